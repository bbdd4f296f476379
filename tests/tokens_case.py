"""Small MoE-layer cases over stored weights, shared by the CPU and GPU tests."""
import numpy as np

import oracle as O


def weights(rng, E, N, K, fmt, group):
    """Raw bf16 weights with outliers, and the quantizer's parameters."""
    w = rng.standard_normal((E, N, K)).astype(np.float32) * 0.05
    flat = w.reshape(-1)
    flat[rng.choice(flat.size, max(1, flat.size // 200), replace=False)] *= 10.0
    bits = O.f32_to_bf16(w)
    if fmt == O.FMT_NONE:
        return bits, (None, None, None)
    s, zp, g = O.observer_weight(bits, fmt, group)
    if fmt == O.FMT_NVFP4:
        s = s.copy()
        s[0, 0, 0] = 0.0                       # a zero block
    if fmt == O.FMT_INT4:
        zp = np.rint(np.clip(zp, 0, 15)).astype(np.float32)
    return bits, (s, zp, g)


def routing(rng, T, E_all, topk):
    ids = np.stack([rng.permutation(E_all)[:topk] for _ in range(T)]).astype(np.int32)
    p = rng.uniform(0.1, 1.0, (T, topk)).astype(np.float32)
    return ids, (p / p.sum(1, keepdims=True)).astype(np.float32)


def make(seed, T, E, H, F, topk, fmt, group, afmt, E_all=None, begin=0, fmt_d=None, group_d=None):
    rng = np.random.default_rng(seed)
    g_gu = group or (16 if fmt == O.FMT_NVFP4 else H)
    fmt_d = fmt if fmt_d is None else fmt_d
    g_d = group_d or group or (16 if fmt_d == O.FMT_NVFP4 else F)
    c = dict(T=T, E=E, H=H, F=F, topk=topk, afmt=afmt, begin=begin)
    c["gu"] = (fmt, g_gu) + weights(rng, E, 2 * F, H, fmt, g_gu)
    c["d"] = (fmt_d, g_d) + weights(rng, E, H, F, fmt_d, g_d)
    x = rng.standard_normal((T, H)).astype(np.float32)
    if x.size >= 64:
        x.reshape(-1)[:16] = 0.0               # a zero 16-block
    c["x"] = O.f32_to_bf16(x)
    c["ids"], c["probs"] = routing(rng, T, E_all or E, topk)
    d = {O.FMT_FP8: 448.0, O.FMT_INT8: 127.0, O.FMT_NVFP4: 2688.0}.get(afmt, 1.0)
    c["s1"] = np.float32(np.abs(x).max() / d)
    # a's largest magnitude is near h's squared; let some of it saturate
    c["s2"] = np.float32(max((0.06 ** 2) * H * 4.0, 1e-3) / d)
    return c


def reference(c, rel_h=0.0):
    vals = [O.stored_values(bits, fmt, group, *q) for fmt, group, bits, q in (c["gu"], c["d"])]
    return O.moe_tokens(c["x"], c["ids"], c["probs"], c["begin"], *vals, c["afmt"], c["s1"],
                        c["s2"], rel_h)
