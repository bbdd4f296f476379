"""The operators that are timed and compared: the MoE layer over stored codes
for a few tokens, and the 8-bit activation checkpoints with the SwiGLU step
that saves and uses them.

``run`` computes each in its plain form (elementary torch operations in
float32), or, with ``own`` true, makes the library calls a user makes.

The codec steps (a scale's reciprocal, z = x * r, the rounding to a grid) are
defined in fp32, so ``exact`` takes them in fp32 too, in a form of its own,
and everything else in float64.
"""
import math

import torch

own = False

DEV = "cuda"
D_OF = {"int8": 127.0, "fp8": 448.0, "nvfp4": 2688.0}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decoded token through the NVFP4 layer of the default workload: latency counts
        dict(name="moe-nvfp4-t1", op="moe", wfmt="nvfp4", afmt="nvfp4", group=16, T=1, E=128,
             H=2048, F=768, topk=8, E_all=128, begin=0),
        # a decode batch of 64 sequences: nearly every expert is read
        dict(name="moe-nvfp4-t64", op="moe", wfmt="nvfp4", afmt="nvfp4", group=16, T=64, E=128,
             H=2048, F=768, topk=8, E_all=128, begin=0),
        # a small decode batch of the FP8 preset (per-channel weights, per-tensor activations)
        dict(name="moe-fp8-t16", op="moe", wfmt="fp8", afmt="fp8", group=-2, T=16, E=128, H=2048,
             F=768, topk=8, E_all=128, begin=0),
        # a few sequences of the w4a16 preset: int4 codes with zero points, bf16 activations
        dict(name="moe-int4-t7", op="moe", wfmt="int4", afmt="none", group=128, T=7, E=128, H=2048,
             F=768, topk=8, E_all=128, begin=0),
        # one rank's 16 of 128 experts under the largest batch: most pairs are routed elsewhere
        dict(name="moe-int8-local-t128", op="moe", wfmt="int8", afmt="int8", group=-2, T=128, E=16,
             H=2048, F=768, topk=8, E_all=128, begin=48),
        # the quantization-off layer (frozen bf16 stacks) at odd sizes, as a small model has them
        dict(name="moe-bf16-odd-t13", op="moe", wfmt="none", afmt="none", group=0, T=13, E=24,
             H=1040, F=368, topk=3, E_all=24, begin=0),
        # the default workload's routed rows, NVFP4 activations, int8 checkpoint
        dict(name="swiglu-int8-r131072", op="swiglu", cfmt="int8", group=128, afmt="nvfp4",
             R=131072, live=131072, F=768),
        # the FP8 preset, an odd number of rows and fewer than there is room for, E4M3 checkpoint
        dict(name="swiglu-fp8-r9731", op="swiglu", cfmt="fp8", group=32, afmt="fp8", R=10240, live=9731,
             F=768),
        # one token's eight rows: the launch counts
        dict(name="swiglu-int8-r8", op="swiglu", cfmt="int8", group=64, afmt="none", R=8, live=8, F=768),
        # the layer input of the default workload, saved and loaded
        dict(name="save-int8-t16384", op="save", cfmt="int8", group=128, rows=16384, K=2048),
        # a single token row in wide E4M3 groups
        dict(name="save-fp8-t1", op="save", cfmt="fp8", group=512, rows=1, K=2048),
        # an odd number of rows of an odd width, in the smallest groups
        dict(name="save-int8-odd", op="save", cfmt="int8", group=16, rows=4099, K=1040),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pow2_groups(*dims):
    return [g for g in (16, 32, 64, 128, 256, 512) if all(d % g == 0 for d in dims)]


def draw(rng):
    limit = {c: max(work(k)["bytes"] for k in listed() if k["op"] == c)
             for c in ("moe", "swiglu", "save")}
    while True:
        op = rng.choice(["moe", "moe", "swiglu", "save"])
        if op == "moe":
            wfmt = rng.choice(["nvfp4", "fp8", "int4", "int8", "none"])
            afmt = rng.choice({"nvfp4": ["nvfp4", "none"], "fp8": ["fp8", "none"],
                               "int4": ["none", "fp8"], "int8": ["int8", "none"],
                               "none": ["none"]}[wfmt])
            H, F = 16 * _log_int(rng, 8, 256), 16 * _log_int(rng, 4, 128)
            group = {"nvfp4": 16, "none": 0}.get(wfmt)
            if wfmt == "int4":
                ok = [g for g in (32, 64, 96, 128) if H % g == 0 and F % g == 0]
                group = rng.choice(ok) if ok else -2
            elif group is None:
                ok = [g for g in (32, 128) if H % g == 0 and F % g == 0]
                group = rng.choice(ok + [-2, -1])
            E_all = _log_int(rng, 4, 256)
            local = rng.random() < 0.3
            E = max(1, E_all // 4) if local else E_all
            c = dict(op="moe", wfmt=wfmt, afmt=afmt, group=group, T=_log_int(rng, 1, 128), E=E,
                     H=H, F=F, topk=rng.randint(1, min(8, E_all)), E_all=E_all,
                     begin=rng.randint(0, E_all - E))
            stack = 3 * E * H * F * {"nvfp4": 0.5625, "int4": 0.54, "none": 2.0}.get(wfmt, 1.01)
            if stack > 3 << 30:
                continue
        elif op == "swiglu":
            F = 16 * _log_int(rng, 4, 128)
            afmt = rng.choice(["none", "fp8", "int8", "nvfp4"])
            R = _log_int(rng, 1, 131072)
            c = dict(op="swiglu", cfmt=rng.choice(["int8", "fp8"]),
                     group=rng.choice(_pow2_groups(F)), afmt=afmt, R=R,
                     live=rng.randint(max(1, R // 2), R), F=F)
        else:
            K = 16 * _log_int(rng, 1, 512)
            c = dict(op="save", cfmt=rng.choice(["int8", "fp8"]), group=rng.choice(_pow2_groups(K)),
                     rows=_log_int(rng, 1, 65536), K=K)
        if work(c)["bytes"] <= limit[op]:
            return c


def _weight_bytes(c, n, k):
    """Stored bytes of one expert's [n, k] matrix."""
    g = {-2: k, -1: n * k}.get(c["group"], c["group"])
    return {"none": 2 * n * k, "int8": n * k + 4 * n * k // max(g, 1),
            "fp8": n * k + 4 * n * k // max(g, 1), "int4": n * k // 2 + 5 * n * k // max(g, 1),
            "nvfp4": n * k // 2 + n * k // 16}[c["wfmt"]]


def work(case):
    c = case
    if c["op"] == "moe":
        T, H, F = c["T"], c["H"], c["F"]
        # experts read: the expected number of distinct local ones
        distinct = c["E"] * (1.0 - (1.0 - c["topk"] / c["E_all"]) ** T)
        pairs = T * c["topk"] * c["E"] / c["E_all"]
        by = distinct * (_weight_bytes(c, 2 * F, H) + _weight_bytes(c, H, F))
        return {"bytes": by + 4 * T * H + 8 * T * c["topk"], "flops": 6.0 * pairs * F * H}
    if c["op"] == "swiglu":
        r, F = c["live"], c["F"]
        ckpt = 2 * F + 4 * (2 * F // c["group"])
        # forward: h in, aq and the checkpoint out; backward: the checkpoint and daq in, dh and aq out
        return {"bytes": r * (4 * F + 2 * F + ckpt) + r * (ckpt + 2 * F + 4 * F + 2 * F),
                "flops": 60.0 * r * F}
    n = c["rows"] * c["K"]
    ckpt = n + 4 * n // c["group"]
    # save: the tensor in, codes and scales out; load: the reverse
    return {"bytes": 2 * (2 * n + ckpt), "flops": 6.0 * n}


# ------------------------------------------- grids and codecs (plain form) --
def _minifloat(z, mant, emin):
    """z rounded to a float grid of `mant` stored mantissa bits and smallest
    exponent emin: multiples of 2^(e - mant), ties to even."""
    _, e = torch.frexp(z)                       # |z| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(z), torch.clamp(e - 1, min=emin) - mant)
    return torch.round(z / step) * step


def _e4m3(z):
    return _minifloat(torch.clamp(z, -448.0, 448.0), 3, -6)


def _e2m1(z):
    return _minifloat(torch.clamp(z, -6.0, 6.0), 1, 0)


def _fake_quant(x, fmt, scale):
    """x [rows, K] fp32 -> (dequantized values, straight-through mask)."""
    if fmt == "none":
        return x, torch.ones_like(x, dtype=torch.bool)
    if fmt == "nvfp4":
        b = x.reshape(*x.shape[:-1], -1, 16)
        theta = _e4m3(torch.clamp(b.abs().amax(-1, keepdim=True) * (1.0 / (6.0 * scale)), max=448.0))
        s = theta * scale
        r = torch.where(s == 0, torch.zeros_like(s), 1.0 / s)
        z = b * r
        v = _e2m1(z) * s
        m = (z.abs() <= 6.0) & (s != 0)
        return v.reshape(x.shape), m.reshape(x.shape)
    z = x * (1.0 / scale)
    if fmt == "fp8":
        q = _e4m3(z)
        m = z.abs() <= 448.0
    else:
        q = torch.round(torch.clamp(z, -128.0, 127.0))
        m = (z >= -128.0) & (z <= 127.0)
    return q * scale, m


def _ckpt_scale(x, cfmt, group):
    amax = x.reshape(x.shape[0], -1, group).abs().amax(-1)
    s = torch.clamp(amax / D_OF[cfmt], min=2.0 ** -126)
    return torch.where(amax == 0, torch.ones_like(s), s)


def _ckpt_values(x, s, cfmt, group):
    """The values the 8-bit codes of x [rows, K] (fp32) stand for."""
    z = x.reshape(x.shape[0], -1, group) * (1.0 / s)[..., None]
    q = _e4m3(z) if cfmt == "fp8" else torch.round(torch.clamp(z, -128.0, 127.0))
    return (q * s[..., None]).reshape(x.shape)


# -------------------------------------------------------------- the inputs --
def _stack(gen, E, N, K, wfmt, group):
    """A weight stack in its stored form, quantized from normal weights with
    a few outliers (scales from each group's largest magnitude)."""
    g = {-2: K, -1: N * K}.get(group, group)
    out = {"codes": [], "scale": [], "sbytes": [], "zp": [], "g": []}
    per = max(1, (32 << 20) // (N * K))
    for e0 in range(0, E, per):
        n = min(per, E - e0)
        w = torch.randn(n, N, K, generator=gen, device=DEV) * 0.02
        w.view(-1)[::997] *= 4.0
        if wfmt == "none":
            out["codes"].append(w.to(torch.bfloat16))
            continue
        if wfmt == "nvfp4":
            b = w.reshape(n, -1, 16)
            amax = b.abs().amax(-1)
            gs = amax.amax(-1) / 2688.0
            th = _e4m3(torch.clamp(amax / (6.0 * gs[:, None]), max=448.0))
            z = b / (th * gs[:, None])[..., None]
            q = _e2m1(torch.nan_to_num(z))
            mag = q.abs()
            code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4))
            code = (code.to(torch.uint8) | (torch.signbit(z).to(torch.uint8) << 3)).reshape(n, -1)
            out["codes"].append(code[:, 0::2] | (code[:, 1::2] << 4))
            out["sbytes"].append(th.to(torch.float8_e4m3fn).view(torch.uint8))
            out["g"].append(gs)
            continue
        b = w.reshape(n, -1, g)
        if wfmt == "int4":
            lo, hi = b.amin(-1).clamp(max=0), b.amax(-1).clamp(min=0)
            s = (hi - lo) / 15.0
            zp = torch.round(-lo / s).clamp(0, 15)
            code = (torch.round(b / s[..., None]) + zp[..., None]).clamp(0, 15)
            code = code.to(torch.uint8).reshape(n, -1)
            out["codes"].append(code[:, 0::2] | (code[:, 1::2] << 4))
            out["zp"].append(zp.to(torch.uint8))
        else:
            s = b.abs().amax(-1) / D_OF[wfmt]
            z = b / s[..., None]
            if wfmt == "int8":
                out["codes"].append(torch.round(z).clamp(-128, 127).to(torch.int8).view(torch.uint8))
            else:
                out["codes"].append(z.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        out["scale"].append(s)
    cat = {k: torch.cat([t.reshape(t.shape[0], -1) for t in v]).contiguous() if v else None
           for k, v in out.items()}
    if cat["g"] is not None:
        cat["g"] = cat["g"].reshape(-1)
    cat.update(fmt=wfmt, group=group, E=E, N=N, K=K)
    return cat


def _routing(gen, c):
    """Distinct random experts per token, softmax weights renormalised over them."""
    logits = torch.randn(c["T"], c["E_all"], generator=gen, device=DEV)
    top, ids = logits.topk(c["topk"], dim=-1)
    return ids.to(torch.int32).contiguous(), torch.softmax(top, -1).contiguous()


def _one(v):
    return torch.tensor([v], dtype=torch.float32, device=DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    bf = torch.bfloat16
    st = {"case": c}
    if c["op"] == "moe":
        T, H, F, E = c["T"], c["H"], c["F"], c["E"]
        st["w_gu"] = _stack(gen, E, 2 * F, H, c["wfmt"], c["group"])
        st["w_d"] = _stack(gen, E, H, F, c["wfmt"], c["group"])
        st["x"] = torch.randn(T, H, generator=gen, device=DEV).to(bf)
        st["ids"], st["probs"] = _routing(gen, c)
        # calibrated per-tensor scales: the input's largest magnitude, and one
        # that the SwiGLU values of these sizes reach
        amax_a = 0.0032 * H
        d = D_OF.get(c["afmt"], 1.0)
        st["s1"] = (st["x"].float().abs().amax() / d).reshape(1)
        st["s2"] = _one(amax_a / d)
        if own:
            import moe_fake_quant_amd as fq
            fmts = fq.FMT_BY_NAME
            st["own"] = dict(
                w_gu=_stored(fq, st["w_gu"]), w_d=_stored(fq, st["w_d"]),
                a1=fq.ActQ(fmts[c["afmt"]], st["s1"]), a2=fq.ActQ(fmts[c["afmt"]], st["s2"]),
                ws=torch.empty(fq.fq_workspace_bytes(fq.FQ_OP_MOE_TOKENS, (E, H, F), T * c["topk"],
                                                     c["topk"]), dtype=torch.uint8, device=DEV),
                out=torch.empty(T, H, dtype=bf, device=DEV))
        return st
    if c["op"] == "swiglu":
        R, F, live = c["R"], c["F"], c["live"]
        # gate_up outputs: normal, with channels of different size
        chan = torch.exp(0.5 * torch.randn(2 * F, generator=gen, device=DEV))
        h = torch.empty(R, 2 * F, dtype=bf, device=DEV)
        daq = torch.empty(R, F, dtype=bf, device=DEV)
        for r in range(0, R, 16384):
            n = min(16384, R - r)
            h[r:r + n] = (torch.randn(n, 2 * F, generator=gen, device=DEV) * chan).to(bf)
            daq[r:r + n] = (torch.randn(n, F, generator=gen, device=DEV) * 1e-3).to(bf)
        st["h"], st["daq"] = h, daq
        g = h[:live, :F].float()
        amax = (g * torch.sigmoid(g) * h[:live, F:].float()).abs().amax()
        st["s"] = (amax / D_OF.get(c["afmt"], 1.0)).reshape(1)
        st["n_rows"] = torch.tensor([live], dtype=torch.int32, device=DEV)
        st["buf"] = dict(aq=torch.zeros(R, F, dtype=bf, device=DEV),
                         aq2=torch.zeros(R, F, dtype=bf, device=DEV),
                         dh=torch.zeros(R, 2 * F, dtype=bf, device=DEV),
                         scale=torch.zeros(R, 2 * F // c["group"], device=DEV))
        if own:
            import moe_fake_quant_amd as fq
            st["own"] = dict(codes=torch.empty(R, 2 * F, dtype=torch.uint8, device=DEV),
                             aq=fq.ActQ(fq.FMT_BY_NAME[c["afmt"]], st["s"]))
        return st
    rows, K = c["rows"], c["K"]
    chan = torch.exp(0.5 * torch.randn(K, generator=gen, device=DEV))
    st["x"] = (torch.randn(rows, K, generator=gen, device=DEV) * chan).to(bf)
    st["out"] = torch.empty(rows, K, dtype=bf, device=DEV)
    st["scale"] = torch.empty(rows, K // c["group"], device=DEV)
    if own:
        st["codes"] = torch.empty(rows, K, dtype=torch.uint8, device=DEV)
    return st


def _stored(fq, w):
    """The stack as the library's export leaves it."""
    group = {-2: w["K"], -1: fq.FQ_GROUP_TENSOR, 0: 16}.get(w["group"], w["group"])
    return fq.StoredW(fmt=fq.FMT_BY_NAME[w["fmt"]], group=group, codes=w["codes"],
                      scale=w["scale"], scale_bytes=w["sbytes"], zero_point_bytes=w["zp"],
                      global_scale=w["g"])


# ------------------------------------------------------------------ passes --
def _decode(w, e):
    """Expert e's matrix [N, K] in fp32 from its stored form."""
    N, K = w["N"], w["K"]
    c = w["codes"][e]
    if w["fmt"] == "none":
        return c.reshape(N, K).float()
    if w["fmt"] == "int8":
        v = c.view(torch.int8).float()
    elif w["fmt"] == "fp8":
        v = c.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack((c & 15, c >> 4), -1).reshape(-1)
        if w["fmt"] == "int4":
            v = c.float().reshape(w["zp"].shape[1], -1) - w["zp"][e].float()[:, None]
        else:
            mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV)
            v = torch.cat((mag, -mag))[c.to(torch.int32)]
    if w["fmt"] == "nvfp4":
        s = w["sbytes"][e].view(torch.float8_e4m3fn).float() * w["g"][e]
    else:
        s = w["scale"][e]
    return (v.reshape(s.numel(), -1) * s[:, None]).reshape(N, K)


def _moe(st, c):
    """The layer expert by expert."""
    xq = _fake_quant(st["x"].float(), c["afmt"], st["s1"])[0]
    out = torch.zeros(c["T"], c["H"], device=DEV)
    for e in range(c["E"]):
        tok, slot = (st["ids"] == e + c["begin"]).nonzero(as_tuple=True)
        if tok.numel() == 0:
            continue
        h = xq[tok] @ _decode(st["w_gu"], e).t()
        g, u = h[:, :c["F"]], h[:, c["F"]:]
        a = _fake_quant(g / (1.0 + torch.exp(-g)) * u, c["afmt"], st["s2"])[0]
        o = a @ _decode(st["w_d"], e).t()
        out.index_add_(0, tok, o * st["probs"][tok, slot][:, None])
    return out.to(torch.bfloat16)


def _swiglu(st, c):
    """Forward and backward of the SwiGLU step, in blocks of rows so that the
    temporaries stay small; the backward uses the saved values of h."""
    b, F, bf = st["buf"], c["F"], torch.bfloat16

    def act(v):
        g, u = v[:, :F], v[:, F:]
        sg = 1.0 / (1.0 + torch.exp(-g))
        # A is stored in bf16 by definition, and the quantizer sees that
        return g, u, sg, _fake_quant((g * sg * u).to(bf).float(), c["afmt"], st["s"])

    for r in range(0, c["live"], 16384):
        rows = slice(r, min(r + 16384, c["live"]))
        h = st["h"][rows].float()
        s = _ckpt_scale(h, c["cfmt"], c["group"])
        saved = _ckpt_values(h, s, c["cfmt"], c["group"])
        b["scale"][rows] = s
        b["aq"][rows] = act(h)[3][0].to(bf)
        g, u, sg, (aq, m) = act(saved)
        b["aq2"][rows] = aq.to(bf)
        d = st["daq"][rows].float()
        da = torch.where(m, d, torch.zeros_like(d))
        b["dh"][rows, :F] = (da * u * sg * (1.0 + g * (1.0 - sg))).to(bf)
        b["dh"][rows, F:] = (da * g * sg).to(bf)
    return dict(b)


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["op"] == "moe":
        return _moe(state, c)
    if c["op"] == "swiglu":
        return _swiglu(state, c)
    x = state["x"].float()
    s = _ckpt_scale(x, c["cfmt"], c["group"])
    return {"x": _ckpt_values(x, s, c["cfmt"], c["group"]).to(torch.bfloat16), "scale": s}


def _run_own(st, c):
    import moe_fake_quant_amd as fq
    if c["op"] == "moe":
        o = st["own"]
        fq.fq_moe_tokens(st["x"], c["T"], c["H"], c["F"], st["ids"], st["probs"], c["topk"],
                         c["begin"], c["E"], o["w_gu"], o["w_d"], o["a1"], o["a2"], o["out"],
                         o["ws"])
        return o["out"]
    cfmt = fq.FMT_BY_NAME[c["cfmt"]]
    if c["op"] == "swiglu":
        o, b = st["own"], st["buf"]
        R, F, g = c["R"], c["F"], c["group"]
        fq.fq_swiglu_actfq_ckpt(st["h"], R, st["n_rows"], F, o["aq"], cfmt, g, None, b["aq"],
                                o["codes"], b["scale"])
        fq.fq_swiglu_bwd_ckpt(st["daq"], o["codes"], b["scale"], R, st["n_rows"], F, cfmt, g,
                              o["aq"], b["dh"], b["aq2"])
        return dict(b)
    fq.fq_ckpt_save(st["x"], c["rows"], c["K"], None, cfmt, c["group"], st["codes"], st["scale"])
    fq.fq_ckpt_load(st["codes"], st["scale"], c["rows"], c["K"], None, cfmt, c["group"], st["out"])
    return {"x": st["out"], "scale": st["scale"]}


# ------------------------------------------------------------ the definition --
def _table_round(z, grid):
    """Nearest entry of an increasing grid of magnitudes (sign kept); halfway
    goes to the entry of even index."""
    a = torch.clamp(z.abs(), max=grid[-1].item())
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.bucketize(a, mid)                     # entries whose midpoint is below a
    hi = torch.bucketize(a, mid, right=True)         # ... or equal to it
    idx = torch.where(lo % 2 == 0, lo, hi)
    return torch.copysign(grid[idx], z)


def _grids():
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                        [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1],
                        device=DEV)
    return e2m1, e4m3


def _exact_fq(v, fmt, s):
    """The quantizer's value and mask of fp32 rows: its steps
    are fp32 by definition, its value is returned in float64."""
    e2m1, e4m3 = _grids()
    f64 = torch.float64
    if fmt == "none":
        return v.to(f64), torch.ones_like(v, dtype=torch.bool)
    if fmt == "nvfp4":
        b = v.view(v.shape[0], v.shape[1] // 16, 16)
        top = b.abs().max(dim=2).values * (1.0 / (s * 6.0))
        sb = _table_round(top.clamp(max=448.0), e4m3) * s
        live = (sb != 0)[:, :, None]
        z = torch.where(live, b * torch.where(sb == 0, sb, 1.0 / sb)[:, :, None], 0.0)
        q = _table_round(z, e2m1).to(f64) * sb[:, :, None].to(f64)
        return q.reshape(v.shape), (live & (z.abs() <= 6.0)).reshape(v.shape)
    z = v * (1.0 / s)
    if fmt == "fp8":
        q, m = _table_round(z, e4m3), (z <= 448.0) & (z >= -448.0)
    else:
        q, m = z.clamp(-128.0, 127.0).round(), (z <= 127.0) & (z >= -128.0)
    return q.to(f64) * s.to(f64), m


def _exact_matrix(w, e):
    """Expert e's matrix in float64, element by element from its code."""
    f64, N, K = torch.float64, w["N"], w["K"]
    c = w["codes"][e]
    if w["fmt"] == "none":
        return c.to(f64).reshape(N, K)
    if w["fmt"] in ("int4", "nvfp4"):
        both = torch.empty(2 * c.numel(), dtype=torch.int64, device=DEV)
        both[0::2], both[1::2] = (c % 16).long(), (c // 16).long()
        c = both
    else:
        c = c.long()
    if w["fmt"] == "int8":
        v = (c - 256 * (c > 127)).to(f64)
    elif w["fmt"] == "int4":
        v = (c - w["zp"][e].long().repeat_interleave(c.numel() // w["zp"].shape[1])).to(f64)
    else:
        grid = _grids()[0 if w["fmt"] == "nvfp4" else 1].to(f64)
        half = 8 if w["fmt"] == "nvfp4" else 128
        v = grid[(c % half).clamp(max=grid.numel() - 1)]
        v = torch.where(c >= half, -v, v)
    if w["fmt"] == "nvfp4":
        s = (_grids()[1][w["sbytes"][e].long()] * w["g"][e]).to(f64)
    else:
        s = w["scale"][e].to(f64)
    return (v * s.repeat_interleave(c.numel() // s.numel())).view(N, K)


def _exact_moe(st, c):
    f64 = torch.float64
    xq = _exact_fq(st["x"].float(), c["afmt"], st["s1"])[0]
    out = torch.zeros(c["T"], c["H"], dtype=f64, device=DEV)
    pairs, probs = {}, st["probs"].to(f64)
    for t, row in enumerate(st["ids"].tolist()):
        for j, e in enumerate(row):
            if c["begin"] <= e < c["begin"] + c["E"]:
                pairs.setdefault(e - c["begin"], []).append((t, j))
    for e, tj in pairs.items():
        tok = torch.tensor([t for t, _ in tj], device=DEV)
        h = torch.matmul(_exact_matrix(st["w_gu"], e), xq[tok].t())           # [2F, pairs]
        a = (h[:c["F"]] * torch.sigmoid(h[:c["F"]]) * h[c["F"]:]).t()
        if c["afmt"] != "none":
            a = _exact_fq(a.float().contiguous(), c["afmt"], st["s2"])[0]
        o = torch.matmul(_exact_matrix(st["w_d"], e), a.t())                  # [H, pairs]
        for i, (t, j) in enumerate(tj):
            out[t] += probs[t, j] * o[:, i]
    return out


def _exact_saved(x, c):
    """The saved values of rows x (fp32) in float64, and their scales."""
    b = x.view(x.shape[0], x.shape[1] // c["group"], c["group"])
    amax = torch.maximum(b.max(dim=2).values, -b.min(dim=2).values)
    s = torch.where(amax > 0, torch.clamp(amax / D_OF[c["cfmt"]], min=2.0 ** -126), 1.0)
    z = b * (1.0 / s)[:, :, None]
    q = _table_round(z, _grids()[1]) if c["cfmt"] == "fp8" else z.clamp(-128.0, 127.0).round()
    return (q.to(torch.float64) * s[:, :, None].to(torch.float64)).view(x.shape), s


def _exact_swiglu(st, c):
    f64, F, R, live = torch.float64, c["F"], c["R"], c["live"]
    out = dict(aq=torch.zeros(R, F, dtype=f64, device=DEV),
               aq2=torch.zeros(R, F, dtype=f64, device=DEV),
               dh=torch.zeros(R, 2 * F, dtype=f64, device=DEV),
               scale=torch.zeros(R, 2 * F // c["group"], dtype=f64, device=DEV))
    for r0 in range(0, live, 8192):
        rows = slice(r0, min(r0 + 8192, live))
        h = st["h"][rows].float()
        saved, out["scale"][rows] = _exact_saved(h, c)
        h = h.to(f64)
        # A is stored in bf16 by definition, and the quantizer sees that
        a = (h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]).to(torch.bfloat16).float()
        out["aq"][rows] = _exact_fq(a, c["afmt"], st["s"])[0]
        g, u = saved.split(F, dim=1)
        sig = torch.sigmoid(g)
        a = (g * sig * u).to(torch.bfloat16).float()
        out["aq2"][rows], m = _exact_fq(a, c["afmt"], st["s"])
        d = st["daq"][rows].to(f64)
        out["dh"][rows, :F] = d * m * u * (sig + g * sig * torch.sigmoid(-g))
        out["dh"][rows, F:] = d * m * (g * sig)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "moe":
        return _exact_moe(st, case)
    if case["op"] == "swiglu":
        return _exact_swiglu(st, case)
    x, s = _exact_saved(st["x"].float(), case)
    return {"x": x, "scale": s.to(torch.float64)}
