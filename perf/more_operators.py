"""Operators that are timed and compared: the int8 product with a scale for each
token and channel, the gated feed-forward block (gate and up projections,
activation and product in one pass) with its recomputing backward, and the
norms around a block with its gate and residual scale.

``run`` computes each in its plain form (elementary torch operations in
float32), or, with ``own`` true, makes the library calls a user makes.

The codec steps (a scale's reciprocal, z = x * r, the rounding to a grid) are
defined in fp32, so ``exact`` takes them in fp32 too, and everything else in
float64.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
EPS = 1e-6
D_OF = {"int8": 127.0, "fp8": 448.0}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decoded token through a dense int8 linear: latency counts
        dict(name="int8-dense-t1", op="int8", E=1, N=4096, K=4096, rows=1, live=1, scales="channel"),
        # the dense linear of 4096 x 4096 under 2048 tokens, as the int4 workload has them
        dict(name="int8-dense-t2048", op="int8", E=1, N=4096, K=4096, rows=2048, live=2048,
             scales="channel"),
        # the down projection of the 128-expert workload over its routed rows
        dict(name="int8-moe-down", op="int8", E=128, N=2048, K=768, rows=131072, live=131072,
             scales="channel"),
        # a small model's experts at odd sizes, fewer rows than there is room for
        dict(name="int8-odd", op="int8", E=5, N=1040, K=368, rows=400, live=333, scales="tensor"),
        # gate_up and SwiGLU of the FP8 preset: 8192 tokens, 128 experts, top-8
        dict(name="gated-fp8-t8192", op="gated", dir="fwd", w="bf16", afmt="fp8", T=8192, topk=8, E=128,
             E_all=128, begin=0, H=2048, F=768),
        # its backward in training, h recomputed, 16384 tokens with bf16 activations
        dict(name="gated-bwd-t16384", op="gated", dir="bwd", w="bf16", afmt="none", T=16384, topk=8,
             E=128, E_all=128, begin=0, H=2048, F=768),
        # a prefill of 2048 tokens over int8 codes, one rank's 32 of 128 experts
        dict(name="gated-int8-local-t2048", op="gated", dir="fwd", w="int8", afmt="none", T=2048, topk=8,
             E=32, E_all=128, begin=64, H=2048, F=768),
        # a dense gated block for four sequences that decode: the weights' stream counts
        dict(name="gated-dense-t4", op="gated", dir="fwd", w="bf16", afmt="none", T=4, topk=1, E=1,
             E_all=1, begin=0, H=2048, F=4096),
        # the backward of a small model's layer at odd sizes, int8 activations
        dict(name="gated-bwd-odd", op="gated", dir="bwd", w="bf16", afmt="int8", T=77, topk=3, E=6,
             E_all=6, begin=0, H=208, F=80),
        # one token's residual, next norm and int8 codes, with the small product that reads them
        dict(name="norm-int8-t1", op="norm", dir="int8", T=1, H=2048, N=512, post=True, pre=True,
             gate=True, block=True),
        # both norms around a block of the 16384-token workload
        dict(name="norm-t16384", op="norm", dir="fwd", T=16384, H=2048, N=0, post=True, pre=True,
             gate=True, block=True),
        # their backward with every gradient, an odd number of tokens
        dict(name="norm-bwd-t8191", op="norm", dir="bwd", T=8191, H=2048, N=0, post=True, pre=True,
             gate=True, block=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50.0)


def draw(rng):
    limit = {op: max(_cost(k) for k in listed() if k["op"] == op) for op in ("int8", "gated", "norm")}
    while True:
        op = rng.choice(["int8", "gated", "gated", "norm"])
        if op == "int8":
            rows = _log_int(rng, 1, 131072)
            c = dict(op=op, E=_log_int(rng, 1, 128), N=16 * _log_int(rng, 1, 512),
                     K=16 * _log_int(rng, 1, 512), rows=rows, live=rng.randint(max(1, rows // 2), rows),
                     scales=rng.choice(["channel", "channel", "tensor"]))
            if c["E"] * c["N"] * c["K"] > 1 << 29:
                continue
        elif op == "gated":
            E_all = _log_int(rng, 1, 128)
            E = max(1, E_all // 4) if rng.random() < 0.3 else E_all
            w = rng.choice(["bf16", "bf16", "int8"])
            dir_ = "fwd" if w == "int8" else rng.choice(["fwd", "bwd"])
            topk = rng.randint(1, min(8, E_all))
            c = dict(op=op, dir=dir_, w=w, afmt="none" if w == "int8" else rng.choice(["none", "fp8"]),
                     T=_log_int(rng, 1, 16384), topk=topk, E=E, E_all=E_all,
                     begin=rng.randint(0, E_all - E), H=16 * _log_int(rng, 1, 256),
                     F=16 * _log_int(rng, 1, 256))
            if c["E"] * c["H"] * c["F"] > 1 << 28 or c["T"] * topk * (c["H"] + 2 * c["F"]) > 1 << 29:
                continue
        else:
            block = rng.random() < 0.8
            c = dict(op=op, dir=rng.choice(["fwd", "bwd", "int8"]), T=_log_int(rng, 1, 16384),
                     H=16 * _log_int(rng, 1, 512), N=0, post=block and rng.random() < 0.6,
                     pre=rng.random() < 0.8 or not block, gate=block and rng.random() < 0.6, block=block)
            if c["dir"] == "int8":
                c.update(pre=True, N=16 * rng.randint(1, 32))
        if _cost(c) <= limit[op]:
            return c


def work(case):
    """The experts read are the expected number of distinct ones that get a row."""
    c = case
    if c["op"] == "int8":
        R, N, K, E = c["live"], c["N"], c["K"], c["E"]
        used = E * (1.0 - (1.0 - 1.0 / E) ** R) if E > 1 else 1
        # x in bf16, the used experts' codes and scales in; y and the token scales out
        return {"bytes": 2.0 * R * K + used * (N * K + 4 * N) + 2.0 * R * N + 4 * R,
                "flops": 2.0 * R * N * K}
    if c["op"] == "gated":
        T, H, F = c["T"], c["H"], c["F"]
        R = T * c["topk"] * c["E"] / c["E_all"]
        used = c["E"] * (1.0 - (1.0 - c["topk"] / c["E_all"]) ** T)
        by = 2.0 * T * H + used * 2 * F * H * (1 if c["w"] == "int8" else 2) + 2.0 * R * F
        fl = 4.0 * R * F * H
        if c["dir"] == "bwd":  # dA in, dH and dX out, and the product with dH
            by += 2.0 * R * F + 4.0 * R * F + 2.0 * R * H
            fl *= 2
        return {"bytes": by, "flops": fl}
    T, H, k = c["T"], c["H"], 2.0 * c["T"] * c["H"]
    if c["dir"] == "bwd":  # y, b, dy, dn in; dx, db out
        return {"bytes": k * (3 + 2 * c["block"] + c["pre"]) + 8.0 * H, "flops": 20.0 * T * H}
    by = k * (1 + 2 * c["block"] + c["pre"]) + 4.0 * H
    if c["dir"] == "int8":
        by += c["N"] * H + 2 * T * c["N"] - T * H
    return {"bytes": by, "flops": 10.0 * T * H + 2.0 * T * H * c["N"]}


# -------------------------------------------------------------- the inputs --
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _tokens(gen, rows, K):
    """Rows of activations: channels and tokens of different size."""
    chan = torch.exp(0.5 * _normal(gen, K))
    return (_normal(gen, rows, K) * chan * torch.exp(0.3 * _normal(gen, rows, 1))).to(BF)


def _int8_stack(gen, E, N, K, scales):
    """Int8 codes [E, N, K] of normal weights with outliers, with a scale for each
    output channel or for each matrix."""
    codes = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    scale = torch.empty((E, N) if scales == "channel" else (E,), device=DEV)
    per = max(1, (32 << 20) // (N * K))
    for e in range(0, E, per):
        w = _normal(gen, min(per, E - e), N, K) * 0.02
        w.view(-1)[::997] *= 4.0
        s = (w.abs().amax(-1) if scales == "channel" else w.abs().amax((1, 2))) / 127.0
        codes[e:e + per] = torch.round(w / s.reshape(w.shape[0], -1, 1)).to(torch.int8)
        scale[e:e + per] = s
    return codes, scale


def _bf16_stack(gen, E, N, K):
    w = torch.empty(E, N, K, dtype=BF, device=DEV)
    per = max(1, (32 << 20) // (N * K))
    for e in range(0, E, per):
        w[e:e + per] = (_normal(gen, min(per, E - e), N, K) * 0.02).to(BF)
    return w


def _segments(counts):
    seg = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=DEV)
    seg[1:] = torch.cumsum(counts, 0)
    return seg


def _route(gen, c):
    """Distinct random experts for each token; the local (token, slot) pairs in
    expert order, as the library's permute gives them."""
    ids = _normal(gen, c["T"], c["E_all"]).topk(c["topk"], dim=-1).indices.reshape(-1) - c["begin"]
    local = (ids >= 0) & (ids < c["E"])
    order = torch.argsort(torch.where(local, ids, c["E"]), stable=True)
    seg = _segments(torch.bincount(ids[local], minlength=c["E"]))
    return order.to(torch.int32), seg


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "int8":
        E, N, K, rows, live = c["E"], c["N"], c["K"], c["rows"], c["live"]
        st["codes"], st["wscale"] = _int8_stack(gen, E, N, K, c["scales"])
        st["x"] = _tokens(gen, rows, K)
        st["seg"] = _segments(torch.bincount(torch.randint(0, E, (live,), generator=gen, device=DEV),
                                             minlength=E))
        st["y"] = torch.zeros(rows, N, dtype=BF, device=DEV)
        st["scale"] = torch.zeros(rows, device=DEV)
        st["xcodes"] = torch.empty(rows, K, dtype=torch.uint8, device=DEV)
    elif c["op"] == "gated":
        T, H, F, E = c["T"], c["H"], c["F"], c["E"]
        R = T * c["topk"]
        st["x"] = _tokens(gen, T, H)
        st["perm"], st["seg"] = _route(gen, c)
        st["aq"] = torch.zeros(R, F, dtype=BF, device=DEV)
        if c["w"] == "int8":
            st["codes"], st["wscale"] = _int8_stack(gen, E, 2 * F, H, "channel")
            st["scale"] = torch.empty(T, device=DEV)
            st["xcodes"] = torch.empty(T, H, dtype=torch.uint8, device=DEV)
        else:
            st["w"] = _bf16_stack(gen, E, 2 * F, H)
        # a calibrated scale for A with room above what these sizes reach: A's
        # largest value is about 60 times the product of its factors' deviations
        st["ascale"] = torch.full((1,), 60.0 * (0.02 * 0.02 * 1.65 * 1.2 * H + 1e-3) / D_OF.get(c["afmt"], 1.0),
                                  device=DEV)
        if c["dir"] == "bwd":
            st["daq"] = torch.empty(R, F, dtype=BF, device=DEV)
            for r in range(0, R, 16384):
                st["daq"][r:r + 16384] = (_normal(gen, min(16384, R - r), F) * 1e-3).to(BF)
            st["dh"] = torch.zeros(R, 2 * F, dtype=BF, device=DEV)
            st["dx"] = torch.zeros(R, H, dtype=BF, device=DEV)
    else:
        T, H = c["T"], c["H"]
        st["x"] = _tokens(gen, T, H)
        st["b"] = _tokens(gen, T, H) if c["block"] else None
        st["gate"] = torch.sigmoid(_normal(gen, T)) if c["gate"] else None
        st["w_post"] = (1.0 + 0.1 * _normal(gen, H)).to(BF) if c["post"] else None
        st["w_pre"] = (1.0 + 0.1 * _normal(gen, H)).to(BF) if c["pre"] else None
        st["alpha"] = 0.5
        if c["dir"] == "bwd":
            st["dy"] = (_normal(gen, T, H) * 1e-2).to(BF)
            st["dn"] = (_normal(gen, T, H) * 1e-2).to(BF) if c["pre"] else None
        if c["dir"] == "int8":
            st["codes"], st["wscale"] = _int8_stack(gen, 1, c["N"], H, "channel")
            st["seg"] = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    if "seg" in st:
        st["segs"] = st["seg"].tolist()
    if own:
        _prepare_own(st, c)
    return st


def _prepare_own(st, c):
    """The quantizers, workspaces and buffers that a program keeps."""
    import moe_fake_quant_amd as fq

    def ws(op, shape, rows, fmts=0):
        return torch.empty(max(256, fq.fq_workspace_bytes(op, shape, rows, fmts)), dtype=torch.uint8,
                           device=DEV)

    def stored(shape):
        group = shape[2] if st["wscale"].dim() == 2 else fq.FQ_GROUP_TENSOR
        return fq.StoredW(fq.FMT_INT8, group, st["codes"], st["wscale"])

    if c["op"] == "int8":
        st["shape"] = (c["E"], c["N"], c["K"])
        st["own"] = dict(w=stored(st["shape"]), ws=ws(fq.FQ_OP_GEMM_INT8, st["shape"], c["rows"]))
    elif c["op"] == "gated":
        R = c["T"] * c["topk"]
        st["shape"] = (c["E"], 2 * c["F"], c["H"])
        o = st["own"] = dict(aq=fq.ActQ(fq.FMT_BY_NAME[c["afmt"]], st["ascale"]),
                             ws=ws(fq.FQ_OP_GATED, st["shape"], R))
        if c["w"] == "int8":
            o["w"] = stored(st["shape"])
        if c["dir"] == "bwd":
            o["ws2"] = ws(fq.FQ_OP_GEMM_BWD, st["shape"], R)
            o["wq"] = fq.WeightQ(fq.FMT_INT8, c["H"], torch.ones(c["E"], 2 * c["F"], device=DEV))
    else:
        T, H = c["T"], c["H"]
        full = dict(dtype=BF, device=DEV)
        if c["dir"] == "bwd":
            f32 = dict(dtype=torch.float32, device=DEV)
            st["own"] = dict(dx=torch.empty(T, H, **full),
                             db=torch.empty(T, H, **full) if c["block"] else None,
                             dgate=torch.empty(T, **f32) if c["gate"] else None,
                             dw_post=torch.empty(H, **f32) if c["post"] else None,
                             dw_pre=torch.empty(H, **f32) if c["pre"] else None,
                             ws=ws(fq.FQ_OP_NORM, (1, T, H), 0))
        else:
            o = st["own"] = dict(y=torch.empty(T, H, **full) if c["block"] else None)
            if c["dir"] == "int8":
                o.update(codes=torch.empty(T, H, dtype=torch.uint8, device=DEV),
                         scale=torch.empty(T, device=DEV), z=torch.empty(T, c["N"], **full),
                         w=stored((1, c["N"], H)), ws=ws(fq.FQ_OP_GEMM_INT8, (1, c["N"], H), T))
            elif c["pre"]:
                o["n"] = torch.empty(T, H, **full)


# ------------------------------------------------------------ plain forms --
def _token_codes(x):
    """Int8 code values of rows x (fp32) and their scales."""
    amax = x.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), torch.clamp(amax * (1.0 / 127.0), min=2.0 ** -126))
    return torch.round(torch.clamp(x * (1.0 / s)[:, None], -128.0, 127.0)), s


def _experts(st):
    """(expert, its rows) of every expert that has rows."""
    segs = st["segs"]
    return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(segs[:-1], segs[1:])) if b > a]


def _int8_values(st, e):
    return st["codes"][e].float(), st["wscale"][e].reshape(1, -1)


def _fq_act(a, afmt, s):
    """Values and straight-through mask of A (fp32) after the activation quantizer;
    A is stored in bf16 by definition, and the quantizer sees that."""
    if afmt == "none":
        return a, torch.ones_like(a)
    z = a.to(BF).float() * (1.0 / s)
    d = -128.0 if afmt == "int8" else -448.0
    top = 127.0 if afmt == "int8" else 448.0
    m = ((z >= d) & (z <= top)).float()
    z = torch.clamp(z, d, top)
    if afmt == "int8":
        return torch.round(z) * s, m
    e = torch.clamp(torch.frexp(z)[1] - 1, min=-6) - 3
    step = torch.ldexp(torch.ones_like(z), e)
    return torch.round(z / step) * step * s, m


def _plain_int8(st, c):
    st["scale"].zero_()
    for e, r in _experts(st):
        q, s = _token_codes(st["x"][r].float())
        w, ws = _int8_values(st, e)
        st["y"][r] = (q @ w.t() * s[:, None] * ws).to(BF)
        st["scale"][r] = s
    return {"y": st["y"], "scale": st["scale"]}


def _plain_gated(st, c):
    F = c["F"]
    x = st["x"].float()
    tok = (st["perm"] // c["topk"]).long()
    if c["w"] == "int8":
        x, st["scale"] = _token_codes(x)
    for e, r in _experts(st):
        xe = x[tok[r]]
        if c["w"] == "int8":
            w, ws = _int8_values(st, e)
            h = xe @ w.t() * st["scale"][tok[r]][:, None] * ws
        else:
            w = st["w"][e].float()
            h = xe @ w.t()
        g, u = h[:, :F], h[:, F:]
        sg = 1.0 / (1.0 + torch.exp(-g))
        aq, m = _fq_act(g * sg * u, c["afmt"], st["ascale"])
        st["aq"][r] = aq.to(BF)
        if c["dir"] == "bwd":
            da = m * st["daq"][r].float()
            dh = torch.cat((da * u * sg * (1.0 + g * (1.0 - sg)), da * g * sg), 1).to(BF)
            st["dh"][r] = dh
            st["dx"][r] = (dh.float() @ w).to(BF)
    if c["dir"] == "bwd":
        return {"aq": st["aq"], "dh": st["dh"], "dx": st["dx"]}
    return {"aq": st["aq"]}


def _plain_norm(st, c):
    x, b = st["x"].float(), st["b"].float() if c["block"] else None
    y = x
    if c["block"]:
        p = b
        if c["post"]:
            p = p * torch.rsqrt(b.square().mean(-1, keepdim=True) + EPS) * st["w_post"].float()
        if c["gate"]:
            p = p * st["gate"][:, None]
        y = x + st["alpha"] * p
    out = {"y": y.to(BF)} if c["block"] else {}
    if c["pre"]:
        n = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["w_pre"].float()
        if c["dir"] == "int8":
            q, s = _token_codes(n)
            w, ws = _int8_values(st, 0)
            out.update(z=(q @ w.t() * s[:, None] * ws).to(BF), scale=s)
        else:
            out["n"] = n.to(BF)
    return out


def _plain_norm_bwd(st, c):
    """x stands for the stored sum y here; dn reaches it through the next norm."""
    y, gy = st["x"].float(), st["dy"].float()
    out = {}
    if c["pre"]:
        r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        dn = st["dn"].float()
        v = dn * st["w_pre"].float()
        gy = gy + r * (v - y * r * r * (v * y).mean(-1, keepdim=True))
        out["dw_pre"] = (dn * y * r).sum(0)
    out["dx"] = gy.to(BF)
    if not c["block"]:
        return out
    b = st["b"].float()
    rb = torch.rsqrt(b.square().mean(-1, keepdim=True) + EPS) if c["post"] else torch.ones_like(b[:, :1])
    w = st["w_post"].float() if c["post"] else torch.ones_like(b[0])
    if c["gate"]:
        out["dgate"] = st["alpha"] * (gy * b * rb * w).sum(-1)
    dp = st["alpha"] * gy * (st["gate"][:, None] if c["gate"] else 1.0)
    if not c["post"]:
        out["db"] = dp.to(BF)
        return out
    out["dw_post"] = (dp * b * rb).sum(0)
    v = dp * w
    out["db"] = (rb * (v - b * rb * rb * (v * b).mean(-1, keepdim=True))).to(BF)
    return out


# ------------------------------------------------------------------ passes --
def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["op"] == "int8":
        return _plain_int8(state, c)
    if c["op"] == "gated":
        return _plain_gated(state, c)
    return _plain_norm_bwd(state, c) if c["dir"] == "bwd" else _plain_norm(state, c)


def _run_own(st, c):
    import moe_fake_quant_amd as fq
    o = st["own"]
    if c["op"] == "int8":
        rows = c["rows"]
        fq.fq_quantize_tokens(st["x"], rows, c["K"], st["seg"][c["E"]:], st["xcodes"], st["scale"])
        fq.fq_grouped_gemm_int8(st["xcodes"], st["scale"], rows, None, 1, rows, st["seg"], st["shape"],
                                o["w"], st["y"], o["ws"])
        return {"y": st["y"], "scale": st["scale"]}
    if c["op"] == "gated":
        T, R, topk = c["T"], c["T"] * c["topk"], c["topk"]
        if c["w"] == "int8":
            fq.fq_quantize_tokens(st["x"], T, c["H"], None, st["xcodes"], st["scale"])
            fq.fq_grouped_gated_int8(st["xcodes"], st["scale"], T, st["perm"], topk, R, st["seg"],
                                     st["shape"], o["w"], st["aq"], o["ws"])
        elif c["dir"] == "fwd":
            fq.fq_grouped_gated_fwd(st["x"], T, st["perm"], topk, R, st["seg"], st["shape"], st["w"],
                                    o["aq"], st["aq"], o["ws"])
        else:
            fq.fq_grouped_gated_bwd(st["daq"], st["x"], T, st["perm"], topk, R, st["seg"], st["shape"],
                                    st["w"], o["aq"], st["dh"], st["aq"], o["ws"])
            fq.fq_grouped_gemm_bwd_scale(st["dh"], None, R, st["seg"], st["shape"], st["w"], st["w"],
                                         o["wq"], None, st["dx"], None, None, o["ws2"])
            return {"aq": st["aq"], "dh": st["dh"], "dx": st["dx"]}
        return {"aq": st["aq"]}
    T, H = c["T"], c["H"]
    norm = (st["gate"], st["alpha"], st["w_post"], st["w_pre"], EPS, T, H)
    if c["dir"] == "bwd":
        fq.fq_norm_residual_bwd(st["dy"], st["dn"], st["x"], st["b"], *norm, o["dx"], o["db"], o["dgate"],
                                o["dw_post"], o["dw_pre"], o["ws"])
        return {k: v for k, v in o.items() if k != "ws" and v is not None}
    if c["dir"] == "int8":
        fq.fq_norm_residual_fwd(st["x"], st["b"], *norm, o["y"], None, o["codes"], o["scale"])
        fq.fq_grouped_gemm_int8(o["codes"], o["scale"], T, None, 1, T, st["seg"], (1, c["N"], H), o["w"],
                                o["z"], o["ws"])
        return {k: o[k] for k in ("y", "z", "scale") if o[k] is not None}
    fq.fq_norm_residual_fwd(st["x"], st["b"], *norm, o["y"], o.get("n"))
    return {k: v for k, v in o.items() if v is not None}


# ------------------------------------------------------------ the definition --
def _exact_codes(v):
    """Token codes and scales of rows v, steps in fp32, as float64."""
    v = v.float()
    top = torch.maximum(v.max(1).values, -v.min(1).values)
    s = torch.where(top > 0, torch.clamp(top * (1.0 / 127.0), min=2.0 ** -126), 1.0)
    z = v * (1.0 / s).unsqueeze(1)
    return z.clamp(-128.0, 127.0).round().double(), s.double()


def _exact_act(a, afmt, s):
    if afmt == "none":
        return a, torch.ones_like(a)
    z = a.to(BF).float() * (1.0 / s)
    if afmt == "int8":
        q, m = z.clamp(-128.0, 127.0).round(), (z >= -128.0) & (z <= 127.0)
    else:
        grid = torch.tensor([k * 2.0 ** -9 for k in range(8)] +
                            [(8 + k) * 2.0 ** e for e in range(-9, 6) for k in range(8)][:-1], device=DEV)
        mid = (grid[1:] + grid[:-1]) / 2
        v = z.abs().clamp(max=448.0)
        lo, hi = torch.bucketize(v, mid), torch.bucketize(v, mid, right=True)
        q, m = torch.copysign(grid[torch.where(lo % 2 == 0, lo, hi)], z), z.abs() <= 448.0
    return q.double() * s.double(), m.double()


def _exact_product(st, c):
    R, out = c["rows"], {}
    out["y"] = torch.zeros(R, c["N"], dtype=torch.float64, device=DEV)
    out["scale"] = torch.zeros(R, dtype=torch.float64, device=DEV)
    per_row = st["wscale"].double().reshape(c["E"], -1, 1).expand(c["E"], c["N"], 1)
    for e in range(c["E"]):
        a, b = st["segs"][e], st["segs"][e + 1]
        if a == b:
            continue
        q, out["scale"][a:b] = _exact_codes(st["x"][a:b])
        w = st["codes"][e].double() * per_row[e]
        out["y"][a:b] = torch.matmul(q * out["scale"][a:b].unsqueeze(1), w.t())
    return out


def _exact_gated(st, c):
    F, R, H = c["F"], c["T"] * c["topk"], c["H"]
    f64 = dict(dtype=torch.float64, device=DEV)
    out = {"aq": torch.zeros(R, F, **f64)}
    if c["dir"] == "bwd":
        out.update(dh=torch.zeros(R, 2 * F, **f64), dx=torch.zeros(R, H, **f64))
    if c["w"] == "int8":
        q, s = _exact_codes(st["x"])
        x = q * s.unsqueeze(1)
    else:
        x = st["x"].double()
    for e in range(c["E"]):
        a, b = st["segs"][e], st["segs"][e + 1]
        if a == b:
            continue
        rows = torch.div(st["perm"][a:b], c["topk"], rounding_mode="floor").long()
        if c["w"] == "int8":
            w = st["codes"][e].double() * st["wscale"][e].double().unsqueeze(1)
        else:
            w = st["w"][e].double()
        g = torch.matmul(x[rows], w[:F].t())
        u = torch.matmul(x[rows], w[F:].t())
        sig = torch.sigmoid(g)
        out["aq"][a:b], m = _exact_act(g * sig * u, c["afmt"], st["ascale"])
        if c["dir"] == "bwd":
            d = m * st["daq"][a:b].double()
            dg = d * u * (sig + g * sig * torch.sigmoid(-g))
            out["dh"][a:b, :F], out["dh"][a:b, F:] = dg, d * g * sig
            out["dx"][a:b] = torch.matmul(dg, w[:F]) + torch.matmul(d * g * sig, w[F:])
    return out


def _exact_rms(v, w):
    """(v / rms(v) * w, 1 / rms(v)) in float64; w None: v itself."""
    if w is None:
        return v, None
    r = 1.0 / torch.sqrt((v * v).sum(1) / v.shape[1] + EPS)
    return v * r.unsqueeze(1) * w.double(), r


def _exact_rms_grad(d, v, w, r):
    if w is None:
        return d
    d = d * w.double()
    k = (d * v).sum(1) * r ** 3 / v.shape[1]
    return d * r.unsqueeze(1) - v * k.unsqueeze(1)


def _exact_norm(st, c):
    y = st["x"].double()
    out = {}
    scale = st["alpha"] * (st["gate"].double() if c["gate"] else torch.ones(c["T"], device=DEV).double())
    if c["block"]:
        p, rb = _exact_rms(st["b"].double(), st["w_post"])
    if c["dir"] != "bwd":
        if c["block"]:
            y = y + scale.unsqueeze(1) * p
            out["y"] = y
        n = _exact_rms(y, st["w_pre"])[0]
        if c["dir"] == "int8":
            q, s = _exact_codes(n)
            w = st["codes"][0].double() * st["wscale"][0].double().unsqueeze(1)
            out.update(scale=s, z=torch.matmul(q * s.unsqueeze(1), w.t()))
        elif c["pre"]:
            out["n"] = n
        return out
    gy = st["dy"].double()
    if c["pre"]:
        r = _exact_rms(y, st["w_pre"])[1]
        dn = st["dn"].double()
        gy = gy + _exact_rms_grad(dn, y, st["w_pre"], r)
        out["dw_pre"] = (dn * y * r.unsqueeze(1)).sum(0)
    out["dx"] = gy
    if c["block"]:
        b = st["b"].double()
        dp = gy * scale.unsqueeze(1)
        out["db"] = _exact_rms_grad(dp, b, st["w_post"], rb)
        if c["gate"]:
            out["dgate"] = st["alpha"] * (gy * p).sum(1)
        if c["post"]:
            out["dw_post"] = (dp * b * rb.unsqueeze(1)).sum(0)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "int8":
        return _exact_product(st, case)
    return _exact_gated(st, case) if case["op"] == "gated" else _exact_norm(st, case)
