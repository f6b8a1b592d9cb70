"""The feed-forward operators in 8 bits as they are measured: their cases, inputs, plain
forms in elementary torch operations, the same calls of this package, and the definitions in
64 bits.

norm        root-mean-square norm after the residual's addition, out as fp8 codes and scales
norm_back   its gradient by the input and the weight
gated       both projections of a gated feed-forward block, the activation and their product,
            out as fp8 codes and scales (dense, contiguous grouped, masked grouped)
gated_back  the gradient by both projections, from their 8-bit checkpoint, as codes
wgrad       a weight's gradient from two 8-bit matrices (dense, contiguous grouped)
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def norm_case(op, T, K, dtype, residual, weight=True, fmt="e4m3", y=False, wide=0):
    """residual: a second input is added (norm), or the sum's own gradient is (norm_back);
    y: the bf16 output as well; wide: the input is the first K columns of rows this much
    longer."""
    return dict(op=op, T=T, K=K, dtype=dtype, residual=residual, weight=weight, fmt=fmt, y=y, wide=wide)


def gated_case(op, form, T, G, N, K, fmt="e4m3", act="silu", save=False, dtype="bf16"):
    """T: rows (dense), rows with their padding (contiguous) or the capacity (masked)."""
    return dict(op=op, form=form, T=T, G=G, N=N, K=K, fmt=fmt, act=act, save=save, dtype=dtype)


def wgrad_case(form, T, G, N, K, out="bf16", p_fmt="e4m3"):
    return dict(op="wgrad", form=form, T=T, G=G, N=N, K=K, out=out, p_fmt=p_fmt)


def listed():
    cases = {
        # one token of one request, before a projection
        "norm_token": norm_case("norm", 1, 7168, "bf16", True),
        # a prefill's rows; the bf16 output feeds the gate and the adapters
        "norm_prefill_4096x7168": norm_case("norm", 4096, 7168, "bf16", True, y=True),
        # fp32 activations inside wider rows, no residual, E5M2 codes
        "norm_odd_1093x1536": norm_case("norm", 1093, 1536, "f32", False, fmt="e5m2", wide=8),
        # the training step's backward pass, the residual stream's gradient added
        "norm_back_8192x7168": norm_case("norm_back", 8192, 7168, "bf16", True),
        # an odd number of fp32 rows without it
        "norm_back_517x2048": norm_case("norm_back", 517, 2048, "f32", False),
        # a decode step of 64 requests
        "gated_decode_64": gated_case("gated", "dense", 64, 1, 2048, 7168),
        # a decode step over a rank's experts, counts uniform in [0, cap]
        "gated_masked_4x256": gated_case("gated", "masked", 256, 4, 2048, 7168),
        # the largest: a training step's experts, gate and up kept in 8 bits
        "gated_train_16384": gated_case("gated", "contiguous", 16384, 8, 2048, 7168, save=True),
        # its backward pass up to the codes of both gradients
        "gated_back_16384": gated_case("gated_back", "contiguous", 16384, 8, 2048, 7168),
        # a short odd batch through a wide dense block
        "gated_back_517": gated_case("gated_back", "dense", 517, 1, 12288, 1536, fmt="e5m2", act="gelu"),
        # the down projection's weight, an odd number of rows
        "wgrad_dense_1093": wgrad_case("dense", 1093, 1, 7168, 2048),
        # both projections' weights of the training step's experts
        "wgrad_train_16384": wgrad_case("contiguous", 16384, 8, 4096, 7168),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    most = {w: max(work(c)[w] for c in listed()) for w in ("bytes", "flops")}
    while True:
        case = _draw(rng)
        if all(work(case)[w] <= most[w] for w in most) and _plain_bytes(case) <= 16 << 30:
            return case


def _plain_bytes(case):
    """What the grouped plain forms hold at once: a weight (or its gradient) for each block
    of 128 rows, in fp32."""
    if case.get("form") != "contiguous" or case["op"] == "gated_back":
        return 0
    return 4 * (case["T"] // 128 + 1) * case["N"] * case["K"] * (2 if case["op"] == "gated" else 1)


def _draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "gated", "gated", "gated", "gated_back", "wgrad", "wgrad"])
    if op in ("norm", "norm_back"):
        K = rng.choice([512, 1536, 2048, 4096, 7168, 16384, 128 * _log(rng, 1, 128)])
        return norm_case(op, _log(rng, 1, 16384), K, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6,
                         rng.random() < 0.8, rng.choice(["e4m3", "e4m3", "e5m2"]),
                         op == "norm" and rng.random() < 0.4, rng.choice([0, 0, 8, 40]))
    N, K = rng.choice([(2048, 7168), (12288, 1536), (16384, 512), (1024, 2048),
                       (128 * _log(rng, 1, 32), 128 * _log(rng, 1, 56))])
    form = rng.choice(["dense", "contiguous"] if op != "gated" else ["dense", "dense", "masked", "contiguous"])
    G = 1 if form == "dense" else rng.randint(1, 8)
    if form == "dense":
        T = _log(rng, 1, 8192)
    elif form == "masked":
        T = _log(rng, 1, 1024)
    else:
        T = 128 * max(2 * G, _log(rng, 1, 128)) + rng.choice([0, 0, 61])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "wgrad":
        return wgrad_case(form, T, G, *rng.choice([(2 * N, K), (K, N)]), p_fmt=fmt)
    return gated_case(op, form, T, G, N, K, fmt, rng.choice(["silu", "silu", "gelu"]),
                      form != "masked" and rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------------------- inputs
def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _segments(case):
    """(group, rows, rows with padding) of the contiguous form: blocks of 128 rows dealt
    out 4 : 2 : 1 : 1 ..., the last block of each segment partly filled; of three groups or
    more the last but one has no rows."""
    G, blocks = case["G"], case["T"] // 128
    share = ([4, 2] + [1] * G)[:G]
    if G >= 3:
        share[G - 2] = 0
    n = [blocks * s // sum(share) for s in share]
    n[0] += blocks - sum(n)
    return [(g, 128 * b - (41 * g + 17) % 128, 128 * b) for g, b in enumerate(n) if b]


def _counts(case):
    """Rows of each group of the masked form, spread over [0, cap], the first full; they go
    by the case, so that its work does."""
    cap = case["T"]
    return [cap if i == 0 else (i * 2654435761 >> 7) % (cap + 1) for i in range(case["G"])]


def _rows(case):
    """Rows that have work."""
    if case.get("form") == "contiguous":
        return sum(r for _, r, _ in _segments(case))
    if case.get("form") == "masked":
        return sum(_counts(case))
    return case["T"]


def _group_idx(case, g):
    """The rows' group index: segments in a drawn order, -1 for padding and behind the last."""
    segs = _segments(case)
    idx = torch.full((case["T"],), -1, device=DEV, dtype=torch.int32)
    at = 0
    for i in torch.randperm(len(segs), generator=g, device=DEV).tolist():
        group, rows, padded = segs[i]
        idx[at:at + rows] = group
        at += padded
    return idx


def _codes(x, fmt):
    """fp8 codes and scales of each 1x128 of x (..., n), fp32."""
    dtype, most = FP8[fmt]
    b = x.reshape(*x.shape[:-1], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax == 0, 1.0, amax / most)
    return (b / s).clamp(-most, most).to(dtype).reshape(x.shape), s[..., 0]


def _weight_codes(w):
    """E4M3 codes and scales of each 128x128 of w (..., n, k), fp32."""
    *lead, n, k = w.shape
    b = w.reshape(*lead, n // 128, 128, k // 128, 128)
    s = b.abs().amax((-3, -1), keepdim=True) / 448.0
    return (b / s).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(w.shape), s[..., 0, :, 0].contiguous()


def _spoil(codes, scales, bad):
    """Rows that are padding may hold anything: NaN here."""
    codes.view(torch.uint8)[bad] = 0x7F
    scales[bad] = float("nan")


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    made = {"norm": _prepare_norm, "norm_back": _prepare_norm, "gated": _prepare_gated,
            "gated_back": _prepare_gated_back, "wgrad": _prepare_wgrad}[case["op"]](case, g)
    return dict(made, case=case)


def _prepare_norm(case, g):
    T, K, dt = case["T"], case["K"], DTYPES[case["dtype"]]
    wide = _normal(g, T, K + case["wide"])
    wide[torch.rand(wide.shape, generator=g, device=DEV) < 0.001] *= 50    # a stream's outliers
    s = dict(x=wide.to(dt)[:, :K], w=1 + 0.2 * _normal(g, K) if case["weight"] else None, r=None)
    if case["op"] == "norm":
        if case["residual"]:
            s["r"] = (3 * _normal(g, T, K)).to(dt)
            s["h"] = torch.empty(T, K, device=DEV, dtype=dt)
        s["q"] = torch.empty(T, K, device=DEV, dtype=FP8[case["fmt"]][0])
        s["s"] = torch.empty(T, K // 128, device=DEV)
        s["y"] = torch.empty(T, K, device=DEV, dtype=torch.bfloat16) if case["y"] else None
        s["rstd"] = torch.empty(T, device=DEV)
    else:
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
        s["dy"] = (0.01 * _normal(g, T, K)).to(dt)
        s["dh"] = (0.01 * _normal(g, T, K)).to(dt) if case["residual"] else None
        s["dx"] = torch.empty(T, K, device=DEV, dtype=dt)
        s["dw"] = torch.empty(K, device=DEV) if case["weight"] else None
    return s


def _prepare_gated(case, g):
    form, T, G, N, K = (case[n] for n in ("form", "T", "G", "N", "K"))
    lead = (G, T) if form == "masked" else (T,)
    x = _normal(g, *lead, K)
    x[torch.rand(x.shape, generator=g, device=DEV) < 0.01] *= 10           # activations' outliers
    a, sa = _codes(x, "e4m3")
    del x
    b, sb = _weight_codes(_normal(g, *(() if form == "dense" else (G,)), 2 * N, K) * K ** -0.5)
    s = dict(a=a, sa=sa, b=b, sb=sb, idx=None, counts=None)
    if form == "contiguous":
        s["idx"] = _group_idx(case, g)
        _spoil(a, sa, s["idx"] < 0)
    elif form == "masked":
        s["counts"] = torch.tensor(_counts(case), device=DEV, dtype=torch.int32)
        _spoil(a, sa, torch.arange(T, device=DEV) >= s["counts"][:, None])
    dt = FP8[case["fmt"]][0]
    s["h"] = torch.zeros(*lead, N, device=DEV, dtype=torch.uint8).view(dt)
    s["sh"] = torch.zeros(*lead, N // 128, device=DEV)
    s["gu"] = torch.zeros(*lead, 2 * N, device=DEV, dtype=torch.uint8).view(dt) if case["save"] else None
    s["sgu"] = torch.zeros(*lead, N // 64, device=DEV) if case["save"] else None
    return s


def _prepare_gated_back(case, g):
    T, N = case["T"], case["N"]
    gu, sgu = _codes(_normal(g, T, 2 * N), "e4m3")
    s = dict(gu=gu, sgu=sgu, dh=(0.01 * _normal(g, T, N)).to(DTYPES[case["dtype"]]), idx=None)
    if case["form"] == "contiguous":
        s["idx"] = _group_idx(case, g)
        _spoil(gu, sgu, s["idx"] < 0)
    s["d"] = torch.zeros(T, 2 * N, device=DEV, dtype=torch.uint8).view(FP8[case["fmt"]][0])
    s["sd"] = torch.zeros(T, N // 64, device=DEV)
    return s


def _prepare_wgrad(case, g):
    T, G, N, K = (case[n] for n in ("T", "G", "N", "K"))
    dense = case["form"] == "dense"
    # a gradient's rows differ in size, as tokens do
    p, sp = _codes(0.01 * _normal(g, T, N) * torch.exp(_normal(g, T, 1)), case["p_fmt"])
    q, sq = _codes(_normal(g, T, K), "e4m3")
    s = dict(p=p, sp=sp, q=q, sq=sq, idx=None)
    if not dense:
        s["idx"] = _group_idx(case, g)
        _spoil(q, sq, s["idx"] < 0)
    s["dw"] = torch.empty(*(() if dense else (G,)), N, K, device=DEV, dtype=DTYPES[case["out"]])
    return s


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "norm_back": _norm_back_own, "gated": _gated_own,
                "gated_back": _gated_back_own, "wgrad": _wgrad_own}[op](state)
    return {"norm": _norm_plain, "norm_back": _norm_back_plain, "gated": _gated_plain,
            "gated_back": _gated_back_plain, "wgrad": _wgrad_plain}[op](state)


def _norm_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    c = s["case"]
    q, sc, h, y, rstd = dg.dg_rms_norm_fp8(s["x"], s["w"], residual=s["r"], eps=EPS, fmt=c["fmt"], Q=s["q"],
                                           S=s["s"], H=s.get("h"), Y=s["y"], rstd=s["rstd"])
    return q, sc, h, y, rstd


def _norm_back_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    return dg.dg_rms_norm_backward(s["dy"], s["x"], s["rstd"], s["w"], grad_h=s["dh"], grad_x=s["dx"],
                                   grad_weight=s["dw"])


def _gated_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    c = s["case"]
    how = dict(activation=c["act"], fmt=c["fmt"])
    args = s["a"], s["sa"], s["b"], s["sb"]
    if c["form"] == "masked":
        return dg.dg_grouped_gated_fp8_masked(*args, s["counts"], s["h"], s["sh"], **how)
    how.update(save=c["save"], GU=s["gu"], sGU=s["sgu"])
    if c["form"] == "dense":
        return dg.dg_gated_fp8_nt(*args, s["h"], s["sh"], **how)
    return dg.dg_grouped_gated_fp8_contiguous(*args, s["idx"], s["h"], s["sh"], **how)


def _gated_back_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    c = s["case"]
    return dg.dg_gated_backward(s["dh"], s["gu"], s["sgu"], s["d"], s["sd"], group_idx=s["idx"],
                                groups=c["G"], activation=c["act"], fmt=c["fmt"])


def _wgrad_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    c = s["case"]
    if c["form"] == "dense":
        return dg.dg_wgrad_fp8(s["p"], s["sp"], s["q"], s["sq"], s["dw"])
    return dg.dg_grouped_wgrad_fp8_contiguous(s["p"], s["sp"], s["q"], s["sq"], s["idx"], c["G"], s["dw"])


def _values(codes, scales):
    return (codes.float().view(*scales.shape, 128) * scales[..., None]).view(codes.shape)


def _norm_plain(s):
    c = s["case"]
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    v = h.float()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    y = v * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"]
    q, sc = _codes(y, c["fmt"])
    return q, sc, h, y.to(torch.bfloat16) if c["y"] else None, rstd


def _norm_back_plain(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy if s["w"] is None else dy * s["w"]
    dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["x"].dtype), None if s["w"] is None else (dy * h * r).sum(0)


def _sigmoid_of(g, act):
    """The factor that the activation puts on g, and its derivative's two parts: act(g) =
    g sigmoid(z), z = g (silu) or 2 sqrt(2/pi) (g + 0.044715 g^3) (gelu's tanh form)."""
    if act == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (g + 0.044715 * g * g * g), c * (1 + 3 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s, dz


def _live(s):
    """Rows that are written: their group is one, and their 128-row block's first row's."""
    idx, c = s["idx"], s["case"]
    lead = idx[torch.arange(c["T"], device=DEV) // 128 * 128]
    return (idx >= 0) & (idx < c["G"]) & (idx == lead)


def _blocks(v, live):
    """Rows of v, padding as zeros, in blocks of 128."""
    v = torch.where(live[:, None], v, torch.zeros((), device=DEV))
    pad = -v.shape[0] % 128
    return torch.cat([v, v.new_zeros(pad, v.shape[1])]).view(-1, 128, v.shape[1])


def _gated_plain(s):
    c = s["case"]
    N, K, T = c["N"], c["K"], c["T"]
    x = _values(s["a"], s["sa"])
    w = (s["b"].float().view(*s["sb"].shape[:-1], 128, K // 128, 128) *
         s["sb"][..., None, :, None]).view(s["b"].shape)
    if c["form"] == "dense":
        gu, live = x @ w.t(), None
    elif c["form"] == "masked":
        live = torch.arange(T, device=DEV) < s["counts"][:, None]
        gu = torch.bmm(torch.where(live[..., None], x, torch.zeros((), device=DEV)), w.transpose(1, 2))
    else:
        live = _live(s)
        of = s["idx"][::128].long().clamp(0, c["G"] - 1)
        gu = torch.bmm(_blocks(x, live), w[of].transpose(1, 2)).view(-1, 2 * N)[:T]
    g, u = gu[..., :N], gu[..., N:]
    outs = list(_codes(g * _sigmoid_of(g, c["act"])[0] * u, c["fmt"]))
    outs += list(_codes(gu, c["fmt"])) if c["save"] else [None, None]
    if live is not None:                      # the other rows stay what they were: zero
        zero = torch.zeros((), device=DEV)
        outs = [o if o is None else torch.where(live[..., None], o.float(), zero).to(o.dtype) for o in outs]
    return tuple(outs)


def _gated_back_plain(s):
    c = s["case"]
    N = c["N"]
    gu = _values(s["gu"], s["sgu"])
    if s["idx"] is not None:
        live = _live(s)[:, None]
        gu = torch.where(live, gu, torch.zeros((), device=DEV))
    g, u, dh = gu[:, :N], gu[:, N:], s["dh"].float()
    sg, dz = _sigmoid_of(g, c["act"])
    d, sd = _codes(torch.cat([dh * u * (sg + g * sg * (1 - sg) * dz), dh * g * sg], 1), c["fmt"])
    if s["idx"] is not None:
        d = torch.where(live, d.float(), torch.zeros((), device=DEV)).to(d.dtype)
        sd = torch.where(live, sd, torch.zeros((), device=DEV))
    return d, sd


def _wgrad_plain(s):
    c = s["case"]
    p, q = _values(s["p"], s["sp"]), _values(s["q"], s["sq"])
    if c["form"] == "dense":
        return (p.t() @ q).to(s["dw"].dtype)
    live = _live(s)
    parts = torch.bmm(_blocks(p, live).transpose(1, 2), _blocks(q, live))
    of = s["idx"][::128].long().clamp(0, c["G"] - 1)      # blocks of padding add zeros
    dw = torch.zeros(c["G"], c["N"], c["K"], device=DEV)
    return dw.index_add_(0, of, parts).to(s["dw"].dtype)


# -------------------------------------------------------------------------------- work
def work(case):
    K, T = case["K"], case["T"]
    if case["op"] in ("norm", "norm_back"):
        e = 2 if case["dtype"] == "bf16" else 4
        w = 4 * K if case["weight"] else 0
        if case["op"] == "norm":
            return {"bytes": T * K * (e * (3 if case["residual"] else 1) + 1 + (2 if case["y"] else 0)) +
                    T * K // 32 + w + 4 * T, "flops": 8 * T * K}
        return {"bytes": T * K * e * (4 if case["residual"] else 3) + 2 * w + 4 * T, "flops": 10 * T * K}
    N, G, rows = case["N"], case["G"], _rows(case)
    code = 33 / 32                                            # a code and its part of a scale
    idx = 4 * T if case["form"] == "contiguous" else 0
    if case["op"] == "wgrad":
        e = 2 if case["out"] == "bf16" else 4
        return {"bytes": code * rows * (N + K) + idx + G * N * K * e, "flops": 2 * rows * N * K}
    if case["op"] == "gated_back":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * N * (e + 4 * code) + idx, "flops": 20 * rows * N}
    used = len(_segments(case)) if case["form"] == "contiguous" else \
        sum(n > 0 for n in _counts(case)) if case["form"] == "masked" else 1
    return {"bytes": code * rows * K + used * 2 * N * K + code * rows * N * (3 if case["save"] else 1) + idx,
            "flops": 4 * rows * N * K}


# -------------------------------------------------------------------- the definitions
def _scaled(y, fmt):
    """Each 1x128 of y over its scale, rounded to 8 bits, and the scale."""
    dtype, most = FP8[fmt]
    b = y.view(*y.shape[:-1], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    s = amax / most
    s[amax == 0] = 1
    return (b / s).clamp(-most, most).to(dtype).double().view(y.shape), s[..., 0]


def _activation64(g, act):
    if act == "silu":
        return torch.nn.functional.silu(g)
    return torch.nn.functional.gelu(g, approximate="tanh")


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(s["x"].dtype).double()      # the sum is kept in its type
        rstd = (h.square().mean(1) + EPS).rsqrt()
        y = h * rstd[:, None] * (1 if s["w"] is None else s["w"].double())
        return (*_scaled(y, case["fmt"]), None, y if case["y"] else None, rstd)
    if case["op"] == "norm_back":
        h = s["x"].double().requires_grad_()
        w = torch.ones(case["K"], device=DEV, dtype=torch.float64) if s["w"] is None else s["w"].double()
        w.requires_grad_()
        y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * w
        dx, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        return dx if s["dh"] is None else dx + s["dh"].double(), None if s["w"] is None else dw
    if case["op"] == "wgrad":
        p = s["p"].double() * s["sp"].double().repeat_interleave(128, 1)
        q = s["q"].double() * s["sq"].double().repeat_interleave(128, 1)
        if case["form"] == "dense":
            return p.t() @ q
        return torch.stack([p[s["idx"] == i].t() @ q[s["idx"] == i] for i in range(case["G"])])
    N = case["N"]
    if case["op"] == "gated_back":
        gu = s["gu"].double() * s["sgu"].double().repeat_interleave(128, 1)
        live = torch.ones(case["T"], device=DEV, dtype=torch.bool) if s["idx"] is None else s["idx"] >= 0
        gu = gu[live].requires_grad_()
        h = _activation64(gu[:, :N], case["act"]) * gu[:, N:]
        got = _scaled(torch.autograd.grad(h, gu, s["dh"][live].double())[0], case["fmt"])
        outs = []
        for v in got:
            outs.append(torch.zeros(case["T"], v.shape[1], device=DEV, dtype=torch.float64))
            outs[-1][live] = v
        return tuple(outs)
    lead = s["h"].shape[:-1]
    outs = [torch.zeros(*lead, n, device=DEV, dtype=torch.float64) for n in (N, N // 128, 2 * N, N // 64)]
    for i in range(case["G"]):
        if case["form"] == "dense":
            at, b, sb = slice(None), s["b"], s["sb"]
        elif case["form"] == "masked":
            at, b, sb = (i, slice(0, int(s["counts"][i]))), s["b"][i], s["sb"][i]
        else:
            at, b, sb = s["idx"] == i, s["b"][i], s["sb"][i]
        x = s["a"][at].double() * s["sa"][at].double().repeat_interleave(128, 1)
        if x.shape[0] == 0:
            continue
        w = b.double() * sb.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        gu = x @ w.t()
        h = _activation64(gu[:, :N], case["act"]) * gu[:, N:]
        for o, v in zip(outs, (*_scaled(h, case["fmt"]), *_scaled(gu, case["fmt"]))):
            o[at] = v
    return tuple(outs) if case["save"] else (outs[0], outs[1], None, None)
