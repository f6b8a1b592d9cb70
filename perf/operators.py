"""The router and the adapters as they are measured: their cases, inputs, plain forms in
elementary torch operations, the same calls of this package, and the definitions in 64
bits.

route     the gate of a mixture of experts: scores, the k experts of each row, their
          weights, rows per expert, and (training) the balance loss
backward  the gradient of that gate's weights and loss by the logits
lora      low-rank adapters of many requests added to a shared projection's output
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------------------- cases
def route_case(op, T, E, k, dtype, score, normalize, balance, bias, padded, closed=0, pad_to=0):
    """padded: rows that are padding; closed: experts that may not be chosen (a bias of
    -inf); pad_to: the logits are the first E columns of rows of this many."""
    return dict(op=op, T=T, E=E, k=k, dtype=dtype, score=score, normalize=normalize,
                balance=balance, bias=bias, padded=padded, closed=closed, pad_to=pad_to)


def lora_case(T, N, K, R, L, used, layout, plain_rows=0, mixed_ranks=False):
    """used: how many of the L adapters the rows name; layout: "mixed" (rows of all
    requests interleaved, as in a decode batch), "segments" (each request's rows
    together, as in a prefill) or "both" (segments, then single rows); plain_rows: rows
    that name no adapter."""
    return dict(op="lora", T=T, N=N, K=K, R=R, L=L, used=used, layout=layout,
                plain_rows=plain_rows, mixed_ranks=mixed_ranks)


def listed():
    cases = {
        # one decode step of 64 requests: sigmoid scores with a selection bias, the counts
        # are the masked GEMM's masked_m
        "route_decode_64x256": route_case("route", 64, 256, 8, "bf16", "sigmoid", True, 0.0, True, 0),
        # the router of a training step over the 4x8192 rows of the contiguous GEMM
        "route_train_32768x256": route_case("route", 32768, 256, 8, "f32", "softmax", False, 1e-3,
                                            False, 1000),
        # an odd count of rows and experts, rows inside wider ones, two experts closed
        "route_train_4099x60": route_case("route", 4099, 60, 4, "bf16", "softmax", True, 1e-2, True,
                                          37, closed=2, pad_to=64),
        # the backward pass of that training step
        "backward_32768x256": route_case("backward", 32768, 256, 8, "f32", "softmax", False, 1e-3,
                                         False, 1000),
        # few experts, two a row, bf16 gradients
        "backward_8192x8": route_case("backward", 8192, 8, 2, "bf16", "sigmoid", True, 1e-2, False, 0),
        # a single request's token
        "lora_token": lora_case(1, 2112, 7168, 16, 8, 1, "mixed"),
        # a decode batch in which every request has an adapter of its own
        "lora_decode_64_distinct": lora_case(64, 4096, 7168, 16, 64, 64, "mixed"),
        # a decode batch over a few adapters of several ranks, some rows without one
        "lora_decode_128_shared": lora_case(128, 24576, 1536, 64, 8, 8, "mixed", plain_rows=16,
                                            mixed_ranks=True),
        # a chunk of a long prompt beside single tokens of other requests
        "lora_both_1093": lora_case(1093, 7168, 2048, 32, 32, 24, "both", plain_rows=5),
        # an output width that no vector of 8 divides
        "lora_prefill_odd_517x2111": lora_case(517, 2111, 7168, 16, 4, 3, "segments"),
        # a prefill of four prompts
        "lora_prefill_4096": lora_case(4096, 7168, 2048, 16, 8, 4, "segments"),
        # the largest: long prompts through the deepest projection, rank 64
        "lora_prefill_8192": lora_case(8192, 7168, 16384, 64, 16, 8, "segments", mixed_ranks=True),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    most = listed()[-1]
    while True:
        case = _draw(rng)
        if all(work(case)[w] <= work(most)[w] for w in ("bytes", "flops")) and (
                case["op"] != "lora" or _all_adapters(case) <= _all_adapters(most)):
            return case


def _all_adapters(case):
    """Operations of the plain form, which takes every row through every adapter."""
    return case["T"] * case["L"] * case["R"] * (case["K"] + case["N"])


def _draw(rng):
    if rng.random() < 0.5:
        op = rng.choice(["route", "route", "backward"])
        T = _log(rng, 1, 32768)
        E = rng.choice([8, 16, 32, 64, 128, 256, 384, 512]) if rng.random() < 0.6 else _log(rng, 2, 512)
        k = rng.randint(1, min(8, E))
        train = op == "backward" or rng.random() < 0.6
        return route_case(op, T, E, k, rng.choice(["f32", "bf16"]), rng.choice(["softmax", "sigmoid"]),
                          rng.random() < 0.5, rng.choice([1e-3, 1e-2]) if train else 0.0,
                          rng.random() < 0.5, rng.choice([0, 0, T // 8, T // 2]),
                          closed=rng.choice([0, 0, (E - k) // 4]),
                          pad_to=rng.choice([0, 0, 0, E + 3]))
    T = _log(rng, 1, 8192)
    N, K = rng.choice([(2112, 7168), (24576, 1536), (32768, 512), (7168, 16384), (4096, 7168),
                       (7168, 2048), (_log(rng, 64, 16384), 128 * _log(rng, 1, 64))])
    L = _log(rng, 1, 64)
    used = min(T, rng.randint(1, L))
    layout = "mixed" if T <= 128 else rng.choice(["segments", "segments", "both"])
    return lora_case(T, N, K, rng.choice([8, 16, 16, 32, 64]), L, used, layout,
                     plain_rows=rng.choice([0, 0, (T - used) // 4]),
                     mixed_ranks=rng.random() < 0.3)


# ------------------------------------------------------------------------------- inputs
def _ranks(case):
    """Rank of each adapter: all R, or R, R/2, R/4, R, ... (rounded up)."""
    R = case["R"]
    return [max(1, R >> (i % 3)) if case["mixed_ranks"] else R for i in range(case["L"])]


def _rows_of(case):
    """Rows of each used adapter: one each, and the rest dealt out 4 : 2 : 1 : 1 ..."""
    T, used, left = case["T"], case["used"], case["T"] - case["used"] - case["plain_rows"]
    share = [4, 2] + [1] * (used - 2) if used > 2 else [1] * used
    if case["layout"] == "both":                # long prompts of the first two requests
        share = [3, 1][:used] + [0] * (used - 2)
    rows = [1 + left * s // sum(share) for s in share]
    rows[0] += T - case["plain_rows"] - sum(rows)
    return rows


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    return (_prepare_lora if case["op"] == "lora" else _prepare_route)(case, g)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _prepare_route(case, g):
    T, E, k, dt = case["T"], case["E"], case["k"], DTYPES[case["dtype"]]
    wide = torch.full((T, max(E, case["pad_to"])), float("nan"), device=DEV, dtype=dt)
    logits = wide[:, :E]
    logits.copy_(1.5 * _normal(g, T, E) + 0.5 * _normal(g, E))
    s = dict(case=case, logits=logits, bias=None, valid=None)
    if case["bias"] or case["closed"]:
        s["bias"] = 0.1 * _normal(g, E)
        if case["closed"]:
            s["bias"][torch.randperm(E, generator=g, device=DEV)[:case["closed"]]] = -math.inf
    if case["padded"]:
        rows = torch.randperm(T, generator=g, device=DEV)[:case["padded"]]
        s["valid"] = torch.ones(T, device=DEV, dtype=torch.uint8)
        s["valid"][rows] = 0
        logits[rows] = float("nan")                       # padding may hold anything
    s["ids"] = torch.empty(T, k, device=DEV, dtype=torch.int32)
    if case["op"] == "route":
        s["weights"] = torch.empty(T, k, device=DEV)
        s["counts"] = torch.empty(E, device=DEV, dtype=torch.int32)
        s["loss"] = torch.empty((), device=DEV) if case["balance"] else None
        s["coef"] = torch.empty(E, device=DEV) if case["balance"] else None
    else:                                                 # what the forward pass has left
        ids, _, _, _, s["coef"] = _route_plain(s)
        s["ids"].copy_(ids)
        s["grad_weights"] = _normal(g, T, k)
        s["grad_loss"] = torch.rand((), generator=g, device=DEV) + 0.5
        s["grad_logits"] = torch.empty(T, E, device=DEV, dtype=dt)
    return s


def _prepare_lora(case, g):
    T, N, K, R, L = (case[n] for n in ("T", "N", "K", "R", "L"))
    x = _normal(g, T, K, dtype=torch.bfloat16)
    x[torch.rand(T, K, generator=g, device=DEV) < 0.01] *= 30          # activations' outliers
    A = _normal(g, L, R, K, dtype=torch.bfloat16).mul_(K ** -0.5)
    B = _normal(g, L, N, R, dtype=torch.bfloat16).mul_(0.05)
    ranks = torch.tensor(_ranks(case), device=DEV, dtype=torch.int32)
    names = torch.randperm(L, generator=g, device=DEV)
    # adapters of rank r sit at the names with that rank's index: the work is the case's
    names = torch.arange(L, device=DEV) if case["mixed_ranks"] else names
    rows = torch.tensor(_rows_of(case) + [case["plain_rows"]], device=DEV)
    which = torch.cat([names[:case["used"]], torch.tensor([-1], device=DEV)])
    ids = torch.repeat_interleave(which, rows, output_size=T).int()
    if case["layout"] == "mixed":
        ids = ids[torch.randperm(T, generator=g, device=DEV)].contiguous()
    return dict(case=case, x=x, A=A, B=B, ids=ids,
                ranks=ranks if case["mixed_ranks"] else None,
                scales=0.5 + torch.rand(L, generator=g, device=DEV),
                base=_normal(g, T, N, dtype=torch.bfloat16),
                out=torch.empty(T, N, device=DEV, dtype=torch.bfloat16))


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _route_own, "backward": _backward_own, "lora": _lora_own}[op](state)
    return {"route": _route_plain, "backward": _backward_plain, "lora": _lora_plain}[op](state)


def _route_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    c = s["case"]
    return dg.dg_moe_route(s["logits"], c["k"], bias=s["bias"], row_valid=s["valid"], score=c["score"],
                           normalize=c["normalize"], scale=2.5, balance=c["balance"] or None,
                           ids=s["ids"], weights=s["weights"], counts=s["counts"], loss=s["loss"],
                           coef=s["coef"])


def _backward_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    c = s["case"]
    return dg.dg_moe_route_backward(s["logits"], s["ids"], coef=s["coef"], grad_loss=s["grad_loss"],
                                    grad_weights=s["grad_weights"], row_valid=s["valid"],
                                    score=c["score"], normalize=c["normalize"], scale=2.5,
                                    grad_logits=s["grad_logits"])


def _lora_own(s):
    import moe_grouped_gemm_lhs_amd as dg
    return dg.dg_lora_bf16(s["x"], s["A"], s["B"], s["ids"], s["base"], s["out"], scales=s["scales"],
                           ranks=s["ranks"])


def _scores(s):
    """The live rows' scores and probabilities (softmax, or sigmoid and its share)."""
    z = s["logits"].float()
    if s["valid"] is not None:
        z = torch.where(s["valid"][:, None] != 0, z, torch.zeros((), device=DEV))
    if s["case"]["score"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        return z, p, p
    sc = 1.0 / (1.0 + torch.exp(-z))
    return z, sc, sc / sc.sum(1, keepdim=True)


def _route_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    z, sc, p = _scores(s)
    key = z if s["bias"] is None else z + s["bias"]
    key, order = torch.sort(key, dim=1, descending=True, stable=True)
    live = key[:, :k] > -math.inf
    if s["valid"] is not None:
        live = live & (s["valid"][:, None] != 0)
    ids = torch.where(live, order[:, :k], -1)
    w = torch.where(live, torch.gather(sc, 1, order[:, :k]), torch.zeros((), device=DEV))
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones((), device=DEV))
    counts = torch.zeros(E + 1, device=DEV, dtype=torch.int32)
    counts.index_add_(0, torch.where(live, ids, E).reshape(-1),
                      torch.ones(T * k, device=DEV, dtype=torch.int32))
    counts = counts[:E]
    loss = coef = None
    if c["balance"]:
        if s["valid"] is not None:
            rows = s["valid"].sum().float()
            p = torch.where(s["valid"][:, None] != 0, p, torch.zeros((), device=DEV))
        else:
            rows = torch.full((), float(T), device=DEV)
        coef = (c["balance"] * E / k) * counts.float() / rows / rows
        loss = (coef * p.sum(0)).sum()
    return ids.int(), 2.5 * w, counts, loss, coef


def _backward_plain(s):
    c = s["case"]
    _, sc, p = _scores(s)
    live = s["ids"] >= 0
    at = torch.where(live, s["ids"], 0).long()
    zero = torch.zeros((), device=DEV)
    gw = torch.where(live, 2.5 * s["grad_weights"], zero)
    if c["normalize"]:
        chosen = torch.where(live, torch.gather(sc, 1, at), zero)
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones((), device=DEV))
        gw = torch.where(live, (gw - (gw * chosen).sum(1, keepdim=True) / total) / total, zero)
    by_score = torch.zeros_like(sc).scatter_add_(1, at, gw)
    u = (s["grad_loss"] * s["coef"])[None, :]
    if c["score"] == "softmax":
        g = by_score + u
        dz = sc * (g - (g * sc).sum(1, keepdim=True))
    else:
        g = by_score + (u - (u * p).sum(1, keepdim=True)) / sc.sum(1, keepdim=True)
        dz = g * sc * (1 - sc)
    if s["valid"] is not None:
        dz = torch.where(s["valid"][:, None] != 0, dz, zero)
    return dz.to(s["logits"].dtype)


def _lora_plain(s):
    """All adapters' products at once, each row keeping its own adapter's."""
    A, B = s["A"].float(), s["B"].float()
    L, R, K = A.shape
    N = B.shape[1]
    mine = (s["ids"][:, None] == torch.arange(L, device=DEV))[:, :, None]
    if s["ranks"] is not None:
        mine = mine & (torch.arange(R, device=DEV) < s["ranks"][:, None])
    h = (s["x"].float() @ A.view(L * R, K).t()).view(-1, L, R) * s["scales"][:, None]
    h = torch.where(mine, h, torch.zeros((), device=DEV)).reshape(-1, L * R)
    delta = h @ B.permute(0, 2, 1).reshape(L * R, N)
    return (s["base"].float() + delta).to(torch.bfloat16)


# -------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "lora":
        T, N, K = case["T"], case["N"], case["K"]
        r = _ranks(case)[:case["used"]]
        rows = _rows_of(case)
        some = T - case["plain_rows"]
        return {"bytes": 2 * some * K + 4 * T * N + 4 * T + sum(2 * x * (K + N) for x in r),
                "flops": sum(2 * m * x * (K + N) for m, x in zip(rows, r))}
    T, E, k = case["T"], case["E"], case["k"]
    elt = 2 if case["dtype"] == "bf16" else 4
    live = T - case["padded"]
    b = live * E * elt + (T if case["padded"] else 0)
    if case["op"] == "route":
        b += 8 * T * k + 4 * E + (4 * E if case["bias"] else 0) + (4 * E + 4 if case["balance"] else 0)
        return {"bytes": b, "flops": 6 * live * E}
    return {"bytes": b + 8 * live * k + T * E * elt + 4 * E, "flops": 10 * live * E}


# -------------------------------------------------------------------- the definitions
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        out = s["base"].double()
        for i in range(case["L"]):
            rows = (s["ids"] == i).nonzero()[:, 0]
            if rows.numel():
                r = _ranks(case)[i]
                h = s["x"][rows].double() @ s["A"][i, :r].double().t().contiguous()
                d = h @ s["B"][i, :, :r].double().t().contiguous()
                out[rows] += s["scales"][i].double() * d
        return out
    live = torch.ones(case["T"], device=DEV, dtype=torch.bool) if s["valid"] is None else s["valid"].bool()
    z = s["logits"][live].double()
    sm = case["score"] == "softmax"
    sc = torch.softmax(z, 1) if sm else torch.sigmoid(z)
    p = sc if sm else sc / sc.sum(1, keepdim=True)
    if case["op"] == "route":
        key = s["logits"][live].float() + (0 if s["bias"] is None else s["bias"])
        order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["k"]]
        open_ = torch.isfinite(key.gather(1, order))
        w = sc.gather(1, order) * open_
        if case["normalize"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        weights = torch.zeros(case["T"], case["k"], device=DEV, dtype=torch.float64)
        weights[live] = 2.5 * w
        if not case["balance"]:
            return None, weights, None, None, None
        n = torch.bincount(order[open_], minlength=case["E"]).double()
        rows = float(live.sum())
        coef = case["balance"] * case["E"] * n / (case["k"] * rows * rows)
        return None, weights, None, coef @ p.sum(0), coef
    # the gradient of  sum(grad_weights * weights) + grad_loss * sum(coef * p)  by autograd
    z.requires_grad_()
    sc = torch.softmax(z, 1) if sm else torch.sigmoid(z)
    p = sc if sm else sc / sc.sum(1, keepdim=True)
    ids = s["ids"][live].long()
    w = sc.gather(1, ids.clamp_min(0)) * (ids >= 0)
    if case["normalize"]:
        w = w / w.sum(1, keepdim=True)
    total = (2.5 * w * s["grad_weights"][live].double()).sum() + \
        s["grad_loss"].double() * (p * s["coef"].double()).sum()
    grad = torch.zeros(case["T"], case["E"], device=DEV, dtype=torch.float64)
    grad[live] = torch.autograd.grad(total, z)[0]
    return grad
