"""The operators around the experts' products, as cases to be timed and compared.

Routing tokens to experts and its gradient, sorting token rows by expert, summing the experts' rows back into tokens
and its gradients, and products of a few unquantized tokens with NVFP4 weights, shared or one expert's.  ``run``
computes them in their plain form (elementary torch operations), or, where ``own`` is true, makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # E2M1 magnitudes


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step's router: bf16 logits (equal ones among them), plain softmax scores
        dict(name="route decode", op="route", T=64, E=64, k=6, score="softmax", renorm=False, bias=False, groups=1, kept=1, pair=False,
             fp32=False, scale=1.0, masked=2),
        # a long prefill or a training batch: sigmoid scores, a balancing bias, the four best of eight groups
        dict(name="route training", op="route", T=32768, E=256, k=8, score="sigmoid", renorm=True, bias=True, groups=8, kept=4, pair=True,
             fp32=True, scale=2.5, masked=0),
        # gradient of softmax scores, which reach every expert; odd sizes
        dict(name="route backward softmax", op="route_backward", T=16301, E=160, k=6, score="softmax", renorm=False, bias=False, groups=8,
             kept=3, pair=False, fp32=False, scale=16.0, masked=13),
        # gradient of renormalised sigmoid scores, which reaches the chosen experts alone
        dict(name="route backward sigmoid", op="route_backward", T=32768, E=256, k=8, score="sigmoid", renorm=True, bias=True, groups=8,
             kept=4, pair=True, fp32=True, scale=2.5, masked=0),
        # decode: 64 requests' tokens copied next to their experts' others
        dict(name="dispatch decode", op="dispatch", T=64, k=8, E=256, C=4096, masked=3),
        # a training batch's tokens on their way into 64 experts
        dict(name="dispatch training", op="dispatch", T=16384, k=8, E=64, C=4096, masked=0),
        # the end of a decode step's expert layer, added to the residual stream
        dict(name="combine decode", op="combine", T=64, k=8, E=256, C=4096, weights=True, residual=True, masked=3),
        # an odd training batch
        dict(name="combine training", op="combine", T=16301, k=6, E=64, C=4096, weights=True, residual=False, masked=0),
        # gradients of the experts' rows and of the routing weights
        dict(name="combine backward", op="combine_backward", T=16384, k=8, E=64, C=4096, masked=0),
        # one token through a dense projection
        dict(name="product one token", op="gemv", T=1, k=1, E=1, N=14336, K=4096, dense=True, shared=True, fp32=False, masked=0),
        # the tokens of a small decode batch through another projection, the other way round
        dict(name="product few tokens", op="gemv", T=24, k=1, E=1, N=4096, K=14336, dense=True, shared=True, fp32=True, masked=0),
        # eight tokens, two experts each, into the experts' up-projection
        dict(name="product by expert", op="gemv", T=8, k=2, E=8, N=14336, K=4096, dense=False, shared=True, fp32=False, masked=1),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))

    op = rng.choice(["route", "route_backward", "dispatch", "combine", "combine_backward", "gemv"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8, 6])
        per = size(max(2, 8 // groups), 512 // groups)
        kept = rng.randrange((groups + 1) // 2, groups + 1)
        T = size(1, 32768)
        return dict(op=op, T=T, E=groups * per, k=size(1, min(16, kept * per)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, bias=rng.random() < 0.5, groups=groups, kept=kept, pair=rng.random() < 0.5,
                    fp32=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), masked=rng.randrange(0, T // 16 + 1))
    if op == "gemv":
        T, dense = size(1, 32), rng.random() < 0.4
        E, k = (1, 1) if dense else (size(2, 32), size(1, 4))
        k = min(k, E)
        N = size(128, 14336, 128)
        most = max(64, min(14336, 8 * 14336 * 4096 // (E * N) // 64 * 64))
        return dict(op=op, T=T, k=k, E=E, N=N, K=size(64, most, 64), dense=dense, shared=dense or rng.random() < 0.5,
                    fp32=rng.random() < 0.3, masked=0 if dense else rng.randrange(0, T // 4 + 1))
    T, E = size(1, 16384), size(8, 256)
    k = size(1, 8)
    C = size(64, min(14336, max(64, 16384 * 8 * 4096 // (T * k))), 8)
    c = dict(op=op, T=T, k=k, E=E, C=C, masked=rng.choice([0, rng.randrange(0, T // 8 + 1)]))
    if op == "combine":
        c.update(weights=rng.random() < 0.7, residual=rng.random() < 0.5)
    return c


def work(case):
    c = case
    T, k, E = c["T"], c["k"], c["E"]
    if c["op"] == "route":
        size = 4 if c["fp32"] else 2
        return {"bytes": T * E * size + T * k * 8, "flops": T * E * 12}
    if c["op"] == "route_backward":
        size = 4 if c["fp32"] else 2
        whole = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * E * size * (2 if whole else 1) + T * k * (8 if whole else 8 + size), "flops": T * (12 * E if whole else 12 * k)}
    if c["op"] == "gemv":
        P = T * k
        used = 1 if c["dense"] else min(E, max(1, P - c["masked"]))
        return {"bytes": int(0.5625 * used * c["N"] * c["K"]) + 2 * (T if c["shared"] else P) * c["K"] + P * c["N"] * (4 if c["fp32"] else 2),
                "flops": 2 * P * c["N"] * c["K"]}
    P, C = T * k, c["C"]
    if c["op"] == "dispatch":
        return {"bytes": 2 * C * (T + P) + 8 * P + 4 * E, "flops": P}
    if c["op"] == "combine":
        return {"bytes": 2 * C * (P + T * (2 if c["residual"] else 1)) + 4 * P * (2 if c["weights"] else 1), "flops": 2 * P * C}
    return {"bytes": 2 * C * (T + 2 * P) + 12 * P, "flops": 3 * P * C}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _logits(c, gen):
    """Router logits: some experts are liked more than others; some tokens are padding (every expert masked)."""
    z = torch.randn((c["T"], c["E"]), generator=gen, device="cuda") * 1.5 + 0.5 * torch.randn(c["E"], generator=gen, device="cuda")
    z = z if c["fp32"] else z.bfloat16()
    if c["masked"]:
        z[torch.randperm(c["T"], generator=gen, device="cuda")[: c["masked"]]] = -math.inf
    return z


def _choices(c, gen):
    """k different experts of each token, unevenly liked; -1 for padding tokens."""
    T, E, k = c["T"], c["E"], c["k"]
    p = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
    ids = torch.sort(p, dim=-1, descending=True).indices[:, :k].to(torch.int32)
    if c["masked"]:
        ids[torch.randperm(T, generator=gen, device="cuda")[: c["masked"]]] = -1
    return ids


def _hidden(T, C, gen):
    v = torch.randn((T, C), generator=gen, device="cuda")
    v[:, torch.randint(0, C, (max(1, C // 1000),), generator=gen, device="cuda")] *= 20   # outlier channels
    return v.bfloat16()


def _weight(N, K, gen):
    """One NVFP4 weight: codes [N, K/2], scales in the GEMM layout, tensor scale [1]."""
    w = torch.randn((N, K), generator=gen, device="cuda") * 0.02
    alpha = (w.abs().amax() / 2688.0).view(1)
    b = w.view(N, K // 16, 16)
    delta = (b.abs().amax(-1) / (alpha * 6.0)).to(torch.float8_e4m3fn)
    a = b.abs() / (delta.float() * alpha).clamp(min=1e-30).unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    q = (torch.bucketize(a, edges, out_int32=True) | (torch.signbit(b).int() << 3)).to(torch.uint8).view(N, K // 2, 2)
    scales = delta.view(torch.uint8).view(N // 128, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return q[..., 0] | (q[..., 1] << 4), scales, alpha


def _softly(T, k, gen):
    return torch.softmax(torch.randn((T, k), generator=gen, device="cuda"), -1) * 2.5


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] in ("route", "route_backward"):
        s["logits"] = _logits(c, gen)
        s["bias"] = 0.1 * torch.randn(c["E"], generator=gen, device="cuda") if c["bias"] else None
        if c["op"] == "route_backward":
            s["ids"] = _plain_route(s)["ids"]
            s["dweights"] = torch.randn((c["T"], c["k"]), generator=gen, device="cuda") * 1e-3
    elif c["op"] == "gemv":
        made = [_weight(c["N"], c["K"], gen) for _ in range(c["E"])]
        s["W"], s["sW"], s["alphaW"] = (torch.stack([m[i] for m in made]) for i in range(3))
        s["alphaW"] = s["alphaW"].view(-1)
        if c["dense"]:
            s["W"], s["sW"], s["ids"] = s["W"][0], s["sW"][0], None
        else:
            s["ids"] = _choices(c, gen)
        s["x"] = _hidden(c["T"] * (1 if c["shared"] else c["k"]), c["K"], gen)
    else:
        T, k, C = c["T"], c["k"], c["C"]
        s["ids"] = _choices(c, gen)
        if c["op"] == "dispatch":
            s["x"] = _hidden(T, C, gen)
        else:
            s["rows"] = _plain_sort(s["ids"], c["E"])[0]
            s["y"] = torch.randn((T * k, C), generator=gen, device="cuda").bfloat16()
            s["weights"] = _softly(T, k, gen) if c.get("weights", True) else None
            if c["op"] == "combine_backward":
                s["dout"] = (torch.randn((T, C), generator=gen, device="cuda") * 1e-2).bfloat16()
            else:
                s["residual"] = torch.randn((T, C), generator=gen, device="cuda").bfloat16() if c["residual"] else None
        if c["masked"] and c["op"] != "combine":
            s["out"] = torch.zeros((T * k, C), dtype=torch.bfloat16, device="cuda")   # rows of no token stay as they are
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _share(z, score):
    """softmax or sigmoid of rows z; rows that are masked throughout give zeros."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=torch.finfo(z.dtype).min))
    return e / e.sum(-1, keepdim=True).clamp(min=torch.finfo(z.dtype).tiny)


def _first(v, n):
    """The n largest of the last axis, equal ones in the order of their places."""
    r = torch.sort(v, dim=-1, descending=True, stable=True)
    return r.values[..., :n], r.indices[..., :n]


def _plain_route(s):
    c, z = s["case"], s["logits"]
    T, E = z.shape
    open_ = z > torch.finfo(z.dtype).min
    v = z.double()
    if s["bias"] is not None or c["groups"] > 1:
        v = _share(v, c["score"])
    if s["bias"] is not None:
        v = v + s["bias"].double()
    v = v.masked_fill(~open_, -math.inf)
    if c["groups"] > 1:
        of_group = v.view(T, c["groups"], -1)
        two = _first(of_group, 2)[0]
        best = two[..., 0]
        if c["pair"] and two.shape[-1] > 1:
            best = best + two[..., 1].masked_fill(two[..., 1] == -math.inf, 0.0)
        kept = torch.zeros((T, c["groups"]), dtype=torch.bool, device=z.device).scatter_(1, _first(best, c["kept"])[1], True)
        v = of_group.masked_fill(~kept.unsqueeze(-1), -math.inf).view(T, E)
    top, ids = _first(v, c["k"])
    got = top > -math.inf
    share = _share(z.float(), c["score"]).gather(1, ids).masked_fill(~got, 0.0)
    if c["renorm"]:
        share = share / share.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
    return {"ids": ids.masked_fill(~got, -1).to(torch.int32), "weights": share * c["scale"]}


def _plain_route_backward(s):
    c = s["case"]
    z, ids = s["logits"].float(), s["ids"].long()
    got = ids >= 0
    at = ids.clamp(min=0)
    g = (s["dweights"] * c["scale"]).masked_fill(~got, 0.0)
    share = _share(z, c["score"])
    mine = share.gather(1, at).masked_fill(~got, 0.0)
    if c["renorm"]:
        p = mine / mine.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
        g = p * (g - (p * g).sum(-1, keepdim=True))
        if c["score"] == "sigmoid":
            g = g * (1 / (1 + torch.exp(z.gather(1, at)))).masked_fill(~got, 0.0)
        d = torch.zeros_like(z).scatter_add_(1, at, g)
    elif c["score"] == "sigmoid":
        d = torch.zeros_like(z).scatter_add_(1, at, g * mine / (1 + torch.exp(z.gather(1, at))))
    else:
        d = share * (torch.zeros_like(z).scatter_add_(1, at, g) - (mine * g).sum(-1, keepdim=True))
    return d.to(s["logits"].dtype)


def _plain_sort(ids, E):
    """Places of the pairs (token, choice) in the order of their experts, and where each expert's begin."""
    flat = ids.reshape(-1).long()
    key = flat.masked_fill(flat < 0, E)
    order = torch.sort(key, dim=0, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:E], 0)])
    return place.masked_fill(flat < 0, -1).view(ids.shape).to(torch.int32), offsets.to(torch.int32)


def _plain_dispatch(s):
    x, ids = s["x"], s["ids"]
    rows, offsets = _plain_sort(ids, s["case"]["E"])
    P = ids.numel()
    xs = torch.zeros((P + 1, x.shape[1]), dtype=x.dtype, device=x.device)
    at = rows.view(-1).long()
    xs[at.masked_fill(at < 0, P)] = x.repeat_interleave(ids.shape[1], 0)
    return {"xs": xs[:P], "rows": rows, "offsets": offsets}


def _taken(y, rows):
    """y's rows of each token [T, k, C] in 32 bits, zeros where there is none."""
    return torch.cat([y, y.new_zeros((1, y.shape[1]))])[rows.long()].float()   # row -1 is the last one


def _plain_combine(s):
    v = _taken(s["y"], s["rows"])
    if s["weights"] is not None:
        v = v * s["weights"].unsqueeze(-1)
    out = v.sum(1)
    return (out if s["residual"] is None else out + s["residual"].float()).bfloat16()


def _plain_combine_backward(s):
    rows, P = s["rows"], s["y"].shape[0]
    dout = s["dout"].float().unsqueeze(1)
    dw = (_taken(s["y"], rows) * dout).sum(-1)
    dy = torch.zeros((P + 1, s["y"].shape[1]), dtype=torch.bfloat16, device=rows.device)
    at = rows.view(-1).long()
    dy[at.masked_fill(at < 0, P)] = (dout * s["weights"].unsqueeze(-1)).bfloat16().view(P, -1)
    return {"dy": dy[:P], "dweights": dw}


def _read(codes, scales):
    """q * Delta of packed codes [..., N, K/2] with scales in the GEMM layout, exact in 32 bits."""
    N, K = codes.shape[-2], codes.shape[-1] * 2
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], -1).view(-1).int()
    delta = scales.view(-1, N // 128, K // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1, N, K // 16, 1)
    return (grid.index_select(0, nib).view(-1, N, K // 16, 16) * delta.view(torch.float8_e4m3fn).float()).view(-1, N, K)


def _plain_gemv(s):
    c = s["case"]
    y = torch.matmul(s["x"].float(), _read(s["W"], s["sW"]).transpose(1, 2)) * s["alphaW"].view(-1, 1, 1)   # [E, rows of x, N]
    if c["dense"]:
        y = y[0]
    else:
        ids = s["ids"].view(-1).long()
        pair = torch.arange(ids.numel(), device=ids.device)
        y = y[ids.clamp(min=0), pair // c["k"] if c["shared"] else pair].masked_fill((ids < 0).unsqueeze(-1), 0.0)
    return y if c["fp32"] else y.bfloat16()


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "dispatch": _plain_dispatch, "combine": _plain_combine,
          "combine_backward": _plain_combine_backward, "gemv": _plain_gemv}


# ---------------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    from nvfp4_block_quantization_amax_b200 import api
    c = s["case"]
    if c["op"] in ("route", "route_backward"):
        score = api.NVFP4_ROUTE_SIGMOID if c["score"] == "sigmoid" else api.NVFP4_ROUTE_SOFTMAX
        flags = api.NVFP4_ROUTE_RENORM if c["renorm"] else 0
        if c["op"] == "route":
            if c["pair"]:
                flags |= api.NVFP4_ROUTE_GROUP_PAIR
            ids, weights = api.nvfp4_route(s["logits"], c["k"], score, flags, bias=s["bias"], groups=c["groups"], groups_kept=c["kept"],
                                           scale=c["scale"])
            return {"ids": ids, "weights": weights}
        return api.nvfp4_route_backward(s["dweights"], s["ids"], s["logits"], score, flags, scale=c["scale"])
    if c["op"] == "dispatch":
        xs, rows, offsets = api.nvfp4_dispatch(s["x"], s["ids"], c["E"], out=s.get("out"))
        return {"xs": xs, "rows": rows, "offsets": offsets}
    if c["op"] == "combine":
        return api.nvfp4_combine(s["y"], s["rows"], s["weights"], residual=s["residual"])
    if c["op"] == "combine_backward":
        dy, dweights = api.nvfp4_combine_backward(s["dout"], s["rows"], s["weights"], s["y"], out=s.get("out"))
        return {"dy": dy, "dweights": dweights}
    return api.nvfp4_gemv(s["x"], s["W"], s["sW"], s["alphaW"], ids=s["ids"],
                          out_dtype=api.NVFP4_OUT_DTYPE_FP32 if c["fp32"] else api.NVFP4_OUT_DTYPE_BF16)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _log_share(z, score):
    if score == "sigmoid":
        return -np.logaddexp(0.0, -z)
    with np.errstate(invalid="ignore", divide="ignore"):
        return z - np.logaddexp.reduce(z, axis=1, keepdims=True)


def _exact_weights(c, z, ids):
    """Routing weights of the chosen experts, and the scores they come from; zeros where there is no choice."""
    got = ids >= 0
    ls = np.where(got, np.take_along_axis(_log_share(z, c["score"]), np.maximum(ids, 0), 1), -np.inf)
    share = np.where(got, np.exp(ls), 0.0)
    w = share
    if c["renorm"]:
        m = np.where(got.any(1, keepdims=True), ls.max(1, keepdims=True), 0.0)
        e = np.exp(ls - m)
        w = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    return share, w


def _exact_route(c, s):
    z = s["logits"].double().cpu().numpy()
    low = torch.finfo(s["logits"].dtype).min
    T, E = z.shape
    value = z
    if c["bias"] or c["groups"] > 1:
        with np.errstate(over="ignore", invalid="ignore"):
            if c["score"] == "sigmoid":
                value = 1.0 / (1.0 + np.exp(-z))
            else:
                e = np.exp(z - np.maximum(z.max(1, keepdims=True), low))
                value = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    if c["bias"]:
        value = value + s["bias"].double().cpu().numpy()
    value = np.where(z > low, value, -np.inf)
    if c["groups"] > 1:
        g = -np.sort(-value.reshape(T, c["groups"], -1), axis=2)
        best = g[:, :, 0].copy()
        if c["pair"] and g.shape[2] > 1:
            best += np.where(np.isinf(g[:, :, 1]), 0.0, g[:, :, 1])
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
        value = np.where(np.repeat(rank < c["kept"], E // c["groups"], axis=1), value, -np.inf)
    ids = np.argsort(-value, axis=1, kind="stable")[:, : c["k"]]
    ids = np.where(np.take_along_axis(value, ids, 1) > -np.inf, ids, -1)
    return {"ids": ids.astype(np.int32), "weights": _exact_weights(c, z, ids)[1] * c["scale"]}


def _exact_route_backward(c, s):
    z, ids = s["logits"].double().cpu().numpy(), s["ids"].cpu().numpy().astype(np.int64)
    g = np.where(ids >= 0, s["dweights"].double().cpu().numpy() * c["scale"], 0.0)
    share, p = _exact_weights(c, z, ids)
    at = np.maximum(ids, 0)
    zs = np.take_along_axis(z, at, 1)
    with np.errstate(over="ignore"):
        other = 1.0 / (1.0 + np.exp(zs)) if c["score"] == "sigmoid" else np.ones_like(zs)
    d = np.zeros_like(z)
    t = np.arange(z.shape[0])[:, None]
    if c["renorm"]:
        np.add.at(d, (t, at), np.where(ids >= 0, other * p * (g - (p * g).sum(1, keepdims=True)), 0.0))
    elif c["score"] == "sigmoid":
        np.add.at(d, (t, at), np.where(ids >= 0, g * share * other, 0.0))
    else:
        np.add.at(d, (t, at), g)
        live = np.isfinite(z.max(1, keepdims=True))
        d = np.where(live, np.exp(np.where(live, _log_share(z, "softmax"), 0.0)) * (d - (share * g).sum(1, keepdims=True)), 0.0)
    return d


def _exact_dispatch(c, s):
    ids = s["ids"].cpu().numpy().reshape(-1)
    rows = np.full(ids.size, -1, dtype=np.int32)
    live = np.nonzero(ids >= 0)[0]
    order = live[np.lexsort((live, ids[live]))]
    rows[order] = np.arange(order.size)
    xs = torch.zeros((ids.size, c["C"]), dtype=torch.float64, device="cuda")
    xs[: order.size] = s["x"].double()[torch.from_numpy(order // c["k"]).cuda()]
    return {"xs": xs, "rows": rows.reshape(c["T"], c["k"]), "offsets": np.searchsorted(np.sort(ids[live]), np.arange(c["E"] + 1)).astype(np.int32)}


def _exact_combine(c, s):
    out = torch.zeros((c["T"], c["C"]), dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
    for j in range(c["k"]):
        r = s["rows"][:, j].long()
        live = torch.nonzero(r >= 0).view(-1)
        w = 1.0 if s["weights"] is None else s["weights"][live, j].double().view(-1, 1)
        out[live] += w * s["y"][r[live]].double()
    return out


def _exact_combine_backward(c, s):
    dy = torch.zeros((c["T"] * c["k"], c["C"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((c["T"], c["k"]), dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        r = s["rows"][:, j].long()
        live = torch.nonzero(r >= 0).view(-1)
        d = s["dout"][live].double()
        dy[r[live]] = d * s["weights"][live, j].double().view(-1, 1)
        dw[live, j] = (d * s["y"][r[live]].double()).sum(1)
    return {"dy": dy, "dweights": dw}


def _exact_gemv(c, s):
    N, K = c["N"], c["K"]
    magnitude = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    n, j = torch.arange(N, device="cuda").view(-1, 1), torch.arange(K // 16, device="cuda").view(1, -1)
    place = ((n // 128) * (K // 64) + j // 4) * 512 + (n % 32) * 16 + ((n // 32) % 4) * 4 + j % 4
    codes, scales = s["W"].view(-1, N, K // 2), s["sW"].view(-1, N * K // 16)
    pairs = torch.arange(c["T"] * c["k"], device="cuda")
    ids = torch.zeros_like(pairs) if c["dense"] else s["ids"].view(-1).long()
    y = torch.zeros((len(pairs), N), dtype=torch.float64, device="cuda")
    for e in range(codes.shape[0]):
        mine = torch.nonzero(ids == e).view(-1)
        if len(mine) == 0:
            continue
        low, high = (codes[e] & 15).int(), (codes[e] >> 4).int()
        q = torch.stack([magnitude[v & 7] * (1.0 - 2.0 * (v >> 3)) for v in (low, high)], -1).view(N, K // 16, 16)
        w = (q * scales[e][place].view(torch.float8_e4m3fn).double().unsqueeze(-1)).view(N, K)
        y[mine] = s["x"][mine // c["k"] if c["shared"] else mine].double() @ w.t() * s["alphaW"][e].double()
    return y


_EXACT = {"route": _exact_route, "route_backward": _exact_route_backward, "dispatch": _exact_dispatch, "combine": _exact_combine,
          "combine_backward": _exact_combine_backward, "gemv": _exact_gemv}


def exact(case, seed):
    return _EXACT[case["op"]](dict(case), prepare(case, seed))
