"""The ragged operators beside the NVFP4 linear layer, as cases to be timed and compared.

Five operators: quantizing rows that are sorted by expert (and reading them back), the products of such rows with
their expert's weight, the experts' weight gradients, and many requests' low-rank adapters beside a shared
projection, forward and backward.  ``run`` computes them in their plain form (elementary torch operations in 32
bits), or, where ``own`` is true, makes the library's calls.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # E2M1 magnitudes
RTN, FOUR_SIX = "rtn", "four_six"


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step's tokens on their way into the experts' up-projection: 8 tokens, two experts each
        dict(name="quantize decode", op="quantize", T=16, C=4096, E=8, empty=2, mode=FOUR_SIX, rht=False, col=False, grad=False),
        # the same layer in training: activations encoded for the forward product and for the weight gradient
        dict(name="quantize activations", op="quantize", T=16384, C=4096, E=8, empty=0, mode=FOUR_SIX, rht=False, col=True, grad=False),
        # output gradients of many small experts, rotated, both orientations; an odd number of rows
        dict(name="quantize gradients", op="quantize", T=16301, C=14336, E=64, empty=3, mode=RTN, rht=True, col=True, grad=True),
        # decode: the experts' weights are read for a few rows
        dict(name="gemm decode", op="gemm", T=16, E=8, empty=2, N=14336, K=4096, fp32=False),
        # a training or prefill layer of eight large experts
        dict(name="gemm prefill", op="gemm", T=16384, E=8, empty=0, N=14336, K=4096, fp32=False),
        # a medium batch over many small experts, fp32 results, ragged everywhere
        dict(name="gemm many experts", op="gemm", T=5003, E=64, empty=5, N=1408, K=2112, fp32=True),
        # weight gradients of eight large experts
        dict(name="wgrad", op="wgrad", T=16384, E=8, empty=0, M=14336, N=4096, fp32=True),
        # weight gradients of many small experts, some of which saw no token
        dict(name="wgrad many experts", op="wgrad", T=4001, E=64, empty=7, M=1408, N=2048, fp32=False),
        # a decode step: one token of each of 64 requests, 32 adapters between them
        dict(name="adapters decode", op="lora", T=64, K=4096, N=14336, r=16, n=32, none=4, runs=False),
        # a prefill batch of a few requests of uneven length
        dict(name="adapters prefill", op="lora", T=8192, K=4096, N=14336, r=16, n=6, none=1, runs=True),
        # training several adapters on one batch
        dict(name="adapters backward", op="lora_backward", T=8192, K=4096, N=14336, r=16, n=4, none=1, runs=True),
        # a short odd batch with a larger rank
        dict(name="adapters backward odd", op="lora_backward", T=517, K=1000, N=2056, r=40, n=5, none=1, runs=True),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))

    op = rng.choice(["quantize", "gemm", "wgrad", "lora", "lora_backward"])
    if op in ("lora", "lora_backward"):
        runs = op == "lora_backward" or rng.random() < 0.5
        n = size(1, 8) if runs else size(1, 64)
        return dict(op=op, T=size(1, 8192) if runs else size(1, 256), K=size(64, 4096, 8), N=size(64, 14336, 8),
                    r=size(8, 128, 8), n=n, none=rng.choice([0, 1]) if n > 1 else 0, runs=runs)
    E = size(1, 64)
    T = size(1, 16384)
    empty = max(E - T, rng.randrange(0, E // 4 + 1))
    if op == "quantize":
        col = rng.random() < 0.6
        return dict(op=op, T=T, C=size(128, 14336, 128 if col else 64), E=E, empty=empty, mode=rng.choice([RTN, FOUR_SIX]),
                    rht=rng.random() < 0.4, col=col, grad=rng.random() < 0.5)
    big = size(128, 14336, 128)
    most = max(128, min(4096, 8 * 14336 * 4096 // (E * big) // 128 * 128))
    if op == "gemm":
        return dict(op=op, T=T, E=E, empty=empty, N=big, K=size(64, most, 64), fp32=rng.random() < 0.3)
    return dict(op=op, T=T, E=E, empty=empty, M=big, N=size(128, most, 128), fp32=rng.random() < 0.6)


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["T"] * c["C"]
        both = 2 if c["col"] else 1
        return {"bytes": 2 * n + both * 2 * n, "flops": both * n * (64 if c["mode"] == FOUR_SIX else 24)}
    if c["op"] == "gemm":
        used = c["E"] - c["empty"]
        return {"bytes": int(0.5625 * c["K"] * (c["T"] + used * c["N"])) + c["T"] * c["N"] * (4 if c["fp32"] else 2),
                "flops": 2 * c["T"] * c["N"] * c["K"]}
    if c["op"] == "wgrad":
        return {"bytes": int(0.5625 * c["T"] * (c["M"] + c["N"])) + c["E"] * c["M"] * c["N"] * (4 if c["fp32"] else 2),
                "flops": 2 * c["T"] * c["M"] * c["N"]}
    used = min(c["n"], c["T"])
    weights = used * c["r"] * (c["K"] + c["N"])
    T, K, N, r = c["T"], c["K"], c["N"], c["r"]
    if c["op"] == "lora":
        return {"bytes": 2 * weights + 2 * T * (K + 2 * N) + 4 * T * r, "flops": 2 * T * r * (K + N)}
    return {"bytes": 2 * weights + 4 * c["n"] * r * (K + N) + 2 * T * (N + 3 * K) + 4 * T * r, "flops": 4 * T * r * (K + N)}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _counts(case, host):
    """Rows of each expert: `empty` experts get none, the others share T rows unevenly."""
    E, T = case["E"], case["T"]
    used = torch.randperm(E, generator=host)[: E - case["empty"]]
    p = torch.softmax(0.7 * torch.randn(len(used), generator=host), 0)
    counts = torch.zeros(E, dtype=torch.int64)
    counts[used] = 1
    if T > len(used):
        counts += torch.bincount(used[torch.multinomial(p, T - len(used), replacement=True, generator=host)], minlength=E)
    return counts.tolist()


def _starts(counts, step=1):
    out = [0]
    for c in counts:
        out.append(out[-1] + -(-c // step) * step)
    return out


def _capacity(T, E, step):
    """The most rows that E ragged groups of T rows in all take up, each padded to a multiple of `step`."""
    return (T + min(T, E) * (step - 1)) // step * step


def _rows(T, C, grad, gen):
    if grad:   # heavy-tailed small values, a few tokens with much larger ones
        u = torch.rand((T, C), generator=gen, device="cuda") - 0.5
        v = torch.sign(u) * torch.log1p(-2 * u.abs()).clamp_(min=-20) * -1e-4
        v[torch.rand((T, 1), generator=gen, device="cuda").expand(T, C) < 0.001] *= 50
        return v.bfloat16()
    v = torch.randn((T, C), generator=gen, device="cuda")
    v[:, torch.randint(0, C, (max(1, C // 1000),), generator=gen, device="cuda")] *= 50   # outlier channels
    return v.bfloat16()


def _operand(x, alpha_rows, mode=RTN):
    """Packed codes [R, C/2] and scales in the GEMM layout of rows x (R a multiple of 128), in slices of rows."""
    R, C = x.shape
    step = max(128, (1 << 26) // C // 128 * 128)
    codes, scales = [], []
    for i in range(0, R, step):
        q, sign, delta = _encode(x[i:i + step].float().view(-1, C // 16, 16), alpha_rows[i:i + step], mode)
        nib = (q | (sign << 3)).view(-1, C // 2, 2)
        codes.append(nib[..., 0] | (nib[..., 1] << 4))
        s = delta.to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 4, 32, C // 64, 4)
        scales.append(s.permute(0, 3, 2, 1, 4).reshape(-1))
    return torch.cat(codes), torch.cat(scales)


def _group_alpha(x, counts):
    a = torch.stack([x[s:e].abs().amax().float() if e > s else x.new_zeros((), dtype=torch.float32)
                     for s, e in zip(_starts(counts), _starts(counts)[1:])])
    return a / torch.full_like(a, 2688.0)


def _padded(x, counts, step):
    """x's rows with each group moved to a multiple of `step` rows; zero rows fill the gaps, up to the capacity."""
    out = x.new_zeros((_capacity(x.shape[0], len(counts), step), x.shape[1]))
    out[_places(counts, step).to(x.device)] = x
    return out


def _places(counts, step):
    shift = torch.tensor([p - s for p, s in zip(_starts(counts, step), _starts(counts))][: len(counts)])
    return torch.arange(sum(counts)) + torch.repeat_interleave(shift, torch.tensor(counts))


def _spread(alpha, counts, step):
    """alpha of each row's group, for rows padded to `step` (rows behind the last group get the last group's)."""
    padded = torch.tensor([-(-c // step) * step for c in counts], device=alpha.device)
    a = torch.repeat_interleave(alpha, padded)
    more = _capacity(sum(counts), len(counts), step) - a.shape[0]
    return torch.cat([a, alpha[-1:].expand(more)]).view(-1, 1)


def _row_operand(x, counts):
    """A ragged row operand: dense codes [T, C/2], scales of the 128-row padded groups, one alpha per group."""
    alpha = _group_alpha(x, counts)
    codes, scales = _operand(_padded(x, counts, 128), _spread(alpha, counts, 128))
    return codes[_places(counts, 128).cuda()].contiguous(), scales, alpha


def _col_operand(x, counts):
    """A ragged column operand: codes [C, cap/2] and scales of the transpose, groups padded to 64 rows."""
    alpha = _group_alpha(x, counts)
    xp = _padded(x, counts, 64)
    per_col = _spread(alpha, counts, 64).view(-1, 16)[:, :1]   # one alpha per 16-row block
    R, cap = x.shape[1], xp.shape[0]
    codes = torch.empty((R, cap // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty(R * (cap // 16), dtype=torch.uint8, device="cuda")
    step = max(128, (1 << 26) // cap // 128 * 128)
    for i in range(0, R, step):
        blocks = xp[:, i:i + step].t().float().reshape(-1, cap // 16, 16)
        q, sign, delta = _encode(blocks, per_col.view(1, -1), RTN)
        nib = (q | (sign << 3)).view(-1, cap // 2, 2)
        codes[i:i + step] = nib[..., 0] | (nib[..., 1] << 4)
        s = delta.to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 4, 32, cap // 64, 4)
        scales[i * (cap // 16):(i + blocks.shape[0]) * (cap // 16)] = s.permute(0, 3, 2, 1, 4).reshape(-1)
    return codes, scales, alpha


def _weights(E, N, K, gen):
    """The experts' weights [E, N, K], quantized one tensor scale each."""
    codes, scales, alpha = [], [], []
    for _ in range(E):
        w = (torch.randn((N, K), generator=gen, device="cuda") * 0.02).bfloat16()
        a = w.abs().amax().float().view(1)
        a = a / torch.full_like(a, 2688.0)
        c, s = _operand(w, a.expand(N, 1))
        codes.append(c)
        scales.append(s)
        alpha.append(a)
    return torch.stack(codes), torch.stack(scales), torch.cat(alpha)


def _requests(case, host):
    """Adapter of each token (-1: none): runs of uneven length in any order, or one request per token."""
    T, n = case["T"], case["n"]
    if not case["runs"]:
        ids = torch.randint(0, n, (T,), generator=host)
        ids[torch.randperm(T, generator=host)[: min(case["none"], T - 1)]] = -1
        return ids
    kinds = torch.cat([torch.arange(n), torch.randint(0, n, (2,), generator=host), torch.full((case["none"],), -1)])
    kinds = kinds[torch.randperm(len(kinds), generator=host)]
    cuts = torch.sort(torch.randint(0, T + 1, (len(kinds) - 1,), generator=host)).values.tolist()
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    return torch.repeat_interleave(kinds, torch.tensor(lengths))


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    c = dict(case)
    state = {"case": c}
    if c["op"] in ("lora", "lora_backward"):
        T, K, N, r, n = c["T"], c["K"], c["N"], c["r"], c["n"]
        ids = _requests(c, host)
        # the plan of the plain form: the tokens of each adapter, padded with T (a row that is dropped)
        most = max(1, int(torch.bincount(ids[ids >= 0], minlength=1).max()))
        place = torch.full((n, most), T, dtype=torch.int64)
        for a in range(n):
            at = torch.nonzero(ids == a).view(-1)
            place[a, : len(at)] = at
        state.update(ids=ids.to(torch.int32).cuda(), place=place.cuda(),
                     x=_rows(T, K, False, gen),
                     A=(torch.randn((n, r, K), generator=gen, device="cuda") / math.sqrt(K)).bfloat16(),
                     B=(torch.randn((n, N, r), generator=gen, device="cuda") * 0.05).bfloat16(),
                     scaling=0.5 + torch.rand(n, generator=gen, device="cuda") * 2)
        if c["op"] == "lora":
            state["y"] = torch.randn((T, N), generator=gen, device="cuda").bfloat16()
        else:
            state["dy"] = _rows(T, N, True, gen)
            state["dx"] = (torch.randn((T, K), generator=gen, device="cuda") * 1e-4).bfloat16()
            state["h"] = _shrink(state)
        return state
    counts = _counts(c, host)
    state["counts"] = counts
    state["offsets"] = torch.tensor(_starts(counts), dtype=torch.int32).cuda()
    if c["op"] == "quantize":
        state["x"] = _rows(c["T"], c["C"], c["grad"], gen)
        state["seed"] = seed * 7919 + 1
    elif c["op"] == "gemm":
        state["A"], state["sA"], state["alphaA"] = _row_operand(_rows(c["T"], c["K"], False, gen), counts)
        state["B"], state["sB"], state["alphaB"] = _weights(c["E"], c["N"], c["K"], gen)
    else:
        state["A"], state["sA"], state["alphaA"] = _col_operand(_rows(c["T"], c["M"], True, gen), counts)
        state["B"], state["sB"], state["alphaB"] = _col_operand(_rows(c["T"], c["N"], False, gen), counts)
    return state


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _signs(seed):
    """The rotation's 16 signs: the low word of one Philox4x32-10 draw, counter (0, 0, 0, 3), key = seed."""
    x, k = [0, 0, 0, 3], [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF]
    for _ in range(10):
        a, b = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
        x = [(b >> 32) ^ x[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ x[3] ^ k[1], a & 0xFFFFFFFF]
        k = [k[0] + 0x9E3779B9 & 0xFFFFFFFF, k[1] + 0xBB67AE85 & 0xFFFFFFFF]
    return [-1.0 if x[0] >> i & 1 else 1.0 for i in range(16)]


def _rotate(v, seed):
    """(1/4) H16 D of the last axis, butterflies in the order 1, 2, 4, 8."""
    v = v * torch.tensor(_signs(seed), device=v.device)
    for h in (1, 2, 4, 8):
        p = v.view(*v.shape[:-1], 8 // h, 2, h)
        v = torch.stack([p[..., 0, :] + p[..., 1, :], p[..., 0, :] - p[..., 1, :]], -2).reshape(v.shape)
    return v * 0.25


def _nearest(a):
    """Index of the E2M1 magnitude nearest to a >= 0, ties to the even code, saturating."""
    i = (a > 0.25).to(torch.uint8)
    for edge, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (a >= edge) if tie_up else (a > edge)
    return i


def _candidate(v, amax, alpha, top):
    den = alpha * top
    delta = torch.where(den == 0, 0.0, amax / den).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    s = alpha * delta
    r = torch.where(s == 0, 0.0, 1.0 / s)
    r = torch.where(torch.isinf(r), 0.0, r).unsqueeze(-1)
    q = _nearest((v * r).abs_())
    return q, delta, s


def _decoded(q, v, s):
    g = torch.tensor(GRID, device=v.device).index_select(0, q.view(-1).int()).view(q.shape)
    return torch.copysign(g, v) * s.unsqueeze(-1)


def _error(v, q, s):
    e = (v - _decoded(q, v, s)).square_()
    for w in (8, 4, 2, 1):
        e = e[..., :w] + e[..., w:]
    return e.squeeze(-1)


def _encode(v, alpha, mode):
    """Magnitude codes, sign bits and block scales of 16-element blocks v [..., 16] with tensor scale alpha."""
    amax = v.abs().amax(-1)
    q, delta, s = _candidate(v, amax, alpha, 6.0)
    if mode == FOUR_SIX:
        q4, delta4, s4 = _candidate(v, amax, alpha, 4.0)
        better = _error(v, q4, s4) < _error(v, q, s)
        q, delta = torch.where(better.unsqueeze(-1), q4, q), torch.where(better, delta4, delta)
    return q, torch.signbit(v).to(torch.uint8), delta


def _values(blocks, alpha_of, mode):
    q, _, delta = _encode(blocks, alpha_of, mode)
    return _decoded(q, blocks, alpha_of * delta)


def _amax_of_groups(v, group, E):
    """max |v| of the rows of each group (0 where there are none)."""
    return torch.zeros(E, device=v.device).scatter_reduce_(0, group, v.abs().flatten(1).amax(1), "amax")


def _plain_quantize(s):
    c, counts = s["case"], s["counts"]
    E, C = c["E"], c["C"]
    group = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    v = s["x"].float().view(c["T"], C // 16, 16)
    if c["rht"]:
        v = _rotate(v, s["seed"])
    a = _amax_of_groups(v, group, E)
    alpha = a / torch.full_like(a, 2688.0)
    out = {"alpha_row": alpha, "row": _values(v, alpha[group].view(-1, 1), c["mode"]).view(c["T"], C).bfloat16()}
    if c["col"]:
        # blocks of 16 rows of one column, group by group, zero rows behind each group
        places = _places(counts, 16).cuda()
        v = torch.zeros((_capacity(c["T"], E, 16), C), device="cuda")
        v[places] = s["x"].float()
        v = v.view(-1, 16, C).transpose(1, 2).contiguous()
        if c["rht"]:
            v = _rotate(v, s["seed"])
        of_block = torch.zeros(v.shape[0], dtype=torch.int64, device="cuda")
        of_block[places // 16] = group
        a = _amax_of_groups(v, of_block, E)
        alpha = a / torch.full_like(a, 2688.0)
        y = _values(v, alpha[of_block].view(-1, 1), c["mode"]).transpose(1, 2).reshape(-1, C)[places]
        out.update(alpha_col=alpha, col=y.bfloat16())
    return out


def _read(codes, scales):
    """q * Delta of packed codes [R, K/2] with scales in the GEMM layout (R a multiple of 128), exact in fp32."""
    R, K = codes.shape[0], codes.shape[1] * 2
    nib = torch.stack([codes & 15, codes >> 4], -1).view(-1).int()
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    delta = scales.view(R // 128, K // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, K // 16)
    return (grid.index_select(0, nib).view(R, K // 16, 16) * delta.view(torch.float8_e4m3fn).float().unsqueeze(-1)).view(R, K)


def _plain_gemm(s):
    c, counts = s["case"], s["counts"]
    places = _places(counts, 128).cuda()
    rows = torch.zeros((_capacity(c["T"], c["E"], 128), c["K"] // 2), dtype=torch.uint8, device="cuda")
    rows[places] = s["A"]
    a = _read(rows, s["sA"])[places]
    ab = s["alphaA"] * s["alphaB"]
    # one product per expert that has rows: a padded batch would multiply rows that are not there
    at = _starts(counts)
    d = [a[i:j] @ _read(s["B"][e], s["sB"][e]).t() * ab[e] for e, (i, j) in enumerate(zip(at, at[1:])) if j > i]
    d = torch.cat(d)
    return d if c["fp32"] else d.bfloat16()


def _plain_wgrad(s):
    c, counts = s["case"], s["counts"]
    a, b = _read(s["A"], s["sA"]), _read(s["B"], s["sB"])
    ab = s["alphaA"] * s["alphaB"]
    at = _starts(counts, 64)
    d = torch.stack([a[:, i:j] @ b[:, i:j].t() * ab[e] for e, (i, j) in enumerate(zip(at, at[1:]))])
    return d if c["fp32"] else d.bfloat16()


def _taken(t, place):
    """Rows of t for each adapter, [n, most, width]; place holds len(t) where there is none, which reads zeros."""
    return torch.cat([t.float(), t.new_zeros((1, t.shape[1]), dtype=torch.float32)])[place]


def _put(base, place, rows):
    out = torch.cat([base, base.new_zeros((1, base.shape[1]))])
    out[place.view(-1)] = rows.view(-1, rows.shape[-1])
    return out[:-1]


def _shrink(s):
    h = _taken(s["x"], s["place"]) @ s["A"].float().transpose(1, 2)
    return _put(h.new_zeros((s["x"].shape[0], h.shape[-1])), s["place"], h)


def _plain_lora(s):
    place = s["place"]
    h = _taken(s["x"], place) @ s["A"].float().transpose(1, 2)
    d = h @ s["B"].float().transpose(1, 2) * s["scaling"].view(-1, 1, 1)
    out = _put(s["y"].float(), place, _taken(s["y"], place) + d).bfloat16()
    return {"out": out, "h": _put(h.new_zeros((out.shape[0], h.shape[-1])), place, h)}


def _plain_lora_backward(s):
    place, by = s["place"], s["scaling"].view(-1, 1, 1)
    dy, x = _taken(s["dy"], place), _taken(s["x"], place)
    g = dy @ s["B"].float()
    dx = _put(s["dx"].float(), place, _taken(s["dx"], place) + g @ s["A"].float() * by).bfloat16()
    dA = g.transpose(1, 2) @ x * by
    dB = dy.transpose(1, 2) @ _taken(s["h"], place) * by
    return {"dx": dx, "dA": dA, "dB": dB}


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "wgrad": _plain_wgrad, "lora": _plain_lora,
            "lora_backward": _plain_lora_backward}[c["op"]](state)


def _own(s):
    from nvfp4_block_quantization_amax_b200 import api
    c = s["case"]
    if c["op"] == "quantize":
        mode = api.NVFP4_FOUR_SIX if c["mode"] == FOUR_SIX else api.NVFP4_RTN
        flags = api.NVFP4_ROWWISE | (api.NVFP4_COLWISE if c["col"] else 0) | (api.NVFP4_RHT if c["rht"] else 0)
        q = api.nvfp4_quantize_grouped(s["x"], s["offsets"], mode, flags, seed=s["seed"])
        out = {"alpha_row": q.alpha_row,
               "row": api.nvfp4_dequantize_grouped(q.codes_row, q.scales_row, q.alpha_row, s["offsets"], c["T"], c["C"],
                                                   api.NVFP4_ROWWISE | api.NVFP4_OUT_BF16)}
        if c["col"]:
            out["alpha_col"] = q.alpha_col
            out["col"] = api.nvfp4_dequantize_grouped(q.codes_col, q.scales_col, q.alpha_col, s["offsets"], c["T"], c["C"],
                                                      api.NVFP4_COLWISE | api.NVFP4_OUT_BF16)
        return out
    if c["op"] in ("gemm", "wgrad"):
        kind = api.NVFP4_OUT_DTYPE_FP32 if c["fp32"] else api.NVFP4_OUT_DTYPE_BF16
        if c["op"] == "gemm":
            return api.nvfp4_gemm_grouped(s["A"], s["sA"], s["alphaA"], s["B"], s["sB"], s["alphaB"], s["offsets"],
                                          out_dtype=kind)
        return api.nvfp4_gemm_grouped_wgrad(s["A"], s["sA"], s["alphaA"], s["B"], s["sB"], s["alphaB"], s["offsets"],
                                            c["T"], out_dtype=kind)
    if c["op"] == "lora":
        out, h = api.nvfp4_lora_apply(s["x"], s["A"], s["B"], s["scaling"], s["ids"], y=s["y"])
        return {"out": out, "h": h}
    dx, dA, dB = api.nvfp4_lora_backward(s["dy"], s["x"], s["h"], s["A"], s["B"], s["scaling"], s["ids"], dx=s["dx"],
                                         out_dtype=api.NVFP4_OUT_DTYPE_FP32)
    return {"dx": dx, "dA": dA, "dB": dB}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _f32(v):
    """Round to 32 bits where the format's definition rounds (scales and scaled values are binary32 numbers)."""
    return v.float().double()


def _to_e4m3(v):
    """v >= 0 rounded to the nearest E4M3 value, ties to even, at most 448."""
    e = torch.floor(torch.log2(v.clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _to_e2m1(a):
    grid = torch.tensor(GRID, dtype=torch.float64, device=a.device)
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.searchsorted(mid, a.contiguous()), torch.searchsorted(mid, a.contiguous(), right=True)
    return grid[torch.where(low % 2 == 0, low, high)]


def _exact_blocks(v, alpha, mode):
    """Values that blocks v [n, 16] stand for once encoded, alpha [n, 1]."""
    best = None
    for top in (6.0, 4.0) if mode == FOUR_SIX else (6.0,):
        den = _f32(alpha * top)
        delta = _to_e4m3(torch.where(den > 0, _f32(v.abs().amax(1, keepdim=True) / den), 0.0))
        s = _f32(alpha * delta)
        r = _f32(1 / s)
        r = torch.where((s == 0) | torch.isinf(r), 0.0, r)
        y = torch.sign(v) * _to_e2m1(_f32(v * r).abs()) * s
        if mode != FOUR_SIX:
            return y
        d = _f32(v - _f32(y))
        e = _f32(d * d)
        for w in (8, 4, 2, 1):
            e = _f32(e[:, :w] + e[:, w:])
        best = (y, e) if best is None else (torch.where(e < best[1], y, best[0]), None)
    return best[0]


def _hadamard(seed):
    i = torch.arange(16)
    bits = sum(((i.view(-1, 1) & i) >> b) & 1 for b in range(4))
    return (torch.where(bits % 2 == 0, 0.25, -0.25).double() * torch.tensor(_signs(seed)).double()).cuda()


def _exact_quantize(s):
    c, at = s["case"], _starts(s["counts"])
    out = {}
    turn = _hadamard(s["seed"]) if c["rht"] else None
    for side in ("row", "col") if c["col"] else ("row",):
        alphas, parts = [], []
        for i, j in zip(at, at[1:]):
            x = s["x"][i:j].double()
            if side == "col":
                x = torch.nn.functional.pad(x, (0, 0, 0, -(j - i) % 16)).t().contiguous()
            v = x.view(-1, 16)
            if turn is not None and len(v):
                v = v @ turn.t()
                # sums of 16 bf16 values: every partial sum of the definition's butterflies is rounded to 32 bits,
                # which differs from the exact sum only where the values span more than 16 bits
                w = x.view(-1, 16) * torch.tensor(_signs(s["seed"]), device="cuda").double()
                for h in (1, 2, 4, 8):
                    k = torch.arange(16, device="cuda")
                    w = _f32(torch.where(k & h == 0, w[:, k] + w[:, k ^ h], w[:, k ^ h] - w[:, k]))
                v = w / 4
            a = _f32((v.abs().max() if v.numel() else x.new_zeros(())) / 2688)
            alphas.append(a)
            y = _exact_blocks(v, a.view(1, 1), c["mode"]).view(x.shape) if len(v) else x
            parts.append(y if side == "row" else y.t()[: j - i])
        out["alpha_" + side] = torch.stack(alphas)
        out[side] = torch.cat(parts)
    return out


def _exact_operand(codes, scales, rows):
    """q * Delta of the given rows of an operand in 64 bits; scales are found by their place in the GEMM layout."""
    K = codes.shape[1] * 2
    byte = codes[:, torch.arange(K, device="cuda") // 2]
    nib = torch.where(torch.arange(K, device="cuda") % 2 == 0, byte & 15, byte >> 4).long()
    mag, exp = nib & 1, (nib >> 1) & 3
    q = torch.where(exp == 0, mag * 0.5, (1 + mag * 0.5) * torch.exp2(exp.double() - 1)) * torch.where(nib > 7, -1.0, 1.0).double()
    m, j = rows.view(-1, 1), torch.arange(K // 16, device="cuda").view(1, -1)
    b = scales[((m // 128) * (K // 64) + j // 4) * 512 + (m % 32) * 16 + (m // 32 % 4) * 4 + j % 4].long()
    e, f = b >> 3, (b & 7).double()
    delta = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2(e.double() - 7))
    return q * delta.repeat_interleave(16, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        return _exact_quantize(s)
    if c["op"] == "gemm":
        out, at, pad = [], _starts(s["counts"]), _starts(s["counts"], 128)
        n = torch.arange(c["N"], device="cuda")
        for e in range(c["E"]):
            if at[e + 1] > at[e]:
                rows = torch.arange(at[e + 1] - at[e], device="cuda") + pad[e]
                a = _exact_operand(s["A"][at[e]:at[e + 1]], s["sA"], rows)
                out.append(a @ _exact_operand(s["B"][e], s["sB"][e], n).t() * (s["alphaA"][e].double() * s["alphaB"][e].double()))
        return torch.cat(out)
    if c["op"] == "wgrad":
        pad = _starts(s["counts"], 64)
        a = _exact_operand(s["A"], s["sA"], torch.arange(c["M"], device="cuda"))
        b = _exact_operand(s["B"], s["sB"], torch.arange(c["N"], device="cuda"))
        out = torch.empty((c["E"], c["M"], c["N"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            torch.matmul(a[:, pad[e]:pad[e + 1]], b[:, pad[e]:pad[e + 1]].t(), out=out[e])
            out[e] *= s["alphaA"][e].double() * s["alphaB"][e].double()
        return out
    ids, x = s["ids"].long(), s["x"].double()
    h = torch.zeros((c["T"], c["r"]), dtype=torch.float64, device="cuda")
    if c["op"] == "lora":
        out = s["y"].double()
        for a in range(c["n"]):
            t = torch.nonzero(ids == a).view(-1)
            h[t] = x[t] @ s["A"][a].double().t()
            out[t] += s["scaling"][a].double() * (h[t] @ s["B"][a].double().t())
        return {"out": out, "h": h}
    dx, dA, dB, dy = s["dx"].double(), [], [], s["dy"].double()
    for a in range(c["n"]):
        t, by = torch.nonzero(ids == a).view(-1), s["scaling"][a].double()
        g = by * (dy[t] @ s["B"][a].double())
        dx[t] += g @ s["A"][a].double()
        dA.append(g.t() @ x[t])
        dB.append(by * (dy[t].t() @ s["h"][t].double()))
    return {"dx": dx, "dA": torch.stack(dA), "dB": torch.stack(dB)}
