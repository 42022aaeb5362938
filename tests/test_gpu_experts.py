"""Routing, dispatch, combine and the few-row products against plain 64-bit
forms.

Tolerances.  U = 2^-24 is half a step of fp32 (relative).
  route: expf is off by at most 2 steps (4 U), 1 + e, the division, the product
    with the scale by U each; a softmax's exponent z - max is rounded (|z - max|
    U), and its row sum uses ex2.approx (2^-22 = 4 U and the rounded exponent's
    |z - max| 2^-23.5 < 2 |z - max| U, whose mean over a softmax is at most
    ln E) and E / 32 + 5 additions.  share(): (d + 16 + 2 ln E + E / 32) U with
    d = |z - max|; a renormalised weight is a quotient of a share and a sum of
    at most k shares, added in 5 steps: (2 max (d + 16) + 12) U.
  route backward: products of such factors; the differences g - <p, g> are off by
    their magnitudes |g| + sum |p g| times those errors and 8 U.
  combine: k + 1 fused multiply-adds, U of the sum of magnitudes each, then half
    a step of bf16, 2^-8.
  combine backward: dy is exactly bf16(fp32(w dout)); dw sums C products.
  gemv: products are exact; K additions that may truncate (2 U each), 8 warps'
    sums and two factors: (2 K + 32) U of the sum of magnitudes.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = torch.finfo(torch.bfloat16).eps / 2
INF = math.inf
SOFTMAX, SIGMOID, RENORM, PAIR = 0, 1, 1, 2


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_quantization_amax_b200 import api as _api
    return _api


def within(got, ref, bound, what):
    over = (got.double().cpu() - ref).abs() - bound
    assert bool((over <= 0).all()), f"{what}: {float(over.max()):.3g} over the bound"


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def scores(z, score):
    if score == SIGMOID:
        return 1 / (1 + torch.exp(-z))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == -INF, 0.0, m))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300)


def route_reference(z, k, score, flags, bias, groups, kept, scale):
    """Experts and weights token by token, in 64 bits."""
    low = torch.finfo(z.dtype).min
    z64 = z.double().cpu()
    T, E = z64.shape
    s = scores(z64, score)
    value = z64 if bias is None and groups == 1 else s if bias is None else s + bias.double().cpu()
    open_ = z64 > low
    if bias is not None:
        open_ &= bias.cpu() > torch.finfo(torch.float32).min
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    n = E // groups
    for t in range(T):
        v = [float(value[t, e]) if open_[t, e] else -INF for e in range(E)]
        if groups > 1:
            of = []
            for g in range(groups):
                two = sorted(v[g * n:(g + 1) * n], reverse=True)[:2]
                of.append(two[0] + two[1] if flags & PAIR and len(two) == 2 and two[1] > -INF else two[0])
            best = sorted(range(groups), key=lambda g: (-of[g], g))[:kept]
            v = [v[e] if e // n in best else -INF for e in range(E)]
        order = [e for e in sorted(range(E), key=lambda e: (-v[e], e)) if v[e] > -INF][:k]
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
        if order:
            if flags & RENORM:
                zs = z64[t, order]
                ls = -torch.logaddexp(torch.zeros_like(zs), -zs) if score == SIGMOID else zs
                w[t, :len(order)] = torch.softmax(ls, 0) * scale
            else:
                w[t, :len(order)] = s[t, order] * scale
    return ids, w


def share_error(z64, ids, score, flags):
    """Relative error of each weight, by the figures above."""
    E = z64.shape[1]
    fin = torch.where(torch.isfinite(z64), z64, torch.full_like(z64, -1e30))
    at = ids.clamp(min=0).long()
    zs = fin.gather(1, at)
    top = torch.where(ids >= 0, zs, torch.full_like(zs, -1e30)).amax(1, keepdim=True) if flags & RENORM else fin.amax(1, keepdim=True)
    d = (top - zs).abs() if score == SOFTMAX or flags & RENORM else torch.zeros_like(zs)
    d = torch.where(ids >= 0, d, 0.0)
    if flags & RENORM:
        return (2 * (d.amax(1, keepdim=True) + 16) + 12) * U
    return (d + 16 + (2 * math.log(E) + E / 32 if score == SOFTMAX else 0)) * U


def logits_of(T, E, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * spread).to(dtype)


def check_route(api, z, k, score, flags, bias=None, groups=1, kept=1, scale=1.0):
    z = z.cuda()
    bias = None if bias is None else bias.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w = api.nvfp4_route(z, k, score, flags, bias=bias, groups=groups, groups_kept=kept, scale=scale, status=status)
    want, w64 = route_reference(z, k, score, flags, bias, groups, kept, scale)
    assert torch.equal(ids.cpu(), want), torch.nonzero((ids.cpu() != want).any(1)).view(-1)[:8]
    within(w, w64, share_error(z.double().cpu(), want, score, flags) * w64.abs() + 2.0 ** -149, "weights")
    assert int(status) == 0
    # the same rows many times over, which may take another kernel
    times = -(-2100 // z.shape[0])
    many, wm = api.nvfp4_route(z.repeat(times, 1), k, score, flags, bias=bias, groups=groups, groups_kept=kept, scale=scale, status=status)
    assert torch.equal(many.cpu(), want.repeat(times, 1)) and int(status) == 0
    within(wm, w64.repeat(times, 1), (share_error(z.double().cpu(), want, score, flags) * w64.abs() + 2.0 ** -149).repeat(times, 1), "weights")
    return ids, w


@pytest.mark.parametrize("T,E,k,groups,kept", [
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 7, 7, 1, 1), (5, 32, 32, 1, 1), (33, 33, 4, 3, 2), (64, 64, 6, 1, 1), (17, 160, 6, 8, 3),
    (40, 256, 8, 8, 4), (9, 100, 10, 4, 2), (130, 128, 5, 32, 7), (6, 512, 22, 1, 1), (4, 1000, 9, 10, 4), (3, 1024, 32, 32, 32),
    (12, 24, 3, 12, 5), (10, 96, 4, 24, 9), (700, 16, 2, 2, 1), (90, 512, 8, 8, 3), (60, 257, 8, 1, 1), (70, 72, 8, 8, 1), (80, 200, 7, 5, 4),
    (50, 500, 3, 4, 4), (64, 40, 8, 8, 2)])
@pytest.mark.parametrize("score,flags", [(SOFTMAX, 0), (SOFTMAX, RENORM | PAIR), (SIGMOID, PAIR), (SIGMOID, RENORM)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_shapes(api, T, E, k, groups, kept, score, flags, dtype):
    z = logits_of(T, E, dtype, seed=T * E + k)
    check_route(api, z, k, score, flags, groups=groups, kept=kept)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.3
    check_route(api, z, k, score, flags, bias=bias, groups=groups, kept=kept, scale=2.5)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_ties_go_to_the_lowest_index(api, score, groups, kept, dtype):
    g = torch.Generator().manual_seed(5)
    z = torch.randint(-2, 3, (200, 64), generator=g).to(dtype) / 2
    z[0] = 0.0
    z[1, ::2] = -0.0
    z[2:4] = 60.0              # sigmoid 1 - 2^-86: 1 in 64 bits
    z[3, 5] = 70.0
    for bias in (None, torch.zeros(64), torch.randint(0, 2, (64,), generator=g).float() / 4):
        for flags in (0, RENORM, PAIR):
            check_route(api, z, 6, score, flags, bias=bias, groups=groups, kept=kept)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("base", [0.0, 7.0, -3.0])
def test_route_orders_values_that_32_bits_cannot(api, score, base):
    """Biases a few steps of 2^-30 apart beside logits whose scores differ by
    as little: only the values in 64 bits tell the experts apart."""
    g = torch.Generator().manual_seed(11)
    z = 1.0 + torch.randint(-40, 40, (300, 96), generator=g).float() * 2.0 ** -23
    bias = base + torch.randint(-3, 4, (96,), generator=g).float() * 2.0 ** -22
    for groups, kept in ((1, 1), (6, 2)):
        check_route(api, z, 8, score, RENORM | PAIR, bias=bias, groups=groups, kept=kept)
    check_route(api, z, 8, score, 0)


@pytest.mark.parametrize("E,k,groups,kept", [(5, 2, 1, 1), (64, 8, 1, 1), (64, 4, 8, 3), (256, 8, 8, 4), (300, 20, 1, 1), (600, 32, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_pairs_that_32_bits_cannot_part(api, E, k, groups, kept, biased):
    """One pair of neighbours in each row, among the choices or at their end,
    whose values are a few 2^-27 apart or equal, in either order."""
    g = torch.Generator().manual_seed(E + k)
    T = 250
    z = torch.argsort(torch.rand((T, E), generator=g), 1).float() * (8.0 / E) - 4.0    # far apart
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    b64 = bias.double() if biased else torch.zeros(E, dtype=torch.float64)
    sig = biased or groups > 1
    c = (1 / (1 + torch.exp(-z.double())) if sig else z.double()) + b64
    order = torch.argsort(c, 1, descending=True)
    for t in range(T):
        r = min(t % (k + 1), E - 2)
        first, second = int(order[t, r]), int(order[t, r + 1])
        target = c[t, first] - b64[second] + (t % 5 - 2) * 2.0 ** -27
        if sig and not 0 < target < 1:
            continue
        z[t, second] = torch.log(target / (1 - target)).float() if sig else z[t, first] * (1 + (t % 5 - 2) * 2.0 ** -23)
    check_route(api, z, k, SIGMOID, RENORM, bias=bias, groups=groups, kept=kept)
    check_route(api, z, k, SOFTMAX, 0, bias=bias, groups=groups, kept=kept)


@pytest.mark.parametrize("score,flags", [(SOFTMAX, 0), (SOFTMAX, RENORM), (SIGMOID, 0), (SIGMOID, RENORM)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_far_logits(api, score, flags, dtype):
    """Scores below the smallest number, and all at once: shares stay shares."""
    z = logits_of(60, 40, dtype, seed=3)
    z[:10] -= 200.0
    z[10:20] *= 40.0
    z[20:30] += 3000.0
    z[30:40] = z[30:40] * 1e36
    check_route(api, z, 5, score, flags)
    check_route(api, z[:20], 5, score, flags, groups=8, kept=3)
    _, w = api.nvfp4_route(z.cuda(), 5, score, flags)
    assert bool(torch.isfinite(w).all())
    if flags & RENORM:
        assert bool(((w.sum(1) - 1).abs() < 1e-5).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,flags", [(SOFTMAX, 0), (SIGMOID, RENORM | PAIR)])
@pytest.mark.parametrize("mask", [-INF, None])
def test_route_masked_experts(api, dtype, score, flags, mask):
    mask = torch.finfo(dtype).min if mask is None else mask
    g = torch.Generator().manual_seed(8)
    z = logits_of(50, 48, dtype, seed=9)
    z[torch.rand((50, 48), generator=g) < 0.7] = mask
    z[0] = mask
    z[1] = mask
    z[1, 47] = -1.0
    z[2, 1:] = mask
    bias = torch.randn(48, generator=g) * 0.2
    for b in (None, bias):
        for groups, kept in ((1, 1), (6, 3)):
            ids, w = check_route(api, z, 8, score, flags, bias=b, groups=groups, kept=kept)
            assert ids[0].tolist() == [-1] * 8 and ids[1].tolist() == [47] + [-1] * 7 and not bool(w[0].any())
    bias[::3] = -INF
    bias[1] = torch.finfo(torch.float32).min
    ids, _ = check_route(api, z, 8, score, flags, bias=bias)
    assert not bool(((ids >= 0) & (ids % 3 == 0)).any())


@pytest.mark.parametrize("bad", [math.nan, INF])
def test_route_nonfinite_rows(api, bad):
    z = logits_of(20, 30, torch.float32, seed=4)
    want = api.nvfp4_route(z.cuda(), 3)
    z[7, 29] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.cat([z, z], 1).repeat(150, 1).cuda()              # 60 experts, 3000 tokens
    ids, w = api.nvfp4_route(wide, 3, status=status)
    rest = torch.arange(3000) % 20 != 7
    assert int(status) == -4 and bool((ids[~rest] == -1).all()) and not bool(w[~rest].any()) and bool((ids[rest] >= 0).all())
    status.zero_()
    ids, w = api.nvfp4_route(z.cuda(), 3, status=status)
    assert int(status) == -4 and ids[7].tolist() == [-1] * 3 and w[7].tolist() == [0.0] * 3
    keep = [t for t in range(20) if t != 7]
    assert torch.equal(ids[keep], want[0][keep]) and torch.equal(w[keep], want[1][keep])
    bias = torch.zeros(30, device="cuda")
    bias[3] = bad
    status.zero_()
    ids, w = api.nvfp4_route(logits_of(20, 30, torch.float32, seed=4).cuda(), 3, bias=bias, status=status)
    assert int(status) == -4 and bool((ids == -1).all()) and not bool(w.any())


def backward_reference(z, ids, dw, score, flags, scale):
    """Gradient and its bound, in 64 bits."""
    z64, dw = z.double().cpu(), dw.double().cpu()
    ids = ids.cpu().long()
    T, E = z64.shape
    got = ids >= 0
    at = ids.clamp(min=0)
    s = scores(z64, score)
    g = torch.where(got, dw * scale, 0.0)
    mine = torch.where(got, s.gather(1, at), 0.0)
    zs = z64.gather(1, at)
    rel = torch.where(got, share_error(z64, ids, score, flags), 0.0).amax(1, keepdim=True) + 16 * U
    other = torch.where(got, 1 / (1 + torch.exp(zs)), 0.0) if score == SIGMOID else got.double()
    zero = torch.zeros_like(z64)
    if flags & RENORM:
        ls = torch.where(got, -torch.logaddexp(torch.zeros_like(zs), -zs) if score == SIGMOID else zs, torch.full_like(zs, -INF))
        p = torch.where(got.any(1, keepdim=True), torch.nan_to_num(torch.softmax(ls, 1)), 0.0)
        inner = g - (p * g).sum(1, keepdim=True)
        mag = g.abs() + (p * g).abs().sum(1, keepdim=True)
        return zero.scatter_add(1, at, other * p * inner), zero.scatter_add(1, at, other * p * mag * 2 * rel)
    if score == SIGMOID:
        v = g * mine * other
        return zero.scatter_add(1, at, v), zero.scatter_add(1, at, v.abs() * 2 * rel)
    d = zero.scatter_add(1, at, g)
    a = zero.scatter_add(1, at, g.abs())
    fin = torch.where(torch.isfinite(z64), z64, torch.full_like(z64, -1e30))
    far = (fin.amax(1, keepdim=True) - fin).clamp(max=200.0)
    rel = (3 * far + 40 + 2 * math.log(E) + E / 32) * U
    dot, mag = (mine * g).sum(1, keepdim=True), (mine * g).abs().sum(1, keepdim=True)
    live = got.any(1, keepdim=True)
    return torch.where(live, s * (d - dot), 0.0), torch.where(live, s * (a + mag) * (rel + rel.amax(1, keepdim=True)), 0.0)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 33, 4), (64, 64, 6), (17, 160, 6), (40, 256, 8), (7, 1000, 32), (301, 16, 3)])
@pytest.mark.parametrize("score,flags", [(SOFTMAX, 0), (SOFTMAX, RENORM), (SIGMOID, 0), (SIGMOID, RENORM)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward(api, T, E, k, score, flags, dtype):
    z = logits_of(T, E, dtype, seed=T + E)
    if T > 4:
        z[1] = -INF
        z[2, : E - 1] = -INF
        z[3] -= 150.0
    z = z.cuda()
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(k)).cuda()
    ids, _ = api.nvfp4_route(z, k, score, flags)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = api.nvfp4_route_backward(dw, ids, z, score, flags, scale=1.5, status=status)
    want, bound = backward_reference(z, ids, dw, score, flags, 1.5)
    bound = bound + 2.0 ** -126
    if dtype == torch.bfloat16:
        bound = bound + HALF * (want.abs() + bound)
    within(d, want, bound, "dlogits")
    assert int(status) == 0 and d.dtype == dtype
    # in place, and into rows further apart
    wide = torch.full((T, E + 5), 7.0, dtype=dtype, device="cuda")
    assert torch.equal(api.nvfp4_route_backward(dw, ids, z, score, flags, scale=1.5, out=wide[:, :E]), d)
    assert bool((wide[:, E:] == 7.0).all())
    zz = z.clone()
    assert api.nvfp4_route_backward(dw, ids, zz, score, flags, scale=1.5, out=zz) is zz and torch.equal(zz, d)


@pytest.mark.parametrize("score,flags", [(SOFTMAX, 0), (SOFTMAX, RENORM), (SIGMOID, 0), (SIGMOID, RENORM)])
def test_route_backward_against_differences(api, score, flags):
    """d loss = <dw, w> along random directions, by central differences of the
    64-bit weights at fixed choices."""
    g = torch.Generator().manual_seed(21)
    z = torch.randn((6, 20), generator=g)
    dw = torch.randn((6, 4), generator=g)
    ids, _ = api.nvfp4_route(z.cuda(), 4, score, flags)
    d = api.nvfp4_route_backward(dw.cuda(), ids, z.cuda(), score, flags, scale=2.0).double().cpu()
    at = ids.cpu().long()

    def loss(z64):
        w = scores(z64, score).gather(1, at)
        w = w / w.sum(1, keepdim=True) if flags & RENORM else w
        return float((w * 2.0 * dw.double()).sum())

    for _ in range(5):
        v = torch.randn((6, 20), generator=g, dtype=torch.float64)
        h = 1e-5
        num = (loss(z.double() + h * v) - loss(z.double() - h * v)) / (2 * h)
        # the differences' own error is about h^2 and 1e-16 / h; fp32 gradients add 1e-6 of their magnitudes
        assert abs(num - float((d * v).sum())) <= 1e-5 * float((d * v).abs().sum()) + 1e-8


def test_route_backward_bad_and_repeated_ids(api):
    z = logits_of(4, 12, torch.float32, seed=2).cuda()
    dw = torch.ones((4, 3), device="cuda")
    ids = torch.tensor([[0, 1, 2], [3, 12, 4], [5, -2, -1], [6, 6, 7]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = api.nvfp4_route_backward(dw, ids, z, SIGMOID, 0, status=status)
    assert int(status) == -1
    ids[1, 1] = ids[2, 1] = -1
    want, bound = backward_reference(z, ids, dw, SIGMOID, 0, 1.0)   # an expert named twice gets both parts
    within(d, want, bound + 2.0 ** -126, "dlogits")


def test_route_strided_logits_and_given_outputs(api):
    z = logits_of(30, 70, torch.bfloat16, seed=1).cuda()
    wide = torch.full((30, 91), INF, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:73] = z
    ids = torch.full((30, 4), 9, dtype=torch.int32, device="cuda")
    w = torch.zeros((30, 4), device="cuda")
    got = api.nvfp4_route(wide[:, 3:73], 4, ids=ids, weights=w)
    want = api.nvfp4_route(z, 4)
    assert got[0] is ids and got[1] is w and torch.equal(ids, want[0]) and torch.equal(w, want[1])
    empty = api.nvfp4_route(z[:0], 4)
    assert empty[0].shape == (0, 4) and empty[1].shape == (0, 4)


# ---------------------------------------------------------------------------
# dispatch and combine
# ---------------------------------------------------------------------------
def choices(T, k, E, seed, none=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.argsort(torch.rand((T, E), generator=g), 1)[:, :k] if k <= E else torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(ids.shape, generator=g) < none] = -1
    return ids.to(torch.int32)


def sort_reference(ids, E):
    flat = ids.reshape(-1).numpy()
    rows = np.full(flat.size, -1, dtype=np.int32)
    order = [p for e in range(E) for p in np.nonzero(flat == e)[0]] if flat.size < 5000 else \
        np.argsort(np.where(flat < 0, E, flat), kind="stable")[: int((flat >= 0).sum())]
    rows[np.asarray(order, dtype=np.int64)] = np.arange(len(order))
    counts = np.bincount(flat[flat >= 0], minlength=E)
    return torch.from_numpy(rows).view(ids.shape), torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def rows_of(T, C, seed):
    return torch.randn((T, C), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("T,k,E,C,none", [
    (1, 1, 1, 8, 0.0), (1, 8, 256, 64, 0.0), (2, 3, 4, 24, 0.5), (31, 2, 8, 72, 0.1), (64, 8, 256, 4096, 0.05), (33, 1, 1024, 128, 0.0),
    (500, 6, 64, 200, 0.2), (1025, 4, 60, 2056, 0.0), (3000, 8, 7, 64, 0.0), (40000, 8, 160, 8, 0.1), (257, 32, 1000, 16, 0.3),
    (100, 4, 16, 64, 1.0)])
def test_dispatch(api, T, k, E, C, none):
    ids = choices(T, k, E, seed=T + k, none=none)
    x = rows_of(T, C, seed=T)
    out = torch.full((T * k, C), 5.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xs, rows, offsets = api.nvfp4_dispatch(x, ids.cuda(), E, out=out, status=status)
    want_rows, want_offsets = sort_reference(ids, E)
    assert torch.equal(rows.cpu(), want_rows) and torch.equal(offsets.cpu(), want_offsets)
    want = torch.full((T * k, C), 5.0, dtype=torch.bfloat16, device="cuda")
    live = (want_rows.view(-1) >= 0).cuda()
    want[want_rows.view(-1).long().cuda()[live]] = x.repeat_interleave(k, 0)[live]
    assert torch.equal(xs, want) and xs is out and int(status) == 0
    none_xs, r2, o2 = api.nvfp4_dispatch(None, ids.cuda(), E)
    assert none_xs is None and torch.equal(r2, rows) and torch.equal(o2, offsets)


def test_dispatch_bad_ids_and_no_tokens(api):
    ids = torch.tensor([[0, 5], [4, -1], [3, -7], [1, 1 << 30]], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = rows_of(4, 16, seed=1)
    xs, rows, offsets = api.nvfp4_dispatch(x, ids.cuda(), 5, status=status)
    assert int(status) == -1
    assert rows.tolist() == [[0, -1], [3, -1], [2, -1], [1, -1]] and offsets.tolist() == [0, 1, 2, 2, 3, 4]
    assert torch.equal(xs[:4], x[[0, 3, 2, 1]])
    xs, rows, offsets = api.nvfp4_dispatch(x[:0], torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert xs.shape == (0, 16) and rows.shape == (0, 2) and offsets.tolist() == [0] * 6


def combine_reference(y, rows, w, residual):
    """Sums and their magnitudes in 64 bits."""
    y, rows = y.double().cpu(), rows.cpu().long()
    T, k = rows.shape
    out = torch.zeros((T, y.shape[1]), dtype=torch.float64) if residual is None else residual.double().cpu()
    mag = out.abs()
    for j in range(k):
        live = rows[:, j] >= 0
        part = y[rows[live, j]] * (1.0 if w is None else w.double().cpu()[live, j:j + 1])
        out[live] += part
        mag[live] += part.abs()
    return out, mag


@pytest.mark.parametrize("T,k,E,C,none", [(1, 1, 4, 8, 0.0), (1, 8, 64, 4096, 0.0), (3, 2, 8, 24, 0.4), (65, 6, 16, 520, 0.1),
                                          (200, 9, 32, 2056, 0.1), (33, 32, 64, 72, 0.2), (1000, 4, 8, 64, 0.0), (7, 17, 40, 14336, 0.1)])
@pytest.mark.parametrize("weighted,res", [(True, False), (True, True), (False, False), (False, True)])
def test_combine(api, T, k, E, C, none, weighted, res):
    rows = sort_reference(choices(T, k, E, seed=T, none=none), E)[0].cuda()
    rows[T // 2] = -1
    y, residual = rows_of(T * k, C, seed=k), rows_of(T, C, seed=k + 1) if res else None
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(C)).cuda() - 0.3 if weighted else None
    dead = torch.ones(T * k, dtype=torch.bool)
    dead[rows.view(-1).cpu().long()[rows.view(-1).cpu() >= 0]] = False
    y[dead.cuda()] = math.nan                 # rows of no pair are not read
    out = api.nvfp4_combine(y, rows, w, residual=residual)
    want, mag = combine_reference(y, rows, w, residual)
    bound = (k + 1) * U * mag
    within(out, want, bound + HALF * (want.abs() + bound), "out")
    empty = torch.zeros(C, dtype=torch.bfloat16, device="cuda") if residual is None else residual[T // 2]
    assert torch.equal(out[T // 2], empty)
    if res:
        into = residual.clone()
        assert api.nvfp4_combine(y, rows, w, residual=into, out=into) is into and torch.equal(into, out)


@pytest.mark.parametrize("T,k,E,C,none", [(1, 1, 4, 8, 0.0), (1, 8, 64, 4096, 0.0), (3, 2, 8, 24, 0.4), (65, 6, 16, 520, 0.1),
                                          (200, 9, 32, 2056, 0.1), (33, 32, 64, 72, 0.2), (1000, 4, 8, 64, 0.0), (9, 17, 40, 14336, 0.1)])
def test_combine_backward(api, T, k, E, C, none):
    rows = sort_reference(choices(T, k, E, seed=T, none=none), E)[0].cuda()
    y, dout = rows_of(T * k, C, seed=k), rows_of(T, C, seed=k + 1)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(C)).cuda() - 0.3
    out = torch.full((T * k, C), 5.0, dtype=torch.bfloat16, device="cuda")
    dy, dw = api.nvfp4_combine_backward(dout, rows, w, y, out=out)
    live = rows.view(-1) >= 0
    at = rows.view(-1).long()[live]
    want = torch.full((T * k, C), 5.0, dtype=torch.bfloat16, device="cuda")
    want[at] = (dout.float().repeat_interleave(k, 0) * w.view(-1, 1)).bfloat16()[live]
    assert dy is out and torch.equal(dy, want)
    prod = torch.zeros((T * k, C), dtype=torch.float64, device="cuda")
    prod[live] = dout.double().repeat_interleave(k, 0)[live] * y.double()[at]
    within(dw, prod.sum(1).view(T, k).cpu(), (C + 32) * U * prod.abs().sum(1).view(T, k).cpu(), "dweights")
    # one of the two alone; without weights
    a, none_dw = api.nvfp4_combine_backward(dout, rows, w, y, need_dweights=False, out=torch.full_like(out, 5.0))
    none_dy, b = api.nvfp4_combine_backward(dout, rows, w, y, need_dy=False)
    assert none_dw is None and none_dy is None and torch.equal(a, dy) and torch.equal(b, dw)
    c, d = api.nvfp4_combine_backward(dout, rows, None, y, out=torch.full_like(out, 5.0))
    want[at] = dout.repeat_interleave(k, 0)[live]
    assert torch.equal(c, want) and torch.equal(d, dw)


def test_combine_is_dispatchs_gradient_and_bad_rows(api):
    T, k, E, C = 50, 3, 6, 40
    ids = choices(T, k, E, seed=1).cuda()
    dxs = rows_of(T * k, C, seed=2)
    _, rows, _ = api.nvfp4_dispatch(None, ids, E)
    want, mag = combine_reference(dxs, rows, None, None)
    bound = k * U * mag
    within(api.nvfp4_combine(dxs, rows), want, bound + HALF * (want.abs() + bound), "dx")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = rows.clone()
    bad[3, 1], bad[4, 0] = T * k, -2
    none = rows.clone()
    none[3, 1] = none[4, 0] = -1
    w = torch.rand((T, k), device="cuda")
    assert torch.equal(api.nvfp4_combine(dxs, bad, w, status=status), api.nvfp4_combine(dxs, none, w)) and int(status) == -1
    status.zero_()
    dout = rows_of(T, C, seed=3)
    outs = [api.nvfp4_combine_backward(dout, r, w, dxs, out=torch.zeros_like(dxs), status=status) for r in (bad, none)]
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]) and int(status) == -1
    same = torch.full((T, k), 7, dtype=torch.int32, device="cuda")      # one place any number of times
    want, mag = combine_reference(dxs, same, w, None)
    within(api.nvfp4_combine(dxs, same, w), want, k * U * mag + HALF * (want.abs() + k * U * mag), "out")


def test_combine_strided_rows_and_pair_order(api):
    T, k, C = 20, 4, 48
    w = torch.rand((T, k), device="cuda")
    y, res = rows_of(T * k, C, seed=2), rows_of(T, C, seed=4)
    order = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    want = api.nvfp4_combine(y, order, w, residual=res)
    assert torch.equal(api.nvfp4_combine(y, None, w, residual=res), want)
    wide = torch.zeros((T * k, 80), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:56] = y
    out = torch.full((T, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    api.nvfp4_combine(wide[:, 8:56], order, w, residual=res, out=out[:, :C])
    assert torch.equal(out[:, :C], want) and bool((out[:, C:] == 3.0).all())
    dout = rows_of(T, 64, seed=5)[:, 8:56]
    assert not dout.is_contiguous()
    a = api.nvfp4_combine_backward(dout, order, w, wide[:, 8:56])
    b = api.nvfp4_combine_backward(dout.contiguous(), None, w, y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# few-row products
# ---------------------------------------------------------------------------
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] + [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], dtype=torch.float64)


def random_weight(E, N, K, seed):
    """Random codes and random scale bytes (every finite E4M3 magnitude)."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    delta = torch.randint(0, 127, (E, N, K // 16), generator=g, dtype=torch.uint8)
    layout = delta.view(E, N // 128, 4, 32, K // 64, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1)
    alpha = torch.rand(E, generator=g) * 1e-3 + 1e-4
    q = GRID[torch.stack([codes & 15, codes >> 4], -1).view(E, N, K).long()]
    w = q * delta.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return codes.cuda(), layout.cuda(), alpha.cuda(), w


def check_gemv(api, x, W, sW, alpha, w, ids, out_dtype, **kw):
    y = api.nvfp4_gemv(x, W if ids is not None else W[0], sW, alpha, ids=ids, out_dtype=out_dtype, **kw)
    x64, a = x.double().cpu(), alpha.double().cpu()
    if ids is None:
        e, src = torch.zeros(x.shape[0], dtype=torch.long), torch.arange(x.shape[0])
    else:
        e = ids.view(-1).cpu().long()
        src = torch.arange(e.numel())
        src = src // ids.shape[1] if x.shape[0] == ids.shape[0] else src
    want = torch.zeros((e.numel(), w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(want)
    for i in range(w.shape[0]):
        at = torch.nonzero(e == i).view(-1)
        want[at] = a[i] * (x64[src[at]] @ w[i].t())
        mag[at] = a[i] * (x64[src[at]].abs() @ w[i].abs().t())
    bound = (2 * x.shape[1] + 32) * U * mag
    within(y, want, bound + (HALF if out_dtype == api.NVFP4_OUT_DTYPE_BF16 else U) * (want.abs() + bound), "y")
    assert not bool(y[(e < 0).cuda()].any())
    return y


@pytest.mark.parametrize("P", [1, 2, 7, 8, 9, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("N,K", [(128, 64), (256, 192), (128, 1024), (640, 2112)])
def test_gemv_dense(api, P, N, K):
    W, sW, alpha, w = random_weight(1, N, K, seed=N + K)
    x = rows_of(P, K, seed=P)
    check_gemv(api, x, W, sW, alpha, w, None, api.NVFP4_OUT_DTYPE_FP32)
    check_gemv(api, x, W, sW, alpha, w, None, api.NVFP4_OUT_DTYPE_BF16)


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 128, 64), (1, 8, 64, 128, 128), (1, 2, 8, 256, 4096), (8, 2, 8, 128, 320), (5, 4, 4, 256, 64),
                                       (64, 8, 256, 128, 128), (100, 2, 3, 128, 192), (32, 32, 1024, 128, 64), (12, 6, 40, 384, 960)])
@pytest.mark.parametrize("shared", [True, False])
def test_gemv_by_expert(api, T, k, E, N, K, shared):
    W, sW, alpha, w = random_weight(E, N, K, seed=E + K)
    ids = choices(T, k, E, seed=T + E, none=0.0 if T == 1 else 0.15).cuda()
    x = rows_of(T if shared else T * k, K, seed=K)
    check_gemv(api, x, W, sW, alpha, w, ids, api.NVFP4_OUT_DTYPE_FP32)
    check_gemv(api, x, W, sW, alpha, w, ids, api.NVFP4_OUT_DTYPE_BF16)


def test_gemv_every_code_and_scale(api):
    """Every product of a code and an E4M3 magnitude comes out exactly."""
    N, K = 128, 2048
    n, kb = torch.arange(N).view(-1, 1), torch.arange(K // 16).view(1, -1)
    delta = ((n * 0 + kb) % 127).to(torch.uint8)
    code = ((torch.arange(K).view(1, -1) + n) % 16).to(torch.uint8)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    layout = delta.view(N // 128, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    w = GRID[code.long()] * delta.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    alpha = torch.ones(1, device="cuda")
    for first in range(0, K, 1024):
        x = torch.zeros((1024, K), dtype=torch.bfloat16, device="cuda")
        x[torch.arange(1024), first + torch.arange(1024)] = 1.0
        y = api.nvfp4_gemv(x, codes.cuda(), layout.cuda(), alpha, out_dtype=api.NVFP4_OUT_DTYPE_FP32)
        assert torch.equal(y.double().cpu(), w[:, first:first + 1024].t())


def test_gemv_bad_ids_strides_and_infinities(api):
    W, sW, alpha, w = random_weight(4, 128, 192, seed=3)
    ids = torch.tensor([[0, 4], [3, -1], [-5, 3]], dtype=torch.int32, device="cuda")
    good = torch.tensor([[0, -1], [3, -1], [-1, 3]], dtype=torch.int32, device="cuda")
    wide = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:200] = rows_of(3, 192, seed=1)
    x = wide[:, 8:200]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((6, 200), 9.0, device="cuda")
    y = check_gemv(api, x, W, sW, alpha, w, good, 1)
    api.nvfp4_gemv(x, W, sW, alpha, ids=ids, out_dtype=1, out=out[:, :128], status=status)
    assert int(status) == -1 and torch.equal(out[:, :128], y) and bool((out[:, 128:] == 9.0).all())
    # an infinity stays in its own row
    x = rows_of(9, 192, seed=2)
    clean = api.nvfp4_gemv(x, W[0], sW[0], alpha[:1], out_dtype=1)
    x[4, 100] = INF
    y = api.nvfp4_gemv(x, W[0], sW[0], alpha[:1], out_dtype=1)
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(y[keep], clean[keep])
    col = w[0, :, 100]
    assert bool((y[4].cpu()[col > 0] == INF).all()) and bool((y[4].cpu()[col < 0] == -INF).all())
    assert bool(torch.isnan(y[4].cpu()[col == 0]).all())
    assert api.nvfp4_gemv(x[:0], W[0], sW[0], alpha[:1]).shape == (0, 128)


# ---------------------------------------------------------------------------
# sizes past 2^31 elements
# ---------------------------------------------------------------------------
def test_rows_past_2_31_elements(api):
    T, k, C, E = 70000, 8, 4096, 64
    x = torch.randn((T, C), device="cuda", dtype=torch.bfloat16)
    ids = (torch.arange(T * k, device="cuda").view(T, k) * 37 % E).to(torch.int32)
    xs, rows, offsets = api.nvfp4_dispatch(x, ids, E)
    want_rows, want_offsets = sort_reference(ids.cpu(), E)
    assert torch.equal(rows.cpu(), want_rows) and torch.equal(offsets.cpu(), want_offsets)
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    assert torch.equal(xs[rows[at].long()], x[at].unsqueeze(1).expand(-1, k, -1))
    w = torch.full((T, k), 0.125, device="cuda")
    assert torch.equal(api.nvfp4_combine(xs, rows, w), x)         # eight eighths, exact
    dy, dw = api.nvfp4_combine_backward(x, rows, w, xs, out=xs.new_zeros(xs.shape))
    assert torch.equal(dy[rows[at].long()], (x[at] * 0.125).unsqueeze(1).expand(-1, k, -1))
    want = x[at].double().square()
    within(dw[at], want.sum(1, keepdim=True).expand(-1, k).cpu(), (C + 32) * U * want.sum(1, keepdim=True).expand(-1, k).cpu(), "dweights")


def test_logits_past_2_31_elements(api):
    T, E = (1 << 23) + 1000, 256
    few = logits_of(512, E, torch.bfloat16, seed=1).cuda()
    z = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    z[-512:] = few
    z[:-512] = 0.0
    ids, w = api.nvfp4_route(z, 4)
    a, b = api.nvfp4_route(few, 4)
    assert torch.equal(ids[-512:], a) and torch.allclose(w[-512:], b, rtol=64 * U, atol=0) and ids[0].tolist() == [0, 1, 2, 3]
    dw = torch.ones((T, 4), device="cuda")
    dw[:, 1:] = 0.5
    for flags in (0, RENORM):
        d = api.nvfp4_route_backward(dw, ids, z, flags=flags)
        assert torch.equal(d[-512:], api.nvfp4_route_backward(dw[-512:], a, few, flags=flags))


def test_weights_past_2_31_bytes(api):
    E, N, K = 76, 14336, 4096
    W = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    sW = torch.randint(40, 70, (E, N * K // 16), device="cuda", dtype=torch.uint8)
    alpha = torch.full((E,), 1e-3, device="cuda")
    ids = torch.tensor([[E - 1, 0], [E - 1, 40]], dtype=torch.int32, device="cuda")
    x = rows_of(2, K, seed=1)
    y = api.nvfp4_gemv(x, W, sW, alpha, ids=ids, out_dtype=1)
    for t in range(2):
        for j in range(2):
            e = int(ids[t, j])
            assert torch.equal(y[2 * t + j], api.nvfp4_gemv(x[t:t + 1], W[e].clone(), sW[e].clone(), alpha[:1], out_dtype=1)[0])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def expert_layer(api, x, z, W, sW, alpha, k, status, residual):
    """Route, dispatch, quantize, multiply by expert, combine."""
    ids, w = api.nvfp4_route(z, k, SIGMOID, RENORM | PAIR, groups=4, groups_kept=2, scale=1.5, status=status)
    xs, rows, offsets = api.nvfp4_dispatch(x, ids, W.shape[0], status=status)
    q = api.nvfp4_quantize_grouped(xs, offsets, api.NVFP4_FOUR_SIX, api.NVFP4_ROWWISE, status=status)
    y = api.nvfp4_gemm_grouped(q.codes_row, q.scales_row, q.alpha_row, W, sW, alpha, offsets, status=status)
    out = api.nvfp4_combine(y, rows, w, residual=residual, status=status)
    return ids, w, xs, rows, offsets, q, y, out


def test_expert_layer(api):
    T, E, k, K, N = 90, 8, 3, 256, 128
    W, sW, alpha, w64 = random_weight(E, N, K, seed=1)
    x, z, res = rows_of(T, K, seed=2), logits_of(T, E, torch.float32, seed=3).cuda(), rows_of(T, N, seed=4)
    z[5] = -INF
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w, xs, rows, offsets, q, y, out = expert_layer(api, x, z, W, sW, alpha, k, status, res)
    assert int(status) == 0 and torch.equal(out[5], res[5]) and int(offsets[-1]) == (T - 1) * k
    # the products in 64 bits of the operands as they were quantized
    xq = api.nvfp4_dequantize_grouped(q.codes_row, q.scales_row, q.alpha_row, offsets, T * k, K, api.NVFP4_ROWWISE).double().cpu()
    off = offsets.cpu().tolist()
    y64 = torch.zeros((T * k, N), dtype=torch.float64)
    for e in range(E):
        y64[off[e]:off[e + 1]] = xq[off[e]:off[e + 1]] @ w64[e].t() * float(alpha[e])
    ymag = (y.double().cpu() - y64)[: off[-1]].norm() / y64[: off[-1]].norm()
    assert ymag < 2 * HALF
    want, mag = combine_reference(y, rows, w, res)
    within(out, want, (k + 1) * U * mag + HALF * (want.abs() + (k + 1) * U * mag), "out")
    # the same layer without quantized activations, as a decode step runs it
    yd = api.nvfp4_gemv(x, W, sW, alpha, ids=ids)
    direct = api.nvfp4_combine(yd, None, w, residual=res)
    exact = torch.zeros((T * k, N), dtype=torch.float64)
    flat = ids.view(-1).cpu().long()
    for p in range(T * k):
        if flat[p] >= 0:
            exact[p] = w64[flat[p]] @ x[p // k].double().cpu() * float(alpha[flat[p]])
    want, mag = combine_reference(exact, torch.arange(T * k).view(T, k), w, res)
    within(direct, want, 3 * HALF * mag, "direct")


def test_expert_layer_in_a_graph_with_changing_choices(api):
    T, E, k, K, N = 40, 8, 2, 128, 128
    W, sW, alpha, _ = random_weight(E, N, K, seed=5)
    x, z, res = rows_of(T, K, seed=6), logits_of(T, E, torch.float32, seed=7).cuda(), rows_of(T, N, seed=8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    expert_layer(api, x, z, W, sW, alpha, k, status, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = expert_layer(api, x, z, W, sW, alpha, k, status, res)
        step = api.nvfp4_combine(api.nvfp4_gemv(x, W, sW, alpha, ids=held[0]), None, held[1])
    for seed in (11, 12):
        x.copy_(rows_of(T, K, seed=seed))
        z.copy_(logits_of(T, E, torch.float32, seed=seed + 20))
        z[seed] = -INF
        graph.replay()
        ids, w, xs, rows, offsets, q, y, out = expert_layer(api, x, z, W, sW, alpha, k, status, res)
        live = int(offsets[-1])
        for a, b in ((held[0], ids), (held[1], w), (held[3], rows), (held[4], offsets), (held[2][:live], xs[:live]),
                     (held[6][:live], y[:live]), (held[7], out)):
            assert torch.equal(a, b)
        assert torch.equal(step, api.nvfp4_combine(api.nvfp4_gemv(x, W, sW, alpha, ids=ids), None, w))
    assert int(status) == 0


def test_training_step_gradients(api):
    """Gradients of sum(dout out) through combine, a fixed row map and route
    against differences of the 64-bit composition."""
    T, E, k, C = 12, 6, 2, 16
    g = torch.Generator().manual_seed(31)
    z = torch.randn((T, E), generator=g)
    x = rows_of(T, C, seed=32)
    dout = rows_of(T, C, seed=33)
    ids, w = api.nvfp4_route(z.cuda(), k, SOFTMAX, RENORM)
    xs, rows, _ = api.nvfp4_dispatch(x, ids, E)
    ys = (2 * xs).bfloat16()                                        # the experts: y = 2 x, exact
    dys, dw = api.nvfp4_combine_backward(dout, rows, w, ys)
    dz = api.nvfp4_route_backward(dw, ids, z.cuda(), SOFTMAX, RENORM).double().cpu()
    dx = api.nvfp4_combine((2 * dys).bfloat16(), rows).double().cpu()
    at = ids.cpu().long()

    def loss(z64, x64):
        p = scores(z64, SOFTMAX).gather(1, at)
        p = p / p.sum(1, keepdim=True)
        return float((dout.double().cpu() * (p.unsqueeze(-1) * 2 * x64.unsqueeze(1)).sum(1)).sum())

    z64, x64 = z.double(), x.double().cpu()
    for _ in range(4):
        vz, vx = torch.randn((T, E), generator=g, dtype=torch.float64), torch.randn((T, C), generator=g, dtype=torch.float64)
        h = 1e-5
        num = (loss(z64 + h * vz, x64) - loss(z64 - h * vz, x64)) / (2 * h)
        mag = float(((dw.double().cpu().abs().sum(1, keepdim=True) + 1) * vz.abs()).sum())
        assert abs(num - float((dz * vz).sum())) <= 1e-5 * mag
        num = (loss(z64, x64 + h * vx) - loss(z64, x64 - h * vx)) / (2 * h)
        # dys and dx are rounded to bf16 once each
        assert abs(num - float((dx * vx).sum())) <= 2 * HALF * float((2 * dout.double().cpu().abs() * vx.abs()).sum()) + 1e-6


def test_streams_and_equal_calls(api):
    """Calls on two streams at once, and twice, give the same bits."""
    T, E, k, C = 300, 64, 6, 512
    z, x = logits_of(T, E, torch.bfloat16, seed=1).cuda(), rows_of(T, C, seed=2)
    W, sW, alpha, _ = random_weight(1, 256, C, seed=3)

    def all_of():
        ids, w = api.nvfp4_route(z, k)
        xs, rows, offsets = api.nvfp4_dispatch(x, ids, E)
        out = api.nvfp4_combine(xs, rows, w)
        return (ids, w, xs, rows, offsets, out, api.nvfp4_gemv(x[:20], W[0], sW, alpha), api.nvfp4_route_backward(w, ids, z)) \
            + api.nvfp4_combine_backward(out, rows, w, xs)

    want = all_of()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(all_of())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("P", [1, 9, 20, 30])
def test_gemv_numbers_far_apart(api, P):
    """Rows whose numbers lie up to 250 powers of two apart, the largest often
    next to codes of zero: every product counts, in fp32's range."""
    N, K = 128, 640
    W, sW, alpha, w = random_weight(1, N, K, seed=P)
    g = torch.Generator().manual_seed(P)
    mant = 1 + torch.randint(0, 128, (P, K), generator=g).double() / 128
    for kind in range(4):
        span = ((-120, 100), (-40, 0), (-133, -100), (60, 110))[kind]
        ex = torch.randint(span[0], span[1] + 1, (P, K), generator=g).double()
        x64 = mant * torch.pow(2.0, ex)
        if kind < 2:
            x64[:, : K // 2] = 0.0                       # and many that are nothing
        x = x64.to(torch.bfloat16).cuda()
        y = api.nvfp4_gemv(x, W[0], sW, alpha, out_dtype=1).double().cpu()
        x64 = x.double().cpu()
        want, mag = float(alpha[0]) * (x64 @ w[0].t()), float(alpha[0]) * (x64.abs() @ w[0].abs().t())
        within(y, want, (2 * K + 40) * U * mag + 2.0 ** -126, f"kind {kind}")
    # one number of 2^100 beside ones of 2^-60: weights of 0 leave the small ones' sum
    x = torch.full((P, K), 2.0 ** -60, dtype=torch.bfloat16, device="cuda")
    x[:, 7] = 2.0 ** 100
    y = api.nvfp4_gemv(x, W[0], sW, alpha, out_dtype=1).double().cpu()
    x64 = x.double().cpu()
    want, mag = float(alpha[0]) * (x64 @ w[0].t()), float(alpha[0]) * (x64.abs() @ w[0].abs().t())
    assert bool((w[0, :, 7] == 0).any())
    within(y, want, (2 * K + 40) * U * mag, "beside 2^100")


def test_gemv_infinities_of_both_kinds_and_numbers_far_apart(api):
    N, K = 128, 512
    W, sW, alpha, w = random_weight(1, N, K, seed=77)
    x = rows_of(5, K, seed=1)
    x[1, 3], x[2, 300], x[3, 5] = INF, -INF, math.nan
    x[0, 9] = 2.0 ** -130
    x[0, 10] = 2.0 ** 120
    x[4] = 0.0
    y = api.nvfp4_gemv(x, W[0], sW, alpha, out_dtype=1).cpu()
    want = float(alpha[0]) * (x.double().cpu() @ w[0].t())
    for r, k in ((1, 3), (2, 300)):
        col = w[0, :, k]
        assert bool((y[r][col != 0] == want[r][col != 0].float()).all()) and bool(torch.isnan(y[r][col == 0]).all())
    assert bool(torch.isnan(y[3]).all()) and not bool(y[4].any())
    mag = float(alpha[0]) * (x[0].double().cpu().abs() @ w[0].abs().t())
    within(y[0], want[0], (2 * K + 40) * U * mag, "row 0")


# ---------------------------------------------------------------------------
# the two host paths
# ---------------------------------------------------------------------------
class Declines:
    """A C++ host path that takes no call: the binding's checks make them all."""
    def __getattr__(self, name):
        return lambda *args: None


class Answers:
    """The C++ host path; counts the calls that it made."""
    def __init__(self, fast):
        self.fast, self.made = fast, []

    def __getattr__(self, name):
        def call(*args):
            done = getattr(self.fast, name)(*args)
            if type(done) is tuple:
                self.made.append(name)
            return done
        return call


def every_call(api, given, strided):
    """Results of the six calls; outputs and status given, or new; rows of
    their own stride, or contiguous."""
    T, k, E, C, N = 13, 3, 9, 64, 128
    g = torch.Generator().manual_seed(5)

    def rows(n, c, dtype=torch.bfloat16):
        t = torch.randn(n, c + 8, generator=g).cuda().to(dtype)
        return t[:, :c] if strided else t[:, :c].contiguous()

    def new(n, c, dtype=torch.bfloat16):
        return torch.zeros(n, c, dtype=dtype, device="cuda") if given else None

    status = torch.zeros(1, dtype=torch.int32, device="cuda") if given else None
    z = rows(T, 16)[:, :E] if strided else rows(T, E)
    bias = torch.randn(E, generator=g).cuda() if given else None
    ids, w = api.nvfp4_route(z, k, 0, 0, bias, ids=new(T, k, torch.int32), weights=new(T, k, torch.float32), status=status)
    dz = api.nvfp4_route_backward(w, ids, z, 0, 0, 2.0, out=new(T, E), status=status)
    x = rows(T, C)
    xs, places, offsets = api.nvfp4_dispatch(
        x, ids, E, out=new(T * k, C), rows=new(T, k, torch.int32),
        offsets=torch.zeros(E + 1, dtype=torch.int32, device="cuda") if given else None, status=status)
    out = api.nvfp4_combine(xs, places, w, residual=x if given else None, out=new(T, C), status=status)
    back = api.nvfp4_combine_backward(x, places, w, xs, out=new(T * k, C), status=status)
    W = torch.randint(0, 256, (E, N, C // 2), generator=g, dtype=torch.uint8).cuda()
    sW = torch.randint(40, 80, (E, N * (C // 16)), generator=g, dtype=torch.uint8).cuda()
    y = api.nvfp4_gemv(x, W, sW, torch.ones(E, device="cuda"), ids, out=new(T * k, N), status=status)
    return [ids, w, dz, xs, places, offsets, out, *back, y]


SIX = ["route", "route_backward", "dispatch", "combine", "combine_backward", "gemv"]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_both_host_paths_make_the_same_call(api, monkeypatch, given, strided):
    fast = Answers(api._load_fast())
    monkeypatch.setattr(api, "_fast", fast)
    a = every_call(api, given, strided)
    assert fast.made == SIX
    monkeypatch.setattr(api, "_fast", Declines())
    b = every_call(api, given, strided)
    for u, v in zip(a, b):
        assert u.shape == v.shape and u.dtype == v.dtype and u.is_contiguous() and torch.equal(u, v)


def test_fast_host_path_gives_back_the_callers_tensors(api):
    z = torch.randn(4, 8, device="cuda")
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    got = api._load_fast().route(z, 2, 0, 0, None, 1, 1, 1.0, ids, w, None)
    assert got[0] is ids and got[1] is w
    assert api._load_fast().dispatch(None, ids, 8, None, None, None, None)[0] is None


def test_fast_host_path_refuses_as_the_checks_do(api):
    """Host-side refusals: nothing is launched."""
    z = torch.zeros(4, 8, device="cuda")
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    y = torch.zeros(8, 64, device="cuda").bfloat16()
    fast = api._load_fast()
    for bad in ((ids[:3], None, None), (ids.long(), None, None), (None, w[:, :1], None), (None, w.cpu(), None), (None, None, w)):
        assert fast.route(z, 2, 0, 0, None, 1, 1, 1.0, *bad) is None
        with pytest.raises((TypeError, ValueError)):
            api.nvfp4_route(z, 2, ids=bad[0], weights=bad[1], status=bad[2])
    for kw in (dict(score=7), dict(flags=9), dict(groups=3), dict(k=9), dict(k=0)):
        with pytest.raises(api.NVFP4Error):
            api.nvfp4_route(z, **{"k": 2, **kw})
    with pytest.raises(api.NVFP4Error):
        api.nvfp4_combine(y[:, :60], ids, w)                      # C not a multiple of 8
    with pytest.raises(ValueError):
        api.nvfp4_combine(y, ids, w, out=torch.zeros(4, 32, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        api.nvfp4_combine_backward(y[:4], ids, w, y, need_dy=False, out=y)
    with pytest.raises(ValueError):
        api.nvfp4_dispatch(None, ids, 8, out=y)
    with pytest.raises(ValueError):
        api.nvfp4_gemv(y, torch.zeros(8, 30, dtype=torch.uint8, device="cuda"), ids.byte(), w.view(-1))


def test_fast_host_path_takes_the_current_stream(api):
    """The call goes to the stream that is current, behind its earlier work."""
    z = torch.zeros(64, 64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z.add_(torch.arange(64, device="cuda"))
        ids, _ = api.nvfp4_route(z, 2)
    torch.cuda.current_stream().wait_stream(s)
    assert ids.cpu().tolist() == [[63, 62]] * 64
