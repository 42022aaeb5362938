"""Low-rank adapters beside a shared projection: nvfp4_lora_apply and
nvfp4_lora_backward against 64-bit products.

Tolerances, element by element.  A product of two bf16 numbers is exact in
fp32; a sum of k of them in fp32 is off by at most k steps of 2^-23 of the sum
of magnitudes (truncating adds included).  So with u = 2^-23 and |.| taken
element by element:
  h:  E_h = (K + 32) u |x| |A|^T        (32: the partial sums of the splits)
  h enters a product as two bf16 numbers: + 2^-17 |h|
  out: s (E_h + 2^-17 |h|) |B|^T + s (2 r + 3) u |h| |B|^T, then one rounding
       to bf16 of the sum with y: half a step, 2^-8 of its magnitude
and the same for g, dx; dA and dB are sums over at most T tokens (2 T + 16).
"""
import pytest
import torch

from nvfp4_block_quantization_amax_b200 import synthetic

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF = torch.finfo(torch.bfloat16).eps / 2
FP32, BF16 = 1, 0


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_quantization_amax_b200 import api as _api
    return _api


def ids_of(kind, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((T,), n - 1, dtype=torch.int32)
    if kind == "random":
        return torch.randint(-1, n, (T,), generator=g).to(torch.int32)
    cuts = torch.sort(torch.randint(0, T + 1, (n + 1,), generator=g)).values.tolist()
    order = torch.randperm(n + 2, generator=g) - 1                 # runs, one without an adapter, one id twice
    order[order == n] = 0
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    return torch.repeat_interleave(order, torch.tensor(lengths)).to(torch.int32)


def problem(T, K, N, r, n, kind, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    rnd = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    return dict(x=rnd(T, K).bfloat16().cuda(), A=(rnd(n, r, K) / K ** 0.5).bfloat16().cuda(),
                B=(rnd(n, N, r) * 0.1).bfloat16().cuda(), scaling=(torch.rand(n, generator=g) + 0.5).cuda(),
                ids=ids_of(kind, T, n, seed).cuda(), y=rnd(T, N).bfloat16().cuda(), dy=(rnd(T, N) * 1e-2).bfloat16().cuda(),
                dx=(rnd(T, K) * 1e-2).bfloat16().cuda())


def within(got, ref, bound, what):
    over = (got.double() - ref).abs() - bound
    assert bool((over <= 0).all()), f"{what}: {float(over.max()):.3g} over the bound"


def reference(p, h=None):
    """64-bit results and bounds of both directions; h: the forward's h as the backward was given it."""
    x, A, B, s, y, dy, dx = (p[k].double() for k in ("x", "A", "B", "scaling", "y", "dy", "dx"))
    T, K = x.shape
    n, N, r = B.shape
    f = dict(h=torch.zeros((T, r), dtype=torch.float64, device="cuda"), out=y.clone(), dx=dx.clone(),
             dA=torch.zeros_like(A), dB=torch.zeros_like(B))
    e = {k: torch.zeros_like(v) for k, v in f.items()}
    for a in range(n):
        t = torch.nonzero(p["ids"] == a).view(-1)
        if len(t) == 0:
            continue
        f["h"][t] = x[t] @ A[a].t()
        e["h"][t] = (K + 32) * U * (x[t].abs() @ A[a].abs().t())
        habs = f["h"][t].abs()
        f["out"][t] += s[a] * (f["h"][t] @ B[a].t())
        e["out"][t] = s[a] * ((e["h"][t] + (2.0 ** -17 + (2 * r + 3) * U) * habs) @ B[a].abs().t())
        g = dy[t] @ B[a]
        eg = (N + 32) * U * (dy[t].abs() @ B[a].abs())
        gb = eg + 2.0 ** -17 * g.abs()
        f["dx"][t] += s[a] * (g @ A[a])
        e["dx"][t] = s[a] * ((gb + (2 * r + 3) * U * g.abs()) @ A[a].abs())
        f["dA"][a] = s[a] * (g.t() @ x[t])
        e["dA"][a] = s[a] * ((gb + (2 * T + 16) * U * g.abs()).t() @ x[t].abs())
        hh = (f["h"] if h is None else h.double())[t]
        f["dB"][a] = s[a] * (dy[t].t() @ hh)
        e["dB"][a] = s[a] * (dy[t].abs().t() @ ((2.0 ** -17 + (2 * T + 16) * U) * hh.abs()))
    for k in ("out", "dx"):
        e[k] += HALF * (f[k].abs() + e[k])
    return f, e


def check(api, p, out_dtype=FP32):
    none = p["ids"] < 0
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
    f, e = reference(p, h)
    within(h, f["h"], e["h"], "h")
    within(out, f["out"], e["out"], "out")
    assert torch.equal(out[none], p["y"][none]) and not bool(h[none].any())
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], dx=p["dx"],
                                         out_dtype=out_dtype)
    within(dx, f["dx"], e["dx"], "dx")
    assert torch.equal(dx[none], p["dx"][none])
    for got, k in ((dA, "dA"), (dB, "dB")):
        assert got.dtype == (torch.float32 if out_dtype == FP32 else torch.bfloat16)
        within(got, f[k], e[k] + (HALF if out_dtype == BF16 else 2.0 ** -24) * (f[k].abs() + e[k]), k)
    return out, h, dx, dA, dB


@pytest.mark.parametrize("T,K,N,r,n,kind", [
    (1, 64, 64, 16, 1, "one"), (1, 8, 8, 8, 3, "random"), (3, 72, 136, 8, 2, "random"), (16, 512, 256, 16, 40, "random"),
    (63, 128, 128, 24, 4, "runs"), (64, 200, 264, 32, 5, "random"), (65, 256, 128, 40, 3, "runs"),
    (130, 136, 520, 64, 4, "runs"), (200, 320, 1032, 128, 3, "random"), (300, 1000, 2056, 16, 6, "runs"),
    (517, 384, 200, 72, 9, "random"), (70, 64, 64, 16, 4, "none"), (129, 2048, 384, 16, 1, "one"),
    (1030, 640, 384, 104, 2, "runs"), (2, 4096, 128, 128, 2, "random"),
])
def test_shapes_and_orders(api, T, K, N, r, n, kind):
    check(api, problem(T, K, N, r, n, kind, seed=T))


@pytest.mark.parametrize("T,n,kind", [(5000, 2, "runs"), (4100, 3, "random"), (900, 200, "random")])
def test_many_tokens_and_many_adapters(api, T, n, kind):
    check(api, problem(T, 136, 264, 16, n, kind, seed=3))


def test_bf16_gradients(api):
    check(api, problem(300, 256, 384, 16, 3, "runs"), out_dtype=BF16)


def test_without_a_base_and_in_place(api):
    p = problem(150, 256, 264, 16, 3, "runs", seed=5)
    args = (p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    want, h = api.nvfp4_lora_apply(*args, y=p["y"])
    y = p["y"].clone()
    got, _ = api.nvfp4_lora_apply(*args, y=y, out=y)
    assert got is y and torch.equal(y, want)
    alone, _ = api.nvfp4_lora_apply(*args)
    zero, _ = api.nvfp4_lora_apply(*args, y=torch.zeros_like(y))
    assert torch.equal(alone, zero)
    back = (p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"])
    want = api.nvfp4_lora_backward(*back, dx=p["dx"])
    dx = p["dx"].clone()
    got = api.nvfp4_lora_backward(*back, dx=dx, dx_out=dx)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    alone = api.nvfp4_lora_backward(*back)
    zero = api.nvfp4_lora_backward(*back, dx=torch.zeros_like(dx))
    assert all(torch.equal(a, b) for a, b in zip(alone, zero))


def test_strided_rows(api):
    p = problem(90, 256, 136, 24, 3, "random", seed=6)
    want = check(api, p)
    wide = {k: torch.full((90, p[k].shape[1] + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
            for k in ("x", "y", "dy", "dx")}
    q = dict(p)
    for k, w in wide.items():
        q[k] = w[:, 16:16 + p[k].shape[1]]
        q[k].copy_(p[k])
    got = check(api, q)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.full((90, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    api.nvfp4_lora_apply(q["x"], q["A"], q["B"], q["scaling"], q["ids"], y=q["y"], out=out[:, 32:168])
    assert torch.equal(out[:, 32:168], want[0]) and bool((out[:, :32] == 3).all()) and bool((out[:, 168:] == 3).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_reaches_no_other_adapter(api, bad):
    p = problem(140, 136, 128, 16, 3, "random", seed=7)
    p["ids"][70], p["ids"][71] = 1, -1
    for k in ("x", "y", "dy", "dx"):
        p[k][70:72] = bad
    clean = dict(p, **{k: p[k].clone() for k in ("x", "y", "dy", "dx")})
    for k in ("x", "y", "dy", "dx"):
        clean[k][70:72] = 0
    def run(q):
        out, h = api.nvfp4_lora_apply(q["x"], q["A"], q["B"], q["scaling"], q["ids"], y=q["y"])
        return (out, h) + api.nvfp4_lora_backward(q["dy"], q["x"], h, q["A"], q["B"], q["scaling"], q["ids"], dx=q["dx"])
    got, want = run(p), run(clean)
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[70:72] = False
    for i in (0, 1, 2):
        assert torch.equal(got[i][keep], want[i][keep])
    for i in (3, 4):
        assert torch.equal(got[i][[0, 2]], want[i][[0, 2]])
        assert not bool(torch.isfinite(got[i][1]).all())


def test_an_infinite_h_gives_infinities_where_the_formula_does(api):
    p = problem(1, 64, 64, 16, 1, "one", seed=8)
    p["A"].zero_()
    p["A"][0, 0] = 1.0
    p["x"].fill_(3e38)                       # h[0] overflows to +inf, the other h are 0
    p["B"].fill_(0.0)
    p["B"][0, :, 0] = 1.0
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    assert h[0, 0] == float("inf") and bool((out == float("inf")).all())


def test_many_tokens_in_place_strided_and_with_a_bad_token(api):
    """The forward pass of more tokens than are gathered: out is y, rows are
    slices of wider ones, and a NaN token stays alone."""
    T, K, N, r, n = 333, 264, 200, 24, 4
    p = problem(T, K, N, r, n, "random", seed=21)
    want, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
    f, e = reference(p, h)
    within(want, f["out"], e["out"], "out")
    wide_x = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_y = torch.full((T, N + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    x, y = wide_x[:, 8:8 + K], wide_y[:, 16:16 + N]
    x.copy_(p["x"])
    y.copy_(p["y"])
    got, h2 = api.nvfp4_lora_apply(x, p["A"], p["B"], p["scaling"], p["ids"], y=y, out=y)
    assert torch.equal(got, want) and torch.equal(h2, h)
    assert bool((wide_y[:, :16] == 3).all()) and bool((wide_y[:, 16 + N:] == 3).all())
    alone, _ = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    zero, _ = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=torch.zeros_like(p["y"]))
    assert torch.equal(alone, zero)
    p["x"][100] = float("nan")
    bad, _ = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
    keep = torch.arange(T, device="cuda") != 100
    assert torch.equal(bad[keep], want[keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [130, 300])
def test_a_bad_adapter_reaches_no_other_token(api, bad, T):
    p = problem(T, 72, 72, 16, 3, "random", seed=22)
    args = lambda q: (q["x"], q["A"], q["B"], q["scaling"], q["ids"])   # noqa: E731
    want, h = api.nvfp4_lora_apply(*args(p), y=p["y"])
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, *args(p)[1:], dx=p["dx"])
    q = dict(p, A=p["A"].clone(), B=p["B"].clone())
    q["A"][1] = bad
    q["B"][1] = bad
    others = p["ids"] != 1
    got, h2 = api.nvfp4_lora_apply(*args(q), y=p["y"])
    gx, gA, gB = api.nvfp4_lora_backward(p["dy"], p["x"], h2, *args(q)[1:], dx=p["dx"])
    assert torch.equal(got[others], want[others]) and torch.equal(gx[others], dx[others])
    assert torch.equal(gA[[0, 2]], dA[[0, 2]]) and torch.equal(gB[[0, 2]], dB[[0, 2]])


@pytest.mark.parametrize("T", [40, 300])
def test_parts_of_the_results_through_the_c_abi(api, T):
    """h may stay in the workspace; dx, dA and dB are each optional."""
    L = api.L
    K, N, r, n = 136, 200, 24, 3
    p = problem(T, K, N, r, n, "random", seed=23)
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], dx=p["dx"], out_dtype=FP32)
    d = {k: v.data_ptr() for k, v in p.items()}
    stream = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(L.nvfp4_lora_workspace_size(T, K, N, r, n, 1), dtype=torch.uint8, device="cuda")
    got = torch.empty_like(out)
    assert L.nvfp4_lora_apply(d["x"], K, d["A"], d["B"], d["scaling"], d["ids"], T, K, N, r, n, d["y"], N, got.data_ptr(), N,
                              None, ws.data_ptr(), L.nvfp4_lora_workspace_size(T, K, N, r, n, 0), None, stream) == 0
    assert torch.equal(got, out)
    for want in ("x", "A", "B", "xA", "AB", "xB"):
        gx, gA, gB = torch.empty_like(dx), torch.empty_like(dA), torch.empty_like(dB)
        ws.fill_(0xFF)
        assert L.nvfp4_lora_backward(d["dy"], N, d["x"], K, h.data_ptr(), d["A"], d["B"], d["scaling"], d["ids"], T, K, N, r, n,
                                     d["dx"], K, gx.data_ptr() if "x" in want else None, K,
                                     gA.data_ptr() if "A" in want else None, gB.data_ptr() if "B" in want else None, FP32,
                                     ws.data_ptr(), ws.numel(), None, stream) == 0
        for k, a, b in (("x", gx, dx), ("A", gA, dA), ("B", gB, dB)):
            assert k not in want or torch.equal(a, b), (want, k)


def test_bad_ids_set_the_status(api):
    p = problem(80, 128, 128, 16, 3, "one", seed=9)
    for bad in (3, -2, 1 << 30):
        ids = p["ids"].clone()
        ids[41] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], ids, y=p["y"], status=st)
        assert st.item() == -1 and torch.equal(out[41], p["y"][41])
        st.zero_()
        api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], ids, status=st)
        assert st.item() == -1


def test_no_tokens(api):
    p = problem(0, 128, 64, 16, 2, "none")
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
    assert out.shape == (0, 64) and h.shape == (0, 16)
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"])
    assert dx.shape == (0, 128) and not bool(dA.any()) and not bool(dB.any())


def test_same_call_same_bits(api):
    p = problem(700, 512, 384, 24, 4, "random", seed=10)
    first = check(api, p)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(check(api, p), first))


def test_gradients_against_differences(api):
    """out is linear in A for fixed B and the other way round, so a finite
    step gives the derivative without truncation error; steps and weights are
    small dyadic numbers, exact in bf16.  What is left is the rounding of the
    two outputs to bf16 (half a step each), weighted by dy."""
    T, K, N, r, n = 90, 64, 72, 16, 3
    p = problem(T, K, N, r, n, "runs", seed=11)
    g = torch.Generator().manual_seed(12)
    for k in ("A", "B"):
        p[k] = (torch.randint(-8, 9, p[k].shape, generator=g) / 8).bfloat16().cuda()
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], out_dtype=FP32)
    dy = p["dy"].double()
    for k, grad in (("A", dA), ("B", dB), ("x", dx)):
        d = torch.randint(-1, 2, p[k].shape, generator=g).cuda() / 8
        q = dict(p)
        if k == "x":
            q["x"] = (p["x"].double() + d).bfloat16()
            d = q["x"].double() - p["x"].double()
        else:
            q[k] = (p[k].double() + d).bfloat16()
            assert torch.equal(q[k].double(), p[k].double() + d)
        moved, _ = api.nvfp4_lora_apply(q["x"], q["A"], q["B"], q["scaling"], q["ids"])
        diff = float((dy * (moved.double() - out.double())).sum())
        noise = float((dy.abs() * HALF * (moved.double().abs() + out.double().abs())).sum()) * 1.01
        if k == "x":
            noise += float((HALF * dx.double().abs() * d.abs()).sum())
        assert abs(diff - float((grad.double() * d).sum())) <= noise


def test_beside_the_shared_projection_forward_and_backward(api):
    """As a layer uses them: y = x W^T in NVFP4, the adapters added in place;
    backward: dx of the frozen NVFP4 weight, the adapters' part on top."""
    T, K, N, r, n = 256, 512, 768, 16, 3
    p = problem(T, K, N, r, n, "runs", seed=13)
    w = synthetic.weight(N, K, seed=14).cuda()
    ROW, COL, GEMM = api.NVFP4_ROWWISE, api.NVFP4_COLWISE, api.NVFP4_GEMM_SCALE_LAYOUT
    qw = api.nvfp4_quantize(w, 0, ROW | COL | GEMM)
    qx = api.nvfp4_quantize(p["x"], 1, ROW | GEMM)
    y = api.nvfp4_gemm(qx.codes_row, qx.scales_row, qx.alpha_row, qw.codes_row, qw.scales_row, qw.alpha_row)
    base = y.clone()
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=y, out=y)
    qd = api.nvfp4_quantize(p["dy"], 1, ROW | GEMM)
    dx0 = api.nvfp4_gemm(qd.codes_row, qd.scales_row, qd.alpha_row, qw.codes_col, qw.scales_col, qw.alpha_col)
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], dx=dx0,
                                         out_dtype=FP32)
    f, e = reference(dict(p, y=base, dx=dx0), h)
    within(out, f["out"], e["out"], "out")
    within(dx, f["dx"], e["dx"], "dx")
    within(dA, f["dA"], e["dA"] + 2.0 ** -24 * f["dA"].abs(), "dA")
    within(dB, f["dB"], e["dB"] + 2.0 ** -24 * f["dB"].abs(), "dB")


def test_captured_and_on_two_streams(api):
    p = problem(300, 256, 384, 16, 4, "runs", seed=15)

    def step(q):
        out, h = api.nvfp4_lora_apply(q["x"], q["A"], q["B"], q["scaling"], q["ids"], y=q["y"])
        return (out, h) + api.nvfp4_lora_backward(q["dy"], q["x"], h, q["A"], q["B"], q["scaling"], q["ids"], dx=q["dx"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(p)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(p)
    for kind, s in (("random", 16), ("none", 17), ("one", 18)):
        q = problem(300, 256, 384, 16, 4, kind, seed=s)
        for k in p:
            p[k].copy_(q[k])
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step(q)))
    qs = [problem(300, 256, 384, 16, 4, "random", seed=s) for s in (19, 20)]
    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        res = []
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                res.append(step(q))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for u, v in zip(res, want) for a, b in zip(u, v))


def test_offsets_past_32_bits(api):
    """Rows past 2^31 elements: only the last tokens have an adapter, and their
    results are those of a call on them alone (bounds of both calls)."""
    T, K, N, r, n, last = 150016, 128, 14400, 16, 2, 320
    p = problem(last, K, N, r, n, "random", seed=61)
    first = T - last
    long = dict(p)
    for k, v in (("x", p["x"]), ("y", p["y"]), ("dy", p["dy"]), ("dx", p["dx"])):
        long[k] = torch.zeros((T, v.shape[1]), dtype=torch.bfloat16, device="cuda")
        long[k][first:] = v
    long["ids"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    long["ids"][first:] = p["ids"]
    out, h = api.nvfp4_lora_apply(long["x"], p["A"], p["B"], p["scaling"], long["ids"], y=long["y"], out=long["y"])
    f, e = reference(p, h[first:])
    within(h[first:], f["h"], e["h"], "h")
    within(out[first:], f["out"], e["out"], "out")
    assert not bool(h[:first].any()) and not bool(out[:first].any())
    dx, dA, dB = api.nvfp4_lora_backward(long["dy"], long["x"], h, p["A"], p["B"], p["scaling"], long["ids"], dx=long["dx"],
                                         out_dtype=FP32)
    within(dx[first:], f["dx"], e["dx"], "dx")
    assert not bool(dx[:first].any())
    for got, k in ((dA, "dA"), (dB, "dB")):
        within(got, f[k], e[k] + 2.0 ** -24 * (f[k].abs() + e[k]), k)


def test_on_a_side_stream(api):
    """Calls on a side stream, inputs made on the default one, results read
    after a wait; the workspace of each call is its own."""
    p = problem(300, 256, 512, 24, 3, "random", seed=62)
    want = check(api, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
        got = (out, h) + tuple(api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], dx=p["dx"],
                                                       out_dtype=FP32))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def cut_short(api, call, want, monkeypatch, limit):
    """`call` with the kernels' waits limited to `limit` ns returns; its results
    are `want` or the status says otherwise.  The next call with the usual limit
    gives `want` again."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("NVFP4_WAIT_TIMEOUT_NS", str(limit))
    got = call(st)
    torch.cuda.synchronize()
    monkeypatch.delenv("NVFP4_WAIT_TIMEOUT_NS")
    assert st.item() in (0, api.L.NVFP4_ERR_TIMEOUT)
    assert st.item() != 0 or all(torch.equal(a, b) for a, b in zip(got, want))
    st.zero_()
    assert all(torch.equal(a, b) for a, b in zip(call(st), want)) and st.item() == 0


@pytest.mark.parametrize("limit", [0, 2500])
@pytest.mark.parametrize("r,kind", [(16, "random"), (16, "runs"), (40, "random"), (128, "random")])
def test_waits_that_give_up_end_the_backward_pass(api, monkeypatch, limit, r, kind):
    """Ring waits cut short on purpose, in tiles of several adapters and of
    one: every kernel ends, and the context stays usable."""
    p = problem(5000, 520, 776, r, 3, kind, seed=24)
    _, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    call = lambda st: api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], dx=p["dx"],   # noqa: E731
                                              out_dtype=FP32, status=st)
    want = call(None)
    for _ in range(3):
        cut_short(api, call, want, monkeypatch, limit)


@pytest.mark.parametrize("limit", [0, 2500])
@pytest.mark.parametrize("r,kind", [(16, "random"), (40, "runs"), (128, "random")])
def test_waits_that_give_up_end_the_forward_pass(api, monkeypatch, limit, r, kind):
    p = problem(5000, 1160, 776, r, 3, kind, seed=25)
    call = lambda st: api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"], status=st)   # noqa: E731
    want = call(None)
    for _ in range(3):
        cut_short(api, call, want, monkeypatch, limit)


def same_kind(got, ref, bound, what):
    """NaN where the formula gives NaN, its infinities where it gives those,
    and within the bound elsewhere (where the bound itself is a number)."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what
    at = torch.isfinite(ref) & torch.isfinite(bound)
    within(got[at], ref[at], bound[at], what)


@pytest.mark.parametrize("T", [30, 300, 4200])
@pytest.mark.parametrize("r,kind", [(16, "random"), (24, "runs"), (64, "random"), (128, "runs")])
@pytest.mark.parametrize("where", ["A", "B", "x", "dy"])
@pytest.mark.parametrize("out_dtype", [FP32, BF16])
def test_infinities_stay_infinities(api, T, r, kind, where, out_dtype):
    """An infinite weight, input or gradient of a token's own: the results are
    the formula's in 64 bits, infinities with their signs and NaN only where
    infinities of both signs (or an infinity and a zero) meet."""
    p = problem(T, 72, 136, r, 3, kind, seed=26)
    t = int(torch.nonzero(p["ids"] >= 0)[T // 3])
    a = int(p["ids"][t])
    inf = float("inf")
    if where == "A":
        p["A"][a, 3, 10], p["A"][a, 5, 11] = inf, -inf
    elif where == "B":
        p["B"][a, 20, 1], p["B"][a, 21, 7] = -inf, inf
    elif where == "x":
        p["x"][t, 17] = -inf
    else:
        p["dy"][t, 100] = inf
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"], y=p["y"])
    dx, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], dx=p["dx"],
                                         out_dtype=out_dtype)
    f, e = reference(p, h)
    step = HALF if out_dtype == BF16 else 2.0 ** -24
    for got, k in ((h, "h"), (out, "out"), (dx, "dx")):
        same_kind(got, f[k], e[k], k)
    for got, k in ((dA, "dA"), (dB, "dB")):
        same_kind(got, f[k], e[k] + step * (f[k].abs() + e[k]), k)
    assert any(bool(torch.isinf(f[k]).any()) for k in ("out", "dx", "dA", "dB"))


@pytest.mark.parametrize("T", [30, 300])
def test_products_at_the_ends_of_the_range(api, T):
    """h next to the largest and the smallest fp32 numbers: its leading bf16
    part is neither an infinity nor zero."""
    p = problem(T, 64, 64, 16, 1, "one", seed=27)
    p["A"].zero_()
    p["A"][0, 0, 0] = p["A"][0, 1, 1] = p["A"][0, 2, 2] = 1.0
    p["x"].zero_()
    p["x"][:, 0] = 3.3895e38                     # the largest bf16 number, and half of its last step on top
    p["A"][0, 0, 3], p["x"][:, 3] = 1.0, 2.0 ** 119
    p["x"][:, 1] = 2.0 ** -133
    p["A"][0, 1, 1] = 2.0 ** -2                  # h[1] = 2^-135
    p["B"].zero_()
    p["B"][0, :, 0] = 2.0 ** -10
    p["B"][0, 5, 1] = float("inf")
    p["scaling"].fill_(1.0)
    out, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    assert bool(torch.isfinite(h).all()) and float(h[0, 0]) > 3.3961e38 and float(h[0, 1]) == 2.0 ** -135
    ref = h.double() @ p["B"][0].double().t()
    assert bool((out[:, 5] == float("inf")).all())
    keep = torch.arange(64, device="cuda") != 5
    within(out[:, keep], ref[:, keep], (2.0 ** -17 + 35 * U + HALF) * 1.01 * ref[:, keep].abs(), "out")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -1.0])
@pytest.mark.parametrize("T", [64, 5000])
@pytest.mark.parametrize("out_dtype", [FP32, BF16])
def test_an_adapter_without_tokens_gets_zeros_whatever_its_scale(api, value, T, out_dtype):
    """Slots of a pool that no request uses: their scaling says nothing."""
    p = problem(T, 136, 264, 16, 4, "random", seed=28)
    p["ids"][p["ids"] == 2] = 1
    p["scaling"][2] = value
    p["A"][2], p["B"][2] = value, value
    _, h = api.nvfp4_lora_apply(p["x"], p["A"], p["B"], p["scaling"], p["ids"])
    _, dA, dB = api.nvfp4_lora_backward(p["dy"], p["x"], h, p["A"], p["B"], p["scaling"], p["ids"], out_dtype=out_dtype)
    for d in (dA, dB):
        assert bool((d[2] == 0).all()) and not bool(torch.signbit(d[2]).any())
        assert bool(torch.isfinite(d).all()) and bool(d[1].any())


@pytest.mark.parametrize("r", [8, 24, 32, 56, 64, 96, 128])
@pytest.mark.parametrize("T,kind", [(300, "random"), (4200, "runs"), (8300, "random")])
@pytest.mark.parametrize("out_dtype", [FP32, BF16])
def test_every_rank_class_and_gradient_type(api, r, T, kind, out_dtype):
    """Gradients in both types for every padded rank, with the rows in one
    range and in several (whose sums are added by a kernel of their own)."""
    check(api, problem(T, 136, 264, r, 3, kind, seed=29), out_dtype=out_dtype)
