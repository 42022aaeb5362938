"""Routing, dispatch and the few-row products where their fast paths end.
Tolerances as in test_gpu_experts.py."""
import threading

import pytest
import torch

from test_gpu_experts import (INF, PAIR, RENORM, SIGMOID, SOFTMAX, api, check_gemv, check_route, choices,  # noqa: F401
                              random_weight, rows_of, sort_reference)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def tied_rows(T, E, k, step, seed):
    """Logits far apart but for three neighbours at the end of the k choices:
    two equal ones and one `step` units in the last place away, in any order."""
    g = torch.Generator().manual_seed(seed)
    order = torch.argsort(torch.rand((T, E), generator=g), 1)
    z = torch.zeros((T, E))
    z.scatter_(1, order, (4.0 - torch.arange(E) * (8.0 / E)).expand(T, E).contiguous())
    at = order[:, k - 1:k + 2]
    v = torch.round(z.gather(1, at[:, 1:2]) * 32) / 32 + 0.0
    odd = torch.randint(0, 3, (T, 1), generator=g)
    three = v.expand(T, 3).clone()
    three.scatter_(1, odd, (v.double() + step * (2.0 ** torch.floor(torch.log2(v.double().abs().clamp(min=0.03)))) * 2.0 ** -23).float())
    return z.scatter_(1, at, three)


@pytest.mark.parametrize("E,k", [(5, 1), (33, 1), (64, 1), (64, 6), (100, 3), (128, 8), (160, 2), (256, 8), (300, 20), (500, 1), (700, 9), (1024, 32)])
@pytest.mark.parametrize("step", [1, 3, -2])
def test_route_equal_experts_at_the_end_hide_no_better_one(api, E, k, step):
    z = tied_rows(150, E, k, step, seed=E + k)
    check_route(api, z, k, SOFTMAX, 0)
    check_route(api, z, k, SIGMOID, RENORM)
    bias = torch.zeros(E)
    check_route(api, z, k, SIGMOID, 0, bias=bias)
    check_route(api, z, k, SOFTMAX, RENORM, bias=bias)


@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (512, 4)])
def test_route_many_equal_experts_around_the_end(api, E, k):
    """Rows of one value but for one or two experts a step above or below."""
    g = torch.Generator().manual_seed(E)
    z = torch.full((120, E), 1.5)
    z[40:80] = torch.tensor([1.5, 1.25])[torch.randint(0, 2, (40, E), generator=g)]
    z[torch.arange(120), torch.randint(0, E, (120,), generator=g)] = 1.5 + 2.0 ** -23
    z[torch.arange(100), torch.randint(0, E, (100,), generator=g)] = 1.5 - 2.0 ** -23
    z[110:] = 0.0
    for bias in (None, torch.zeros(E)):
        check_route(api, z, k, SOFTMAX, 0, bias=bias)
        check_route(api, z, k, SIGMOID, RENORM, bias=bias)
    check_route(api, z, k, SIGMOID, PAIR, groups=8, kept=3)


@pytest.mark.parametrize("E,groups", [(40, 4), (128, 4), (256, 8), (512, 4), (96, 12)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_group_values_past_32_bits(api, E, groups, score):
    """Sums of two biases below -FLT_MAX are still ordered, and stand above a
    group without an open expert; sums above FLT_MAX are as well."""
    n = E // groups
    z = torch.randn((20, E), generator=torch.Generator().manual_seed(E))
    low = torch.finfo(torch.float32).min
    for values in ([-INF, -3.0e38, -2.5e38, -3.2e38], [-3.3e38, low, -3.1e38, -2.0e38], [3.0e38, 2.6e38, -3.0e38, 3.2e38],
                   [-3.0e38, -3.0e38, -INF, -3.0e38]):
        bias = torch.tensor(values).repeat(groups // 4).repeat_interleave(n)
        for kept in (1, 2, groups - 1):
            check_route(api, z, 3, score, PAIR, bias=bias, groups=groups, kept=kept)
    # the second value next to the lowest number
    bias = torch.zeros(E)
    bias[:n] = torch.nextafter(torch.tensor(low), torch.tensor(0.0))
    bias[0] = 2.0
    check_route(api, z, 2, score, PAIR, bias=bias, groups=groups, kept=1)


# ---------------------------------------------------------------------------
# dispatch
# ---------------------------------------------------------------------------
def test_dispatch_from_two_host_threads(api):
    """Calls of different numbers of experts, whose sorts need different
    amounts of shared memory, at once: each thread has its own stream."""
    T, k = 700, 8
    cases = {E: choices(T, k, E, seed=E) for E in (400, 1024, 600, 1000)}
    want = {E: sort_reference(ids, E) for E, ids in cases.items()}
    gpu = {E: ids.cuda() for E, ids in cases.items()}
    failures = []
    start = threading.Barrier(len(cases))

    def work(E):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(400):
                    _, rows, offsets = api.nvfp4_dispatch(None, gpu[E], E)
                assert torch.equal(rows.cpu(), want[E][0]) and torch.equal(offsets.cpu(), want[E][1])
        except Exception as e:   # noqa: BLE001
            failures.append((E, e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(E,)) for E in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


@pytest.mark.parametrize("T,k,E", [(1, 1, 5), (300, 1, 7), (1024, 1, 256), (1023, 2, 16), (2048, 2, 64), (4096, 1, 128), (4095, 1, 1000),
                                   (1365, 3, 8), (4097, 1, 60)])
def test_dispatch_one_or_two_choices(api, T, k, E):
    ids = choices(T, k, E, seed=T, none=0.05)
    x = rows_of(T, 72, seed=T)
    xs, rows, offsets = api.nvfp4_dispatch(x, ids.cuda(), E)
    want_rows, want_offsets = sort_reference(ids, E)
    assert torch.equal(rows.cpu(), want_rows) and torch.equal(offsets.cpu(), want_offsets)
    live = (want_rows.view(-1) >= 0).cuda()
    assert torch.equal(xs[want_rows.view(-1).cuda()[live].long()], x.repeat_interleave(k, 0)[live])


@pytest.mark.parametrize("T,k,launches", [(64, 8, 1), (512, 8, 1), (1024, 1, 1), (1024, 2, 1), (2048, 1, 2), (4096, 1, 2), (2048, 2, 2),
                                          (1024, 4, 2), (682, 6, 2), (128, 32, 2), (700, 8, 2), (1, 32, 1)])
def test_dispatch_goes_by_rounds_and_pairs(api, T, k, launches):
    """One launch where its count is the cheaper one, else sort and copy."""
    from nvfp4_block_quantization_amax_b200 import _lib
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the sizes are those of 148 SMs")
    ids, x = choices(T, k, 64, seed=T).cuda(), rows_of(T, 64, seed=T)
    before = _lib.nvfp4_launch_count()
    api.nvfp4_dispatch(x, ids, 64)
    assert _lib.nvfp4_launch_count() - before == launches


# ---------------------------------------------------------------------------
# few-row products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hot,T,k,E", [(9, 40, 1, 64), (40, 64, 2, 128), (300, 500, 1, 300)])
def test_gemv_a_hot_expert_among_many(api, hot, T, k, E):
    """More than 8 rows of one weight where few are likely, in several passes."""
    W, sW, alpha, w = random_weight(E, 128, 192, seed=E)
    ids = choices(T, k, E, seed=T, none=0.1)
    ids.view(-1)[torch.randperm(T * k, generator=torch.Generator().manual_seed(hot))[:hot]] = E - 2
    for rows in (T, T * k):
        x = rows_of(rows, 192, seed=rows)
        check_gemv(api, x, W, sW, alpha, w, ids.cuda(), api.NVFP4_OUT_DTYPE_FP32)


@pytest.mark.parametrize("T,k,E,K", [(20, 2, 4, 448), (36, 1, 4, 64), (30, 2, 5, 1024), (45, 1, 3, 320), (64, 2, 8, 128), (90, 1, 2, 192),
                                      (14, 1, 2, 1152), (16, 2, 2, 1152), (40, 1, 2, 1088), (60, 1, 2, 1088), (150, 1, 3, 1088)])
def test_gemv_7_to_50_rows_of_each_expert(api, T, k, E, K):
    W, sW, alpha, w = random_weight(E, 256, K, seed=E + K)
    ids = choices(T, k, E, seed=T, none=0.05).cuda()
    for rows in (T, T * k):
        x = rows_of(rows, K, seed=rows)
        check_gemv(api, x, W, sW, alpha, w, ids, api.NVFP4_OUT_DTYPE_FP32)
        check_gemv(api, x, W, sW, alpha, w, ids, api.NVFP4_OUT_DTYPE_BF16)


@pytest.mark.parametrize("P", [25, 31, 32, 40, 65, 72, 100])
@pytest.mark.parametrize("N,K", [(128, 64), (128, 14336), (4096, 1088)])
def test_gemv_25_rows_and_more(api, P, N, K):
    W, sW, alpha, w = random_weight(1, N, K, seed=N + K)
    check_gemv(api, rows_of(P, K, seed=P), W, sW, alpha, w, None, api.NVFP4_OUT_DTYPE_FP32)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_sizes_are_refused_before_results_of_them_are_allocated(api):
    """Host-side refusals: nothing is launched, and no memory asked for."""
    z = torch.zeros((64, 64), device="cuda")
    ids = torch.zeros((1 << 16, 32), dtype=torch.int32, device="cuda")
    W, sW, alpha, _ = random_weight(1, 128, 64, seed=1)
    x = torch.zeros((1 << 16, 64), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    used = torch.cuda.memory_allocated()
    for call in [lambda k=k: api.nvfp4_route(z, k) for k in (-1, 0, 33, 1 << 33, 1 << 70)] + \
                [lambda E=E: api.nvfp4_dispatch(None, ids[:8], E) for E in (-5, 0, 1025, 1 << 40, 1 << 70)] + \
                [lambda: api.nvfp4_gemv(x, W[0], sW[0], alpha), lambda: api.nvfp4_gemv(x, W, sW, alpha, ids=ids),
                 lambda: api.nvfp4_gemv(x[:1025], W, sW, alpha, ids=ids[:1025, :1].contiguous())]:
        with pytest.raises(api.NVFP4Error) as e:
            call()
        assert e.value.status == -2
    assert torch.cuda.max_memory_allocated() - used < 1 << 20
