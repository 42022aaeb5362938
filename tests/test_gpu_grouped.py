"""Ragged groups on the GPU: nvfp4_quantize_grouped, nvfp4_dequantize_grouped,
nvfp4_gemm_grouped and nvfp4_gemm_grouped_wgrad.

Quantization is bit-exact with the CPU oracle run on every group as a tensor
of its own (padded with zero rows to a multiple of 64, stream id + group).
The products are compared with 64-bit products of the same operands.

Tolerance of a product, element by element: products of E2M1 x E4M3 values are
exact in fp32, so the error is that of the accumulation, at most one step of
2^-23 of the running magnitude (truncation included) for each of at most K
additions, plus the three roundings of the scales: (K + 3) 2^-23 sum |a b|;
a bf16 result adds half a step, 2^-8 of its magnitude.  The whole fp32 result
keeps the plain GEMM's relative Frobenius error of 1e-5.
"""
import numpy as np
import pytest
import torch

import oracle
from nvfp4_block_quantization_amax_b200 import synthetic

pytestmark = pytest.mark.gpu

ROW, COL, GEMM, RHT, HEADROOM, INV, BF = 0x1, 0x2, 0x20, 0x40, 0x200, 0x80, 0x100
MODES = {"rtn": 0, "four_six": 1, "rht_sr": 2, "ms_eden": 3, "rht_sr_hw": 4}
FP32, BF16 = 1, 0
COUNTS = {
    "one row": [1],
    "ragged": [37, 0, 1, 64, 65, 200, 0, 15],
    "whole": [128, 256, 64],
    "empty ends": [0, 0, 5, 0],
    "many": [(7 * i) % 23 for i in range(70)],
}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_quantization_amax_b200 import api as _api
    return _api


def starts(counts, step=1):
    out = [0]
    for c in counts:
        out.append(out[-1] + -(-c // step) * step)
    return out


def capacity(T, E, step):
    return (T + min(T, E) * (step - 1)) // step * step


def offsets_of(counts, first=0):
    return torch.tensor([first + s for s in starts(counts)], dtype=torch.int32, device="cuda")


def gemm_to_plain(flat, rows, kb):
    m = np.arange(rows)[:, None]
    j = np.arange(kb)[None, :]
    return np.asarray(flat)[((m >> 7) * (kb >> 2) + (j >> 2)) * 512 + (m & 31) * 16 + ((m >> 5) & 3) * 4 + (j & 3)]


def plain_to_gemm(s):
    rows, kb = s.shape
    flat = np.empty(rows * kb, np.uint8)
    m = np.arange(rows)[:, None]
    j = np.arange(kb)[None, :]
    flat[((m >> 7) * (kb >> 2) + (j >> 2)) * 512 + (m & 31) * 16 + ((m >> 5) & 3) * 4 + (j & 3)] = s
    return flat


def rows_of(T, C, seed):
    t = synthetic.normal_with_channel_outliers(max(T, 1), C, seed=seed)[:T].float()
    g = torch.Generator().manual_seed(seed)
    return (t * torch.exp2(torch.randint(-5, 6, (T, 1), generator=g).float())).bfloat16()


def oracle_group(x, mode, flags, seed, sid):
    """The oracle on one group's rows, padded to 64 with zero rows."""
    pad = torch.zeros((-len(x) % 64, x.shape[1]), dtype=torch.bfloat16)
    return oracle.quantize(synthetic.bf16_bits(torch.cat([x, pad])), mode, flags & (ROW | COL | RHT | HEADROOM),
                           seed=seed, stream_id=sid)


def check_quantize(api, x, counts, mode, flags, first=0, seed=5, sid=3):
    T, C = x.shape
    E = len(counts)
    q = api.nvfp4_quantize_grouped(x.cuda(), offsets_of(counts, first), mode, flags, seed=seed, stream_id=sid)
    torch.cuda.synchronize()
    at, p128, p64 = starts(counts), starts(counts, 128), starts(counts, 64)
    if flags & ROW:
        srow = gemm_to_plain(q.scales_row.cpu().numpy(), capacity(T, E, 128), C // 16)
    if flags & COL:
        kcap = capacity(T, E, 64)
        scol = gemm_to_plain(q.scales_col.cpu().numpy(), C, kcap // 16)
    for e, n in enumerate(counts):
        if n == 0:
            for side, bit in (("row", ROW), ("col", COL)):
                if flags & bit:
                    assert float(getattr(q, f"alpha_{side}")[e]) == 0.0
            continue
        o = oracle_group(x[first + at[e]:first + at[e + 1]], mode, flags, seed, sid + e)
        if flags & ROW:
            assert float(q.alpha_row[e]) == o["alpha_row"], e
            assert float(q.amax[0, e]) == o["amax_row"], e
            assert np.array_equal(q.codes_row[first + at[e]:first + at[e + 1]].cpu().numpy(), o["codes_row"][:n]), e
            assert np.array_equal(srow[p128[e]:p128[e] + n], o["scales_row"][:n]), e
        if flags & COL:
            assert float(q.alpha_col[e]) == o["alpha_col"], e
            assert float(q.amax[1, e]) == o["amax_col"], e
            assert np.array_equal(q.codes_col[:, p64[e] // 2:p64[e + 1] // 2].cpu().numpy(), o["codes_col"]), e
            assert np.array_equal(scol[:, p64[e] // 16:p64[e + 1] // 16], o["scales_col"]), e
    return q


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("orient", ["row", "col", "dual"])
def test_quantize_every_mode_and_orientation(api, mode, orient):
    counts = COUNTS["ragged"]
    flags = {"row": ROW, "col": COL, "dual": ROW | COL}[orient]
    check_quantize(api, rows_of(sum(counts), 384, 11), counts, MODES[mode], flags)


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("flags", [ROW | COL, ROW | COL | RHT | HEADROOM])
def test_quantize_group_shapes(api, counts, flags):
    counts = COUNTS[counts]
    check_quantize(api, rows_of(sum(counts), 128, 12), counts, MODES["four_six"], flags)


@pytest.mark.parametrize("C", [64, 192, 1088])
def test_quantize_row_widths(api, C):
    check_quantize(api, rows_of(100, C, 13), [3, 97], MODES["rtn"], ROW)


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("counts,C", [([1], 64), ([3, 0, 1, 20], 192), ([0, 0, 64, 0], 4096), ([2] * 30, 14336 // 7),
                                      ([5, 0, 40], 14336)])
def test_quantize_few_rows(api, mode, counts, C):
    """Rowwise and at most 64 rows: the single-launch path, every mode."""
    x = rows_of(sum(counts) + 2, C, 17)
    check_quantize(api, x, counts, MODES[mode], ROW, first=1)
    check_quantize(api, x, counts, MODES[mode], ROW | RHT | HEADROOM, first=1)


def test_quantize_few_rows_strided_and_nonfinite(api):
    x = rows_of(12, 512, 18)
    wide = torch.zeros((12, 648), dtype=torch.bfloat16, device="cuda")
    wide[:, 64:576] = x.cuda()
    got = api.nvfp4_quantize_grouped(wide[:, 64:576], offsets_of([5, 0, 7]), 1, ROW)
    want = check_quantize(api, x, [5, 0, 7], 1, ROW, seed=0, sid=0)
    assert torch.equal(got.codes_row, want.codes_row) and torch.equal(got.alpha_row, want.alpha_row)
    for flags in (ROW, ROW | RHT):
        y = x.clone()
        y[9, 500] = float("nan")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = api.nvfp4_quantize_grouped(y.cuda(), offsets_of([5, 0, 7]), 0, flags, status=st)
        assert st.item() == -4 and float(q.alpha_row[0]) > 0.0
        st.zero_()
        api.nvfp4_quantize_grouped(y.cuda(), offsets_of([5, 0, 4]), 0, flags, status=st)
        assert st.item() == 0


def test_quantize_strided_rows_and_rows_of_no_group(api):
    x = rows_of(90, 512, 14)
    wide = torch.zeros((90, 640), dtype=torch.bfloat16, device="cuda")
    wide[:, 64:576] = x.cuda()
    counts = [20, 0, 41]                                  # rows 7 .. 67 of 90
    q = api.grouped_alloc_outputs(90, 512, 3, ROW | COL, torch.device("cuda"))
    q.codes_row.fill_(0xA5)
    api.nvfp4_quantize_grouped(wide[:, 64:576], offsets_of(counts, 7), 1, ROW | COL, seed=2, stream_id=1, out=q)
    want = check_quantize(api, x, counts, 1, ROW | COL, first=7, seed=2, sid=1)
    assert torch.equal(q.codes_row[7:68], want.codes_row[7:68]) and torch.equal(q.alpha_col, want.alpha_col)
    assert bool((q.codes_row[:7] == 0xA5).all()) and bool((q.codes_row[68:] == 0xA5).all())


def test_quantize_without_rows(api):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    q = api.nvfp4_quantize_grouped(x, offsets_of([0, 0]), 0, ROW | COL)
    assert q.alpha_row.tolist() == [0.0, 0.0] and q.alpha_col.tolist() == [0.0, 0.0]


def test_quantize_zero_group_tiny_and_nonfinite(api):
    x = rows_of(60, 128, 15)
    x[10:30] = 0.0                                        # group 1: all zeros
    x[30:] *= 2.0 ** -100                                 # group 2: tiny, its own scale
    check_quantize(api, x, [10, 20, 30], 1, ROW | COL)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[35, 7] = bad
        for flags in (ROW, ROW | COL, ROW | COL | RHT, COL | RHT):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            api.nvfp4_quantize_grouped(y.cuda(), offsets_of([10, 20, 30]), 0, flags, status=st)
            assert st.item() == -4
            st.zero_()
            api.nvfp4_quantize_grouped(y.cuda(), offsets_of([10, 20]), 0, flags, status=st)   # not in any group
            assert st.item() == 0


@pytest.mark.parametrize("orient", [ROW, COL])
@pytest.mark.parametrize("extra", [0, BF, RHT, RHT | BF])
def test_dequantize(api, orient, extra):
    counts = COUNTS["ragged"]
    T, C = sum(counts) + 9, 256
    x = rows_of(T, C, 16)
    q = api.nvfp4_quantize_grouped(x.cuda(), offsets_of(counts, 4), 0, orient | (extra & RHT), seed=9)
    flags = orient | (extra & BF) | (INV if extra & RHT else 0)
    y = torch.full((T, C), 7.0, dtype=torch.bfloat16 if extra & BF else torch.float32, device="cuda")
    side = ("codes_row", "scales_row", "alpha_row") if orient == ROW else ("codes_col", "scales_col", "alpha_col")
    api.nvfp4_dequantize_grouped(*(getattr(q, k) for k in side), offsets_of(counts, 4), T, C, flags, seed=9, out=y)
    at = starts(counts)
    for e, n in enumerate(counts):
        if n == 0:
            continue
        o = oracle_group(x[4 + at[e]:4 + at[e + 1]], 0, orient | (extra & RHT), 9, e)
        k = "row" if orient == ROW else "col"
        rows, cols = (n + -n % 64, C) if orient == ROW else (C, n + -n % 64)
        want = oracle.dequantize(o[f"codes_{k}"], o[f"scales_{k}"], o[f"alpha_{k}"], rows, cols,
                                 flags=oracle.INVERSE_RHT if extra & RHT else 0, seed=9)
        want = torch.from_numpy(want if orient == ROW else np.ascontiguousarray(want.T))[:n]
        assert torch.equal(y[4 + at[e]:4 + at[e + 1]].cpu(), want.to(y.dtype)), e
    assert bool((y[:4] == 7).all()) and bool((y[4 + at[-1]:] == 7).all())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def values(codes, scales):
    """q * Delta of a plain operand in 64 bits."""
    R, K2 = codes.shape
    return torch.from_numpy(oracle.dequantize(np.ascontiguousarray(codes), np.ascontiguousarray(scales), 1.0, R,
                                              2 * K2)).double()


def close(got, a, b, ab, K, fp32):
    """got against ab * a @ b^T, element by element (see the head of this file)."""
    got = got.double().cpu()
    ref = a @ b.t() * ab
    bound = (K + 3) * 2.0 ** -23 * (a.abs() @ b.abs().t()) * abs(ab)
    if fp32:
        n = float(ref.norm())
        assert float((got - ref).norm()) <= 1e-5 * n or n == 0
    else:
        bound = bound + torch.finfo(torch.bfloat16).eps / 2 * (ref.abs() + bound)
    assert bool(((got - ref).abs() <= bound).all()), float(((got - ref).abs() - bound).max())


def weights(api, E, N, K, seed):
    w = synthetic.weight(E * N, K, seed=seed).cuda()
    qs = [api.nvfp4_quantize(w[e * N:(e + 1) * N], 0, ROW | GEMM) for e in range(E)]
    return (torch.stack([q.codes_row for q in qs]), torch.cat([q.scales_row for q in qs]),
            torch.cat([q.alpha_row for q in qs]))


def check_gemm(api, counts, N, K, fp32, seed=21, first=0, behind=0, ldd=None):
    T, E = first + sum(counts) + behind, len(counts)
    q = api.nvfp4_quantize_grouped(rows_of(T, K, seed).cuda(), offsets_of(counts, first), 1, ROW)
    B, sB, aB = weights(api, E, N, K, seed + 1)
    dt = torch.float32 if fp32 else torch.bfloat16
    buf = torch.full((T, ldd or N), 3.0, dtype=dt, device="cuda")
    out = buf[:, :N]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.nvfp4_gemm_grouped(q.codes_row, q.scales_row, q.alpha_row, B, sB, aB, offsets_of(counts, first),
                           out_dtype=FP32 if fp32 else BF16, out=out, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    srow = gemm_to_plain(q.scales_row.cpu().numpy(), capacity(T, E, 128), K // 16)
    at, p128 = starts(counts), starts(counts, 128)
    for e, n in enumerate(counts):
        if n == 0:
            continue
        rows = slice(first + at[e], first + at[e + 1])
        a = values(q.codes_row[rows].cpu().numpy(), srow[p128[e]:p128[e] + n])
        b = values(B[e].cpu().numpy(), gemm_to_plain(sB.view(E, -1)[e].cpu().numpy(), N, K // 16))
        close(out[rows], a, b, float(q.alpha_row[e]) * float(aB[e]), K, fp32)
    assert bool((buf[:first] == 3).all()) and bool((buf[first + at[-1]:] == 3).all())
    assert bool((buf[:, N:] == 3).all())


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 64), ([1], 256, 256), ([3, 0, 5], 384, 320), ([256], 256, 512), ([300, 1, 0, 129], 256, 192),
    ([16, 17, 15, 31, 33], 640, 1088), ([0, 0, 2], 128, 128), ([513, 255, 257], 384, 640),
    ([32, 33, 127, 128, 129, 0, 300], 128, 320), ([600], 256, 64), ([79, 81, 79], 128, 256), ([81, 81, 81], 384, 256),
])
def test_gemm_shapes(api, counts, N, K, fp32):
    check_gemm(api, counts, N, K, fp32)


def test_gemm_many_groups(api):
    check_gemm(api, COUNTS["many"], 256, 256, True)
    check_gemm(api, [1] * 200, 128, 128, False)


def test_gemm_rows_of_no_group_and_wide_output(api):
    check_gemm(api, [20, 0, 41], 256, 256, False, first=5, behind=11, ldd=320)
    check_gemm(api, [20, 0, 300], 128, 256, True, first=130, behind=3, ldd=132)


def test_gemm_many_tiles_per_pair(api):
    """More tiles than CTA pairs: the ring and the accumulator are reused."""
    check_gemm(api, [700, 300, 0, 1100], 2048, 448, False)


def check_wgrad(api, counts, M, N, fp32, seed=31, mode=0, extra=0):
    T, E = sum(counts), len(counts)
    off = offsets_of(counts)
    qa = api.nvfp4_quantize_grouped(rows_of(T, M, seed).cuda(), off, mode, COL | extra, seed=4)
    qb = api.nvfp4_quantize_grouped(rows_of(T, N, seed + 1).cuda(), off, mode, COL | extra, seed=4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D = api.nvfp4_gemm_grouped_wgrad(qa.codes_col, qa.scales_col, qa.alpha_col, qb.codes_col, qb.scales_col,
                                     qb.alpha_col, off, T, out_dtype=FP32 if fp32 else BF16, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    kcap = capacity(T, E, 64)
    sa = gemm_to_plain(qa.scales_col.cpu().numpy(), M, kcap // 16)
    sb = gemm_to_plain(qb.scales_col.cpu().numpy(), N, kcap // 16)
    p = starts(counts, 64)
    for e, n in enumerate(counts):
        if n == 0:
            assert not bool(D[e].any())
            continue
        k = slice(p[e], p[e + 1])
        a = values(qa.codes_col[:, k.start // 2:k.stop // 2].cpu().numpy(), sa[:, k.start // 16:k.stop // 16])
        b = values(qb.codes_col[:, k.start // 2:k.stop // 2].cpu().numpy(), sb[:, k.start // 16:k.stop // 16])
        close(D[e], a, b, float(qa.alpha_col[e]) * float(qb.alpha_col[e]), p[e + 1] - p[e], fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("counts,M,N", [
    ([1], 128, 128), ([64], 256, 256), ([3, 0, 70], 384, 128), ([300, 1, 0, 129], 256, 640), ([0, 5], 128, 384),
    ([1000, 260, 513], 512, 256),
])
def test_wgrad_shapes(api, counts, M, N, fp32):
    check_wgrad(api, counts, M, N, fp32)


def test_wgrad_many_groups_and_rotation(api):
    check_wgrad(api, COUNTS["many"], 256, 128, True, extra=RHT)
    check_wgrad(api, [100, 0, 900], 1536, 1024, False, mode=3)


def test_wgrad_without_rows(api):
    z = torch.empty((128, 0), dtype=torch.uint8, device="cuda")
    s = torch.empty(0, dtype=torch.uint8, device="cuda")
    al = torch.zeros(2, dtype=torch.float32, device="cuda")
    D = torch.full((2, 128, 128), 5.0, device="cuda")
    api.nvfp4_gemm_grouped_wgrad(z, s, al, z, s, al, offsets_of([0, 0]), 0, out_dtype=FP32, out=D)
    assert not bool(D.any())


def test_bad_offsets_set_the_status_and_write_nothing(api):
    T, C = 64, 128
    x = rows_of(T, C, 41).cuda()
    good = offsets_of([32, 32])
    q = api.nvfp4_quantize_grouped(x, good, 0, ROW | COL)
    B, sB, aB = weights(api, 2, 128, C, 42)
    for bad in ([0, 40, 30], [0, 32, 65], [-1, 32, 64], [70, 70, 70]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        api.nvfp4_gemm_grouped(q.codes_row, q.scales_row, q.alpha_row, B, sB, aB, off, out=out, status=st)
        assert st.item() == -1 and bool((out == 3).all())
        st.zero_()
        api.nvfp4_quantize_grouped(x, off, 0, ROW | COL, status=st)
        assert st.item() == -1
        st.zero_()
        y = torch.full((T, C), 3.0, device="cuda")
        api.nvfp4_dequantize_grouped(q.codes_row, q.scales_row, q.alpha_row, off, T, C, ROW, out=y, status=st)
        assert st.item() == -1 and bool((y == 3).all())
        st.zero_()
        api.nvfp4_gemm_grouped_wgrad(q.codes_col, q.scales_col, q.alpha_col, q.codes_col, q.scales_col, q.alpha_col,
                                     off, T, status=st)
        assert st.item() == -1


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
def expert_layer(api, x, dy, off, W, WT, seed):
    """Forward and backward of one expert layer in NVFP4: returns y, dx, dW."""
    B, sB, aB = W
    Bt, sBt, aBt = WT
    T = x.shape[0]
    qx = api.nvfp4_quantize_grouped(x, off, 1, ROW)
    y = api.nvfp4_gemm_grouped(qx.codes_row, qx.scales_row, qx.alpha_row, B, sB, aB, off)
    qd = api.nvfp4_quantize_grouped(dy, off, 0, ROW | COL | RHT, seed=seed)
    dx = api.nvfp4_gemm_grouped(qd.codes_row, qd.scales_row, qd.alpha_row, Bt, sBt, aBt, off)
    qw = api.nvfp4_quantize_grouped(x, off, 0, COL | RHT, seed=seed)
    dW = api.nvfp4_gemm_grouped_wgrad(qd.codes_col, qd.scales_col, qd.alpha_col, qw.codes_col, qw.scales_col,
                                      qw.alpha_col, off, T)
    return y, dx, dW


def make_layer(api, E, N, K, seed):
    w = synthetic.weight(E * N, K, seed=seed).cuda()
    qf = [api.nvfp4_quantize(w[e * N:(e + 1) * N], 0, ROW | GEMM) for e in range(E)]
    qb = [api.nvfp4_quantize(w[e * N:(e + 1) * N], 0, COL | GEMM | RHT, seed=77) for e in range(E)]
    W = (torch.stack([q.codes_row for q in qf]), torch.cat([q.scales_row for q in qf]), torch.cat([q.alpha_row for q in qf]))
    WT = (torch.stack([q.codes_col for q in qb]), torch.cat([q.scales_col for q in qb]), torch.cat([q.alpha_col for q in qb]))
    return w.view(E, N, K), W, WT


def test_expert_layer_forward_backward(api):
    """The layer against 64-bit products of the unquantized tensors: NVFP4
    keeps about 10% of the norm as error per operand (4 mantissa steps per
    binade: rms relative rounding error near 0.1), so two operands stay below
    0.25; a product with a wrong group, row or scale is off by order 1."""
    counts = [150, 0, 40, 1, 129]
    T, N, K, E = sum(counts), 384, 256, 5
    x = rows_of(T, K, 51).clamp(-50, 50).cuda()
    dy = (torch.randn((T, N), generator=torch.Generator().manual_seed(52)) * 1e-3).bfloat16().cuda()
    w, W, WT = make_layer(api, E, N, K, 53)
    off = offsets_of(counts)
    y, dx, dW = expert_layer(api, x, dy, off, W, WT, seed=77)
    at = starts(counts)
    for e, n in enumerate(counts):
        if n == 0:
            assert not bool(dW[e].any())
            continue
        r = slice(at[e], at[e + 1])
        for got, ref in ((y[r], x[r].double() @ w[e].double().t()), (dx[r], dy[r].double() @ w[e].double()),
                         (dW[e], dy[r].double().t() @ x[r].double())):
            assert float((got.double() - ref).norm() / ref.norm()) < 0.25


def test_expert_layer_captured_with_changing_offsets(api):
    """One graph, replayed with other inputs and other group sizes in place."""
    T, N, K, E = 200, 256, 128, 4
    _, W, WT = make_layer(api, E, N, K, 61)
    x = rows_of(T, K, 62).cuda()
    dy = rows_of(T, N, 63).cuda()
    off = offsets_of([50, 50, 50, 50])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        expert_layer(api, x, dy, off, W, WT, 77)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = expert_layer(api, x, dy, off, W, WT, 77)
    for counts, s in (([7, 0, 64, 129], 64), ([200, 0, 0, 0], 65), ([0, 1, 2, 3], 66)):
        x.copy_(rows_of(T, K, s))
        dy.copy_(rows_of(T, N, s + 10))
        off.copy_(offsets_of(counts))
        for t in got:
            t.zero_()
        g.replay()
        want = expert_layer(api, x, dy, off, W, WT, 77)
        n = sum(counts)
        assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:n], want[1][:n])
        assert torch.equal(got[2], want[2])
        assert not bool(got[0][n:].any())


def test_two_streams_at_once(api):
    counts = [100, 0, 33, 67]
    x = [rows_of(200, 256, s).cuda() for s in (71, 72)]
    off = offsets_of(counts)
    B, sB, aB = weights(api, 4, 256, 256, 73)

    def pass_(t):
        q = api.nvfp4_quantize_grouped(t, off, 1, ROW)
        return api.nvfp4_gemm_grouped(q.codes_row, q.scales_row, q.alpha_row, B, sB, aB, off)

    want = [pass_(t) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for t, s in zip(x, streams):
            with torch.cuda.stream(s):
                got.append(pass_(t))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# buffers as they come, and sizes past 32 bits
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("counts", [[37, 0, 1, 64, 65], [300, 0, 129, 200]])
def test_bytes_of_no_group_do_not_matter(api, counts):
    """Outputs full of 0xFF (codes of -6, scales and alphas of NaN) before the
    call: the products and the decoded rows are those of zeroed outputs."""
    T, C, N, E = sum(counts), 256, 384, len(counts)
    x, g = rows_of(T, C, 41).cuda(), rows_of(T, N, 42).cuda()
    off, B = offsets_of(counts), weights(api, E, N, C, 43)
    got = []
    for fill in (0xFF, 0):
        qs = []
        for t in (x, g):
            q = api.grouped_alloc_outputs(T, t.shape[1], E, ROW | COL, t.device)
            for b in (q.codes_row, q.scales_row, q.codes_col, q.scales_col, q.alpha_row, q.alpha_col, q.amax):
                b.view(torch.uint8).fill_(fill)
            qs.append(api.nvfp4_quantize_grouped(t, off, 1, ROW | COL, out=q))
        qx, qg = qs
        got.append((api.nvfp4_gemm_grouped(qx.codes_row, qx.scales_row, qx.alpha_row, *B, off),
                    api.nvfp4_gemm_grouped_wgrad(qg.codes_col, qg.scales_col, qg.alpha_col, qx.codes_col, qx.scales_col,
                                                 qx.alpha_col, off, T),
                    api.nvfp4_dequantize_grouped(qx.codes_row, qx.scales_row, qx.alpha_row, off, T, C, ROW),
                    api.nvfp4_dequantize_grouped(qx.codes_col, qx.scales_col, qx.alpha_col, off, T, C, COL)))
    for a, b in zip(*got):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


def test_offsets_past_32_bits_quantize(api):
    """More than 2^31 elements: the last group is that of a call of its own."""
    T, C, last = 139000, 16384, 1000
    x = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    x[:] = rows_of(1000, C, 51).cuda().repeat(139, 1)
    off = torch.tensor([0, 70001, T - last, T], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, last], dtype=torch.int32, device="cuda")
    q = api.nvfp4_quantize_grouped(x, off, 1, ROW | COL, stream_id=0)
    own = api.nvfp4_quantize_grouped(x[T - last:].clone(), tail, 1, ROW | COL, stream_id=2)
    assert float(q.alpha_row[2]) == float(own.alpha_row[0]) and float(q.alpha_col[2]) == float(own.alpha_col[0])
    assert torch.equal(q.codes_row[T - last:], own.codes_row)
    at = -(-70001 // 64) * 32 + -(-(T - last - 70001) // 64) * 32
    assert torch.equal(q.codes_col[:, at:at + own.codes_col.shape[1]], own.codes_col)
    for side, bit in (("row", ROW), ("col", COL)):
        y = api.nvfp4_dequantize_grouped(*(getattr(q, f"{k}_{side}") for k in ("codes", "scales", "alpha")), off, T, C,
                                         bit | BF)
        z = api.nvfp4_dequantize_grouped(*(getattr(own, f"{k}_{side}") for k in ("codes", "scales", "alpha")), tail, last, C,
                                         bit | BF)
        assert torch.equal(y[T - last:], z)
        del y


def test_offsets_past_32_bits_products(api):
    """Results and weights of more than 2^31 elements or bytes: the last group
    against its own product, which has one group and the same tiles."""
    T, N, K, last = 139000, 16384, 64, 1000
    x = rows_of(1000, K, 52).cuda().repeat(139, 1)
    off = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, last], dtype=torch.int32, device="cuda")
    q = api.nvfp4_quantize_grouped(x, off, 0, ROW)
    own = api.nvfp4_quantize_grouped(x[T - last:], tail, 0, ROW)
    B, sB, aB = weights(api, 2, N, K, 53)
    D = api.nvfp4_gemm_grouped(q.codes_row, q.scales_row, q.alpha_row, B, sB, aB, off, out_dtype=FP32)
    want = api.nvfp4_gemm_grouped(own.codes_row, own.scales_row, own.alpha_row, B[1:].contiguous(), sB[N * K // 16:],
                                  aB[1:], tail, out_dtype=FP32)
    assert torch.equal(D[T - last:], want)
    del D, x
    # a column of D per expert row: E M N elements, few tokens
    E, M = 33, 8192
    counts = [3] * E
    g = rows_of(sum(counts), M, 54).cuda()
    qc = api.nvfp4_quantize_grouped(g, offsets_of(counts), 0, COL)
    one = api.nvfp4_quantize_grouped(g[-3:].clone(), offsets_of([3]), 0, COL)
    W = api.nvfp4_gemm_grouped_wgrad(*(t for _ in range(2) for t in (qc.codes_col, qc.scales_col, qc.alpha_col)),
                                     offsets_of(counts), sum(counts))
    assert torch.equal(W[-1], api.nvfp4_gemm_grouped_wgrad(
        *(t for _ in range(2) for t in (one.codes_col, one.scales_col, one.alpha_col)), offsets_of([3]), 3)[0])
    del W
    # weights of more than 2^31 bytes of codes, few tokens each
    E, N, K = 40, 8192, 16384
    w = synthetic.weight(N, K, seed=55).cuda()
    qw = api.nvfp4_quantize(w, 0, ROW | GEMM)
    B = qw.codes_row[None].repeat(E, 1, 1)
    sB, aB = qw.scales_row.repeat(E), qw.alpha_row.repeat(E)
    xs = rows_of(2 * E, K, 56).cuda()
    q = api.nvfp4_quantize_grouped(xs, offsets_of([2] * E), 0, ROW)
    own = api.nvfp4_quantize_grouped(xs[-2:].clone(), offsets_of([2]), 0, ROW)
    D = api.nvfp4_gemm_grouped(q.codes_row, q.scales_row, q.alpha_row, B, sB, aB, offsets_of([2] * E))
    want = api.nvfp4_gemm_grouped(own.codes_row, own.scales_row, own.alpha_row, B[:1], qw.scales_row, qw.alpha_row,
                                  offsets_of([2]))
    assert torch.equal(D[-2:], want)


@pytest.mark.parametrize("T", [40, 64, 300])
@pytest.mark.parametrize("flags", [ROW, COL, ROW | COL, ROW | RHT, ROW | COL | RHT])
def test_bad_offsets_leave_everything_empty(api, T, flags):
    """Bad offsets count as no group at all: alphas 0, no code or scale byte
    written, decoded rows left alone, weight gradients zeros - in the kernels of
    few rows as in the others."""
    C, E = 128, 2
    x = rows_of(T, C, 44).cuda()
    good = api.nvfp4_quantize_grouped(x, offsets_of([T - 9, 9]), 0, ROW | COL)
    for bad in ([0, T, T - 1], [0, T // 2, T + 1], [-1, T // 2, T], [T + 6] * 3):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = api.grouped_alloc_outputs(T, C, E, flags, x.device)
        sides = [s for s, bit in (("row", ROW), ("col", COL)) if flags & bit]
        for s in sides:
            for k in ("codes", "scales"):
                getattr(q, f"{k}_{s}").fill_(0xA5)
            getattr(q, f"alpha_{s}").fill_(7.0)
        api.nvfp4_quantize_grouped(x, off, 1, flags, out=q, status=st)
        assert st.item() == -1
        for s in sides:
            assert getattr(q, f"alpha_{s}").tolist() == [0.0, 0.0]
            assert all(bool((getattr(q, f"{k}_{s}") == 0xA5).all()) for k in ("codes", "scales"))
            for extra in (0, INV | BF):
                st.zero_()
                y = torch.full((T, C), 3.0, dtype=torch.bfloat16 if extra & BF else torch.float32, device="cuda")
                api.nvfp4_dequantize_grouped(getattr(good, f"codes_{s}"), getattr(good, f"scales_{s}"), getattr(good, f"alpha_{s}"),
                                             off, T, C, (ROW if s == "row" else COL) | extra, out=y, status=st)
                assert st.item() == -1 and bool((y == 3).all())
        for dt, out in ((FP32, torch.float32), (BF16, torch.bfloat16)):
            st.zero_()
            D = torch.full((E, C, C), 5.0, dtype=out, device="cuda")
            api.nvfp4_gemm_grouped_wgrad(*(t for _ in range(2) for t in (good.codes_col, good.scales_col, good.alpha_col)), off, T,
                                         out_dtype=dt, out=D, status=st)
            assert st.item() == -1 and not bool(D.any())


@pytest.mark.parametrize("counts", [[(5 * i) % 4 for i in range(1024)], [0] * 1000 + [1] * 24])
def test_as_many_groups_as_there_may_be(api, counts):
    check_quantize(api, rows_of(sum(counts), 128, 45), counts, 1, ROW | COL)
    check_gemm(api, counts, 128, 64, True, seed=46)
    check_wgrad(api, counts, 128, 128, False, seed=48)


@pytest.mark.parametrize("flags", [ROW, ROW | COL, ROW | RHT, COL | RHT])
@pytest.mark.parametrize("T", [48, 100])
def test_values_at_the_ends_of_the_range(api, T, flags):
    """Groups of the largest, of the smallest and of mixed numbers: as the
    oracle does each by itself."""
    x = rows_of(T, 128, 47).float().sign()
    x[: T // 3] *= 2.0 ** 123
    x[T // 3: T // 2] *= 2.0 ** -133
    x[T // 2:, ::3] *= 2.0 ** 100
    x[T // 2:, 1::3] *= 2.0 ** -120
    check_quantize(api, x.bfloat16(), [T // 3, T // 2 - T // 3, T - T // 2], 0, flags)
    check_quantize(api, x.bfloat16(), [T // 3, T // 2 - T // 3, T - T // 2], 1, flags)
