"""Host-side checks of the grouped calls (CPU): refusals return before
anything is launched, and the binding checks the buffers it is given."""
import pytest
import torch

from nvfp4_block_quantization_amax_b200 import _lib as L
from nvfp4_block_quantization_amax_b200 import api

ROW, COL, RHT = L.NVFP4_ROWWISE, L.NVFP4_COLWISE, L.NVFP4_RHT
FAKE = 0x10000   # never dereferenced: every call fails its checks first
OUT = L.nvfp4_qtensor_t(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from nvfp4_block_quantization_amax_b200 import build
    build.build()
    return L.load()


@pytest.mark.parametrize("T,E,step", [(0, 4, 64), (1, 4, 64), (5, 1, 128), (64, 3, 64), (1000, 8, 128), (7, 1024, 64)])
def test_capacity_holds_every_split(T, E, step):
    cap = L.nvfp4_grouped_capacity(T, E, step)
    assert cap % step == 0
    # the worst split: as many groups as possible one row past a multiple
    n = min(T, E)
    worst = [1] * n
    if n:
        worst[0] += T - n
        assert sum(-(-c // step) * step for c in worst) <= cap
    one_each = [T] + [0] * (E - 1)
    assert sum(-(-c // step) * step for c in one_each) <= cap
    assert cap <= T + n * (step - 1)


def quantize(x=FAKE, T=64, C=128, ld=128, off=FAKE, E=2, mode=0, flags=ROW, sid=0, out=OUT, ws=FAKE, nws=1 << 20):
    return L.nvfp4_quantize_grouped(x, T, C, ld, off, E, mode, flags, 0, sid, out, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=0), -1), (dict(flags=ROW | L.NVFP4_BLOCK2D), -1), (dict(flags=ROW | L.NVFP4_SINGLE_PASS), -1),
    (dict(flags=ROW | L.NVFP4_ALPHA_PROVIDED), -1), (dict(flags=ROW | L.NVFP4_VECTOR_SCALES), -1), (dict(mode=5), -1),
    (dict(mode=-1), -1), (dict(E=0), -2), (dict(E=1025), -2), (dict(T=-1), -2), (dict(T=1 << 31), -2),
    (dict(off=None), -1), (dict(off=FAKE + 2), -3), (dict(C=0), -2), (dict(C=96, ld=96), -2), (dict(ld=64), -2),
    (dict(C=192, ld=192, flags=COL), -2), (dict(C=1 << 20, ld=1 << 20, T=1 << 20), -2), (dict(x=None), -1),
    (dict(x=FAKE + 8), -3), (dict(ld=132), -3), (dict(sid=0x7FFFFFFF), -1), (dict(ws=None), -8), (dict(nws=15), -8),
    (dict(ws=FAKE + 8), -8), (dict(out=L.nvfp4_qtensor_t(FAKE, FAKE, None, None, None, None, None, None)), -1),
    (dict(out=L.nvfp4_qtensor_t(FAKE + 8, FAKE, FAKE, None, None, None, None, None)), -3),
    (dict(flags=COL, out=L.nvfp4_qtensor_t(None, None, None, FAKE, None, FAKE, None, None)), -1),
])
def test_quantize_refusals(kw, status):
    assert quantize(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(flags=0), -1), (dict(flags=ROW | COL), -1), (dict(flags=ROW | L.NVFP4_BLOCK2D), -1), (dict(E=0), -2),
    (dict(C=72), -2), (dict(C=192, flags=COL), -2), (dict(codes=None), -1), (dict(y=None), -1), (dict(y=FAKE + 8), -3),
    (dict(off=None), -1), (dict(T=0, codes=None), 0),
])
def test_dequantize_refusals(kw, status):
    a = dict(codes=FAKE, scales=FAKE, alpha=FAKE, T=64, C=128, off=FAKE, E=2, flags=ROW, y=FAKE)
    a.update(kw)
    assert L.nvfp4_dequantize_grouped(a["codes"], a["scales"], a["alpha"], a["T"], a["C"], a["off"], a["E"], a["flags"],
                                      0, a["y"], None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=64), -2), (dict(N=192), -2), (dict(K=32), -2), (dict(K=96), -2), (dict(ldd=64), -2), (dict(E=0), -2),
    (dict(E=2000), -2), (dict(dt=2), -1), (dict(A=None), -1), (dict(D=None), -1), (dict(A=FAKE + 8), -3),
    (dict(D=FAKE + 8), -3), (dict(ldd=132), -3), (dict(ldd=130, dt=1), -3), (dict(off=None), -1),
    (dict(E=1024, N=1 << 22), -2), (dict(T=0, A=None), 0),
])
def test_gemm_refusals(kw, status):
    a = dict(A=FAKE, off=FAKE, E=2, T=64, N=128, K=128, D=FAKE, dt=0, ldd=128)
    a.update(kw)
    assert L.nvfp4_gemm_grouped(a["A"], FAKE, FAKE, FAKE, FAKE, FAKE, a["off"], a["E"], a["T"], a["N"], a["K"], a["D"],
                                a["dt"], a["ldd"], None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=64), -2), (dict(N=130), -2), (dict(M=0), -2), (dict(E=0), -2), (dict(dt=3), -1), (dict(A=None), -1),
    (dict(D=None), -1), (dict(A=FAKE + 4), -3), (dict(D=FAKE + 4), -3), (dict(off=None), -1),
    (dict(E=1024, M=1 << 22), -2),
])
def test_wgrad_refusals(kw, status):
    a = dict(A=FAKE, off=FAKE, E=2, T=64, M=128, N=128, D=FAKE, dt=1)
    a.update(kw)
    assert L.nvfp4_gemm_grouped_wgrad(a["A"], FAKE, FAKE, FAKE, FAKE, FAKE, a["off"], a["E"], a["T"], a["M"], a["N"],
                                      a["D"], a["dt"], None, None) == status


def test_binding_refuses_wrong_tensors():
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    with pytest.raises(TypeError, match="bfloat16 CUDA"):
        api.nvfp4_quantize_grouped(torch.zeros((5, 128)), off, 0, ROW)
    for bad in (off.long(), off.view(1, 3)):
        with pytest.raises(TypeError, match="offsets"):
            api._check_groups(bad, torch.device("cpu"))
    with pytest.raises(ValueError, match="offsets"):
        api._check_groups(off[:1], torch.device("cpu"))
    with pytest.raises(ValueError, match="contiguous"):
        api._check_groups(torch.zeros(6, dtype=torch.int32)[::2], torch.device("cpu"))
    u8 = dict(dtype=torch.uint8)
    A, B, f = torch.zeros((5, 64), **u8), torch.zeros((2, 128, 64), **u8), torch.zeros(2)
    sA, sB = torch.zeros(256 * 8, **u8), torch.zeros(2 * 128 * 8, **u8)
    with pytest.raises(ValueError, match="codes"):
        api.nvfp4_gemm_grouped(A, sA, f, B[..., :32], sB, f, off)
    with pytest.raises(ValueError, match="experts"):
        api.nvfp4_gemm_grouped(A, sA, f, B[:1], sB, f, off)
    with pytest.raises(ValueError, match="sA"):
        api.nvfp4_gemm_grouped(A, sA[:100], f, B, sB, f, off)
    with pytest.raises(ValueError, match="sB"):
        api.nvfp4_gemm_grouped(A, sA, f, B, sB[:100], f, off)
    with pytest.raises(ValueError, match="alphaB"):
        api.nvfp4_gemm_grouped(A, sA, f, B, sB, f[:1], off)
    with pytest.raises(ValueError, match="out"):
        api.nvfp4_gemm_grouped(A, sA, f, B, sB, f, off, out=torch.zeros((4, 128), dtype=torch.bfloat16))
    cap = api.L.nvfp4_grouped_capacity(5, 2, 64)
    W = torch.zeros((128, cap // 2), **u8)
    with pytest.raises(ValueError, match="bytes per row"):
        api.nvfp4_gemm_grouped_wgrad(W, sA, f, W[:, :16], sB, f, off, 5)
    q = api.grouped_alloc_outputs(5, 128, 2, ROW | COL, torch.device("cpu"))
    api.grouped_check_outputs(q, 5, 128, 2, ROW | COL, torch.device("cpu"))
    q.scales_col = q.scales_col[:-1]
    with pytest.raises(ValueError, match="scales_col"):
        api.grouped_check_outputs(q, 5, 128, 2, ROW | COL, torch.device("cpu"))


def test_binding_refuses_host_tensors():
    """Tensors that pass every other check but are not on a GPU."""
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    u8 = dict(dtype=torch.uint8)
    A, B, f = torch.zeros((5, 64), **u8), torch.zeros((2, 128, 64), **u8), torch.zeros(2)
    sA, sB = torch.zeros(256 * 8, **u8), torch.zeros(2 * 128 * 8, **u8)
    with pytest.raises(TypeError, match="CUDA"):
        api.nvfp4_gemm_grouped(A, sA, f, B, sB, f, off)
    with pytest.raises(TypeError, match="CUDA"):
        api.nvfp4_dequantize_grouped(A, sA, f, off, 5, 128, ROW)
    W, sW = torch.zeros((128, 64), **u8), torch.zeros(128 * 8, **u8)   # 5 rows of 2 groups: 128 padded rows
    with pytest.raises(TypeError, match="CUDA"):
        api.nvfp4_gemm_grouped_wgrad(W, sW, f, W, sW, f, off, 5)


def qt(**kw):
    f = dict(codes_row=FAKE, scales_row=FAKE, alpha_row=FAKE, codes_col=FAKE, scales_col=FAKE, alpha_col=FAKE,
             amax_out=FAKE, status=FAKE)
    f.update(kw)
    return L.nvfp4_qtensor_t(*f.values())


@pytest.mark.parametrize("name", ["alpha_row", "alpha_col", "amax_out", "status"])
@pytest.mark.parametrize("T", [0, 16, 200])
def test_quantize_refuses_misaligned_words(name, T):
    assert quantize(T=T, flags=ROW | COL, out=qt(**{name: FAKE + 2})) == -3


def test_words_of_the_other_orientation_are_not_looked_at():
    assert quantize(flags=ROW, ws=None, out=qt(alpha_col=FAKE + 2)) == -8
    assert quantize(flags=COL, ws=None, out=qt(alpha_row=FAKE + 2)) == -8


@pytest.mark.parametrize("alpha,status", [(FAKE + 2, None), (FAKE, FAKE + 1)])
def test_dequantize_refuses_misaligned_words(alpha, status):
    assert L.nvfp4_dequantize_grouped(FAKE, FAKE, alpha, 64, 128, FAKE, 2, ROW, 0, FAKE, status, None) == -3


def test_products_refuse_misaligned_words():
    assert L.nvfp4_gemm_grouped(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 64, 128, 128, FAKE, 0, 128, FAKE + 2, None) == -3
    assert L.nvfp4_gemm_grouped_wgrad(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 64, 128, 128, FAKE, 1, FAKE + 2, None) == -3
