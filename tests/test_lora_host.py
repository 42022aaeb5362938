"""Host-side checks of the adapter calls (CPU): refusals return before
anything is launched, and the binding checks the tensors it is given."""
import pytest
import torch

from nvfp4_block_quantization_amax_b200 import _lib as L
from nvfp4_block_quantization_amax_b200 import api

FAKE = 0x10000   # never dereferenced: every call fails its checks first


@pytest.fixture(scope="module", autouse=True)
def lib():
    from nvfp4_block_quantization_amax_b200 import build
    build.build()
    return L.load()


BAD = [(dict(T=-1), -2), (dict(T=1 << 31), -2), (dict(K=12), -2), (dict(N=4), -2), (dict(r=12), -2), (dict(r=0), -2),
       (dict(r=136), -2), (dict(n=0), -2), (dict(n=70000), -2), (dict(K=1 << 23), -2), (dict(A=None), -1),
       (dict(ids=None), -1), (dict(A=FAKE + 8), -3), (dict(ids=FAKE + 2), -3), (dict(x=None), -1),
       (dict(x=FAKE + 8), -3), (dict(ws=None), -8), (dict(nws=15), -8), (dict(ws=FAKE + 8), -8)]


@pytest.mark.parametrize("kw,status", BAD + [
    (dict(ldx=120), -2), (dict(ldx=132), -3), (dict(out=None), -1), (dict(ldo=64), -2), (dict(y=FAKE + 2), -3),
    (dict(y=FAKE, ldy=8), -2), (dict(h=FAKE + 4), -3), (dict(T=0, x=None), 0),
])
def test_apply_refusals(kw, status):
    a = dict(x=FAKE, ldx=128, A=FAKE, ids=FAKE, T=64, K=128, N=256, r=16, n=2, y=None, ldy=256, out=FAKE, ldo=256, h=FAKE,
             ws=FAKE, nws=1 << 30)
    a.update(kw)
    assert L.nvfp4_lora_apply(a["x"], a["ldx"], a["A"], FAKE, FAKE, a["ids"], a["T"], a["K"], a["N"], a["r"], a["n"],
                              a["y"], a["ldy"], a["out"], a["ldo"], a["h"], a["ws"], a["nws"], None, None) == status


@pytest.mark.parametrize("kw,status", BAD + [
    (dict(dt=2), -1), (dict(dy=None), -1), (dict(dx=None, dA=None, dB=None), -1), (dict(h=None), -1),
    (dict(h=FAKE + 4), -3), (dict(dA=FAKE + 2), -3), (dict(lddx=64), -2), (dict(dxi=FAKE + 8), -3),
])
def test_backward_refusals(kw, status):
    a = dict(dy=FAKE, x=FAKE, ldx=128, h=FAKE, A=FAKE, ids=FAKE, T=64, K=128, N=256, r=16, n=2, dxi=None, dx=FAKE,
             lddx=128, dA=FAKE, dB=FAKE, dt=1, ws=FAKE, nws=1 << 30)
    a.update(kw)
    assert L.nvfp4_lora_backward(a["dy"], 256, a["x"], a["ldx"], a["h"], a["A"], FAKE, FAKE, a["ids"], a["T"], a["K"],
                                 a["N"], a["r"], a["n"], a["dxi"], 128, a["dx"], a["lddx"], a["dA"], a["dB"], a["dt"],
                                 a["ws"], a["nws"], None, None) == status


def test_workspace_sizes():
    assert L.nvfp4_lora_workspace_size(0, 128, 128, 16, 2, 0) == 0
    assert L.nvfp4_lora_workspace_size(64, 128, 128, 16, 2, 0) > 0
    assert L.nvfp4_lora_workspace_size(64, 128, 128, 16, 2, 1) > L.nvfp4_lora_workspace_size(64, 128, 128, 16, 2, 0)


def test_binding_refuses_wrong_tensors():
    dev = torch.device("cpu")
    bf = dict(dtype=torch.bfloat16)
    A, B, s, ids = torch.zeros((2, 16, 64), **bf), torch.zeros((2, 32, 16), **bf), torch.zeros(2), torch.zeros(5, dtype=torch.int32)
    assert api._check_lora(A, B, s, ids, 5, dev) == (64, 32, 16, 2)
    with pytest.raises(ValueError, match="A must be"):
        api._check_lora(A, B[:, :, :8], s, ids, 5, dev)
    with pytest.raises(TypeError, match="B"):
        api._check_lora(A, B.float(), s, ids, 5, dev)
    with pytest.raises(ValueError, match="ids"):
        api._check_lora(A, B, s, ids, 6, dev)
    with pytest.raises(TypeError, match="ids"):
        api._check_lora(A, B, s, ids.long(), 5, dev)
    with pytest.raises(ValueError, match="contiguous"):
        api._check_lora(A.transpose(1, 2).contiguous().transpose(1, 2), B, s, ids, 5, dev)
    with pytest.raises(TypeError, match="CUDA"):
        api.nvfp4_lora_apply(torch.zeros((5, 64), **bf), A, B, s, ids)
    assert api._rows(torch.zeros((5, 80), **bf)[:, :64], 5, 64, "x", dev) == 80
    with pytest.raises(ValueError, match="row-major"):
        api._rows(torch.zeros((64, 5), **bf).t(), 5, 64, "x", dev)
    with pytest.raises(ValueError, match="row-major"):
        api._rows(torch.zeros((4, 64), **bf), 5, 64, "x", dev)


@pytest.mark.parametrize("name", ["x", "dy"])
def test_backward_refuses_dx_over_an_input_of_the_weight_gradients(name):
    a = dict(dy=FAKE, x=2 * FAKE)
    call = lambda dA, dB: L.nvfp4_lora_backward(   # noqa: E731
        a["dy"], 128, a["x"], 128, FAKE, FAKE, FAKE, FAKE, FAKE, 64, 128, 128, 16, 2, None, 128, a[name], 128, dA, dB, 1,
        FAKE, 1 << 30, None, None)
    assert call(FAKE, None) == -1 and call(None, FAKE) == -1 and call(FAKE, FAKE) == -1


def test_a_misaligned_status_word_is_refused():
    assert L.nvfp4_lora_apply(FAKE, 128, FAKE, FAKE, FAKE, FAKE, 64, 128, 256, 16, 2, None, 256, FAKE, 256, FAKE, FAKE, 1 << 30,
                              FAKE + 2, None) == -3
    assert L.nvfp4_lora_backward(FAKE, 256, 2 * FAKE, 128, FAKE, FAKE, FAKE, FAKE, FAKE, 64, 128, 256, 16, 2, None, 128, 3 * FAKE,
                                 128, FAKE, FAKE, 1, FAKE, 1 << 30, FAKE + 2, None) == -3
