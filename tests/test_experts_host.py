"""Host-side checks of routing, dispatch, combine and the few-row products
(CPU): refusals return before anything is launched, and the binding checks the
tensors it is given."""
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


ROUTE_BAD = [(dict(dt=2), -1), (dict(score=2), -1), (dict(flags=4), -1), (dict(T=-1), -2), (dict(T=1 << 31), -2),
             (dict(T=1 << 30), -2), (dict(E=0), -2), (dict(E=1025, ld=1025), -2), (dict(k=0), -2), (dict(k=33), -2),
             (dict(k=9, E=8), -2), (dict(ld=63), -2), (dict(z=None), -1), (dict(z=FAKE + 2), -3), (dict(z=FAKE + 1, dt=0), -3),
             (dict(ids=None), -1), (dict(ids=FAKE + 2), -3), (dict(w=None), -1), (dict(w=FAKE + 1), -3),
             (dict(status=FAKE + 2), -3), (dict(T=0, z=None, ids=None, w=None), 0)]


@pytest.mark.parametrize("kw,status", ROUTE_BAD + [
    (dict(groups=0), -2), (dict(groups=3), -2), (dict(groups=64), -2), (dict(kept=0), -2), (dict(groups=4, kept=5), -2),
    (dict(groups=16, kept=1, k=5), -2), (dict(bias=FAKE + 2), -3)])
def test_route_refusals(kw, status):
    a = dict(z=FAKE, ld=64, dt=1, bias=None, T=4, E=64, k=4, groups=1, kept=1, score=0, flags=0, ids=FAKE, w=FAKE, status=None)
    a.update(kw)
    assert L.nvfp4_route(a["z"], a["ld"], a["dt"], a["bias"], a["T"], a["E"], a["k"], a["groups"], a["kept"], a["score"],
                         a["flags"], 1.0, a["ids"], a["w"], a["status"], None) == status


@pytest.mark.parametrize("kw,status", ROUTE_BAD + [
    (dict(d=None), -1), (dict(d=FAKE + 2), -3), (dict(ldd=60), -2), (dict(d=FAKE, ld=72), -1)])
def test_route_backward_refusals(kw, status):
    a = dict(z=FAKE, ld=64, dt=1, T=4, E=64, k=4, score=0, flags=0, ids=FAKE, w=FAKE, d=3 * FAKE, ldd=64, status=None)
    a.update(kw)
    if a["E"] > 64:
        a["ldd"] = a["E"]
    assert L.nvfp4_route_backward(a["w"], a["ids"], a["z"], a["ld"], a["dt"], a["T"], a["E"], a["k"], a["score"], a["flags"],
                                  1.0, a["d"], a["ldd"], a["status"], None) == status


PAIRS_BAD = [(dict(T=-1), -2), (dict(T=1 << 31), -2), (dict(k=0), -2), (dict(k=33), -2), (dict(T=1 << 28, k=8), -2),
             (dict(C=0), -2), (dict(C=12), -2), (dict(C=4), -2), (dict(rows=FAKE + 2), -3), (dict(status=FAKE + 2), -3)]


@pytest.mark.parametrize("kw,status", PAIRS_BAD + [
    (dict(E=0), -2), (dict(E=1025), -2), (dict(ids=None), -1), (dict(ids=FAKE + 1), -3), (dict(rows=None), -1),
    (dict(offsets=None), -1), (dict(offsets=FAKE + 2), -3), (dict(x=None), -1), (dict(xs=None), -1), (dict(xs=FAKE), -1),
    (dict(x=FAKE + 8), -3), (dict(ldx=56), -2), (dict(ldx=68), -3), (dict(ldxs=8), -2), (dict(xs=3 * FAKE + 2), -3)])
def test_dispatch_refusals(kw, status):
    a = dict(x=FAKE, ldx=64, ids=FAKE, T=4, k=2, E=8, C=64, xs=3 * FAKE, ldxs=64, offsets=FAKE, rows=FAKE, status=None)
    a.update(kw)
    assert L.nvfp4_dispatch(a["x"], a["ldx"], a["ids"], a["T"], a["k"], a["E"], a["C"], a["xs"], a["ldxs"], a["offsets"],
                            a["rows"], a["status"], None) == status


ROWS_BAD = PAIRS_BAD + [(dict(R=-1), -2), (dict(R=1 << 31), -2), (dict(rows=None, R=7), -2), (dict(w=FAKE + 2), -3),
                        (dict(y=None), -1), (dict(y=FAKE + 8), -3), (dict(ldy=60), -2), (dict(ldy=68), -3)]


@pytest.mark.parametrize("kw,status", ROWS_BAD + [
    (dict(out=None), -1), (dict(out=FAKE), -1), (dict(ldo=32), -2), (dict(out=3 * FAKE + 4), -3), (dict(res=FAKE + 4), -3),
    (dict(res=FAKE, ldr=32), -2), (dict(res=3 * FAKE, ldr=72), -1), (dict(T=0, y=None, rows=None, out=None), 0)])
def test_combine_refusals(kw, status):
    a = dict(y=FAKE, ldy=64, R=8, rows=FAKE, w=FAKE, T=4, k=2, C=64, res=None, ldr=64, out=3 * FAKE, ldo=64, status=None)
    a.update(kw)
    assert L.nvfp4_combine(a["y"], a["ldy"], a["R"], a["rows"], a["w"], a["T"], a["k"], a["C"], a["res"], a["ldr"], a["out"],
                           a["ldo"], a["status"], None) == status


@pytest.mark.parametrize("kw,status", ROWS_BAD + [
    (dict(dy=None, dw=None), -1), (dict(dout=None), -1), (dict(dout=FAKE + 8), -3), (dict(lddo=8), -2), (dict(dy=FAKE), -1),
    (dict(dy=3 * FAKE), -1), (dict(lddy=8), -2), (dict(dw=FAKE + 2), -3), (dict(T=0, y=None, rows=None, dout=None), 0)])
def test_combine_backward_refusals(kw, status):
    a = dict(dout=3 * FAKE, lddo=64, y=FAKE, ldy=64, R=8, rows=FAKE, w=FAKE, T=4, k=2, C=64, dy=4 * FAKE, lddy=64, dw=FAKE,
             status=None)
    a.update(kw)
    assert L.nvfp4_combine_backward(a["dout"], a["lddo"], a["y"], a["ldy"], a["R"], a["rows"], a["w"], a["T"], a["k"], a["C"],
                                    a["dy"], a["lddy"], a["dw"], a["status"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), -1), (dict(P=-1), -2), (dict(P=1025), -2), (dict(rep=0), -2), (dict(E=0), -2), (dict(E=1025), -2),
    (dict(ids=None), -2), (dict(N=64, ldo=64), -2), (dict(N=0), -2), (dict(N=(1 << 25) + 128, ldo=1 << 26), -2), (dict(K=96), -2), (dict(K=0), -2), (dict(ldo=64), -2),
    (dict(x=None), -1), (dict(W=None), -1), (dict(sW=None), -1), (dict(alpha=None), -1), (dict(out=None), -1),
    (dict(x=FAKE + 8), -3), (dict(ldx=64), -2), (dict(ldx=132), -3), (dict(W=FAKE + 8), -3), (dict(sW=FAKE + 4), -3),
    (dict(alpha=FAKE + 2), -3), (dict(ids=FAKE + 2), -3), (dict(status=FAKE + 2), -3), (dict(out=FAKE + 2), -3),
    (dict(out=FAKE + 1, dt=0), -3), (dict(P=0, x=None, out=None), 0)])
def test_gemv_refusals(kw, status):
    a = dict(x=FAKE, ldx=128, ids=FAKE, P=4, rep=2, W=FAKE, sW=FAKE, alpha=FAKE, E=2, N=128, K=128, out=FAKE, dt=1, ldo=128,
             status=None)
    a.update(kw)
    assert L.nvfp4_gemv(a["x"], a["ldx"], a["ids"], a["P"], a["rep"], a["W"], a["sW"], a["alpha"], a["E"], a["N"], a["K"],
                        a["out"], a["dt"], a["ldo"], a["status"], None) == status


def test_binding_refuses_wrong_tensors():
    dev = torch.device("cpu")
    ids = torch.zeros((5, 2), dtype=torch.int32)
    assert api._pairs(ids, torch.int32, "ids", dev) == (5, 2)
    with pytest.raises(ValueError, match="need"):
        api._pairs(ids.view(-1), torch.int32, "ids", dev)
    with pytest.raises(TypeError, match="ids"):
        api._pairs(ids.long(), torch.int32, "ids", dev)
    with pytest.raises(ValueError, match="contiguous"):
        api._pairs(torch.zeros((2, 5), dtype=torch.int32).t(), torch.int32, "ids", dev)
    with pytest.raises(ValueError, match="weights"):
        api._places(ids, torch.zeros((5, 3)), dev)
    with pytest.raises(ValueError, match="rows or weights"):
        api._places(None, None, dev)
    assert api._places(None, torch.zeros((5, 3)), dev) == (5, 3)
    bf = torch.zeros((5, 64), dtype=torch.bfloat16)
    for call in (lambda: api.nvfp4_route(bf, 2), lambda: api.nvfp4_dispatch(bf, ids, 4), lambda: api.nvfp4_combine(bf, ids),
                 lambda: api.nvfp4_combine_backward(bf, ids, None, bf),
                 lambda: api.nvfp4_gemv(bf, torch.zeros((128, 32), dtype=torch.uint8), None, None),
                 lambda: api.nvfp4_route_backward(torch.zeros((5, 2)), ids, bf)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_fast_host_path_declines_what_is_not_on_the_gpu():
    """The C++ host path leaves every call it does not know to the binding's
    checks: nothing is done, None is the answer."""
    f = api._load_fast()
    z, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    x, codes, alpha = torch.zeros(4, 32).bfloat16(), torch.zeros(8, 16, dtype=torch.uint8), torch.ones(1)
    assert f.route(z, 2, 0, 0, None, 1, 1, 1.0, None, None, None) is None
    assert f.route(None, "2", 0, 0, None, 1, 1, 1.0, None, None, None) is None
    assert f.route_backward(w, ids, z, 0, 0, 1.0, None, None) is None
    assert f.dispatch(x, ids, 8, None, None, None, None) is None
    assert f.combine(x, ids, w, None, None, None) is None
    assert f.combine_backward(x, ids, w, x, True, True, None, None) is None
    assert f.gemv(x, codes, codes, alpha, None, 0, None, None) is None
    assert f.route() is None and f.gemv(x) is None
    with pytest.raises(ValueError):
        f.use(1, 2)
