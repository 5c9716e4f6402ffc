"""Argument checks of the layer norm and the AdamW step: refused on the host, before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x100008)


@pytest.fixture(scope="module")
def L():
    from soft_clustering_gmm_amd import gmm
    return gmm.lib()


def test_layer_norm_refusals(L):
    def call(X=FAKE, xt=2, N=10, D=64, wt=2, eps=1e-5, Y=FAKE, yt=2):
        return L.gmm_layer_norm(X, xt, N, D, FAKE, FAKE, wt, eps, Y, yt, None, None)
    assert call(xt=3) == -1 and call(yt=-1) == -1 and call(wt=5) == -1
    assert call(xt=2, yt=0, wt=0) == -1 and call(xt=1, yt=2) == -1  # only float X has an Y of another type
    assert call(wt=1) == -1  # neither Y's type nor float
    assert call(N=-1) == -1 and call(D=0) == -1 and call(X=None) == -1 and call(Y=None) == -1
    assert call(eps=0.0) == -1 and call(eps=-1.0) == -1 and call(eps=float("inf")) == -1 and call(eps=float("nan")) == -1
    assert call(D=65537) == -2 and call(N=1 << 31) == -2
    assert call(N=0, X=None, Y=None) == 0

    def back(dY=FAKE, yt=2, X=FAKE, xt=2, N=10, D=64, stats=FAKE, wt=2, dX=FAKE, dg=FAKE, ws=FAKE, wsb=1 << 40):
        return L.gmm_layer_norm_backward(dY, yt, X, xt, N, D, stats, FAKE, wt, dX, dg, None, ws, wsb, None)
    assert back(dY=None) == -1 and back(X=None) == -1 and back(stats=None) == -1 and back(yt=0) == -1
    assert back(wt=1) == -1 and back(N=-3) == -1 and back(D=1 << 20) == -2
    assert back(ws=None) == -3 and back(ws=ODD) == -3 and back(wsb=64) == -3
    assert back(dX=None, dg=None, ws=None) == 0  # nothing wanted
    assert L.gmm_layer_norm_workspace_bytes(-1, 64, 2) == 0 and L.gmm_layer_norm_workspace_bytes(5, 64, 9) == 0
    assert L.gmm_layer_norm_workspace_bytes(5, 70000, 2) == 0
    for n in (0, 1, 1000, 1 << 20):
        for d in (1, 64, 16384, 65536):
            for t in (0, 1, 2):
                assert 256 <= L.gmm_layer_norm_workspace_bytes(n, d, t) <= 1024 * 8 * max(d, 4096)


def arrays(sizes, params, grads):
    n = len(sizes)
    return (ctypes.c_int64 * n)(*sizes), (ctypes.c_void_p * n)(*params), (ctypes.c_void_p * n)(*grads)


def test_adamw_refusals(L):
    def call(sizes=(10, 300), params=(0x100000, 0x200000), grads=(0x300000, 0x400000), pt=2, gt=2, master=None, m=FAKE,
             v=FAKE, bits=32, ms=None, vs=None, step=FAKE, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, count=None):
        s, p, g = arrays(sizes, params, grads)
        return L.gmm_adamw_step(len(sizes) if count is None else count, s, p, pt, g, gt, master, m, v, bits, ms, vs, step,
                                lr, b1, b2, eps, wd, None, None, None)
    assert call(pt=3) == -1 and call(gt=1) == -1 and call(pt=0, gt=2) == -1 and call(bits=16) == -1
    assert call(b1=1.0) == -1 and call(b2=-0.1) == -1 and call(b2=float("nan")) == -1
    assert call(eps=0.0) == -1 and call(eps=1e-60) == -1 and call(lr=-1.0) == -1 and call(lr=float("inf")) == -1
    assert call(wd=-0.1) == -1 and call(wd=float("nan")) == -1
    assert call(count=-1) == -1 and call(sizes=(10, -1)) == -1
    assert call(step=None) == -1 and call(step=ctypes.c_void_p(0x100004)) == -1
    assert call(m=None) == -1 and call(v=None) == -1 and call(m=ODD) == -1 and call(v=ODD) == -1 and call(master=ODD) == -1
    assert call(bits=8) == -1 and call(bits=8, ms=FAKE) == -1  # 8 bits need scales
    assert call(pt=0, gt=0, master=FAKE) == -1
    assert call(params=(0x100000, None)) == -1
    assert L.gmm_adamw_step(2, None, None, 2, None, 2, None, FAKE, FAKE, 32, None, None, FAKE, 1e-3, 0.9, 0.99, 1e-8, 0.0,
                            None, None, None) == -1

    def elements(*sizes):
        return L.gmm_adamw_state_elements(len(sizes), (ctypes.c_int64 * len(sizes))(*sizes))
    assert elements() == 0 and elements(1) == 256 and elements(256, 257, 0) == 768 and elements(5, -1) == -1
    assert elements(1 << 40) == -1 and L.gmm_adamw_state_elements(-1, None) == -1
    assert L.gmm_adamw_state_elements(1, None) == -1


def test_adamw_state():
    from soft_clustering_gmm_amd import gmm
    params = [torch.arange(300.0).view(3, 100).bfloat16(), torch.ones(1).bfloat16(), torch.full((256,), 2.0).bfloat16()]
    s = gmm.adamw_state(params, master=True)
    assert sorted(s) == ["m", "master", "step", "v"] and s["m"].shape == s["v"].shape == (1024,)
    assert torch.equal(s["master"][:300], params[0].float().view(-1)) and (s["master"][300:512] == 0).all()
    assert s["master"][512] == 1 and (s["master"][768:] == 2).all() and s["step"].tolist() == [0, 0]
    s = gmm.adamw_state(params, bits=8)
    assert s["m"].dtype == s["v"].dtype == torch.float8_e4m3fn and s["m_scale"].shape == (4,) and "master" not in s
    with pytest.raises(ValueError):
        gmm.adamw_state(params, bits=16)
    with pytest.raises(ValueError):
        gmm.adamw_state([])
