"""Argument checks of the linear layer and the layer of experts: refused on the host, before any launch."""
import ctypes
import os

import pytest

from tests import layer_oracle as oracle

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x100008)


@pytest.fixture(scope="module")
def L():
    from soft_clustering_gmm_amd import gmm
    return gmm.lib()


def test_linear_refusals(L):
    def call(X=FAKE, xt=2, N=100, d_in=64, W=FAKE, d_out=32, act=0, Y=FAKE, yt=2, ws=FAKE, wsb=1 << 40):
        return L.gmm_linear(X, xt, N, d_in, W, d_out, None, act, None, Y, yt, None, ws, wsb, None)
    assert call(xt=3) == -1 and call(yt=1) == -1 and call(xt=0, yt=2) == -1
    assert call(act=4) == -1 and call(act=-1) == -1
    assert call(N=-1) == -1 and call(d_in=0) == -1 and call(d_out=0) == -1
    assert call(X=None) == -1 and call(W=None) == -1 and call(Y=None) == -1
    assert call(X=ODD) == -1 and call(W=ODD) == -1  # whole 16-byte rows off a 16-byte border
    assert call(d_in=65537) == -2 and call(d_out=65537) == -2 and call(N=1 << 31) == -2
    # 100 rows of 63 two-byte elements are copied to rows of 64
    assert call(d_in=63, ws=None) == -3 and call(d_in=63, wsb=100) == -3 and call(d_in=63, ws=ODD) == -3
    assert call(N=0, X=None, Y=None, ws=None) == 0


def test_linear_backward_refusals(L):
    def call(dY=FAKE, yt=2, X=FAKE, xt=2, N=100, d_in=64, W=FAKE, d_out=32, pre=FAKE, act=2, ws=FAKE, wsb=1 << 40):
        return L.gmm_linear_backward(dY, yt, X, xt, N, d_in, W, d_out, pre, act, FAKE, FAKE, FAKE, ws, wsb, None)
    assert call(dY=None) == -1 and call(pre=None) == -1 and call(X=None) == -1 and call(W=None) == -1
    assert call(yt=1) == -1 and call(act=7) == -1 and call(N=-5) == -1 and call(X=ODD) == -1 and call(W=ODD) == -1
    assert call(d_out=1 << 17) == -2
    assert call(ws=None) == -3 and call(wsb=8) == -3


def test_linear_workspace_bytes(L):
    assert L.gmm_linear_workspace_bytes(10, 0, 5, 2, 0) == 0
    assert L.gmm_linear_workspace_bytes(10, 5, 5, 7, 0) == 0
    assert L.gmm_linear_workspace_bytes(1 << 31, 5, 5, 2, 0) == 0
    assert L.gmm_linear_workspace_bytes(0, 5, 5, 2, 1) > 0
    # aligned rows with enough tiles need no copies; odd ones one copy each
    aligned = L.gmm_linear_workspace_bytes(1 << 18, 1024, 1024, 2, 0)
    assert aligned <= 1 << 20
    assert L.gmm_linear_workspace_bytes(1 << 18, 1023, 1024, 2, 0) >= (1 << 18) * 1024 * 2
    for n in (1, 64, 65, 1000, 12345):
        for b in (0, 1):
            assert L.gmm_linear_workspace_bytes(n, 100, 77, 1, b) > 0


def test_expert_refusals(L):
    def call(X=FAKE, xt=2, N=8, D=64, P=FAKE, d=16, K=4, top=2, W1=FAKE, F=32, act=3, idx=FAKE, ws=FAKE, wsb=1 << 40):
        return L.gmm_expert_layer(X, xt, N, D, P, d, FAKE, FAKE, FAKE, K, top, ctypes.c_float(0), 0, W1, None, FAKE,
                                  None, F, act, 1, None, FAKE, idx, FAKE, ws, wsb, None)
    assert call(xt=5) == -1 and call(act=9) == -1 and call(N=-1) == -1 and call(D=0) == -1 and call(K=0) == -1
    assert call(top=0) == -1 and call(F=0) == -1 and call(d=0) == -1
    assert call(X=None) == -1 and call(P=None) == -1 and call(W1=None) == -1 and call(idx=None) == -1
    assert call(N=129) == -2 and call(top=9) == -2 and call(d=129) == -2 and call(D=65537) == -2
    assert call(K=65537) == -2 and call(F=65537) == -2
    assert call(ws=None) == -3 and call(ws=ODD) == -3 and call(wsb=64) == -3

    def rows(X=FAKE, N=8, idx=FAKE, wts=FAKE, top=2, ws=FAKE):
        return L.gmm_expert_rows(X, 2, N, 64, idx, wts, top, 4, FAKE, None, FAKE, None, 32, 3, 1, None, FAKE, ws,
                                 1 << 40, None)
    assert rows(X=None) == -1 and rows(idx=None) == -1 and rows(wts=None) == -1 and rows(top=0) == -1
    assert rows(N=129) == -2 and rows(ws=None) == -3
    assert L.gmm_expert_workspace_bytes(129, 64, 4, 32, 16, 2, 2) == 0
    assert L.gmm_expert_workspace_bytes(8, 64, 4, 32, 129, 2, 2) == 0
    assert 0 < L.gmm_expert_workspace_bytes(1, 64, 4, 32, 0, 1, 2) < L.gmm_expert_workspace_bytes(128, 64, 4, 32, 16, 8, 0)


@pytest.mark.parametrize("name", oracle.ACTS)
def test_oracle_slopes_against_differences(name):
    z = torch.linspace(-6, 6, 401, dtype=torch.float64) + 1e-3
    h = 1e-5
    d = (oracle.act(z + h, name) - oracle.act(z - h, name)) / (2 * h)
    assert (d - oracle.slope(z, name)).abs().max() < 1e-9


def test_oracle_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    X, W, b, dY = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((7, 5), (4, 5), (4,), (7, 4)))
    _, z, _ = oracle.linear(X.float(), W.float(), b.float(), "gelu", None)
    X, W, b = X.float(), W.float(), b.float()
    (dx, dw, db), _ = oracle.gradients(dY.float(), X, W, z, "gelu")
    h = 1e-4

    def loss(x, w, c):
        return float((oracle.act(x @ w.T + c, "gelu") * dY.float().double()).sum())
    base = [X.double(), W.double(), b.double()]
    for at, grad in enumerate((dx, dw, db)):
        v = torch.randn(base[at].shape, generator=g, dtype=torch.float64)
        ends = [loss(*[t + (s * v if i == at else 0) for i, t in enumerate(base)]) for s in (h, -h)]
        assert abs((ends[0] - ends[1]) / (2 * h) - float((grad * v).sum())) < 1e-5


def test_planted_errors_are_seen():
    """The bounds see a swapped pick, a lost bias and one wrong product."""
    g = torch.Generator().manual_seed(0)
    X, W = torch.randn(20, 300, generator=g).bfloat16(), (torch.randn(30, 300, generator=g) * 300 ** -0.5).bfloat16()
    y, z, zb = oracle.linear(X, W, None, "none", None)
    bound = oracle.y_bound(y, z, zb, "none", torch.bfloat16)
    good = y.to(torch.bfloat16)
    oracle.check(good, y, bound, "rounded")
    X2 = X.clone()
    X2[3, 17] = 0
    bad = oracle.linear(X2, W, None, "none", None)[0].to(torch.bfloat16)
    with pytest.raises(AssertionError):
        oracle.check(bad, y, bound, "one product")
    with pytest.raises(AssertionError):
        oracle.check(good + 0.05, y, bound, "bias")
