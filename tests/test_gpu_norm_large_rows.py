"""Rows of the layer norm's backward pass with a mean as large as float holds, and deviations of 0: finite numbers, which
give finite gradients, whatever part of the row's threads has columns."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


# rows shorter than a piece, and of pieces for some of their threads; for powers of 2 alone the mean of equal values is
# exact, so that the deviations are 0
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 4, 8, 16, 32, 64, 1024])
def test_constant_rows(G, t, D):
    g = torch.Generator(device="cuda").manual_seed(D)
    X = torch.zeros(5, D, device="cuda")
    # powers of 2, so that their sums are exact, and below 2^126
    X[0], X[1], X[2], X[3] = 2.0 ** 110, -2.0 ** 110, 2.0 ** 111, 2.0 ** 108
    X[4] = torch.randn(D, generator=g, device="cuda")
    X = X.to(t)
    dY = torch.randn(5, D, generator=g, device="cuda").to(t)
    gamma = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(t)
    eps = 1e-12  # 1 / sqrt(eps) is 2^20: 2^110 times that is beyond float
    Y, stats = G.layer_norm(X, gamma, None, eps=eps, want_stats=True)
    assert (Y[:4] == 0).all() and Y.isfinite().all() and stats.isfinite().all()
    assert torch.equal(stats[:4, 0], X[:4, 0].float())
    dx, dgamma, dbeta = G.layer_norm_backward(dY, X, stats, gamma)
    # the deviations are 0, so dX = rstd (k - mean k)
    k = dY[:4].double() * gamma.double()
    want = stats[:4, 1:].double() * (k - k.mean(1, keepdim=True))
    bound = 100 * 2.0 ** -24 * stats[:4, 1:].double() * (k.abs() + k.abs().mean(1, keepdim=True))
    assert ((dx[:4].double() - want).abs() <= bound + oracle.rounding(want.abs() + bound, t)).all()
    assert dx.isfinite().all() and dgamma.isfinite().all() and dbeta.isfinite().all()


# pieces for some of the threads of every number of threads that share a row
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D", [3, 12, 24, 25, 72, 136, 300, 520, 1000, 1032, 2056, 2504, 4104, 6000, 9000, 12000, 17000, 40000])
def test_given_statistics(G, x, y, D):
    """Rows of one value, which is their mean, under statistics that the caller gives: dX = rstd (k - mean k)."""
    t = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
    g = torch.Generator(device="cuda").manual_seed(D)
    top = 2.0 ** 110 if x != "f16" else 2.0 ** 15
    X = torch.full((5, D), top, device="cuda", dtype=t[x])
    X[1::2] = -top
    dY = torch.randn(5, D, generator=g, device="cuda").to(t[y])
    gamma = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(t[y])
    rstd = 2.0 ** 20 if x != "f16" else 2.0 ** 114  # top times rstd is beyond float
    if x == "f16":
        dY.zero_()  # 2^114 times anything else is beyond half
    stats = torch.tensor([top, rstd], device="cuda").expand(5, 2).contiguous()
    stats[1::2, 0] = -top
    dx, dgamma, dbeta = G.layer_norm_backward(dY, X, stats, gamma)
    k = dY.double() * gamma.double()
    want = rstd * (k - k.mean(1, keepdim=True))
    bound = 100 * 2.0 ** -24 * rstd * (k.abs() + k.abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= bound + oracle.rounding(want.abs() + bound, t[x])).all()
    assert (dgamma == 0).all() and dbeta.isfinite().all()
