"""The cross entropy's gradients of few features under many logits, which are computed twice, and of a few more, which are
computed once and kept, against 64 bits; and of few rows around the number of picks from which on a launch prepares them."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402
from tests.test_gpu_cross_entropy import NAMES, TYPES, compare, inputs, reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("N,d,V,top", [(4090, 64, 8190, 2), (2040, 40, 33001, 1), (1200, 64, 9001, 8), (1200, 65, 9001, 8),
                                       (4090, 72, 4101, 3), (9001, 7, 1300, 1),
                                       (64, 96, 700, 8), (65, 96, 700, 8), (512, 136, 300, 1), (513, 136, 300, 1), (512, 45, 300, 1),
                                       (170, 64, 5000, 3), (171, 64, 5000, 3), (255, 64, 60000, 2), (257, 64, 60000, 2)])
def test_against_64_bits(G, monkeypatch, N, d, V, top, dtype):
    monkeypatch.setattr(oracle, "ON", "cuda")
    X, W, b, idx, wts, dloss = inputs(N, d, V, top, TYPES[dtype], True, True, seed=N + d, masked=0.1)
    want, bounds = reference(X, W, b, idx, wts, dloss)
    got = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    for a, w, bd, what in zip(got, want, bounds, NAMES):
        compare(a, w, bd, what)
    again = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    assert all(torch.equal(a, o) for a, o in zip(got, again))
    only = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b, want_dw=False, want_db=False)
    assert torch.equal(only[2], got[2])
