"""The linear layer's workspace query: 256 bytes mean that a call needs none, and nothing else."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: the calls below are refused on the host


@pytest.fixture(scope="module")
def L():
    from soft_clustering_gmm_amd import gmm
    return gmm.lib()


def test_small_partial_sums_are_not_taken_for_none(L):
    """A contraction in three parts with one output column: 17 to 21 rows of 3 floats are 204 to 252 bytes."""
    for N in range(17, 22):
        for d_in in range(164, 193, 4):
            assert L.gmm_linear_workspace_bytes(N, d_in, 1, 0, 0) > 256, (N, d_in)
            assert L.gmm_linear(FAKE, 0, N, d_in, FAKE, 1, None, 0, None, FAKE, 0, None, None, 0, None) == -3


@pytest.mark.parametrize("x_dtype", [0, 1, 2])
def test_none_or_more(L, x_dtype):
    """A call that needs a workspace is told more than 256 bytes, and is refused without one."""
    for N in (*range(1, 40), 64, 100, 257):
        for d_in in (*range(1, 40, 3), *range(100, 400, 12), 1000, 4096):
            for d_out in (1, 2, 3, 5, 8, 33):
                n = L.gmm_linear_workspace_bytes(N, d_in, d_out, x_dtype, 0)
                assert n == 256 or n >= 512, (N, d_in, d_out)
                if n > 256:
                    assert L.gmm_linear(FAKE, x_dtype, N, d_in, FAKE, d_out, None, 0, None, FAKE, x_dtype, None, None,
                                        0, None) == -3, (N, d_in, d_out)


@pytest.mark.gpu
def test_calls_with_small_partial_sums():
    from soft_clustering_gmm_amd import gmm as G
    from tests import layer_oracle as oracle
    g = torch.Generator().manual_seed(0)
    for N, d_in in ((17, 192), (21, 164), (17, 168), (19, 180), (22, 192)):
        X, W = torch.randn(N, d_in, generator=g).cuda(), torch.randn(1, d_in, generator=g).cuda()
        y, z, zb = oracle.linear(X, W, None, "none", None)
        oracle.check(G.linear(X, W)[0], y, oracle.y_bound(y, z, zb, "none", torch.float32), (N, d_in))
