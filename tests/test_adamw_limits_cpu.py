"""Numbers of the AdamW step that float cannot hold as they are meant: refused on the host, before any launch."""
import ctypes

import pytest

pytest.importorskip("torch")
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def L():
    from soft_clustering_gmm_amd import gmm
    return gmm.lib()


def call(L, lr=1e-3, eps=1e-8, wd=0.01):
    s, p, g = (ctypes.c_int64 * 1)(10), (ctypes.c_void_p * 1)(0x100000), (ctypes.c_void_p * 1)(0x200000)
    return L.gmm_adamw_step(1, s, p, 2, g, 2, None, FAKE, FAKE, 32, None, None, FAKE, lr, 0.9, 0.999, eps, wd, None, None,
                            None)


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.17e-38, 3.5e38, 1e300])
def test_eps_is_a_normal_float(L, eps):
    """The device's reciprocal takes less for 0: an element without a gradient would become 0 times infinity. What float
    takes for infinity would end every update."""
    assert call(L, eps=eps) == -1


@pytest.mark.parametrize("number", [3.5e38, 1e300])
def test_rate_and_decay_are_finite_floats(L, number):
    assert call(L, lr=number) == -1 and call(L, wd=number) == -1
