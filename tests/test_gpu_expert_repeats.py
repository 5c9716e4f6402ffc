"""Few picks (the product that gathers a row's experts) with an expert picked more than once, skipped picks and weights
of any size and sign: gmm_expert_rows against the plain 64-bit form, alone and among more picks."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# picks and weights of at most 8 picks
CASES = {
    "small weight first": ([[0, 0]], [[1e-6, 1.0]], 1),
    "a thousandth first": ([[0, 0], [2, 1]], [[1e-3, 1.0], [0.5, 0.5]], 1),
    "zero weight first": ([[0, 0]], [[0.0, 1e-6]], 10000),
    "skipped between": ([[1, -1, 1, 4], [2, 0, 7, 2]], [[1e-5, 9.0, -2.0, 0.25], [0.125, 1.0, 8.0, -1.0]], 1),
    "all eight the same": ([[3] * 8], [[1e-7, 0.25, -0.5, 1.0, 0.0, 2.0, -1e-3, 0.125]], 1),
    "cancelled": ([[1, 1, 0]], [[1.0, -1.0, 1e-6]], 10000),
}


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("name", sorted(CASES))
def test_repeated_picks(name, dtype):
    from soft_clustering_gmm_amd import gmm as G
    i, w, lift = CASES[name]
    idx, wts, t = torch.tensor(i, dtype=torch.int32), torch.tensor(w), TYPES[dtype]
    T, (K, D, F) = idx.shape[0], (5, 72, 60)
    g = torch.Generator().manual_seed(len(name))

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(t).cuda()
    X, W1, W2 = normal(T, D, scale=3.0), normal(K, 2 * F, D, scale=D ** -0.5), normal(K, D, F, scale=lift * F ** -0.5)
    b1, b2 = normal(K, 2 * F), normal(K, D)
    want, bound = oracle.experts(X, idx, wts, W1, b1, W2, b2, "silu", True, None)
    y = G.expert_rows(X, idx.cuda(), wts.cuda(), W1, W2, b1=b1, b2=b2)
    oracle.check(y, want, bound, "few picks")
    n = 8 // idx.numel() + 1  # copies that make more than 8 picks
    more = G.expert_rows(X.repeat(n, 1), idx.repeat(n, 1).cuda(), wts.repeat(n, 1).cuda(), W1, W2, b1=b1, b2=b2)
    oracle.check(more, want.repeat(n, 1), bound.repeat(n, 1), "more picks")
