"""The cross entropy of rows that are sure of their pick: the largest logit, the sum and the pick's logit come from one
product, so that the loss is a sum of non-negative terms and is as exact as its logits' differences."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
# rows, features, classes, picks: few rows; one tile and many; a long contraction that gradients split; few features
# under many logits, which the gradients compute twice; rows that share a wave
SHAPES = [(9, 2048, 500, 1), (16, 1000, 9000, 3), (400, 2048, 600, 1), (300, 2056, 70001, 2), (60, 4096, 100, 1),
          (1200, 256, 9001, 2), (1200, 88, 9001, 8), (5000, 136, 260, 2), (33, 777, 1025, 5)]


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


def confident(N, d, V, top, t, seed=0):
    """Rows whose first pick's class lies in their direction, so that its logit is 8 to 64 and the others' are small."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(N, d, generator=g, device="cuda").to(t)
    W = torch.randn(V, d, generator=g, device="cuda") * d ** -0.5
    first = torch.randperm(V, generator=g, device="cuda")[torch.arange(N, device="cuda") % V]
    size = torch.linspace(8, 64, N, device="cuda")
    x = X.float()
    W[first] = (x * (size / (x * x).sum(1))[:, None])[:len(first)]
    idx = torch.randint(0, V, (N, top), generator=g, device="cuda", dtype=torch.int32)
    idx[:] = first[:, None].int()  # all picks are the sure one
    return X, W.to(t), idx


def bounds(X, W, idx, bias):
    """(loss, its bound): log(1 + r) with r = sum exp(z_v - z_pick), each logit off by its sum's worst case."""
    x, w = X.double(), W.double()
    z, zb = x @ w.T, oracle.sum_bound(X.double(), W.double(), X.shape[1])
    if bias is not None:
        z = z + bias.double()
        zb = zb + 2 * U * z.abs()
    i = idx[:, :1].long()
    own, ownb = torch.gather(z, 1, i), torch.gather(zb, 1, i)
    far = (z - own).scatter(1, i, -float("inf"))
    r = torch.exp(far)
    # Each term is off by its exponent's error, and by the exponential's and its own sums' roundings: 512 at most.
    rb = (r * torch.expm1(zb + ownb + 2 * U * far.abs().clamp(max=200))).sum(1)
    r = r.sum(1)
    # The largest entry is 1, and the others are added to it: a sum S >= 1 becomes the float next to S + t, off by half a
    # step of S + t and, as S is a float itself, by t at most. The largest entry's part passes through at most 64 additions
    # in a lane, 32 parts in a lane, 6 steps over the wave and 16 waves; what they add is r altogether.
    loss = torch.log1p(r)
    return loss, rb + 512 * U * r + torch.minimum(r, 118 * U * (1 + r)) + 4 * U * loss


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "x".join(map(str, SHAPES[i])))
def test_sure_rows(G, i, dtype):
    N, d, V, top = SHAPES[i]
    X, W, idx = confident(N, d, V, top, TYPES[dtype], seed=i)
    bias = (torch.randn(V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)) * 0.1).to(X.dtype)
    for b in (None, bias):
        want, off = bounds(X, W, idx, b)
        fwd, lse = G.cross_entropy(X, W, idx, bias=b)
        back = G.cross_entropy_gradients(X, W, idx, bias=b, want_dw=False, want_db=False)[0]
        for loss in (fwd, back):
            assert (loss >= 0).all(), (float(loss.min()), int((loss < 0).sum()))
            bad = ~((loss.double() - top * want).abs() <= top * off + (top - 1) * 4 * U * top * want)
            assert not bad.any(), (int(bad.sum()), float(loss[bad][0]), float(top * want[bad][0]))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_picks_anywhere(G, dtype):
    """Picks in every column of a tile, in the last classes and outside, each row its own."""
    V, N, d = 777, 2000, 300
    g = torch.Generator(device="cuda").manual_seed(0)
    X = torch.randn(N, d, generator=g, device="cuda").to(TYPES[dtype])
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).to(TYPES[dtype])
    i = torch.arange(N, device="cuda")
    idx = torch.stack([i % (V + 9) - 4, (i * 7 + 3) % V, V - 1 - i % 5, torch.full_like(i, V + 40)], 1).int()
    z, zb = X.double() @ W.double().T, oracle.sum_bound(X.double(), W.double(), d)
    lse, real = torch.logsumexp(z, 1), (idx >= 0) & (idx < V)
    at = torch.where(real, idx, 0).long()
    want = torch.where(real, lse[:, None] - torch.gather(z, 1, at), 0.0).sum(1)
    off = 3 * (2 * zb.amax(1) + 600 * U * (1 + lse.abs() + z.abs().amax(1)))
    for out in (G.cross_entropy(X, W, idx)[0], G.cross_entropy_gradients(X, W, idx)[0]):
        assert ((out.double() - want).abs() <= off).all()
