"""The gradient of each logit of 2-byte operands, one by one: rows of X are those of the identity, so that dW's entries
are G's. What is kept of a logit between the products is off by no more than G's own rounding."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("N,V,spread", [(320, 20000, 3.0), (320, 20000, 0.5), (280, 30001, 5.0)])
def test_entries(G, t, N, V, spread):
    g = torch.Generator(device="cuda").manual_seed(N + V)
    W = (torch.randn(V, N, generator=g, device="cuda") * spread).to(t)
    X = torch.eye(N, device="cuda").to(t)
    idx = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    z = W.double().T  # a product of one term: exact
    p = torch.softmax(z, 1)
    size = 2.0 ** 14
    want = (p - torch.zeros_like(p).scatter_(1, idx.long()[:, None], 1.0)) * size
    dloss = torch.full((N,), size, device="cuda")
    _, _, _, dw, _ = G.cross_entropy_gradients(X, W, idx, dloss=dloss, want_dx=False, want_db=False)
    got = dw.double().T
    far = (z.amax(1, keepdim=True) - z).clamp(max=200)
    # Kept: half a step of half, 2^-11 of p, and below 2^-29 of the group's largest, 2^-40 of that. Exponentials and sums in float: the row's
    # sum is off by 512 roundings at most, an exponent by 2 of itself. G, scaled by 2^11 / size, and the output: half a
    # step each, and half of the smallest number where they are that small.
    rel = 2.0 ** -11 + (512 + 24) * U + 2 * U * far
    kept = p * size * rel + 2.0 ** -40 * size * p.amax(1, keepdim=True)
    half = torch.finfo(t).eps / 2
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[t]
    bound = kept + 2 * half * (want.abs() + kept) * (1 + half) + tiny * (size / 2048 + 1) + 12 * U * want.abs()
    # the pick's entry is p - 1: a difference
    bound = bound.scatter_add(1, idx.long()[:, None], torch.full((N, 1), 8 * U * size, dtype=torch.float64, device="cuda"))
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / bound).max()))


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_groups_far_below(G, t):
    """Groups of columns whose largest logit lies far below the row's, entries far below their group's, classes taken out."""
    N, V = 264, 4000
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(V, N, generator=g, device="cuda")
    W -= (torch.arange(V, device="cuda") // 64 % 5 * 9)[:, None]
    W[::7] -= 20
    W, X = W.to(t), torch.eye(N, device="cuda").to(t)
    bias = torch.zeros(V, device="cuda", dtype=t)
    bias[5::11] = -float("inf")
    bias[640:960] = -float("inf")
    idx = torch.randint(0, V // 11, (N,), generator=g, device="cuda", dtype=torch.int32) * 11
    idx[(idx >= 640) & (idx < 960)] = 0
    p = torch.softmax((W.double() + bias.double()[:, None]).T, 1)
    want = p - torch.zeros_like(p).scatter_(1, idx.long()[:, None], 1.0)
    dw = G.cross_entropy_gradients(X, W, idx, bias=bias, want_dx=False)[3].double().T
    half = torch.finfo(t).eps / 2
    # G and the output are rounded, in half also below its smallest normal number; the bias's sum in float
    bound = (2.0 ** -11 + 2.1 * half + 700 * U) * want.abs() + 2.0 ** -40 + (2.0 ** -24 if t == torch.float16 else 0.0) + 8 * U
    assert ((dw - want).abs() <= bound).all(), float(((dw - want).abs() / bound).max())
    assert (dw[:, 5::11] == 0).all() and (dw[:, 640:960] == 0).all()
