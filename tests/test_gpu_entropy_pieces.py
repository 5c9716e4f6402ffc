"""The cross entropy's gradients over several pieces of rows: what is added up over them, whatever their number and sizes."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


# two and three pieces of 2^20 rows, the last one of few rows or of many; pieces of 1536 rows, their logits computed once or twice
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("N,d,V", [((1 << 20) + 5, 16, 6), ((1 << 21) + 70001, 24, 40), (3 * 1792 + 20, 300, 300000),
                                   (2 * 1792 + 1000, 64, 300000)])
def test_sums_over_pieces(G, dtype, N, d, V):
    t = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(N)
    X = torch.randn(N, d, generator=g, device="cuda").to(t)
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).to(t)
    b = torch.zeros(V, device="cuda", dtype=t)
    idx = torch.randint(0, 2, (N,), generator=g, device="cuda", dtype=torch.int32)  # two classes: no sum cancels
    idx[7::11] = -1
    dloss = torch.full((N,), 1 / 64, device="cuda")
    loss, lse, dx, dw, db = G.cross_entropy_gradients(X, W, idx, dloss=dloss, bias=b)
    dww, dbw = torch.zeros(V, d, dtype=torch.float64, device="cuda"), torch.zeros(V, dtype=torch.float64, device="cuda")
    w, rows, dxe, dxn = W.double(), max(256, (1 << 27) // V), 0.0, 0.0
    for r in range(0, N, rows):
        part = slice(r, min(N, r + rows))
        x, i, real = X[part].double(), idx[part].long().clamp(min=0)[:, None], (idx[part] >= 0)[:, None]
        z = x @ w.T
        p = torch.softmax(z, 1).mul_(real).scatter_add_(1, i, -real.double()).mul_(1 / 64)
        dww += p.T @ x
        dbw += p.sum(0)
        want = p @ w
        dxe, dxn = dxe + float((dx[part].double() - want).square().sum()), dxn + float(want.square().sum())
        del z, p
    half = torch.finfo(t).eps / 2
    # p is off by 1e-4 of itself at most (|z| is below 16, a sum of 300 products), G is rounded, and the output
    for off, size in ((dxe ** 0.5, dxn ** 0.5), (float((dw.double() - dww).norm()), float(dww.norm()))):
        assert off <= (2e-4 + 2 * half) * size
    # db: each of a chunk's 1024 rows, of a piece's 1024 chunks (in 16 slices) and of the pieces is added in float
    assert ((db.double() - dbw).abs() <= (2e-4 + 2100 * 2.0 ** -24 + 2 * half) * dbw.abs().clamp(min=2.0 ** -14)).all()
    # without db, and db alone
    one = G.cross_entropy_gradients(X, W, idx, dloss=dloss, bias=b, want_dx=False, want_dw=False)
    assert torch.equal(one[4], db) and torch.equal(one[0], loss) and torch.equal(one[1], lse)
    two = G.cross_entropy_gradients(X, W, idx, dloss=dloss, bias=b, want_db=False)
    assert torch.equal(two[2], dx) and torch.equal(two[3], dw)
