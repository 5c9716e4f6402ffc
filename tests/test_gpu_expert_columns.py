"""What is not a number in an expert's weights reaches the rows that picked it and no others, whatever the call's size."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ODD = {"inf": float("inf"), "nan": float("nan")}


def weights(K, D, F, t, seed):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(*s, generator=g) * s[-1] ** -0.5).to(t).cuda() for s in ((K, 2 * F, D), (K, D, F))], g


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("odd", sorted(ODD))
@pytest.mark.parametrize("idx", [[[0, 3], [3, 1]], [[2], [3], [-1], [0]], [[1, 0], [2, 1], [0, 3], [2, 0]],
                                 [[0], [1], [2], [3], [4], [2], [0], [1]], [[0, 3], [3, 1], [1, 1], [2, 0], [0, -1]]],
                         ids=lambda i: f"{len(i)}x{len(i[0])}")
def test_given_picks(idx, odd, dtype):
    from soft_clustering_gmm_amd import gmm as G
    t, (K, D, F), T = TYPES[dtype], (5, 136, 200), len(idx)
    (W1, W2), g = weights(K, D, F, t, T)
    X, R = (torch.randn(T, D, generator=g).to(t).cuda() for _ in range(2))
    i = torch.tensor(idx, dtype=torch.int32)
    w = torch.rand(*i.shape, generator=g).add(0.1).cuda()
    want = G.expert_rows(X, i.cuda(), w, W1, W2, residual=R)
    assert want.isfinite().all()
    for where in ("one value", "all values", "first product"):
        A, B = W1.clone(), W2.clone()
        if where == "one value":
            B[3, 7, F - 1] = ODD[odd]
        elif where == "all values":
            B[3] = ODD[odd]
        else:
            A[3] = ODD[odd]
        y = G.expert_rows(X, i.cuda(), w, A, B, residual=R)
        for r in range(T):
            if 3 in idx[r]:
                assert not (y[r, 7] if where == "one value" else y[r]).isfinite().any(), (where, r)
            else:
                assert torch.equal(y[r], want[r]), (where, r)


@pytest.mark.parametrize("odd", sorted(ODD))
def test_picks_of_the_gate(odd):
    from soft_clustering_gmm_amd import gmm as G
    K, D, F, d = 6, 64, 96, 12
    (W1, W2), g = weights(K, D, F, torch.bfloat16, 1)
    X = torch.randn(4, D, generator=g).bfloat16().cuda()
    P = (torch.randn(d, D, generator=g) * D ** -0.5).bfloat16().cuda()
    mu, var, logw = torch.randn(K, d, generator=g).cuda(), torch.ones(K, d).cuda(), torch.zeros(K).cuda()
    want, idx, _ = G.expert_layer(X, P, mu, var, logw, W1, W2, top=2, renorm=True)
    picks = idx.cpu().tolist()
    alone = [e for e in range(K) if 0 < sum(e in p for p in picks) < 4]
    assert alone
    for e in alone:
        B = W2.clone()
        B[e, :, 5] = ODD[odd]
        y, again, _ = G.expert_layer(X, P, mu, var, logw, W1, B, top=2, renorm=True)
        assert torch.equal(again, idx)
        for r, p in enumerate(picks):
            assert not y[r].isfinite().any() if e in p else torch.equal(y[r], want[r]), (e, r)
