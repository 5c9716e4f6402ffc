"""The layers in torch's graph: tensors that require gradients get them, or a backward pass that has none says so."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def leaves(N, d_in, d_out, t, out, seed=0):
    g = torch.Generator().manual_seed(seed)
    made = [torch.randn(N, d_in, generator=g).to(t), (torch.randn(d_out, d_in, generator=g) * d_in ** -0.5).to(t),
            torch.randn(d_out, generator=g).to(t), torch.randn(N, d_out, generator=g).to(out)]
    return [m.cuda().requires_grad_() for m in made], torch.randn(N, d_out, generator=g).to(out).cuda()


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_gradients_are_those_of_linear_backward(name, dtype, out):
    from soft_clustering_gmm_amd import gmm as G
    act, o = getattr(G, "ACT_" + name.upper()), TYPES[out]
    (X, W, b, R), dY = leaves(70, 45, 33, TYPES[dtype], o)
    with torch.no_grad():
        want_y, pre = G.linear(X, W, bias=b, act=act, residual=R, out_dtype=o, want_pre=True)
        want = G.linear_backward(dY, X, W, pre=pre, act=act)
    assert want_y.grad_fn is None
    for asked in (False, True):
        Y, p = G.linear(X, W, bias=b, act=act, residual=R, out_dtype=o, want_pre=asked)
        assert torch.equal(Y, want_y) and Y.requires_grad
        assert p is None if not asked else torch.equal(p, pre) and not p.requires_grad
        got = torch.autograd.grad(Y, (X, W, b, R), dY)
        for a, e in zip(got, (*want, dY)):
            assert a.dtype == e.dtype and torch.equal(a, e)


def test_only_what_requires_gradients():
    from soft_clustering_gmm_amd import gmm as G
    (X, W, b, R), dY = leaves(20, 24, 16, torch.bfloat16, torch.bfloat16)
    every = torch.autograd.grad(G.linear(X, W, bias=b, act=G.ACT_GELU, residual=R)[0], (X, W, b, R), dY)
    for i in range(4):
        part = [t.detach().requires_grad_(i == j) for j, t in enumerate((X, W, b, R))]
        Y, _ = G.linear(part[0], part[1], bias=part[2], act=G.ACT_GELU, residual=part[3])
        Y.backward(dY)
        assert torch.equal(part[i].grad, every[i]) and all(p.grad is None for j, p in enumerate(part) if j != i)
    assert not G.linear(X.detach(), W.detach(), bias=b.detach())[0].requires_grad


def test_two_layers_spread_gradients_and_shared_weights():
    """A chain whose loss gives a gradient with strides of zero, one weight used twice, against float autograd."""
    from soft_clustering_gmm_amd import gmm as G
    (X, W, b, _), _ = leaves(30, 24, 24, torch.float32, torch.float32, seed=3)

    def chain(lin):
        h = lin(X, W, b)
        return lin(h, W, b).t().sum() + (h * h).mean()

    def plain(x, w, c):
        return torch.nn.functional.silu(x.double() @ w.double().t() + c.double())
    got = torch.autograd.grad(chain(lambda x, w, c: G.linear(x, w, bias=c, act=G.ACT_SILU)[0]), (X, W, b))
    want = torch.autograd.grad(chain(plain), (X, W, b))
    for a, e in zip(got, want):
        assert (a.double() - e.double()).norm() <= 1e-5 * e.double().norm()
    with pytest.raises(RuntimeError, match="no second derivatives"):  # not gradients that count as constants
        torch.autograd.grad(G.linear(X, W, bias=b, act=G.ACT_SILU)[0].sum(), X, create_graph=True)


def test_experts_say_that_they_have_no_gradients():
    from soft_clustering_gmm_amd import gmm as G
    g = torch.Generator().manual_seed(0)
    T, D, F, K, d = 4, 32, 16, 5, 6
    X, P, W1, W2 = (torch.randn(*s, generator=g).cuda() for s in ((T, D), (d, D), (K, 2 * F, D), (K, D, F)))
    mu, var, logw = torch.randn(K, d, generator=g).cuda(), torch.ones(K, d).cuda(), torch.zeros(K).cuda()
    y, idx, resp = G.expert_layer(X, P, mu, var, logw, W1, W2)
    assert not y.requires_grad
    for t in (X, P, mu, var, logw, W1, W2):
        t.requires_grad_()
        y2, idx2, resp2 = G.expert_layer(X, P, mu, var, logw, W1, W2)
        assert torch.equal(y2, y) and torch.equal(idx2, idx) and torch.equal(resp2, resp)
        with pytest.raises(RuntimeError, match="expert_layer has no backward pass"):
            (y2.sum() + resp2.sum()).backward()
        t.requires_grad_(False)
    want = G.expert_rows(X, idx, resp, W1, W2, residual=X)
    for t in (X, resp, W1, W2):
        t.requires_grad_()
        y2 = G.expert_rows(X, idx, resp, W1, W2, residual=X)
        assert torch.equal(y2, want)
        with pytest.raises(RuntimeError, match="expert_rows has no backward pass"):
            y2.sum().backward()
        with torch.no_grad():
            assert not G.expert_rows(X, idx, resp, W1, W2, residual=X).requires_grad
        t.requires_grad_(False)


@pytest.mark.parametrize("N", [0, 1, 19])
def test_empty_few_and_unaligned_batches(N):
    """Rows of odd length from inside a batch, and gradients that start off a 16-byte border."""
    from soft_clustering_gmm_amd import gmm as G
    (X, W, b, R), dY = leaves(N + 3, 45, 33, torch.float16, torch.float32)
    Y, _ = G.linear(X[3:], W, bias=b, act=G.ACT_SILU, residual=R[3:], out_dtype=torch.float32)
    got = torch.autograd.grad(Y, (X, W, b, R), dY[3:])
    with torch.no_grad():
        _, pre = G.linear(X[3:], W, bias=b, act=G.ACT_SILU, out_dtype=torch.float32, want_pre=True)
        want = G.linear_backward(dY[3:], X[3:], W, pre=pre, act=G.ACT_SILU)
    assert torch.equal(got[0][3:], want[0]) and (got[0][:3] == 0).all() and torch.equal(got[3][3:], dY[3:])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
