"""A training step around the mixture: layer norm, linear layer, the head's cross entropy against the components that the
mixture picks, and the AdamW step, together as they are used, against 64-bit torch."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
N, WIDTH, HIDDEN, FEATURES, K = 700, 96, 160, 16, 45


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


def problem(G, t):
    """Rows, the picks of a mixture over some of their features, and a network's parameters."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale
    rows = normal(N, WIDTH) * 2 + 1
    mu, var = normal(K, FEATURES), torch.rand(K, FEATURES, generator=g, device="cuda") + 0.5
    idx, resp = G.assign_top2(rows[:, :FEATURES].contiguous(), mu, var, torch.full((K,), -3.8, device="cuda"))
    idx[5::9] = -1  # rows that nobody labelled
    params = [1 + normal(WIDTH, scale=0.1), normal(WIDTH, scale=0.1), normal(HIDDEN, WIDTH, scale=WIDTH ** -0.5),
              normal(HIDDEN, scale=0.1), normal(K, HIDDEN, scale=HIDDEN ** -0.5), normal(K, scale=0.1)]
    return rows.to(t), idx, resp, [p.to(t).requires_grad_() for p in params]


def forward(G, rows, idx, resp, params):
    gamma, beta, w, b, head, hb = params
    h, _ = G.layer_norm(rows, gamma, beta)
    y, _ = G.linear(h, w, bias=b, act=G.ACT_GELU)
    loss, _ = G.cross_entropy(y, head, idx, wts=resp, bias=hb)
    return loss.mean()


def plain(rows, idx, resp, params):
    gamma, beta, w, b, head, hb = params
    d = rows - rows.mean(1, keepdim=True)
    h = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * gamma + beta
    z = h @ w.T + b
    z = z * 0.5 * torch.special.erfc(-z / 2 ** 0.5) @ head.T + hb
    c = resp.double() * (idx >= 0)
    return (c * (torch.logsumexp(z, 1)[:, None] - torch.gather(z, 1, idx.clamp(min=0).long()))).sum(1).mean()


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_step(G, t, bits):
    rows, idx, resp, params = problem(G, t)
    wide = [p.detach().double().requires_grad_() for p in params]
    want = plain(rows.double(), idx, resp, wide)
    want.backward()
    loss = forward(G, rows, idx, resp, params)
    loss.backward()
    # float: sums of up to 700 terms; 2 bytes: the forward values, dZ and G and the gradient are rounded, 8 times in all
    off = 2e-5 if t == torch.float32 else 8 * torch.finfo(t).eps / 2
    assert abs(float(loss) - float(want)) <= off * abs(float(want))
    for p, w in zip(params, wide):
        assert p.grad.dtype == t
        assert (p.grad.double() - w.grad).norm() <= off * w.grad.norm()
    state = G.adamw_state(params, bits=bits, master=t != torch.float32)
    grads = [p.grad for p in params]
    before = [p.detach().double() for p in params]
    with torch.no_grad():
        G.adamw_step(params, grads, **state, **HYPER)
    assert state["step"].tolist() == [1, 0]
    for p, b, g in zip(params, before, grads):
        # the first step is lr in the gradient's direction, eps aside
        new = b - HYPER["lr"] * HYPER["weight_decay"] * b - HYPER["lr"] * g.double() / (g.double().abs() + HYPER["eps"])
        assert (p.detach().double() - new).abs().max() <= 1e-6 + new.abs().max() * torch.finfo(t).eps / 2
    # and the next forward pass takes the new parameters
    again = forward(G, rows, idx, resp, params)
    after = plain(rows.double(), idx, resp, [p.detach().double() for p in params])
    assert abs(float(again) - float(after)) <= off * abs(float(after)) and float(again) != float(loss)


def test_captured_steps(G):
    """The same as a captured step without torch's graph: replays go on from each other, as eager steps do."""
    rows, idx, resp, params = problem(G, torch.bfloat16)
    params = [p.detach() for p in params]
    twin = [p.clone() for p in params]
    a, b = G.adamw_state(params, bits=8, master=True), G.adamw_state(twin, bits=8, master=True)
    share = torch.full((N,), 1 / N, device="cuda")

    def step(p, state):
        gamma, beta, w, bias, head, hb = p
        h, st = G.layer_norm(rows, gamma, beta, want_stats=True)
        y, pre = G.linear(h, w, bias=bias, act=G.ACT_GELU, want_pre=True)
        loss, _, dy, dhead, dhb = G.cross_entropy_gradients(y, head, idx, dloss=share, wts=resp, bias=hb)
        dh, dw, db = G.linear_backward(dy, h, w, pre=pre, act=G.ACT_GELU)
        _, dgamma, dbeta = G.layer_norm_backward(dh, rows, st, gamma, want_dx=False)
        G.adamw_step(p, [dgamma, dbeta, dw, db, dhead, dhb], **state, **HYPER)
        return loss
    with torch.no_grad():
        step(params, a), step(twin, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss = step(params, a)
        for _ in range(4):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(loss, step(twin, b))
            assert all(torch.equal(x, y) for x, y in zip(params, twin))
            for k in a:
                assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
