"""The layer of experts (gmm_expert_layer, gmm_expert_rows) against its plain 64-bit form, entry by entry, within
bounds derived from the arithmetic (tests/layer_oracle.py); picks and missing picks exactly."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


def layer(T, D, F, K, d, dtype, glu, bias, residual, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0, t=dtype):
        return (torch.randn(*shape, generator=g) * scale).to(t).cuda()
    up = 2 * F if glu else F
    f32 = torch.float32
    s = {"X": normal(T, D), "P": normal(d, D, scale=D ** -0.5), "mu": normal(K, d, scale=0.7, t=f32),
         "var": ((0.5 + torch.rand(K, d, generator=g)) * max(1.0, d / 16)).cuda(),
         "logw": torch.log_softmax(torch.randn(K, generator=g), 0).cuda(),
         "W1": normal(K, up, D, scale=D ** -0.5), "W2": normal(K, D, F, scale=F ** -0.5)}
    opt = {"b1": normal(K, up) if bias else None, "b2": normal(K, D) if bias else None,
           "residual": normal(T, D) if residual else None}
    return s, opt


# rows, width, hidden, experts, features, top
SHAPES = [(1, 64, 32, 4, 8, 2), (1, 1000, 333, 7, 17, 3), (1, 8, 1, 1, 1, 2), (5, 256, 128, 64, 64, 2),
          (16, 96, 200, 300, 128, 8), (17, 130, 40, 3, 65, 2), (40, 264, 72, 2, 5, 1), (128, 72, 56, 5, 33, 4),
          (128, 40, 24, 1, 9, 1), (33, 1, 16, 6, 2, 2), (20, 17, 19, 65, 100, 8)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "x".join(map(str, SHAPES[i])))
def test_layer(G, i, dtype):
    T, D, F, K, d, top = SHAPES[i]
    name, glu, renorm, thr = oracle.ACTS[i % 4], i % 2 == 0, i % 3 == 0, (0.0, 0.05, 0.3)[i % 3]
    s, opt = layer(T, D, F, K, d, TYPES[dtype], glu, i % 2 == 1, i % 4 != 2, seed=i)
    y, idx, resp = G.expert_layer(s["X"], s["P"], s["mu"], s["var"], s["logw"], s["W1"], s["W2"],
                                  act=getattr(G, "ACT_" + name.upper()), glu=glu, top=top, border_threshold=thr,
                                  renorm=renorm, **opt)
    want_idx, want_resp, w = oracle.gate(s["X"], s["P"], s["mu"], s["var"], s["logw"], top, thr, renorm)
    assert torch.equal(idx.cpu().long(), want_idx)
    # 64-bit scores, rounded once to float
    oracle.check(resp, want_resp, want_resp * (2.0 ** -24 + 1e-9) + 2.0 ** -149, "resp")
    y64, bound = oracle.experts(s["X"], want_idx, w, s["W1"], opt["b1"], s["W2"], opt["b2"], name, glu,
                                opt["residual"])
    oracle.check(y, y64, bound, f"y {name}")
    again = G.expert_layer(s["X"], s["P"], s["mu"], s["var"], s["logw"], s["W1"], s["W2"],
                           act=getattr(G, "ACT_" + name.upper()), glu=glu, top=top, border_threshold=thr,
                           renorm=renorm, **opt)
    assert torch.equal(again[0], y) and torch.equal(again[2], resp)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("T,K,top", [(1, 5, 1), (9, 4, 3), (64, 3, 8), (128, 2, 8), (128, 200, 2)])
def test_given_picks(G, T, K, top, dtype):
    """Picks outside the experts, rows without any, the same expert twice in a row, negative and zero weights."""
    D, F = 104, 60
    s, opt = layer(T, D, F, K, 4, TYPES[dtype], True, True, True, seed=T + K)
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-1, K + 1, (T, top), generator=g, dtype=torch.int32)
    if T > 2:
        idx[1] = -1
        idx[2] = 0
        idx[0, -1] = 2 ** 31 - 1
    wts = torch.randn(T, top, generator=g)
    wts[T - 1, 0] = 0
    y = G.expert_rows(s["X"], idx.cuda(), wts.cuda(), s["W1"], s["W2"], **opt)
    y64, bound = oracle.experts(s["X"], idx, wts, s["W1"], opt["b1"], s["W2"], opt["b2"], "silu", True,
                                opt["residual"])
    oracle.check(y, y64, bound, "y")
    if T > 2:
        assert torch.equal(y[1], opt["residual"][1])  # a row whose mask leaves nothing


def test_rows_without_a_posterior(G):
    """NaN and infinite rows: no picks, y NaN, the other rows as without them; components of weight zero and fewer
    components than picks."""
    for T in (6, 50):
        s, opt = layer(T, 64, 40, 6, 12, torch.bfloat16, True, False, True, seed=T)
        s["logw"][2] = float("-inf")
        args = [s[k] for k in ("P", "mu", "var", "logw", "W1", "W2")]
        y, idx, resp = G.expert_layer(s["X"], *args, top=8, **opt)
        assert not (idx == 2).any() and (idx[:, 5:] == -1).all() and (resp[:, 5:] == 0).all() and (idx[:, :5] >= 0).all()
        X = s["X"].clone()
        X[1, 3], X[4, 0] = float("nan"), float("inf")
        y2, idx2, resp2 = G.expert_layer(X, *args, top=8, **opt)
        for t in (1, 4):
            assert y2[t].isnan().all() and (idx2[t] == -1).all() and (resp2[t] == 0).all()
        keep = [t for t in range(T) if t not in (1, 4)]
        assert torch.equal(y2[keep], y[keep]) and torch.equal(idx2[keep], idx[keep])
        s["logw"].fill_(float("-inf"))
        y3, idx3, _ = G.expert_layer(s["X"], *args, top=2, **opt)
        assert y3.isnan().all() and (idx3 == -1).all()


def test_ties_go_to_the_lower_component(G):
    s, opt = layer(9, 32, 16, 40, 6, torch.float32, False, False, False, seed=1)
    for k in ("mu", "var"):
        s[k][:] = s[k][:1]
    s["logw"].fill_(-1.0)
    _, idx, resp = G.expert_layer(s["X"], s["P"], s["mu"], s["var"], s["logw"], s["W1"], s["W2"], glu=False, top=3)
    assert (idx.cpu() == torch.tensor([0, 1, 2], dtype=torch.int32)).all()
    assert (resp == torch.tensor(1 / 40).cuda()).all()


@pytest.mark.parametrize("T,K,d,top", [(1, 64, 128, 8), (3, 512, 20, 8), (2, 513, 20, 8), (5, 4096, 7, 3), (4, 4100, 3, 8),
                                       (2, 65536, 2, 2), (128, 65, 128, 2)])
def test_gate_sizes(G, T, K, d, top):
    """Few and many components: picks and responsibilities against 64 bits, experts of one value."""
    s, _ = layer(T, 48, 1, K, d, torch.float32, False, False, False, seed=K)
    _, idx, resp = G.expert_layer(s["X"], s["P"], s["mu"], s["var"], s["logw"], s["W1"], s["W2"], glu=False, top=top)
    want_idx, want_resp, _ = oracle.gate(s["X"], s["P"], s["mu"], s["var"], s["logw"], top, 0.0, False)
    assert torch.equal(idx.cpu().long(), want_idx)
    oracle.check(resp, want_resp, want_resp * (2.0 ** -24 + 1e-9) + 2.0 ** -149, "resp")


def test_empty_batch_and_in_place(G):
    s, opt = layer(0, 64, 40, 6, 12, torch.float16, True, True, True, seed=0)
    y, idx, resp = G.expert_layer(*[s[k] for k in ("X", "P", "mu", "var", "logw", "W1", "W2")], **opt)
    assert y.shape == (0, 64) and idx.shape == (0, 2) and resp.shape == (0, 2)


def test_projection_mixture_lists_and_experts_together(G):
    """As they are used: wide rows projected (gmm_linear), a mixture fitted on the features, rows assigned and listed,
    and a serving batch through the experts, once with the gate inside and once with the picks of gmm_assign_top2."""
    g = torch.Generator().manual_seed(4)
    N, D, d, K, F = 5000, 512, 24, 6, 96
    centres = torch.randn(K, D, generator=g) * 2
    rows = (centres[torch.randint(0, K, (N,), generator=g)] + torch.randn(N, D, generator=g)).to(torch.bfloat16).cuda()
    P = (torch.randn(d, D, generator=g) * D ** -0.5).to(torch.bfloat16).cuda()
    feats, _ = G.linear(rows, P, out_dtype=torch.float32)
    mu, var = feats[:K].clone(), torch.ones(K, d, device="cuda")
    logw = torch.full((K,), -1.79, device="cuda")
    hist = G.em_iterate(feats, mu, var, logw, 4, 1e-3)
    assert (hist[1:] >= hist[:-1] - 1e-6 * hist[:-1].abs()).all()
    idx, resp = G.assign_top2(feats, mu, var, logw)
    offsets, members = G.border_lists(idx, resp, K, 0.05)
    assert int(offsets[-1]) >= N
    W1 = (torch.randn(K, 2 * F, D, generator=g) * D ** -0.5).to(torch.bfloat16).cuda()
    W2 = (torch.randn(K, D, F, generator=g) * F ** -0.5).to(torch.bfloat16).cuda()
    batch = rows[:48].contiguous()
    y, i2, r2 = G.expert_layer(batch, P, mu, var, logw, W1, W2, residual=batch)
    # the features were rounded to float in between: a responsibility moves by that much times its slopes
    sure = (r2.cpu()[:, 0] - r2.cpu()[:, 1] > 1e-3)
    assert sure.any() and torch.equal(i2.cpu()[sure][:, 0], idx[:48].cpu()[sure][:, 0])
    assert (r2.cpu() - resp[:48].cpu()).abs()[sure].max() < 1e-4
    y2 = G.expert_rows(batch, i2, r2, W1, W2, residual=batch)
    assert torch.equal(y, y2)


def test_captured_layer(G):
    s, opt = layer(8, 256, 128, 32, 48, torch.bfloat16, True, False, True, seed=2)
    args = [s[k] for k in ("X", "P", "mu", "var", "logw", "W1", "W2")]
    ws = G.expert_workspace(8, 256, 32, 128, 48, 2, torch.bfloat16, s["X"].device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.expert_layer(*args, ws=ws, **opt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.expert_layer(*args, ws=ws, **opt)
    for i in range(4):
        s["X"].copy_(torch.randn(8, 256, generator=torch.Generator().manual_seed(i)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, G.expert_layer(*args, ws=ws, **opt)):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_two_graphs_share_a_workspace(G):
    """Two captured layers of different sizes on one workspace, replayed in turn: each call sets up what it reads."""
    sets = [layer(T, 128, 64, K, 24, torch.float16, True, True, True, seed=T) for T, K in ((5, 9), (33, 4))]
    ws = torch.empty(max(G.expert_workspace(T, 128, K, 64, 24, 2, torch.float16, "cuda").numel()
                         for T, K in ((5, 9), (33, 4))), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    call = [lambda s=s, o=o: G.expert_layer(*[s[k] for k in ("X", "P", "mu", "var", "logw", "W1", "W2")], ws=ws, **o)
            for s, o in sets]
    want = [[t.clone() for t in c()] for c in call]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in call:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(c())
        graphs.append(g)
    for _ in range(3):
        for g, a, b in zip(graphs, got, want):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_weights_past_32_bit_offsets(G):
    """300 experts of 2 x 1800 x 4096 and 4096 x 1800: the last one's weights lie past 2^31 elements."""
    K, F, D = 300, 1800, 4096
    W1 = torch.zeros(K, 2 * F, D, dtype=torch.bfloat16, device="cuda")
    W2 = torch.zeros(K, D, F, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for k in (0, K - 1):
        W1[k].normal_(generator=g).mul_(D ** -0.5)
        W2[k].normal_(generator=g).mul_(F ** -0.5)
    X = torch.randn(3, D, generator=g, device="cuda").bfloat16()
    idx = torch.tensor([[K - 1, 0], [K - 1, -1], [7, K - 1]], dtype=torch.int32, device="cuda")
    wts = torch.tensor([[0.75, 0.25], [1.0, 0.0], [0.5, 0.5]], device="cuda")
    for top in (2, 1):  # the gathering product, and the one by expert (more picks)
        i, w, x = (idx, wts, X) if top == 2 else (idx.repeat(4, 1), wts.repeat(4, 1), X.repeat(4, 1))
        y = G.expert_rows(x.contiguous(), i.contiguous(), w.contiguous(), W1, W2)
        keep = torch.tensor([0, 7, K - 1])
        small = {0: 0, 7: 1, K - 1: 2, -1: -1}
        j = torch.tensor([[small[int(v)] for v in r] for r in i.cpu()])
        y64, bound = oracle.experts(x, j, w, W1[keep], None, W2[keep], None, "silu", True, None)
        oracle.check(y, y64, bound, "y")


def test_refusals(G):
    s, opt = layer(4, 64, 40, 6, 12, torch.float16, True, True, True, seed=0)
    args = [s[k] for k in ("P", "mu", "var", "logw", "W1", "W2")]
    with pytest.raises(ValueError):
        G.expert_layer(s["X"].float(), *args)
    with pytest.raises(ValueError):
        G.expert_layer(s["X"], *args, glu=False)
    with pytest.raises(ValueError):
        G.expert_layer(s["X"], *args, b1=opt["b1"][:, :3])
    with pytest.raises(ValueError):  # more rows than a call takes
        G.expert_layer(s["X"].repeat(33, 1), *args)
    with pytest.raises(ValueError):
        G.expert_layer(s["X"], *args, top=9)
    with pytest.raises(ValueError):
        G.expert_rows(s["X"], torch.zeros(4, 2, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, device="cuda"),
                      s["W1"], s["W2"])
