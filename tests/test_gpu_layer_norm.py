"""The layer norm (gmm_layer_norm, gmm_layer_norm_backward) against its plain 64-bit form, entry by entry, within bounds
derived from the arithmetic."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# X, Y, weights
COMBOS = [("f32", "f32", "f32"), ("f16", "f16", "f16"), ("bf16", "bf16", "f32"), ("f32", "bf16", "f32"),
          ("f32", "f16", "f16"), ("bf16", "bf16", "bf16")]
# A sum over a row runs over at most 64 elements in a thread, 6 steps over a wave and 16 waves, that over the rows over
# at most N in a thread, a block's 64 groups, 16 slices of at most 64 parts: 96 and N + 160 additions at most, each off
# by 2^-24 of a partial sum. U is a rounding.
ROW, COLUMN, U = 96, 160, 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


def inputs(N, D, x, y, w, seed=0, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    X = (torch.randn(N, D, generator=g) * (0.1 + torch.rand(N, 1, generator=g) * 3)
         + mean * torch.randn(N, 1, generator=g)).to(TYPES[x]).cuda()
    gamma, beta = ((torch.randn(D, generator=g) * 0.3 + o).to(TYPES[w]).cuda() for o in (1, 0))
    return X, gamma, beta, torch.randn(N, D, generator=g).to(TYPES[y]).cuda()


def reference(X, gamma, beta, dY, eps, stats=None):
    """(y, dx, dgamma, dbeta, mean, rstd) in 64 bits and the bounds of all six before their own rounding."""
    x, dy = oracle.wide(X), oracle.wide(dY)
    N, D = x.shape
    ga = torch.ones(D, dtype=torch.float64, device=x.device) if gamma is None else oracle.wide(gamma)
    be = torch.zeros(D, dtype=torch.float64, device=x.device) if beta is None else oracle.wide(beta)
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    h = d * rstd
    y = h * ga + be
    # The deviations are rounded, their mean is off by ROW U mean |d| and rstd by half of the relative error of the sum of
    # squares, ROW + 4, and 2 of its own; the first mean's error e0 leaves (e0 rstd)^2 of the squares' sum
    e0 = ROW * U * x.abs().mean(1, keepdim=True)
    hb = U * (ROW * d.abs().mean(1, keepdim=True) * rstd + h.abs() * (ROW / 2 + 8) * (1 + (e0 * rstd) ** 2)
              + 2 * e0 * rstd)
    yb = hb * ga.abs() + 2 * U * (y.abs() + (h * ga).abs())
    mb = 2 * U * (mean.abs() + e0) + ROW * U * d.abs().mean(1, keepdim=True)
    rb = rstd * U * (ROW / 2 + 8) * (1 + (e0 * rstd) ** 2)
    # the backward pass starts from the rounded mean and rstd
    hb = U * h.abs() * 2 + rstd * mb + d.abs() * rb + U * rstd * mean.abs() * 2
    k = dy * ga
    s1, s2 = k.mean(1, keepdim=True), (k * h).mean(1, keepdim=True)
    dx = rstd * (k - s1 - h * s2)
    s1b = (ROW + 2) * U * k.abs().mean(1, keepdim=True)
    s2b = (ROW + 2) * U * (k * h).abs().mean(1, keepdim=True) + (k.abs() * hb).mean(1, keepdim=True)
    terms = k.abs() + s1.abs() + (h * s2).abs()
    dxb = rstd * (s1b + h.abs() * s2b + hb * (s2.abs() + s2b) + 6 * U * terms) + rb * terms
    dgamma, dbeta = (dy * h).sum(0), dy.sum(0)
    dgb = (dy.abs() * hb).sum(0) + (N + COLUMN) * U * (dy * h).abs().sum(0)
    dbb = (N + COLUMN) * U * dy.abs().sum(0)
    return (y, dx, dgamma, dbeta, mean, rstd), (yb, dxb, dgb, dbb, mb, rb)


def compare(got, want, bound, what):
    oracle.check(got, want, bound + oracle.rounding(want.abs() + bound, got.dtype), what)


# one element, the pieces of every group of threads, one more and one less, and the widest
WIDTHS = [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 96, 128, 129, 200, 255, 256, 257, 512, 513, 777, 1024, 1025, 2048, 2050, 4096, 5000, 8192,
          8193, 16384, 16390, 30000, 32768, 65535, 65536]


@pytest.mark.parametrize("x,y,w", COMBOS)
@pytest.mark.parametrize("D", WIDTHS)
def test_both_passes(G, D, x, y, w):
    N = [1, 2, 5, 33, 70][WIDTHS.index(D) % 5]
    X, gamma, beta, dY = inputs(N, D, x, y, w, seed=D)
    plain = D % 3 == 2
    if plain:
        gamma, beta = None, beta if D % 2 else None
    eps = 1e-5 if D % 2 else 1e-3
    want, bounds = reference(X, gamma, beta, dY, eps)
    Y, stats = G.layer_norm(X, gamma, beta, eps=eps, out_dtype=TYPES[y], want_stats=True)
    compare(Y, want[0], bounds[0], "y")
    compare(stats[:, :1], want[4], bounds[4], "mean")
    compare(stats[:, 1:], want[5], bounds[5], "rstd")
    again, none = G.layer_norm(X, gamma, beta, eps=eps, out_dtype=TYPES[y])
    assert none is None and torch.equal(again, Y)
    got = G.layer_norm_backward(dY, X, stats, gamma, param_dtype=TYPES[w] if plain else None)
    for a, b, bd, what in zip(got, want[1:4], bounds[1:4], ("dx", "dgamma", "dbeta")):
        compare(a, b, bd, what)
    assert got[0].dtype == X.dtype and got[1].dtype == got[2].dtype == TYPES[w]
    for part in range(3):  # each alone is the same
        asked = {f"want_{n}": i == part for i, n in enumerate(("dx", "dgamma", "dbeta"))}
        one = G.layer_norm_backward(dY, X, stats, gamma, param_dtype=TYPES[w] if plain else None, **asked)
        for i in range(3):
            assert one[i] is None if i != part else torch.equal(one[i], got[i])


@pytest.mark.parametrize("x,y,w", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "f16", "f32")])
@pytest.mark.parametrize("N,D", [(70001, 16), (20011, 100), (9001, 520), (5003, 2048), (2999, 4100), (700, 16384),
                                 (700, 20000)])
def test_many_rows(G, monkeypatch, N, D, x, y, w):
    """More rows than the device holds at once."""
    monkeypatch.setattr(oracle, "ON", "cuda")
    X, gamma, beta, dY = inputs(N, D, x, y, w, seed=N)
    want, bounds = reference(X, gamma, beta, dY, 1e-5)
    Y, stats = G.layer_norm(X, gamma, beta, out_dtype=TYPES[y], want_stats=True)
    compare(Y, want[0], bounds[0], "y")
    for a, b, bd, what in zip(G.layer_norm_backward(dY, X, stats, gamma), want[1:4], bounds[1:4],
                              ("dx", "dgamma", "dbeta")):
        compare(a, b, bd, what)
        if a.dtype == torch.float32:  # the worst case is far: errors of either sign add up as their root
            assert (a.double() - b).norm() <= 2e-6 * b.norm(), what


def test_mean_far_from_zero_and_constant_rows(G):
    X, gamma, beta, dY = inputs(40, 300, "f32", "f32", "f32", seed=3, mean=1000.0)
    X[7] = 4096.25
    X[8] = 0
    want, bounds = reference(X, gamma, beta, dY, 1e-5)
    Y, stats = G.layer_norm(X, gamma, beta, want_stats=True)
    compare(Y, want[0], bounds[0], "y")
    assert torch.equal(Y[7], beta) and torch.equal(Y[8], beta)
    for a, b, bd, what in zip(G.layer_norm_backward(dY, X, stats, gamma), want[1:4], bounds[1:4],
                              ("dx", "dgamma", "dbeta")):
        compare(a, b, bd, what)


def test_gradients_against_differences(G):
    """The formula itself: central differences of the 64-bit form along random directions."""
    X, gamma, beta, dY = inputs(9, 37, "f32", "f32", "f32", seed=11)
    _, stats = G.layer_norm(X, gamma, beta, want_stats=True)
    grads = [g.cpu().double() for g in G.layer_norm_backward(dY, X, stats, gamma)]
    base = [t.cpu().double() for t in (X, gamma, beta)]

    def loss(x, ga, be):
        d = x - x.mean(1, keepdim=True)
        return float(((d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * ga + be) * dY.cpu().double()).sum())
    g = torch.Generator().manual_seed(0)
    for at, grad in enumerate(grads):
        v = torch.randn(base[at].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        ends = [loss(*[t + (s * v if i == at else 0) for i, t in enumerate(base)]) for s in (h, -h)]
        slope = float((grad * v).sum())
        # the differences are good to h^2, the gradient to float roundings of its entries
        assert abs((ends[0] - ends[1]) / (2 * h) - slope) <= 1e-5 * float((grad * v).abs().sum()) + 1e-6


def test_what_is_not_finite_stays_in_its_row(G):
    for D in (20, 300, 3000, 20000):
        X, gamma, beta, dY = inputs(6, D, "f32", "f32", "f32", seed=D)
        clean, stats = G.layer_norm(X, gamma, beta, want_stats=True)
        dx, _, _ = G.layer_norm_backward(dY, X, stats, gamma)
        bad = X.clone()
        bad[1, D // 2], bad[4, 0] = float("nan"), float("inf")
        Y, st = G.layer_norm(bad, gamma, beta, want_stats=True)
        dxb, _, dbeta = G.layer_norm_backward(dY, bad, st, gamma)
        rows = torch.tensor([0, 2, 3, 5], device="cuda")
        assert torch.equal(Y[rows], clean[rows]) and torch.equal(dxb[rows], dx[rows])
        assert Y[1].isnan().all() and Y[4].isnan().any() and dbeta.isfinite().all()


@pytest.mark.parametrize("D", [5, 77, 1023, 4099, 16383, 20001, 65535])
def test_rows_from_any_element_and_in_place(G, D):
    """Views that start off every 16-byte border, outputs over their inputs, and nothing written beside them."""
    t = torch.float16
    X, gamma, beta, dY = inputs(11, D, "f16", "f16", "f16", seed=D)
    Y, stats = G.layer_norm(X, gamma, beta, want_stats=True)
    grads = G.layer_norm_backward(dY, X, stats, gamma)
    for o in (1, 3):
        def place(src):
            flat = torch.full((src.numel() + 64,), 7.0, dtype=t, device="cuda")
            flat[o:o + src.numel()] = src.reshape(-1)
            return flat, flat[o:o + src.numel()].view(src.shape)
        xf, x = place(X)
        gf, ga = place(gamma)
        bf, be = place(beta)
        st = torch.empty_like(stats)
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        L = G.lib()
        assert L.gmm_layer_norm(x.data_ptr(), 1, 11, D, ga.data_ptr(), be.data_ptr(), 1, 1e-5, x.data_ptr(), 1,
                                st.data_ptr(), s) == 0
        assert torch.equal(x, Y) and torch.equal(st, stats)
        df, d = place(dY)
        ws = G.layer_norm_workspace(11, D, t, "cuda")
        dg, db = torch.empty_like(gamma), torch.empty_like(beta)
        assert L.gmm_layer_norm_backward(d.data_ptr(), 1, X.data_ptr(), 1, 11, D, st.data_ptr(), ga.data_ptr(), 1,
                                         d.data_ptr(), dg.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
        assert torch.equal(d, grads[0]) and torch.equal(dg, grads[1]) and torch.equal(db, grads[2])
        for flat, n in ((xf, X.numel()), (df, dY.numel()), (gf, D), (bf, D)):
            assert (flat[:o] == 7).all() and (flat[o + n:] == 7).all()


def test_offsets_past_32_bits(G):
    N, D = 140001, 16400
    X = torch.empty(N, D, dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for i in range(0, N, 20000):
        X[i:i + 20000] = torch.randn(min(20000, N - i), D, generator=g, device="cuda", dtype=torch.float16)
    Y, stats = G.layer_norm(X, want_stats=True)
    # sums of N ones: half ends at 65504, so the weights' gradients are float
    dx, dg, db = G.layer_norm_backward(Y, X, stats, param_dtype=torch.float32)
    for r in (0, 70000, 131000, N - 1):
        one, st = G.layer_norm(X[r:r + 1], want_stats=True)
        assert torch.equal(one[0], Y[r]) and torch.equal(st[0], stats[r])
        assert torch.equal(G.layer_norm_backward(Y[r:r + 1], X[r:r + 1], st)[0][0], dx[r])
    # Y is h in half: the sum over N of h^2 is N, and its roundings leave 2^-11 of it at most
    total = float(dg.double().sum()) / D
    assert abs(total - N) <= N * (2.0 ** -10) and db.isfinite().all()


def test_no_rows(G):
    X, gamma, beta, dY = inputs(3, 40, "f16", "f16", "f16")
    Y, stats = G.layer_norm(X[:0], gamma, beta, want_stats=True)
    assert Y.shape == (0, 40) and stats.shape == (0, 2)
    dx, dg, db = G.layer_norm_backward(dY[:0], X[:0], stats, gamma)
    assert dx.shape == (0, 40) and (dg == 0).all() and (db == 0).all()


@pytest.mark.parametrize("x,y,w", COMBOS)
def test_graph(G, x, y, w):
    """torch's graph gives layer_norm_backward's gradients, from a loss whose gradient has strides of zero too."""
    X, gamma, beta, dY = inputs(21, 77, x, y, w, seed=5)
    with torch.no_grad():
        want, stats = G.layer_norm(X, gamma, beta, out_dtype=TYPES[y], want_stats=True)
        grads = G.layer_norm_backward(dY, X, stats, gamma)
    for t in (X, gamma, beta):
        t.requires_grad_()
    Y, none = G.layer_norm(X, gamma, beta, out_dtype=TYPES[y])
    assert none is None and torch.equal(Y, want)
    for a, b in zip(torch.autograd.grad(Y, (X, gamma, beta), dY), grads):
        assert torch.equal(a, b) and a.dtype == b.dtype
    Y, st = G.layer_norm(X, gamma, beta, out_dtype=TYPES[y], want_stats=True)
    assert not st.requires_grad and torch.equal(st, stats)
    (db,) = torch.autograd.grad(Y.sum(), (beta,))
    assert (db == 21).all()
    with pytest.raises(RuntimeError, match="no second derivatives"):
        torch.autograd.grad(G.layer_norm(X, gamma, beta, out_dtype=TYPES[y])[0].sum(), X, create_graph=True)
    only = G.layer_norm(X.detach(), None, beta, out_dtype=TYPES[y])[0]
    (b,) = torch.autograd.grad(only, (beta,), dY)
    assert torch.equal(b, grads[2])


def test_captured_and_replayed(G):
    X, gamma, beta, dY = inputs(300, 700, "bf16", "bf16", "bf16", seed=9)
    x, dy = X.clone(), dY.clone()
    ws = G.layer_norm_workspace(300, 700, torch.bfloat16, "cuda")

    def step():
        Y, st = G.layer_norm(x, gamma, beta, want_stats=True)
        return (Y, *G.layer_norm_backward(dy, x, st, gamma, ws=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(X.roll(i, 0) * (i + 1))
        dy.copy_(dY.roll(2 * i, 1))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_refusals(G):
    X, gamma, beta, dY = inputs(4, 24, "bf16", "bf16", "bf16")
    _, stats = G.layer_norm(X, gamma, beta, want_stats=True)
    for call in (lambda: G.layer_norm(X.t(), gamma, beta), lambda: G.layer_norm(X.cpu(), gamma, beta),
                 lambda: G.layer_norm(X, gamma[:-1], beta), lambda: G.layer_norm(X, gamma, beta.float()),
                 lambda: G.layer_norm(X, gamma.half(), beta.half()), lambda: G.layer_norm(X, out_dtype=torch.float32),
                 lambda: G.layer_norm(X.double()), lambda: G.layer_norm(X.float(), out_dtype=torch.float64),
                 lambda: G.layer_norm_backward(dY.float(), X, stats, gamma),
                 lambda: G.layer_norm_backward(dY[:-1], X, stats, gamma),
                 lambda: G.layer_norm_backward(dY, X, stats[:-1], gamma),
                 lambda: G.layer_norm_backward(dY, X, stats.half(), gamma),
                 lambda: G.layer_norm_backward(dY, X, stats, gamma, ws=torch.empty(8, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: G.layer_norm(X, eps=0.0), lambda: G.layer_norm(X, eps=float("nan")),
                 lambda: G.layer_norm_backward(dY, X, stats, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(G.GmmError):
            call()
