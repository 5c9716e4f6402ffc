"""The cross entropy of a linear head (gmm_cross_entropy, gmm_cross_entropy_gradients) against its plain 64-bit form,
entry by entry, within bounds derived from the arithmetic."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
# additions that an entry of a row's sum passes through, and the exponentials that rescale it: at most 64 in a lane, 32
# parts in a lane, 6 steps over the wave and 16 waves, with 4 roundings each
SUM = 4 * (64 + 32 + 6 + 16)


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


def inputs(N, d, V, top, t, soft, bias, seed=0, masked=0.2, on="cpu"):
    g = torch.Generator(device=on).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=on)
    X, W = normal(N, d).to(t).cuda(), (normal(V, d) * 2 * d ** -0.5).to(t).cuda()
    idx = torch.randint(-1, V + 1, (N, top), generator=g, device=on, dtype=torch.int32)
    idx[torch.rand(N, generator=g, device=on) < masked] = -1
    if top > 1:
        idx[::3, 1] = idx[::3, 0]  # a class picked twice
    wts = None
    if soft:
        wts = torch.rand(N, top, generator=g, device=on)
        wts[::5, 0] = 0
    dloss = normal(N)
    dloss[3::7] = 0
    return (X, W, (normal(V) * 0.5).to(t).cuda() if bias else None, idx.cuda(), None if wts is None else wts.cuda(),
            dloss.cuda())


def reference(X, W, bias, idx, wts, dloss):
    """(loss, lse, dx, dw, db) in 64 bits, and the bounds of all five before the outputs' rounding."""
    x, w, b = oracle.wide(X), oracle.wide(W), oracle.wide(bias)
    N, V = x.shape[0], w.shape[0]
    z = x @ w.T
    zb = oracle.sum_bound(x, w, x.shape[1])
    if b is not None:
        z = z + b
        zb += 2 * U * z.abs()
    lse = torch.logsumexp(z, 1)
    most = z.amax(1)
    p = torch.exp(z - lse[:, None])
    far = (most[:, None] - z).clamp(max=90)  # beyond it the exponential is 0
    lb = (p * (zb + 2 * U * far)).sum(1) + SUM * U
    lseb = lb + 4 * U * (most.abs() + lse.abs() + (lse - most).abs())
    i = idx.to(x.device).long()
    i = i[:, None] if i.dim() == 1 else i
    real = (i >= 0) & (i < V)
    c = real.double() if wts is None else torch.where(real, oracle.wide(wts).view(i.shape), 0.0)
    i = torch.where(real, i, 0)
    picked = torch.gather(z, 1, i)
    terms = lse[:, None] - picked
    # the picks' logits are a sum of their own, or the product's
    off = lseb[:, None] + torch.gather(zb, 1, i) + 4 * U * (most[:, None].abs() + picked.abs())
    loss, lossb = (c * terms).sum(1), (c.abs() * (off + 10 * U * (terms.abs() + off))).sum(1)
    d = torch.ones(N, dtype=torch.float64, device=x.device) if dloss is None else oracle.wide(dloss)
    s = c.sum(1)
    grad = d[:, None] * s[:, None] * p
    # p is off by its logit's error and the sum's, and the roundings of the exponential and of three products
    gb = grad.abs() * (zb + lb[:, None] + 2 * U * far + 16 * U)
    if X.dtype != torch.float32:  # a difference from a largest logit around it in half: half a step, 2^-11 of it
        gb += grad.abs() * (2.0 ** -11 * far + 2.0 ** -25)
    gb += (d * c.abs().sum(1))[:, None].abs() * p * 10 * U  # s may cancel
    grad.scatter_add_(1, i, -d[:, None] * c)
    pick = torch.zeros_like(grad).scatter_add_(1, i, (d[:, None] * c).abs())
    gb += 10 * U * pick
    if X.dtype != torch.float32:  # rounded to the operands' type, of which the scale makes the largest pick 2^11
        largest = float((d.abs() * c.abs().amax(1)).max()) if N else 0.0
        gb += (grad.abs() + gb) * (oracle.EPS[X.dtype] / 2 + 4 * U) + oracle.TINY[X.dtype] * max(largest, 1e-30) / 2048
    dx, dw, db = grad @ w, grad.T @ x, grad.sum(0)
    size = grad.abs() + gb
    dxb = gb @ w.abs() + oracle.sum_bound(size, w.T, V) + 2 * U * dx.abs()
    # the rows' pieces are added up in float
    dwb = gb.T @ x.abs() + oracle.sum_bound(size.T, x.T, N) + 8 * U * dw.abs()
    dbb = gb.sum(0) + (N + 300) * 2 * U * size.sum(0)
    return (loss, lse, dx, dw, db), (lossb, lseb, dxb, dwb, dbb)


def compare(got, want, bound, what):
    oracle.check(got, want, bound + oracle.rounding(want.abs() + bound, got.dtype), what)


NAMES = ("loss", "lse", "dx", "dw", "db")
# rows, features, classes, picks: one of each; few rows (up to 16), also of very many classes; sizes that no tile or
# 16-byte piece divides; long contractions with few outputs (split); rows of more classes than a wave or a block strides
SHAPES = [(1, 1, 1, 1), (1, 64, 5, 2), (2, 7, 300, 1), (16, 64, 1000, 3), (5, 24, 70001, 1), (17, 129, 31, 2),
          (65, 72, 200, 1), (130, 8, 2600, 8), (256, 512, 256, 1), (513, 264, 5000, 2), (1000, 96, 96, 1),
          (300, 4096, 24, 2), (700, 1, 19, 1), (20, 40, 33000, 2), (129, 1000, 4097, 1), (33, 3000, 2049, 4)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "x".join(map(str, SHAPES[i])))
def test_against_64_bits(G, monkeypatch, i, dtype):
    monkeypatch.setattr(oracle, "ON", "cuda")
    N, d, V, top = SHAPES[i]
    soft, bias = i % 2 == 0, i % 3 != 1
    X, W, b, idx, wts, dloss = inputs(N, d, V, top, TYPES[dtype], soft, bias, seed=i)
    if i % 5 == 2:
        dloss = None
    want, bounds = reference(X, W, b, idx, wts, dloss)
    loss, lse = G.cross_entropy(X, W, idx, wts=wts, bias=b)
    compare(loss, want[0], bounds[0], "loss")
    compare(lse, want[1], bounds[1], "lse")
    got = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    for a, w, bd, what in zip(got, want, bounds, NAMES):
        compare(a, w, bd, what)
    for part in ("dx", "dw", "db"):  # each alone is the same
        asked = {f"want_{n}": n == part for n in ("dx", "dw", "db")}
        one = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b, **asked)
        for a, o, n in zip(got, one, NAMES):
            assert o is None if n in ("dx", "dw", "db") and n != part else torch.equal(a, o)
    if top == 1:  # labels as kmeans_assign gives them
        flat = G.cross_entropy_gradients(X, W, idx[:, 0].contiguous(), dloss=dloss,
                                         wts=None if wts is None else wts[:, 0].contiguous(), bias=b)
        assert all(torch.equal(a, o) for a, o in zip(got, flat))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,V", [(4090, 520, 8190), (4090, 200, 8190), (8200, 1000, 2050), (2040, 136, 33001), (4090, 72, 4101),
                                   (5001, 100, 90), (4999, 700, 300)])
def test_large_tiles(G, monkeypatch, N, d, V, dtype):
    monkeypatch.setattr(oracle, "ON", "cuda")
    t = TYPES[dtype]
    X, W, b, idx, wts, _ = inputs(N, d, V, 2, t, True, True, seed=N)
    dloss = torch.full((N,), 1 / N, device="cuda")
    want, bounds = reference(X, W, b, idx, wts, dloss)
    got = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    for a, w, bd, what in zip(got, want, bounds, NAMES):
        compare(a, w, bd, what)
        # the bounds are those of the worst signs; in the 2-norm two roundings remain, G's and the output's
        off = float((a.double() - w).norm() / w.norm())
        assert off <= (1e-5 if a.dtype == torch.float32 else 2 * oracle.EPS[t] / 2), (what, off)
    for part in ("dx", "dw", "db"):  # each alone is the same
        asked = {f"want_{n}": n == part for n in ("dx", "dw", "db")}
        one = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b, **asked)
        assert all(o is None or torch.equal(a, o) for a, o in zip(got, one))
    loss, lse = G.cross_entropy(X, W, idx, wts=wts, bias=b)
    compare(loss, want[0], bounds[0], "loss")
    compare(lse, want[1], bounds[1], "lse")


@pytest.mark.parametrize("dtype,N,d", [("f32", 1100, 16), ("f16", 1100, 16), ("bf16", 1100, 16), ("bf16", 600, 904)])
def test_pieces_of_rows(G, dtype, N, d):
    """A million classes: 512 rows of logits at a time, with dW and db summed over the pieces."""
    V = 1 << 20
    t = TYPES[dtype]
    X, W, b, idx, wts, dloss = inputs(N, d, V, 2, t, True, True, seed=3, on="cuda")
    got = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    fwd = G.cross_entropy(X, W, idx, wts=wts, bias=b)
    dw, db = torch.zeros(V, d, dtype=torch.float64, device="cuda"), torch.zeros(V, dtype=torch.float64, device="cuda")
    for r in range(0, N, 512):  # in pieces in 64 bits too, with memory for the bounds
        part = slice(r, min(N, r + 512))
        x, w = X[part].double(), W.double()
        z = x @ w.T + b.double()
        lse = torch.logsumexp(z, 1)
        i = idx[part].long()
        real = (i >= 0) & (i < V)
        c = torch.where(real, wts[part].double(), 0.0)
        i = torch.where(real, i, 0)
        loss = (c * (lse[:, None] - torch.gather(z, 1, i))).sum(1)
        # |z| is below 16 here, so a logit is off by (d + 8) 2^-23 of 16 d^(1/2) at most: far below 1e-4
        for out in (got, fwd):
            assert (out[0][part].double() - loss).abs().max() < 2e-4 and (out[1][part].double() - lse).abs().max() < 1e-4
        g = z.sub_(lse[:, None]).exp_().mul_((dloss[part].double() * c.sum(1))[:, None])
        g.scatter_add_(1, i, -dloss[part].double()[:, None] * c)
        dx = g @ w
        # G's entries are off by 1e-4 of themselves and a rounding; errors of either sign add up as their root
        assert (got[2][part].double() - dx).norm() <= (2e-4 + 2 * oracle.EPS[t] / 2) * dx.norm()
        dw += g.T @ x
        db += g.sum(0)
        del z, g
    for a, w, what in ((got[3], dw, "dw"), (got[4], db, "db")):
        assert (a.double() - w).norm() <= (2e-4 + 2 * oracle.EPS[t] / 2) * w.norm(), what
    # pieces of another size, the same rows: the last piece alone
    tail = slice(N // 512 * 512, N)
    alone = G.cross_entropy_gradients(X[tail], W, idx[tail], dloss=dloss[tail], wts=wts[tail], bias=b)
    assert (alone[1] - got[1][tail]).abs().max() < 1e-4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_of_few_classes(G, monkeypatch, dtype):
    """Thousands of tiles, each with sums of the bias's gradient."""
    monkeypatch.setattr(oracle, "ON", "cuda")
    N, d, V, t = 70001, 16, 130, TYPES[dtype]
    X, W, b, idx, wts, _ = inputs(N, d, V, 2, t, True, True, seed=1)
    dloss = torch.full((N,), 1 / N, device="cuda")
    want, bounds = reference(X, W, b, idx, wts, dloss)
    got = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    for a, w, bd, what in zip(got, want, bounds, NAMES):
        compare(a, w, bd, what)
        # errors of either sign add up as their root: of a sum of 70001 terms, and two roundings
        assert (a.double() - w).norm() <= (1e-5 if t == torch.float32 else 2 * oracle.EPS[t] / 2) * w.norm(), what


def test_gradients_against_differences(G):
    X, W, b, idx, wts, dloss = inputs(9, 12, 31, 2, torch.float32, True, True, seed=11)
    _, _, *grads = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    base = [t.cpu().double() for t in (X, W, b)]
    i = idx.cpu().long()
    real = (i >= 0) & (i < 31)
    c = torch.where(real, wts.cpu().double(), 0.0)

    def loss(x, w, bb):
        z = x @ w.T + bb
        return float((dloss.cpu().double() * (c * (torch.logsumexp(z, 1)[:, None]
                                                   - torch.gather(z, 1, torch.where(real, i, 0)))).sum(1)).sum())
    g = torch.Generator().manual_seed(0)
    for at, grad in enumerate(grads):
        v = torch.randn(base[at].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        ends = [loss(*[t + (s * v if k == at else 0) for k, t in enumerate(base)]) for s in (h, -h)]
        grad = grad.cpu().double()
        assert abs((ends[0] - ends[1]) / (2 * h) - float((grad * v).sum())) <= 1e-5 * float((grad * v).abs().sum()) + 1e-6


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("N,V", [(12, 40), (300, 3000)])
def test_rows_without_a_gradient_hold_anything(G, dtype, N, V):
    """Rows of no picks, of picks that weigh nothing and of a loss that nobody asks for, with NaN and infinity in X."""
    t = TYPES[dtype]
    X, W, b, idx, wts, dloss = inputs(N, 72, V, 2, t, True, True, seed=5, masked=0.0)
    idx, wts = idx.clamp(0, V - 1), wts + 0.1
    idx[1], idx[4] = -1, V
    wts[6] = 0
    dloss[8] = 0
    off = torch.tensor([1, 4, 6, 8], device="cuda")
    clean = X.clone()
    clean[off] = 0
    bad = X.clone()
    bad[off[0]], bad[off[1], 5], bad[off[2]], bad[off[3], 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    want = G.cross_entropy_gradients(clean, W, idx, dloss=dloss, wts=wts, bias=b)
    got = G.cross_entropy_gradients(bad, W, idx, dloss=dloss, wts=wts, bias=b)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[off] = False
    for a, w in zip(got[2:], want[2:]):
        assert torch.equal(a, w) and a.isfinite().all()
    assert (got[2][off] == 0).all() and (got[0][off[:3]] == 0).all()
    assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1][rest], want[1][rest])
    fwd = G.cross_entropy(bad, W, idx, wts=wts, bias=b)
    assert (fwd[0][off[:3]] == 0).all() and fwd[1][off[0]].isnan() and fwd[0][rest].isfinite().all()
    none = G.cross_entropy_gradients(bad, W, torch.full_like(idx, -1), wts=wts, bias=b)
    assert all((a == 0).all() for a in (none[0], *none[2:]))


@pytest.mark.parametrize("N", [7, 200])
def test_classes_taken_out(G, N):
    """A bias of -infinity (a weight of 0), or of the type's lowest value, leaves a class out, tiles of them too."""
    V, keep = 700, torch.arange(700) % 3 == 1
    keep[64:400] = False
    X, W, b, idx, wts, dloss = inputs(N, 40, V, 2, torch.bfloat16, True, True, seed=8)
    kept = keep.nonzero()[:, 0].int().cuda()
    few = torch.randint(0, len(kept), idx.shape, device="cuda")
    small = G.cross_entropy_gradients(X, W[keep].contiguous(), few.int(), dloss=dloss, wts=wts, bias=b[keep].contiguous())
    for low in (float("-inf"), torch.finfo(torch.bfloat16).min):
        masked = torch.where(keep.cuda(), b, torch.full_like(b, low))
        for out in (G.cross_entropy_gradients(X, W, kept[few], dloss=dloss, wts=wts, bias=masked),
                    G.cross_entropy(X, W, kept[few], wts=wts, bias=masked)):
            # |z| is below 16 and a sum of 40 products: both are off by 1e-4 at most
            assert (out[0] - small[0]).abs().max() < 2e-4 and (out[1] - small[1]).abs().max() < 1e-4
            if len(out) == 5:
                assert (out[3][~keep] == 0).all() and (out[4][~keep] == 0).all()
                for a, w in ((out[2], small[2]), (out[3][keep], small[3]), (out[4][keep], small[4])):
                    assert (a.double() - w.double()).norm() <= (2e-4 + 2.0 ** -7) * w.double().norm()
    gone = (~keep).nonzero()[0, 0].int()
    masked = torch.where(keep.cuda(), b, torch.full_like(b, float("-inf")))
    loss, _ = G.cross_entropy(X, W, torch.full((N,), int(gone), dtype=torch.int32, device="cuda"), bias=masked)
    assert (loss == float("inf")).all()
    loss, lse = G.cross_entropy(X, W, kept[few], wts=wts, bias=torch.full_like(b, float("-inf")))
    assert (lse == float("-inf")).all()


def test_extreme_logits(G):
    """Logits far apart, and a loss that is nearly 0: lse - z loses nothing to the size of either."""
    V = 300
    X, W = torch.eye(20, 24, device="cuda") * 200, torch.zeros(V, 24, device="cuda")
    W[:24] = torch.eye(24, device="cuda")
    idx = torch.arange(20, device="cuda", dtype=torch.int32)
    loss, lse, dx, dw, _ = G.cross_entropy_gradients(X, W, idx)
    assert (loss.abs() < 1e-6).all() and (lse == 200).all() and dx.abs().max() < 1e-30
    loss, lse, dx, _, _ = G.cross_entropy_gradients(-X, W, idx)
    assert ((loss - 200 - torch.tensor(299.0).log()).abs() < 1e-4).all()
    off, _ = G.cross_entropy(X * 1e30, W, (idx + 1) % 20)
    assert (off > 1e31).all() and off.isfinite().all()


@pytest.mark.parametrize("N", [5, 700])
@pytest.mark.parametrize("top", [1, 3, 7])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weights_that_all_rows_share(G, dtype, top, N):
    """Under a mean all picks weigh the same: whatever that is, its rounding is no common factor of the gradients."""
    t = TYPES[dtype]
    for seed, share in enumerate((1 / N, 1 / 7373, 1 / 3, 0.7)):
        X, W, _, idx, _, _ = inputs(N, 104, 20000, top, t, False, False, seed=seed)
        dloss = torch.full((N,), share, device="cuda")
        (_, _, dx, dw, _), _ = reference(X.cpu(), W.cpu(), None, idx.cpu(), None, dloss.cpu())
        got = G.cross_entropy_gradients(X, W, idx, dloss=dloss, want_db=False)
        for a, w in ((got[2], dx), (got[3], dw)):
            # The outputs' own rounding, and G's: a pick's entry 2^11 (1 - p) is off by half a step below 2^11, u / 2 (u
            # half a step above), u / 2 / sqrt 3 in the root mean square; the other entries' squares sum to exp(2^2) /
            # 20000 of a pick's for logits of deviation 2, times 7 picks at most: 0.02 u^2 / 3. Together 0.30 u. 1.1 for
            # the fluctuation of a norm over 520 entries.
            u = torch.finfo(t).eps / 2
            rounded = float((w.to(t).double() - w).norm() / w.norm())
            off = float((a.cpu().double() - w).norm() / w.norm())
            assert off <= 1.1 * (rounded ** 2 + (0.31 * u) ** 2) ** 0.5, (seed, share, off, rounded)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-12, 1e-4, 1.0, 1e6])
def test_gradients_of_any_size(G, monkeypatch, dtype, size):
    """A float dloss far outside half's range: the scale keeps the products' operands inside it."""
    monkeypatch.setattr(oracle, "ON", "cuda")
    t = TYPES[dtype]
    X, W, b, idx, wts, dloss = inputs(200, 64, 500, 1, t, False, True, seed=4)
    unit = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    got = G.cross_entropy_gradients(X, W, idx, dloss=dloss * size, wts=wts, bias=b)
    if t == torch.bfloat16:
        for a, u in zip(got[2:], unit[2:]):
            assert (a.double() / size - u.double()).norm() <= 2.0 ** -6 * u.double().norm()
    else:
        want, bounds = reference(X, W, b, idx, wts, dloss * size)
        for a, w, bd, what in zip(got[2:], want[2:], bounds[2:], NAMES[2:]):
            over = w.abs() + bd >= 65504  # half ends there
            assert torch.equal(a.isinf() & ~over, torch.zeros_like(over))
            fine = ~over
            compare(torch.where(fine, a, torch.zeros_like(a)), torch.where(fine, w, 0.0), bd, what)


def test_rows_from_any_element(G):
    """Rows that are no whole 16-byte pieces may start anywhere; others are refused off a border."""
    X, W, b, idx, wts, dloss = inputs(90, 45, 333, 2, torch.float16, True, True, seed=2)
    want = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    flat = torch.zeros(X.numel() + 1, dtype=X.dtype, device="cuda")
    flat[1:] = X.reshape(-1)
    x = flat[1:].view(X.shape)
    for a, w in zip(G.cross_entropy_gradients(x, W, idx, dloss=dloss, wts=wts, bias=b), want):
        assert torch.equal(a, w)
    for a, w in zip(G.cross_entropy(x, W, idx, wts=wts, bias=b), G.cross_entropy(X, W, idx, wts=wts, bias=b)):
        assert torch.equal(a, w)
    y = flat[1:1 + 80 * 48].view(80, 48)
    for call in (lambda: G.cross_entropy(y, y[:20], idx[:80]), lambda: G.cross_entropy_gradients(y, y[:20], idx[:80])):
        with pytest.raises(G.GmmError):
            call()


def test_no_rows(G):
    X, W, b, idx, _, _ = inputs(3, 40, 50, 1, torch.float16, False, True)
    loss, lse = G.cross_entropy(X[:0], W, idx[:0], bias=b)
    assert loss.shape == lse.shape == (0,)
    _, _, dx, dw, db = G.cross_entropy_gradients(X[:0], W, idx[:0], bias=b)
    assert dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_graph(G, dtype):
    X, W, b, idx, wts, dloss = inputs(70, 45, 333, 2, TYPES[dtype], True, True, seed=6)
    want = G.cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=b)
    for t in (X, W, b):
        t.requires_grad_()
    loss, lse = G.cross_entropy(X, W, idx, wts=wts, bias=b)
    ws = G.cross_entropy_workspace(70, 45, 333, TYPES[dtype], "cuda")
    assert torch.equal(G.cross_entropy(X, W, idx, wts=wts, bias=b, ws=ws)[0], loss)
    assert loss.requires_grad and not lse.requires_grad
    for a, w in zip(torch.autograd.grad(loss, (X, W, b), dloss), want[2:]):
        assert torch.equal(a, w)
    (dw,) = torch.autograd.grad(G.cross_entropy(X.detach(), W, idx, wts=wts, bias=b.detach())[0], W, dloss)
    assert torch.equal(dw, want[3])
    mean = torch.autograd.grad(G.cross_entropy(X, W, idx, wts=wts, bias=b)[0].mean(), (X, W, b))
    even = G.cross_entropy_gradients(X.detach(), W.detach(), idx, dloss=torch.full((70,), 1 / 70, device="cuda"), wts=wts,
                                     bias=b.detach())
    assert all(torch.equal(a, w) for a, w in zip(mean, even[2:]))
    with pytest.raises(RuntimeError, match="no second derivatives"):
        torch.autograd.grad(G.cross_entropy(X, W, idx, wts=wts, bias=b)[0].sum(), X, create_graph=True)
    wts.requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient of wts"):
        G.cross_entropy(X, W, idx, wts=wts, bias=b)[0].sum().backward()


def test_captured_and_replayed(G):
    X, W, b, idx, wts, dloss = inputs(200, 136, 900, 2, torch.bfloat16, True, True, seed=6)
    x, i = X.clone(), idx.clone()
    ws = G.cross_entropy_workspace(200, 136, 900, torch.bfloat16, "cuda", gradients=True)
    ws2 = G.cross_entropy_workspace(200, 136, 900, torch.bfloat16, "cuda")

    def step():
        return (*G.cross_entropy_gradients(x, W, i, dloss=dloss, wts=wts, bias=b, ws=ws),
                *G.cross_entropy(x, W, i, wts=wts, bias=b, ws=ws2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(X.roll(k, 0))
        i.copy_(idx.roll(3 * k, 0))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, w in zip(got, step()):
            assert torch.equal(a, w)


def test_overlapping_streams(G):
    """Calls on two streams at once, each with scratch of its own."""
    made = [inputs(300, 264, 2000, 1, torch.float16, False, True, seed=s) for s in (0, 1)]
    want = [G.cross_entropy_gradients(m[0], m[1], m[3], dloss=m[5], bias=m[2]) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        got = []
        for m, s in zip(made, streams):
            with torch.cuda.stream(s):
                got.append(G.cross_entropy_gradients(m[0], m[1], m[3], dloss=m[5], bias=m[2]))
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, w))


def test_refusals(G):
    X, W, b, idx, wts, dloss = inputs(20, 24, 30, 2, torch.bfloat16, True, True)
    for call in (lambda: G.cross_entropy(X.t(), W, idx), lambda: G.cross_entropy(X, W.float(), idx),
                 lambda: G.cross_entropy(X, W[:, :-1], idx), lambda: G.cross_entropy(X, W, idx.long()),
                 lambda: G.cross_entropy(X, W, idx[:-1]), lambda: G.cross_entropy(X, W, idx, wts=wts[:, :1]),
                 lambda: G.cross_entropy(X, W, idx, wts=wts.half()), lambda: G.cross_entropy(X, W, idx, bias=b[1:]),
                 lambda: G.cross_entropy(X, W, idx, bias=b.float()), lambda: G.cross_entropy(X, W, idx.cpu()),
                 lambda: G.cross_entropy(X, W, idx[None]), lambda: G.cross_entropy(X.double(), W.double(), idx),
                 lambda: G.cross_entropy_gradients(X, W, idx, dloss=dloss[:-1]),
                 lambda: G.cross_entropy_gradients(X, W, idx, dloss=dloss.half()),
                 lambda: G.cross_entropy_gradients(X, W, idx, ws=torch.empty(8, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    nine = torch.zeros(20, 9, dtype=torch.int32, device="cuda")
    for call in (lambda: G.cross_entropy(X, W, nine), lambda: G.cross_entropy_gradients(X, W, nine),
                 lambda: G.cross_entropy(X, W, idx, ws=torch.empty(8, dtype=torch.uint8, device="cuda")),
                 lambda: G.cross_entropy_gradients(X, W, idx, ws=torch.empty(512, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(G.GmmError):
            call()
