"""The linear layer (gmm_linear, gmm_linear_backward) against its plain 64-bit form, entry by entry, within bounds
derived from the arithmetic (tests/layer_oracle.py)."""
import ctypes

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


def act_of(G, name):
    return getattr(G, "ACT_" + name.upper())


def inputs(N, d_in, d_out, dtype, out, bias, residual, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, t=dtype):
        return torch.randn(*shape, generator=g).to(t).cuda()
    X, W = normal(N, d_in), (normal(d_out, d_in, t=torch.float32) * d_in ** -0.5).to(dtype)
    return X, W, normal(d_out) if bias else None, normal(N, d_out, t=out) if residual else None, normal(N, d_out, t=out)


# rows, d_in, d_out: one value; few rows (one, two and four groups of 16); just above; sizes that no tile or 16-byte
# piece divides; exact tiles; long contractions with few outputs (split); one output column
SHAPES = [(1, 1, 1), (1, 4096, 33), (2, 7, 300), (16, 64, 64), (17, 129, 31), (64, 500, 130), (65, 72, 200),
          (127, 1023, 77), (128, 128, 128), (130, 8, 260), (256, 512, 256), (513, 264, 520), (1000, 96, 96),
          (300, 8192, 24), (2050, 40, 1), (700, 1, 19), (1500, 200, 513)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "x".join(map(str, SHAPES[i])))
def test_forward(G, i, dtype):
    N, d_in, d_out = SHAPES[i]
    for name in oracle.ACTS[i % 2::2]:
        out = torch.float32 if (i + len(name)) % 3 == 0 else TYPES[dtype]
        X, W, b, R, _ = inputs(N, d_in, d_out, TYPES[dtype], out, i % 3 != 1, i % 2 == 0, seed=i)
        Y, pre = G.linear(X, W, bias=b, act=act_of(G, name), residual=R, out_dtype=out, want_pre=True)
        y, z, zb = oracle.linear(X, W, b, name, R)
        oracle.check(pre, z, zb + oracle.rounding(z, out), f"pre {name}")
        oracle.check(Y, y, oracle.y_bound(y, z, zb, name, out), f"y {name}")
        again, none = G.linear(X, W, bias=b, act=act_of(G, name), residual=R, out_dtype=out)
        assert none is None and torch.equal(again, Y)  # the same with and without pre, and every time


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "x".join(map(str, SHAPES[i])))
def test_backward(G, i, dtype):
    N, d_in, d_out = SHAPES[i]
    name = oracle.ACTS[i % 4]
    out = torch.float32 if i % 5 == 2 else TYPES[dtype]
    X, W, b, _, dY = inputs(N, d_in, d_out, TYPES[dtype], out, True, False, seed=100 + i)
    _, pre = G.linear(X, W, bias=b, act=act_of(G, name), out_dtype=out, want_pre=True)
    pre = None if name == "none" else pre
    dX, dW, db = G.linear_backward(dY, X, W, pre=pre, act=act_of(G, name))
    want, bounds = oracle.gradients(dY, X, W, pre, name)
    for got, w, bd, what in zip((dX, dW, db), want, bounds, ("dx", "dw", "db")):
        oracle.check(got, w, bd + oracle.rounding(w.abs() + bd, TYPES[dtype]), f"{what} {name}")
    one = G.linear_backward(dY, X, W, pre=pre, act=act_of(G, name), want_dw=False, want_db=False)
    two = G.linear_backward(dY, X, W, pre=pre, act=act_of(G, name), want_dx=False)
    assert torch.equal(one[0], dX) and one[1] is None and one[2] is None
    assert two[0] is None and torch.equal(two[1], dW) and torch.equal(two[2], db)
    three = G.linear_backward(dY, X, W, pre=pre, act=act_of(G, name), want_dx=False, want_dw=False)
    assert torch.equal(three[2], db)


# Sizes whose products take the 256-row and the 128-row tiles, each a little short of whole tiles, with rows of whole
# 16-byte pieces and without
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d_in,d_out", [(8190, 4088, 4090), (4094, 2041, 2040), (4090, 1016, 8190)])
def test_large_tiles(G, monkeypatch, N, d_in, d_out, dtype):
    monkeypatch.setattr(oracle, "ON", "cuda")
    t = TYPES[dtype]
    X, W, b, R, dY = inputs(N, d_in, d_out, t, t, True, True, seed=N)
    Y, pre = G.linear(X, W, bias=b, act=G.ACT_SILU, residual=R, want_pre=True)
    y, z, zb = oracle.linear(X, W, b, "silu", R)
    oracle.check(pre, z, zb + oracle.rounding(z, t), "pre")
    oracle.check(Y, y, oracle.y_bound(y, z, zb, "silu", t), "y")
    del y, z, zb
    got = G.linear_backward(dY, X, W, pre=pre, act=G.ACT_SILU)
    want, bounds = oracle.gradients(dY, X, W, pre, "silu")
    for g, w, bd, what in zip(got, want, bounds, ("dx", "dw", "db")):
        oracle.check(g, w, bd + oracle.rounding(w.abs() + bd, t), what)
        # the bounds are those of the worst signs; the 2-norm stays near the roundings': dZ's and the output's
        off = float((g.double() - w).norm() / w.norm())
        assert off <= (1e-5 if dtype == "f32" else 2 * oracle.EPS[t] / 2), (what, off)


def test_more_rows_than_a_launch_and_elements_than_32_bits(G):
    """2^20 + 77 rows of 2080: two launches, offsets past 2^31 elements; rows at both ends and at the seam, and the
    gradients against sums in 64 bits."""
    N, d_in, d_out = (1 << 20) + 77, 2080, 24
    g = torch.Generator(device="cuda").manual_seed(0)
    X = torch.randn(N, d_in, generator=g, device="cuda", dtype=torch.float16)
    W = torch.randn(d_out, d_in, generator=g, device="cuda", dtype=torch.float16) * d_in ** -0.5
    dY = torch.randn(N, d_out, generator=g, device="cuda", dtype=torch.float16)
    Y, _ = G.linear(X, W)
    dX, dW, db = G.linear_backward(dY, X, W)
    rows = torch.tensor([0, 1, (1 << 20) - 1, 1 << 20, N - 2, N - 1], device="cuda")
    y, z, zb = oracle.linear(X[rows], W, None, "none", None)
    oracle.check(Y[rows], y, oracle.y_bound(y, z, zb, "none", torch.float16), "y")
    want, bounds = oracle.gradients(dY[rows], X[rows], W, None, "none")
    oracle.check(dX[rows], want[0], bounds[0] + oracle.rounding(want[0].abs() + bounds[0], torch.float16), "dx")
    w64 = torch.zeros(d_out, d_in, dtype=torch.float64, device="cuda")
    for r in range(0, N, 1 << 17):
        w64 += torch.mm(dY[r:r + (1 << 17)].double().t().contiguous(), X[r:r + (1 << 17)].double())
    # float sums of 2^20 terms of either sign: far below the output's own rounding of half a step
    assert float((dW.double() - w64).norm() / w64.norm()) <= oracle.EPS[torch.float16] / 2
    b64 = dY.double().sum(0)
    assert float((db.double() - b64).norm() / b64.norm()) <= oracle.EPS[torch.float16] / 2


def test_two_streams_at_once(G):
    """Calls that overlap on two streams, each with its own workspace."""
    sets = [inputs(700, 1030, 260, torch.bfloat16, torch.bfloat16, True, True, seed=s) for s in (1, 2)]
    alone = [G.linear(X, W, bias=b, act=G.ACT_GELU, residual=R)[0] for X, W, b, R, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, (X, W, b, R, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(G.linear(X, W, bias=b, act=G.ACT_GELU, residual=R)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(alone, got))


@pytest.mark.parametrize("name", oracle.ACTS)
def test_gradients_against_differences(G, name):
    """sum(Y dY) by central differences along random directions of X, W and bias, h = 2^-5. The difference's own
    error is h^2/6 times a third derivative (smooth activations) plus float rounding over h; relu away from 0."""
    X, W, b, _, dY = inputs(37, 29, 23, torch.float32, torch.float32, True, False, seed=7)
    if name == "relu":  # every z at least 0.5 from 0: flipped signs would not be differences of a smooth function
        b = b + torch.sign(b) * 20
    h, act = 2.0 ** -5, act_of(G, name)
    _, pre = G.linear(X, W, bias=b, act=act, want_pre=True)
    grads = G.linear_backward(dY, X, W, pre=pre, act=act)

    def loss(x, w, c):
        return float((G.linear(x, w, bias=c, act=act)[0].double() * dY.double()).sum())
    g = torch.Generator().manual_seed(1)
    for at, grad in enumerate(grads):
        base = [X, W, b]
        v = torch.randn(base[at].shape, generator=g).cuda()
        v = v / v.norm()
        ends = []
        for s in (h, -h):
            moved = list(base)
            moved[at] = base[at] + s * v
            ends.append(loss(*moved))
        slope = float((grad.double() * v.double()).sum())
        # third derivatives of gelu and silu stay below 2; sum |dY| |direction of z|^3 h^2 / 6 with |dz| <= 8
        # float rounding: (terms + 8) 2^-23 of sum |Y dY|, over h
        size = float((G.linear(X, W, bias=b, act=act)[0].double() * dY.double()).abs().sum())
        dz = (v @ W.T) if at == 0 else (X @ v.T) if at == 1 else v.expand(37, 23)
        curve = 0.0 if name in ("none", "relu") else 2 * float((dY.abs() * dz.abs() ** 3).sum()) * h * h / 6
        assert abs((ends[0] - ends[1]) / (2 * h) - slope) <= curve + 40 * 2.0 ** -23 * size / h, (name, at)


@pytest.mark.parametrize("N", [3, 50, 300])
def test_values_that_are_not_numbers_stay_in_their_rows(G, N):
    X, W, b, R, dY = inputs(N, 136, 72, torch.bfloat16, torch.bfloat16, True, True, seed=3)
    clean = G.linear(X, W, bias=b, act=G.ACT_GELU, residual=R)[0]
    X2, R2 = X.clone(), R.clone()
    X2[1, 5] = float("nan")
    X2[2, 7] = float("inf")
    R2[0, 3] = float("nan")
    got = G.linear(X2, W, bias=b, act=G.ACT_GELU, residual=R2)[0]
    assert got[1].isnan().all() and not got[2].isfinite().any()
    assert got[0, 3].isnan() and torch.equal(got[0, 4:], clean[0, 4:]) and torch.equal(got[3:], clean[3:])
    W2 = W.clone()
    W2[70, 3] = float("nan")  # next to the ragged end of the columns
    got = G.linear(X, W2, bias=b, act=G.ACT_GELU, residual=R)[0]
    assert got[:, 70].isnan().all() and torch.equal(got[:, :70], clean[:, :70]) and torch.equal(got[:, 71], clean[:, 71])
    pre = G.linear(X, W, bias=b, act=G.ACT_RELU, want_pre=True)[1]
    dY[1, 4] = float("nan")
    dX, dW, db = G.linear_backward(dY, X, W, pre=pre, act=G.ACT_RELU)
    assert dX[1].isnan().all() and not dX[0].isnan().any() and not dX[2:].isnan().any()
    assert dW[4].isnan().all() and not dW[5:].isnan().any() and db.isnan().sum() == 1


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_rows_of_odd_length_may_start_anywhere(G, dtype):
    """Slices of a batch with odd rows start off 16-byte borders; residual and output in place."""
    t = TYPES[dtype]
    X, W, b, R, dY = inputs(203, 45, 67, t, t, True, True, seed=5)
    for n0, n1 in ((1, 203), (3, 20), (7, 100)):
        y = G.linear(X[n0:n1], W[:], bias=b, act=G.ACT_SILU, residual=R[n0:n1])[0]
        want, z, zb = oracle.linear(X[n0:n1], W, b, "silu", R[n0:n1])
        oracle.check(y, want, oracle.y_bound(want, z, zb, "silu", t), "slice")
    pre = G.linear(X, W, bias=b, act=G.ACT_SILU, want_pre=True)[1]
    got = G.linear_backward(dY[5:], X[5:], W, pre=pre[5:], act=G.ACT_SILU)
    want, bounds = oracle.gradients(dY[5:], X[5:], W, pre[5:], "silu")
    for g, w, bd in zip(got, want, bounds):
        oracle.check(g, w, bd + oracle.rounding(w.abs() + bd, t), "slice gradient")


def test_in_place_residual_and_nothing_behind_the_output(G):
    for N, d_in, d_out in ((5, 64, 30), (90, 64, 30), (300, 4096, 40), (300, 64, 264)):
        X, W, b, R, _ = inputs(N, d_in, d_out, torch.bfloat16, torch.bfloat16, True, True, seed=N)
        want = G.linear(X, W, bias=b, act=G.ACT_RELU, residual=R)[0]
        buf = torch.full((N + 4, d_out), 7.0, dtype=torch.bfloat16, device="cuda")
        buf[:N] = R
        ws = G.linear_workspace(N, d_in, d_out, torch.bfloat16, X.device)
        P = ctypes.c_void_p
        code = G.lib().gmm_linear(P(X.data_ptr()), G.GMM_BF16, N, d_in, P(W.data_ptr()), d_out, P(b.data_ptr()),
                                  G.ACT_RELU, P(buf.data_ptr()), P(buf.data_ptr()), G.GMM_BF16, None,
                                  P(ws.data_ptr()), ws.numel(), P(torch.cuda.current_stream().cuda_stream))
        assert code == 0
        assert torch.equal(buf[:N], want) and (buf[N:] == 7).all()


def test_empty_batch(G):
    X, W, b, R, dY = inputs(0, 24, 16, torch.float16, torch.float16, True, True)
    assert G.linear(X, W, bias=b, residual=R)[0].shape == (0, 16)
    dX, dW, db = G.linear_backward(dY, X, W)
    assert dX.shape == (0, 24) and (dW == 0).all() and (db == 0).all()


def test_captured_step_on_its_own_stream(G):
    """Forward and backward captured once and replayed with new data between eager work on another stream."""
    N, d_in, d_out = 200, 520, 136
    X, W, b, R, dY = inputs(N, d_in, d_out, torch.bfloat16, torch.bfloat16, True, True, seed=9)
    ws = G.linear_workspace(N, d_in, d_out, X.dtype, X.device)
    wb = G.linear_workspace(N, d_in, d_out, X.dtype, X.device, backward=True)

    def step():
        Y, pre = G.linear(X, W, bias=b, act=G.ACT_GELU, residual=R, want_pre=True, ws=ws)
        return (Y, *G.linear_backward(dY, X, W, pre=pre, act=G.ACT_GELU, ws=wb))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        X.copy_(torch.randn(N, d_in, generator=torch.Generator().manual_seed(i)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, c in zip(kept, step()):
            assert torch.equal(a, c), i
        torch.cuda.synchronize()


def test_refusals(G):
    X, W, b, R, dY = inputs(4, 16, 8, torch.float16, torch.float16, True, True)
    with pytest.raises(ValueError):
        G.linear(X, W.float())
    with pytest.raises(ValueError):
        G.linear(X.t(), W)
    with pytest.raises(ValueError):
        G.linear(X, W, bias=b[:4])
    with pytest.raises(ValueError):
        G.linear(X, W, residual=R.float())
    with pytest.raises(ValueError):
        G.linear(X, W, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        G.linear_backward(dY, X, W, act=G.ACT_RELU)
    with pytest.raises(G.GmmError):
        G.linear(X, W, act=9)
    flat = torch.zeros(4 * 16 + 1, dtype=torch.float16, device="cuda")
    with pytest.raises(G.GmmError):  # whole 16-byte rows that start off a 16-byte border
        G.linear(flat[1:].view(4, 16), W)
