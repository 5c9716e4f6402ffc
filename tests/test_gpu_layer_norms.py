"""The layers in the 2-norm, where a lost piece of a long sum shows that the worst-case bounds of single entries would
let pass; large half products; the experts in place."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests import layer_bounds as bounds  # noqa: E402
from tests import layer_oracle as oracle  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def inputs(N, d_in, d_out, t, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    X = torch.randn(N, d_in, generator=g, device=device).to(t)
    W = (torch.randn(d_out, d_in, generator=g, device=device) * d_in ** -0.5).to(t)
    return X, W, torch.randn(N, d_out, generator=g, device=device).to(t), torch.randn(d_out, generator=g, device=device).to(t)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", sorted(TYPES))
# one row, 16 and 17; short sums; long ones in one part and in several; 128-row and 256-row tiles, whole and ragged
@pytest.mark.parametrize("N,d_in,d_out", [(1, 8192, 700), (16, 4093, 8200), (17, 8192, 64), (300, 8192, 24), (64, 65536, 40),
                                          (700, 1000, 333), (1537, 1023, 777), (2048, 2048, 1024), (8190, 4088, 4090),
                                          (4094, 2041, 2040)])
def test_forward_in_norm(N, d_in, d_out, dtype):
    from soft_clustering_gmm_amd import gmm as G
    t = TYPES[dtype]
    X, W, R, b = inputs(N, d_in, d_out, t, seed=N)
    z = X.double() @ W.double().t().contiguous() + b.double()
    for out in {t, torch.float32}:
        r = R.to(out)
        for name, scale in (("none", 1.0), ("silu", 2.0)):
            # |silu'| <= 1.1, and silu of a normal z is 0.6 of its norm, so a sum's error counts twice
            Y, pre = G.linear(X, W, bias=b, act=getattr(G, "ACT_" + name.upper()), residual=r, out_dtype=out,
                              want_pre=True)
            bounds.norm_check(pre, z, d_in, out, "pre")
            bounds.norm_check(Y.double(), oracle.act(z, name) + r.double(), d_in * scale ** 2, out, f"y {name}")


@pytest.mark.gpu
@pytest.mark.parametrize("N,d_in,d_out", [(8190, 4088, 4090), (4094, 2041, 2040), (4090, 1016, 8190)])
def test_large_half_gradients(N, d_in, d_out):
    from soft_clustering_gmm_amd import gmm as G
    X, W, dY, b = inputs(N, d_in, d_out, torch.float16, seed=N)
    _, pre = G.linear(X, W, bias=b, act=G.ACT_SILU, want_pre=True)
    got = G.linear_backward(dY, X, W, pre=pre, act=G.ACT_SILU)
    dz = dY.double() * oracle.slope(pre.double(), "silu")
    want = (dz @ W.double(), dz.t().contiguous() @ X.double(), dz.sum(0))
    for g, w, n, what in zip(got, want, (d_out, N, N), ("dx", "dw", "db")):
        bounds.norm_check(g, w, n, torch.float16, what, roundings=2)  # dZ's and the output's


def test_a_lost_piece_is_seen():
    """One 16-byte piece of 2048 left out of a sum, and operands rounded to bfloat16: within the worst-case bounds, but
    not in the norm."""
    X, W, _, b = inputs(40, 8192, 30, torch.float32, seed=0, device="cpu")
    z = X.double() @ W.double().t()
    bounds.norm_check(z.float(), z, 8192, torch.float32, "right")
    lost = X.clone()
    lost[:, 8188:] = 0
    for wrong in (lost.double() @ W.double().t(), X.bfloat16().double() @ W.bfloat16().double().t()):
        with pytest.raises(AssertionError):
            bounds.norm_check(wrong.float(), z, 8192, torch.float32, "wrong")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("T", [1, 3, 9, 60])  # up to 8 picks, and more
def test_experts_in_place(T, dtype):
    """Y over X, over the residual, and over both where they are one."""
    from soft_clustering_gmm_amd import gmm as G
    t, g = TYPES[dtype], torch.Generator().manual_seed(T)
    D, F, K, d, top = 200, 96, 6, 10, 2

    def normal(*shape, scale=1.0, t=t):
        return (torch.randn(*shape, generator=g) * scale).to(t).cuda()
    X, R, P = normal(T, D), normal(T, D), normal(d, D, scale=D ** -0.5)
    W1, W2, b1, b2 = normal(K, 2 * F, D, scale=D ** -0.5), normal(K, D, F, scale=F ** -0.5), normal(K, 2 * F), normal(K, D)
    mu, var, logw = normal(K, d, t=torch.float32), torch.ones(K, d, device="cuda"), torch.zeros(K, device="cuda")
    V, L = ctypes.c_void_p, G.lib()
    at = {torch.float32: G.GMM_F32, torch.float16: G.GMM_F16, torch.bfloat16: G.GMM_BF16}[t]
    ws = G.expert_workspace(T, D, K, F, d, top, t, X.device)
    stream = V(torch.cuda.current_stream().cuda_stream)

    def p(x):
        return V(x.data_ptr())

    def layer(x, r, y):
        idx, resp = torch.empty(T, top, dtype=torch.int32, device="cuda"), torch.empty(T, top, device="cuda")
        code = L.gmm_expert_layer(p(x), at, T, D, p(P), d, p(mu), p(var), p(logw), K, top, ctypes.c_float(0.0), 1, p(W1),
                                  p(b1), p(W2), p(b2), F, G.ACT_SILU, 1, p(r), p(y), p(idx), p(resp), p(ws), ws.numel(),
                                  stream)
        assert code == 0
        return idx, resp

    def rows(x, r, y, idx, resp):
        assert L.gmm_expert_rows(p(x), at, T, D, p(idx), p(resp), top, K, p(W1), p(b1), p(W2), p(b2), F, G.ACT_SILU, 1,
                                 p(r), p(y), p(ws), ws.numel(), stream) == 0
    for res_is_x in (False, True):
        want = torch.empty_like(X)
        picks, resp = layer(X, X if res_is_x else R, want)
        want_rows = torch.empty_like(X)
        rows(X, X if res_is_x else R, want_rows, picks, resp)
        for over in ("X", "residual"):
            x, r = X.clone(), R.clone()
            if res_is_x:
                r = x
            y = x if over == "X" else r
            idx, _ = layer(x, r, y)
            assert torch.equal(y, want) and torch.equal(idx, picks), (over, res_is_x)
            x, r = X.clone(), R.clone()
            if res_is_x:
                r = x
            y = x if over == "X" else r
            rows(x, r, y, picks, resp)
            assert torch.equal(y, want_rows), (over, res_is_x)
