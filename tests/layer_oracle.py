"""Plain 64-bit forms of the linear layer, its gradients and the layer of experts (on the CPU, or where a test of
large shapes puts ON), with worst-case error bounds of the library's arithmetic (tests/layer_bounds.py has those that
are relative to the value, and those of the 2-norm). Shares no code with the library."""
import math

import torch

EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
ACTS = ("none", "relu", "gelu", "silu")
# The functions' own error: value and slope within 2^-20 of max(1, |z|). That is their bound for float results (2^-20
# of the value); for results of 2 bytes the tail of the normal distribution is off by half of 6.3e-7 at most.
FUNCTION = 2.0 ** -20


ON = "cpu"


def wide(t):
    return None if t is None else t.detach().to(ON).double()


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


def sum_bound(a, b, terms):
    """Worst error of float accumulation of `terms` products: each addition is off by at most one unit of the last
    place of a partial sum (truncation included), at most sum |a b|."""
    return (terms + 8) * 2.0 ** -23 * (a.abs() @ b.abs().T)


def rounding(t, dtype):
    """Half a step of the output's type."""
    return t.abs() * EPS[dtype] / 2 + TINY[dtype]


def linear(X, W, bias, name, residual):
    """(y, z, bound of z's error before rounding)."""
    x, w = wide(X), wide(W)
    z = x @ w.T
    bound = sum_bound(x, w, x.shape[1])
    if bias is not None:
        z = z + wide(bias)
        bound = bound + 2.0 ** -23 * z.abs()
    y = act(z, name)
    if residual is not None:
        y = y + wide(residual)
    return y, z, bound


def y_bound(y, z, zb, name, dtype):
    # every activation's slope is at most 1.13
    fn = 0.0 if name in ("none", "relu") else FUNCTION * torch.clamp(z.abs(), min=1.0)
    return 1.13 * zb + fn + 2.0 ** -23 * y.abs() + rounding(y, dtype)


def gradients(dY, X, W, pre, name):
    """((dx, dw, db), (bounds before their own rounding)) for the given pre. dZ is rounded to X's type for the
    products: half a step of it per term, on top of the accumulation."""
    x, w, dy = wide(X), wide(W), wide(dY)
    dz, fn = dy, torch.zeros_like(dy)
    if name != "none":
        z = wide(pre)
        dz = dy * slope(z, name)
        fn = dy.abs() * (0.0 if name == "relu" else FUNCTION) * torch.clamp(z.abs(), min=1.0) + 2.0 ** -23 * dz.abs()
    per = rounding(dz, X.dtype) + fn
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    bx = per @ w.abs() + sum_bound(dz.abs() + per, w.T, w.shape[0])
    bw = per.T @ x.abs() + sum_bound((dz.abs() + per).T, x.T, x.shape[0])
    bb = fn.sum(0) + (x.shape[0] + 8) * 2.0 ** -23 * dz.abs().sum(0)
    return (dx, dw, db), (bx, bw, bb)


def gate(X, P, mu, var, logw, top, threshold, renorm):
    """(idx, resp, weights) of every row's picks, -1 and 0 for a dropped or missing one."""
    f = wide(X) @ wide(P).T
    m, v = wide(mu), wide(var)
    s = wide(logw) - 0.5 * ((2 * math.pi * v).log().sum(1) + ((f[:, None] - m) ** 2 / v).sum(2))
    T, K = s.shape
    post = torch.softmax(s, 1)
    val, order = torch.sort(s, dim=1, descending=True, stable=True)
    idx = torch.full((T, top), -1, dtype=torch.int64)
    resp = torch.zeros(T, top, dtype=torch.float64)
    n = min(top, K)
    for t in range(T):
        for j in range(n):
            k = int(order[t, j])
            if val[t, j] > -math.inf and (j == 0 or post[t, k] >= threshold):
                idx[t, j], resp[t, j] = k, post[t, k]
    w = resp / resp.sum(1, keepdim=True) if renorm else resp
    return idx, resp, w


def experts(X, idx, wts, W1, b1, W2, b2, name, glu, residual):
    """(y, bound): every pick's expert on its row, in 64 bits, with the bound of the library's roundings."""
    x, dtype = wide(X), X.dtype
    T, D = x.shape
    K, F = W2.shape[0], W2.shape[2]
    y = torch.zeros(T, D, dtype=torch.float64) if residual is None else wide(residual).clone()
    bound, size = torch.zeros_like(y), y.abs()
    for t in range(T):
        for j in range(idx.shape[1]):
            k, c = int(idx[t, j]), float(wts[t, j])
            if not 0 <= k < K:
                continue
            w1, w2 = wide(W1[k]), wide(W2[k])
            row = x[t:t + 1]
            z = row @ w1.T
            zb = sum_bound(row, w1, D)
            if b1 is not None:
                z = z + wide(b1[k])
                zb = zb + 2.0 ** -23 * z.abs()
            g, gb = z[:, :F], zb[:, :F]
            fn = 0.0 if name in ("none", "relu") else FUNCTION * torch.clamp(g.abs(), min=1.0)
            a, ab = act(g, name), 1.13 * gb + fn
            if glu:
                u, ub = z[:, F:], zb[:, F:]
                a, ab = a * u, ab * (u.abs() + ub) + a.abs() * ub
            ab = ab + rounding(a.abs() + ab, dtype) + 2.0 ** -23 * a.abs()
            o = a @ w2.T
            ob = ab @ w2.abs().T + sum_bound(a.abs() + ab, w2, F)
            if b2 is not None:
                o = o + wide(b2[k])
            y[t:t + 1] += c * o
            bound[t:t + 1] += abs(c) * (ob + 2.0 ** -22 * o.abs())
            size[t:t + 1] += abs(c) * o.abs()
    return y, bound + 2.0 ** -22 * size + rounding(y, dtype)


def check(got, want, bound, what):
    got = wide(got)
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((off / bound).nan_to_num(posinf=1e30).max()):.3g} of the bound, first at "
                           f"{bad.nonzero()[0].tolist()}")
