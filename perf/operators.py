"""Measured cases of the learned products around the mixture: the matrix product with its epilogue (the projection of
wide rows to the mixture's features, a layer of a feature network), the same with its backward pass, and the layer of
experts gated by the mixture's posterior, for a few rows.

`own = False` computes plain forms in elementary torch operations; `own = True` calls the library."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
ACTS = ("none", "relu", "gelu", "silu")


def linear(name, rows, d_in, d_out, dtype, out, act, bias, residual, op="linear"):
    return {"name": name, "op": op, "rows": rows, "d_in": d_in, "d_out": d_out, "dtype": dtype, "out": out, "act": act,
            "bias": bias, "residual": residual}


def experts(name, rows, width, hidden, count, features, top, dtype, act, glu, bias, residual, threshold, renorm):
    return {"name": name, "op": "experts", "rows": rows, "width": width, "hidden": hidden, "experts": count,
            "features": features, "top": top, "dtype": dtype, "act": act, "glu": glu, "bias": bias,
            "residual": residual, "threshold": threshold, "renorm": renorm}


def listed():
    return [
        # one row through a wide layer while serving: the weights are read once, latency counts
        linear("linear one row", 1, 4096, 4096, "bf16", "bf16", "silu", True, True),
        # the embeddings of an index projected to the 96 features that the mixture is fitted on
        linear("linear projection", 262144, 1024, 96, "bf16", "f32", "none", True, False),
        # the first layer of a feature network over a large batch
        linear("linear large", 8192, 4096, 16384, "bf16", "bf16", "gelu", True, False),
        # a ragged batch, sizes that no tile divides and rows that are not aligned
        linear("linear odd", 1537, 1023, 777, "f16", "f16", "relu", True, True),
        # single precision, as the mixture's own rows are by default
        linear("linear f32", 4096, 1024, 1024, "f32", "f32", "none", True, True),
        # a training step of a feature network's layer: forward, then every gradient
        linear("train layer", 4096, 2048, 8192, "bf16", "bf16", "gelu", True, True, "train"),
        # the projection to the mixture's features, trained in single precision
        linear("train projection f32", 16384, 512, 128, "f32", "f32", "none", True, False, "train"),
        # a ragged last batch
        linear("train odd", 1001, 516, 1000, "f16", "f16", "silu", True, True, "train"),
        # one row through a layer of experts while serving
        experts("experts one row", 1, 4096, 1408, 64, 64, 2, "bf16", "silu", True, False, True, 0.05, True),
        # a small batch of serving, border vectors to two experts
        experts("experts 16 rows", 16, 2048, 1024, 128, 96, 2, "bf16", "silu", True, False, True, 0.05, True),
        # the largest batch: most experts are read
        experts("experts 128 rows", 128, 4096, 2048, 64, 128, 2, "bf16", "silu", True, False, True, 0.0, True),
        # few experts with biases, ragged sizes, three picks weighted by the posterior itself
        experts("experts odd", 27, 1001, 333, 5, 17, 3, "f16", "gelu", False, True, False, 0.02, False),
    ]


def spread(rng, lo, hi):
    """A whole number, even over the logarithm of the range."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def sized(rng, lo, hi):
    """As spread(), a multiple of 64 or of 8 two times in three."""
    n, m = spread(rng, lo, hi), rng.choice((1, 8, 64))
    return max(lo, n // m * m)


def draw(rng):
    while True:
        op = rng.choice(("linear", "train", "experts"))
        dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
        act = rng.choice(ACTS)
        if op == "train" and dtype == "f32" and act == "relu":
            continue  # the sign of a sum next to zero, and with it the slope, is not settled in 32 bits
        if op == "experts":
            c = {"op": op, "rows": spread(rng, 1, 128), "width": sized(rng, 64, 4096), "hidden": sized(rng, 64, 4096),
                 "experts": spread(rng, 2, 256), "features": spread(rng, 8, 128), "top": rng.choice((1, 2, 2, 3, 4, 8)),
                 "dtype": dtype, "act": act, "glu": rng.random() < 0.5, "bias": rng.random() < 0.5,
                 "residual": rng.random() < 0.5, "threshold": rng.choice((0.0, 0.05)), "renorm": rng.random() < 0.5}
            weights = c["experts"] * (3 if c["glu"] else 2) * c["width"] * c["hidden"]
            if weights * SIZE[dtype] <= 64 * 3 * 4096 * 2048 * 2:
                return c
            continue
        c = {"op": op, "rows": spread(rng, 1, 262144 if op == "linear" else 16384), "d_in": sized(rng, 16, 8192),
             "d_out": sized(rng, 16, 16384), "dtype": dtype, "out": rng.choice((dtype, dtype, "f32")), "act": act,
             "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}
        work = c["rows"] * c["d_in"] * c["d_out"]
        most = 8192 * 4096 * 16384 if op == "linear" else 4096 * 2048 * 8192
        # single precision runs at a fraction of the others' rate
        if work * (16 if dtype == "f32" else 1) <= most and c["rows"] * (c["d_in"] + 2 * c["d_out"]) <= 1 << 29:
            return c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype if dtype != torch.float64 else torch.float32)
                * scale).to(dtype)

    s = dict(case)
    if case["op"] == "experts":
        T, D, F, K, d = case["rows"], case["width"], case["hidden"], case["experts"], case["features"]
        up = 2 * F if case["glu"] else F
        s["x"] = normal(T, D)
        s["proj"] = normal(d, D, scale=D ** -0.5)
        f32 = torch.float32
        s["mu"] = normal(K, d, scale=0.7, dtype=f32)
        # variances that leave a row between a few components, as at the border between lists
        s["var"] = (0.5 + torch.rand(K, d, generator=g, device="cuda")) * max(1.0, d / 16)
        s["logw"] = torch.log_softmax(0.5 * normal(K, dtype=f32), 0)
        s["w1"] = normal(K, up, D, scale=D ** -0.5)
        s["w2"] = normal(K, D, F, scale=2 * F ** -0.5)
        s["b1"] = normal(K, up, scale=0.5) if case["bias"] else None
        s["b2"] = normal(K, D, scale=0.5) if case["bias"] else None
        s["res"] = normal(T, D) if case["residual"] else None
        return s
    N, I, O, o = case["rows"], case["d_in"], case["d_out"], TYPES[case["out"]]
    s["x"] = normal(N, I)
    s["w"] = normal(O, I, scale=I ** -0.5)
    s["b"] = normal(O, scale=0.5) if case["bias"] else None
    s["res"] = normal(N, O, dtype=o) if case["residual"] else None
    if case["op"] == "train":
        s["dy"] = normal(N, O, dtype=o)
    return s


def act_of(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope_of(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


def plain_linear(s):
    z = s["x"].float() @ s["w"].float().T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = act_of(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(TYPES[s["out"]]), z


def plain_train(s):
    y, z = plain_linear(s)
    dz = s["dy"].float() * slope_of(z, s["act"])
    t = s["x"].dtype
    out = {"y": y, "dx": (dz @ s["w"].float()).to(t), "dw": (dz.T @ s["x"].float()).to(t)}
    if s["b"] is not None:
        out["db"] = dz.sum(0).to(t)
    return out


def plain_gate(s):
    """Picks in 64 bits, which a border between two components needs."""
    f = s["x"].double() @ s["proj"].double().T
    mu, var = s["mu"].double(), s["var"].double()
    score = s["logw"].double() - 0.5 * (torch.log(2 * math.pi * var).sum(1)
                                        + ((f[:, None, :] - mu) ** 2 / var).sum(2))
    T, K = score.shape
    top = min(s["top"], K)
    val, idx = torch.sort(score, dim=1, descending=True, stable=True)
    resp = torch.exp(val - torch.logsumexp(score, 1, keepdim=True))[:, :top]
    idx = idx[:, :top]
    keep = resp >= s["threshold"]
    keep[:, 0] = True
    idx = torch.where(keep, idx, torch.full_like(idx, -1))
    resp = torch.where(keep, resp, torch.zeros_like(resp))
    if top < s["top"]:
        more = s["top"] - top
        idx = torch.cat([idx, idx.new_full((T, more), -1)], 1)
        resp = torch.cat([resp, resp.new_zeros((T, more))], 1)
    return idx, resp


def plain_experts(s):
    idx, resp = plain_gate(s)
    wts = resp / resp.sum(1, keepdim=True) if s["renorm"] else resp
    T, D = s["x"].shape
    flat = idx.reshape(-1)
    at = torch.nonzero(flat >= 0)[:, 0]  # the picks, each with its row, grouped by expert
    at = at[torch.sort(flat[at], stable=True)[1]]
    rows = at // s["top"]
    used, group, counts = torch.unique_consecutive(flat[at], return_inverse=True, return_counts=True)
    place = torch.arange(at.numel(), device=at.device) - (torch.cumsum(counts, 0) - counts)[group]
    x = torch.zeros(used.numel(), int(counts.max()), D, device=at.device)
    x[group, place] = s["x"][rows].float()
    h = torch.bmm(x, s["w1"][used].float().transpose(1, 2).contiguous())
    if s["b1"] is not None:
        h = h + s["b1"][used].float()[:, None, :]
    if s["glu"]:
        a, b = h.chunk(2, 2)
        h = act_of(a, s["act"]) * b
    else:
        h = act_of(h, s["act"])
    o = torch.bmm(h, s["w2"][used].float().transpose(1, 2).contiguous())
    if s["b2"] is not None:
        o = o + s["b2"][used].float()[:, None, :]
    y = s["res"].float() if s["res"] is not None else torch.zeros(T, D, device=at.device)
    y = y.index_add(0, rows, o[group, place] * wts.reshape(-1)[at].float()[:, None])
    return {"y": y.to(s["x"].dtype), "idx": idx.to(torch.int32), "resp": resp.float()}


def run(state):
    s = state
    if own:
        from soft_clustering_gmm_amd import gmm
        act = getattr(gmm, "ACT_" + s["act"].upper())
        if s["op"] == "experts":
            y, idx, resp = gmm.expert_layer(
                s["x"], s["proj"], s["mu"], s["var"], s["logw"], s["w1"], s["w2"], b1=s["b1"], b2=s["b2"], act=act,
                glu=s["glu"], top=s["top"], border_threshold=s["threshold"], renorm=s["renorm"], residual=s["res"])
            return {"y": y, "idx": idx, "resp": resp}
        out = TYPES[s["out"]]
        if s["op"] == "linear":
            y, _ = gmm.linear(s["x"], s["w"], bias=s["b"], act=act, residual=s["res"], out_dtype=out)
            return {"y": y}
        y, pre = gmm.linear(s["x"], s["w"], bias=s["b"], act=act, residual=s["res"], out_dtype=out,
                            want_pre=s["act"] != "none")
        dx, dw, db = gmm.linear_backward(s["dy"], s["x"], s["w"], pre=pre, act=act, want_db=s["b"] is not None)
        got = {"y": y, "dx": dx, "dw": dw}
        if db is not None:
            got["db"] = db
        return got
    if s["op"] == "experts":
        return plain_experts(s)
    if s["op"] == "linear":
        return {"y": plain_linear(s)[0]}
    return plain_train(s)


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "experts":
        T, D, F, K, d = case["rows"], case["width"], case["hidden"], case["experts"], case["features"]
        top = min(case["top"], K)
        mats = 3 if case["glu"] else 2
        read = K * (1 - (1 - min(1.0, top / K)) ** T)  # experts that some row picks, were the picks even
        return {"bytes": read * mats * D * F * e + d * D * e + 8 * K * d + T * D * e * (3 if case["residual"] else 2),
                "flops": 2.0 * T * top * mats * D * F + 2.0 * T * d * D + 4.0 * T * K * d}
    N, I, O, o = case["rows"], case["d_in"], case["d_out"], SIZE[case["out"]]
    b = (N * I + O * I) * e + N * O * o * (2 if case["residual"] else 1)
    f = 2.0 * N * I * O
    if case["op"] == "train":
        b += N * O * o + (N * I + O * I) * e
        f *= 3
    return {"bytes": b, "flops": f}


def exact_act(z, act, slope=False):
    phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
    q = torch.sigmoid(z)
    if slope:
        return {"none": torch.ones_like(z), "relu": torch.heaviside(z, torch.zeros_like(z)),
                "gelu": phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                "silu": q + z * q * (1 - q)}[act]
    return {"none": z, "relu": torch.relu(z), "gelu": z * phi, "silu": z * q}[act]


def exact(case, seed):
    s = prepare(case, seed)

    def wide(name):
        return None if s[name] is None else s[name].double()

    if case["op"] != "experts":
        z = torch.nn.functional.linear(wide("x"), wide("w"), wide("b"))
        y = exact_act(z, case["act"])
        y = y if s["res"] is None else y + wide("res")
        if case["op"] == "linear":
            return {"y": y}
        dz = wide("dy") * exact_act(z, case["act"], slope=True)
        got = {"y": y, "dx": torch.mm(dz, wide("w")), "dw": torch.mm(dz.t().contiguous(), wide("x"))}
        if s["b"] is not None:
            got["db"] = dz.sum(0)
        return got
    T, K, F = case["rows"], case["experts"], case["hidden"]
    x = wide("x")
    gate = torch.distributions.Normal(wide("mu"), wide("var").sqrt(), validate_args=False)
    feats = torch.nn.functional.linear(x, wide("proj"))
    log_joint = torch.stack([gate.log_prob(f).sum(1) + wide("logw") for f in feats])
    post = torch.softmax(log_joint, 1).cpu()
    order = [sorted(range(K), key=lambda k: (-row[k], k))[:case["top"]] for row in log_joint.tolist()]
    y = torch.zeros_like(x) if s["res"] is None else wide("res")
    resp = torch.zeros(T, case["top"], dtype=torch.float64)
    rows_of = {}
    for t in range(T):
        for j, k in enumerate(order[t]):
            if j == 0 or post[t, k] >= case["threshold"]:
                resp[t, j] = post[t, k]
                rows_of.setdefault(k, []).append((t, j))
    wts = resp / resp.sum(1, keepdim=True) if case["renorm"] else resp
    for k, places in sorted(rows_of.items()):
        ts = torch.tensor([t for t, _ in places], device=x.device)
        c = torch.tensor([[float(wts[t, j])] for t, j in places], dtype=torch.float64, device=x.device)
        h = torch.nn.functional.linear(x[ts], s["w1"][k].double(), None if s["b1"] is None else s["b1"][k].double())
        h = exact_act(h[:, :F], case["act"]) * h[:, F:] if case["glu"] else exact_act(h, case["act"])
        o = torch.nn.functional.linear(h, s["w2"][k].double(), None if s["b2"] is None else s["b2"][k].double())
        y[ts] = y[ts] + c * o
    return {"y": y, "idx": None, "resp": resp.to(x.device)}
