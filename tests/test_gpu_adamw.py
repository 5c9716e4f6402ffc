"""The AdamW step (gmm_adamw_step) against its plain 64-bit form, and its 8-bit states against the rounding that the
header writes down."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
U = 2.0 ** -24
SIZES = [1, 255, 256, 257, 0, 1000, 4096, 5, 70000, 3]
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def G():
    from soft_clustering_gmm_amd import gmm
    gmm.lib()
    return gmm


def parts(sizes):
    at = 0
    for n in sizes:
        yield slice(at, at + n)
        at += -(-n // 256) * 256


def make(sizes, t, gt, seed=0, offset=0):
    """Parameters and gradients, each `offset` elements into memory of its own."""
    g = torch.Generator().manual_seed(seed)

    def place(n, scale, dtype):
        flat = torch.full((n + 2 * offset,), 9.0, dtype=dtype)
        flat[offset:offset + n] = (torch.randn(n, generator=g) * scale).to(dtype)
        return flat.cuda()[offset:offset + n]
    return [place(n, 0.5, t) for n in sizes], [place(n, 0.1, gt) for n in sizes]


def shown(state, name):
    """The state's values in 64 bits."""
    t = state[name]
    if t.dtype == torch.float32:
        return t.cpu().double()
    return t.cpu().float().double() * state[name + "_scale"].cpu().double().repeat_interleave(256)


def reference(p, g, m, v, n, lr, beta1, beta2, eps, weight_decay):
    """(p, m, v) in 64 bits and the bound of p's error: m and v are off by 4 roundings, the step by 10."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    step = lr * (m / (1 - beta1 ** n)) / ((v / (1 - beta2 ** n)).sqrt() + eps)
    # m may cancel: its error is relative to its terms
    terms = (beta1 * (m - (1 - beta1) * g) / beta1 if beta1 else 0 * m).abs() + (1 - beta1) * g.abs()
    bound = lr / (1 - beta1 ** n) * 4 * U * terms / ((v / (1 - beta2 ** n)).sqrt() + eps) + 10 * U * step.abs()
    new = p - lr * weight_decay * p - step
    return new, m, v, bound + 3 * U * (p.abs() + step.abs()), 4 * U * terms


def off(got, want, bound, what):
    bad = ~((got.cpu().double() - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t,gt,master", [("f32", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", False),
                                         ("f16", "f16", False), ("f16", "f32", True), ("bf16", "bf16", False)])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps(G, t, gt, master, bits, offset):
    t, gt = TYPES[t], TYPES[gt]
    params, _ = make(SIZES, t, gt, offset=offset)
    around = [p._base if p._base is not None else p for p in params]
    state = G.adamw_state(params, bits=bits, master=master)
    factor, grad_factor = (torch.full((), x, device="cuda") for x in (0.5, 0.25))
    skipped = SIZES.index(1000)
    for n in range(1, 5):
        _, grads = make(SIZES, t, gt, seed=n, offset=offset)
        given = [None if i == skipped and n == 2 else g for i, g in enumerate(grads)]
        held = {k: x.clone() for k, x in state.items()}
        before = [p.clone() for p in params]
        G.adamw_step(params, given, **state, **HYPER, lr_factor=factor, grad_factor=grad_factor)
        assert state["step"].tolist() == [n, 0]
        old_m, old_v = shown(held, "m"), shown(held, "v")
        old_v = old_v if bits == 32 else old_v ** 2
        new_m, new_v = shown(state, "m"), shown(state, "v")
        hyper = dict(HYPER, lr=float(torch.tensor(HYPER["lr"])) * 0.5)
        for i, part in enumerate(parts(SIZES)):
            if given[i] is None:
                assert torch.equal(params[i], before[i])
                for k in ("m", "v", "master"):
                    if k in state:
                        assert torch.equal(state[k][part].view(torch.uint8), held[k][part].view(torch.uint8))
                continue
            p0 = (held["master"][part] if master else before[i]).cpu().double()
            want, m, v, pb, mb = reference(p0, given[i].cpu().double() * 0.25, old_m[part], old_v[part], n, **hyper)
            if master:
                off(state["master"][part], want, pb, "master")
                assert torch.equal(state["master"][part].to(t), params[i])
            else:
                off(params[i], want, pb + (want.abs() + pb) * EPS[t] / 2 + TINY[t], "p")
            if bits == 32:
                off(new_m[part], m, mb, "m")
                off(new_v[part], v, 6 * U * v, "v")
        # nothing beside the tensors: their surroundings and what lies between the parts of the state
        for a, p in zip(around, params):
            assert a is p or ((a[:offset] == 9).all() and (a[offset + p.numel():] == 9).all())
        inside = torch.zeros(state["m"].numel(), dtype=torch.bool)
        for part in parts(SIZES):
            inside[part] = True
        for k in ("m", "v", "master"):
            if k in state:
                assert (state[k].cpu().float()[~inside] == 0).all()


def chance(n, step, device):
    mask = 0xFFFFFFFF
    x = (torch.arange(n, device=device) ^ (step * 0x9E3779B1 & mask)) & mask
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ x >> shift) * factor) & mask
    x = x ^ x >> 16
    return (x & 0xFFFF).double() / 65536, (x >> 16).double() / 65536


@pytest.mark.parametrize("sizes", [[3000, 513], [17, (1 << 25) + 300]], ids=["small", "past the caches"])
def test_held_in_eight_bits(G, sizes):
    """Every held value is the neighbour that the hash decides, of the 64-bit value over its block's scale; where that is
    within a float rounding of the border either is."""
    on = "cuda"
    params, _ = make(sizes, torch.bfloat16, torch.float32)
    state = G.adamw_state(params, bits=8)
    N = state["m"].numel()

    def held(name):
        return state[name].to(on).float().double() * state[name + "_scale"].to(on).double().repeat_interleave(256)
    for n in range(1, 4):
        _, grads = make(sizes, torch.bfloat16, torch.float32, seed=n)
        k = min(700, sizes[0])
        grads[0][:k] *= 10.0 ** torch.linspace(-8, 0, k, device="cuda")  # far below their block's largest
        old_m, old_v = held("m"), held("v") ** 2
        G.adamw_step(params, grads, **state, **HYPER)
        g = torch.zeros(N, dtype=torch.float64, device=on)
        inside = torch.zeros(N, dtype=torch.bool, device=on)
        for part, x in zip(parts(sizes), grads):
            g[part], inside[part] = x.to(on).double(), True
        m = torch.where(inside, 0.9 * old_m + (1 - 0.9) * g, 0 * g)
        r = torch.where(inside, 0.99 * old_v + (1 - 0.99) * g * g, 0 * g).sqrt()
        for name, x, part in (("m", m, chance(N, n, on)[0]), ("v", r, chance(N, n, on)[1])):
            scale = state[name + "_scale"].to(on).double()
            want = x.abs().view(-1, 256).amax(1) / 448
            assert ((scale - want).abs() <= 8 * U * want).all()
            up = 1 / want.clamp(min=1e-300).repeat_interleave(256)
            y = x * up
            exponent = torch.frexp(y)[1].clamp(min=-5)
            unit = torch.ldexp(torch.ones_like(y), exponent - 4)
            a = y.abs() / unit  # neighbours are 1 apart
            # m may cancel: off by a few roundings of its terms
            wide = 1e-6 + 8 * U * (a + old_m.abs() * up / unit if name == "m" else a)
            got = state[name].to(on).float().double()
            low, high = (torch.floor(a + part - wide) * unit, torch.floor(a + part + wide) * unit)
            if name == "v":
                low, high = (torch.where(x > 0, q.clamp(min=2.0 ** -9), q) for q in (low, high))
            size = got.abs()
            ok = (size >= low.clamp(max=448) - 1e-12) & (size <= high.clamp(max=448) + 1e-12)
            ok &= (got == 0) | (torch.sign(got) == torch.sign(x))
            assert (ok | ~inside).all(), (name, n, (~ok & inside).nonzero()[:3].tolist())
            assert (got[~inside] == 0).all()
            if name == "m":  # the hash moves about half of them up
                moved = (size > torch.floor(a) * unit) & inside & (a > 1)
                assert 0.3 < float(moved.double().sum() / (inside & (a > 1)).sum()) < 0.7


def test_averages_keep_moving_in_eight_bits(G):
    """Rounded to the nearest, an average of 1 in 1000 would stay where its first step put it."""
    p = [torch.zeros(4096, device="cuda")]
    g = [torch.where(torch.arange(4096, device="cuda") % 2 == 0, 1.0, -0.5)]
    state = G.adamw_state(p, bits=8)
    for n in range(1500):
        G.adamw_step(p, g, **state, beta2=0.999, lr=0.0)
    v, m = shown(state, "v") ** 2, shown(state, "m")
    want = (1 - 0.999 ** 1500) * g[0].cpu().double() ** 2
    # neighbours of v are 2^-3 to 2^-2 apart, so a step of 1 in 1000 is a walk whose spread is sqrt(2^-2 / 2) of v at
    # most; over 2048 entries the mean is within a few hundredths, and held sqrt(v) are as often above as below
    for half in (0, 1):
        ratio = float((v / want)[half::2].mean())
        assert 0.8 < ratio < 1.25, ratio
        assert 0.9 < float((m / g[0].cpu().double())[half::2].mean()) < 1.1


def test_large_states(G):
    """A state that goes past the caches is that of its parts in calls of their own."""
    n = 9_000_064
    params, grads = make([n], torch.bfloat16, torch.float32)
    start = params[0].clone()
    state = G.adamw_state(params, master=True)
    for _ in range(2):
        G.adamw_step(params, grads, **state, **HYPER)
    for o, k in ((0, 5000), (4_000_000 // 256 * 256, 70_000), (n - 64 - 2560, 2624)):
        p = [start[o:o + k].clone()]
        one = G.adamw_state(p, master=True)
        for _ in range(2):
            G.adamw_step(p, [grads[0][o:o + k]], **one, **HYPER)
        assert torch.equal(p[0], params[0][o:o + k])
        for name in ("m", "v", "master"):
            assert torch.equal(one[name][:k], state[name][o:o + k])


def test_elements_past_32_bits(G):
    """A tensor of more than 2^31 elements, behind another one: its ends are those of calls of their own."""
    n = (1 << 31) + 777
    p = [torch.ones(300, dtype=torch.bfloat16, device="cuda"), torch.empty(n, dtype=torch.bfloat16, device="cuda")]
    ramp = torch.arange(1 << 20, device="cuda", dtype=torch.float32).sub_(1 << 19).div_(1 << 19).bfloat16()
    for o in range(0, n, 1 << 20):
        p[1][o:o + (1 << 20)] = ramp[:n - o]
    g = [t.clone() for t in p]
    ends = [(0, 5000), ((1 << 30) + 256, 4096), ((1 << 31) - 512, 1289)]
    start = [p[1][o:o + k].clone() for o, k in ends]
    state = G.adamw_state(p)
    G.adamw_step(p, g, **state, **HYPER)
    for (o, k), q in zip(ends, start):
        one = G.adamw_state([q])
        G.adamw_step([q], [g[1][o:o + k]], **one, **HYPER)
        assert torch.equal(q, p[1][o:o + k])
        for name in ("m", "v"):
            assert torch.equal(one[name][:k], state[name][512 + o:512 + o + k])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [96, 97, 250])
def test_many_tensors(G, count, bits):
    sizes = [(i * 37) % 600 for i in range(count)]
    params, grads = make(sizes, torch.float32, torch.float32)
    alone = [p.clone() for p in params]
    state = G.adamw_state(params, bits=bits)
    G.adamw_step(params, grads, **state, **HYPER)
    G.adamw_step(params, [g * 0.5 for g in grads], **state, **HYPER)
    assert state["step"].tolist() == [2, 0]
    if bits == 8:
        return  # a tensor's rounding goes by its place in the state
    for p, a, g, part in zip(params, alone, grads, parts(sizes)):
        one = G.adamw_state([a])
        G.adamw_step([a], [g], **one, **HYPER)
        G.adamw_step([a], [g * 0.5], **one, **HYPER)
        n = a.numel()
        assert torch.equal(a, p) and torch.equal(one["m"][:n], state["m"][part])


@pytest.mark.parametrize("bits", [32, 8])
def test_what_is_not_finite_reaches_no_other(G, bits):
    params, grads = make([1000], torch.float32, torch.float32)
    clean = [p.clone() for p in params]
    other = [g.clone() for g in grads]
    other[0][3], other[0][300], other[0][301] = float("nan"), float("inf"), -float("inf")
    for g in (grads, other):
        g[0][5] = 0.0
    a, b = G.adamw_state(params, bits=bits), G.adamw_state(params, bits=bits)
    for _ in range(3):
        G.adamw_step(clean, grads, **a, **HYPER)
        G.adamw_step(params, other, **b, **HYPER)
    bad = torch.tensor([3, 300, 301], device="cuda")
    fine = torch.ones(1000, dtype=torch.bool, device="cuda")
    fine[bad] = False
    assert torch.equal(params[0][fine], clean[0][fine])
    assert not shown(b, "m")[bad.cpu()].isfinite().any() and not shown(b, "v")[bad.cpu()].isfinite().any()
    for k in ("m", "v"):
        x, y = shown(a, k)[:1000][fine.cpu()], shown(b, k)[:1000][fine.cpu()]
        assert torch.equal(x, y)


def test_zeros_and_tiny_values(G):
    """No gradient yet, blocks of zeros, values below the smallest scale."""
    for bits in (32, 8):
        p = [torch.linspace(-1, 1, 600, device="cuda")]
        start = p[0].clone()
        state = G.adamw_state(p, bits=bits)
        G.adamw_step(p, [torch.zeros(600, device="cuda")], **state, lr=0.1, weight_decay=0.5)
        off(p[0], start.cpu().double() * (1 - 0.05), 4 * U * start.cpu().double().abs(), "decay alone")
        assert (shown(state, "m") == 0).all() and (shown(state, "v") == 0).all()
        G.adamw_step(p, [torch.full((600,), 1e-38, device="cuda")], **state, lr=0.1)
        assert p[0].isfinite().all() and shown(state, "m").isfinite().all() and shown(state, "v").isfinite().all()


def test_beta_zero_and_no_tensors(G):
    p = [torch.ones(10, device="cuda")]
    state = G.adamw_state(p)
    G.adamw_step(p, [torch.full((10,), 0.5, device="cuda")], **state, lr=0.25, beta1=0.0, beta2=0.0, weight_decay=0.0)
    off(p[0], torch.full((10,), 0.75, dtype=torch.float64), 1e-6, "sign step")
    state["step"].fill_(0)
    G.adamw_step(p, [None], **state)
    assert state["step"].tolist() == [1, 0] and (state["m"][:10] == 0.5).all()
    empty = dict(m=torch.empty(0, device="cuda"), v=torch.empty(0, device="cuda"), step=state["step"])
    G.adamw_step([], [], **empty)
    assert state["step"].tolist() == [2, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_replayed(G, bits):
    """A captured step counts on, and takes its rate and the gradients' factor from device memory."""
    sizes = [700, 33, 5000]
    params, grads = make(sizes, torch.bfloat16, torch.bfloat16)
    twin = [p.clone() for p in params]
    a, b = G.adamw_state(params, bits=bits, master=True), G.adamw_state(twin, bits=bits, master=True)
    rate, factor = torch.ones((), device="cuda"), torch.ones((), device="cuda")

    def step(p, state):
        G.adamw_step(p, grads, **state, **HYPER, lr_factor=rate, grad_factor=factor)
    step(params, a)  # before the capture, as on the other side
    step(twin, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(params, a)
    for i in range(4):
        rate.fill_(0.5 ** i)
        factor.fill_(1.0 + i)
        for g in grads:
            g.mul_(-0.7)
        graph.replay()
        torch.cuda.synchronize()
        step(twin, b)
        assert all(torch.equal(x, y) for x, y in zip(params, twin))
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    assert a["step"].tolist() == [6 - 1, 0]


def test_graphs_see_the_update(G):
    """A graph that has saved a parameter refuses its backward pass after the step."""
    w = torch.ones(20, 24, device="cuda", requires_grad=True)
    x = torch.ones(30, 24, device="cuda", requires_grad=True)
    y, _ = G.linear(x, w)
    state = G.adamw_state([w])
    G.adamw_step([w], [torch.ones_like(w)], **state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_refusals(G):
    params, grads = make([300, 20], torch.bfloat16, torch.bfloat16)
    state = G.adamw_state(params)
    f32 = [p.float() for p in params]

    def call(p=params, g=grads, **other):
        return G.adamw_step(p, g, **{**state, **other})
    half = {k: torch.zeros(768, device="cuda", dtype=torch.uint8).view(F8) for k in ("m", "v")}
    for bad in (lambda: call(g=grads[:1]), lambda: call(g=[grads[0], grads[0]]), lambda: call(p=[params[0], f32[1]]),
                lambda: call(g=[grads[0], f32[1]]), lambda: call(p=[p.cpu() for p in params]),
                lambda: call(p=[params[0], params[0][:20]], g=[grads[0], grads[1]]),
                lambda: call(p=[params[0], torch.zeros(40, device="cuda", dtype=torch.bfloat16)[::2]]),
                lambda: call(m=state["m"][:-1]), lambda: call(v=state["v"].half()), lambda: call(**half),
                lambda: call(step=state["step"].int()), lambda: call(master=state["m"][:5]),
                lambda: call(p=f32, g=f32, master=state["m"]), lambda: call(lr_factor=torch.ones(2, device="cuda")),
                lambda: call(grad_factor=torch.ones(())), lambda: call(m=state["m"].cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: call(lr=-1.0), lambda: call(beta1=1.0), lambda: call(eps=0.0), lambda: call(lr=math.nan)):
        with pytest.raises(G.GmmError):
            bad()
    assert state["step"].tolist() == [0, 0] and (state["m"] == 0).all()
