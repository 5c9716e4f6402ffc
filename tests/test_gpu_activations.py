"""The activations and their slopes over the whole line, with bounds relative to the value: gelu's and silu's negative
tails are far below 1 and a bound next to 1 would not see them."""
import pytest

torch = pytest.importorskip("torch")

from tests import layer_bounds as bounds  # noqa: E402
from tests import layer_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def line(t):
    """From the left tail to where both functions are the identity, small and large ones of either sign."""
    small = torch.logspace(-7, 0, 200, dtype=torch.float64)
    large = torch.tensor([14.5, 50.0, 87.0, 88.5, 100.0, 3e4, 6e4], dtype=torch.float64)
    z = torch.cat([torch.linspace(-14, 10, 2400, dtype=torch.float64), small, -small, large, -large, torch.zeros(1)])
    if t != torch.float16:
        z = torch.cat([z, torch.tensor([1e20, -1e20, 3e38, -3e38])])
    return z.to(t)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_values(name, dtype, out):
    from soft_clustering_gmm_amd import gmm as G
    t, o = TYPES[dtype], TYPES[out]
    z, act = line(t), getattr(G, "ACT_" + name.upper())
    want = oracle.act(z.double(), name)
    bound = bounds.value_bound(want, o)
    # one row times many weights (the stream over the weights), many rows times eight and three ones (the tiled product)
    Y, _ = G.linear(torch.ones(1, 1, dtype=t, device="cuda"), z[:, None].contiguous().cuda(), act=act, out_dtype=o)
    oracle.check(Y[0], want, bound, "few rows")
    for n in (8, 3):
        Y, pre = G.linear(z[:, None].contiguous().cuda(), torch.ones(n, 1, dtype=t, device="cuda"), act=act, out_dtype=o,
                          want_pre=True)
        assert torch.equal(pre.cpu().double(), z.double()[:, None].expand(-1, n))
        oracle.check(Y, want[:, None].expand(-1, n), bound[:, None].expand(-1, n), f"{n} columns")


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_values_in_the_experts(name, dtype):
    """One expert of one input, act(z) times 1: h is what the second product takes."""
    from soft_clustering_gmm_amd import gmm as G
    t = TYPES[dtype]
    z = line(t)
    want = oracle.act(z.double(), name)
    n = z.numel()
    eye = torch.zeros(1, 1, n, dtype=t)  # the first product's row i is z_i; the second takes one of them
    for i in range(0, n, 97):
        eye.zero_()
        eye[0, 0, i] = 1
        y = G.expert_rows(torch.ones(1, 1, dtype=t, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                          torch.ones(1, 1, device="cuda"), z[None, :, None].contiguous().cuda(), eye.cuda(),
                          act=getattr(G, "ACT_" + name.upper()), glu=False)
        # the sum's zero products are exact; h and y are rounded to the same type
        oracle.check(y, want[i].reshape(1, 1), bounds.value_bound(want[i], t).reshape(1, 1), f"{float(z[i])}")


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_slopes(name, dtype):
    """One row, dY = 1: the bias's gradient is the slope, not rounded before."""
    from soft_clustering_gmm_amd import gmm as G
    t = TYPES[dtype]
    z = line(t)
    one = torch.ones(1, 1, dtype=t, device="cuda")
    want, size = bounds.slope_parts(z.double(), name)
    bound = bounds.RELATIVE[t.itemsize] * size + bounds.FLOOR + oracle.rounding(want, t)
    for out in {t, torch.float32}:
        pre = z[None].to(out).cuda()
        db = G.linear_backward(torch.ones_like(pre), one, z[:, None].contiguous().cuda(), pre=pre,
                               act=getattr(G, "ACT_" + name.upper()))[2]
        oracle.check(db, want, bound, str(out))
