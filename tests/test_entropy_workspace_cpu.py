"""The workspace of the cross entropy and its gradients: pieces of rows pass through it, so it does not grow with the rows
of a call once they are many."""
import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    from soft_clustering_gmm_amd import gmm
    return gmm.lib()


@pytest.mark.parametrize("t", [0, 1, 2], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,V", [(64, 1 << 20), (520, 1 << 20), (7, 1 << 20), (64, 65536), (2048, 65536), (300, 9001), (33, 50),
                                 (16, 1)])
def test_bounded(L, t, d, V):
    e = 4 if t == 0 else 2
    lx = -(-d * e // 16) * 16  # bytes of a padded row
    for gradients in (0, 1):
        sizes = [L.gmm_cross_entropy_workspace_bytes(N, d, V, t, gradients) for N in (1 << 20, 1 << 22, 1 << 24, 1 << 30)]
        # logits (float) and their gradient, 256 rows at least, or as many as 2^29 logits; two copies of X's rows and 128
        # bytes a row beside; W padded, dW so far; partial sums of products (2 GB at most); the bias's sums, of 16 rows
        # each at least, or 1024 of them, once more where they are folded
        rows = min(1 << 20, max(256, (1 << 29) // V))
        sums = 2 * max(rows // 16, 1024) + 257
        most = rows * V * (4 + e) * 1.01 + rows * (2 * lx + 128) + V * (lx + 4 * d) + (2 << 30) + sums * V * 4
        stats = rows * -(-V // 32) * 8 * 1.1 + (300 << 20)
        assert all(s <= most + stats for s in sizes), (gradients, sizes, most + stats)


def test_many_rows_of_many_classes(L):
    # 2^24 rows of 64 features to 2^20 classes: far inside the limits, and has to fit a device beside W and dW
    for N in (1 << 20, 1 << 22, 1 << 24, 1 << 30):
        assert L.gmm_cross_entropy_workspace_bytes(N, 64, 1 << 20, 2, 1) <= 4 << 30
