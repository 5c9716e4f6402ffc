"""A caller's workspace for the layers: where it lies and what it holds are checked before its address goes on."""
import pytest

torch = pytest.importorskip("torch")

from soft_clustering_gmm_amd import gmm  # noqa: E402


def test_space():
    cpu = torch.device("cpu")
    assert gmm._space(None, cpu) == (None, 0)
    ws = torch.empty(1000, dtype=torch.uint8)
    assert gmm._space(ws, cpu) == (ws.data_ptr(), 1000)
    assert gmm._space(torch.empty(8, 3, dtype=torch.float64), cpu)[1] == 192
    with pytest.raises(ValueError):  # memory of another device
        gmm._space(ws, torch.device("cuda", 0))
    with pytest.raises(ValueError):
        gmm._space(torch.empty(8, dtype=torch.uint8, device="meta"), cpu)
    with pytest.raises(ValueError):  # a million elements in one byte
        gmm._space(torch.empty(1, dtype=torch.uint8).expand(1 << 20), cpu)
    with pytest.raises(ValueError):
        gmm._space(ws[::2], cpu)


@pytest.mark.gpu
def test_calls_refuse_a_workspace_elsewhere():
    X, W = torch.ones(40, 45, device="cuda"), torch.ones(20, 45, device="cuda")
    here = gmm.linear_workspace(40, 45, 20, torch.float32, X.device, backward=True)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), here[:1].expand(1 << 20)):
        with pytest.raises(ValueError):
            gmm.linear(X, W, ws=ws)
        with pytest.raises(ValueError):
            gmm.linear_backward(torch.ones(40, 20, device="cuda"), X, W, ws=ws)
        with pytest.raises(ValueError):
            gmm.expert_rows(X, torch.zeros(40, 1, dtype=torch.int32, device="cuda"), torch.ones(40, 1, device="cuda"),
                            torch.ones(2, 6, 45, device="cuda"), torch.ones(2, 45, 3, device="cuda"), ws=ws)
        with pytest.raises(ValueError):
            gmm.expert_layer(X, W[:4], torch.zeros(2, 4, device="cuda"), torch.ones(2, 4, device="cuda"),
                             torch.zeros(2, device="cuda"), torch.ones(2, 6, 45, device="cuda"),
                             torch.ones(2, 45, 3, device="cuda"), ws=ws)
    with pytest.raises(gmm.GmmError):  # too small
        gmm.linear(X, W, ws=here[:256])
    assert (gmm.linear(X, W, ws=here.view(torch.int64))[0] == 45).all()
