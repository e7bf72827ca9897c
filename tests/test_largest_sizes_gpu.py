"""k3moe_gate at the largest count of tokens that its argument holds, and
k3moe_linear at the largest it takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 4])
def test_gate_most_tokens(T):
    """One expert, its score 1 by softmax; the last token and one in the middle
    without any expert.  21 GB."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory free")
    logits = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    out = (T // 2, T - 1)
    for t in out:
        logits[t] = float("-inf")
    idx = torch.full((T, 1), 7, dtype=torch.int32, device="cuda")
    weight = torch.full((T, 1), 7.0, device="cuda")
    m.check(m.k3moe_gate(logits, T, None, m.make_gate(1, 1, flags=m.K3MOE_LOGITS_BF16), idx, weight))
    torch.cuda.synchronize()
    for t in out:
        assert int(idx[t]) == -1 and float(weight[t]) == 0
        idx[t] = 0
        weight[t] = 1
    assert int(idx.min()) == int(idx.max()) == 0
    assert float(weight.min()) == float(weight.max()) == 1


@pytest.mark.parametrize("T,n", [(2 ** 30, 1), (2 ** 30 - 3, 3)])
def test_linear_most_tokens(T, n):
    """Small whole numbers, so that every sum is exact.  26 GB at most."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory free")
    x = torch.ones((T, 8), dtype=torch.bfloat16, device="cuda")
    rows = [0, 255, T // 2, T - 1]
    for i, t in enumerate(rows):
        x[t] = i + 2
    w = torch.arange(1, n + 1, device="cuda").to(torch.bfloat16)[:, None].expand(n, 8).contiguous()
    lin = m.make_linear(n, 8)
    ws = m.new_linear_workspace(lin, T)
    out = torch.full((T, n), 7.0, dtype=torch.bfloat16, device="cuda")
    m.check(m.k3moe_linear(x, T, w, None, None, None, None, lin, out, ws))
    torch.cuda.synchronize()
    m.check(m.k3moe_device_status(ws))
    for i, t in enumerate(rows):
        assert out[t].tolist() == [8.0 * (c + 1) * (i + 2) for c in range(n)]
        out[t] = out[1]
    for c in range(n):
        assert float(out[:, c].min()) == float(out[:, c].max()) == 8 * (c + 1)
