"""How exactly k3moe_linear carries its sums, as include/k3moe.h states it: with
terms of one sign (the worst case of a sum that is cut towards zero) and the
bias at minus the exact sum, the output is the sum's error itself.

Bounds: a step of 16 products cuts at most 2^-23 of the running sum, so a chain
of n steps at most n 2^-23 of the whole sum S, and chains added to nearest keep
the longest chain's factor (32 steps of 16 with an fp32 output; all of K with a
bf16 one).  To that 32 further half units of 2^-23 for the parts' additions,
2^-24 S for the bias, and the output's own rounding of a small number."""
import pytest
import torch

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("K", [512, 7168, 32768])
@pytest.mark.parametrize("T,n", [(1, 900), (8, 1024), (12, 300), (40, 130), (300, 512), (2048, 4096)])
def test_sums_of_one_sign(T, n, K, fp32):
    g = torch.Generator(device="cuda")
    g.manual_seed(K + T)
    x = torch.randn(1, K, generator=g, device="cuda").abs().to(torch.bfloat16)
    w = torch.randn(n, K, generator=g, device="cuda").abs().to(torch.bfloat16)
    exact = (w.double() @ x.double().T)[:, 0]
    bias = -exact.float()
    lin = m.make_linear(n, K, 0, m.K3MOE_OUT_FP32 if fp32 else 0)
    out = torch.empty((T, n), dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    ws = m.new_linear_workspace(lin, T)
    m.check(m.k3moe_linear(x.expand(T, K).contiguous(), T, w, None, bias, None, None, lin, out, ws))
    torch.cuda.synchronize()
    m.check(m.k3moe_device_status(ws))
    assert (out == out[:1]).all()  # equal tokens, equal sums
    err = ((out[0].double() - (exact + bias.double())).abs() / exact).max()
    steps = 32 if fp32 or T <= 8 else K // 16
    assert float(err) <= ((steps + 32) * 2.0 ** -23 + 2.0 ** -24) * (1 + 2.0 ** -8)
