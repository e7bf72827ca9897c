"""Waits of the dense product that run out, without any GPU fault: the
library's failure-path hook leaves out some of the copies waited for.  The call
records K3MOE_ERR_DEVICE_TIMEOUT and ends in bounded time with nothing of
its own in flight, the device stays usable, and on a workspace zero-filled
again the next call gives the bytes from before the failure."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    m.k3moe_debug_set_fault(0, 0)
    torch.cuda.empty_cache()


def product(T, n, k, gated, fp32):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + n + k)

    def r(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(BF)

    x, w, wg = r(T, k), r(n, k, std=k ** -0.5), r(n, k, std=k ** -0.5) if gated else None
    lin = m.make_linear(n, k, m.K3MOE_ACT_SILU if gated else 0, m.K3MOE_OUT_FP32 if fp32 else 0)
    ws = m.new_linear_workspace(lin, T)

    def run():
        out = torch.zeros((T, n), dtype=torch.float32 if fp32 else BF, device="cuda")
        m.check(m.k3moe_linear(x, T, w, wg, None, None, None, lin, out, ws), "k3moe_linear")
        torch.cuda.synchronize()
        return out, m.k3moe_device_status(ws)

    return run, ws


def runs_out_and_recovers(T, n, k, gated, fp32):
    run, ws = product(T, n, k, gated, fp32)
    want, status = run()
    assert status == m.K3MOE_OK
    t0 = time.monotonic()
    try:
        assert m.k3moe_debug_set_fault(1, 1_000_000) == m.K3MOE_OK  # 1 ms for each wait
        for _ in range(3):
            _, status = run()
            assert status == m.K3MOE_ERR_DEVICE_TIMEOUT
    finally:
        m.k3moe_debug_set_fault(0, 0)
    # three calls of a few waits of 1 ms each: no drain ran to its limit of 2 s
    assert time.monotonic() - t0 < 1.5
    ws.zero_()
    for _ in range(2):
        got, status = run()
        assert status == m.K3MOE_OK
        assert torch.equal(got, want)


@pytest.mark.parametrize("gated,fp32", [(False, True), (True, False)])
@pytest.mark.parametrize("T,n,k", [(1, 896, 7168), (8, 5000, 1536), (4, 40, 64), (12, 2600, 520)])
def test_few_tokens(T, n, k, gated, fp32):
    runs_out_and_recovers(T, n, k, gated, fp32)


@pytest.mark.parametrize("gated,fp32", [(False, True), (True, False)])
@pytest.mark.parametrize("T,n,k", [(40, 200, 64), (40, 200, 128), (130, 300, 136)])  # too short to be split
def test_tiles(T, n, k, gated, fp32):
    runs_out_and_recovers(T, n, k, gated, fp32)


@pytest.mark.parametrize("gated,fp32", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("T,n,k", [(64, 896, 7168), (100, 1536, 7168), (40, 130, 20000), (129, 65, 9000)])
def test_split_reductions(T, n, k, gated, fp32):
    """One CTA of each cluster gives up; the others get its part late or not in
    time, and leave only after it has landed."""
    runs_out_and_recovers(T, n, k, gated, fp32)


@pytest.mark.parametrize("gated,fp32", [(False, False), (True, False), (False, True)])
def test_a_wait_bounds_a_step_and_not_the_call(gated, fp32):
    """Some 5 ms of work in steps of 0.05 ms at most: with 1 ms for each wait
    nothing runs out, and every tile is written."""
    T, n, k = 65536, 3584 if gated else 7168, 7168
    run, ws = product(T, n, k, gated, fp32)
    want, status = run()
    assert status == m.K3MOE_OK
    try:
        assert m.k3moe_debug_set_fault(0, 1_000_000) == m.K3MOE_OK
        got, status = run()
    finally:
        m.k3moe_debug_set_fault(0, 0)
    assert status == m.K3MOE_OK
    assert torch.equal(got, want)


@pytest.mark.parametrize("gated,fp32", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,n,k", [(4096, 4104, 72), (2047, 2500, 520), (4095, 2304, 1096), (1500, 3001, 584)])
def test_pairs(T, n, k, gated, fp32):
    """One CTA of each pair stops a copy short of the other."""
    runs_out_and_recovers(T, n, k, gated, fp32)
