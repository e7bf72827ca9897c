"""Waits of a routed layer call that run out, without any GPU fault: the
library's failure-path hook withholds the signal that the routing is loaded.
The roles of a CTA that go through barriers together leave together, so the
call ends, records K3MOE_ERR_DEVICE_TIMEOUT, and on a workspace zero-filled
again gives the same bytes as before."""
import time

import numpy as np
import pytest
import torch

import k3gen
from gpu_helpers import dims_of
from k3gen import device as kdev

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    m.k3moe_debug_set_fault(0, 0)
    kdev.release_all()


# scale rows by TMA, by the scale warps in gate/up, in both passes; a shared
# expert of more work than the limit leaves time for, a small one, none
CFGS = [k3gen.Config("tma", d=512, ff=512, E=64, k=8, ff_shared=192, T=0),
        k3gen.Config("rows22", d=704, ff=192, E=48, k=8, ff_shared=64, T=0),
        k3gen.Config("wide_shared", d=704, ff=64, E=32, k=4, ff_shared=1536, T=0),
        k3gen.Config("none", d=320, ff=192, E=40, k=5, ff_shared=0, T=0)]


@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("cfg", CFGS, ids=lambda c: c.name)
def test_waits_that_run_out(cfg, T):
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    flags = m.K3MOE_OUT_FP32 | (0 if cfg.ff_shared else m.K3MOE_NO_SHARED)
    dims = dims_of(cfg, flags)
    ws = m.new_workspace(dims, T)
    rng = np.random.default_rng(T)
    idx = torch.from_numpy(np.stack([rng.permutation(cfg.E)[:cfg.k] for _ in range(T)]).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.random((T, cfg.k)).astype(np.float32)).cuda()

    def run():
        y = torch.zeros((T, cfg.d), device="cuda")
        m.check(m.k3moe_layer_routed(inp.x, T, idx, w, W.blob_ptrs, *W.shared, dims, y, ws), "k3moe_layer_routed")
        torch.cuda.synchronize()
        return y, m.k3moe_device_status(ws)

    want, status = run()
    assert status == m.K3MOE_OK
    for limit in (1_000, 20_000, 1_000_000):
        try:
            assert m.k3moe_debug_set_fault(1, limit) == m.K3MOE_OK
            _, status = run()
        finally:
            m.k3moe_debug_set_fault(0, 0)
        assert status == m.K3MOE_ERR_DEVICE_TIMEOUT
        ws.zero_()
        got, status = run()
        assert status == m.K3MOE_OK
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("cfg", [k3gen.CONFIGS["tiny"], CFGS[0], CFGS[2]], ids=lambda c: c.name)
def test_one_launch_waits_that_run_out(cfg, T):
    """The decode pass as one launch: the same end, well before the limit of a
    drain (2 s)."""
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    dims = dims_of(cfg, m.K3MOE_OUT_FP32 | m.K3MOE_ONE_LAUNCH)
    ws = m.new_workspace(dims, T)

    def run():
        y = torch.zeros((T, cfg.d), device="cuda")
        m.check(m.k3moe_layer(inp.x, T, W.w_router, None, W.blob_ptrs, *W.shared, dims, y, None, None, ws))
        torch.cuda.synchronize()
        return y, m.k3moe_device_status(ws)

    want, status = run()
    assert status == m.K3MOE_OK
    t0 = time.monotonic()
    try:
        assert m.k3moe_debug_set_fault(1, 1_000_000) == m.K3MOE_OK
        _, status = run()
    finally:
        m.k3moe_debug_set_fault(0, 0)
    assert status == m.K3MOE_ERR_DEVICE_TIMEOUT
    assert time.monotonic() - t0 < 1.0
    ws.zero_()
    got, status = run()
    assert status == m.K3MOE_OK
    assert torch.equal(got, want)
