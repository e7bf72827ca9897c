"""k3moe_layer_routed on the GPU: against the fp64 oracle's combine under the
same routing (gate G1), against k3moe_layer under the layer's own routing, and
the chain of the bf16 router product, the routing and the layer."""
import numpy as np
import pytest
import torch

import k3gen
from gpu_helpers import dims_of, run_layer, sample_tokens
from k3gen import device as kdev
from operator_refs import gate_ref
from parity import G1_TOL, g1_error

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None

SMALL = k3gen.Config("small", d=512, ff=256, E=64, k=8, ff_shared=192, T=0)
TINY = k3gen.CONFIGS["tiny"]
ODD = k3gen.Config("odd", d=320, ff=192, E=40, k=5, ff_shared=64, T=0)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    kdev.release_all()


def routed(cfg, W, x, idx, w, flags=0, ws_tokens=None, ptrs=None, status=0, ws=None, y=None):
    T = idx.shape[0]
    dims = dims_of(cfg, flags)
    ws = m.new_workspace(dims, T if ws_tokens is None else ws_tokens) if ws is None else ws
    if y is None:
        y = torch.full((T, cfg.d), float("nan"), device="cuda",
                       dtype=torch.float32 if flags & m.K3MOE_OUT_FP32 else torch.bfloat16)
    sh = W.shared if not (flags & m.K3MOE_NO_SHARED) else (None, None, None)
    m.check(m.k3moe_layer_routed(x, T, torch.as_tensor(idx, dtype=torch.int32, device="cuda"),
                                 torch.as_tensor(w, dtype=torch.float32, device="cuda"),
                                 W.blob_ptrs if ptrs is None else ptrs, *sh, dims, y, ws), "k3moe_layer_routed")
    torch.cuda.synchronize()
    assert m.k3moe_device_status(ws) == status
    return y


def oracle_y(orc, cfg, W, x_host, idx, w, tokens, shared=True):
    xs = x_host[tokens]
    weight = np.where(idx[tokens] >= 0, w[tokens], 0.0).astype(np.float64)
    cache = {}
    blobs = [cache.setdefault(e, W.blob_host(e)) for t in tokens for e in (int(max(v, 0)) for v in idx[t])]
    return orc.combine(xs, weight, blobs, W.shared_host if shared else None, cfg.d, cfg.ff)


def random_routing(cfg, T, seed, missing=0.0):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(cfg.E)[:cfg.k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, cfg.k)).astype(np.float32) + 0.05
    gone = rng.random((T, cfg.k)) < missing
    return np.where(gone, -1, idx).astype(np.int32), w


@pytest.mark.parametrize("cfg,T,ws_tokens", [(TINY, 1, 1), (TINY, 4, 4), (SMALL, 8, 8), (SMALL, 20, 8), (TINY, 9, 9),
                                             (SMALL, 33, 33), (SMALL, 200, 200), (ODD, 3, 3), (ODD, 70, 70)])
@pytest.mark.parametrize("missing", [0.0, 0.3])
@pytest.mark.parametrize("shared", [True, False])
def test_against_the_oracle(orc, cfg, T, ws_tokens, missing, shared):
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, T, missing)
    flags = m.K3MOE_OUT_FP32 | (0 if shared else m.K3MOE_NO_SHARED)
    y = routed(cfg, W, inp.x, idx, w, flags, ws_tokens).cpu().numpy()
    tokens = sample_tokens(T, 12)
    err = g1_error(y[tokens], oracle_y(orc, cfg, W, inp.x_host, idx, w, tokens, shared))
    assert err.max() <= G1_TOL, err


SCALES = [k3gen.Config("rows22", d=704, ff=192, E=48, k=8, ff_shared=64, T=0),    # scale rows of 22 and 6 bytes
          k3gen.Config("rows20", d=640, ff=384, E=48, k=8, ff_shared=128, T=0),   # 20 and 12
          k3gen.Config("rows24", d=768, ff=256, E=48, k=8, ff_shared=64, T=0),    # 24 and 8
          k3gen.Config("rows2", d=1216, ff=64, E=48, k=8, ff_shared=64, T=0)]     # 38 and 2


@pytest.mark.parametrize("cfg", SCALES, ids=lambda c: c.name)
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 60, 400])
def test_scale_rows_of_every_alignment(orc, cfg, T):
    """Reduction lengths whose scale rows no tensor map reaches, with several
    items and several expert groups per CTA."""
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, T + 1, 0.1)
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32).cpu().numpy()
    tokens = sample_tokens(T, 12)
    err = g1_error(y[tokens], oracle_y(orc, cfg, W, inp.x_host, idx, w, tokens))
    assert err.max() <= G1_TOL, err


@pytest.mark.parametrize("T", [1, 8, 9, 40, 100])
def test_wide_shared_expert(orc, T):
    """A shared expert with more rows than the hidden size and the routed
    experts have, so with more row blocks than any of theirs."""
    cfg = k3gen.Config("wide_shared", d=256, ff=64, E=32, k=4, ff_shared=1536, T=0)
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, T + 2, 0.1)
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32).cpu().numpy()
    tokens = sample_tokens(T, 12)
    assert g1_error(y[tokens], oracle_y(orc, cfg, W, inp.x_host, idx, w, tokens)).max() <= G1_TOL
    yl, il, wl = run_layer(cfg, W, inp.x, None, T)
    got = routed(cfg, W, inp.x, il, wl)
    assert np.array_equal(got.view(torch.int16).cpu().numpy(), yl)


@pytest.mark.parametrize("T", [9, 33, 63, 64, 65])
def test_sort_in_one_launch_and_in_five(orc, T):
    """Both sides of the number of tokens up to which one CTA sorts, with all
    tokens on one expert, with 32 picks a token and with picks left out."""
    cfg = k3gen.Config("many", d=128, ff=64, E=200, k=32, ff_shared=64, T=0)
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, T, 0.2)
    idx[:, 0] = 7
    idx[:, 1:] = np.where(idx[:, 1:] == 7, -1, idx[:, 1:])
    idx[3] = -1
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32).cpu().numpy()
    tokens = sample_tokens(T, 16)
    assert g1_error(y[tokens], oracle_y(orc, cfg, W, inp.x_host, idx, w, tokens)).max() <= G1_TOL


@pytest.mark.parametrize("cfg,T", [(TINY, 1), (SMALL, 8), (SMALL, 100), (k3gen.CONFIGS["k3_decode"], 1),
                                   (k3gen.CONFIGS["k3_decode"], 3)])
def test_the_layers_own_routing_gives_the_layer(cfg, T):
    """Under the routing k3moe_layer chose, the outputs are the layer's, bit
    for bit: the same kernels run on the same dispatch."""
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    y, idx, w = run_layer(cfg, W, inp.x, None, T)
    got = routed(cfg, W, inp.x, idx, w)
    assert np.array_equal(got.view(torch.int16).cpu().numpy(), y)


@pytest.mark.parametrize("T,ws_tokens", [(2, 2), (8, 8), (40, 40)])
def test_repeated_experts(orc, T, ws_tokens):
    """The same expert in several places of a row: its weights add up."""
    cfg = SMALL
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, 5)
    idx[0, :] = idx[0, 0]
    idx[1, 3] = idx[1, 1]
    idx[1, 6] = idx[1, 1]
    idx[T - 1, 7] = idx[T - 1, 0]
    w[0, 2] = -0.5
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32, ws_tokens).cpu().numpy()
    tokens = sample_tokens(T, 12)
    assert g1_error(y[tokens], oracle_y(orc, cfg, W, inp.x_host, idx, w, tokens)).max() <= G1_TOL


@pytest.mark.parametrize("T,ws_tokens", [(1, 1), (8, 8), (24, 24), (24, 8)])
def test_rows_without_any_expert(orc, T, ws_tokens):
    """No pick anywhere: the shared expert alone, or zero; weights of missing
    picks are not read."""
    cfg = SMALL
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx = np.full((T, cfg.k), -1, np.int32)
    w = np.full((T, cfg.k), np.nan, np.float32)
    none = torch.zeros_like(W.blob_ptrs)
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32 | m.K3MOE_NO_SHARED, ws_tokens, ptrs=none)
    assert (y == 0).all()
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32, ws_tokens, ptrs=none).cpu().numpy()
    tokens = sample_tokens(T, 8)
    ref = oracle_y(orc, cfg, W, inp.x_host, np.zeros_like(idx), np.zeros_like(w), tokens)
    assert g1_error(y[tokens], ref).max() <= G1_TOL
    if T > 1:  # some rows with, some without
        idx2, w2 = random_routing(cfg, T, 3)
        idx2[::2] = -5
        w2[::2] = np.inf
        y = routed(cfg, W, inp.x, idx2, w2, m.K3MOE_OUT_FP32, ws_tokens).cpu().numpy()
        ref = oracle_y(orc, cfg, W, inp.x_host, idx2, w2, tokens)
        assert g1_error(y[tokens], ref).max() <= G1_TOL


@pytest.mark.parametrize("T,ws_tokens", [(3, 3), (30, 30)])
def test_ids_past_the_last_expert_are_reported(orc, T, ws_tokens):
    cfg = SMALL
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, 8)
    idx[1, 2] = cfg.E
    idx[2, 0] = 2 ** 31 - 1
    y = routed(cfg, W, inp.x, idx, w, m.K3MOE_OUT_FP32, ws_tokens, status=m.K3MOE_ERR_DEVICE_CHECK).cpu().numpy()
    idx[1, 2] = idx[2, 0] = -1
    tokens = sample_tokens(T, 8)
    assert g1_error(y[tokens], oracle_y(orc, cfg, W, inp.x_host, idx, w, tokens)).max() <= G1_TOL


@pytest.mark.parametrize("T", [2, 30])
def test_missing_blobs_of_unpicked_experts(T):
    """A pointer table that holds only the picked experts; a picked one that is
    missing is reported."""
    cfg = SMALL
    W = kdev.weights(cfg)
    inp = kdev.DeviceInputs(cfg, T=T)
    idx, w = random_routing(cfg, T, 4)
    idx %= 11  # repetitions too
    ptrs = W.blob_ptrs.clone()
    ptrs[11:] = 0
    full = routed(cfg, W, inp.x, idx, w)
    assert torch.equal(routed(cfg, W, inp.x, idx, w, ptrs=ptrs), full)
    ptrs[int(idx[0, 0])] = 0
    routed(cfg, W, inp.x, idx, w, ptrs=ptrs, status=m.K3MOE_ERR_DEVICE_CHECK)


def test_one_workspace_between_layer_and_routed_calls(orc):
    """Layer, routed and single-expert calls in turn on one workspace give what
    each gives on its own."""
    cfg = SMALL
    W = kdev.weights(cfg)
    dims = dims_of(cfg)
    ws = m.new_workspace(dims, 64)
    for T in (3, 64, 8, 1, 40):
        inp = kdev.DeviceInputs(cfg, T=T)
        y0, idx, w = run_layer(cfg, W, inp.x, None, T)
        idx2, w2 = random_routing(cfg, T, T, 0.2)
        alone = routed(cfg, W, inp.x, idx2, w2)
        y = torch.empty((T, cfg.d), dtype=torch.int16, device="cuda")
        got = torch.empty((T, cfg.d), dtype=torch.bfloat16, device="cuda")
        # ordered on the stream, no wait in between
        i2, v2 = torch.from_numpy(idx2).cuda(), torch.from_numpy(w2).cuda()
        for _ in range(3):
            m.check(m.k3moe_layer_routed(inp.x, T, i2, v2, W.blob_ptrs, *W.shared, dims, got, ws))
            m.check(m.k3moe_layer(inp.x, T, W.w_router, None, W.blob_ptrs, *W.shared, dims, y, None, None, ws))
        torch.cuda.synchronize()
        assert m.k3moe_device_status(ws) == 0
        assert np.array_equal(y.cpu().numpy(), y0)
        assert torch.equal(got, alone)


@pytest.mark.parametrize("T", [1, 6, 48])
def test_router_gate_layer_chain_in_a_graph(orc, T):
    """The chain a serving step runs: the bf16 router's product, the routing by
    sigmoid scores with a bias and groups, the layer on it; captured once,
    replayed with new tokens."""
    cfg = SMALL
    W = kdev.weights(cfg)
    dims = dims_of(cfg, m.K3MOE_OUT_FP32)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    wr = (torch.randn(cfg.E, cfg.d, generator=g, device="cuda") * cfg.d ** -0.5).to(torch.bfloat16)
    bias = torch.randn(cfg.E, generator=g, device="cuda") * 0.05
    lin = m.make_linear(cfg.E, cfg.d, m.K3MOE_ACT_NONE, m.K3MOE_OUT_FP32)
    gate = m.make_gate(cfg.E, cfg.k, m.K3MOE_SCORE_SIGMOID, 8, 4, 2, 2.5, m.K3MOE_RENORM_TOPK)
    lws, ws = m.new_linear_workspace(lin, T), m.new_workspace(dims, T)
    logits = torch.empty((T, cfg.E), device="cuda")
    idx = torch.empty((T, cfg.k), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, cfg.k), device="cuda")
    y = torch.empty((T, cfg.d), device="cuda")
    x = kdev.DeviceInputs(cfg, T=T).x.clone()

    def step():
        m.check(m.k3moe_linear(x, T, wr, None, None, None, None, lin, logits, lws))
        m.check(m.k3moe_gate(logits, T, bias, gate, idx, wt))
        m.check(m.k3moe_layer_routed(x, T, idx, wt, W.blob_ptrs, *W.shared, dims, y, ws))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        inp = kdev.DeviceInputs(cfg, seed=seed, T=T)
        x.copy_(inp.x)
        graph.replay()
        torch.cuda.synchronize()
        assert m.k3moe_device_status(ws) == 0 and m.k3moe_device_status(lws) == 0
        # the picks follow from the logits as computed; the logits from x
        ri, rw = gate_ref(logits.double().cpu().numpy(), cfg.k, "sigmoid", bias.double().cpu().numpy(), 8, 4, 2, True,
                          2.5)
        assert np.array_equal(idx.cpu().numpy(), ri)
        ref = x.view(torch.bfloat16).double() @ wr.double().T
        assert float((logits.double() - ref).norm() / ref.norm()) <= 1e-6
        tokens = sample_tokens(T, 8)
        yo = oracle_y(orc, cfg, W, inp.x_host, ri, rw, tokens)
        assert g1_error(y.cpu().numpy()[tokens], yo).max() <= G1_TOL


def test_dense_block_chain():
    """A dense gated block on the residual stream, both products: h + W_d
    (silu(W_g h) * W_u h), the second added in place."""
    T, d, ff = 37, 512, 320
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
    h, wg, wu, wd = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16), r(ff, d), r(ff, d), r(d, ff)
    up, down = m.make_linear(ff, d, m.K3MOE_ACT_SILU), m.make_linear(d, ff)
    ws = torch.zeros(max(m.k3moe_linear_workspace_size(l, T) for l in (up, down)), dtype=torch.uint8, device="cuda")
    mid = torch.empty((T, ff), dtype=torch.bfloat16, device="cuda")
    out = h.clone()
    m.check(m.k3moe_linear(out, T, wu, wg, None, None, None, up, mid, ws))
    m.check(m.k3moe_linear(mid, T, wd, None, None, None, out, down, out, ws))
    torch.cuda.synchronize()
    hd = h.double()
    a = torch.nn.functional.silu(hd @ wg.double().T) * (hd @ wu.double().T)
    ref = hd + a @ wd.double().T
    # the middle is rounded to bf16 (2^-8 of each value at most), then once more at the end
    tol = 2.0 ** -8 * (a.abs() @ wd.double().abs().T + ref.abs()) * 1.01 + 1e-5
    assert ((out.double() - ref).abs() <= tol).all()
