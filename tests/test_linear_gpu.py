"""k3moe_linear on the GPU against the plain 64-bit product, with the error
bounds of operator_refs."""
import pytest
import torch

from operator_refs import linear_norm_tol, linear_ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None
BF = torch.bfloat16
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def data(T, n, k, seed=0, gated=False, bias=False, resid=False, fp32=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(*s, std=1.0, dtype=BF):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)

    return {"x": r(T, k), "w": r(n, k, std=k ** -0.5), "wg": r(n, k, std=k ** -0.5) if gated else None,
            "b": r(n, dtype=torch.float32) if bias else None,
            "bg": r(n, dtype=torch.float32) if bias and gated else None,
            "r": r(T, n, dtype=torch.float32 if fp32 else BF) if resid else None}


def call(d, act="none", fp32=False, out=None, ws=None, stream=None):
    T, k = d["x"].shape
    n = d["w"].shape[0]
    lin = m.make_linear(n, k, ACTS[act], m.K3MOE_OUT_FP32 if fp32 else 0)
    ws = m.new_linear_workspace(lin, T) if ws is None else ws
    if out is None:
        out = torch.full((T, n), float("nan"), dtype=torch.float32 if fp32 else BF, device="cuda")
    m.check(m.k3moe_linear(d["x"], T, d["w"], d["wg"], d["b"], d["bg"], d["r"], lin, out, ws, stream=stream),
            "k3moe_linear")
    return out, ws


def check(d, act="none", fp32=False, out=None, ws=None):
    out, ws = call(d, act, fp32, out, ws)
    torch.cuda.synchronize()
    m.check(m.k3moe_device_status(ws), "device status")
    compare(out, d, act, fp32)
    return out


def compare(out, d, act, fp32):
    bits = 24 if fp32 else 8
    ref, tol = linear_ref(d["x"], d["w"], d["wg"], d["b"], d["bg"], d["r"], act, bits)
    err = (out.double() - ref).abs()
    bad = (~(err <= tol)).nonzero()
    assert len(bad) == 0, (len(bad), bad[:4].tolist(), float(err.max()))
    rel = float(err.norm() / ref.norm()) if float(ref.norm()) else 0.0
    assert rel <= linear_norm_tol(d["x"].shape[1], bits), rel


TOKENS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 511, 512, 700,
          1025]


@pytest.mark.parametrize("T", TOKENS)
def test_tokens(T):
    """Every count of tokens, on a shape with ragged edges and on one without."""
    i = TOKENS.index(T)
    check(data(T, 300, 520, seed=T, bias=True), list(ACTS)[i % 5], fp32=i % 3 == 0)
    check(data(T, 256, 1024, seed=T, resid=True, fp32=i % 2 == 0), fp32=i % 2 == 0)
    check(data(T, 200, 264, seed=T, gated=True, bias=True, resid=i % 2 == 1), "silu")


@pytest.mark.parametrize("n,k", [(1, 8), (1, 4096), (7, 8), (8, 16), (15, 24), (16, 72), (17, 64), (33, 40), (63, 128),
                                 (64, 56), (65, 1000), (127, 136), (128, 2048), (129, 8), (1001, 1000), (896, 7168),
                                 (2050, 48), (4000, 264)])
@pytest.mark.parametrize("T", [1, 5, 8, 13, 24, 40, 130, 400])
def test_sizes(n, k, T):
    check(data(T, n, k, seed=n + k, bias=n % 2 == 0, resid=T % 2 == 0), "gelu" if n % 3 == 0 else "none")
    check(data(T, n, k, seed=n + k, gated=True, bias=True, fp32=True, resid=True), "silu", fp32=True)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T", [1, 12, 60, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue(act, T, gated):
    for fp32 in (False, True):
        for bias in (False, True):
            check(data(T, 192, 256, 3, gated, bias, resid=fp32 != bias, fp32=fp32), act, fp32)


@pytest.mark.parametrize("T,n,k,gated,act,resid,fp32", [
    (1, 1536, 7168, True, "silu", False, False), (8, 7168, 1536, False, "none", True, False),
    (64, 896, 7168, False, "none", False, True), (512, 896, 7168, False, "none", False, True),
    (1000, 1536, 7168, True, "silu", False, False), (2049, 7168, 1536, False, "none", True, False),
    (4096, 1536, 7168, True, "silu", False, False), (3001, 2000, 1000, False, "gelu_tanh", True, True)])
def test_layer_sizes(T, n, k, gated, act, resid, fp32):
    d = data(T, n, k, 11, gated, resid=resid, fp32=fp32)
    a = check(d, act, fp32)
    b, _ = call(d, act, fp32)
    torch.cuda.synchronize()
    assert torch.equal(a, b)  # the same inputs, the same bits


@pytest.mark.parametrize("T,n,k,gated,act,resid,fp32", [
    # rings that go round, and CTAs that go from group to group of columns
    (3, 5000, 320, False, "none", True, False), (5, 4803, 4104, False, "relu", False, True),
    (8, 3001, 1032, True, "silu", True, False), (1, 20000, 64, False, "gelu", False, False),
    (2, 40, 30000, False, "none", True, True), (8, 17, 20008, True, "silu", False, True),
    (12, 5001, 520, True, "gelu_tanh", False, False), (16, 2600, 1000, False, "none", True, False),
    (9, 9001, 72, False, "relu", False, True),
    # split reductions, chains longer than one
    (17, 896, 7168, False, "none", False, True), (40, 130, 20000, False, "gelu", True, True),
    (300, 64, 16384, False, "none", False, True), (100, 1536, 7168, True, "silu", False, False),
    (129, 65, 9000, True, "silu", True, True), (500, 129, 2504, False, "relu", True, False),
    (600, 300, 40000, False, "none", True, False), (20, 3000, 70000, True, "relu", False, False),
    # few tokens in tiles, for more weights than are streamed for them
    (12, 3001, 3504, True, "silu", True, False), (16, 2600, 8200, False, "none", True, True),
    (9, 2563, 8008, False, "gelu", False, False),
    # fp32 outputs in tiles of up to 256 tokens, chain after chain
    (4095, 900, 1024, False, "none", True, True), (1300, 1024, 1096, True, "silu", False, True),
    (2500, 1001, 1240, False, "gelu", True, True), (3000, 896, 576, False, "none", False, True),
    # CTA pairs: ragged rows, columns and K
    (1500, 3001, 520, True, "silu", True, False), (2047, 1000, 328, False, "none", False, False),
    (1111, 2500, 1000, False, "gelu", True, False), (5000, 130, 2056, True, "relu", False, False),
    (4096, 4104, 72, False, "none", True, False),
    # CTA pairs with fp32 outputs: one chain, several, a last one of one K-step
    (4096, 4104, 72, False, "none", True, True), (2047, 2500, 520, False, "gelu", False, True),
    (1500, 3001, 584, True, "silu", True, True), (4095, 2304, 1096, True, "relu", False, True),
    (3000, 7168, 1536, False, "none", True, True), (2100, 2600, 2600, False, "none", False, True)])
def test_variants(T, n, k, gated, act, resid, fp32):
    check(data(T, n, k, T + n, gated, bias=n % 2 == 0, resid=resid, fp32=fp32), act, fp32)


def test_first_call_is_captured():
    """The library's set-up on a device happens in whichever call comes first,
    also one that is captured."""
    import subprocess
    import sys
    code = """
import torch, mxfp4_routed_expert_softmax_b200 as m
for T in (2, 40, 600):
    x, w = torch.randn(T, 512, device="cuda").bfloat16(), torch.randn(256, 512, device="cuda").bfloat16()
    lin = m.make_linear(256, 512, 0, m.K3MOE_OUT_FP32)
    ws, out = m.new_linear_workspace(lin, T), torch.zeros(T, 256, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.check(m.k3moe_linear(x, T, w, None, None, None, None, lin, out, ws))
    g.replay()
    torch.cuda.synchronize()
    ref = x.double() @ w.double().T
    assert float((out.double() - ref).norm() / ref.norm()) < 1e-5
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_fp32_precision():
    """Long reductions with fp32 output stay within a few units of fp32: the
    partial sums are short enough that the error does not grow with K (a plain
    fp32 product of 7168 random terms is off by about 3e-7)."""
    for T in (1, 8, 16, 64, 300, 600):
        d = data(T, 896, 7168, T)
        out, _ = call(d, fp32=True)
        ref = d["x"].double() @ d["w"].double().T
        assert float((out.double() - ref).norm() / ref.norm()) <= 1e-6


@pytest.mark.parametrize("T", [1, 4, 8, 11, 40, 150, 300, 600])
def test_rows_of_wider_tensors(T):
    """Operands as slices of wider rows, the output too: what lies beside and
    behind the slice stays as it was."""
    n, k = 130, 136
    d = data(T, n, k, 5, gated=True, bias=True, resid=True)
    wide = {a: torch.full((d[a].shape[0] + 2, d[a].shape[1] + 24), float("nan"), dtype=BF, device="cuda")
            for a in ("x", "w", "wg", "r")}
    s = dict(d)
    for a, off in (("x", 8), ("w", 16), ("wg", 16), ("r", 3)):
        s[a] = wide[a][:d[a].shape[0], off:off + d[a].shape[1]]
        s[a].copy_(d[a])
    for off in (0, 8, 5):
        o = torch.full((T + 2, n + 24), 77.0, dtype=BF, device="cuda")
        check(s, "silu", out=o[:T, off:off + n])
        o[:T, off:off + n] = 77.0
        assert (o == 77.0).all()


@pytest.mark.parametrize("T", [1, 8, 20, 128, 384])
def test_in_place_residual(T):
    for fp32 in (False, True):
        d = data(T, 264, 512, 9, resid=True, fp32=fp32)
        h = d["r"].clone()
        out, ws = call({**d, "r": h}, fp32=fp32, out=h)
        torch.cuda.synchronize()
        compare(out, d, "none", fp32)


@pytest.mark.parametrize("T", [3, 8, 40, 130, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_infinities_and_nans_stay_in_their_rows(T, gated):
    """A token with NaN or infinite entries touches its own row only, a weight
    row its own column, also next to rows and columns that do not exist."""
    n, k = 72, 200
    d = data(T, n, k, 2, gated)
    d["x"][T - 1, 3] = float("nan")
    d["x"][0, 5] = float("inf")
    d["w"][n - 1, 7] = float("inf")
    out, ws = call(d, "silu", True)
    ok = torch.ones(T, n, dtype=torch.bool, device="cuda")
    ok[T - 1], ok[0], ok[:, n - 1] = False, False, False
    assert torch.isnan(out[T - 1]).all()
    assert not torch.isfinite(out[:, n - 1]).any() or gated
    clean = {a: None if v is None else v.clone() for a, v in d.items()}
    clean["x"][T - 1, 3], clean["x"][0, 5], clean["w"][n - 1, 7] = 0, 0, 0
    ref, tol = linear_ref(clean["x"], clean["w"], clean["wg"], act="silu")
    assert (((out.double() - ref).abs() <= tol) | ~ok).all()


def test_zero_and_huge_values():
    d = data(33, 40, 64, 1, bias=True)
    d["x"].zero_()
    check(d, "gelu")
    d = data(20, 64, 64, 1)
    d["x"] *= 2.0 ** 60
    d["w"] *= 2.0 ** 60
    check(d, "none", True)
    d["x"] *= 2.0 ** 40  # past fp32's range
    out, _ = call(d, "none", True)
    assert not torch.isfinite(out).all()


def test_offsets_past_32_bits():
    """The output's rows span more than 2^31 elements, and x's."""
    T, n, k = 70000, 64, 64
    d = data(T, n, k, 3)
    wide = torch.empty((T, 32768), dtype=BF, device="cuda")
    out = wide[:, 512:512 + n]
    xw = torch.empty((T, 32768), dtype=BF, device="cuda")
    xs = xw[:, 1024:1024 + k]
    xs.copy_(d["x"])
    check({**d, "x": xs}, out=out)


def test_one_workspace_many_calls():
    """Calls of all kinds one after the other on one workspace, sized for the
    largest, on one stream."""
    ws = None
    for T, n, k in ((300, 200, 512), (1, 896, 7168), (8, 200, 4096), (64, 128, 2048), (2, 64, 64), (300, 200, 512)):
        d = data(T, n, k, T)
        need = m.k3moe_linear_workspace_size(m.make_linear(896, 7168), 1024)
        need = max(need, m.k3moe_linear_workspace_size(m.make_linear(n, k), T))
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if ws is None or ws.numel() < need else ws
        check(d, fp32=True, ws=ws)


@pytest.mark.parametrize("T,n,k", [(1, 896, 7168), (8, 1024, 1536), (50, 256, 4096), (300, 512, 512)])
def test_streams_and_graph(T, n, k):
    """Two calls at once on two streams with a workspace each; captured and
    replayed with new inputs."""
    a, b = data(T, n, k, 1), data(T, n, k, 2)
    oa, wa = call(a, fp32=True)
    ob, wb = call(b, fp32=True)
    torch.cuda.synchronize()
    ra, rb = oa.clone(), ob.clone()
    oa.zero_(), ob.zero_()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        call(a, fp32=True, out=oa, ws=wa, stream=s1)
        call(b, fp32=True, out=ob, ws=wb, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a, fp32=True, out=oa, ws=wa)
        call(b, fp32=True, out=ob, ws=wa)
    a["x"].copy_(b["x"])
    a["w"].copy_(b["w"])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, rb) and torch.equal(ob, rb)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,n,k", [(2047, 2500, 520), (1500, 3001, 584)])
def test_many_tokens_in_wider_rows_in_place(T, n, k, gated, fp32):
    """Many tokens: the residual in place, in rows of a wider tensor; what lies
    beside and behind them stays as it was, and a token or a weight row with
    NaN touches its own row or column only."""
    d = data(T, n, k, 4, gated, bias=True, resid=True, fp32=fp32)
    d["x"][T - 1, 3] = float("nan")
    d["w"][n - 1, 7] = float("nan")
    clean = {a: None if v is None else v.clone() for a, v in d.items()}
    clean["x"][T - 1, 3], clean["w"][n - 1, 7] = 0, 0
    xw = torch.full((T + 2, k + 24), float("nan"), dtype=BF, device="cuda")
    xs = xw[:T, 8:8 + k]
    xs.copy_(d["x"])
    for off in (0, 16, 5):
        o = torch.full((T + 2, n + 28), 77.0, dtype=d["r"].dtype, device="cuda")
        h = o[:T, off:off + n]
        h.copy_(d["r"])
        _, ws = call({**d, "x": xs, "r": h}, "silu", fp32, out=h)
        torch.cuda.synchronize()
        m.check(m.k3moe_device_status(ws), "device status")
        assert torch.isnan(h[T - 1]).all() and torch.isnan(h[:, n - 1]).all()
        ref, tol = linear_ref(clean["x"], clean["w"], clean["wg"], clean["b"], clean["bg"], clean["r"], "silu",
                              24 if fp32 else 8)
        ok = (h.double() - ref).abs() <= tol
        assert ok[:T - 1, :n - 1].all()
        o[:T, off:off + n] = 77.0
        assert (o == 77.0).all()


def test_fp32_precision_of_many_tokens():
    """As above, in tiles of more tokens and in pairs of CTAs."""
    for T, n, k in ((1300, 2560, 4096), (3000, 896, 7168)):
        d = data(T, n, k, T)
        out, _ = call(d, fp32=True)
        ref = d["x"].double() @ d["w"].double().T
        assert float((out.double() - ref).norm() / ref.norm()) <= 1e-6


@pytest.mark.parametrize("fp32", [False, True])
def test_many_tokens_on_two_streams(fp32):
    """Two calls of many tokens at once, a workspace each, between calls of few
    tokens; then captured and replayed."""
    a, b, c = data(2047, 2500, 520, 1), data(1500, 3001, 584, 2), data(5, 896, 2048, 3)
    want = [call(d, fp32=fp32)[0] for d in (a, b, c)]
    torch.cuda.synchronize()
    outs, wss = zip(*[call(d, fp32=fp32) for d in (a, b, c, c)])
    torch.cuda.synchronize()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(8):
        call(a, fp32=fp32, out=outs[0], ws=wss[0], stream=s1)
        call(c, fp32=fp32, out=outs[2], ws=wss[2], stream=s1)
        call(b, fp32=fp32, out=outs[1], ws=wss[1], stream=s2)
        call(c, fp32=fp32, out=outs[3], ws=wss[3], stream=s2)
    torch.cuda.synchronize()
    for o, w in zip(outs, want + [want[2]]):
        assert torch.equal(o, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for d, o in zip((a, b, c), outs):
            call(d, fp32=fp32, out=o, ws=wss[0])
    for o in outs:
        o.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
