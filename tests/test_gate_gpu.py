"""k3moe_gate on the GPU against the plain 64-bit statement of the routing:
picks equal, weights within the bound of operator_refs."""
import numpy as np
import pytest
import torch

from operator_refs import GATE_ATOL, GATE_RTOL, gate_ref

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def desc(E, k, score="softmax", groups=1, kept=1, group_top=1, renorm=False, scale=1.0, bf16=False):
    return m.make_gate(E, k, m.K3MOE_SCORE_SIGMOID if score == "sigmoid" else m.K3MOE_SCORE_SOFTMAX, groups, kept,
                       group_top, scale, (m.K3MOE_RENORM_TOPK if renorm else 0) | (m.K3MOE_LOGITS_BF16 if bf16 else 0))


def run(l, k, bias=None, stream=None, **kw):
    T, E = l.shape
    g = desc(E, k, bf16=l.dtype == torch.bfloat16, **kw)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    m.check(m.k3moe_gate(l, T, bias, g, idx, w, stream), "k3moe_gate")
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def compare(l, k, bias=None, **kw):
    idx, w = run(l, k, bias, **kw)
    ri, rw = gate_ref(l.double().cpu().numpy(), k, bias=None if bias is None else bias.double().cpu().numpy(), **kw)
    bad = np.nonzero((idx != ri).any(1))[0]
    assert bad.size == 0, (bad[:5], idx[bad[:2]], ri[bad[:2]])
    np.testing.assert_allclose(w, rw, rtol=GATE_RTOL, atol=GATE_ATOL)


def logits(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * spread).to(dtype)


def biases(E, seed, std=0.05):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 + seed)
    return torch.randn(E, generator=g, device="cuda") * std


SHAPES = [(1, 1, 1), (3, 2, 1), (1, 8, 2), (5, 8, 8), (2, 31, 31), (7, 32, 32), (4, 33, 32), (9, 64, 6), (1, 896, 16),
          (37, 896, 16), (2, 897, 17), (5, 1000, 1), (3, 1024, 32), (33, 1023, 24), (130, 160, 6), (257, 256, 8),
          (11, 121, 13), (600, 384, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_shapes(T, E, k, score, biased):
    for dtype in (torch.float32, torch.bfloat16):
        compare(logits(T, E, E + k, dtype), k, biases(E, k) if biased else None, score=score, renorm=(E + T) % 2 == 0,
                scale=2.5 if T % 2 else 1.0)


GROUPS = [(256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (160, 6, 8, 3, 1), (896, 16, 7, 3, 2), (896, 16, 8, 1, 2), (64, 3, 32, 2, 2),
          (1020, 32, 17, 9, 2), (1023, 30, 31, 4, 1), (62, 2, 31, 30, 2), (9, 2, 3, 1, 2), (30, 9, 3, 2, 2), (2, 1, 2, 1, 1),
          (1024, 32, 2, 1, 2), (512, 20, 4, 3, 2), (72, 8, 12, 5, 2), (32, 8, 32, 9, 1)]


@pytest.mark.parametrize("E,k,groups,kept,group_top", GROUPS)
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_groups(E, k, groups, kept, group_top, score, biased):
    for T, dtype in ((1, torch.float32), (70, torch.float32), (41, torch.bfloat16)):
        compare(logits(T, E, 3 * E + k, dtype), k, biases(E, k, 0.2) if biased else None, score=score, groups=groups,
                kept=kept, group_top=group_top, renorm=True, scale=2.5)


@pytest.mark.parametrize("groups,kept,group_top", [(1, 1, 1), (8, 3, 2), (8, 5, 1)])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_ties(groups, kept, group_top, score, biased):
    """Equal inputs tie to the lower id: constant rows, rows of few values, and
    more equal values than any list of candidates holds."""
    E, k = 896, 16
    l = logits(64, E, 5)
    l[0] = 0.25
    l[1] = torch.where(torch.arange(E, device="cuda") % 3 == 0, 1.0, -1.0)
    l[2:20] = torch.round(l[2:20])
    l[20:30] = torch.round(l[20:30] * 2) / 2
    l[30, :] = -3.0
    l[30, ::200] = 2.0
    l[31] = torch.arange(E, device="cuda") / E
    l[32] = -torch.arange(E, device="cuda") / E
    l[33:40] = l[33:40].clamp(max=1.0)  # a plateau at the top
    b = torch.round(biases(E, 1, 1.0)) / 4 if biased else None
    compare(l, k, b, score=score, groups=groups, kept=kept, group_top=group_top, renorm=True)
    compare(l, 32, b, score=score, groups=groups, kept=kept, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties(score):
    """Scores closer than fp32 can tell are still ranked as the formula says:
    one-unit steps of the logits, and biases that nearly cancel the scores."""
    E, k = 128, 12
    base = logits(40, E, 9)
    l = torch.nextafter(base[:, :1].expand(-1, E).contiguous(), torch.full((40, E), 100.0, device="cuda"))
    step = torch.randint(0, 4, (40, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    for i in range(1, 4):
        l = torch.where(step >= i, torch.nextafter(l, torch.full_like(l, 100.0)), l)
    compare(l, k, None, score=score)
    compare(l, k, biases(E, 3, 1e-8), score=score)
    row = base[:1].expand(40, E).contiguous()
    z = torch.sigmoid(row[0].double()) if score == "sigmoid" else torch.softmax(row[0].double(), 0)
    compare(row, k, (0.5 - z).float(), score=score, renorm=True)
    # saturated sigmoids: equal in fp32, some still apart in 64 bits, some not
    sat = torch.randint(10, 50, (40, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).float()
    compare(sat, k, None, score=score)
    compare(sat, k, torch.zeros(E, device="cuda"), score=score)


@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("groups,kept,group_top", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_masks(score, biased, groups, kept, group_top):
    """-inf and NaN logits, masks that leave fewer than k experts or none,
    infinite and lowest values, biases of +-inf and NaN."""
    E, k = 64, 8
    inf = float("inf")
    low = torch.finfo(torch.float32).min
    l = logits(24, E, 21)
    l[0] = -inf
    l[1, 1:] = -inf
    l[2, :-3] = -inf
    l[3, ::2] = -inf
    l[4] = low
    l[5, 3:] = low
    l[6, 5] = float("nan")
    l[7, 5] = inf
    l[8, 5], l[8, 6] = inf, inf
    l[9] = float("nan")
    l[10, 10:] = float("nan")
    l[11, 16:] = -inf
    l[12, :48] = -inf
    l[13] = 3.0e38
    l[14, 7] = 88.0
    l[15] = -100.0
    l[16, 1::16] = -inf
    l[16, 2::16] = -inf
    l[17, 17:32] = -inf
    b = None
    if biased:
        b = biases(E, 4, 0.3)
        b[20], b[21], b[40] = -inf, float("nan"), inf
    kw = dict(score=score, groups=groups, kept=kept, group_top=group_top)
    compare(l, k, b, **kw)
    compare(l, k, b, renorm=True, scale=-1.5, **kw)
    lb = l.to(torch.bfloat16)
    compare(lb, k, b, **kw)


def vector_ref(l, k, bias, sigmoid):
    """The picks of many tokens at once, in 64 bits: sorts that keep the order of equal values."""
    l = l.double()
    c = (torch.sigmoid(l) if sigmoid else torch.softmax(l, 1)) + bias.double()
    top, idx = c.sort(dim=1, descending=True, stable=True)
    return torch.where(top[:, :k] > -np.inf, idx[:, :k], -1).to(torch.int32), c


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["spread", "zero", "tiny", "masked", "huge", "coarse", "saturated"])
def test_biased_picks_of_many_tokens(score, kind):
    """Where the biased scores are told apart in 32 bits, where only 64 bits
    do, and where there are more candidates than the list holds."""
    T, E, k = 3000, 896, 16
    l = logits(T, E, 77, torch.bfloat16 if kind in ("zero", "coarse") else torch.float32)
    b = {"spread": biases(E, 3), "zero": torch.zeros(E, device="cuda"), "tiny": biases(E, 3, 1e-7),
         "masked": biases(E, 3), "huge": biases(E, 3, 1e6), "coarse": torch.round(biases(E, 3, 1.0)),
         "saturated": biases(E, 3, 1e-9)}[kind]
    if kind == "masked":
        b[::3] = -float("inf")
    if kind == "coarse":
        l = torch.round(l)
    if kind == "saturated":
        l = l.abs() * 4 + 14
    idx, w = run(l, k, b, score=score)
    ri, c = vector_ref(l, k, b, score == "sigmoid")
    got = torch.as_tensor(idx, device="cuda")
    # torch's exponentials and sums may differ from the definition's in the
    # last bit of 64: a few units of the sum of score and bias
    a = c.gather(1, got.clamp(min=0).long())
    e = c.gather(1, ri.clamp(min=0).long())
    gap = (a - e).abs() > 2.0 ** -48 * (1 + e.abs())
    assert not bool((gap & (got != ri)).any())
    assert float((got != ri).float().mean()) < (1e-3 if kind not in ("saturated", "tiny", "huge") else 2e-2)


def test_small_scores_keep_their_ratios():
    """Scores far below fp32's range, renormalised: the ratios of the formula."""
    E, k = 96, 6
    l = logits(20, E, 3) - 120.0
    compare(l, k, None, score="sigmoid", renorm=True)
    b = torch.where(torch.arange(E, device="cuda") < 20, 5.0, 0.0)  # picks the bias makes, with scores near 0
    l = logits(20, E, 4)
    l[:, :20] -= 150.0
    compare(l, k, b, score="softmax", renorm=True)
    compare(l, k, b, score="sigmoid", renorm=True)
    compare(l, k, b, score="sigmoid")


def test_row_distance_and_rows_behind():
    """Logits as a slice of wider rows; nothing behind the last row is written."""
    T, E, k = 19, 250, 9
    wide = logits(T, 301, 6)
    for off in (0, 1, 7):
        l = wide[:, off:off + E]
        g = desc(E, k, "sigmoid")
        idx = torch.full((T + 3, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T + 3, k), -7.0, device="cuda")
        m.check(m.k3moe_gate(l, T, None, g, idx, w))
        ri, rw = gate_ref(l.double().cpu().numpy(), k, "sigmoid")
        assert np.array_equal(idx[:T].cpu().numpy(), ri)
        np.testing.assert_allclose(w[:T].cpu().numpy(), rw, rtol=GATE_RTOL)
        assert (idx[T:] == -7).all() and (w[T:] == -7).all()
    lb = wide.to(torch.bfloat16)
    for off in (0, 1, 8):
        compare(lb[:, off:off + E], k, score="sigmoid")


def test_offsets_past_32_bits():
    """Rows further apart than 2^31 elements in all."""
    T, E, k = 70, 64, 4
    wide = torch.empty((T, 1 << 25), dtype=torch.bfloat16, device="cuda")
    l = wide[:, 12345 * 8:12345 * 8 + E]
    l.copy_(logits(T, E, 8))
    compare(l, k, score="softmax")


def test_many_tokens_and_repeats():
    """More tokens than any one wave of warps, twice: equal bits; a sample
    against the reference."""
    T, E, k = 70001, 96, 5
    l = logits(T, E, 31)
    a, b = run(l, k, None, score="softmax", renorm=True), run(l, k, None, score="softmax", renorm=True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    pick = np.r_[0:50, T - 50:T]
    ri, rw = gate_ref(l[torch.from_numpy(pick).cuda()].double().cpu().numpy(), k, renorm=True)
    assert np.array_equal(a[0][pick], ri)
    np.testing.assert_allclose(a[1][pick], rw, rtol=GATE_RTOL)


def test_streams_and_graph():
    """On a stream of its own, two calls at once, and captured and replayed
    with new inputs."""
    E, k, T = 896, 16, 33
    la, lb = logits(T, E, 41), logits(T, E, 42)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    g = desc(E, k)
    out = [(torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        m.check(m.k3moe_gate(la, T, None, g, *out[0], stream=s1))
        m.check(m.k3moe_gate(lb, T, None, g, *out[1], stream=s2))
    torch.cuda.synchronize()
    for l, (i, w) in ((la, out[0]), (lb, out[1])):
        ri, _ = gate_ref(l.double().cpu().numpy(), k)
        assert np.array_equal(i.cpu().numpy(), ri)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.check(m.k3moe_gate(la, T, None, g, *out[0]))
    la.copy_(lb)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
