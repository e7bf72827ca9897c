"""Refusals of k3moe_gate, k3moe_linear and k3moe_layer_routed (every argument
is checked before anything is launched, so no GPU is needed), and the plain
statement of the routing on cases worked by hand."""
import ctypes

import numpy as np
import pytest

from operator_refs import gate_ref
from test_abi_cpu import A16, BIG, _build


@pytest.fixture(scope="module")
def m():
    _build()
    import mxfp4_routed_expert_softmax_b200 as m
    return m


INVALID, SHAPE, WORKSPACE = 1, 2, 3


@pytest.mark.parametrize("args,want", [
    ((0, 1), SHAPE), ((1025, 1), SHAPE), ((8, 0), INVALID), ((8, 9), INVALID), ((64, 33), INVALID),
    ((64, 4, 2), INVALID), ((64, 4, -1), INVALID), ((64, 4, 0, 0), SHAPE), ((64, 4, 0, 33), SHAPE),
    ((64, 4, 0, 7), SHAPE), ((64, 4, 0, 8, 0), INVALID), ((64, 4, 0, 8, 9), INVALID), ((64, 9, 0, 8, 1), INVALID),
    ((64, 4, 0, 8, 2, 0), INVALID), ((64, 4, 0, 8, 2, 3), INVALID), ((8, 4, 0, 8, 4, 2), INVALID),
    ((64, 4, 0, 1, 1, 1, float("nan")), INVALID), ((64, 4, 0, 1, 1, 1, float("inf")), INVALID),
    ((64, 4, 0, 1, 1, 1, 1.0, 1), INVALID), ((64, 4, 0, 1, 1, 1, 1.0, 256), INVALID)])
def test_gate_rejects_bad_descriptors(m, args, want):
    g = m.make_gate(*args)
    assert m.lib.k3moe_gate(A16, 0, 1, None, ctypes.byref(g), A16, A16, None) == want


def test_gate_rejects_bad_arguments(m):
    g = m.make_gate(64, 4)

    def call(l=A16, ld=0, T=1, bias=None, desc=g, idx=A16, w=A16):
        return m.lib.k3moe_gate(l, ld, T, bias, ctypes.byref(desc) if desc else None, idx, w, None)

    assert call(l=None) == call(T=0) == call(T=-1) == call(ld=63) == call(ld=-1) == INVALID
    assert call(l=A16 + 2) == call(bias=A16 + 2) == call(idx=None) == call(w=None) == INVALID
    assert call(idx=A16 + 1) == call(w=A16 + 3) == call(desc=None) == INVALID
    b = m.make_gate(64, 4, flags=m.K3MOE_LOGITS_BF16)
    assert call(l=A16 + 1, desc=b) == INVALID


@pytest.mark.parametrize("args,want", [
    ((0, 64), SHAPE), ((-5, 64), SHAPE), ((64, 0), SHAPE), ((64, 4), SHAPE), ((64, 12), SHAPE),
    ((1 << 25, 64), SHAPE), ((64, 1 << 25), SHAPE), ((64, 64, 5), INVALID), ((64, 64, -1), INVALID),
    ((64, 64, 0, 2), INVALID), ((64, 64, 0, 64), INVALID)])
def test_linear_rejects_bad_descriptors(m, args, want):
    d = m.make_linear(*args)
    assert m.k3moe_linear_workspace_size(d, 1) == 0
    assert m.lib.k3moe_linear(A16, 0, 1, A16, None, 0, None, None, None, 0, ctypes.byref(d), A16, 0, A16, BIG,
                              None) == want


def test_linear_rejects_bad_arguments(m):
    d, f = m.make_linear(100, 64), m.make_linear(100, 64, 0, m.K3MOE_OUT_FP32)

    def call(x=A16, ldx=0, T=1, w=A16, wg=None, ldw=0, b=None, bg=None, r=None, ldr=0, lin=d, out=2 * A16, ldo=0,
             ws=A16 * 16, wsb=BIG):
        return m.lib.k3moe_linear(x, ldx, T, w, wg, ldw, b, bg, r, ldr, ctypes.byref(lin) if lin else None, out, ldo,
                                  ws, wsb, None)

    for bad in (dict(x=None), dict(x=A16 + 8), dict(T=0), dict(w=None), dict(w=A16 + 8), dict(wg=A16 + 2),
                dict(ldx=56), dict(ldx=68), dict(ldw=60), dict(ldw=65), dict(ldr=99), dict(ldo=99), dict(ldo=-1),
                dict(b=A16 + 2), dict(bg=A16), dict(wg=A16, bg=A16 + 1), dict(r=A16 + 1), dict(out=None),
                dict(out=A16 + 1), dict(lin=f, out=A16 + 2), dict(lin=f, r=A16 + 2), dict(r=2 * A16, ldr=104),
                dict(lin=None), dict(ws=None), dict(ws=A16 + 16)):
        assert call(**bad) == INVALID, bad
    assert call(wsb=16) == WORKSPACE
    assert call(wsb=m.k3moe_linear_workspace_size(d, 1) - 1) == WORKSPACE
    assert call(T=(1 << 30) + 1) == SHAPE


def test_linear_workspace_covers_every_smaller_call(m):
    """A workspace for T tokens serves every smaller T."""
    for n, k in ((896, 7168), (7168, 1536), (100, 64), (1, 8)):
        d = m.make_linear(n, k)
        sizes = [m.k3moe_linear_workspace_size(d, t) for t in (1, 2, 8, 9, 16, 33, 64, 200, 256, 257, 4096, 10 ** 6)]
        assert sizes == sorted(sizes) and sizes[0] >= 256
        assert m.k3moe_linear_workspace_size(d, 0) == 0


def test_binding_rejects_wrong_tensors(m):
    """The Python calls refuse tensors whose type or layout the pointers cannot carry."""
    import torch
    g = m.make_gate(64, 4)
    i, w = torch.empty(2, 4, dtype=torch.int32), torch.empty(2, 4)
    l = torch.empty(2, 64)
    assert m.k3moe_gate(l.to(torch.bfloat16), 2, None, g, i, w, 0) == INVALID
    assert m.k3moe_gate(torch.empty(64, 2).T, 2, None, g, i, w, 0) == INVALID
    assert m.k3moe_gate(torch.empty(2, 63), 2, None, g, i, w, 0) == INVALID
    assert m.k3moe_gate(l, 2, None, g, i.long(), w, 0) == INVALID
    assert m.k3moe_gate(l, 2, None, g, i, torch.empty(4, 2).T, 0) == INVALID
    d = m.make_linear(64, 64)
    x, wt = torch.empty(2, 64, dtype=torch.bfloat16), torch.empty(64, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for bad in (dict(x=x.float()), dict(w=wt.T), dict(out=x.float()), dict(b=torch.empty(64, dtype=torch.bfloat16)),
                dict(x=x[:, :56]), dict(wg=torch.empty(64, 128, dtype=torch.bfloat16)[:, :64])):
        a = {"x": x, "w": wt, "wg": None, "b": None, "out": x.clone(), **bad}
        assert m.k3moe_linear(a["x"], 2, a["w"], a["wg"], a["b"], None, None, d, a["out"], ws, stream=0) == INVALID
    assert m.k3moe_layer_routed(x, 2, i.long(), w, A16, None, None, None, m.make_dims(64, 64, 4, 4, 0), x, ws,
                                stream=0) == INVALID


def test_binding_rejects_host_tensors(m):
    """Right in type and layout, but not in the device's memory."""
    import torch
    bf = torch.bfloat16
    i, w = torch.empty(2, 4, dtype=torch.int32), torch.empty(2, 4)
    assert m.k3moe_gate(torch.empty(2, 64), 2, None, m.make_gate(64, 4), i, w, 0) == INVALID
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    x = torch.empty(2, 64, dtype=bf)
    assert m.k3moe_linear(x, 2, torch.empty(64, 64, dtype=bf), None, None, None, None, m.make_linear(64, 64), x.clone(), ws,
                          stream=0) == INVALID
    assert m.k3moe_layer_routed(x, 2, i, w, A16, None, None, None, m.make_dims(64, 64, 4, 4, 0), x, ws,
                                stream=0) == INVALID


def test_binding_argument_errors(m):
    """What is not an address, a descriptor or a number raises; addresses go
    to the library, which refuses these before any launch."""
    g, d = m.make_gate(64, 4), m.make_linear(64, 64)
    for bad in (("x", 1, None, g, A16, A16, 0), (A16, "1", None, g, A16, A16, 0), (A16, 1, None, d, A16, A16, 0),
                (A16, 1, None, 5, A16, A16, 0), (A16, 1, None, g, 1.5, A16, 0), (A16, 1, None, g, A16, A16, "s")):
        with pytest.raises((TypeError, AttributeError)):
            m.k3moe_gate(*bad)
    with pytest.raises(OverflowError):
        m.k3moe_gate(A16, 1 << 31, None, g, A16, A16, 0)
    with pytest.raises(TypeError):  # a workspace given as an address needs its size
        m.k3moe_linear(A16, 1, A16, None, None, None, None, d, A16, A16 * 16, stream=0)
    assert m.k3moe_linear(A16, 0, A16, None, None, None, None, d, 2 * A16, A16 * 16, BIG, 0) == INVALID
    assert m.k3moe_linear(A16, 1, A16, None, None, None, None, d, 2 * A16, A16 * 16, 16, 0) == WORKSPACE
    assert m.k3moe_gate(A16 + 2, 1, None, g, A16, A16, 0) == INVALID

    class Stream:
        cuda_stream = 0
    assert m.k3moe_gate(A16, 0, None, g, A16, A16, Stream()) == INVALID


def test_layer_routed_rejects_bad_arguments(m):
    dims = m.make_dims(256, 128, 32, 4, 128)

    def call(x=A16, T=4, idx=A16, w=A16, blobs=A16, sg=A16, d=dims, y=A16, ws=A16 * 16, wsb=BIG):
        return m.lib.k3moe_layer_routed(x, T, idx, w, blobs, sg, sg, sg, ctypes.byref(d), y, ws, wsb, None)

    for bad in (dict(idx=None), dict(idx=A16 + 2), dict(w=None), dict(w=A16 + 1), dict(x=None), dict(x=A16 + 2),
                dict(T=0), dict(blobs=None), dict(sg=None), dict(y=None), dict(ws=None), dict(ws=A16 + 16)):
        assert call(**bad) == INVALID, bad
    assert call(wsb=16) == WORKSPACE
    assert call(d=m.make_dims(100, 128, 32, 4, 128)) == SHAPE


def test_routing_worked_by_hand():
    """Logits 0, ln 2, ln 4, ln 8: softmax 1/15, 2/15, 4/15, 8/15; sigmoid 1/2, 2/3, 4/5, 8/9."""
    l = np.log([[1.0, 2.0, 4.0, 8.0]])
    i, w = gate_ref(l, 2)
    assert i.tolist() == [[3, 2]] and np.allclose(w, [[8 / 15, 4 / 15]])
    i, w = gate_ref(l, 2, renorm=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]])
    i, w = gate_ref(l, 2, "sigmoid", renorm=True)
    assert np.allclose(w, [[(8 / 9) / (8 / 9 + 4 / 5), (4 / 5) / (8 / 9 + 4 / 5)]])
    # the bias moves the picks, not the weights: 1/2 + 1 > 8/9
    i, w = gate_ref(l, 2, "sigmoid", bias=[1.0, 0, 0, 0])
    assert i.tolist() == [[0, 3]] and np.allclose(w, [[1 / 2, 8 / 9]])
    # two groups: 1/2 + 2/3 < 4/5 + 8/9; by one value with a bias: 1/2 + 1 > 8/9
    assert gate_ref(l, 2, "sigmoid", groups=2, kept=1, group_top=2)[0].tolist() == [[3, 2]]
    assert gate_ref(l, 2, "sigmoid", bias=[1.0, 0, 0, 0], groups=2, kept=1)[0].tolist() == [[0, 1]]
    # masks, ties, nothing left
    assert gate_ref(np.array([[0.0, -np.inf, 0.0, 0.0]]), 4)[0].tolist() == [[0, 2, 3, -1]]
    i, w = gate_ref(np.full((1, 4), -np.inf), 2, renorm=True)
    assert i.tolist() == [[-1, -1]] and (w == 0).all()
