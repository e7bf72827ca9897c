"""What the Python calls of k3moe_gate, k3moe_linear and k3moe_layer_routed
refuse of tensors in the device's memory: each call with one defect returns
K3MOE_ERR_INVALID_ARGUMENT before anything is launched, and the same call
without it is carried out."""
import pytest
import torch

pytestmark = pytest.mark.gpu
m = pytest.importorskip("mxfp4_routed_expert_softmax_b200") if torch.cuda.is_available() else None
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def zeros(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def strided(t):
    """The same shape in rows twice as far apart."""
    return torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype, device=t.device)[:, :t.shape[1]]


def columns(t):
    """The same shape with elements that do not follow one another."""
    return torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype, device=t.device).T


T, E, K = 5, 64, 4


def gate_args(bf16=False):
    return {"logits": zeros(T, E, dtype=BF if bf16 else F32), "T": T, "bias": zeros(E, dtype=F32),
            "gate": m.make_gate(E, K, flags=m.K3MOE_LOGITS_BF16 if bf16 else 0), "idx": zeros(T, K, dtype=I32),
            "weight": zeros(T, K, dtype=F32)}


def gate(**a):
    return m.k3moe_gate(*(a[x] for x in ("logits", "T", "bias", "gate", "idx", "weight")))


GATE = {
    "T past the logits": lambda a: {"logits": a["logits"][:T - 1]},
    "one row for many tokens": lambda a: {"logits": a["logits"][0]},
    "T past the picks": lambda a: {"idx": a["idx"][:T - 1]},
    "T past the weights": lambda a: {"weight": a["weight"][:T - 1]},
    "T past all": lambda a: {"T": T + 1},
    "narrow logits": lambda a: {"logits": a["logits"][:, :E - 1]},
    "wide logits": lambda a: {"logits": zeros(T, E + 1, dtype=a["logits"].dtype)},
    "logits by columns": lambda a: {"logits": columns(a["logits"])},
    "overlapping logits": lambda a: {"logits": a["logits"][0].expand(T, E)},
    "fp16 logits": lambda a: {"logits": a["logits"].half()},
    "fp64 logits": lambda a: {"logits": a["logits"].double()},
    "integer picks as logits": lambda a: {"logits": zeros(T, E, dtype=I32)},
    "short bias": lambda a: {"bias": a["bias"][:E - 1]},
    "strided bias": lambda a: {"bias": zeros(2 * E, dtype=F32)[::2]},
    "bf16 bias": lambda a: {"bias": a["bias"].to(BF)},
    "integer bias": lambda a: {"bias": a["bias"].to(I32)},
    "fp32 picks": lambda a: {"idx": a["idx"].float()},
    "64-bit picks": lambda a: {"idx": a["idx"].long()},
    "integer weights": lambda a: {"weight": a["weight"].to(I32)},
    "strided weights": lambda a: {"weight": strided(a["weight"])},
    "strided picks": lambda a: {"idx": strided(a["idx"])},
    "host logits": lambda a: {"logits": a["logits"].cpu()},
}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("defect", list(GATE))
def test_gate(defect, bf16):
    a = gate_args(bf16)
    assert gate(**{**a, **GATE[defect](a)}) == m.K3MOE_ERR_INVALID_ARGUMENT
    m.check(gate(**a))
    torch.cuda.synchronize()


def test_gate_takes_larger_and_sliced_tensors():
    a = gate_args()
    m.check(gate(**{**a, "logits": zeros(T + 3, E + 5, dtype=F32)[:, 1:1 + E], "bias": zeros(E + 1, dtype=F32),
                    "idx": zeros(T + 2, K, dtype=I32), "weight": zeros((T + 2) * K, dtype=F32)}))
    m.check(gate(**{**gate_args(True), "logits": zeros(T, E, dtype=torch.int16)}))  # the bits of bf16
    torch.cuda.synchronize()


N, D = 48, 64


def linear_args(fp32=False):
    return {"x": zeros(T, D), "T": T, "w": zeros(N, D), "wg": zeros(N, D), "b": zeros(N, dtype=F32),
            "bg": zeros(N, dtype=F32), "r": zeros(T, N, dtype=F32 if fp32 else BF),
            "lin": m.make_linear(N, D, m.K3MOE_ACT_SILU, m.K3MOE_OUT_FP32 if fp32 else 0),
            "out": zeros(T, N, dtype=F32 if fp32 else BF), "ws": zeros(1 << 16, dtype=torch.uint8), "ws_bytes": None}


def linear(**a):
    return m.k3moe_linear(*(a[x] for x in ("x", "T", "w", "wg", "b", "bg", "r", "lin", "out", "ws", "ws_bytes")))


LINEAR = {
    "T past x": lambda a: {"x": a["x"][:T - 1]},
    "one row for many tokens": lambda a: {"x": a["x"][0]},
    "T past the residual": lambda a: {"r": a["r"][:T - 1]},
    "T past the output": lambda a: {"out": a["out"][:T - 1]},
    "T past all": lambda a: {"T": T + 1},
    "few rows of w": lambda a: {"w": a["w"][:N - 1]},
    "few rows of w_gate": lambda a: {"wg": a["wg"][:N - 1]},
    "one row of w": lambda a: {"w": a["w"][0]},
    "narrow x": lambda a: {"x": a["x"][:, :D - 8]},
    "wide w": lambda a: {"w": zeros(N, D + 8)},
    "narrow output": lambda a: {"out": a["out"][:, :N - 1]},
    "wide residual": lambda a: {"r": zeros(T, N + 1, dtype=a["r"].dtype)},
    "x by columns": lambda a: {"x": columns(a["x"])},
    "w by columns": lambda a: {"w": columns(a["w"])},
    "output by columns": lambda a: {"out": columns(a["out"])},
    "overlapping output": lambda a: {"out": a["out"][0].expand(T, N)},
    "w and w_gate of unlike rows": lambda a: {"wg": strided(a["wg"])},
    "three dimensions": lambda a: {"x": a["x"][None]},
    "fp16 x": lambda a: {"x": a["x"].half()},
    "fp32 x": lambda a: {"x": a["x"].float()},
    "fp16 w": lambda a: {"w": a["w"].half()},
    "fp16 w_gate": lambda a: {"wg": a["wg"].half()},
    "an output of another type": lambda a: {"out": a["out"].to(BF if a["out"].dtype == F32 else F32)},
    "an fp16 output": lambda a: {"out": a["out"].half()},
    "an integer output": lambda a: {"out": a["out"].to(I32)},
    "a residual of another type": lambda a: {"r": a["r"].to(BF if a["r"].dtype == F32 else F32)},
    "an fp16 residual": lambda a: {"r": a["r"].half()},
    "short bias": lambda a: {"b": a["b"][:N - 1]},
    "short gate bias": lambda a: {"bg": a["bg"][:N - 1]},
    "bf16 bias": lambda a: {"b": a["b"].to(BF)},
    "integer gate bias": lambda a: {"bg": a["bg"].to(I32)},
    "strided bias": lambda a: {"b": zeros(2 * N, dtype=F32)[::2]},
    "strided workspace": lambda a: {"ws": zeros(1 << 17, dtype=torch.uint8)[::2]},
    "more workspace than there is": lambda a: {"ws_bytes": (1 << 16) + 1},
    "host x": lambda a: {"x": a["x"].cpu()},
}


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("defect", list(LINEAR))
def test_linear(defect, fp32):
    a = linear_args(fp32)
    assert linear(**{**a, **LINEAR[defect](a)}) == m.K3MOE_ERR_INVALID_ARGUMENT
    m.check(linear(**a))
    torch.cuda.synchronize()


def test_linear_takes_larger_and_sliced_tensors():
    a = linear_args()
    m.check(linear(**{**a, "x": zeros(T + 3, D + 16)[:, 8:8 + D], "w": zeros(N + 2, D + 8)[:, :D],
                      "wg": zeros(N, D + 8)[:, :D], "b": zeros(N + 1, dtype=F32), "r": zeros(T + 1, N + 3)[:, 2:2 + N],
                      "out": zeros(T + 1, N + 3)[:, 2:2 + N]}))
    m.check(linear(**{**a, "T": 1, "x": zeros(D), "out": zeros(N), "r": None}))
    m.check(linear(**{**a, "x": zeros(T, D, dtype=torch.int16), "w": zeros(N, D, dtype=torch.int16)}))
    torch.cuda.synchronize()


H, FF, NE, FS = 128, 64, 16, 64


def routed_args(fp32=False, T=T):
    dims = m.make_dims(H, FF, NE, K, FS, m.K3MOE_OUT_FP32 if fp32 else 0)
    blobs = torch.zeros(NE, m.k3moe_blob_bytes(dims), dtype=torch.uint8, device="cuda")
    return {"x": zeros(T, H), "T": T, "idx": zeros(T, K, dtype=I32), "weight": zeros(T, K, dtype=F32),
            "blobs": torch.tensor([b.data_ptr() for b in blobs], dtype=torch.int64, device="cuda"), "_keep": blobs,
            "sg": zeros(FS, H), "su": zeros(FS, H), "sd": zeros(H, FS), "dims": dims,
            "y": zeros(T, H, dtype=F32 if fp32 else BF), "ws": m.new_workspace(dims, T), "ws_bytes": None}


def routed(**a):
    return m.k3moe_layer_routed(*(a[x] for x in ("x", "T", "idx", "weight", "blobs", "sg", "su", "sd", "dims", "y",
                                                 "ws", "ws_bytes")))


ROUTED = {
    "T past x": lambda a: {"x": a["x"][:-1]},
    "T past the picks": lambda a: {"idx": a["idx"][:-1]},
    "T past the weights": lambda a: {"weight": a["weight"][:-1]},
    "T past the output": lambda a: {"y": a["y"][:-1]},
    "T past all": lambda a: {"T": a["T"] + 1},
    "x in wider rows": lambda a: {"x": strided(a["x"])},
    "output in wider rows": lambda a: {"y": strided(a["y"])},
    "x by columns": lambda a: {"x": columns(a["x"])},
    "strided picks": lambda a: {"idx": strided(a["idx"])},
    "strided weights": lambda a: {"weight": strided(a["weight"])},
    "shared gate in wider rows": lambda a: {"sg": strided(a["sg"])},
    "shared up in wider rows": lambda a: {"su": strided(a["su"])},
    "shared down transposed": lambda a: {"sd": columns(a["sd"])},
    "short shared gate": lambda a: {"sg": a["sg"][:-1]},
    "short shared up": lambda a: {"su": a["su"][:-1]},
    "short shared down": lambda a: {"sd": a["sd"][:-1]},
    "short pointer table": lambda a: {"blobs": a["blobs"][:-1]},
    "32-bit pointer table": lambda a: {"blobs": a["blobs"].to(I32)},
    "strided pointer table": lambda a: {"blobs": a["blobs"].repeat_interleave(2)[::2]},
    "fp16 x": lambda a: {"x": a["x"].half()},
    "fp32 x": lambda a: {"x": a["x"].float()},
    "fp32 picks": lambda a: {"idx": a["idx"].float()},
    "64-bit picks": lambda a: {"idx": a["idx"].long()},
    "integer weights": lambda a: {"weight": a["weight"].to(I32)},
    "fp16 shared matrix": lambda a: {"su": a["su"].half()},
    "an output of another type": lambda a: {"y": a["y"].to(BF if a["y"].dtype == F32 else F32)},
    "an fp16 output": lambda a: {"y": a["y"].half()},
    "strided workspace": lambda a: {"ws": torch.zeros(2 * a["ws"].numel(), dtype=torch.uint8, device="cuda")[::2]},
    "more workspace than there is": lambda a: {"ws_bytes": a["ws"].numel() + 1},
    "host x": lambda a: {"x": a["x"].cpu()},
}


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("defect", list(ROUTED))
def test_layer_routed(defect, fp32):
    a = routed_args(fp32)
    assert routed(**{**a, **ROUTED[defect](a)}) == m.K3MOE_ERR_INVALID_ARGUMENT
    m.check(routed(**a))
    torch.cuda.synchronize()
    assert m.k3moe_device_status(a["ws"]) == m.K3MOE_OK


def test_layer_routed_takes_larger_and_flat_tensors():
    a = routed_args()
    m.check(routed(**{**a, "x": zeros(T + 3, H), "idx": zeros((T + 1) * K, dtype=I32), "y": zeros(T, 1, H),
                      "blobs": a["blobs"].repeat(2), "sg": zeros(FS * H, dtype=torch.int16)}))
    b = {**a, "dims": m.make_dims(H, FF, NE, K, FS, m.K3MOE_NO_SHARED), "sg": None, "su": None, "sd": None}
    m.check(routed(**b))
    torch.cuda.synchronize()
    assert m.k3moe_device_status(a["ws"]) == m.K3MOE_OK
