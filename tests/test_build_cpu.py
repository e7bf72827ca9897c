"""What the package needs of torch: the compiled Python entry points alone,
which are built for one torch.  Without them, or with ones that do not load, the
package imports, every other call works, and the calls that need them say so."""
import importlib.util
import os
import subprocess
import sys

import pytest

from test_abi_cpu import ROOT, _build

PKG = os.path.join(ROOT, "mxfp4_routed_expert_softmax_b200")


@pytest.fixture(scope="module")
def build():
    _build()
    spec = importlib.util.spec_from_file_location("k3moe_build_again", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


USE = """
import {first}
import mxfp4_routed_expert_softmax_b200 as m
assert m.k3moe_blob_bytes(m.make_dims(128, 64, 16, 4, 64)) > 0
try:
    print("gate", m.k3moe_gate(16, 0, None, m.make_gate(16, 4), 16, 16, 0))
except ImportError as e:
    print("ImportError", e)
"""


def use(root, first):
    r = subprocess.run([sys.executable, "-c", USE.format(first=first)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


@pytest.mark.parametrize("first", ["torch", "os"])  # before the package, or by its first call
@pytest.mark.parametrize("binding", ["there", "missing", "not loadable"])
def test_package_without_the_entry_points(build, tmp_path, first, binding):
    pkg = tmp_path / "mxfp4_routed_expert_softmax_b200"
    pkg.mkdir()
    for f in ("__init__.py", "build.py", "libk3moe.so"):
        os.symlink(os.path.join(PKG, f), pkg / f)
    path = pkg / os.path.basename(build.binding_path())
    if binding == "there":
        os.symlink(build.binding_path(), path)
    elif binding == "not loadable":
        path.write_bytes(b"of another torch")
    out = use(tmp_path, first)
    if binding == "there":
        assert out.startswith("gate 1")
    else:
        assert out.startswith("ImportError") and "build.py" in out and path.name in out


def test_another_torch_is_noticed(build, monkeypatch):
    assert not build.stale()
    monkeypatch.setattr(build, "torch_version", lambda: "0.0.1+other")
    assert build.stale()


def test_library_alone(build, monkeypatch):
    """Without torch, and where only the library is asked for, nothing of
    torch's is compiled."""
    monkeypatch.setattr(build, "_binding_command", lambda: pytest.fail("the entry points were to be built"))
    monkeypatch.setattr(build, "torch_version", lambda: "0.0.1+other")
    assert build.build(library_only=True) == build.LIB
    monkeypatch.setattr(build, "torch_version", lambda: None)
    assert build.binding_path() is None and not build.stale()
    assert build.build() == build.LIB
