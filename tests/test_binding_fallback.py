"""The short way from Python to the smallest calls is for speed alone: the library
builds, loads and refuses as ever where it cannot be built or loaded (no GPU needed)."""
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
import bit_vq_routed_gb300 as bv  # noqa: E402
from bit_vq_routed_gb300 import build  # noqa: E402

QUICK = ("_quick_norm", "_quick_rows", "_quick_linear_8bit", "_quick_route_scored")


@pytest.fixture
def binding(tmp_path, monkeypatch):
    """A place of its own for the binding, and none loaded."""
    bv.load()
    p = str(tmp_path / "moe_binding.so")
    monkeypatch.setattr(build, "binding_path", lambda: p)
    monkeypatch.setattr(bv, "_lib", None)
    for n in QUICK:
        monkeypatch.setattr(bv, n, bv._look_again)
    return p


def _works():
    assert all(getattr(bv, n) is bv._look_again for n in QUICK)
    bf = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bv.moe_rms_norm(bf, None, 1e-6, y=bf)
    assert bv.moe_linear_8bit_workspace_size(1, 16, 16) > 0


def test_the_name_tells_python_and_torch(monkeypatch):
    p = build.binding_path()
    assert torch.__version__ in p and os.path.dirname(p) == build.PKG
    monkeypatch.setattr(torch, "__version__", "99.0.0")
    assert build.binding_path() != p and not os.path.exists(build.binding_path()) and not build.binding_settled()


@pytest.mark.parametrize("how", ["no compiler", "no headers"])
def test_a_binding_that_cannot_be_built(binding, monkeypatch, how):
    def run(cmd, **kw):
        assert cmd[0] == "g++"
        if how == "no compiler":
            raise FileNotFoundError("g++")
        return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")

    monkeypatch.setattr(subprocess, "run", run)
    open(binding, "w").close()
    os.utime(binding, (1, 1))  # (of older sources)
    assert not build.binding_settled()
    with pytest.warns(RuntimeWarning, match="ctypes"):
        bv.load()
    assert not os.path.exists(binding) and build.binding_settled()
    _works()
    # and it is not tried again at each start
    monkeypatch.setattr(subprocess, "run", None)
    monkeypatch.setattr(bv, "_lib", None)
    bv.load()
    _works()


def test_a_binding_that_does_not_load(binding):
    with open(binding, "w") as f:
        f.write("of another machine")
    with pytest.warns(RuntimeWarning, match="does not load"):
        bv.load()
    _works()


def test_it_is_built_again(binding):
    open(binding + ".failed", "w").close()
    assert build.binding_settled()
    assert build.build_binding()
    assert os.path.exists(binding) and not os.path.exists(binding + ".failed") and build.binding_settled()
    bv.load()
    assert all(getattr(bv, n) is not bv._look_again for n in QUICK)
