"""What the build compiles again, and for whom."""
import os
import subprocess
import sys
import types

import pytest
import torch

from mixture_experts_ffn_token_b200 import abi
from mixture_experts_ffn_token_b200 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A built tree of its own, with compilers that only note what they are asked for."""
    calls = []

    def run(cmd, check):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(b, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    b.build()
    assert len(calls) == len(b.sources()) + 2 and b.up_to_date()
    calls.clear()
    return calls


def outputs(calls):
    return {os.path.basename(c[c.index("-o") + 1]).split(".")[0] for c in calls}


def test_nothing_to_do(tree):
    b.build()
    assert not tree


@pytest.mark.parametrize("change", ["torch", "python"])
def test_binding_of_another_torch_or_python_is_built_again(tree, monkeypatch, change):
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "2.99.0")
    else:
        monkeypatch.setattr(sys, "version_info", (3, 99, 0, "final", 0))
    assert not b.up_to_date()
    b.build()
    assert outputs(tree) == {"_binding"} and b.up_to_date()
    tree.clear()
    b.build()
    assert not tree


def test_a_change_of_the_binding_compiles_no_kernel(tree, tmp_path):
    os.utime(b.BINDING, (1, 1))
    b.build()
    assert outputs(tree) == {"_binding"}


def test_a_change_of_a_kernel_keeps_the_binding(tree):
    os.utime(b.LIB, (1, 1))
    b.build()
    assert "_binding" not in outputs(tree) and len(tree) == len(b.sources()) + 1


def test_forced(tree):
    b.build(force=True)
    assert len(tree) == len(b.sources()) + 2


def test_the_c_library_needs_no_torch(tree, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch raises ImportError
    assert b.build(force=True) == b.LIB
    assert "_binding" not in outputs(tree) and len(tree) == len(b.sources()) + 1
    assert "torch" in capsys.readouterr().err
    tree.clear()
    b.build()
    assert not tree                                     # the library is not built again


def test_the_build_script_runs_without_torch():
    code = "import sys; sys.modules['torch'] = None; import runpy; print(len(runpy.run_path(sys.argv[1])['sources']()))"
    out = subprocess.run([sys.executable, "-c", code, b.__file__], capture_output=True, text=True)
    assert out.returncode == 0 and int(out.stdout) == len(b.sources()), out.stderr


def test_binding_of_another_torch_is_not_loaded(monkeypatch):
    b.build()
    abi.load_binding()
    monkeypatch.setattr(abi, "_binding", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.99.0")
        with pytest.raises(OSError, match="build it"):
            abi.load_binding()
    abi.load_binding()
