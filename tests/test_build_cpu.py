"""The build of the compiled marshalling module (csrc/torch_calls.cpp): which file the binding takes, and when."""
import os
import shutil
import sysconfig
import types

import pytest

from moe_router_gemm_gb300 import _binding, build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The package's folders with copies of the module's inputs, and a compiler that writes a file of its own."""
    for name, files in (("CSRC", ["torch_calls.cpp"]), ("INCLUDE", ["bf16_linear.h"])):
        d = tmp_path / name
        d.mkdir()
        for f in files:
            shutil.copy(os.path.join(getattr(build, name), f), d)
        monkeypatch.setattr(build, name, str(d))
    (tmp_path / "pkg").mkdir()
    monkeypatch.setattr(build, "PKG", str(tmp_path / "pkg"))
    compiler = types.SimpleNamespace(fails=False, runs=0)

    def run(cmd, **kw):
        compiler.runs += 1
        if not compiler.fails:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("module")
        return types.SimpleNamespace(returncode=int(compiler.fails), stdout="", stderr="no header")

    monkeypatch.setattr(build.subprocess, "run", run)
    return tmp_path, compiler


def _module(tree):
    """The file that the binding would load, or None."""
    return build.calls_path() if os.path.exists(build.calls_path()) else None


@pytest.mark.parametrize("changed", ["INCLUDE/bf16_linear.h", "CSRC/torch_calls.cpp"])
def test_a_module_of_other_sources_is_not_loaded(tree, changed):
    root, compiler = tree
    first = build.build_calls()
    assert first is not None and _module(tree) == first and compiler.runs == 1
    assert build.build_calls() == first and compiler.runs == 1  # nothing changed
    with open(root / changed, "a") as f:
        f.write("\n/* another argument order */\n")
    assert _module(tree) is None
    compiler.fails = True
    assert build.build_calls() is None and compiler.runs == 2
    assert _module(tree) is None  # calls go through ctypes, as the build has said
    compiler.fails = False
    second = build.build_calls()
    assert second != first and _module(tree) == second
    assert os.listdir(root / "pkg") == [os.path.basename(second)]  # the older one is gone


def test_a_module_belongs_to_one_python(tree, monkeypatch):
    here = build.build_calls()
    tag = sysconfig.get_config_var("SOABI")
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-" + tag if name == "SOABI" else None)
    assert _module(tree) is None
    assert build.build_calls() != here and os.path.exists(here)


def test_forcing_builds_again(tree):
    _, compiler = tree
    path = build.build_calls()
    assert build.build_calls(force=True) == path and compiler.runs == 2


def test_the_binding_loads_what_the_build_names(tree):
    assert _binding._load_calls(None) is None  # nothing was built here


def test_what_the_module_build_raises_is_raised(tree, monkeypatch):
    """Only what build_calls itself handles turns into calls through ctypes."""
    root, compiler = tree
    monkeypatch.setattr(build, "LIB", str(root / "pkg" / "lib.so"))
    monkeypatch.setattr(build, "BUILD", str(root / "objects"))
    monkeypatch.setattr(build, "up_to_date", lambda: False)

    def broken(force=False):
        raise ValueError("a mistake in build_calls")

    monkeypatch.setattr(build, "build_calls", broken)
    with pytest.raises(ValueError, match="a mistake"):
        build.build()
    monkeypatch.setattr(build, "build_calls", lambda force=False: None)
    assert build.build() == build.LIB
