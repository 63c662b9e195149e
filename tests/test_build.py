"""What the build makes anew, with compilers that only write their output (CPU only)."""
import os
import shutil
import types

import pytest

from attention_forward_blackwell_gb300 import build as real


class Tools:
    """Stands in for subprocess.run: notes what is made, fails where told to."""

    def __init__(self):
        self.made, self.fail, self.clock = [], None, 2_000_000_000

    def stamp(self, path):
        self.clock += 10
        os.utime(path, (self.clock, self.clock))

    def run(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        if self.fail == name:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="told to fail")
        self.made.append(name)
        with open(out, "w") as f:
            f.write(f"{len(self.made)}")
        self.stamp(out)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build over a copy of the sources, and its tools."""
    pkg, inc = tmp_path / "pkg", tmp_path / "include"
    shutil.copytree(real.CSRC, pkg / "csrc")
    shutil.copytree(real.INCLUDE, inc)
    tools = Tools()
    for name, path in (("HERE", pkg), ("CSRC", pkg / "csrc"), ("INCLUDE", inc), ("OBJDIR", pkg / "_build"),
                       ("LIB_PATH", pkg / "libfa_gb300.so"),
                       ("BIND_PATH", pkg / os.path.basename(real.BIND_PATH))):
        monkeypatch.setattr(real, name, str(path))
    monkeypatch.setattr(real.subprocess, "run", tools.run)
    return types.SimpleNamespace(build=real.build, tools=tools, header=str(inc / "fa.h"),
                                 lib=os.path.basename(real.LIB_PATH), bind=os.path.basename(real.BIND_PATH),
                                 bind_path=real.BIND_PATH, bind_obj=str(pkg / "_build" / "bind.o"))


def made(tree, **kw):
    tree.tools.made.clear()
    tree.build(**kw)
    return list(tree.tools.made)


def test_nothing_is_made_twice(tree):
    first = made(tree)
    assert tree.lib in first and tree.bind in first and "bind.o" in first
    assert made(tree) == []


@pytest.mark.parametrize("failing", ["span.o", "libfa_gb300.so", "bind"])
def test_a_build_that_failed_leaves_no_stale_module(tree, failing):
    """The header changed (an argument more, say) and the build did not come to
    its end: the module of the old header is not left beside the new library, and
    the next build makes it anew."""
    made(tree)
    tree.tools.stamp(tree.header)
    tree.tools.fail = tree.bind if failing == "bind" else failing
    with pytest.raises(RuntimeError):
        made(tree)
    if tree.lib in tree.tools.made:
        assert not os.path.exists(tree.bind_path)
    tree.tools.fail = None
    again = made(tree)
    assert tree.bind in again
    assert os.path.getmtime(tree.bind_path) >= os.path.getmtime(tree.bind_obj)
    assert made(tree) == []


def test_the_module_is_of_one_python(tree, monkeypatch):
    """A CPython extension: another interpreter neither finds it nor keeps it."""
    import sysconfig
    assert real.BIND_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    made(tree)
    of = sysconfig.get_config_var
    monkeypatch.setattr(real.sysconfig, "get_config_var",
                        lambda name: "cpython-399-other" if name == "SOABI" else of(name))
    assert tree.bind in made(tree)
    assert made(tree) == []


def test_the_library_needs_no_torch(tree, monkeypatch):
    """Users of the C ABI build the library without torch; with it, the module follows."""
    with monkeypatch.context() as m:
        m.setattr(real.importlib.util, "find_spec", lambda name: None)
        first = made(tree)
        assert tree.lib in first and "bind.o" not in first and tree.bind not in first
        assert made(tree) == []
    assert tree.bind in made(tree)
