"""The incremental build's decisions: what is compiled and linked when torch is missing, has
changed, or a step before was cut off. Nothing is compiled here: the commands are recorded
and their outputs written as empty files."""
import importlib.util
import os
import subprocess
import sys
import types

import pytest

from stream_decomposition_abft_gb300 import _build


class Tree:
    """A copy's paths under tmp_path, and a torch of a version of one's choice."""

    def __init__(self, tmp_path, monkeypatch):
        self.tmp, self.torch, self.ran, self.fail = tmp_path, None, [], None
        for name, value in (("BUILD", tmp_path / "_build"), ("LIB", tmp_path / "libskgemm.so"),
                            ("BINDING", tmp_path / "_skg_torch.so")):
            monkeypatch.setattr(_build, name, str(value))
        monkeypatch.setattr(_build, "_nvcc", lambda: "nvcc")
        monkeypatch.setattr(_build.subprocess, "run", self._run)
        find = importlib.util.find_spec
        monkeypatch.setattr(_build.importlib.util, "find_spec",
                            lambda name, *a: self._spec() if name == "torch" else find(name, *a))

    def install(self, version):
        """A torch of this version, in a folder of its own; None: no torch."""
        self.torch = version and str(self.tmp / f"torch-{version}")
        if version:
            os.makedirs(self.torch, exist_ok=True)
            with open(os.path.join(self.torch, "version.py"), "w") as f:
                f.write(f"__version__ = '{version}'\n")

    def _spec(self):
        return self.torch and types.SimpleNamespace(
            origin=os.path.join(self.torch, "__init__.py"))

    def _run(self, cmd, **kw):
        self.ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        if self.fail and self.fail in out:
            return subprocess.CompletedProcess(cmd, 1, "", "cut off")
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def build(self, **kw):
        """(sources compiled, names linked) of one build()."""
        self.ran = []
        assert _build.build(**kw) == _build.LIB
        done = [os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in self.ran]
        return [d for d in done if d.endswith(".o")], [d for d in done if not d.endswith(".o")]


@pytest.fixture
def tree(tmp_path, monkeypatch):
    return Tree(tmp_path, monkeypatch)


LIB, BINDING = "libskgemm.so", "_skg_torch.so"


def test_without_torch(tree):
    # The library needs no torch: all of it is built, and nothing of the binding.
    compiled, linked = tree.build()
    assert len(compiled) >= 8 and not any("torch" in c for c in compiled)
    assert linked == [LIB] and not os.path.exists(_build.BINDING)
    assert tree.build() == ([], [])
    # With torch there later, the binding alone is added.
    tree.install("2.9.1")
    compiled, linked = tree.build()
    assert len(compiled) == 1 and "torch" in compiled[0] and linked == [BINDING]
    assert tree.build() == ([], [])


@pytest.mark.parametrize("hide", ["import sys; sys.modules['torch'] = None",
                                  "import importlib.util as u; f = u.find_spec; "
                                  "u.find_spec = lambda n, *a: None if n == 'torch' else f(n, *a)"])
def test_entry_without_torch(hide):
    # The build entry point with torch hidden, on the tree as it is built here.
    _build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", hide + "; import __graft_entry__ as g; g.build()"],
                         cwd=root, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]


def test_torch_changed_and_back(tree):
    # The binding is linked from the object that fits the torch at hand, also when that
    # object was there from before.
    tree.install("2.9.1")
    assert tree.build()[1] == [LIB, BINDING]
    for version, compiled in (("2.11.0", 1), ("2.9.1", 0), ("2.11.0", 0)):
        tree.install(version)
        got = tree.build()
        assert (len(got[0]), got[1]) == (compiled, [BINDING]), version
        link = tree.ran[-1]
        name = "skg_torch_" + "".join(c if c.isalnum() else "_" for c in
                                      f"__version__ = '{version}'\n") + ".o"
        assert any(os.path.basename(a) == name for a in link)
        assert any(tree.torch in a for a in link)  # the libraries of that torch
        assert tree.build() == ([], [])


@pytest.mark.parametrize("step", [LIB, BINDING])
def test_link_cut_off(tree, step):
    # A build that ended between compiling and linking is taken up there.
    tree.install("2.9.1")
    tree.build()
    tree.fail = step
    with pytest.raises(RuntimeError):
        tree.build(force=True)
    tree.fail = None
    assert tree.build() == ([], [LIB, BINDING] if step == LIB else [BINDING])
    assert tree.build() == ([], [])
