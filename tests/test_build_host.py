"""What build() makes, and when: with a compiler that only records what it was asked for, in a folder of its own."""
import os
import subprocess
import sys

import pytest

from mlp_latency_gb300 import _lib

NVCC = """#!{python}
import os, sys
out = sys.argv[sys.argv.index("-o") + 1]
open({log!r}, "a").write(os.path.basename(out).split(".tmp")[0] + "\\n")
if "marshal.cpp" in " ".join(sys.argv) and os.path.exists({broken!r}):
    open(out, "w").write("half a file")
    sys.exit(1)
open(out, "w").write("x")
"""


class Tree:
    def __init__(self, path):
        self.path, self.log, self.broken = path, str(path / "log"), str(path / "broken")

    def asked(self):
        """What the compiler was asked for since the last time: True for the library, the names of other modules."""
        text = open(self.log).read() if os.path.exists(self.log) else ""
        open(self.log, "w").close()
        return sorted(n for n in text.split() if not n.endswith(".o"))

    def made(self):
        return sorted(f for f in os.listdir(self.path / "pkg"))


@pytest.fixture
def tree(tmp_path, monkeypatch):
    t = Tree(tmp_path)
    (tmp_path / "pkg").mkdir()
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC.format(python=sys.executable, log=t.log, broken=t.broken))
    nvcc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setattr(_lib, "PKG", str(tmp_path / "pkg"))
    monkeypatch.setattr(_lib, "LIB_PATH", str(tmp_path / "pkg" / "libmlp_chain.so"))
    return t


def torch_version(monkeypatch, tmp_path, version):
    """A torch of this version, or none."""
    import importlib.util
    found = importlib.util.find_spec

    class Spec:
        submodule_search_locations = [str(tmp_path / f"torch{version}")]

    if version:
        os.makedirs(Spec.submodule_search_locations[0], exist_ok=True)
        open(os.path.join(Spec.submodule_search_locations[0], "version.py"), "w").write(f"__version__ = '{version}'\n")
    monkeypatch.setattr(_lib.importlib.util, "find_spec", lambda n: (Spec if version else None) if n == "torch" else found(n))


def test_the_library_needs_no_torch(tree, monkeypatch):
    torch_version(monkeypatch, tree.path, None)
    _lib.build()
    assert tree.made() == ["libmlp_chain.so"] and tree.asked() == ["libmlp_chain.so"]
    _lib.build()
    assert tree.asked() == []


def test_another_torch_gets_checks_of_its_own(tree, monkeypatch):
    torch_version(monkeypatch, tree.path, "1.0")
    _lib.build()
    first = tree.made()
    assert len(first) == 2 and tree.asked() == first
    _lib.build()
    assert tree.asked() == []
    torch_version(monkeypatch, tree.path, "1.1")
    _lib.build()
    assert len(tree.made()) == 2 and tree.made() != first and len(tree.asked()) == 1


def test_checks_that_do_not_compile_leave_the_library(tree, monkeypatch):
    torch_version(monkeypatch, tree.path, "1.0")
    open(tree.broken, "w").close()
    with pytest.raises(subprocess.CalledProcessError):
        _lib.build()
    assert tree.made() == ["libmlp_chain.so"]
    os.remove(tree.broken)
    tree.asked()
    _lib.build()
    assert len(tree.made()) == 2 and len(tree.asked()) == 1
