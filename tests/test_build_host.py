"""The build on the host, with the compilers replaced: the library does not depend on the binding's extension."""
import os

import pytest

from gated_deltanet_gdn_gb300 import binding
from gated_deltanet_gdn_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Empty build folders, and a _run that writes each command's output file; `broken` fails on the extension."""
    state = {"broken": False, "ran": []}
    for name in ("BUILD_DIR", "LIB_PATH", "EXT_PATH"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))

    def run(what, cmd, verbose):
        state["ran"].append(what)
        if state["broken"] and any("binding_ext" in c for c in cmd):
            raise RuntimeError("Python.h: No such file or directory")
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc_path", lambda: "nvcc")
    return state


def test_the_library_is_built_when_the_extension_is_not(tree):
    tree["broken"] = True
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.EXT_PATH)
    assert not b.lib_is_stale() and b.ext_is_stale()
    tree["ran"].clear()
    assert b.build_lib() == b.LIB_PATH and not tree["ran"]
    tree["broken"] = False
    b.build()  # the extension alone
    assert os.path.exists(b.EXT_PATH) and not b.is_stale()
    assert all("extension" in w or "binding_ext" in w for w in tree["ran"])


def test_the_rule_loads_without_the_extension(monkeypatch):
    def broken():
        raise RuntimeError("Python.h: No such file or directory")

    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_ext", None)
    monkeypatch.setattr(b, "ext_is_stale", lambda: True)
    monkeypatch.setattr(b, "build_ext", broken)
    assert binding.gdn_version() == 100
    with pytest.raises(RuntimeError, match="Python.h"):
        binding.gdn_block_norm_fwd(None)


def test_another_pytorch_or_python_makes_the_extension_stale(tree, monkeypatch):
    """The extension is compiled against their binary interfaces."""
    import sys

    import torch

    b.build()
    assert not b.ext_is_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + ".other")
        assert b.ext_is_stale() and not b.lib_is_stale()
        b.build()
        assert not b.ext_is_stale()
    assert b.ext_is_stale()
    b.build()
    with monkeypatch.context() as m:
        m.setattr(sys, "version", "3.99 " + sys.version)
        assert b.ext_is_stale()
    assert not b.is_stale()
