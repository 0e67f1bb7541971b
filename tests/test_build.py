"""The build of the C library and of the Python extension, with a stand-in for
the compilers: which of them run, and what is there afterwards."""
import os
import sys

import pytest

from routed_moe_decode_router_gb300 import build as B


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """B.build() in a folder of its own; the commands that it ran, by program."""
    ran = []

    def run(cmd, what):
        ran.append(os.path.basename(cmd[0]))
        if run.refuses == ran[-1]:
            raise RuntimeError("%s failed" % what)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return ""
    run.refuses = None
    run.ran = ran
    for name in ("LIB", "BINDING", "BUILT_FOR"):
        if hasattr(B, name):
            monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "_run", run)
    return run


def test_library_without_pytorch(tools, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch raises
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert not os.path.exists(B.BINDING) and set(tools.ran) == {"nvcc"}
    del tools.ran[:]
    B.build()
    assert tools.ran == []


def test_library_without_python_headers(tools, tmp_path, monkeypatch):
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_library_is_there_when_the_extension_fails(tools):
    tools.refuses = "g++"
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_extension_is_built_again_for_another_pytorch(tools, monkeypatch):
    import torch
    B.build()
    assert os.path.exists(B.BINDING)
    del tools.ran[:]
    B.build()
    assert tools.ran == []
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    B.build()
    assert tools.ran == ["g++", "g++"]


def test_extension_of_another_pytorch_is_not_loaded(tools, monkeypatch):
    import torch
    from routed_moe_decode_router_gb300 import native, ops
    B.build()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    monkeypatch.setattr(ops, "_ext", None)
    monkeypatch.setattr(native, "lib", lambda: None)
    with pytest.raises(RuntimeError, match="9.9.9.*build it again"):
        ops.rms_norm(torch.zeros(1, 8), torch.zeros(8))
