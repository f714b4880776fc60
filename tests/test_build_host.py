"""What the build makes, without a GPU."""
import os
import re
import shutil
import subprocess
import sys

import pytest

from self_attention_gb300.build import LIB_PATH, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _dynamic(path):
    return subprocess.run(["readelf", "-d", path], capture_output=True, text=True, check=True).stdout


def test_the_library_needs_no_toolkit(tmp_path):
    """libattn_gb300.so carries its CUDA runtime and no path of the machine it was built on: a copy loads by
    itself in a process without PyTorch and without library paths."""
    text = _dynamic(LIB_PATH)
    needed = re.findall(r"\(NEEDED\).*\[(.*)\]", text)
    assert needed and not [n for n in needed if n.startswith(("libcuda", "libtorch", "libc10", "libpython"))], needed
    assert not re.search(r"\((RPATH|RUNPATH)\)", text), text
    copy = shutil.copy(LIB_PATH, tmp_path)
    code = (f"import ctypes, sys; lib = ctypes.CDLL({str(copy)!r}); f = lib.attn_linear_bwd_workspace_size; "
            "f.restype = ctypes.c_size_t; assert f(16, 64, 32, 2) > 0; assert 'torch' not in sys.modules")
    env = {k: v for k, v in os.environ.items() if k not in ("LD_LIBRARY_PATH", "LD_PRELOAD")}
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, cwd=tmp_path)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build of one small source into an empty folder."""
    import self_attention_gb300.build as b
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / b.LIB_NAME))
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "attn_binding.so"))
    monkeypatch.setattr(b, "SOURCES", ["vector_add.cu"])
    return b


def test_a_binding_that_does_not_compile_leaves_the_library(elsewhere, monkeypatch):
    def fail(*_):
        raise RuntimeError("no compiler for the binding")

    monkeypatch.setattr(elsewhere, "_compile_binding", fail)
    with pytest.raises(RuntimeError, match="no compiler for the binding"):
        elsewhere.build()
    assert os.path.exists(elsewhere.LIB_PATH) and not os.path.exists(elsewhere.BINDING_PATH)
    with pytest.raises(RuntimeError):       # and it is still an error the next time
        elsewhere.build()
    assert elsewhere.build_library() == elsewhere.LIB_PATH


def test_a_binding_for_another_pytorch_is_built_again(elsewhere, monkeypatch):
    """Its C++ interface differs from version to version, whatever the files' times say."""
    built = []
    monkeypatch.setattr(elsewhere, "_compile_binding", lambda *_: built.append("compiled") or "object")
    monkeypatch.setattr(elsewhere, "_run", lambda *_: open(elsewhere.BINDING_PATH + f".{os.getpid()}.tmp", "w").close())
    monkeypatch.setattr(elsewhere.os, "remove", lambda path: None)
    elsewhere.build()
    elsewhere.build()
    assert built == ["compiled"]
    torch_dir = elsewhere._torch_dir()
    other = os.path.join(elsewhere.BUILD_DIR, "torch")
    os.makedirs(other)
    with open(os.path.join(torch_dir, "version.py")) as f, open(os.path.join(other, "version.py"), "w") as g:
        g.write(f.read().replace("__version__ = '", "__version__ = '9"))
    monkeypatch.setattr(elsewhere, "_torch_dir", lambda: other)
    elsewhere.build()
    elsewhere.build()
    assert built == ["compiled"] * 2
