"""What the build gives where the Python binding cannot be built, on a small tree of sources."""
import os

import pytest

from progressive_kv_quantization_gb300 import build as B

KERNEL = 'extern "C" __global__ void k() {}\nextern "C" int answer() { return 42; }\n'
GOOD = 'extern "C" int answer();\nextern "C" int twice() { return 2 * answer(); }\n'
BAD = '#include "a header that is nowhere.h"\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc, out = tmp_path / "csrc", tmp_path / "_build"
    csrc.mkdir()
    (csrc / "k.cu").write_text(KERNEL)
    (csrc / "binding.cpp").write_text(GOOD)
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "SOURCES", ["k.cu"])
    monkeypatch.setattr(B, "BUILD", str(out))
    monkeypatch.setattr(B, "LIB", str(out / "liblynx.so"))
    monkeypatch.setattr(B, "BINDING", str(out / "lynx_binding.so"))
    return csrc


def test_the_library_does_not_need_the_binding(tree):
    """No torch headers, another compiler: the C library is there all the same, and stays
    up to date; a binding of before does not stay behind."""
    B.build()
    assert os.path.exists(B.LIB) and os.path.exists(B.BINDING)
    (tree / "binding.cpp").write_text(BAD)
    (tree / "k.cu").write_text(KERNEL.replace("42", "43"))
    os.remove(B.LIB)
    with pytest.warns(UserWarning, match="nowhere"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING) and B.up_to_date()
    (tree / "binding.cpp").write_text(GOOD)
    made = os.path.getmtime(B.LIB)
    B.build()
    assert os.path.exists(B.BINDING) and os.path.getmtime(B.LIB) == made     # only what was missing is built


def test_no_compiler_for_the_binding(tree, monkeypatch, tmp_path):
    import subprocess
    run = subprocess.run

    def without_gxx(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError(2, "No such file or directory: 'g++'")
        return run(cmd, **kw)
    monkeypatch.setattr(subprocess, "run", without_gxx)
    with pytest.warns(UserWarning, match="g\\+\\+"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_the_binding_follows_torch(tree, monkeypatch):
    """A binding that was built against another torch or Python is built again."""
    B.build()
    first = os.stat(B.BINDING).st_mtime_ns
    B.build()
    assert os.stat(B.BINDING).st_mtime_ns == first
    of = B._binding_of()
    monkeypatch.setattr(B, "_binding_of", lambda: of + " another")
    B.build()
    assert os.stat(B.BINDING).st_mtime_ns > first
