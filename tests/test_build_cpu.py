"""The build of the library and of the native part of the Python binding."""
import os
import subprocess
import sys

import pytest

from scaled_dot_product_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def broken_binding(tmp_path, monkeypatch):
    """A binding that does not compile, in the place of one from an earlier build."""
    build.build()
    (tmp_path / "binding.cpp").write_text("#include <no_such_header.h>\n")
    (tmp_path / "_binding.so").write_bytes(b"older")
    os.utime(tmp_path / "_binding.so", (1, 1))
    monkeypatch.setattr(build, "BINDING_SRC", str(tmp_path / "binding.cpp"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    return tmp_path


def test_the_library_is_built_without_the_binding(broken_binding, capfd):
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "no_such_header" in capfd.readouterr().err
    assert not (broken_binding / "_binding.so").exists()          # no binding rather than an older one


def test_building_the_binding_alone_fails_loudly(broken_binding):
    with pytest.raises(RuntimeError, match="no_such_header"):
        build.build_binding()


def test_the_library_is_built_without_torch():
    code = "import sys; sys.modules['torch'] = None; from scaled_dot_product_gb300 import build as b; " \
           "b.BINDING += '.none'; print(b.build())"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == build.LIB, r.stderr[-2000:]
    assert "torch" in r.stderr
