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


def test_a_bounds_site_names_one_check():
    """The checking build reports a number: it stands for one place in the sources."""
    sites = {}
    for name in sorted(os.listdir(build.CSRC)):
        src = open(os.path.join(build.CSRC, name)).read()
        at = src.find("SDPA_IN_BOUNDS(")
        while at >= 0:
            end, depth = at + len("SDPA_IN_BOUNDS("), 1
            while depth:
                depth += {"(": 1, ")": -1}.get(src[end], 0)
                end += 1
            last = src[at:end - 1].rsplit(",", 1)[1].strip()
            if last.isdigit():                            # not the macro itself
                sites.setdefault(int(last), []).append((name, src.count("\n", 0, at) + 1))
            at = src.find("SDPA_IN_BOUNDS(", end)
    assert len(sites) > 20 and all(len(v) == 1 for v in sites.values()), {k: v for k, v in sites.items() if len(v) > 1}
