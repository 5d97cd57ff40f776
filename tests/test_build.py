"""The build of the C library needs nothing but nvcc: where torch is missing, the Python extension is left out and said to be."""
import os
import subprocess
import sys

import kimi_delta_attention_21_b200.build as build

# the build as a file, in a process that has no torch; everything but the extension is up to date
SCRIPT = """
import importlib.util, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("kda_build", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.MARSHAL = sys.argv[2]
if len(sys.argv) > 3:
    b.shutil.which = lambda name: None
    del sys.modules["torch"]
print(b.build())
"""


def run(tmp_path, *more):
    so = tmp_path / "_marshal.so"
    r = subprocess.run([sys.executable, "-c", SCRIPT, build.__file__, str(so), *more], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == build.LIB and os.path.exists(build.LIB)
    assert not so.exists()
    return r.stderr


def test_the_library_builds_without_torch(tmp_path):
    assert "_marshal.so was not built: torch is missing" in run(tmp_path)


def test_the_library_builds_without_a_compiler_for_the_extension(tmp_path):
    assert "_marshal.so was not built: g++ is missing" in run(tmp_path, "no-compiler")


def test_a_failed_compilation_of_the_extension_is_an_error(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))  # kda.h is not there
    try:
        build.build_marshal()
    except RuntimeError as e:
        assert "g++ failed" in str(e) and "kda.h" in str(e)
    else:
        raise AssertionError("built without kda.h")
