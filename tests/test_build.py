"""The build: what a compiler says about the sources (CPU only)."""
import concurrent.futures as cf
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "bit_quantized_moe_permute_amd")


@pytest.fixture
def script(tmp_path):
    """build.py by path (the package would load the library), writing its objects into a folder of the test."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PACKAGE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    if not os.path.exists(b.HIPCC):
        pytest.skip("no hipcc")
    b.BUILD = str(tmp_path)
    return b


def test_the_sources_have_no_warnings(script):
    """Every source, host and device side."""
    flags = [f for f in script.FLAGS if f not in ("-Xclang", "-target-feature", "-packed-fp32-ops")]    # (the host side warns of it)

    def check(src):
        cmd = [script.HIPCC, *(["-x", "hip"] if src.endswith(".cpp") else []), *flags, "-Wno-unused-command-line-argument", "-fsyntax-only", "-I",
               os.path.join(ROOT, "include"), os.path.join(script.CSRC, src)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return r.returncode, r.stderr
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        for src, (rc, err) in zip(script.SOURCES, ex.map(check, script.SOURCES)):
            assert rc == 0 and not err.strip(), f"{src}:\n{err}"


@pytest.mark.parametrize("text,said", [
    ("int chosen(int n) { if (n > 3) return 1; }\n", "return-type"),
    ("struct __attribute__((packed)) Any { uint4 v; };\n__device__ uint4 get(const void *p) { return ((const Any *)p)->v; }\n",
     "packed-non-pod")])
def test_the_build_stops_at(script, tmp_path, text, said):
    """What has led to a fault, or would: a missing return, a packed struct that keeps its alignment."""
    script.CSRC = str(tmp_path)
    (tmp_path / "wrong.hip").write_text("#include <hip/hip_runtime.h>\n" + text)
    with pytest.raises(RuntimeError, match=said):
        script._compile("wrong.hip")


def test_the_build_shows_warnings(script, tmp_path, capfd):
    script.CSRC = str(tmp_path)
    (tmp_path / "odd.hip").write_text("#include <hip/hip_runtime.h>\nint f(int n) { int unused = n; return n; }\n")
    script._compile("odd.hip")
    assert "unused variable" in capfd.readouterr().err
    (tmp_path / "good.hip").write_text("#include <hip/hip_runtime.h>\nint f(int n) { return n; }\n")
    script._compile("good.hip")
    assert not capfd.readouterr().err
