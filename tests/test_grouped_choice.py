"""Which kernel a call of the grouped products takes (csrc/choice.h), on the CPU: both sides of every border, and that the shapes of
the GPU tests reach the kernels they are named after."""
import os
import shutil
import subprocess

import pytest

import test_grouped_paths as paths

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_moe_permute_amd", "csrc")


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """A function from calls (operation, SwiGLU, groups, rows, n_out, n_in) to their kernels."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("choice") / "choice")
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", exe,
                           os.path.join(ROOT, "tests", "choice_main.cpp")])

    def run(calls):
        text = "".join(f"{op} {int(swiglu)} {n} {rows} {n_out} {n_in}\n" for op, swiglu, n, rows, n_out, n_in in calls)
        return subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    return run


def check(choose, expected):
    calls, want = [e[:-1] for e in expected], [e[-1] for e in expected]
    got = choose(calls)
    assert len(got) == len(want)
    for call, g, w in zip(calls, got, want):
        assert g == w, (call, g, w)


# SwiGLU, groups, rows, weight rows (of one half), columns -> kernel
Q4 = [
    (0, 1, 1, 4096, 4096, "few"), (0, 1, 1, 20480, 4096, "few"), (0, 1, 1, 24576, 4096, "16 halves"),
    (0, 1, 4, 20480, 4096, "few"), (0, 1, 5, 20480, 4096, "16 halves"), (0, 1, 8, 16384, 4096, "few"),
    (0, 1, 8, 24576, 4096, "16 halves"), (0, 1, 9, 16384, 4096, "16 halves"), (0, 1, 16, 12288, 4096, "few"),
    (0, 1, 24, 6144, 4096, "few"), (0, 1, 24, 8192, 4096, "16 halves"), (0, 1, 64, 8192, 4096, "16 halves"),
    (0, 1, 256, 2048, 4096, "16 halves"), (0, 1, 32, 4096, 16384, "few"), (0, 1, 64, 4096, 16384, "16 halves"),
    (0, 1, 32, 4096, 1024, "few"), (0, 1, 128, 4096, 1024, "16"), (0, 1, 64, 8192, 2048, "16 halves"),
    (0, 1, 64, 8192, 1280, "16"), (0, 1, 64, 4096, 1280, "few"), (0, 1, 65, 4096, 1280, "16"), (0, 1, 128, 8192, 4096, "16"), (0, 1, 48, 16384, 4096, "16"),
    (0, 1, 24, 24576, 4096, "64 halves"), (0, 1, 24, 32768, 4096, "64 halves"), (0, 1, 33, 24576, 4096, "64 halves"),
    (0, 1, 33, 16384, 4096, "16"), (0, 1, 64, 24576, 4096, "64 halves"), (0, 1, 1024, 2048, 4096, "64 halves"),
    (0, 1, 128, 24576, 4096, "32"), (0, 1, 128, 16384, 1024, "32"), (0, 1, 256, 16384, 4096, "64"),
    (0, 1, 16, 65536, 4096, "16"), (0, 1, 17, 65536, 4096, "64"), (0, 1, 2048, 4096, 4096, "64"),
    (1, 256, 8, 2048, 4096, "16 halves"), (1, 256, 24, 2048, 4096, "16"), (0, 256, 24, 4096, 2048, "16"),
    (0, 256, 4096, 4096, 2048, "32"), (0, 256, 16000, 4096, 2048, "64"), (0, 8, 1024, 2048, 4096, "32"),
    (0, 16, 1024, 1024, 1024, "32"), (0, 16, 512, 1024, 1024, "16"),
]


def test_q4(choose):
    check(choose, [("q4", *c) for c in Q4])


# SwiGLU, groups, rows, weight rows (of one half), columns -> kernel
FEW_ROWS = [
    (0, 1, 1, 4096, 4096, "few rows"), (0, 1, 4, 32752, 4096, "few rows"), (0, 1, 4, 32768, 4096, "tiles"),
    (0, 1, 5, 16384, 4096, "tiles"), (0, 1, 16, 12288, 4096, "few rows"), (0, 1, 16, 16384, 4096, "tiles"),
    (0, 1, 17, 4096, 4096, "few rows"), (0, 1, 48, 4096, 4096, "few rows"), (0, 1, 49, 4096, 4096, "tiles"),
    (0, 1, 192, 1024, 4096, "few rows"), (0, 1, 193, 1024, 4096, "tiles"), (0, 1, 32, 8192, 4096, "tiles"),
    (0, 64, 4, 1024, 1024, "few rows"), (0, 16, 32, 1024, 1024, "tiles"), (1, 256, 8, 2048, 4096, "tiles"),
    (1, 8, 2, 2048, 4096, "few rows"), (1, 1, 4, 16384, 4096, "tiles"), (1, 1, 4, 16368, 4096, "few rows"),
    (0, 16, 1200, 520, 1000, "tiles"), (1, 16, 80, 264, 520, "few rows"),
]


def test_few_rows(choose):
    check(choose, [("linear", *c) for c in FEW_ROWS])


def test_the_gpu_tests_reach_their_kernels(choose):
    check(choose, [("q4", swiglu, 1, T, N // (1 + swiglu), K, kernel) for kernel, T, N, K in paths.q4_paths() for swiglu in (0, 1)])
    check(choose, [("q4", 0, E, T * max(k, 1), N, K, kernel) for kernel, (T, k, E, K, N) in paths.Q4_EXPERTS])
