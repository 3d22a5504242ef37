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
    """A function from calls (operation, SwiGLU, groups, rows, n_out, n_in, columns to a scale) to their kernels."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("choice") / "choice")
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", exe,
                           os.path.join(ROOT, "tests", "choice_main.cpp")])

    def run(calls):
        text = "".join(" ".join(str(int(v) if isinstance(v, bool) else v) for v in call) + "\n" for call in calls)
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
    (0, 1, 4, 16384, 4096, "few"), (0, 1, 4, 20480, 4096, "16 halves"), (0, 1, 8, 16384, 4096, "few"),
    (0, 1, 8, 24576, 4096, "16 halves"), (0, 1, 16, 16384, 4096, "16 halves"), (0, 1, 16, 12288, 4096, "few"),
    (0, 1, 24, 6144, 4096, "few"), (0, 1, 24, 8192, 4096, "16 halves"), (0, 1, 64, 8192, 4096, "16 halves"),
    (0, 1, 256, 2048, 4096, "16 halves"), (0, 1, 32, 4096, 16384, "few"), (0, 1, 64, 4096, 16384, "16 halves"),
    (0, 1, 32, 4096, 1024, "few"), (0, 1, 128, 4096, 1024, "16"), (0, 1, 64, 8192, 2048, "16 halves"),
    (0, 1, 64, 8192, 1280, "16"), (0, 1, 64, 4096, 1280, "few"), (0, 1, 65, 4096, 1280, "16"),
    (0, 1, 80, 4096, 1536, "16"), (0, 1, 64, 4096, 1664, "few"), (0, 1, 96, 4096, 1664, "16 halves"), (0, 1, 863, 300, 352, "few"),
    (0, 1, 238, 872, 2432, "few"), (0, 1, 420, 872, 2432, "16"),
    (0, 1, 80, 4096, 2048, "16 halves"), (0, 1, 128, 8192, 4096, "16"), (0, 1, 48, 16384, 4096, "16"),
    (0, 1, 24, 24576, 4096, "64 halves"), (0, 1, 24, 32768, 4096, "64 halves"), (0, 1, 33, 24576, 4096, "64 halves"),
    (0, 1, 33, 16384, 4096, "16"), (0, 1, 64, 24576, 4096, "64 halves"), (0, 1, 1024, 2048, 4096, "64 halves"),
    (0, 1, 128, 24576, 4096, "32"), (0, 1, 128, 16384, 1024, "32"), (0, 1, 256, 16384, 4096, "64"),
    (0, 1, 16, 65536, 4096, "16"), (0, 1, 17, 65536, 4096, "64"), (0, 1, 2048, 4096, 4096, "64"),
    (1, 256, 8, 2048, 4096, "16 halves"), (1, 256, 24, 2048, 4096, "16"), (0, 256, 24, 4096, 2048, "16"),
    (0, 256, 4096, 4096, 2048, "32"), (0, 256, 16000, 4096, 2048, "64"), (0, 8, 1024, 2048, 4096, "32"),
    (1, 80, 54, 221, 1216, "few"), (0, 16, 1024, 1024, 1024, "32"), (0, 16, 512, 1024, 1024, "16"),
]

# the same with the columns to a scale
Q4_SCALES = [(0, 1, 80, 4096, 1664, 32, "few"), (0, 1, 80, 4096, 1664, 128, "16 halves"), (0, 1, 1137, 240, 1920, 32, "few"),
             (0, 1, 64, 4096, 1920, 32, "few"), (0, 1, 128, 4096, 1920, 32, "16 halves")]


def test_q4(choose):
    check(choose, [("q4", *c[:5], 64, c[5]) for c in Q4] + [("q4", *c) for c in Q4_SCALES])


# SwiGLU, groups, rows, weight rows (of one half), columns -> kernel
FEW_ROWS = [
    (0, 1, 1, 4096, 4096, "few rows"), (0, 1, 4, 32752, 4096, "few rows"), (0, 1, 4, 32768, 4096, "128x64"),
    (0, 1, 5, 16384, 4096, "128x64"), (0, 1, 16, 12288, 4096, "few rows"), (0, 1, 16, 16384, 4096, "128x64"),
    (0, 1, 17, 4096, 4096, "few rows"), (0, 1, 48, 4096, 4096, "few rows"), (0, 1, 49, 4096, 4096, "128x64"),
    (0, 1, 208, 1024, 4096, "few rows"), (0, 1, 209, 1024, 4096, "128x64"), (0, 1, 32, 8192, 4096, "128x64"),
    (0, 64, 4, 1024, 1024, "few rows"), (0, 16, 32, 1024, 1024, "128x64"), (1, 256, 8, 2048, 4096, "128x64"),
    (0, 8, 8, 2048, 4096, "few rows"), (1, 16, 8, 1024, 1024, "128x64"),
    (1, 8, 2, 2048, 4096, "few rows"), (1, 1, 4, 16384, 4096, "128x64"), (1, 1, 4, 16368, 4096, "few rows"),
    (0, 16, 1200, 520, 1000, "128x64"), (1, 16, 80, 264, 520, "few rows"),
]


def test_few_rows(choose):
    check(choose, [("linear", *c[:5], 0, c[5]) for c in FEW_ROWS])


# SwiGLU, groups, rows, weight rows (of one half), columns -> kernel of the forward product
TILES = [
    (0, 1, 1024, 4096, 4096, "128x64"), (0, 1, 1152, 4096, 4096, "128x64"), (0, 1, 1153, 4096, 4096, "256x128 of 8"),
    (0, 1, 2048, 4096, 4096, "256x128 of 8"), (0, 1, 2049, 4096, 4096, "256x256"), (0, 1, 4096, 4096, 4096, "256x256"),
    (0, 1, 6144, 4096, 4096, "256x128 of 8"), (0, 1, 8192, 4096, 4096, "256x256"), (1, 1, 2048, 2048, 4096, "256x128 of 8"),
    (0, 1, 111, 65536, 4096, "256x128 of 4"), (0, 1, 112, 65536, 4096, "256x128 of 8"), (0, 32, 4096, 2048, 4096, "256x256"),
    (0, 32, 3552, 2048, 4096, "256x128 of 4"), (0, 32, 3584, 2048, 4096, "256x256"), (0, 32, 5120, 1024, 1024, "256x128 of 8"),
    (0, 1, 4096, 4096, 328, "256x256"), (0, 1, 4096, 4096, 320, "256x128 of 4"), (0, 1, 2040, 4096, 256, "256x128 of 4"),
    (0, 32, 8128, 4096, 2048, "256x256"), (0, 32, 8192, 2048, 4096, "256x128 of 8"),
    (1, 256, 16384, 2048, 4096, "256x128 of 4"), (1, 256, 32768, 2048, 4096, "256x256"), (1, 256, 8192, 2048, 4096, "128x64"),
    (1, 32, 93672, 2048, 4096, "256x256"), (0, 16, 1200, 520, 1000, "128x64"), (0, 16, 8192, 520, 1000, "256x128 of 8"),
    (0, 16, 16384, 520, 1000, "256x256"),
]
# groups, rows, n_out, n_in -> kernel of the input's gradient
DGRAD = [
    (1, 1, 4096, 4096, "128x64"), (1, 1024, 4096, 4096, "128x64"), (1, 2048, 4096, 4096, "256x128 of 8"), (1, 4096, 4096, 4096, "256x256"),
    (256, 24, 4096, 2048, "128x64"), (25, 116, 2112, 1728, "128x64"), (220, 6188, 4056, 632, "128x64"), (256, 16, 4096, 2048, "128x64"), (256, 8, 2048, 4096, "128x64"), (256, 16, 2048, 4096, "256x128 of 4"), (256, 32, 4096, 2048, "256x128 of 4"),
    (64, 64, 512, 1024, "128x64"), (64, 64, 1024, 1024, "128x64"), (64, 256, 2048, 1024, "256x128 of 4"), (64, 1024, 512, 1024, "128x64"),
    (32, 1024, 2048, 4096, "256x128 of 4"), (32, 3552, 4096, 2048, "256x128 of 4"), (44, 8448, 144, 320, "128x64"), (32, 4096, 4096, 2048, "256x256"),
    (32, 8192, 4096, 2048, "256x128 of 8"), (32, 8192, 2048, 4096, "256x256"), (32, 16384, 2048, 4096, "256x256"),
    (16, 524, 520, 1000, "128x64"), (16, 4096, 520, 1000, "256x128 of 8"),
]


# groups, rows, n_out, n_in -> kernel of the weights' gradient
WGRAD = [
    (1, 8192, 2048, 2048, "128x128"), (1, 64, 4096, 2048, "128x128"), (1, 64, 4104, 2048, "256x256"), (1, 8192, 2560, 4096, "256x256"),
    (8, 128, 1024, 1024, "128x128"), (9, 128, 1024, 1024, "256x256"), (32, 154, 512, 1000, "256x256"), (4096, 8, 8, 8, "256x256"),
]


def test_weights_gradient(choose):
    check(choose, [("wgrad", 0, *c[:4], 0, c[4]) for c in WGRAD])


def test_tiles(choose):
    check(choose, [("linear", *c[:5], 0, c[5]) for c in TILES])
    check(choose, [("dgrad", 0, *c[:4], 0, c[4]) for c in DGRAD])


def test_the_gpu_tests_reach_their_kernels(choose):
    group = {K: g for K, g, *_ in paths.Q4_COLUMNS}
    check(choose, [("q4", swiglu, 1, T, N // (1 + swiglu), K, group[K], kernel) for kernel, T, N, K in paths.q4_paths() for swiglu in (0, 1)])
    for kernel, forward, (T, k, E, K, P) in paths.BF16_SHAPES:
        rows = T * max(k, 1)
        if forward:
            check(choose, [("linear", 0, E, rows, P, K, 0, kernel), ("linear", 1, E, rows, P // 2, K, 0, kernel)])
        check(choose, [("dgrad", 0, E, rows, K, P, 0, kernel)])
    check(choose, [("wgrad", 0, E, T * max(k, 1), N, K, 0, "256x256") for T, k, E, K, N in paths.WGRAD_256])
    check(choose, [("q4", 0, E, T * max(k, 1), N, K, 32, kernel) for kernel, (T, k, E, K, N) in paths.Q4_EXPERTS])
