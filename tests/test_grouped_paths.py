"""The grouped products where a call's sizes choose another kernel, and the values at the edges of their numerics.

Tolerances are those of test_grouped.py (its docstring derives them)."""
import os

import pytest
import torch

from test_grouped import BF16, F32, LIB, Case, note, run_wgrad


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import bit_quantized_moe_permute_amd as m
    return m


# ----------------------------------------------------------------------------
# adding to gradients
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("E,K,N", [(9, 136, 264), (300, 136, 264)], ids=["few tiles", "many tiles"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_accumulate_leaves_groups_without_rows_as_they_were(m, dtype, E, K, N):
    """Bit for bit, whatever is there: negative zeros (which adding a sum of nothing would make positive), NaNs of any payload."""
    c = Case(20, 2, E, K, N, seed=51, some=3, tail=5)
    empty = [e for e in range(E) if not c.counts[e]]
    assert empty and len(empty) < E
    bits = torch.int32 if dtype == F32 else torch.int16
    info = torch.iinfo(bits)
    dw = torch.randint(info.min, info.max, (E, N, K), generator=torch.Generator().manual_seed(52), dtype=bits)
    dw[:, ::2, ::3] = info.min                                      # -0
    gpu = dw.cuda().view(dtype)
    note(f"accumulate into empty groups {dtype} {E}")
    m.moe_grouped_wgrad(c.groups(m), c.x.cuda(), c.dy.cuda(), gpu, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(gpu.cpu().view(bits)[empty], dw[empty])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(300, 0, 1, 4104, 4104), (90, 2, 300, 264, 136), (40, 3, 12, 200, 136)],
                         ids=lambda s: "x".join(map(str, s)))
def test_accumulate(m, shape, dtype):
    """On the tiles of 256 x 256 (289 of one matrix, 600 of small ones) and of 128 x 128."""
    run_wgrad(m, Case(*shape, seed=53, dst="slots" if shape[1] else "sorted"), dtype, f"accumulate {shape}", accumulate=True)
