"""The workspace of moe_shared_ffn: no more than its calls use, and enough where most of it is in use."""
import pytest

from test_shared_ffn import F32, Case, call, m, needs_lib, note  # noqa: F401


@needs_lib
@pytest.mark.parametrize("R", [8, 64, 256])
def test_bytes_per_token_of_many_tokens(R):
    """Of hundreds of thousands of tokens each more takes three bf16 parts of x, of h and of two projections' low-rank
    results, its place in the plan (8 bytes), and 16 bytes of a work item per 64; partial sums over K are for few tiles."""
    H, I = 64, 32
    a, b = (call(layer=dict(hidden=H, shared_inter=I), pool=dict(n_adapters=2, max_rank=R), T=T, x=None)[2]
            for T in (1 << 19, 1 << 20))
    assert 0 < b - a <= (6 * H + 6 * I + 12 * R + 8 + 0.25) * (1 << 19) + 9 * 256


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4000, 8000, 16300])
def test_partial_sums_stay_in_their_place(m, T):  # noqa: F811
    """Eight, four and two parts of K at the largest numbers of tokens that have them, with guards behind the workspace."""
    note(f"partial sums T={T}")
    c = Case(T, 2048, 64, 1, 16, seed=T)
    c.check(c.run(m, F32))
