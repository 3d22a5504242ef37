"""moe_shared_ffn: the bits that the header promises (24 beside an fp32 result, 16 beside a bf16 one), on every tile.

Measure: the 2-norm of the error over all outputs of a call over that of the root sums of squares of the outputs' terms
(those of W'd h), so that single outputs' deviations average out.

fp32 out.  A chain of n additions of independent terms, whose partial sums grow as the square root of their number, each
rounded by at most 2^-24 of the sum (uniformly: 2^-24 / sqrt(3)): a variance of sum_j j 2^-48 / 3 = n^2 2^-48 / 6 over terms
of n.  A product of K takes up to three parts per value: n = 3 K additions over the K terms' variance, sqrt(K / 2) 2^-24.
Gate and up (K = H, an adapter's A x likewise, B s another R) enter h with a factor of at most 1.1 each; silu's exponential,
sum, quotient and product add at most 10 roundings, their variance 10^2 / 3 < 36; down has K = I, and R.  Together
sqrt(1.21 (H + R) + (I + R) / 2 + 36) 2^-24 = ARITH; the parts themselves leave nothing.

bf16 out.  Two bf16 parts leave at most 2^-16 of a value (uniformly 2^-16 / sqrt(3)): of h and of down's low-rank results once,
of x and of gate's and up's low-rank results with 1.1 each for gate and up, variances 1 + 1 + 2 * 1.21 + 2 * 1.21 < 7.  The result is
rounded once.  What a rounding is off by differs between two values by at most their distance, so
|error| <= |rounding of the exact result| + 2 * (sqrt(7 / 3) 2^-16 + ARITH).

test_bounds_tell_lost_parts plants a lost part in the oracle: each of x, h and the low-rank results with one part less
exceeds these bounds.
"""
import pytest
import torch

from test_shared_ffn import BF16, F32, Case, m, note  # noqa: F401


def parts(v, n):
    """v as n bf16 parts (0: as it is)."""
    if not n:
        return v
    rest, total = v.clone(), torch.zeros_like(v)
    for _ in range(n):
        p = rest.float().to(BF16).double()
        total, rest = total + p, rest - p
    return total


def emulate(c, x_parts=0, h_parts=0, low_parts=0):
    """The operator in binary64, with x, h and the adapters' A x cut to bf16 parts."""
    def project(v, p):
        out = v @ c.w[p].double().T
        for i, r in enumerate(c.ranks()):
            rows = (c.ids == i).nonzero().flatten()
            s = float(c.scale[i]) * (v[rows] @ c.a[p][i, :r].double().T)
            out[rows] += parts(s, low_parts) @ c.b[p][i, :, :r].double().T
        return out

    x = parts(c.x.double(), x_parts)
    g, u = project(x, "gate"), project(x, "up")
    return project(parts(g * torch.sigmoid(g) * u, h_parts), "down")


def error_over_bound(c, got):
    want, size = c.reference()
    norm = torch.linalg.vector_norm
    total = torch.maximum(norm(size), norm(want))
    R = c.R if c.n else 0
    bound = (1.21 * (c.H + R) + (c.I + R) / 2 + 36)**0.5 * 2.0**-24 * total
    if got.dtype == BF16:
        bound = norm(want.float().to(BF16).double() - want) + 2 * (bound + (7 / 3)**0.5 * 2.0**-16 * total)
    return float(norm(got.double() - want) / bound)


def check(m, c, out_t):  # noqa: F811
    got = c.run(m, out_t)
    assert torch.isfinite(got).all()
    over = error_over_bound(c, got)
    assert over <= 1, over


@pytest.mark.parametrize("T,H,I,n,R", [(24, 128, 64, 5, 16), (60, 264, 136, 7, 24), (40, 512, 256, 3, 8)])
def test_bounds_tell_lost_parts(T, H, I, n, R):
    c = Case(T, H, I, n, R, F32, seed=T)
    full, one_less = {F32: 3, BF16: 2}, {F32: 2, BF16: 1}
    for out_t in (F32, BF16):
        whole = dict(x_parts=full[out_t], h_parts=full[out_t], low_parts=full[out_t])
        assert error_over_bound(c, emulate(c, **whole).float().to(out_t)) <= 1
        for lost in whole:
            assert error_over_bound(c, emulate(c, **{**whole, lost: one_less[out_t]}).float().to(out_t)) > 1, (out_t, lost)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 100, 300])
@pytest.mark.parametrize("H,I,n,R", [(128, 64, 0, 0), (520, 264, 0, 0), (128, 64, 5, 16), (264, 136, 7, 24), (1024, 512, 5, 8)])
@pytest.mark.parametrize("x_t,out_t", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
def test_precision(m, T, H, I, n, R, x_t, out_t):  # noqa: F811
    note(f"precision T={T} H={H} I={I} n={n} R={R} x={x_t} out={out_t}")
    check(m, Case(T, H, I, n, R, x_t, seed=T + H), out_t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(1100, 4096, 128), (1100, 4104, 136), (700, 1504, 128), (700, 1504, 136), (2112, 4096, 64),
                                   (700, 512, 1024), (700, 520, 1024), (2112, 320, 2048), (2100, 264, 2056)])
@pytest.mark.parametrize("x_t,out_t", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("n", [0, 3])
def test_precision_of_every_tile(m, T, H, I, x_t, out_t, n):  # noqa: F811
    """Tiles of 64, 128 and 256 tokens and of 64 and 128 weight rows, of gate/up and of down, with K whole and ragged."""
    note(f"tiles T={T} H={H} I={I} n={n} x={x_t} out={out_t}")
    check(m, Case(T, H, I, n, 40, x_t, seed=T + I), out_t)
