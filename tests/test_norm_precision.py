"""The norm calls' rows of every size of values, and the bits of their results, against binary64.

Tolerances.  A square of fp32 is exact in binary64, and so are sums of up to 32768 of them but for 2^-38 of the sum; the factor
from them is used in two fp32 parts (2^-48), and the products by it and the weight are corrected to one rounding: n is off by
2^-24 of itself and less than 2^-36 besides (ARITH).  Outputs add their own rounding: none in fp32 (it is that one), 2^-8 in
bf16, 2^-4 of the value or 2^-10 of the scale in e4m3.  A block's scale is the exact one's unless its largest value
lies within 2^-23 of where the scale changes; a row's scale is rounded once (2^-24).  A combined row is summed in binary64 and
rounded once to fp32, with the residual; without one that rounding enters n twice, by the value and by the row's factor.
"""
import numpy as np
import pytest
import torch

from test_norm import BF16, F32, draw, f64, m, note, outputs  # noqa: F401

HALF, ARITH = 2.0**-24, 2.0**-36


def exact_norm(v, weight, eps):
    return v / np.sqrt((v * v).sum(axis=1, keepdims=True) / v.shape[1] + np.float64(np.float32(eps))) * f64(weight)


def check(y, ys, n, slack=0.0):
    """`slack`: what n may be off by beside its one rounding, relative."""
    T, H = n.shape
    size = np.abs(n)
    if y.dtype in (F32, BF16):
        bad = np.abs(f64(y) - n) > ((HALF if y.dtype == F32 else HALF + 2.0**-8) + ARITH + slack) * size + 2.0**-149
        assert not bad.any(), (np.argwhere(bad)[:4], f64(y)[bad][:4], n[bad][:4])
        return
    if ys.dtype == F32:
        want = np.maximum(size.max(axis=1), 448 * 2.0**-126) / 448
        assert (np.abs(f64(ys) - want) <= (HALF + ARITH + slack) * want).all()
        per = np.repeat(f64(ys)[:, None], H, axis=1)
    else:
        e = ys.view(torch.uint8).cpu().numpy().astype(int) - 127
        pad = np.zeros((T, -(-H // 32) * 32))
        pad[:, :H] = size
        big = pad.reshape(T, -1, 32).max(axis=2)
        least = np.clip(np.ceil(np.log2(np.maximum(big, 1e-300) * (1 - 2 * HALF - slack) / 448)), -127, 127)
        most = np.clip(np.ceil(np.log2(np.maximum(big, 1e-300) * (1 + 2 * HALF + slack) / 448)), -127, 127)
        assert ((e >= least) & (e <= most)).all(), np.argwhere((e < least) | (e > most))[:4]
        per = np.repeat(2.0**e, 32, axis=1)[:, :H]
    bad = np.abs(f64(y) * per - n) > np.maximum(2.0**-4 * size, 2.0**-10 * per) * (1 + 2.0**-20) + (2 * HALF + slack) * size
    assert not bad.any(), (np.argwhere(bad)[:4], (f64(y) * per)[bad][:4], n[bad][:4])


POWERS = [-140, -127, -126, -110, -100, -90, -76, -75, -74, -70, -65, -64, -63, -40, 0, 40, 62, 63, 64, 65, 66, 90, 100, 118, 124]


@pytest.mark.gpu
@pytest.mark.parametrize("H", [7, 64, 515, 4096, 9000, 20001])
@pytest.mark.parametrize("x_t", [F32, BF16])
@pytest.mark.parametrize("y_t", ["f32", "bf16", "block", "row"])
@pytest.mark.parametrize("eps", [0.0, 1e-42])
def test_rows_of_any_scale(m, H, x_t, y_t, eps):  # noqa: F811
    """Values from the smallest that fp32 holds to the largest, where their squares are far outside fp32."""
    note(f"any scale H={H} x={x_t} y={y_t} eps={eps}")
    least = -140 if x_t is F32 else -130                  # bf16 holds values from 2^-133 on
    powers = torch.tensor(POWERS).clamp_min(least).double()
    x = (draw(61, len(POWERS), H).clamp(-3.9, 3.9) * powers.exp2()[:, None]).to(x_t)
    w = draw(62, H, std=0.3, mean=1.0)
    y, ys = outputs(len(POWERS), H, y_t)
    m.moe_add_rms_norm(x.cuda(), None, None, w.cuda(), eps, y, ys)
    torch.cuda.synchronize()
    check(y, ys, exact_norm(f64(x), w, eps))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [5, 72, 1001])
@pytest.mark.parametrize("y_t", ["f32", "block"])
def test_combined_rows_of_any_scale(m, H, y_t):  # noqa: F811
    note(f"combined rows of any scale H={H} y={y_t}")
    T, k = len(POWERS), 2
    scale = torch.tensor(POWERS).double().exp2()
    o = (draw(63, T, k, H).clamp(-3.9, 3.9) * scale[:, None, None]).float().reshape(T * k, H)
    tw, res = torch.softmax(draw(64, T, k), dim=1), (draw(65, T, H).clamp(-3.9, 3.9) * scale[:, None]).float()
    w = draw(66, H, std=0.3, mean=1.0)
    r_out = torch.empty(T, H, device="cuda")
    y, ys = outputs(T, H, y_t)
    m.moe_combine_norm(o.cuda(), tw.cuda(), None, res.cuda(), r_out, w.cuda(), 0.0, y, ys)
    torch.cuda.synchronize()
    v = (f64(o).reshape(T, k, H) * f64(tw)[:, :, None]).sum(axis=1) + f64(res)
    assert (np.abs(f64(r_out) - v) <= HALF * (1 + 2.0**-20) * np.abs(v) + 2.0**-149).all()
    check(y, ys, exact_norm(f64(r_out), w, 0.0))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(37, 4096), (300, 1024), (5, 515), (3, 16384), (2, 20001), (9, 3)])
@pytest.mark.parametrize("x_t,res_t,w_t,y_t", [(F32, BF16, BF16, "f32"), (BF16, F32, F32, "bf16"), (BF16, BF16, BF16, "block"),
                                               (F32, F32, BF16, "row"), (F32, None, F32, "f32")])
def test_bits_of_the_result(m, T, H, x_t, res_t, w_t, y_t):  # noqa: F811
    note(f"bits T={T} H={H} x={x_t} residual={res_t} weight={w_t} y={y_t}")
    x, w = draw(71, T, H, dtype=x_t), draw(72, H, std=0.1, mean=1.0, dtype=w_t)
    res = None if res_t is None else draw(73, T, H, std=2.0, dtype=res_t).cuda()
    r_out = None if res is None else torch.empty_like(res)
    y, ys = outputs(T, H, y_t)
    m.moe_add_rms_norm(x.cuda(), res, r_out, w.cuda(), 1e-6, y, ys)
    torch.cuda.synchronize()
    check(y, ys, exact_norm(f64(x if res is None else r_out), w, 1e-6))


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", [(3, 8, 8192), (2, 8, 16384), (2, 8, 9000), (2, 8, 32768), (1, 8, 32760), (5, 6, 1024), (2, 7, 24576)])
@pytest.mark.parametrize("w_t", [F32, BF16])
@pytest.mark.parametrize("shared,steer,res_t,y_t", [(True, False, BF16, "bf16"), (False, True, F32, "f32"), (True, True, None, "block"),
                                                    (True, False, None, "row")])
def test_long_combined_rows(m, T, k, H, w_t, shared, steer, res_t, y_t):  # noqa: F811
    note(f"combined T={T} k={k} H={H} weight={w_t} shared={shared} steer={steer} residual={res_t} y={y_t}")
    o, tw = draw(81, T * k, H), torch.softmax(draw(82, T, k), dim=1)
    sh, sv = draw(83, T, H) if shared else None, draw(84, H, std=H**-0.5) if steer else None
    w = draw(85, H, std=0.1, mean=1.0, dtype=w_t)
    res = None if res_t is None else draw(86, T, H, std=2.0, dtype=res_t)
    gpu = [None if t is None else t.cuda() for t in (o, tw, sh, res, w, sv)]
    r_out = None if res is None else torch.empty_like(gpu[3])
    y, ys = outputs(T, H, y_t)
    m.moe_combine_norm(gpu[0], gpu[1], gpu[2], gpu[3], r_out, gpu[4], 1e-6, y, ys, steer_v=gpu[5], steer_f=0.75)
    torch.cuda.synchronize()
    v = (f64(o).reshape(T, k, H) * f64(tw)[:, :, None]).sum(axis=1) + (f64(sh) if shared else 0)
    tiny = 2.0**-40                                       # binary64 sums of up to 32768 terms of size 1
    if steer:
        v = v - 0.75 * (v @ f64(sv))[:, None] * f64(sv)
    if res is not None:
        v = v + f64(res)
        half = HALF if res_t is F32 else 2.0**-8 + HALF
        assert (np.abs(f64(r_out) - v) <= half * (1 + 2.0**-20) * np.abs(v) + tiny).all()
        check(y, ys, exact_norm(f64(r_out), w, 1e-6))
        return
    check(y, ys, exact_norm(v.astype(np.float32).astype(np.float64), w, 1e-6), slack=2 * HALF)
