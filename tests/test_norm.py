"""moe_add_rms_norm and moe_combine_norm against a plain binary64 implementation.

Tolerances.  residual_out of moe_add_rms_norm is one fp32 addition and one rounding, so it is compared bit for bit.
The norm's fp32 arithmetic adds, relative to n: the sum of squares, at most 32 sequential fused multiply-adds per
thread, 6 butterfly steps and 16 partials, all of positive terms (54 * 2^-24, halved by the square root), the
division, the addition of eps, the square root, the reciprocal and two products (6 * 2^-24) -- 33 * 2^-24 < 2e-6 = ARITH.
Output rounding adds half a step of the type: 2^-24 (fp32), 2^-8 (bf16), for e4m3 2^-4 of the value or half a subnormal
step, 2^-10 of the scale; forming the value over the scale one more 2^-23, covered by ARITH's slack.
"""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_moe_permute_amd", "libmoe2bit.so")
ARITH = 2e-6
EPS = 1e-6
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def note(msg):
    print(f"[norm] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import bit_quantized_moe_permute_amd as m
    return m


# ----------------------------------------------------------------------------
# reference
# ----------------------------------------------------------------------------
def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def stored(v64, dtype):
    """v (exact in binary64 up to one rounding) as the residual holds it: rounded to fp32, then to its type."""
    t = torch.from_numpy(v64.astype(np.float32))
    return t.to(dtype)


def norm64(v, weight):
    rms = np.sqrt((v * v).sum(axis=1, keepdims=True) / v.shape[1] + np.float64(np.float32(EPS)))
    return v / rms * f64(weight)


def block_exponents(n):
    """Least e with max|n| <= 448 * 2^e per 32 columns, and how near max|n| lies to a value where it changes."""
    T, H = n.shape
    pad = np.zeros((T, -(-H // 32) * 32))
    pad[:, :H] = np.abs(n)
    big = pad.reshape(T, -1, 32).max(axis=2)
    with np.errstate(divide="ignore"):
        e = np.where(big > 0, np.ceil(np.log2(np.maximum(big, 1e-300) / 448.0)), -127)
    e = np.clip(e, -127, 127)
    near = np.abs(big / (448.0 * 2.0**e) - 0.5) < 1e-5
    near |= np.abs(big / (448.0 * 2.0**e) - 1.0) < 1e-5
    return e.astype(int), near


def check_output(y, y_scale, n):
    """The norm call's output against the binary64 n [T][H]."""
    T, H = n.shape
    if y.dtype in (F32, BF16):
        half = 2.0**-24 if y.dtype == F32 else 2.0**-8
        bad = np.abs(f64(y) - n) > (ARITH + half * (1 + ARITH)) * np.abs(n) + 1e-40
        assert not bad.any(), (np.argwhere(bad)[:4], f64(y)[bad][:4], n[bad][:4])
        return
    codes = f64(y)
    assert np.isfinite(codes).all()
    if y_scale.dtype == F32:
        want = np.maximum(np.abs(n).max(axis=1), 448 * 2.0**-126) / 448
        scale = f64(y_scale)
        assert (np.abs(scale - want) <= 2 * ARITH * want).all()
        per = np.repeat(scale[:, None], H, axis=1)
    else:
        e = y_scale.view(torch.uint8).cpu().numpy().astype(int) - 127
        want, near = block_exponents(n)
        assert ((e == want) | (near & (np.abs(e - want) <= 1))).all(), np.argwhere(e != want)[:4]
        per = np.repeat(2.0**e, 32, axis=1)[:, :H]
    bad = np.abs(codes * per - n) > np.maximum(2.0**-4 * np.abs(n), 2.0**-10 * per) * (1 + ARITH) + ARITH * np.abs(n)
    assert not bad.any(), (np.argwhere(bad)[:4], (codes * per)[bad][:4], n[bad][:4])


def outputs(T, H, y, device="cuda"):
    t = torch.full((T, H), float("nan"), device=device).to({"f32": F32, "bf16": BF16}.get(y, E4M3))
    s = (torch.full((T, (H + 31) // 32), 255, dtype=torch.uint8, device=device) if y == "block" else
         torch.full((T,), float("nan"), device=device) if y == "row" else None)
    return t, s


def draw(seed, *shape, std=1.0, mean=0.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


# ----------------------------------------------------------------------------
# moe_add_rms_norm
# ----------------------------------------------------------------------------
SHAPES = [(1, 1), (3, 7), (2, 31), (5, 33), (1, 64), (4, 256), (9, 1000), (3, 1023), (2, 2055), (1, 4096), (37, 4096),
          (2, 4104), (2, 8192), (1, 8193), (2, 9000), (1, 16384), (1, 20001), (1, 32768), (1, 32767)]
TYPES = [(F32, BF16, BF16, "bf16"), (BF16, F32, F32, "f32"), (BF16, BF16, BF16, "block"), (F32, F32, BF16, "row"),
         (BF16, None, F32, "bf16"), (F32, None, BF16, "block")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("x_t,res_t,w_t,y_t", TYPES)
def test_add_rms_norm(m, T, H, x_t, res_t, w_t, y_t):
    note(f"add_rms_norm T={T} H={H} x={x_t} residual={res_t} weight={w_t} y={y_t}")
    x, w = draw(1, T, H, dtype=x_t), draw(2, H, std=0.1, mean=1.0, dtype=w_t)
    res = None if res_t is None else draw(3, T, H, std=2.0, dtype=res_t)
    y, ys = outputs(T, H, y_t)
    r_in = None if res is None else res.cuda()
    r_out = None if res is None else torch.full_like(r_in, float("nan"))
    m.moe_add_rms_norm(x.cuda(), r_in, r_out, w.cuda(), EPS, y, ys)
    torch.cuda.synchronize()
    v = f64(x)
    if res is not None:
        want = stored(v + f64(res), res_t)
        assert torch.equal(r_out.cpu(), want)
        assert torch.equal(r_in.cpu(), res)
        v = f64(want)
    check_output(y, ys, norm64(v, w))
    if res is not None:                                   # in place: the same bits
        y2, ys2 = outputs(T, H, y_t)
        m.moe_add_rms_norm(x.cuda(), r_in, r_in, w.cuda(), EPS, y2, ys2)
        torch.cuda.synchronize()
        assert torch.equal(r_in, r_out)
        assert torch.equal(y2.view(torch.uint8), y.view(torch.uint8))
        assert ys is None or torch.equal(ys2, ys)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [512, 515])
@pytest.mark.parametrize("y_t", ["f32", "bf16", "block", "row"])
def test_rows_that_are_not_finite(m, H, y_t):
    """A NaN makes its row NaN, an infinity (whose row's factor is 0) itself alone; the other rows keep their bits, and rows
    behind the last one are not written."""
    note(f"not finite H={H} y={y_t}")
    x, w = draw(8, 5, H).cuda(), draw(9, H, std=0.1, mean=1.0).cuda()

    def run():
        y, ys = outputs(7, H, y_t)
        before = y.clone()
        m.moe_add_rms_norm(x, None, None, w, EPS, y[:5], None if ys is None else ys[:5])
        torch.cuda.synchronize()
        assert torch.equal(y[5:].view(torch.uint8), before[5:].view(torch.uint8))
        assert ys is None or (ys[5:] == 255).all() or torch.isnan(ys[5:]).all()
        return y[:5].cpu(), None if ys is None else ys[:5].cpu()

    clean, clean_s = run()
    x[1, 3], x[2, 7] = float("nan"), float("inf")
    y, ys = run()
    keep = [0, 3, 4]
    assert torch.equal(y[keep].view(torch.uint8), clean[keep].view(torch.uint8))
    assert ys is None or torch.equal(ys[keep], clean_s[keep])
    assert torch.isnan(y[1].float()).all()
    assert torch.isnan(y[2, 7].float()) and int((y[2].float() != 0).sum()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("H", [512, 515])
@pytest.mark.parametrize("y_t", ["f32", "bf16", "block", "row"])
def test_rows_of_unusual_values(m, H, y_t):
    """Zero rows, tiny rows (eps decides), large rows, one spike, blocks of zeros, negative weights."""
    note(f"unusual rows H={H} y={y_t}")
    x = draw(5, 7, H)
    x[0] = 0.0
    x[1] *= 2.0**-40
    x[2] *= 2.0**40
    x[3] = 0.0
    x[3, H // 2] = 3.0
    x[4, :64] = 0.0
    x[5] = 1.0
    w = draw(6, H)
    y, ys = outputs(7, H, y_t)
    m.moe_add_rms_norm(x.cuda(), None, None, w.cuda(), EPS, y, ys)
    torch.cuda.synchronize()
    check_output(y, ys, norm64(f64(x), w))
    assert (f64(y)[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("off", [1, 2, 8])
def test_rows_at_any_element_offset(m, off):
    """Views that start `off` elements into a buffer (16-byte alignment lost or kept); what lies around the outputs stays."""
    note(f"offset {off}")
    T, H = 3, 520
    x, res, w = draw(7, T * H + 16, dtype=BF16), draw(8, T * H + 16, dtype=BF16), draw(9, H + 16)
    xb, rb, wb = x.cuda(), res.cuda(), w.cuda()
    out = torch.full((T * H + 16,), 7.0, dtype=BF16, device="cuda")
    y = torch.full((T * H + 16,), 7.0, dtype=BF16, device="cuda")
    view = lambda t: t[off:off + T * H].view(T, H)  # noqa: E731
    m.moe_add_rms_norm(view(xb), view(rb), view(out), wb[off:off + H], EPS, view(y))
    torch.cuda.synchronize()
    want = stored(f64(view(x)) + f64(view(res)), BF16)
    assert torch.equal(view(out).cpu(), want)
    check_output(view(y), None, norm64(f64(want), w[off:off + H]))
    for t in (out, y):
        assert (t[:off] == 7).all() and (t[off + T * H:] == 7).all()


@pytest.mark.gpu
def test_rows_do_not_depend_on_each_other(m):
    note("row independence")
    T, H = 300, 2048
    x, w = draw(11, T, H).cuda(), draw(12, H, mean=1.0, std=0.1).cuda()
    y, ys = outputs(T, H, "block")
    m.moe_add_rms_norm(x, None, None, w, EPS, y, ys)
    for t in (0, 17, T - 1):
        y1, ys1 = outputs(1, H, "block")
        m.moe_add_rms_norm(x[t:t + 1], None, None, w, EPS, y1, ys1)
        torch.cuda.synchronize()
        assert torch.equal(y1[0].view(torch.uint8), y[t].view(torch.uint8)) and torch.equal(ys1[0], ys[t])


@pytest.mark.gpu
def test_many_short_rows(m):
    """More than 2^16 rows."""
    note("70001 rows")
    T, H = 70001, 40
    x, w = draw(13, T, H, dtype=BF16), draw(14, H, mean=1.0, std=0.1)
    y, _ = outputs(T, H, "f32")
    m.moe_add_rms_norm(x.cuda(), None, None, w.cuda(), EPS, y)
    torch.cuda.synchronize()
    check_output(y, None, norm64(f64(x), w))


# ----------------------------------------------------------------------------
# moe_combine_norm
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", [(1, 8, 4096), (3, 8, 512), (5, 4, 1024), (2, 1, 72), (4, 3, 100), (2, 8, 1001), (1, 16, 8192),
                                   (2, 2, 16384), (1, 2, 32768), (1, 1, 1), (3, 4, 7), (2, 6, 9), (3, 5, 63), (2, 8, 9001),
                                   (1, 3, 32767)])
@pytest.mark.parametrize("shared,steer,res_t,y_t", [(True, False, BF16, "bf16"), (False, False, F32, "f32"),
                                                    (True, True, F32, "block"), (False, True, None, "row")])
def test_combine_norm(m, T, k, H, shared, steer, res_t, y_t):
    """Against the combine (and steering) calls followed by moe_add_rms_norm, and against binary64."""
    note(f"combine_norm T={T} k={k} H={H} shared={shared} steer={steer} residual={res_t} y={y_t}")
    o, tw = draw(21, T * k, H), torch.softmax(draw(22, T, k), dim=1)
    sh = draw(23, T, H) if shared else None
    w = draw(24, H, std=0.1, mean=1.0, dtype=BF16)
    sv = draw(25, H, std=H**-0.5) if steer else None
    res = None if res_t is None else draw(26, T, H, std=2.0, dtype=res_t)
    dev = [None if t is None else t.cuda() for t in (o, tw, sh, res, w, sv)]
    od, twd, shd, rd, wd, svd = dev
    r_out = None if res is None else torch.full_like(rd, float("nan"))
    y, ys = outputs(T, H, y_t)
    m.moe_combine_norm(od, twd, shd, rd, r_out, wd, EPS, y, ys, steer_v=svd, steer_f=0.75)
    # the separate calls
    yc = torch.empty(T, H, device="cuda")
    if steer:
        m.moe_combine_steer(od, twd, shd, T, k, H, svd, 0.75, yc)
    else:
        m.moe_combine(od, twd, shd, T, k, H, yc)
    torch.cuda.synchronize()
    v = (f64(o).reshape(T, k, H) * f64(tw)[:, :, None]).sum(axis=1) + (f64(sh) if shared else 0)
    mag = (np.abs(f64(o)).reshape(T, k, H) * f64(tw)[:, :, None]).sum(axis=1) + (np.abs(f64(sh)) if shared else 0)
    if steer:
        d = f64(sv)
        dot = v @ d
        v = v - 0.75 * dot[:, None] * d
        # the dot's error: H products in fp32, at most 32 + 6 + 16 sequential sums of terms of size mag * |d|
        mag = mag + 54 * 0.75 * (mag @ np.abs(d))[:, None] * np.abs(d)
    err = (k + 4) * 2.0**-24 * mag                        # k + 1 additions, the update, the residual, before rounding
    if res is not None:
        v = v + f64(res)
        err = err + 2.0**-24 * np.abs(v) + (2.0**-8 * np.abs(v) if res_t is BF16 else 0)
        assert (np.abs(f64(r_out) - v) <= err * (1 + 1e-6)).all()
        if not steer:                                     # one rounding of the whole sum, two in bf16 (fp32 between)
            half = 2.0**-24 if res_t is F32 else 2.0**-8 + 2.0**-24
            assert (np.abs(f64(r_out) - v) <= half * (1 + 1e-6) * np.abs(v)).all()
        v = f64(r_out)
        err = 0 * err
    n = norm64(v, w)
    # what the row's error does to n beyond the arithmetic of the norm: itself over the rms, and through the rms
    rms = np.sqrt((v * v).mean(axis=1, keepdims=True) + EPS)
    slack = err / rms * np.abs(f64(w)) + np.abs(n) * (err * np.abs(v)).mean(axis=1, keepdims=True) / rms**2
    if y_t in ("f32", "bf16"):
        half = 2.0**-24 if y_t == "f32" else 2.0**-8
        assert (np.abs(f64(y) - n) <= slack + (ARITH + half * (1 + ARITH)) * np.abs(n) + 1e-40).all()
    else:
        y2, ys2 = outputs(T, H, y_t)                      # the rounding to 8 bits, on the row as the library formed it
        if res is None:
            m.moe_add_rms_norm(yc, None, None, wd, EPS, y2, ys2)
        else:
            m.moe_add_rms_norm(torch.zeros_like(yc), r_out, torch.empty_like(r_out), wd, EPS, y2, ys2)
        torch.cuda.synchronize()
        if res is not None:
            check_output(y, ys, n)
        else:
            per = np.repeat(f64(ys)[:, None], H, axis=1)
            got = f64(y) * per
            assert (np.abs(got - n) <= slack + np.maximum(2.0**-4 * np.abs(n), 2.0**-10 * per) * (1 + ARITH)
                    + 2 * ARITH * np.abs(n)).all()


# ----------------------------------------------------------------------------
# streams and graphs
# ----------------------------------------------------------------------------
@pytest.mark.gpu
def test_graph_replays_match_eager_calls(m):
    """Both calls captured in one graph, replayed on changed inputs with eager work in between."""
    note("graph")
    T, k, H = 3, 8, 1024
    o, tw, sh = draw(31, T * k, H).cuda(), torch.softmax(draw(32, T, k), 1).cuda(), draw(33, T, H).cuda()
    res, w = draw(34, T, H, dtype=BF16).cuda(), draw(35, H, mean=1.0, std=0.1, dtype=BF16).cuda()
    mid, mid2 = torch.empty_like(res), torch.empty_like(res)
    y, _ = outputs(T, H, "bf16")
    z, zs = outputs(T, H, "block")

    def calls():
        m.moe_combine_norm(o, tw, sh, res, mid, w, EPS, y)
        m.moe_add_rms_norm(y, mid, mid2, w, EPS, z, zs)

    calls()
    torch.cuda.synchronize()
    g, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(g, stream=cap):
            calls()
    for i in range(4):
        o.copy_(draw(40 + i, T * k, H))
        res.copy_(draw(50 + i, T, H, dtype=BF16))
        torch.cuda.synchronize()
        for t in (mid, mid2, y):
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (mid, y, mid2, z.view(torch.uint8), zs)]
        calls()
        torch.cuda.synchronize()
        for a, b in zip(got, (mid, y, mid2, z.view(torch.uint8), zs)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_runs_on_the_current_stream(m):
    """Inputs written and outputs read on a side stream, without any other synchronization."""
    note("side stream")
    T, H = 64, 4096
    w = torch.ones(H, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = torch.zeros(T, H, device="cuda")
        for _ in range(20):
            x.add_(0.25)
        y = torch.empty(T, H, device="cuda")
        m.moe_add_rms_norm(x, None, None, w, 0.0, y)
        got = y.clone()
    s.synchronize()
    assert (got - 1).abs().max() <= ARITH


# ----------------------------------------------------------------------------
# refusals (host only)
# ----------------------------------------------------------------------------
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe2bit.so not built (run __graft_entry__.build())")


@pytest.fixture(scope="module")
def calls():
    import bit_quantized_moe_permute_amd as m
    return m.lib


def _add(L, x=0x10000, x_dt=1, T=4, H=64, res=0x20000, out=0x30000, res_dt=1, w=0x40000, w_dt=1, eps=1e-6, y=0x50000, y_dt=1,
         ys=None):
    st = L.moe_add_rms_norm(x, x_dt, T, H, res, out, res_dt, w, w_dt, eps, y, y_dt, ys, None)
    return st, L.moe_last_error().decode()


@needs_lib
@pytest.mark.parametrize("bad,word", [
    (dict(x=None), "null"), (dict(w=None), "null"), (dict(y=None), "null"), (dict(out=None), "residual_out"),
    (dict(res=None), "residual_out"), (dict(T=0), "n_tokens"), (dict(T=-1), "n_tokens"), (dict(H=0), "hidden"),
    (dict(x_dt=2), "dtype"), (dict(x_dt=-1), "dtype"), (dict(res_dt=2), "dtype"), (dict(w_dt=3), "dtype"),
    (dict(y_dt=4), "dtype"), (dict(y_dt=-1), "dtype"), (dict(y_dt=2), "y_scale"), (dict(ys=0x60000), "y_scale"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(x=0x10001), "misaligned"), (dict(x_dt=0, x=0x10002), "misaligned"), (dict(w=0x40001), "misaligned"),
    (dict(y=0x50001), "misaligned"), (dict(y_dt=3, ys=0x60002), "misaligned"), (dict(res=0x20001), "misaligned"),
    (dict(y=0x10000), "overlap"), (dict(y=0x10002), "overlap"), (dict(y=0x20000), "overlap"), (dict(y=0x30000), "overlap"),
    (dict(out=0x10000), "overlap"), (dict(out=0x20002), "overlap"), (dict(out=0x40000), "overlap"),
    (dict(y_dt=2, ys=0x50000), "overlap"), (dict(y_dt=2, ys=0x10000), "overlap"), (dict(y_dt=3, ys=0x20000), "overlap"),
])
def test_add_rms_norm_refuses(calls, bad, word):
    st, msg = _add(calls, **bad)
    assert st == 1 and word in msg, (st, msg)


@needs_lib
def test_add_rms_norm_refuses_long_rows(calls):
    far = dict(x=1 << 30, res=2 << 30, out=3 << 30, w=4 << 30, y=5 << 30)
    st, msg = _add(calls, H=32769, **far)
    assert st == 2 and "32768" in msg
    st, msg = _add(calls, T=1 << 22, H=8, **far)
    assert st == 2 and "split the batch" in msg


@needs_lib
def test_combine_norm_refuses(calls):
    good = dict(o=0x10000, w=0x20000, sh=0x30000, T=2, k=2, H=64, sv=None, f=0.0, res=0x40000, out=0x50000, res_dt=1,
                wt=0x60000, w_dt=1, eps=1e-6, y=0x70000, y_dt=1, ys=None)

    def call(**bad):
        a = dict(good, **bad)
        st = calls.moe_combine_norm(a["o"], a["w"], a["sh"], a["T"], a["k"], a["H"], a["sv"], a["f"], a["res"], a["out"],
                                    a["res_dt"], a["wt"], a["w_dt"], a["eps"], a["y"], a["y_dt"], a["ys"], None)
        return st, calls.moe_last_error().decode()

    for bad, word in [(dict(o=None), "null"), (dict(w=None), "null"), (dict(k=0), "shape"), (dict(T=0), "n_tokens"),
                      (dict(sh=0x30002), "misaligned"), (dict(sv=0x80001), "misaligned"),
                      (dict(sv=0x80000, f=float("nan")), "finite"), (dict(out=0x10000), "overlap"),
                      (dict(y=0x20000), "overlap"), (dict(y=0x30000), "overlap"), (dict(sv=0x70000), "overlap"),
                      (dict(wt=None), "null"), (dict(out=None), "residual_out"), (dict(y_dt=3), "y_scale")]:
        st, msg = call(**bad)
        assert st == 1 and word in msg, (bad, st, msg)


@needs_lib
def test_binding_refuses():
    import bit_quantized_moe_permute_amd as m
    T, H = 3, 64
    x, w, y = torch.zeros(T, H), torch.ones(H), torch.zeros(T, H)
    with pytest.raises(TypeError, match="GPU"):
        m.moe_add_rms_norm(x, None, None, w, EPS, y)
    with pytest.raises(ValueError, match="tokens"):
        m.moe_add_rms_norm(x[0], None, None, w, EPS, y)
    with pytest.raises(ValueError, match="residual_out"):
        m.moe_add_rms_norm(x, x, None, w, EPS, y)
    with pytest.raises(TypeError, match="residual_out"):
        m.moe_add_rms_norm(x, x, x.to(BF16), w, EPS, y)
    with pytest.raises(ValueError, match="weight"):
        m.moe_add_rms_norm(x, None, None, w[:-1], EPS, y)
    with pytest.raises(ValueError, match="y: "):
        m.moe_add_rms_norm(x, None, None, w, EPS, y[:2])
    with pytest.raises(ValueError, match="y_scale"):
        m.moe_add_rms_norm(x, None, None, w, EPS, y.to(E4M3))
    with pytest.raises(ValueError, match="y_scale"):
        m.moe_add_rms_norm(x, None, None, w, EPS, y, torch.zeros(T))
    with pytest.raises(ValueError, match="y_scale"):
        m.moe_add_rms_norm(x, None, None, w, EPS, y.to(E4M3), torch.zeros(T, 1, dtype=torch.uint8))
    with pytest.raises(TypeError, match="y_scale"):
        m.moe_add_rms_norm(x, None, None, w, EPS, y.to(E4M3), torch.zeros(T, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="unsupported dtype"):
        m.moe_add_rms_norm(x.half(), None, None, w, EPS, y)
    with pytest.raises(ValueError, match="slot_out"):
        m.moe_combine_norm(x, torch.ones(2, 2), None, None, None, w, EPS, y)
    with pytest.raises(TypeError, match="float32"):
        m.moe_combine_norm(x, torch.ones(3, 1), x.to(BF16), None, None, w, EPS, y)
    with pytest.raises(ValueError, match="steer_v"):
        m.moe_combine_norm(x, torch.ones(3, 1), None, None, None, w, EPS, y, steer_v=w[:-1])
