"""The grouped products where a call's sizes choose another kernel, and the values at the edges of their numerics.

Tolerances are those of test_grouped.py (its docstring derives them)."""
import pytest
import torch

from test_grouped import BF16, F32, LAYOUTS, Q4, U, Case, compare, guarded, note, run_dgrad, run_forward, run_q4, run_wgrad, swiglu


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


# ----------------------------------------------------------------------------
# SwiGLU
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 40])
@pytest.mark.parametrize("kind", ["bf16", "q4"])
def test_swiglu_of_far_negative_gates(m, T, kind):
    """silu(g) u for gates whose exp(-g) leaves the floats while the value does not: silu(-90) = -7e-38, times a u of 1e30.
    Exponential, reciprocal and products are off by some 2^-22 (2^-20 taken) down to g = -131, where exp2's own result would be
    below 2^-126 after 2^64 has been taken out; from there the value may be lost, and is at most |g| exp(g) |u|.  Products below
    2^-126 are rounded to steps of 2^-149."""
    step = 2.0**-3 if kind == "q4" else 0.5
    gates = torch.cat([-80.0 - step * torch.arange(200), -105.0 - torch.arange(40)]).to(BF16 if kind == "bf16" else F32).float()
    ups = torch.tensor([1.0, -2.0**60, 2.0**110, -2.0**-80, 2.0**127])
    gates, ups = (t.reshape(-1) for t in torch.broadcast_tensors(gates[:, None], ups))
    K, N = 64, gates.numel()
    x = torch.zeros(T, K, dtype=BF16)
    x[:, :2] = 1.0                                                  # x[0] makes the gate, x[1] the other half
    out = torch.empty(T, N, device="cuda")
    groups = m.RowGroups(T)
    note(f"far negative gates {T} {kind}")
    if kind == "bf16":
        w = torch.zeros(1, 2 * N, K)
        w[0, :N, 0], w[0, N:, 1] = gates, ups
        m.moe_grouped_linear(groups, x.cuda(), w.to(BF16).cuda(), out, m.ACT_SWIGLU)
    else:
        codes = torch.full((1, 2 * N, K), 8, dtype=torch.uint8)
        codes[0, :N, 0] = codes[0, N:, 1] = 9
        s = torch.ones(1, 2 * N, K // 32)
        s[0, :N, 0], s[0, N:, 0] = gates, ups
        m.moe_q4_linear(groups, m.Q4Weights((codes[..., ::2] | codes[..., 1::2] << 4).contiguous().cuda(), s.cuda()), x.cuda(), out,
                        m.ACT_SWIGLU)
    torch.cuda.synchronize()
    g, u = gates.double(), ups.double()
    want = g * torch.sigmoid(g) * u
    tol = torch.where(g >= -131, 2.0**-20 * want.abs() + 2.0**-149, want.abs() + 2.0**-149)
    got = out.cpu().double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, gates {g[bad.any(0)][:8].tolist()}, others {u[bad.any(0)][:8].tolist()}"


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(6, 2, 4, 136, 72), (120, 2, 3, 136, 72), (1300, 0, 1, 136, 2056)], ids=lambda s: "x".join(map(str, s)))
def test_swiglu_of_a_far_negative_gate_leaves_other_rows_alone(m, shape):
    """One row's gates of -90 and below take the wave another way: the other rows' bits do not change."""
    T, k, E, K, N = shape
    c = Case(*shape, seed=66, swiglu=True)
    c.w[:, :N, 0] = 1.0                                             # x[0] moves every gate
    for far in (-100.0, -1000.0, float("-inf")):
        got = []
        for v in (0.5, far):
            c.x[T // 2, 0] = v
            out = torch.empty(c.rows, N, device="cuda")
            note(f"far row {shape} {v}")
            m.moe_grouped_linear(c.groups(m), c.x.cuda(), c.w.cuda(), out, m.ACT_SWIGLU)
            torch.cuda.synchronize()
            got.append(out.cpu())
        rest = [p for p in range(c.rows) if c.r(p) != T // 2]
        assert len(rest) < c.rows and torch.equal(got[0][rest], got[1][rest])


# ----------------------------------------------------------------------------
# 4-bit weights: the ends of the range of x
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("group,zero", [(32, 15), (64, 15), (128, 15), (128, 0)])
@pytest.mark.parametrize("T,N", [(1, 40), (50, 40), (50, 32800)])
def test_q4_of_x_just_below_2_to_116(m, T, N, group, zero):
    """Every x the largest bf16 below 2^116 and of one sign, codes and zero points that add up: an offset product of 32 columns and
    the 3 x 32 columns before it come to at most 2432 |x| < 2^128.  2 K additions, each off by 2^-24 of a partial sum of at most
    2432 |x|, K / group groups to a result."""
    K, code = 256, 15 - zero
    x = torch.full((T, K), 1.9921875 * 2.0**115, dtype=BF16)
    x[1::2] *= -1
    scale = 2.0**-12
    q = m.Q4Weights(torch.full((1, N, K // 2), code * 17, dtype=torch.uint8, device="cuda"),
                    torch.full((1, N, K // group), scale, device="cuda"),
                    torch.full((1, N, K // group), zero, dtype=torch.uint8, device="cuda"))
    out = torch.empty(T, N, device="cuda")
    note(f"q4 of large x {T} {N} {group} {zero}")
    m.moe_q4_linear(m.RowGroups(T), q, x.cuda(), out)
    torch.cuda.synchronize()
    want = (code - zero) * scale * x.double().sum(1, keepdim=True)
    tol = 2 * K * 2.0**-24 * 2432 * x[0, 0].double().abs() * scale
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,N", [(3, 40), (50, 32800)])
def test_q4_of_an_x_that_is_not_finite(m, T, N, value):
    """Its row is NaN throughout: (16 + code) x and -(16 + zero) x are infinities of both signs.  Other rows do not see it."""
    c = Case(T, 0, 1, 192, N, seed=54)
    q = Q4(c, 32, True, F32).on_gpu(m)
    got = []
    for v in (0.5, value):
        c.x[1, 100] = v
        for act in (m.ACT_NONE, m.ACT_SWIGLU):
            out = torch.empty(T, N // (1 + act), device="cuda")
            note(f"q4 of {v}")
            m.moe_q4_linear(c.groups(m), q, c.x.cuda(), out, act)
            torch.cuda.synchronize()
            got.append(out.cpu())
    rest = [t for t in range(T) if t != 1]
    for clean, spoiled in zip(got[:2], got[2:]):
        assert torch.equal(clean[rest], spoiled[rest]) and clean.isfinite().all() and spoiled[1].isnan().all()


# ----------------------------------------------------------------------------
# 4-bit weights: every kernel (test_grouped_choice.py holds the shapes to their kernels)
# ----------------------------------------------------------------------------
# kernel -> rows, weight rows: ends of rows and tiles inside the last block
Q4_ROWS = {"few": (37, 150), "16 halves": (330, 1290), "16": (497, 1290), "32": (2090, 1290), "64 halves": (890, 1290), "64": (3005, 1290)}
# columns, group, scales, zero points: rows that end inside a chunk of 128, a second and third block of 32 groups (from 1024 columns
# with groups of 32, 2048 with 64, 4096 with 128), in one and in two halves
Q4_COLUMNS = [(96, 32, F32, False), (1056, 32, F32, False), (2144, 32, torch.float16, True), (2240, 64, F32, False), (3616, 32, BF16, True),
              (3904, 64, F32, True), (4288, 64, torch.float16, True), (4480, 128, F32, True), (7936, 128, torch.float16, False), (8448, 128, BF16, False)]
Q4_HALVES = (3616, 3904, 7936, 8448)                                # where two halves of K make k_many faster
Q4_EXPERTS = [("16", (6, 4, 24, 192, 2730)), ("16", (3, 8, 30, 160, 2820)), ("64 halves", (64, 2, 8, 2112, 2720)), ("32", (280, 2, 8, 256, 2720))]


def q4_paths():
    return [(kernel, T, N, K) for kernel, (T, N) in Q4_ROWS.items() for K, *_ in Q4_COLUMNS
            if "halves" not in kernel or K in Q4_HALVES or (K > 2048 and kernel == "64 halves")]


@pytest.mark.gpu
@pytest.mark.parametrize("act", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("kernel,T,N,K", q4_paths())
def test_q4_paths(m, kernel, T, N, K, act):
    _, group, scale_t, with_zero = next(c for c in Q4_COLUMNS if c[0] == K)
    g = torch.Generator(device="cuda").manual_seed(55)
    what = f"q4 {kernel} {T} rows, {N} x {K}, groups of {group}, {scale_t}, zero points {with_zero}, swiglu {act}"
    codes = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = ((0.5 + torch.rand(1, N, K // group, generator=g, device="cuda")) * K**-0.5 / 8).to(scale_t)
    zero = torch.randint(0, 16, (1, N, K // group), generator=g, device="cuda", dtype=torch.uint8) if with_zero else None
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    fill = 5.5
    whole, out = guarded(T, N // (1 + act), F32, fill)
    note(what)
    m.moe_q4_linear(m.RowGroups(T), m.Q4Weights(codes, scale, zero), x, out, m.ACT_SWIGLU if act else m.ACT_NONE)
    torch.cuda.synchronize()
    q = torch.stack([codes[0] & 15, codes[0] >> 4], dim=2).view(N, K).double()
    per = lambda t: t.double().repeat_interleave(group, dim=1)
    w = (q - (8.0 if zero is None else per(zero[0]))) * per(scale[0])
    y, t = x.double() @ w.T, 4 * (2 * K)**0.5 * U * torch.sqrt(x.double().square() @ (31 * per(scale[0])).square().T)
    if act:
        y, t = swiglu(y, t)
    more = y.new_zeros(3, y.shape[1])
    compare(whole, torch.cat([y, more]).cpu(), torch.cat([t, more]).cpu(), list(range(T)), fill, what)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,shape", Q4_EXPERTS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_q4_paths_of_experts(m, kernel, shape):
    """Down projections of few and more tokens: no activation, in slot order."""
    c = Case(*shape, seed=56, dst="slots")
    run_q4(m, c, Q4(c, 32, True, torch.float16), F32, f"q4 {kernel} {shape}")


# ----------------------------------------------------------------------------
# bf16 weights: every kernel
# ----------------------------------------------------------------------------
# what test_grouped.LAYOUTS are, on shapes whose groups have more than 16 rows and few weight rows, and more of these
@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda d: "-".join(map(str, d.values())))
@pytest.mark.parametrize("shape", [(140, 3, 9, 328, 136), (140, 3, 9, 328, 616), (33, 2, 3, 1096, 200)], ids=lambda s: "x".join(map(str, s)))
def test_linear_layouts_of_more_rows(m, shape, layout):
    c = Case(*shape, seed=57, **layout)
    run_forward(m, c, F32, f"linear {shape} {layout}")
    c.swiglu, c.w = True, torch.cat([c.w, c.w.flip(1)], dim=1)
    run_forward(m, c, BF16, f"linear {shape} {layout} swiglu")


# kernel, forward too (else the input's gradient alone), (T, k, E, terms of a sum, results of a row): 4 to 17 steps of a ring of two or
# three, ragged ends on every side
BF16_SHAPES = [
    ("128x64", True, (130, 4, 16, 520, 1008)), ("256x128 of 4", True, (300, 4, 16, 200, 4000)), ("256x128 of 4", False, (10, 4, 20, 1032, 3336)),
    ("256x128 of 8", True, (1300, 0, 1, 328, 4112)), ("256x128 of 8", True, (450, 2, 3, 520, 5008)),
    ("256x128 of 8", True, (420, 3, 5, 1032, 3600)), ("256x256", True, (2570, 0, 1, 328, 4112)), ("256x256", True, (420, 3, 5, 520, 7008)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,forward,shape", BF16_SHAPES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_bf16_paths(m, kernel, forward, shape):
    T, k, E, K, P = shape
    tail = 5 if k else 0
    if forward:
        c = Case(T, k, E, K, P, seed=58, dst="slots", tail=tail)
        run_forward(m, c, F32, f"linear {kernel} {shape}")
        run_forward(m, c, BF16, f"linear {kernel} {shape}")
        c = Case(T, k, E, K, P // 2, seed=59, src="sorted", tail=tail, swiglu=True)
        run_forward(m, c, F32, f"linear {kernel} {shape} swiglu")
        run_forward(m, c, BF16, f"linear {kernel} {shape} swiglu")
    c = Case(T, k, E, P, K, seed=60, dst="slots", tail=tail)
    run_dgrad(m, c, F32, f"dgrad {kernel} {shape}")
    run_dgrad(m, c, BF16, f"dgrad {kernel} {shape}")


WGRAD_256 = [(4500, 0, 1, 4104, 4112), (3100, 2, 5, 2056, 2312), (70, 0, 1, 3112, 3304)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", WGRAD_256, ids=lambda s: "x".join(map(str, s)))
def test_wgrad_in_large_tiles(m, shape):
    """Tiles of 256 x 256 (289; 450 in five matrices; 169) with more rows to a group than the kernel keeps indices of at once, whose
    table is filled again while a ring of two steps runs, and with few."""
    T, k, E, K, N = shape
    c = Case(*shape, seed=61, dst="slots" if k else "sorted", some=2 if k else None)
    run_wgrad(m, c, F32, f"wgrad {shape}")
    run_wgrad(m, c, BF16, f"wgrad {shape} accumulate", accumulate=True)


# ----------------------------------------------------------------------------
# stacks of weights, gradients and results behind 4 GiB
# ----------------------------------------------------------------------------
def near(got, want, tol, what):
    """Like compare(), on the GPU."""
    if got.dtype == BF16:
        tol = tol + 2.0**-8 * want.abs()
    worst = float(((got.double() - want).abs() / tol.clamp_min(1e-300)).nan_to_num(nan=1e9).max())
    note(f"{what}: worst {worst:.3f} of the tolerance")
    assert worst <= 1, what


def product(x, w, sizes=None, terms=1):
    """x w^T in binary64 and its tolerance (sizes: what it is taken over, default w)."""
    x, w = x.double(), w.double()
    s = w if sizes is None else sizes
    return x @ w.T, 4 * (x.shape[1] * terms)**0.5 * U * torch.sqrt(x.square() @ s.square().T)


def rows_of(E, T, last):
    """Offsets of E groups: `last` of T positions in the last group, the others in group E - 2."""
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1], off[E] = T - last, T
    return off, ((E - 2, 0, T - last), (E - 1, T - last, T))


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K,T", [(4096, 512, 1032, 3), (4096, 512, 1032, 40), (35, 8192, 8192, 40), (35, 8192, 8192, 4300)])
def test_weights_behind_4_gib(m, E, N, K, T):
    """Forward, with SwiGLU, and the input's gradient, of the last two of a stack of matrices that passes 2^32 bytes before them."""
    assert (E - 2) * N * K * 2 > 2**32
    g = torch.Generator(device="cuda").manual_seed(62)
    w = torch.empty(E, N, K, dtype=BF16, device="cuda")
    for e in (E - 2, E - 1):
        w[e] = (torch.randn(N, K, generator=g, device="cuda") * K**-0.5).to(BF16)
    x, dy = (torch.randn(T, n, generator=g, device="cuda").to(BF16) for n in (K, N))
    off, groups = rows_of(E, T, (T + 1) // 2)
    G = m.RowGroups(T, offsets=off)
    y, s, dx = (torch.full((T, n), 7.0, device="cuda") for n in (N, N // 2, K))
    note(f"weights behind 4 GiB {E} {N} {K} {T}")
    m.moe_grouped_linear(G, x, w, y)
    m.moe_grouped_linear(G, x, w, s, m.ACT_SWIGLU)
    m.moe_grouped_dgrad(G, dy, w, dx)
    torch.cuda.synchronize()
    for e, a, b in groups:
        want, tol = product(x[a:b], w[e])
        near(y[a:b], want, tol, f"linear {e}")
        near(s[a:b], *swiglu(want, tol), f"swiglu {e}")
        near(dx[a:b], *product(dy[a:b], w[e].T), f"dgrad {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("E,N,K,T", [(4096, 256, 8320, 3), (35, 16384, 16384, 2), (35, 16384, 16384, 4), (35, 16384, 16384, 500),
                                     (35, 16384, 16384, 3000)])
def test_codes_behind_4_gib(m, E, N, K, T):
    """4-bit codes likewise, up to the last scale and zero point of the stack; k_few, k_many in halves, in tiles of 16, 32 and 64."""
    assert (E - 2) * N * K // 2 > 2**32
    g = torch.Generator(device="cuda").manual_seed(63)
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(E, N, K // 64, dtype=torch.float16, device="cuda")
    zero = torch.empty(E, N, K // 64, dtype=torch.uint8, device="cuda")
    for e in (E - 2, E - 1):
        codes[e] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale[e] = (0.5 + torch.rand(N, K // 64, generator=g, device="cuda")) * K**-0.5 / 8
        zero[e] = torch.randint(0, 16, (N, K // 64), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    off, groups = rows_of(E, T, (T + 1) // 2)
    G, q = m.RowGroups(T, offsets=off), m.Q4Weights(codes, scale, zero)
    y, s = torch.full((T, N), 7.0, device="cuda"), torch.full((T, N // 2), 7.0, device="cuda")
    note(f"codes behind 4 GiB {E} {N} {K} {T}")
    m.moe_q4_linear(G, q, x, y)
    m.moe_q4_linear(G, q, x, s, m.ACT_SWIGLU)
    torch.cuda.synchronize()
    per = lambda t: t.double().repeat_interleave(64, dim=1)
    for e, a, b in groups:
        w = (torch.stack([codes[e] & 15, codes[e] >> 4], dim=2).view(N, K).double() - per(zero[e])).mul_(per(scale[e]))
        want, tol = product(x[a:b], w, 31 * per(scale[e]), terms=2)
        near(y[a:b], want, tol, f"q4 {e}")
        near(s[a:b], *swiglu(want, tol), f"q4 swiglu {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,E,N,K", [(F32, 35, 8192, 4104), (BF16, 35, 8192, 8200), (F32, 4096, 512, 520)])
def test_weights_gradients_behind_4_gib(m, dtype, E, N, K):
    T = 70
    assert (E - 2) * N * K * (4 if dtype == F32 else 2) > 2**32
    g = torch.Generator(device="cuda").manual_seed(64)
    x, dy = (torch.randn(T, n, generator=g, device="cuda").to(BF16) for n in (K, N))
    off, groups = rows_of(E, T, (T + 1) // 2)
    G = m.RowGroups(T, offsets=off)
    dw = torch.full((E, N, K), 7.0, dtype=dtype, device="cuda")
    note(f"weights' gradients behind 4 GiB {dtype} {E}")
    m.moe_grouped_wgrad(G, x, dy, dw)
    torch.cuda.synchronize()
    assert not any(bool(dw[e].any()) for e in range(E - 2))
    for e, a, b in groups:
        near(dw[e], *product(dy[a:b].T, x[a:b].T), f"wgrad {e}")
    for e, a, b in groups:
        dw[e] = 1.0
    m.moe_grouped_wgrad(G, x, dy, dw, accumulate=True)
    torch.cuda.synchronize()
    for e, a, b in groups:
        want, tol = product(dy[a:b].T, x[a:b].T)
        near(dw[e], want + 1, tol + 2 * U * (want + 1).abs(), f"wgrad accumulate {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 300])
def test_q4_results_behind_4_gib(m, T):
    far, N, K = 2**17 + 7, 2**14 + 64, 128
    g = torch.Generator(device="cuda").manual_seed(65)
    out = torch.zeros(far, N, dtype=BF16, device="cuda")
    rows = far - 1 - 2 * torch.arange(T, device="cuda")
    codes = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = (0.5 + torch.rand(1, N, K // 32, generator=g, device="cuda")) / 90
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    note(f"q4 results behind 4 GiB {T}")
    m.moe_q4_linear(m.RowGroups(T, out_index=rows.to(torch.int32)), m.Q4Weights(codes, scale), x, out)
    torch.cuda.synchronize()
    per = scale[0].double().repeat_interleave(32, dim=1)
    w = (torch.stack([codes[0] & 15, codes[0] >> 4], dim=2).view(N, K).double() - 8) * per
    near(out[rows], *product(x, w, 31 * per, terms=2), "q4 results")
    assert not out[rows - 1].any() and not out[:100].any()
