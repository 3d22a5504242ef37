"""moe_grouped_linear, its two gradients and moe_q4_linear against plain binary64 implementations.

Tolerances, per element.  A sum of K terms in fp32 makes one rounding error of at most 2^-24 of the partial sum per addition.
With terms of random sign the j-th partial sum is about sqrt(j / K) of the terms' root sum of squares S, so the errors, uniform
and independent, add up to a standard deviation of sqrt(K / 2) * 2^-24 / sqrt(3) * S = 0.41 sqrt(K) 2^-24 S; over some 10^6
elements 5 of these are met: 4 * sqrt(K) * 2^-24 * S leaves a factor of two.  Sums of few terms are covered by it too: K
additions are off by at most K 2^-24 sum |terms| <= K^1.5 2^-24 S, less than 4 sqrt(K) 2^-24 S up to K = 4, and shorter chains
of larger K by the argument above.  A bf16 result adds 2^-8 of its value.  SwiGLU y = silu(g) u: errors of g and u enter with
at most 1.1 |u| and |silu(g)|; its own exp, quotient and products are off by some 2^-22 of y (2^-20 taken).
4-bit weights: what is summed is x (16 + code) and -x (16 + zero), both factors below 32, so S is taken over both terms at 31
times scale |x|, and K counts twice; a scaled sum per group and its addition are two roundings more (K / 32 groups at most).
"""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_moe_permute_amd", "libmoe2bit.so")
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0**-24


def note(msg):
    print(f"[grouped] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import bit_quantized_moe_permute_amd as m
    return m


# ----------------------------------------------------------------------------
# inputs and reference
# ----------------------------------------------------------------------------
class Case:
    """Rows of T tokens with k choices among E experts (k = 0: one matrix for all), sorted by expert, CPU tensors.

    src: x has the tokens' rows ("tokens") or sorted rows; dst: outputs in slot order ("slots") or sorted.  head, tail:
    positions before the first and behind the last group."""

    def __init__(self, T, k, E, K, N, src="tokens", dst="sorted", seed=1, head=0, tail=0, some=None, swiglu=False):
        g = torch.Generator().manual_seed(seed)
        self.T, self.k, self.E, self.K, self.N, self.swiglu = T, k, E, K, N, swiglu
        self.src, self.dst = src, dst

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(BF16)

        if k:
            among = E if some is None else some                     # experts that get rows
            expert = torch.stack([torch.randperm(among, generator=g)[:k] for _ in range(T)]).reshape(-1) * (E // among)
            order = torch.sort(expert, stable=True).indices
            counts = torch.bincount(expert, minlength=E)
        else:
            order, counts = torch.arange(T), torch.tensor([T])
        self.R = T * max(k, 1)
        self.rows = self.R + head + tail                            # positions
        self.counts = counts.tolist()
        self.begin = [head + int(c) for c in torch.cat([counts.new_zeros(1), counts.cumsum(0)])]
        self.offsets = torch.tensor(self.begin, dtype=torch.int32) if k else None
        pad = lambda v: torch.cat([torch.full((head,), 2**31 - 1), v, torch.full((tail,), -7)]).to(torch.int32)
        self.perm = pad(order)
        self.x = normal(T if src == "tokens" else self.rows, K)
        self.w = normal(E, N * (2 if swiglu else 1), K, std=K**-0.5)
        self.dy = normal(self.R if dst == "slots" else self.rows, N)
        self.in_index = self.perm if src == "tokens" and k else None
        self.out_index = self.perm if dst == "slots" else None

    def positions(self, e):
        return list(range(self.begin[e], self.begin[e + 1])) if self.k else list(range(self.T))

    def r(self, p):
        """Row of x of position p, by the definition."""
        return int(self.in_index[p]) // self.k if self.in_index is not None else p

    def slot(self, p):
        return int(self.in_index[p]) if self.in_index is not None else p

    def o(self, p):
        return int(self.out_index[p]) if self.out_index is not None else p

    def groups(self, m):
        dev = lambda t: None if t is None else t.cuda()
        return m.RowGroups(self.rows, offsets=dev(self.offsets), in_index=dev(self.in_index),
                           in_div=self.k if self.in_index is not None else 1, out_index=dev(self.out_index))


def guarded(rows, cols, dtype, fill):
    """An output of `rows` rows with guard rows behind it, all of one value."""
    whole = torch.full((rows + 3, cols), fill, dtype=dtype, device="cuda")
    return whole, whole[:rows]


def compare(out, want, tol, written, fill, what):
    """out within tol of want where written (rows), still `fill` elsewhere."""
    out = out.cpu()
    rest = torch.ones(out.shape[0], dtype=torch.bool)
    rest[written] = False
    assert torch.equal(out[rest], torch.full_like(out[rest], fill)), f"{what}: rows that no position names were written"
    got, want, tol = out[written].double(), want[written], tol[written]
    if out.dtype == BF16:
        tol = tol + 2.0**-8 * want.abs()
    bad = ~((got - want).abs() <= tol)
    worst = float(((got - want).abs() / tol.clamp_min(1e-300)).nan_to_num(nan=1e9).max()) if got.numel() else 0.0
    note(f"{what}: {out.dtype} worst {worst:.3f} of the tolerance")
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {worst:.3g} times the tolerance"


def swiglu(y, t):
    """silu(g) * u of y = [g, u] and its tolerance from that of y."""
    n = y.shape[1] // 2
    g, u, tg, tu = y[:, :n], y[:, n:], t[:, :n], t[:, n:]
    s = g * torch.sigmoid(g)
    return s * u, 1.1 * u.abs() * tg + s.abs() * tu + 1.1 * tg * tu + 2.0**-20 * (s * u).abs()


def forward(c, weights=None, sizes=None, terms=1):
    """Results, their tolerances and the written rows of the forward product, binary64.  weights: matrices (default c.w),
    sizes: what S is taken over (default the weights)."""
    rows = c.R if c.dst == "slots" else c.rows
    out, tol, written = torch.zeros(rows, c.N, dtype=F64), torch.zeros(rows, c.N, dtype=F64), []
    for e in range(c.E):
        p = c.positions(e)
        if not p:
            continue
        x = c.x[[c.r(i) for i in p]].double()
        w = (c.w[e].double() if weights is None else weights[e])
        s = w if sizes is None else sizes[e]
        y, t = x @ w.T, 4 * (c.K * terms)**0.5 * U * torch.sqrt(x.square() @ s.square().T)
        if c.swiglu:
            y, t = swiglu(y, t)
        o = [c.o(i) for i in p]
        out[o], tol[o] = y, t
        written += o
    return out, tol, written


def run_forward(m, c, out_t, what):
    fill = 7.25
    whole, out = guarded(c.R if c.dst == "slots" else c.rows, c.N, out_t, fill)
    note(f"{what} {out_t}")
    m.moe_grouped_linear(c.groups(m), c.x.cuda(), c.w.cuda(), out, m.ACT_SWIGLU if c.swiglu else m.ACT_NONE)
    torch.cuda.synchronize()
    want, tol, written = forward(c)
    compare(whole, torch.cat([want, want[:0].new_zeros(3, c.N)]), torch.cat([tol, tol.new_zeros(3, c.N)]), written, fill, what)
    return out


# T, k, E, K, N: single rows, odd rows, tiles' edges, K and N that are no multiples of a tile, empty groups, many groups
SHAPES = [
    (1, 1, 1, 8, 8), (1, 0, 1, 1048, 72), (4, 0, 1, 136, 16520), (16, 0, 1, 136, 1000), (1, 2, 4, 64, 64), (1, 8, 256, 512, 136),
    (3, 2, 5, 72, 40), (5, 4, 16, 264, 520), (16, 1, 3, 128, 256),
    (17, 2, 4, 1000, 264), (33, 4, 8, 192, 128), (64, 1, 1, 256, 128), (65, 2, 3, 64, 192), (130, 4, 16, 520, 1000),
    (257, 2, 2, 128, 272), (300, 1, 300, 64, 64), (600, 2, 3, 320, 384), (1100, 1, 2, 1032, 520), (129, 0, 1, 512, 256),
]


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_linear(m, shape, swiglu):
    c = Case(*shape, swiglu=swiglu)
    run_forward(m, c, BF16, f"linear {shape} swiglu={swiglu}")
    run_forward(m, c, F32, f"linear {shape} swiglu={swiglu}")


# rows outside the groups, before and behind them; groups with rows far apart; both orders on either side
LAYOUTS = [dict(src="sorted", dst="sorted"), dict(src="sorted", dst="slots"), dict(src="tokens", dst="slots"),
           dict(src="tokens", dst="sorted", head=3, tail=9), dict(src="sorted", dst="sorted", head=1, tail=70),
           dict(src="sorted", dst="slots", tail=200, some=3)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda d: "-".join(map(str, d.values())))
@pytest.mark.parametrize("shape", [(1, 2, 12, 128, 72), (19, 3, 12, 96, 200), (140, 3, 9, 328, 136)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_layouts(m, shape, layout):
    c = Case(*shape, seed=2, **layout)
    run_forward(m, c, F32, f"linear {shape} {layout}")
    c.swiglu, c.w = True, torch.cat([c.w, c.w.flip(1)], dim=1)
    run_forward(m, c, BF16, f"linear {shape} {layout} swiglu")


def run_dgrad(m, c, out_t, what):
    fill = -3.5
    rows = c.R if c.in_index is not None else c.rows
    whole, dx = guarded(rows, c.K, out_t, fill)
    note(f"{what} {out_t}")
    m.moe_grouped_dgrad(c.groups(m), c.dy.cuda(), c.w.cuda(), dx)
    torch.cuda.synchronize()
    want, tol, written = torch.zeros(rows + 3, c.K, dtype=F64), torch.zeros(rows + 3, c.K, dtype=F64), []
    for e in range(c.E):
        p = c.positions(e)
        if p:
            dy, w, i = c.dy[[c.o(q) for q in p]].double(), c.w[e].double(), [c.slot(q) for q in p]
            want[i], tol[i] = dy @ w, 4 * c.N**0.5 * U * torch.sqrt(dy.square() @ w.square())
            written += i
    compare(whole, want, tol, written, fill, what)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_dgrad(m, shape):
    c = Case(*shape, seed=3)
    run_dgrad(m, c, BF16, f"dgrad {shape}")
    run_dgrad(m, c, F32, f"dgrad {shape}")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda d: "-".join(map(str, d.values())))
def test_dgrad_layouts(m, layout):
    run_dgrad(m, Case(45, 3, 12, 200, 136, seed=4, **layout), F32, f"dgrad {layout}")


def run_wgrad(m, c, out_t, what, accumulate=False):
    note(f"{what} {out_t}")
    whole = torch.full((c.E * c.N * c.K + 64,), 0.75, dtype=out_t, device="cuda")
    dw = whole[:c.E * c.N * c.K].view(c.E, c.N, c.K)
    if accumulate:
        dw.copy_(torch.randn(c.E, c.N, c.K, generator=torch.Generator().manual_seed(9)))
    else:
        dw.fill_(float("nan"))
    old = dw.cpu().double()
    m.moe_grouped_wgrad(c.groups(m), c.x.cuda(), c.dy.cuda(), dw, accumulate=accumulate)
    torch.cuda.synchronize()
    got = dw.cpu()
    assert torch.equal(whole[c.E * c.N * c.K:].cpu(), torch.full((64,), 0.75, dtype=out_t)), f"{what}: wrote behind dw"
    worst = 0.0
    for e in range(c.E):
        p = c.positions(e)
        dy, x = c.dy[[c.o(q) for q in p]].double(), c.x[[c.r(q) for q in p]].double()
        want, tol = dy.T @ x, 4 * max(len(p), 1)**0.5 * U * torch.sqrt(dy.square().T @ x.square())
        if accumulate:
            want = want + old[e]
            tol = tol + 2 * U * want.abs()
        if out_t == BF16:
            tol = tol + 2.0**-8 * want.abs()
        err = (got[e].double() - want).abs()
        assert (err <= tol).all(), f"{what}: group {e} off by {float((err - tol).max()):.3g} beyond its tolerance"
        worst = max(worst, float((err / tol.clamp_min(1e-300)).max()))
    note(f"{what}: worst {worst:.3f} of the tolerance")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_wgrad(m, shape):
    c = Case(*shape, seed=5)
    run_wgrad(m, c, BF16, f"wgrad {shape}")
    run_wgrad(m, c, F32, f"wgrad {shape}")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2600, 2, 2, 264, 520), (5000, 1, 1, 64, 72), (4097, 0, 1, 136, 72), (2300, 2, 17, 1032, 1000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_wgrad_of_many_rows(m, shape):
    """More rows to a group than the kernel keeps indices of at once."""
    run_wgrad(m, Case(*shape, seed=5, dst="slots"), F32, f"wgrad {shape}")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(700, 4, 12, 520, 1288), (512, 8, 32, 264, 2056), (1300, 0, 1, 328, 5000), (2200, 3, 5, 136, 4104)],
                         ids=lambda s: "x".join(map(str, s)))
def test_large_products(m, shape):
    """The largest tiles: enough rows and weights that they fill the chip, with ragged ends on every side."""
    tail = 3 if shape[1] else 0                                     # (without offsets every position is of the one group)
    c = Case(*shape, seed=6, dst="slots", tail=tail)
    run_forward(m, c, BF16, f"linear {shape}")
    run_dgrad(m, Case(*shape[:3], shape[4], shape[3], seed=6, src="sorted", tail=tail), F32, f"dgrad {shape}")
    c.swiglu, c.w = True, torch.cat([c.w, c.w.flip(1)], dim=1)
    run_forward(m, c, F32, f"linear {shape} swiglu")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda d: "-".join(map(str, d.values())))
def test_wgrad_layouts(m, layout):
    c = Case(77, 3, 12, 200, 136, seed=6, **layout)
    run_wgrad(m, c, F32, f"wgrad {layout}")
    run_wgrad(m, c, F32, f"wgrad {layout} accumulate", accumulate=True)
    run_wgrad(m, c, BF16, f"wgrad {layout} accumulate", accumulate=True)


# ----------------------------------------------------------------------------
# 4-bit weights
# ----------------------------------------------------------------------------
class Q4:
    """Random codes, scales of mixed size and (optionally) zero points for the matrices of a case."""

    def __init__(self, c, group, zero, dtype, seed=11):
        g = torch.Generator().manual_seed(seed)
        n, rows, ng = c.E, c.w.shape[1], c.K // group
        q = torch.randint(0, 16, (n, rows, c.K), generator=g, dtype=torch.uint8)
        self.codes = q[..., 0::2] | (q[..., 1::2] << 4)
        self.scale = ((0.5 + torch.rand(n, rows, ng, generator=g)) * c.K**-0.5 / 8).to(dtype)
        self.zero = torch.randint(0, 16, (n, rows, ng), generator=g, dtype=torch.uint8) if zero else None
        z = torch.full((n, rows, ng), 8.0, dtype=F64) if self.zero is None else self.zero.double()
        per = lambda t: t.repeat_interleave(group, dim=2)
        self.w = (q.double() - per(z)) * per(self.scale.double())
        self.size = 31 * per(self.scale.double().abs())

    def on_gpu(self, m):
        return m.Q4Weights(self.codes.cuda(), self.scale.cuda(), None if self.zero is None else self.zero.cuda())


def run_q4(m, c, q, out_t, what):
    fill = 5.5
    rows = c.R if c.dst == "slots" else c.rows
    whole, out = guarded(rows, c.N, out_t, fill)
    note(f"{what} {out_t}")
    m.moe_q4_linear(c.groups(m), q.on_gpu(m), c.x.cuda(), out, m.ACT_SWIGLU if c.swiglu else m.ACT_NONE)
    torch.cuda.synchronize()
    want, tol, written = forward(c, q.w, q.size, terms=2)
    compare(whole, torch.cat([want, want.new_zeros(3, c.N)]), torch.cat([tol, tol.new_zeros(3, c.N)]), written, fill, what)


Q4_SHAPES = [
    (1, 0, 1, 128, 1), (1, 0, 1, 256, 16), (2, 0, 1, 384, 33), (4, 0, 1, 4096, 48), (5, 0, 1, 512, 64), (16, 0, 1, 1152, 100),
    (17, 0, 1, 256, 37), (40, 0, 1, 640, 130), (64, 0, 1, 256, 256), (65, 0, 1, 128, 31), (200, 0, 1, 384, 96),
    (1, 8, 64, 256, 72), (3, 2, 6, 512, 40), (9, 4, 7, 128, 129), (50, 3, 5, 256, 64), (150, 2, 3, 384, 50),
]


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("group,zero,scale", [(32, True, torch.float16), (64, False, BF16), (128, True, F32),
                                              (32, False, F32), (128, False, torch.float16)],
                         ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("shape", Q4_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_q4(m, shape, group, zero, scale, swiglu):
    c = Case(*shape, seed=7, swiglu=swiglu)
    q = Q4(c, group, zero, scale)
    run_q4(m, c, q, F32, f"q4 {shape} group {group} zero={zero} {scale} swiglu={swiglu}")
    run_q4(m, c, q, BF16, f"q4 {shape} group {group} zero={zero} {scale} swiglu={swiglu}")


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("group,zero,scale", [(32, True, torch.float16), (64, False, F32), (128, True, BF16)],
                         ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("shape", [(1, 0, 1, 128, 32780), (9, 0, 1, 1408, 32801), (16, 0, 1, 256, 33000), (23, 0, 1, 384, 32770),
                                   (33, 0, 1, 640, 32780), (70, 0, 1, 256, 32790), (40, 4, 40, 256, 890), (150, 4, 30, 128, 1300),
                                   (300, 2, 20, 896, 1666), (320, 2, 64, 128, 1100), (600, 2, 40, 1152, 1700)], ids=lambda s: "x".join(map(str, s)))
def test_q4_many_weights(m, shape, group, zero, scale, swiglu):
    """Matrices of many rows or many of them, with one to many rows of x to a group."""
    c = Case(*shape, seed=10, swiglu=swiglu)
    run_q4(m, c, Q4(c, group, zero, scale), F32, f"q4 {shape} group {group} zero={zero} {scale} swiglu={swiglu}")


@pytest.mark.gpu
@pytest.mark.parametrize("group,K", [(32, 96), (64, 192), (32, 1056)])
@pytest.mark.parametrize("T", [2, 20, 70])
def test_q4_many_weights_in_odd_rows(m, T, K, group):
    c = Case(T, 0, 1, K, 32780, seed=10)
    run_q4(m, c, Q4(c, group, True, torch.float16), BF16, f"q4 {T}x{K} group {group}")


@pytest.mark.gpu
@pytest.mark.parametrize("group,K", [(32, 32), (32, 96), (32, 1056), (64, 64), (64, 320)])
@pytest.mark.parametrize("T", [1, 3, 20, 70])
def test_q4_short_and_odd_rows(m, T, K, group):
    """Rows of one group, and of lengths that are no multiple of 128."""
    c = Case(T, 0, 1, K, 45, seed=8)
    run_q4(m, c, Q4(c, group, True, BF16), F32, f"q4 {T}x{K} group {group}")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda d: "-".join(map(str, d.values())))
@pytest.mark.parametrize("T", [1, 30])
def test_q4_layouts(m, T, layout):
    c = Case(T, 3, 12, 256, 80, seed=9, **layout)
    run_q4(m, c, Q4(c, 64, True, torch.float16), F32, f"q4 T={T} {layout}")


# ----------------------------------------------------------------------------
# what stays apart, repeats, graphs, streams
# ----------------------------------------------------------------------------
def all_ops(m, c, q):
    """Every call on one case; name, a function that fills its output, the output."""
    G, x, w, dy, qw = c.groups(m), c.x.cuda(), c.w.cuda(), c.dy.cuda(), q.on_gpu(m)
    rows = c.R if c.dst == "slots" else c.rows
    new = lambda *s: torch.zeros(*s, device="cuda")
    y, s, dx, dw, y4 = new(rows, c.N), new(rows, c.N // 2), new(c.R if c.in_index is not None else c.rows, c.K), new(c.E, c.N, c.K), new(rows, c.N)
    s4 = new(rows, c.N // 2)
    return [("linear", lambda: m.moe_grouped_linear(G, x, w, y), y),
            ("swiglu", lambda: m.moe_grouped_linear(G, x, w, s, m.ACT_SWIGLU), s),
            ("dgrad", lambda: m.moe_grouped_dgrad(G, dy, w, dx), dx),
            ("wgrad", lambda: m.moe_grouped_wgrad(G, x, dy, dw), dw),
            ("q4", lambda: m.moe_q4_linear(G, qw, x, y4), y4),
            ("q4 swiglu", lambda: m.moe_q4_linear(G, qw, x, s4, m.ACT_SWIGLU), s4)], (x, w, dy)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 90])
def test_repeats_and_graph_replays_give_the_same_bits(m, T):
    c = Case(T, 4, 8, 512, 208, dst="slots", seed=12)
    ops, (x, w, dy) = all_ops(m, c, Q4(c, 64, True, torch.float16))
    for name, call, out in ops:
        call()
        torch.cuda.synchronize()
        first = out.clone()
        out.fill_(1.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, first), f"{name}: a repeated call gave other bits"
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            call()
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                call()
        for turn in range(3):
            out.fill_(2.0)
            x.mul_(2.0)                                             # other inputs in the same place, exactly scaled
            dy.mul_(2.0)
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            out.fill_(3.0)
            call()
            torch.cuda.synchronize()
            assert torch.equal(got, out), f"{name}: replay {turn} differs from the eager call"
        x.div_(8.0)
        dy.div_(8.0)


@pytest.mark.gpu
def test_two_streams_at_once(m):
    """Calls that overlap share nothing: no workspace, no counter."""
    cases = [Case(70, 4, 8, 512, 208, seed=s) for s in (13, 14)]
    sets = [all_ops(m, c, Q4(c, 32, True, BF16, seed=s)) for s, c in enumerate(cases)]
    want = []
    for ops, _ in sets:
        for _, call, out in ops:
            call()
        torch.cuda.synchronize()
        want.append([o.clone() for _, _, o in ops])
        for _, _, o in ops:
            o.fill_(4.0)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(len(sets[0][0])):
            for s, (ops, _) in zip(streams, sets):
                with torch.cuda.stream(s):
                    ops[i][1]()
    torch.cuda.synchronize()
    for (ops, _), w in zip(sets, want):
        for (name, _, out), t in zip(ops, w):
            assert torch.equal(out, t), name


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(6, 2, 4), (120, 2, 3)])
def test_non_finite_values_stay_in_their_rows_and_groups(m, T, k, E):
    """NaN and infinities in one row of x or dy reach that row's results only, in one matrix its own rows only."""
    c = Case(T, k, E, 136, 72, src="sorted", seed=15)
    clean = Case(T, k, E, 136, 72, src="sorted", seed=15)
    p = c.begin[1]                                                  # group 1's first position
    assert c.counts[1] > 1
    c.x[p, 5], c.x[p, 100], c.dy[p, 3], c.w[2, 7, 9] = float("nan"), float("inf"), float("-inf"), float("nan")
    for name in ("linear", "dgrad"):
        got = []
        for d in (c, clean):
            out = torch.zeros(d.rows, d.N if name == "linear" else d.K, device="cuda")
            note(f"non-finite {name}")
            if name == "linear":
                m.moe_grouped_linear(d.groups(m), d.x.cuda(), d.w.cuda(), out)
            else:
                m.moe_grouped_dgrad(d.groups(m), d.dy.cuda(), d.w.cuda(), out)
            torch.cuda.synchronize()
            got.append(out.cpu())
        spoiled = [p] + list(range(c.begin[2], c.begin[3]))
        rest = [i for i in range(c.rows) if i not in spoiled]
        assert torch.equal(got[0][rest], got[1][rest]), name
        assert not got[0][p].isfinite().all()
        # a NaN weight touches its own output column only (dgrad: its own input column)
        cols = [j for j in range(got[0].shape[1]) if j != (7 if name == "linear" else 9)]
        rows = list(range(c.begin[2], c.begin[3]))
        assert torch.equal(got[0][rows][:, cols], got[1][rows][:, cols]), name
    got = []
    for d in (c, clean):
        dw = torch.zeros(E, d.N, d.K, device="cuda")
        m.moe_grouped_wgrad(d.groups(m), d.x.cuda(), d.dy.cuda(), dw)
        torch.cuda.synchronize()
        got.append(dw.cpu())
    for e in range(E):
        if e != 1:
            assert torch.equal(got[0][e], got[1][e])
    clean_cols = [j for j in range(c.K) if j not in (5, 100)]
    clean_rows = [j for j in range(c.N) if j != 3]
    assert torch.equal(got[0][1][clean_rows][:, clean_cols], got[1][1][clean_rows][:, clean_cols])
    assert got[0][1][:, 5].isnan().all() and not got[0][1][3].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(6, 4), (1500, 2)])
def test_wgrad_leaves_out_positions_without_either_row(m, T, E):
    """A position without a row of x, or of dy, adds nothing: not even where the other row is not finite."""
    c = Case(T, 2, E, 136, 72, dst="slots", seed=20)
    c.in_index, c.out_index = c.perm.clone(), c.perm.clone()
    c.x = c.x.repeat_interleave(2, 0)                               # a row of its own for every slot
    no_x, no_dy = (next(b + i for e, b in enumerate(c.begin[:-1]) if c.counts[e] > 1) for i in (0, 1))
    c.dy[int(c.perm[no_x])], c.x[int(c.perm[no_dy])] = float("nan"), float("inf")
    c.in_index[no_x], c.out_index[no_dy] = -1, -1
    groups = m.RowGroups(c.rows, offsets=c.offsets.cuda(), in_index=c.in_index.cuda(), out_index=c.out_index.cuda())
    for dtype in (F32, BF16):
        dw = torch.full((c.E, c.N, c.K), 7.0, dtype=dtype, device="cuda")
        note(f"wgrad without either row {T} {dtype}")
        m.moe_grouped_wgrad(groups, c.x.cuda(), c.dy.cuda(), dw)
        torch.cuda.synchronize()
        for e in range(c.E):
            p = [i for i in c.positions(e) if i not in (no_x, no_dy)]
            x, dy = (v[[int(c.perm[i]) for i in p]].double() for v in (c.x, c.dy))
            want, tol = dy.T @ x, (len(p) + 1) * 2.0**-23 * (dy.abs().T @ x.abs())
            if dtype == BF16:
                tol = tol + 2.0**-8 * want.abs()
            assert ((dw[e].cpu().double() - want).abs() <= tol).all()


@pytest.mark.gpu
def test_many_overlapping_groups_touch_nothing_outside(m):
    """4096 groups, every second one of all rows: far more tiles than a launch is made for."""
    R, E, N, K = 300, 4096, 8, 32
    offsets = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    groups = m.RowGroups(R, offsets=offsets)
    x = torch.ones(R, K, dtype=BF16, device="cuda")
    w = torch.ones(E, N, K, dtype=BF16, device="cuda")
    q = m.Q4Weights(torch.full((E, N, K // 2), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(E, N, 1, device="cuda"))
    for name, call in (("linear", lambda out: m.moe_grouped_linear(groups, x, w, out)),
                       ("q4", lambda out: m.moe_q4_linear(groups, q, x, out))):
        whole, out = guarded(R, N, F32, 7.0)
        note(f"overlapping groups {name}")
        call(out)
        torch.cuda.synchronize()
        assert (whole[R:] == 7.0).all() and ((out == 7.0) | (out == float(K))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("kind", ["bf16", "q4"])
def test_swiglu_of_large_and_infinite_gates(m, T, kind):
    """Gates of either sign from 2^-100 to 2^100 and (bf16 weights) past the largest float: no overflow on the way reaches the
    result. x[0] is the gate and x[1] the other half."""
    g = torch.Generator().manual_seed(21)
    K, N = 64, 16
    x = torch.zeros(T, K, dtype=BF16)
    out = torch.zeros(T, N, device="cuda")
    w = torch.zeros(1, 2 * N, K)
    scale = torch.exp2(torch.linspace(-100, 100, N).round())
    scale[4:8] = torch.tensor([64.0, 90.0, 2.0**24, 2.0**26])       # where silu leaves the floats, and 2e7 and more
    w[0, :N, 0], w[0, N:, 1] = scale, 1.0
    x[:, 0] = torch.randn(T, generator=g).to(BF16)
    x[::2, 0] = -x[::2, 0].abs()
    x[:, 1] = torch.randn(T, generator=g).to(BF16)
    groups = m.RowGroups(T)
    note(f"large gates {T} {kind}")
    if kind == "bf16":
        w[0, N - 1, 0] = 3e38                                       # with an x of 4 the sum overflows
        w = w.to(BF16)
        if T > 1:
            x[1, 0] = 4.0
        m.moe_grouped_linear(groups, x.cuda(), w.cuda(), out, m.ACT_SWIGLU)
    else:
        w = w.to(BF16)
        codes = torch.full((1, 2 * N, K), 8, dtype=torch.uint8)
        codes[0, :N, 0] = codes[0, N:, 1] = 9
        s = torch.ones(1, 2 * N, K // 32)
        s[0, :N, 0] = w[0, :N, 0].float()
        m.moe_q4_linear(groups, m.Q4Weights((codes[..., ::2] | codes[..., 1::2] << 4).contiguous().cuda(), s.cuda()), x.cuda(), out,
                        m.ACT_SWIGLU)
    torch.cuda.synchronize()
    gate = (x[:, :1].double() * w[0, :N, 0].double()).float().double()      # one product of each sum is not zero
    want = gate * torch.sigmoid(gate) * x[:, 1:2].double()
    got = out.cpu().double()
    finite = want.abs() < 3e38
    assert ((got - want).abs()[finite] <= (2.0**-20 * want.abs() + 1e-35)[finite]).all()
    large = want.abs() >= 3e38                                       # a gate of -inf: -inf * 0
    assert torch.equal(got[large].sign(), want[large].sign()) and (got[large].abs() > 2.9e38).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
def test_rows_and_results_behind_4_gib(m, T):
    """Rows of x, of the output and of dy and weights whose byte offsets pass 32 bits, against the same rows in small buffers."""
    far, wide, K, N = 2**17 + 7, 2**14 + 64, 128, 136               # far x wide: 4.3 GB of bf16
    g = torch.Generator(device="cuda").manual_seed(22)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    big, near = torch.empty(far, wide, dtype=BF16, device="cuda"), normal(T, wide)
    rows = far - 1 - 2 * torch.arange(T, device="cuda")
    big[rows] = near
    index, one = rows.to(torch.int32), lambda **kw: m.RowGroups(T, **kw)
    w, wt = normal(1, N, wide), normal(1, wide, K)
    q = m.Q4Weights(torch.randint(0, 256, (1, N, wide // 2), generator=g, device="cuda", dtype=torch.uint8),
                    torch.rand(1, N, wide // 32, generator=g, device="cuda"))
    note(f"behind 4 GiB {T}: inputs")
    for cols, side, call in ((N, "in_index", lambda G, x, out: m.moe_grouped_linear(G, x, w, out)),
                             (N, "in_index", lambda G, x, out: m.moe_q4_linear(G, q, x, out)),
                             (K, "out_index", lambda G, x, out: m.moe_grouped_dgrad(G, x, wt, out))):
        got, want = (torch.zeros(T, cols, device="cuda") for _ in range(2))
        call(one(**{side: index}), big, got)
        call(one(), near, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and want.abs().max() > 0
    dw, dw0 = (torch.zeros(1, K, wide, device="cuda") for _ in range(2))
    dy = normal(T, K)
    m.moe_grouped_wgrad(one(in_index=index), big, dy, dw)
    m.moe_grouped_wgrad(one(), near, dy, dw0)
    torch.cuda.synchronize()
    assert torch.equal(dw, dw0) and dw.abs().max() > 0
    note(f"behind 4 GiB {T}: results")
    x, out = normal(T, K), torch.zeros(T, wide, dtype=BF16, device="cuda")
    big.zero_()
    m.moe_grouped_linear(one(out_index=index), x, wt, big)
    m.moe_grouped_linear(one(), x, wt, out)
    torch.cuda.synchronize()
    assert torch.equal(big[rows], out) and out.abs().max() > 0
    assert not big[rows - 1].any() and not big[:100].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 50])
def test_q4_non_finite_values_stay_in_their_rows(m, T):
    c = Case(T, 0, 1, 256, 40, seed=16)
    q = Q4(c, 64, True, F32)
    got = []
    for spoil in (False, True):
        if spoil:
            c.x[1, 17] = float("inf")
            q.scale[0, 3, 2] = float("nan")
        out = torch.zeros(T, 40, device="cuda")
        m.moe_q4_linear(c.groups(m), q.on_gpu(m), c.x.cuda(), out)
        torch.cuda.synchronize()
        got.append(out.cpu())
    rows, cols = [i for i in range(T) if i != 1], [j for j in range(40) if j != 3]
    assert torch.equal(got[0][rows][:, cols], got[1][rows][:, cols])
    assert got[1][:, 3].isnan().all() and not got[1][1].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 40])
def test_indices_outside_the_buffers(m, T):
    """An input row outside x counts as zeros; an output row outside the output is not written."""
    c = Case(T, 2, 4, 128, 64, dst="slots", seed=17)
    c.in_index, c.out_index = c.perm.clone(), c.perm.clone()
    bad_in, bad_out = c.begin[1] if c.counts[1] else 0, c.rows - 1
    lost = int(c.out_index[bad_out])
    c.in_index[bad_in], c.out_index[bad_out] = -5, 10**9
    whole, out = guarded(c.R, c.N, F32, 7.0)
    m.moe_grouped_linear(c.groups(m), c.x.cuda(), c.w.cuda(), out)
    q = Q4(c, 32, False, F32)
    whole4, out4 = guarded(c.R, c.N, F32, 7.0)
    m.moe_q4_linear(c.groups(m), q.on_gpu(m), c.x.cuda(), out4)
    wholeg, dx = guarded(c.R, c.K, F32, 7.0)
    m.moe_grouped_dgrad(c.groups(m), c.dy.cuda(), c.w.cuda(), dx)
    dw = torch.zeros(c.E, c.N, c.K, device="cuda")
    m.moe_grouped_wgrad(c.groups(m), c.x.cuda(), c.dy.cuda(), dw)
    torch.cuda.synchronize()
    for w in (whole, whole4):
        w = w.cpu()
        assert (w[lost] == 7.0).all() and (w[c.R:] == 7.0).all()
        zero = int(c.out_index[bad_in])
        if bad_in != bad_out:
            assert (w[zero] == 0.0).all()
    kept = [p for p in range(c.rows) if p not in (bad_in, bad_out)]
    for e in range(c.E):
        p = [i for i in c.positions(e) if i in kept]
        x, dy = c.x[[c.r(i) for i in p]].double(), c.dy[[c.o(i) for i in p]].double()
        assert torch.allclose(whole.cpu()[[c.o(i) for i in p]].double(), x @ c.w[e].double().T, atol=1e-4)
        assert torch.allclose(dw[e].cpu().double(), dy.T @ x, atol=1e-3)
    slot = int(c.perm[bad_in])
    assert (wholeg.cpu()[slot] == 7.0).all() and (wholeg.cpu()[c.R:] == 7.0).all()


@pytest.mark.gpu
def test_offsets_that_decrease_or_leave_the_rows_touch_nothing_outside(m):
    c = Case(40, 2, 4, 64, 72, seed=18)
    c.offsets = torch.tensor([-9, 50, 20, 2**31 - 1, 60], dtype=torch.int32)
    q = Q4(c, 32, True, F32)
    for name, shape, call in (
            ("linear", (c.rows, c.N), lambda o: m.moe_grouped_linear(c.groups(m), c.x.cuda(), c.w.cuda(), o)),
            ("dgrad", (c.R, c.K), lambda o: m.moe_grouped_dgrad(c.groups(m), c.dy.cuda(), c.w.cuda(), o)),
            ("wgrad", (c.E * c.N, c.K), lambda o: m.moe_grouped_wgrad(c.groups(m), c.x.cuda(), c.dy.cuda(), o.view(c.E, c.N, c.K))),
            ("q4", (c.rows, c.N), lambda o: m.moe_q4_linear(c.groups(m), q.on_gpu(m), c.x.cuda(), o))):
        whole, out = guarded(*shape, F32, 7.0)
        note(name)
        call(out)
        torch.cuda.synchronize()
        assert (whole[shape[0]:] == 7.0).all(), name


# ----------------------------------------------------------------------------
# as they are used together
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("T", [1, 3, 150])
def test_layer_of_unquantized_or_4bit_experts(m, T, kind):
    """moe_route, gate/up with SwiGLU, down into slot order, moe_combine, against binary64 on the routing's choices.
    Tolerance (2-norm per token): h is rounded to bf16, 2^-8 / sqrt(3) of the result's terms; the rest is fp32."""
    H, I, E, k = 512, 256, 16, 4
    g = torch.Generator().manual_seed(21)
    x = torch.randn(T, H, generator=g).to(BF16)
    wr = (torch.randn(E, H, generator=g) * 0.05).to(BF16)
    up, down = Case(T, k, E, H, I, swiglu=True, seed=22), Case(T, k, E, I, H, seed=23)
    q_up, q_down = (Q4(up, 32, True, torch.float16), Q4(down, 64, False, BF16)) if kind == "q4" else (None, None)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, off, perm, act = (torch.empty(n, **i32) for n in (T * k, E + 1, T * k, E + 1))
    tw, xd = torch.empty(T, k, device="cuda"), x.cuda()
    ws = torch.empty(m.moe_route_workspace(T, E, k), dtype=torch.uint8, device="cuda")
    h = torch.empty(T * k, I, dtype=BF16, device="cuda")
    slots, y = torch.empty(T * k, H, device="cuda"), torch.empty(T, H, device="cuda")
    m.moe_route(xd, wr.cuda(), E, k, idx, tw, off, perm, act, ws)
    first = m.RowGroups(T * k, offsets=off, in_index=perm, in_div=k)
    second = m.RowGroups(T * k, offsets=off, out_index=perm)
    if kind == "q4":
        m.moe_q4_linear(first, q_up.on_gpu(m), xd, h, m.ACT_SWIGLU)
        m.moe_q4_linear(second, q_down.on_gpu(m), h, slots)
        wu, wd = q_up.w, q_down.w
    else:
        m.moe_grouped_linear(first, xd, up.w.cuda(), h, m.ACT_SWIGLU)
        m.moe_grouped_linear(second, h, down.w.cuda(), slots)
        wu, wd = up.w.double(), down.w.double()
    m.moe_combine(slots, tw, None, T, k, H, y)
    torch.cuda.synchronize()
    idx, tw, got = idx.cpu().view(T, k), tw.cpu().double(), y.cpu().double()
    for t in range(T):
        want, size = torch.zeros(H, dtype=F64), torch.zeros(H, dtype=F64)
        for j in range(k):
            e = int(idx[t, j])
            z = wu[e] @ x[t].double()
            v = z[:I] * torch.sigmoid(z[:I]) * z[I:]
            want += tw[t, j] * (wd[e] @ v)
            size += tw[t, j]**2 * (wd[e].square() @ v.square())
        assert (got[t] - want).norm() <= 2.0**-8 * size.sqrt().norm(), t


@pytest.mark.gpu
def test_training_step_of_two_products(m):
    """Forward, both gradients of both products, and the gradient of tokens read by several slots, against binary64
    automatic differentiation.  Tolerance (2-norm): bf16 copies of h, dh and the SwiGLU's gradients, four roundings of
    2^-8 at most each."""
    T, k, E, H, I = 60, 2, 6, 256, 136
    c = Case(T, k, E, H, 2 * I, seed=31)
    d = Case(T, k, E, I, H, src="sorted", dst="slots", seed=31)
    assert torch.equal(c.perm, d.perm) and c.begin == d.begin
    gc, gd = c.groups(m), d.groups(m)
    x, wu, wd, dy = c.x.cuda(), c.w.cuda(), d.w.cuda(), d.dy.cuda()
    z = torch.empty(T * k, 2 * I, device="cuda")
    m.moe_grouped_linear(gc, x, wu, z)
    gate, upv = z[:, :I], z[:, I:]
    s = torch.sigmoid(gate)
    h = (gate * s * upv).to(BF16)
    y = torch.empty(T * k, H, device="cuda")
    m.moe_grouped_linear(gd, h, wd, y)
    dh, dwd = torch.empty(T * k, I, device="cuda"), torch.empty_like(wd, dtype=F32)
    m.moe_grouped_dgrad(gd, dy, wd, dh)
    m.moe_grouped_wgrad(gd, h, dy, dwd)
    dz = torch.cat([dh * upv * s * (1 + gate * (1 - s)), dh * gate * s], dim=1).to(BF16)
    dslots, dwu = torch.empty(T * k, H, device="cuda"), torch.empty_like(wu, dtype=F32)
    m.moe_grouped_dgrad(gc, dz, wu, dslots)
    m.moe_grouped_wgrad(gc, x, dz, dwu)
    dx = torch.empty(T, H, device="cuda")
    m.moe_combine(dslots, torch.ones(T, k, device="cuda"), None, T, k, H, dx)
    torch.cuda.synchronize()
    xr, wur, wdr = (t.double().requires_grad_() for t in (c.x, c.w, d.w))
    total = 0.0
    for e in range(E):
        p = c.positions(e)
        zz = xr[[c.r(i) for i in p]] @ wur[e].T
        hh = torch.nn.functional.silu(zz[:, :I]) * zz[:, I:]
        total = total + (d.dy[[d.o(i) for i in p]].double() * (hh @ wdr[e].T)).sum()
    total.backward()
    for name, got, want in (("dx", dx, xr.grad), ("dwu", dwu, wur.grad), ("dwd", dwd, wdr.grad)):
        err = float((got.cpu().double() - want).norm() / want.norm())
        note(f"{name} {err:.2e}")
        assert err <= 4 * 2.0**-8, name


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 100])
def test_gradients_against_differences(m, T):
    """The product is linear in x and in W: a step of one element changes it by its gradient exactly, up to fp32 sums."""
    c = Case(T, 2, 4, 72, 40, seed=41)
    G, w, dy = c.groups(m), c.w.cuda(), c.dy.cuda()

    def loss(x, w):
        y = torch.empty(c.rows, c.N, device="cuda")
        m.moe_grouped_linear(G, x, w, y)
        return float((y.double() * dy.double()).sum())

    dslots, dw = torch.empty(c.R, c.K, device="cuda"), torch.empty(c.E, c.N, c.K, device="cuda")
    m.moe_grouped_dgrad(G, dy, w, dslots)
    m.moe_grouped_wgrad(G, c.x.cuda(), dy, dw)
    dx = dslots.view(T, 2, c.K).sum(dim=1)
    base = c.x.cuda()
    # sums of some 10^4 terms of size 1 in fp32 rows: 10^2 * 2^-24 * sqrt(72) each way, over a step of 4
    for t, j in ((0, 0), (T - 1, c.K - 1), (T // 2, 17)):
        up, dn = base.clone(), base.clone()
        up[t, j], dn[t, j] = 2.0, -2.0
        assert abs((loss(up, w) - loss(dn, w)) / 4 - float(dx[t, j])) < 1e-3
    for e, n, j in ((0, 0, 0), (3, 39, 71), (1, 20, 33)):
        up, dn = w.clone(), w.clone()
        up[e, n, j], dn[e, n, j] = 2.0, -2.0
        assert abs((loss(base, up) - loss(base, dn)) / 4 - float(dw[e, n, j])) < 1e-3


# ----------------------------------------------------------------------------
# refusals (no GPU)
# ----------------------------------------------------------------------------
@pytest.fixture(scope="module")
def host():
    if not os.path.exists(LIB):
        pytest.skip("libmoe2bit.so not built")
    import bit_quantized_moe_permute_amd as m
    return m


P = 0x100000                                                        # never dereferenced


def desc(m, **kw):
    return m.GroupDesc(**{**dict(n_groups=4, n_rows=64, offsets=P, in_index=P, in_div=2, out_index=P), **kw})


def refused(m, status, text, call, *args):
    st = call(*args)
    msg = m.moe_last_error()
    assert st == status and text in msg, (st, msg)


def test_group_descriptions_are_checked(host):
    m, f = host, host.lib.moe_grouped_linear
    A, B, O = 0x10000000, 0x20000000, 0x30000000
    call = lambda g, st, text: refused(m, st, text, f, g, A, 32, B, 64, 64, 0, O, 0, 64, None)
    call(None, 1, "null group")
    call(desc(m, n_groups=0), 1, "n_groups")
    call(desc(m, n_groups=4097), 1, "n_groups")
    call(desc(m, n_rows=0), 1, "n_rows")
    call(desc(m, n_rows=-3), 1, "n_rows")
    call(desc(m, n_rows=(1 << 24) + 1), 2, "n_rows")
    call(desc(m, offsets=None), 1, "offsets")
    call(desc(m, in_div=0), 1, "in_div")
    call(desc(m, in_index=P + 2), 1, "misaligned")
    call(desc(m, out_index=P + 1), 1, "misaligned")
    call(desc(m, offsets=O + 64), 1, "overlaps")
    call(desc(m, in_index=O), 1, "overlaps")


def test_products_are_checked(host):
    m = host
    g, A, B, O = desc(m), 0x10000000, 0x20000000, 0x30000000
    for f, wide in ((m.lib.moe_grouped_linear, True), (m.lib.moe_grouped_dgrad, False)):
        def call(st, text, a=A, ar=32, b=B, n=64, k=64, act=0, o=O, dt=0, orows=64):
            args = (g, a, ar, b, n, k, act, o, dt, orows, None) if wide else (g, a, ar, b, n, k, o, dt, orows, None)
            refused(m, st, text, f, *args)
        call(1, "null", a=None)
        call(1, "null", b=None)
        call(1, "null", o=None)
        call(1, "misaligned", a=A + 2)
        call(1, "misaligned", b=B + 8)
        call(1, "misaligned", o=O + 4)
        call(1, "without rows", ar=0)
        call(1, "without rows", orows=0)
        call(1, "multiples of 8", n=60)
        call(1, "multiples of 8", k=0)
        call(2, "above", n=(1 << 20) + 8)
        call(2, "above", k=(1 << 20) + 8)
        call(1, "dtype", dt=2)
        call(1, "dtype", dt=4)
        call(1, "overlaps", o=A + 64)
        call(1, "overlaps", o=B + 4 * 64 * 64 * 2 - 16)
        if wide:
            call(1, "activation", act=2)
            call(1, "overlaps", act=1, o=B + 2 * 4 * 64 * 64 * 2 - 16)
    f = m.lib.moe_grouped_wgrad

    def call(st, text, x=A, xr=32, dy=B, dyr=64, n=64, k=64, o=O, dt=0):
        refused(m, st, text, f, g, x, xr, dy, dyr, n, k, 0, o, dt, None)
    call(1, "null", x=None)
    call(1, "null", dy=None)
    call(1, "without rows", xr=0)
    call(1, "without rows", dyr=-1)
    call(1, "multiples of 8", k=12)
    call(1, "misaligned", o=O + 8)
    call(1, "dtype", dt=3)
    call(1, "overlaps", o=A)
    call(1, "overlaps", o=B + 64)


def test_q4_weights_are_checked(host):
    m, f = host, host.lib.moe_q4_linear
    A, O, C, S, Z = 0x10000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000

    def call(st, text, act=0, x=A, xr=32, o=O, dt=0, orows=64, groups=None, **kw):
        w = m.Q4Desc(**{**dict(n_mats=4, rows=48, cols=256, group=64, scale_dt=0, codes=C, scale=S, zero=Z), **kw})
        refused(m, st, text, f, groups or desc(m), w, x, xr, act, o, dt, orows, None)
    refused(m, 1, "null", f, desc(m), None, A, 32, 0, O, 0, 64, None)
    call(1, "null", codes=None)
    call(1, "null", scale=None)
    call(1, "null", x=None)
    call(1, "null", o=None)
    call(1, "matrices", n_mats=3)
    call(1, "group must", group=16)
    call(1, "group must", group=256)
    call(1, "multiple of group", cols=224)
    call(1, "multiple of group", cols=0)
    call(1, "multiple of group", rows=0)
    call(1, "even", rows=47, act=1)
    call(1, "activation", act=5)
    call(2, "above", cols=(1 << 20) + 64)
    call(2, "above", rows=(1 << 20) + 1)
    call(1, "dtype", scale_dt=2)
    call(1, "dtype", dt=4)
    call(1, "misaligned", x=A + 8)
    call(1, "misaligned", codes=C + 8)
    call(1, "misaligned", scale=S + 2)
    call(1, "misaligned", o=O + 2)
    call(1, "without rows", xr=0)
    call(1, "without rows", orows=0)
    call(1, "overlaps", o=C + 4 * 48 * 128 - 16)
    call(1, "overlaps", o=S)
    call(1, "overlaps", o=Z)
    call(1, "overlaps", o=A)


@pytest.mark.parametrize("value", [0, -1, 2**31, 2**32 + 4])
def test_row_counts_are_int32(host, value):
    """A number that an int32 does not hold is refused, not cut."""
    with pytest.raises(ValueError, match="n_rows"):
        host.RowGroups(value)
    with pytest.raises(ValueError, match="in_div"):
        host.RowGroups(4, in_div=value)


def test_binding_checks(host):
    m = host
    with pytest.raises(TypeError, match="GPU tensor"):
        m.RowGroups(4, offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="GPU tensor"):
        m.Q4Weights(torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(2, 16, 2))
    with pytest.raises(ValueError, match="32, 64 or 128"):
        m.Q4Weights(torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(2, 16, 8))
    G = m.RowGroups(4)
    x, w = torch.zeros(4, 16, dtype=BF16), torch.zeros(1, 8, 16, dtype=BF16)
    with pytest.raises(TypeError, match="GPU tensor"):
        m.moe_grouped_linear(G, x, w, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="must be"):
        m.moe_grouped_linear(G, x, w, torch.zeros(4, 16))
    with pytest.raises(ValueError, match="must be"):
        m.moe_grouped_linear(G, x[:, :8], w, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="must be"):
        m.moe_grouped_linear(G, x, w[0], torch.zeros(4, 8))
    with pytest.raises(TypeError, match="bfloat16"):
        m.moe_grouped_linear(G, x.float(), w, torch.zeros(4, 8))
    with pytest.raises(TypeError, match="bfloat16"):
        m.moe_grouped_linear(G, x, w.float(), torch.zeros(4, 8))
    with pytest.raises(TypeError, match="dtype"):
        m.moe_grouped_linear(G, x, w, torch.zeros(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="even"):
        m.moe_grouped_linear(G, x, torch.zeros(1, 7, 16, dtype=BF16), torch.zeros(4, 3), m.ACT_SWIGLU)
    with pytest.raises(ValueError, match="must be"):
        m.moe_grouped_dgrad(G, torch.zeros(4, 16, dtype=BF16), w, torch.zeros(4, 16))
    with pytest.raises(ValueError, match="must be"):
        m.moe_grouped_wgrad(G, x, torch.zeros(4, 8, dtype=BF16), torch.zeros(8, 16))


@pytest.mark.gpu
def test_binding_checks_on_the_gpu(m):
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="int32"):
        m.RowGroups(4, offsets=off.long())
    with pytest.raises(ValueError, match="contiguous"):
        m.RowGroups(2, offsets=off, in_index=torch.zeros(4, dtype=torch.int32, device="cuda")[::2])
    with pytest.raises(ValueError, match="need as many"):
        m.RowGroups(4, offsets=off, in_index=torch.zeros(3, dtype=torch.int32, device="cuda"))
    G = m.RowGroups(4, offsets=off)
    x, w, out = (torch.zeros(*s, dtype=BF16, device="cuda") for s in ((4, 16), (2, 8, 16), (4, 8)))
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_grouped_linear(G, torch.zeros(4, 32, dtype=BF16, device="cuda")[:, ::2], w, out)
    with pytest.raises(m.MoeError, match="misaligned"):
        m.moe_grouped_linear(G, torch.zeros(65, dtype=BF16, device="cuda")[1:].view(4, 16), w, out)
    with pytest.raises(m.MoeError, match="overlaps"):
        m.moe_grouped_linear(G, x, w, w.view(-1)[:32].view(4, 8))
    codes = torch.zeros(2, 8, 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="scale"):
        m.Q4Weights(codes, torch.zeros(2, 8, 1, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="zero"):
        m.Q4Weights(codes, torch.zeros(2, 8, 1, device="cuda"), torch.zeros(2, 8, 2, dtype=torch.uint8, device="cuda"))
    q = m.Q4Weights(codes[0], torch.zeros(8, 1, device="cuda"))
    assert (q.n, q.rows, q.cols, q.group) == (1, 8, 32, 32)
    with pytest.raises(m.MoeError, match="matrices"):
        m.moe_q4_linear(G, q, torch.zeros(4, 32, dtype=BF16, device="cuda"), out)
