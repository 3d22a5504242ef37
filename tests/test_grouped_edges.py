"""The grouped products at the edges of what their contract allows: routings that change under a captured call, no positions at all,
divisors and indices of any size, scales and zero points at any alignment, the largest sizes.

Tolerances are those of test_grouped.py (its docstring derives them)."""
import pytest
import torch

from test_grouped import BF16, F32, Q4, Case, guarded, note, swiglu
from test_grouped_paths import near, product


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import bit_quantized_moe_permute_amd as m
    return m


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 30, 400])
def test_captured_calls_follow_a_routing_that_changes_in_place(m, T):
    """Offsets and permutation of another batch in the same buffers, fewer positions than the description has room for among them."""
    c = Case(T, 4, 8, 512, 208, dst="slots", seed=71)
    others = [Case(T, 4, 8, 512, 208, dst="slots", seed=s, some=n) for s, n in ((72, None), (73, 4), (74, None))]
    off, perm = c.offsets.cuda(), c.perm.cuda()
    G = m.RowGroups(c.rows, offsets=off, in_index=perm, in_div=4, out_index=perm)
    x, w, dy, q = c.x.cuda(), c.w.cuda(), c.dy.cuda(), Q4(c, 64, True, torch.float16).on_gpu(m)
    new = lambda *s: torch.zeros(*s, device="cuda")
    outs = dict(linear=new(c.R, 208), swiglu=new(c.R, 104), dgrad=new(c.R, 512), wgrad=new(8, 208, 512), q4=new(c.R, 208))

    def calls():
        m.moe_grouped_linear(G, x, w, outs["linear"])
        m.moe_grouped_linear(G, x, w, outs["swiglu"], m.ACT_SWIGLU)
        m.moe_grouped_dgrad(G, dy, w, outs["dgrad"])
        m.moe_grouped_wgrad(G, x, dy, outs["wgrad"])
        m.moe_q4_linear(G, q, x, outs["q4"])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            calls()
    note(f"routing changes {T}")
    for turn, d in enumerate(others + [others[0], None]):
        if d is None:                                               # half of the positions
            off.copy_((c.offsets.cuda() // 2).to(torch.int32))
        else:
            off.copy_(d.offsets.cuda())
            perm.copy_(d.perm.cuda())
        got = []
        for run in (graph.replay, calls):
            for o in outs.values():
                o.fill_(3.0)
            run()
            torch.cuda.synchronize()
            got.append({k: o.clone() for k, o in outs.items()})
        for k in outs:
            assert torch.equal(got[0][k], got[1][k]), (turn, k)
        if d is not None:
            for e in range(8):
                p = d.positions(e)
                if p:
                    rows, tok = [d.o(i) for i in p], [d.r(i) for i in p]
                    near(got[0]["linear"][rows], *product(x[tok], w[e]), f"linear {turn} {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("n,rows", [(1, 5), (3, 70), (300, 4000)])
def test_no_positions_at_all(m, n, rows):
    """Offsets that name none: nothing is written, the weights' gradient is zero or stays."""
    K, N = 128, 144
    off = torch.full((n + 1,), 3, dtype=torch.int32, device="cuda")
    G = m.RowGroups(rows, offsets=off)
    g = torch.Generator(device="cuda").manual_seed(75)
    x, dy, w = randn(g, rows, K), randn(g, rows, N), randn(g, n, N, K)
    q = m.Q4Weights(torch.zeros(n, N, K // 2, dtype=torch.uint8, device="cuda"), torch.ones(n, N, K // 32, device="cuda"))
    note(f"no positions {n} {rows}")
    for cols, call in ((N, lambda o: m.moe_grouped_linear(G, x, w, o)), (N // 2, lambda o: m.moe_grouped_linear(G, x, w, o, m.ACT_SWIGLU)),
                       (K, lambda o: m.moe_grouped_dgrad(G, dy, w, o)), (N, lambda o: m.moe_q4_linear(G, q, x, o))):
        whole, out = guarded(rows, cols, F32, 7.0)
        call(out)
        torch.cuda.synchronize()
        assert (whole == 7.0).all()
    dw = torch.full((n, N, K), 7.0, device="cuda")
    m.moe_grouped_wgrad(G, x, dy, dw, accumulate=True)
    torch.cuda.synchronize()
    assert (dw == 7.0).all()
    m.moe_grouped_wgrad(G, x, dy, dw)
    torch.cuda.synchronize()
    assert not dw.any()


@pytest.mark.gpu
@pytest.mark.parametrize("div", [1, 2, 3, 5, 6, 7, 10, 127, 641, 65535, 65537, 10**6 + 3, 10**9, 2**30 - 1, 2**30, 2**30 + 1, 2**31 - 1])
def test_divisors_of_the_input_index(m, div):
    """Row in_index / in_div, rounded down, for indices around every multiple that an int32 holds (or 200 of them)."""
    last = (2**31 - 1) // div
    multiples = sorted({*range(min(last, 100) + 1), *(last - i for i in range(min(last, 100) + 1))})
    index = sorted({i for v in multiples for i in (v * div - 1, v * div, v * div + 1, v * div + div - 1) if 0 <= i < 2**31})
    rows = [i // div for i in index]
    low = min(max(rows), 120)                                       # x has rows 0 .. low; the others count as zeros
    x = torch.zeros(low + 1, 32, dtype=BF16, device="cuda")
    x[:, 0] = torch.arange(1, low + 2)
    w = torch.zeros(1, 8, 32, dtype=BF16, device="cuda")
    w[0, 0, 0] = 1.0
    codes = torch.full((1, 8, 16), 0x88, dtype=torch.uint8, device="cuda")
    codes[0, 0, 0] = 0x89
    G = m.RowGroups(len(index), in_index=torch.tensor(index, dtype=torch.int32, device="cuda"), in_div=div)
    want = torch.tensor([r + 1.0 if r <= low else 0.0 for r in rows])
    for call in (lambda o: m.moe_grouped_linear(G, x, w, o),
                 lambda o: m.moe_q4_linear(G, m.Q4Weights(codes, torch.ones(1, 8, 1, device="cuda")), x, o)):
        out = torch.full((len(index), 8), 7.0, device="cuda")
        call(out)
        torch.cuda.synchronize()
        assert torch.equal(out[:, 0].cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, BF16, F32], ids=lambda t: str(t).replace("torch.", ""))
@pytest.mark.parametrize("T,N,K,group", [(3, 50, 1056, 32), (70, 1300, 1056, 32), (497, 1290, 2240, 64), (330, 1290, 7936, 128), (2090, 1290, 96, 32)])
def test_scales_and_zero_points_at_any_alignment(m, T, N, K, group, dtype):
    """Scales aligned to their elements, zero points to bytes: the same bits as from aligned ones."""
    c = Case(T, 0, 1, K, N, seed=76)
    q = Q4(c, group, True, dtype)
    x, G = c.x.cuda(), c.groups(m)
    codes = q.codes.cuda()

    def shifted(t, by):
        flat = torch.empty(t.numel() + by + 8, dtype=t.dtype, device="cuda")
        v = flat[by:by + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    want = torch.empty(T, N, device="cuda")
    note(f"alignment {T} {N} {K} {group} {dtype}")
    m.moe_q4_linear(G, m.Q4Weights(codes, q.scale.cuda(), q.zero.cuda()), x, want)
    for a, b in ((1, 0), (0, 1), (1, 3), (3, 2), (5, 7)):
        got = torch.empty(T, N, device="cuda")
        m.moe_q4_linear(G, m.Q4Weights(codes, shifted(q.scale, a), shifted(q.zero, b)), x, got)
        torch.cuda.synchronize()
        assert torch.equal(got, want), (a, b)


LARGEST = 2**20


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
def test_the_largest_matrices(m, T):
    """n_in and n_out of 2^20, the other side short."""
    g = torch.Generator(device="cuda").manual_seed(77)
    for N, K in ((16, LARGEST), (LARGEST, 16)):
        x, dy, w = randn(g, T, K), randn(g, T, N), randn(g, 1, N, K, std=K**-0.5)
        G = m.RowGroups(T)
        y, s, dx, dw = (torch.full(v, 7.0, device="cuda") for v in ((T, N), (T, N // 2), (T, K), (1, N, K)))
        note(f"largest {T} {N} {K}")
        m.moe_grouped_linear(G, x, w, y)
        m.moe_grouped_linear(G, x, w, s, m.ACT_SWIGLU)
        m.moe_grouped_dgrad(G, dy, w, dx)
        m.moe_grouped_wgrad(G, x, dy, dw)
        torch.cuda.synchronize()
        want, tol = product(x, w[0])
        near(y, want, tol, f"linear {N} {K}")
        near(s, *swiglu(want, tol), f"swiglu {N} {K}")
        near(dx, *product(dy, w[0].T), f"dgrad {N} {K}")
        near(dw[0], *product(dy.T, x.T), f"wgrad {N} {K}")
    for N, K in ((3, LARGEST), (LARGEST, 32)):
        codes = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = (0.5 + torch.rand(1, N, K // 32, generator=g, device="cuda")) * K**-0.5 / 8
        x, out = randn(g, T, K), torch.full((T, N), 7.0, device="cuda")
        note(f"largest q4 {T} {N} {K}")
        m.moe_q4_linear(m.RowGroups(T), m.Q4Weights(codes, scale), x, out)
        torch.cuda.synchronize()
        per = scale[0].double().repeat_interleave(32, dim=1)
        w = (torch.stack([codes[0] & 15, codes[0] >> 4], dim=2).view(N, K).double() - 8) * per
        near(out, *product(x, w, 31 * per, terms=2), f"q4 {N} {K}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 7])
def test_the_most_rows(m, n):
    """2^24 positions, of one group and of seven."""
    R, K = 2**24, 32
    g = torch.Generator(device="cuda").manual_seed(78)
    cut = torch.sort(torch.randint(0, R, (n - 1,), generator=g, device="cuda")).values.tolist()
    edges = [0, *cut, R]
    G = m.RowGroups(R, offsets=torch.tensor(edges, dtype=torch.int32, device="cuda") if n > 1 else None)
    x, w, y = randn(g, R, K), randn(g, n, 8, K, std=0.2), torch.full((R, 8), 7.0, device="cuda")
    q = m.Q4Weights(torch.randint(0, 256, (n, 8, K // 2), generator=g, device="cuda", dtype=torch.uint8), torch.full((n, 8, 1), 0.02, device="cuda"))
    y4, dy = torch.full((R, 8), 7.0, device="cuda"), randn(g, R, 8)
    dx, dw = torch.full((R, K), 7.0, device="cuda"), torch.full((n, 8, K), 7.0, device="cuda")
    note(f"most rows {n}")
    m.moe_grouped_linear(G, x, w, y)
    m.moe_q4_linear(G, q, x, y4)
    m.moe_grouped_dgrad(G, dy, w, dx)
    m.moe_grouped_wgrad(G, x, dy, dw)
    torch.cuda.synchronize()
    for e in range(n):
        a, b = edges[e], edges[e + 1]
        c = q._keep[0][e]
        v = (torch.stack([c & 15, c >> 4], dim=2).view(8, K).double() - 8) * 0.02
        near(y[a:b], *product(x[a:b], w[e]), f"linear {e}")
        near(y4[a:b], *product(x[a:b], v, torch.full_like(v, 31 * 0.02), terms=2), f"q4 {e}")
        near(dx[a:b], *product(dy[a:b], w[e].T), f"dgrad {e}")
        near(dw[e], *product(dy[a:b].T, x[a:b].T), f"wgrad {e}")


@pytest.mark.gpu
def test_a_stream_that_is_named(m):
    """stream=: the call runs there, behind what is there already, and not on the current one."""
    c = Case(90, 4, 8, 512, 208, dst="slots", seed=79)
    G, x, w = c.groups(m), c.x.cuda(), c.w.cuda()
    want = torch.empty(c.R, c.N, device="cuda")
    m.moe_grouped_linear(G, x, w, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.full((c.R, c.N), 7.0, device="cuda")
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            late.add_(0.0)
        late.copy_(x)
    m.moe_grouped_linear(G, late, w, out, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want)
