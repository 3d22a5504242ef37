"""moe_shared_ffn (the shared expert with low-rank adapters of many requests) against a plain binary64 implementation.

Tolerances, per token, on the 2-norm of the error over the root sum of squares of the output's terms, those of
W' = Wd + c B A of the token's adapter: what is off in h passes through all of W'.  fp32 out: x, A x, h and A h keep their
24 bits, so what is left are the fp32 sums.  A chain of up to 16384 terms in random order is off by sqrt(16384) * 2^-24 =
2^-17 of its terms' root sum of squares; gate and up enter h with a factor of at most 1.1 each (the largest slope of silu),
and the down product adds its own: sqrt(2 * 1.1^2 + 1) * 2^-17 < 2^-16.  bf16 out: a rounding to bf16 is off by at most 2^-8,
uniform rounding errors have 1/sqrt(3) of that as their root mean square, and errors of independent terms add in squares:
h and the result at 2^-8 / sqrt(3)
each: 0.82 * 2^-8.  Below 64 terms that averaging is no argument (one term may be most of the sum), and the
bf16 bound is the one of the largest errors: with |e_i| <= 2^-8 and w_i the columns of Wd,
|sum e_i h_i w_i| <= 2^-8 sum |h_i| |w_i| <= 2^-8 sqrt(I) sqrt(sum h_i^2 |w_i|^2), and 2^-8 of the result: 2^-8 (sqrt(I) + 1).
With adapters of low rank an output can be all in one direction b, where the errors of h meet in one number,
c b sum e_i a_i h_i, of standard deviation 2^-8 / sqrt(3) of that term; no averaging over outputs remains, and over some
thousands of tokens 4 deviations are met: 2^-8 sqrt(16 / 3 + 1 / 3) = 2.4 * 2^-8 for a bf16 out.
"""
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_moe_permute_amd", "libmoe2bit.so")
BF16, F32 = torch.bfloat16, torch.float32
TOL = {F32: 2.0**-16, BF16: 2.0**-8}


def note(msg):
    print(f"[shared-ffn] {msg}", flush=True)
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
    """Weights, a pool of n adapters of ranks up to R and tokens with adapters, as CPU tensors."""

    def __init__(self, T, H, I, n=0, R=8, x_t=BF16, seed=1, projections=("gate", "up", "down"), ranks=None, scales=True):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0, dtype=BF16):
            return (torch.randn(*shape, generator=g) * std).to(dtype)

        self.T, self.H, self.I, self.n, self.R = T, H, I, n, R
        self.x = normal(T, H, dtype=x_t)
        self.w = {"gate": normal(I, H, std=H**-0.5), "up": normal(I, H, std=H**-0.5), "down": normal(H, I, std=I**-0.5)}
        shape = {"gate": (I, H), "up": (I, H), "down": (H, I)}
        self.a = {p: normal(n, R, shape[p][1], std=shape[p][1]**-0.5) for p in projections if n}
        self.b = {p: normal(n, shape[p][0], R, std=R**-0.5) for p in projections if n}
        self.rank = None if ranks is None else torch.tensor([ranks[i % len(ranks)] for i in range(n)], dtype=torch.int32)
        self.scale = (torch.rand(n, generator=g) + 0.5) if n and scales else None
        self.ids = torch.randint(-1, n + 1, (T,), generator=g, dtype=torch.int32) if n else None

    def ranks(self):
        return [self.R] * self.n if self.rank is None else [min(max(int(r), 0), self.R) for r in self.rank]

    def spoil(self):
        """NaN behind every adapter's rank and in every adapter that no token uses."""
        used = set(self.ids.tolist())
        for i, r in enumerate(self.ranks()):
            for p in self.a:
                self.a[p][i, r if i in used else 0:] = float("nan")
                self.b[p][i, :, r if i in used else 0:] = float("nan")

    def project(self, v, p):
        """W' v = W v + scale B A v per token, and the root sum of squares of W' v's terms, in binary64."""
        w = self.w[p].double()
        out, size = v @ w.T, torch.sqrt((v * v) @ (w * w).T)
        for i, r in enumerate(self.ranks()):
            rows = (self.ids == i).nonzero().flatten() if self.n else []
            if len(rows) and p in self.a and r:
                scale = float(self.scale[i]) if self.scale is not None else 1.0
                a, b = self.a[p][i, :r].double(), self.b[p][i, :, :r].double()
                out[rows] += scale * (v[rows] @ a.T @ b.T)
                size[rows] = torch.sqrt((v[rows] * v[rows]) @ (w + scale * b @ a).square().T)
        return out, size

    def reference(self):
        x = self.x.double()
        g, u = self.project(x, "gate")[0], self.project(x, "up")[0]
        return self.project(g * torch.sigmoid(g) * u, "down")

    def on_gpu(self, m):
        dev = {p: t.cuda() for p, t in self.w.items()}
        desc = m.LayerDesc(hidden=self.H, shared_inter=self.I, shared_gate=dev["gate"].data_ptr(),
                           shared_up=dev["up"].data_ptr(), shared_down=dev["down"].data_ptr())
        pool = None
        if self.n:
            pool = m.AdapterPool(self.H, self.I, rank=None if self.rank is None else self.rank.cuda(),
                                 scale=None if self.scale is None else self.scale.cuda(),
                                 **{p: (self.a[p].cuda(), self.b[p].cuda()) for p in self.a})
        return dev, desc, pool, None if self.ids is None else self.ids.cuda()

    def run(self, m, out_t=F32):
        """One call with guards behind the output and the workspace."""
        keep, desc, pool, ids = self.on_gpu(m)
        need = m.moe_shared_ffn_workspace(desc, self.T, pool)
        assert need > 0
        ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((self.T + 2, self.H), float("nan"), dtype=out_t, device="cuda")
        m.moe_shared_ffn(desc, self.x.cuda(), out[:self.T], ws[:need], pool, ids)
        torch.cuda.synchronize()
        assert (ws[need:] == 0xA5).all(), "written behind the workspace"
        assert torch.isnan(out[self.T:]).all(), "written behind the last token"
        return out[:self.T].cpu()

    def check(self, out):
        want, size = self.reference()
        got = out.double()
        assert torch.isfinite(got).all()
        err = torch.linalg.vector_norm(got - want, dim=1)
        den = torch.maximum(torch.linalg.vector_norm(want, dim=1), torch.linalg.vector_norm(size, dim=1))
        rel = float((err / den.clamp_min(1e-30)).max())
        tol = TOL[out.dtype]
        if out.dtype == BF16:
            tol = 2.0**-8 * (self.I**0.5 + 1) if self.I < 64 else 2.4 * 2.0**-8 if self.n else tol
        assert rel <= tol, (rel, tol)


# ----------------------------------------------------------------------------
# numerics
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 100, 130, 257])
@pytest.mark.parametrize("H,I", [(8, 8), (40, 24), (64, 128), (136, 72), (520, 264)])
@pytest.mark.parametrize("x_t,out_t", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
def test_without_adapters(m, T, H, I, x_t, out_t):
    note(f"T={T} H={H} I={I} x={x_t} out={out_t}")
    c = Case(T, H, I, x_t=x_t, seed=T)
    c.check(c.run(m, out_t))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 16, 29, 64, 65, 131, 300])
@pytest.mark.parametrize("H,I,n,R", [(8, 8, 1, 8), (72, 40, 3, 8), (264, 136, 7, 24), (512, 256, 40, 16), (128, 64, 2, 256),
                                     (64, 192, 300, 40)])
@pytest.mark.parametrize("x_t,out_t", [(BF16, F32), (F32, BF16), (F32, F32), (BF16, BF16)])
def test_with_adapters(m, T, H, I, n, R, x_t, out_t):
    """Mixed ranks (none, one, odd, full, above the pool's), tokens without an adapter and with indices outside the pool,
    NaN in what no token uses."""
    note(f"T={T} H={H} I={I} n={n} R={R} x={x_t} out={out_t}")
    c = Case(T, H, I, n, R, x_t, seed=T + n, ranks=[R, 1, R // 2 + 1, 0, R - 3, R + 9, 8, -2])
    if T > 2:
        c.ids[0], c.ids[1] = -2**31, 2**31 - 1
    c.spoil()
    c.check(c.run(m, out_t))


@pytest.mark.gpu
@pytest.mark.parametrize("projections", [("gate",), ("up",), ("down",), ("gate", "down"), ("gate", "up")])
@pytest.mark.parametrize("T", [5, 90, 300])
def test_some_projections(m, projections, T):
    note(f"adapters of {projections} T={T}")
    c = Case(T, 136, 88, 4, 16, seed=T, projections=projections, scales=False)
    c.check(c.run(m))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,n,R", [(1, 4096, 2048, 8, 16), (24, 4096, 2048, 32, 64), (200, 4096, 2048, 8, 32),
                                       (700, 1024, 512, 16, 16), (2048, 512, 1024, 3, 8), (4099, 256, 128, 5, 8)])
@pytest.mark.parametrize("out_t", [F32, BF16])
def test_larger_layers(m, T, H, I, n, R, out_t):
    note(f"T={T} H={H} I={I} n={n} R={R} out={out_t}")
    c = Case(T, H, I, n, R, seed=T)
    c.check(c.run(m, out_t))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(2100, 264, 2056), (2100, 4104, 72), (1100, 264, 2056), (1100, 4104, 72), (2112, 320, 2048)])
@pytest.mark.parametrize("n,x_t", [(0, BF16), (3, BF16), (3, F32)])
def test_wide_tiles(m, T, H, I, n, x_t):
    """Tiles of 128 and 256 tokens (where they are enough for every compute unit), whole and with odd ends."""
    note(f"wide tiles T={T} H={H} I={I} n={n} x={x_t}")
    c = Case(T, H, I, n, 24, x_t, seed=T, ranks=[24, 5, 17])
    c.check(c.run(m, BF16))


@pytest.mark.gpu
@pytest.mark.parametrize("T,R", [(1, 8), (1, 16), (2, 8), (1, 24), (2, 16), (3, 8), (1, 32), (4, 8), (5, 8), (1, 40)])
@pytest.mark.parametrize("I", [8, 264, 2056, 8200])
@pytest.mark.parametrize("out_t", [F32, BF16])
def test_few_values(m, T, R, I, out_t):
    """Both sides of the limits up to which the down product forms the low-rank results of h itself."""
    note(f"few values T={T} R={R} I={I} out={out_t}")
    for ranks in ([R], [R - 3, 0, 1]):
        c = Case(T, 72, I, 4, R, seed=T, ranks=ranks)
        c.ids = torch.arange(T, dtype=torch.int32)
        c.spoil()
        c.check(c.run(m, out_t))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 64, 65, 400])
@pytest.mark.parametrize("mix", ["none", "one", "runs", "each"])
def test_token_orders(m, T, mix):
    """All tokens without an adapter, all with the same one, runs of one request each, and a different one per token."""
    note(f"T={T} {mix}")
    n = 400
    c = Case(T, 136, 72, n, 8, seed=T)
    t = torch.arange(T, dtype=torch.int32)
    c.ids = {"none": torch.full((T,), -1, dtype=torch.int32), "one": torch.full((T,), 7, dtype=torch.int32),
             "runs": t // 23 - 1, "each": n - 1 - t}[mix].contiguous()
    c.spoil()
    c.check(c.run(m))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 60, 300, 9000])
def test_the_most_adapters(m, T):
    """A pool of 4096, its last ones among those in use, on a stream that is named."""
    note(f"4096 adapters T={T}")
    c = Case(T, 24, 16, 4096, 8, seed=T)
    c.ids[0], c.ids[-1] = 4095, 4096
    keep, desc, pool, ids = c.on_gpu(m)
    x, out = c.x.cuda(), torch.empty(T, c.H, device="cuda")
    ws = torch.empty(m.moe_shared_ffn_workspace(desc, T, pool), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    m.moe_shared_ffn(desc, x, out, ws, pool, ids, stream=side.cuda_stream)
    side.synchronize()
    c.check(out.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 70, 300])
def test_pools_beyond_32_bits(m, T):
    """The last adapter of a pool whose A matrices pass 2^31 elements."""
    note(f"large pool T={T}")
    n, R, H, I = 520, 256, 16384, 16
    c = Case(T, H, I, seed=T)
    small = Case(T, H, I, 1, R, seed=T + 1, projections=("gate",))
    a = torch.empty(n, R, H, dtype=BF16, device="cuda")
    b = torch.empty(n, I, R, dtype=BF16, device="cuda")
    assert a.numel() - R * H > 2**31
    a[-1], b[-1] = small.a["gate"][0].cuda(), small.b["gate"][0].cuda()
    dev = {p: t.cuda() for p, t in c.w.items()}
    desc = m.LayerDesc(hidden=H, shared_inter=I, shared_gate=dev["gate"].data_ptr(), shared_up=dev["up"].data_ptr(),
                       shared_down=dev["down"].data_ptr())
    pool = m.AdapterPool(H, I, gate=(a, b))
    ids = torch.full((T,), n - 1, dtype=torch.int32, device="cuda")
    out = torch.empty(T, H, device="cuda")
    ws = torch.empty(m.moe_shared_ffn_workspace(desc, T, pool), dtype=torch.uint8, device="cuda")
    m.moe_shared_ffn(desc, c.x.cuda(), out, ws, pool, ids)
    torch.cuda.synchronize()
    c.n, c.R, c.a, c.b, c.scale = 1, R, {"gate": small.a["gate"]}, {"gate": small.b["gate"]}, None
    c.ids = torch.zeros(T, dtype=torch.int32)
    c.check(out.cpu())


# ----------------------------------------------------------------------------
# one request and the others
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 20, 64, 65, 200, 257, 700])
def test_a_token_does_not_depend_on_the_others(m, T):
    """Same bits for a token whatever adapters the other tokens use, in whatever order, and with NaN adapters among
    theirs; the tokens with the NaN adapter alone become NaN."""
    note(f"independence T={T}")
    c = Case(T, 264, 136, 12, 16, seed=T)
    c.ids = (torch.arange(T, dtype=torch.int32) % 13) - 1
    first = c.run(m)
    t = T // 2
    keep = int(c.ids[t])
    c.ids = torch.randint(-1, 12, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    c.ids[t] = keep
    assert torch.equal(c.run(m)[t], first[t])
    bad = (keep + 1) % 12
    c.ids[c.ids == bad] = keep
    clean = c.run(m)
    c.ids[0] = bad
    for p in c.a:
        c.a[p][bad] = float("nan")
        c.b[p][bad] = float("inf")
    got = c.run(m)
    assert torch.isnan(got[0]).all()
    assert torch.equal(got[1:], clean[1:])


@pytest.mark.gpu
def test_a_token_of_two(m):
    """The same where the down product forms the low-rank results itself."""
    note("independence T=2")
    c = Case(2, 264, 136, 3, 8, seed=2)
    c.ids = torch.tensor([0, 1], dtype=torch.int32)
    first = c.run(m)
    c.a["down"][0], c.b["up"][0] = float("nan"), float("inf")
    got = c.run(m)
    assert torch.isnan(got[0]).all() and torch.equal(got[1], first[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 40, 200, 300])
@pytest.mark.parametrize("x_t", [BF16, F32])
def test_a_token_that_is_not_finite(m, T, x_t):
    """A padded row that holds NaN or infinities reaches no other row."""
    note(f"not finite T={T} x={x_t}")
    c = Case(T, 264, 136, 3, 8, x_t=x_t, seed=T)
    clean = c.run(m)
    c.x[0, 3], c.x[0, 90] = float("inf"), float("nan")
    got = c.run(m)
    assert torch.isnan(got[0]).all() and torch.equal(got[1:], clean[1:])


@pytest.mark.gpu
def test_without_adapters_matches_the_layer_call(m):
    """The shared half of moe_expert_ffn and this call agree within both calls' errors."""
    import oracle
    import synth
    from bit_quantized_moe_permute_amd.layer import DeviceLayer, LayerBuffers, forward
    sp = synth.SPECS["small"]
    DL = DeviceLayer.from_synth(synth.make_layer(sp, quantizer=oracle.quantize))
    for T in (1, 5, 40, 150):
        note(f"against the layer's own T={T}")
        x = torch.from_numpy(synth.activations("small", T, sp.hidden, True, seed=60 + T).view(np.int16)).view(BF16).cuda()
        b = LayerBuffers.allocate(DL, T)
        forward(DL, x, b)
        out = torch.empty_like(b.shared_out)
        ws = torch.empty(m.moe_shared_ffn_workspace(DL.desc, T), dtype=torch.uint8, device="cuda")
        m.moe_shared_ffn(DL.desc, x, out, ws)
        torch.cuda.synchronize()
        rel = torch.linalg.vector_norm(out - b.shared_out, dim=1) / torch.linalg.vector_norm(b.shared_out, dim=1)
        assert float(rel.max()) <= 2 * TOL[F32]


# ----------------------------------------------------------------------------
# streams and graphs
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 130, 300])
def test_graph_replays_match_eager_calls(m, T):
    """Captured once, replayed with other activations, other token indices and another adapter loaded into a slot."""
    note(f"graph T={T}")
    c = Case(T, 264, 136, 6, 16, seed=T)
    keep, desc, pool, ids = c.on_gpu(m)
    x = c.x.cuda()
    out, ref = torch.empty(T, c.H, device="cuda"), torch.empty(T, c.H, device="cuda")
    need = m.moe_shared_ffn_workspace(desc, T, pool)
    ws, ws2 = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    m.moe_shared_ffn(desc, x, out, ws, pool, ids)
    torch.cuda.synchronize()
    g, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(g, stream=cap):
            m.moe_shared_ffn(desc, x, out, ws, pool, ids)
    slot = pool._keep[0]
    for i in range(4):
        x.copy_(torch.randn(T, c.H, generator=torch.Generator().manual_seed(70 + i)))
        ids.copy_(torch.randint(-1, 7, (T,), generator=torch.Generator().manual_seed(80 + i)))
        slot[i].mul_(-0.5)
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        m.moe_shared_ffn(desc, x, ref, ws2, pool, ids)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), i


@pytest.mark.gpu
def test_two_graphs_share_a_workspace(m):
    """Two captured calls of other sizes with one workspace, replayed in turn on one stream, eager calls between."""
    note("two graphs, one workspace")
    c = [Case(T, 264, 136, 6, 16, seed=T) for T in (3, 300)]
    want = [k.run(m) for k in c]
    on = [k.on_gpu(m) for k in c]
    xs, outs = [k.x.cuda() for k in c], [torch.empty(k.T, k.H, device="cuda") for k in c]
    ws = torch.empty(max(m.moe_shared_ffn_workspace(o[1], k.T, o[2]) for k, o in zip(c, on)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, cap = [], torch.cuda.Stream()
    for o, x, out in zip(on, xs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(cap):
            with torch.cuda.graph(graphs[-1], stream=cap):
                m.moe_shared_ffn(o[1], x, out, ws, o[2], o[3])
    for i in range(4):
        for out in outs:
            out.fill_(7.0)
        ws.fill_(0xFF if i % 2 else 0)
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out.cpu(), w), i
        m.moe_shared_ffn(on[0][1], xs[0], outs[0], ws, on[0][2], on[0][3])
        torch.cuda.synchronize()
        assert torch.equal(outs[0].cpu(), want[0]), i


@pytest.mark.gpu
def test_two_streams_with_a_workspace_each(m):
    note("two streams")
    c = [Case(T, 264, 136, 6, 16, seed=T) for T in (40, 170, 300)]
    want = [k.run(m) for k in c]
    sides = [torch.cuda.Stream() for _ in c]
    on = [k.on_gpu(m) for k in c]
    xs = [k.x.cuda() for k in c]
    ws = [torch.empty(m.moe_shared_ffn_workspace(o[1], k.T, o[2]), dtype=torch.uint8, device="cuda") for k, o in zip(c, on)]
    outs = [torch.empty(k.T, k.H, device="cuda") for k in c]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, x, w, out in zip(sides, on, xs, ws, outs):
            with torch.cuda.stream(s):
                m.moe_shared_ffn(o[1], x, out, w, o[2], o[3])
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out.cpu(), w)


# ----------------------------------------------------------------------------
# the operators together: a block between its two norms
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 90])
@pytest.mark.parametrize("steer", [False, True])
def test_block_with_adapters(m, T, steer):
    """forward_block: residual norm, routing, routed experts, shared expert with adapters, combine, residual, norm, against
    the oracle's routing and experts and binary64 for the rest (the layer's tolerance, 1e-3 per token)."""
    import oracle
    import synth
    from bit_quantized_moe_permute_amd.layer import DeviceLayer, LayerBuffers, forward, forward_block
    note(f"block T={T} steer={steer}")
    sp = synth.SPECS["small"]
    L = synth.make_layer(sp, quantizer=oracle.quantize)
    DL = DeviceLayer.from_synth(L)
    H, I = sp.hidden, DL.Is
    c = Case(T, H, I, 5, 16, seed=T, ranks=[16, 7])
    c.w = {p: t.cpu() for p, t in zip(("gate", "up", "down"), DL.shared)}
    _, _, pool, ids = c.on_gpu(m)
    DL.set_adapters(pool)
    rng = np.random.default_rng(5)
    if steer:
        DL.set_steering(rng.standard_normal(H) / np.sqrt(H), 0.5)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))
    res = torch.from_numpy(2 * rng.standard_normal((T, H)).astype(np.float32))
    w_in, w_out = (torch.from_numpy((1 + 0.1 * rng.standard_normal(H)).astype(np.float32)) for _ in range(2))
    b = LayerBuffers.allocate(DL, T)
    r, y = res.cuda(), torch.empty(T, H, device="cuda")
    forward_block(DL, x.cuda(), r, w_in.cuda(), w_out.cuda(), 1e-6, b, y, token_adapter=ids)
    torch.cuda.synchronize()
    r1 = (x + res).double()
    xn = r1 / torch.sqrt((r1 * r1).mean(1, keepdim=True) + 1e-6) * w_in.double()
    got_xn = b.xn.cpu()
    assert ((got_xn.double() - xn).abs() <= 1.001 * 2.0**-8 * xn.abs()).all()
    bits = got_xn.view(torch.int16).numpy().view(np.uint16)
    ref = oracle.layer(bits, L.w_router, sp.top_k, sp.n_experts, sp.inter, sp.gate_up_fmt, L.gate, L.up, sp.down_fmt, L.down,
                       L.codebook, shared=L.shared)
    c.x = got_xn
    shared, _ = c.reference()
    layer = torch.from_numpy(ref["y"] - ref["shared_out"]).double() + shared
    if steer:
        v = DL.steer_v.cpu().double()
        layer = layer - 0.5 * torch.outer(layer @ v, v)
    r2 = r1 + layer
    rel = torch.linalg.vector_norm(r.cpu().double() - r2, dim=1) / torch.linalg.vector_norm(r2, dim=1)
    assert float(rel.max()) <= 1e-3
    y2 = r2 / torch.sqrt((r2 * r2).mean(1, keepdim=True) + 1e-6) * w_out.double()
    rel = torch.linalg.vector_norm(y.cpu().double() - y2, dim=1) / torch.linalg.vector_norm(y2, dim=1)
    assert float(rel.max()) <= 2e-3
    # the layer alone, through forward(), on the same rows
    forward(DL, b.xn.clone(), b, token_adapter=ids)
    torch.cuda.synchronize()
    rel = torch.linalg.vector_norm(b.y.cpu().double() - layer, dim=1) / torch.linalg.vector_norm(layer, dim=1)
    assert float(rel.max()) <= 1e-3


# ----------------------------------------------------------------------------
# refusals (host only)
# ----------------------------------------------------------------------------
needs_lib = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe2bit.so not built (run __graft_entry__.build())")
P = {p: 0x1000000 * (i + 1) for i, p in enumerate(("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b"))}


def call(layer=None, pool=None, **bad):
    import bit_quantized_moe_permute_amd as m
    L = m.LayerDesc(**dict(dict(hidden=64, shared_inter=32, shared_gate=0x10000, shared_up=0x20000, shared_down=0x30000),
                           **(layer or {})))
    A = None if pool is None else m.AdapterDesc(**dict(dict(n_adapters=2, max_rank=8, **P), **pool))
    a = dict(dict(x=0x100000, x_dt=1, T=3, ids=0x200000, out=0x300000, out_dt=0, ws=0x400000, size=1 << 22), **bad)
    st = m.lib.moe_shared_ffn(None if bad.get("no_layer") else L, A, a["x"], a["x_dt"], a["T"], a["ids"], a["out"], a["out_dt"],
                              a["ws"], a["size"], None)
    return st, m.moe_last_error(), m.lib.moe_shared_ffn_workspace(L, A, a["T"])


@needs_lib
@pytest.mark.parametrize("bad,word", [
    (dict(no_layer=True), "null layer"), (dict(layer=dict(hidden=60)), "multiples of 8"), (dict(layer=dict(hidden=0)), "multiples"),
    (dict(layer=dict(shared_inter=0)), "multiples of 8"), (dict(layer=dict(shared_inter=-8)), "multiples of 8"),
    (dict(layer=dict(shared_up=None)), "weights"), (dict(layer=dict(shared_down=0x30008)), "aligned"),
    (dict(pool=dict(n_adapters=0)), "n_adapters"), (dict(pool=dict(n_adapters=4097)), "n_adapters"),
    (dict(pool=dict(max_rank=12)), "max_rank"), (dict(pool=dict(max_rank=0)), "max_rank"), (dict(pool=dict(max_rank=264)), "max_rank"),
    (dict(pool=dict(up_b=None)), "neither"), (dict(pool=dict(down_a=0x5000008)), "aligned"), (dict(pool=dict(rank=0x1002)), "misaligned"),
    (dict(pool={}, ids=None), "null"), (dict(x=None), "null"), (dict(out=None), "null"), (dict(ws=None), "null"), (dict(T=0), "n_tokens"),
    (dict(x_dt=2), "dtype"), (dict(out_dt=3), "dtype"), (dict(x=0x100008), "misaligned"), (dict(out=0x300004), "misaligned"),
    (dict(ws=0x400080), "misaligned"), (dict(pool={}, ids=0x200002), "misaligned"), (dict(size=100), "workspace"),
    (dict(out=0x100000), "overlaps"), (dict(x=0x400000), "overlaps"), (dict(out=0x400000), "overlaps"),
    (dict(pool={}, ids=0x300000), "overlaps"), (dict(pool={}, ids=0x400100), "overlaps"),
])
def test_shared_ffn_refuses(bad, word):
    st, msg, _ = call(**bad)
    assert st == 1 and word in msg, (st, msg)


@needs_lib
@pytest.mark.parametrize("bad,word", [
    (dict(layer=dict(hidden=(1 << 20) + 8)), "above"), (dict(layer=dict(shared_inter=(1 << 20) + 8)), "above"),
    (dict(layer=dict(hidden=8, shared_inter=8), T=1 << 22), "n_tokens >"), (dict(layer=dict(hidden=1 << 20), T=1 << 10), "split the batch"),
    (dict(layer=dict(shared_inter=1 << 10), T=1 << 20), "split the batch"),
])
def test_shared_ffn_limits(bad, word):
    st, msg, ws = call(**bad)
    assert st == 2 and word in msg and ws == 0, (st, msg)


@needs_lib
def test_workspace_sizes():
    assert call(T=0)[2] == 0 and call(layer=dict(hidden=60))[2] == 0
    none, some = call(x=None)[2], call(pool={}, x=None)[2]
    assert 0 < none < some
    assert call(pool={}, T=100, x=None)[2] > some
    # a buffer for many tokens serves fewer
    for layer in (dict(hidden=8, shared_inter=8), dict(hidden=64, shared_inter=32), dict(hidden=1024, shared_inter=1024), dict(hidden=1024, shared_inter=1200),
                  dict(hidden=4096, shared_inter=2048)):
        for pool in (None, dict(n_adapters=1, max_rank=256), dict(n_adapters=300, max_rank=8), dict(n_adapters=16, max_rank=32)):
            sizes = [call(layer=layer, pool=pool, T=T, x=None)[2] for T in [*range(1, 700), *range(700, 20000, 61)]]
            assert all(a <= b for a, b in zip(sizes, sizes[1:])), (layer, pool)


@needs_lib
def test_pool_clone():
    import bit_quantized_moe_permute_amd as m
    c = Case(3, 64, 32, 2, 8, projections=("gate", "down"), ranks=[8, 3])
    pool = m.AdapterPool(64, 32, rank=c.rank, scale=c.scale, **{p: (c.a[p], c.b[p]) for p in c.a})
    other = pool.clone()
    assert (other.hidden, other.inter, other.n, other.max_rank) == (64, 32, 2, 8) and other.desc.up_a is None
    assert len(other._keep) == len(pool._keep) == 6
    for s, t in zip(pool._keep, other._keep):
        assert torch.equal(s, t) and s.data_ptr() != t.data_ptr()
    assert other.desc.gate_a == other._keep[0].data_ptr() and other.desc.scale == other._keep[-1].data_ptr()


@needs_lib
def test_binding_refuses():
    import bit_quantized_moe_permute_amd as m
    c = Case(3, 64, 32, 2, 8)
    desc = m.LayerDesc(hidden=64, shared_inter=32, shared_gate=0x10000, shared_up=0x20000, shared_down=0x30000)
    pool = m.AdapterPool(64, 32, **{p: (c.a[p], c.b[p]) for p in c.a})
    out, ws = torch.empty(3, 64), torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(TypeError, match="GPU"):
        m.moe_shared_ffn(desc, c.x, out, ws)
    with pytest.raises(ValueError, match="hidden"):
        m.moe_shared_ffn(desc, c.x[:, :56], out, ws)
    with pytest.raises(ValueError, match="out"):
        m.moe_shared_ffn(desc, c.x, out[:2], ws)
    with pytest.raises(TypeError, match="token_adapter"):
        m.moe_shared_ffn(desc, c.x, out, ws, pool)
    with pytest.raises(TypeError, match="token_adapter"):
        m.moe_shared_ffn(desc, c.x, out, ws, pool, c.ids.long())
    with pytest.raises(ValueError, match="token_adapter"):
        m.moe_shared_ffn(desc, c.x, out, ws, pool, c.ids[:2])
    other = Case(3, 64, 40, 2, 8)
    with pytest.raises(ValueError, match="adapters are for"):
        m.moe_shared_ffn(desc, c.x, out, ws, m.AdapterPool(64, 40, gate=(other.a["gate"], other.b["gate"])), c.ids)
    with pytest.raises(ValueError, match="no projection"):
        m.AdapterPool(64, 32)
    with pytest.raises(ValueError, match="gate_b"):
        m.AdapterPool(64, 32, gate=(c.a["gate"], c.b["gate"][:, :, :4]))
    with pytest.raises(ValueError, match="down_a"):
        m.AdapterPool(64, 32, gate=(c.a["gate"], c.b["gate"]), down=(c.a["gate"], c.b["down"]))
    with pytest.raises(ValueError, match="rank"):
        m.AdapterPool(64, 32, gate=(c.a["gate"], c.b["gate"]), rank=torch.zeros(2))
    with pytest.raises(ValueError, match="scale"):
        m.AdapterPool(64, 32, gate=(c.a["gate"], c.b["gate"]), scale=torch.zeros(3))
