"""layer.forward_block: its refusals, residual and output types, graph replay, and the memory that buffers take for it."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from test_norm import f64, outputs
from test_norm_precision import HALF, check, exact_norm
from test_shared_ffn import BF16, F32, LIB, Case, m, needs_lib, note  # noqa: F401


# ----------------------------------------------------------------------------
# refusals (host only)
# ----------------------------------------------------------------------------
def refused_call(**change):
    """forward_block on CPU tensors of a layer of hidden 64 and buffers of four tokens; what is not refused for another
    reason is refused for being on the CPU, with a TypeError that names the GPU."""
    from bit_quantized_moe_permute_amd.layer import forward_block
    T, H = 4, 64
    L = SimpleNamespace(H=H, Is=32, adapters=None, steer_v=None, steer_f=0.0, desc=None)
    rows = torch.empty(T, H, dtype=BF16)
    b = SimpleNamespace(T=T, xn=rows, ws_shared=None, block_rows=lambda *_: rows)
    a = dict(x=torch.zeros(T, H), residual=torch.zeros(T, H), w_in=torch.ones(H), w_out=torch.ones(H), y=torch.zeros(T, H),
             y_scale=None, token_adapter=None)
    a.update(change)
    forward_block(L, a["x"], a["residual"], a["w_in"], a["w_out"], 1e-6, b, a["y"], a["y_scale"], a["token_adapter"])


@needs_lib
@pytest.mark.parametrize("change,error,word", [
    ({}, TypeError, "GPU"),
    (dict(x=torch.zeros(3, 64)), ValueError, "shape"), (dict(x=torch.zeros(5, 64)), ValueError, "shape"),
    (dict(x=torch.zeros(4, 56)), ValueError, "shape"), (dict(x=torch.zeros(256)), ValueError, "shape"),
    (dict(token_adapter=torch.zeros(4, dtype=torch.int32)), ValueError, "no adapters"),
    (dict(w_out=torch.ones(63)), ValueError, "weight"), (dict(y=torch.zeros(3, 64)), ValueError, "y: "),
    (dict(y=torch.zeros(4, 64, dtype=torch.float16)), TypeError, "y: "), (dict(y_scale=torch.zeros(4)), ValueError, "y_scale"),
    (dict(residual=torch.zeros(3, 64)), ValueError, "residual"),
])
def test_block_refuses(change, error, word):
    with pytest.raises(error, match=word):
        refused_call(**change)


def layer(m, T, n=5):  # noqa: F811
    import oracle
    import synth
    from bit_quantized_moe_permute_amd.layer import DeviceLayer
    sp = synth.SPECS["small"]
    L = synth.make_layer(sp, quantizer=oracle.quantize)
    DL = DeviceLayer.from_synth(L)
    c = Case(T, sp.hidden, DL.Is, n, 16, seed=T, ranks=[16, 7])
    c.w = {p: t.cpu() for p, t in zip(("gate", "up", "down"), DL.shared)}
    return DL, L, c


@pytest.mark.gpu
def test_a_refused_block_leaves_the_residual(m):  # noqa: F811
    from bit_quantized_moe_permute_amd.layer import LayerBuffers, forward_block
    note("refused block")
    T = 5
    DL, _, c = layer(m, T)
    H = DL.H
    _, _, pool, ids = c.on_gpu(m)
    w = torch.ones(H, device="cuda")
    b = LayerBuffers.allocate(DL, T)
    x, r, y = torch.ones(T, H, device="cuda"), torch.zeros(T + 2, H, device="cuda"), torch.empty(T, H, device="cuda")

    def refused(error, x=x, y=y, w_out=w, ids=None, b=b):
        with pytest.raises(error):
            forward_block(DL, x, r, w, w_out, 1e-6, b, y, token_adapter=ids)
        torch.cuda.synchronize()
        assert (r == 0).all()

    refused(ValueError, x=x[:4])
    refused(ValueError, y=y[:4])
    refused(ValueError, w_out=w[:-1])
    refused(TypeError, y=y.half())
    refused(ValueError, ids=ids)                          # a layer without adapters
    DL.set_adapters(pool)
    refused(ValueError, ids=ids)                          # buffers from before it had any
    b2 = LayerBuffers.allocate(DL, T)
    refused(TypeError, ids=ids.long(), b=b2)
    refused(ValueError, ids=ids[:4], b=b2)
    DL.set_adapters(Case(T, H, DL.Is, 40, 256, seed=1).on_gpu(m)[2])
    refused(ValueError, ids=ids, b=b2)                    # buffers for smaller adapters


@pytest.mark.gpu
def test_rows_are_allocated_for_blocks_alone(m):  # noqa: F811
    """Buffers take no memory for forward_block's rows before its first call, on torch's stream, a named one and under capture."""
    from bit_quantized_moe_permute_amd.layer import LayerBuffers, forward, forward_block
    note("rows of a block")
    T = 6
    DL, _, _ = layer(m, T)
    H, w = DL.H, torch.ones(DL.H, device="cuda")
    x, r, y = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    want_r, want = r.clone(), torch.empty_like(y)
    b = LayerBuffers.allocate(DL, T)
    forward(DL, x.to(BF16), b)
    assert b.xn is None
    forward_block(DL, x, want_r, w, w, 1e-6, b, want)
    rows = b.xn
    forward_block(DL, x, r.clone(), w, w, 1e-6, b, y)
    torch.cuda.synchronize()
    assert b.xn is rows and rows.shape == (T, H) and torch.equal(y, want)
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, torch.cuda.default_stream().cuda_stream):
        b, r2 = LayerBuffers.allocate(DL, T), r.clone()
        y.fill_(0)
        torch.cuda.synchronize()
        forward_block(DL, x, r2, w, w, 1e-6, b, y, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(r2, want_r)
    b, r2 = LayerBuffers.allocate(DL, T), r.clone()
    torch.cuda.synchronize()
    g, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(cap):
        with torch.cuda.graph(g, stream=cap):
            forward_block(DL, x, r2, w, w, 1e-6, b, y)
    for _ in range(3):
        r2.copy_(r)
        y.fill_(0)
        junk = torch.full((64, H), float("nan"), device="cuda")
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(r2, want_r)
        del junk
    xn = b.xn.clone()
    del g
    r3 = r.clone()
    forward_block(DL, x, r3, w, w, 1e-6, b, y.fill_(0))      # the rows outlive the graph
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(b.xn, xn)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 90])
@pytest.mark.parametrize("res_t,w_t,y_t", [(BF16, BF16, "bf16"), (BF16, F32, "block"), (F32, BF16, "row"), (BF16, BF16, "f32")])
@pytest.mark.parametrize("adapters", [False, True])
def test_block_types(m, T, res_t, w_t, y_t, adapters):  # noqa: F811
    """A bf16 residual stream and outputs of every type, against the oracle and binary64: the first norm and the last one
    within their roundings of what is stored, the layer between them within its 1e-3 per token, the residual's rounding added."""
    import oracle
    from bit_quantized_moe_permute_amd.layer import LayerBuffers, forward_block
    note(f"block T={T} residual={res_t} weights={w_t} y={y_t} adapters={adapters}")
    DL, L, c = layer(m, T)
    sp, H = L.spec, DL.H
    ids = None
    if adapters:
        _, _, pool, ids = c.on_gpu(m)
        DL.set_adapters(pool)
    else:
        c.n = 0
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(BF16)
    res = torch.from_numpy(2 * rng.standard_normal((T, H)).astype(np.float32)).to(res_t)
    w_in, w_out = (torch.from_numpy((1 + 0.1 * rng.standard_normal(H)).astype(np.float32)).to(w_t) for _ in range(2))
    b = LayerBuffers.allocate(DL, T)
    r = res.cuda()
    y, ys = outputs(T, H, y_t)
    forward_block(DL, x.cuda(), r, w_in.cuda(), w_out.cuda(), 1e-6, b, y, ys, token_adapter=ids)
    torch.cuda.synchronize()
    r1 = f64((x.float() + res.float()).to(res_t))
    check(b.xn, None, exact_norm(r1, w_in, 1e-6))
    xn = b.xn.cpu()
    ref = oracle.layer(xn.view(torch.int16).numpy().view(np.uint16), L.w_router, sp.top_k, sp.n_experts, sp.inter, sp.gate_up_fmt,
                       L.gate, L.up, sp.down_fmt, L.down, L.codebook, shared=L.shared)
    c.x = xn
    out = ref["y"] - ref["shared_out"] + c.reference()[0].numpy()
    r2 = r1 + out
    norm = lambda v: np.linalg.norm(v, axis=1)  # noqa: E731
    half = HALF if res_t is F32 else 2.0**-8 + HALF
    assert (norm(f64(r) - r2) <= 1.01e-3 * norm(out) + half * norm(r2)).all()
    check(y, ys, exact_norm(f64(r), w_out, 1e-6))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 300])
def test_block_replays(m, T):  # noqa: F811
    """A captured block with adapters on a bf16 residual stream, replayed on changed rows and adapters, eager blocks between."""
    from bit_quantized_moe_permute_amd.layer import LayerBuffers, forward_block
    note(f"block graph T={T}")
    DL, _, c = layer(m, T)
    H = DL.H
    _, _, pool, ids = c.on_gpu(m)
    DL.set_adapters(pool)
    w = torch.ones(H, device="cuda")
    x, r = torch.randn(T, H, device="cuda").to(BF16), torch.zeros(T, H, dtype=BF16, device="cuda")
    (y, ys), (want, want_s) = outputs(T, H, "block"), outputs(T, H, "block")
    b, b2 = LayerBuffers.allocate(DL, T), LayerBuffers.allocate(DL, T)
    forward_block(DL, x, r, w, w, 1e-6, b, y, ys, token_adapter=ids)
    torch.cuda.synchronize()
    g, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(g, stream=cap):
            forward_block(DL, x, r, w, w, 1e-6, b, y, ys, token_adapter=ids)
    for i in range(4):
        gen = torch.Generator().manual_seed(90 + i)
        x.copy_(torch.randn(T, H, generator=gen))
        r.copy_(torch.randn(T, H, generator=gen))
        ids.copy_(torch.randint(-1, 6, (T,), generator=gen))
        r2 = r.clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        forward_block(DL, x, r2, w, w, 1e-6, b2, want, want_s, token_adapter=ids)
        torch.cuda.synchronize()
        assert torch.equal(r, r2) and torch.equal(ys, want_s), i
        assert torch.equal(y.view(torch.uint8), want.view(torch.uint8)), i


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 70])
def test_forward_takes_the_description_it_is_given(m, T):  # noqa: F811
    """Another description's shared weights (here gate and up exchanged) are those that tokens with adapters use too: without
    an adapter among the tokens the layer is the same as without token_adapter, within both calls' errors."""
    from bit_quantized_moe_permute_amd.layer import LayerBuffers, forward
    note(f"description T={T}")
    DL, _, c = layer(m, T)
    DL.set_adapters(c.on_gpu(m)[2])
    x = c.x.cuda()
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    b = LayerBuffers.allocate(DL, T)
    other = DL.make_desc()
    other.shared_gate, other.shared_up = other.shared_up, other.shared_gate
    for desc in (None, DL.make_desc(), other):
        want = forward(DL, x, b, desc).clone()
        got = forward(DL, x, b, desc, token_adapter=none)
        torch.cuda.synchronize()
        err = torch.linalg.vector_norm(got - want, dim=1) / torch.linalg.vector_norm(want, dim=1)
        assert float(err.max()) <= 2.0**-15, float(err.max())
