"""layer.forward_block: its refusals, residual and output types, graph replay, and the memory that buffers take for it."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

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
