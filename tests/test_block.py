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
    b = SimpleNamespace(T=T, xn=torch.empty(T, H, dtype=BF16), ws_shared=None)
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
