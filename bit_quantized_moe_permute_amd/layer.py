"""Device-side bookkeeping for one layer: uploads canonical blocks, prepares
them with moe_prepare_weights, allocates per-call buffers with torch, and
chains the three C-ABI calls.  Argument marshalling only; all arithmetic runs
in libmoe2bit's kernels."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import numpy as np
import torch

from . import (FMT_IQ2X, PATH_AUTO, PRECISION_EXACT, AdapterDesc, LayerDesc, moe_add_rms_norm, moe_combine,
               moe_combine_norm, moe_combine_steer, moe_expert_ffn, moe_expert_ffn_workspace, moe_layer,
               moe_layer_workspace, moe_prepare_weights, moe_route, moe_route_workspace, moe_shared_ffn,
               moe_shared_ffn_workspace, moe_weight_bytes, _norm_output)


def _u8(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).reshape(-1)).to(device)


class AdapterPool:
    """Low-rank adapters of a shared expert resident in device memory.

    gate, up, down: (A, B) bf16 tensors, A [n][R][columns of W] and B [n][rows of W][R], or None for a projection
    without adapters; adapter a adds scale[a] * B[a] A[a] to W.  rank: int32 [n] (ranks up to R; None: all R).
    scale: fp32 [n] (None: all 1).  The pool keeps the tensors; their values may be changed in place (an adapter loaded
    into a slot) between calls.
    """

    def __init__(self, hidden, inter, gate=None, up=None, down=None, rank=None, scale=None):
        self.hidden, self.inter = hidden, inter
        pairs = {"gate": (gate, inter, hidden), "up": (up, inter, hidden), "down": (down, hidden, inter)}
        given = [p[0] for p in pairs.values() if p[0] is not None]
        if not given:
            raise ValueError("adapters for no projection")
        n, R = given[0][0].shape[:2]
        self.n, self.max_rank = n, R
        self.device_index = given[0][0].get_device()
        self.desc = AdapterDesc(n_adapters=n, max_rank=R)
        self._given = dict(gate=gate, up=up, down=down, rank=rank, scale=scale)
        self._keep = []
        for name, (ab, rows, cols) in pairs.items():
            if ab is not None:
                self._hold(name + "_a", ab[0], (n, R, cols), torch.bfloat16)
                self._hold(name + "_b", ab[1], (n, rows, R), torch.bfloat16)
        if rank is not None:
            self._hold("rank", rank, (n,), torch.int32)
        if scale is not None:
            self._hold("scale", scale, (n,), torch.float32)

    def _hold(self, name, t, shape, dtype):
        if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape}, got {t.dtype} "
                             f"{tuple(t.shape)}")
        if t.get_device() != self.device_index:
            raise ValueError(f"{name}: adapters on devices {self.device_index} and {t.get_device()}")
        self._keep.append(t)
        setattr(self.desc, name, t.data_ptr())

    def clone(self) -> "AdapterPool":
        """A second copy of every device tensor (distinct addresses, same values)."""
        return AdapterPool(self.hidden, self.inter, **{
            n: t if t is None else t.clone() if n in ("rank", "scale") else tuple(v.clone() for v in t)
            for n, t in self._given.items()})


class DeviceLayer:
    """A routed 2-bit MoE layer resident in device memory.

    hidden, inter, n_experts, top_k: layer shape.  gate/up/down: canonical block
    bytes (numpy uint8) of E stacked [I][H] / [H][I] matrices.  codebook:
    [256][8] uint8.  w_router: [E][H] bf16 bits (uint16) or fp32.  bias: [E]
    fp32 or None.  shared: (Wg, Wu, Wd) bf16 bits or None.
    """

    def __init__(self, hidden, inter, n_experts, top_k, gate_up_fmt, down_fmt, gate, up, down, codebook, w_router,
                 bias=None, shared=None, device="cuda", path=PATH_AUTO):
        self.H, self.I, self.E, self.k = hidden, inter, n_experts, top_k
        self.gate_up_fmt, self.down_fmt = gate_up_fmt, down_fmt
        self.device = torch.device(device)
        self.gate = self._prepare(gate_up_fmt, gate, inter, hidden)
        self.up = self._prepare(gate_up_fmt, up, inter, hidden)
        self.down = self._prepare(down_fmt, down, hidden, inter)
        self.codebook = _u8(codebook, self.device)
        if w_router.dtype == np.uint16:
            self.w_router = torch.from_numpy(np.ascontiguousarray(w_router).view(np.int16)).view(torch.bfloat16).to(self.device)
        else:
            self.w_router = torch.from_numpy(np.ascontiguousarray(w_router, np.float32)).to(self.device)
        self.bias = None if bias is None else torch.from_numpy(np.ascontiguousarray(bias, np.float32)).to(self.device)
        self.Is = 0
        self.shared = None
        if shared is not None:
            self.shared = tuple(torch.from_numpy(np.ascontiguousarray(s).view(np.int16)).view(torch.bfloat16)
                                .to(self.device) for s in shared)
            self.Is = self.shared[0].shape[0]
        self.path = path
        self.desc = self.make_desc(path)
        self.steer_v, self.steer_f = None, 0.0
        self.adapters = None

    def set_adapters(self, pool: AdapterPool | None):
        """Low-rank adapters of this layer's shared expert, for forward() calls that name each token's; None: none."""
        if pool is not None and (pool.hidden, pool.inter) != (self.H, self.Is):
            raise ValueError(f"adapters are for hidden {pool.hidden}, inter {pool.inter}; the layer's shared expert has "
                             f"{self.H}, {self.Is}")
        self.adapters = pool

    def set_steering(self, v, F: float = 1.0):
        """Directional steering of this layer's FFN output, y -= F * v * dot(v, y): v is one fp32 value per hidden
        unit (used as given), or None to turn steering off."""
        if v is None:
            self.steer_v, self.steer_f = None, 0.0
            return
        v = np.ascontiguousarray(v, dtype=np.float32).reshape(-1)
        if v.shape[0] != self.H:
            raise ValueError(f"steering direction has {v.shape[0]} entries, the layer has hidden {self.H}")
        self.steer_v, self.steer_f = torch.from_numpy(v).to(self.device), float(F)

    def _prepare(self, fmt, blocks, rows, cols):
        nbytes = moe_weight_bytes(fmt, self.E, rows, cols)
        assert blocks.size == nbytes, (blocks.size, nbytes)
        canon = _u8(blocks, self.device)
        prep = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        moe_prepare_weights(fmt, self.E, rows, cols, canon, prep)
        torch.cuda.synchronize(self.device)
        del canon
        return prep

    def make_desc(self, path=PATH_AUTO, precision=PRECISION_EXACT) -> LayerDesc:
        d = LayerDesc()
        d.hidden, d.inter, d.n_experts, d.top_k = self.H, self.I, self.E, self.k
        d.gate_up_fmt, d.down_fmt = self.gate_up_fmt, self.down_fmt
        d.gate, d.up, d.down = self.gate.data_ptr(), self.up.data_ptr(), self.down.data_ptr()
        d.codebook = self.codebook.data_ptr() if self.gate_up_fmt == FMT_IQ2X else None
        d.shared_inter = self.Is
        if self.shared is not None:
            d.shared_gate, d.shared_up, d.shared_down = (s.data_ptr() for s in self.shared)
        d.path = path
        d.precision = precision
        return d

    def routed_desc(self, desc: LayerDesc | None = None) -> LayerDesc:
        """The layer without its shared expert (which moe_shared_ffn computes then)."""
        d = LayerDesc.from_buffer_copy(desc or self.desc)
        d.shared_inter, d.shared_gate, d.shared_up, d.shared_down = 0, None, None, None
        return d

    def clone(self) -> "DeviceLayer":
        """A second copy of every device tensor (distinct addresses, same values)."""
        c = object.__new__(DeviceLayer)
        c.__dict__.update(self.__dict__)
        c.gate, c.up, c.down = self.gate.clone(), self.up.clone(), self.down.clone()
        c.codebook = self.codebook.clone()
        c.w_router = self.w_router.clone()
        c.bias = None if self.bias is None else self.bias.clone()
        c.shared = None if self.shared is None else tuple(s.clone() for s in self.shared)
        c.steer_v = None if self.steer_v is None else self.steer_v.clone()
        c.adapters = None if self.adapters is None else self.adapters.clone()
        c.desc = c.make_desc(self.path)
        return c

    @classmethod
    def from_synth(cls, layer, device="cuda", path=PATH_AUTO) -> "DeviceLayer":
        sp = layer.spec
        return cls(sp.hidden, sp.inter, sp.n_experts, sp.top_k, sp.gate_up_fmt, sp.down_fmt, layer.gate, layer.up,
                   layer.down, layer.codebook, layer.w_router, layer.bias, layer.shared, device, path)


@dataclass
class LayerBuffers:
    """Per-call outputs and workspaces for T tokens."""
    T: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    logits: torch.Tensor
    offsets: torch.Tensor
    perm: torch.Tensor
    active: torch.Tensor
    ws_route: torch.Tensor
    slot_out: torch.Tensor
    shared_out: torch.Tensor | None
    ws_ffn: torch.Tensor
    y: torch.Tensor
    ws: torch.Tensor            # one buffer: ws_route and ws_ffn are views into it (the layout moe_layer takes)
    ws_shared: torch.Tensor | None = None       # moe_shared_ffn's, when the layer has adapters
    xn: torch.Tensor | None = None              # the normed rows forward_block() hands to the layer, from its first call on

    @classmethod
    def allocate(cls, L: DeviceLayer, T: int, with_logits: bool = False) -> "LayerBuffers":
        dev = L.device
        i32 = dict(dtype=torch.int32, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        ws_r = (moe_route_workspace(T, L.E, L.k) + 255) // 256 * 256
        ws_l = moe_layer_workspace(L.desc, T)
        ws = torch.empty(max(ws_l, ws_r + 256), dtype=torch.uint8, device=dev)
        ws_s = moe_shared_ffn_workspace(L.desc, T, L.adapters) if L.adapters is not None else 0
        return cls(
            T=T,
            topk_idx=torch.empty(T, L.k, **i32), topk_w=torch.empty(T, L.k, **f32),
            logits=torch.empty(T, L.E, **f32) if with_logits else None,
            offsets=torch.empty(L.E + 1, **i32), perm=torch.empty(T * L.k, **i32),
            active=torch.empty(L.E + 1, **i32),
            ws_route=ws[:ws_r],
            slot_out=torch.empty(T * L.k, L.H, **f32),
            shared_out=torch.empty(T, L.H, **f32) if L.Is else None,
            ws_ffn=ws[ws_r:],
            y=torch.empty(T, L.H, **f32),
            ws=ws,
            ws_shared=torch.empty(ws_s, dtype=torch.uint8, device=dev) if ws_s else None,
        )

    def block_rows(self, L: DeviceLayer, stream=None) -> torch.Tensor:
        """xn, allocated on the stream that writes it first (the memory may have been in use there before)."""
        if self.xn is None:
            shape = dict(size=(self.T, L.H), dtype=torch.bfloat16, device=L.device)
            if stream is None:
                self.xn = torch.empty(**shape)
            else:
                with torch.cuda.stream(torch.cuda.ExternalStream(stream)):
                    self.xn = torch.empty(**shape)
        return self.xn


def _check_adapters(L: DeviceLayer, b: LayerBuffers, token_adapter):
    if token_adapter is None:
        return
    if L.adapters is None:
        raise ValueError("token_adapter given, but the layer has no adapters (set_adapters)")
    if token_adapter.dtype != torch.int32:
        raise TypeError("token_adapter must be an int32 tensor")
    if token_adapter.numel() < b.T:
        raise ValueError(f"token_adapter: {token_adapter.numel()} elements, the call needs {b.T}")
    if b.ws_shared is None:
        raise ValueError("these buffers were allocated before the layer had adapters")
    if b.ws_shared.numel() < moe_shared_ffn_workspace(L.desc, b.T, L.adapters):
        raise ValueError("these buffers were allocated before the layer had these adapters")


def _route_and_experts(L: DeviceLayer, x, b: LayerBuffers, desc, token_adapter, stream):
    """moe_route and the experts: b.slot_out and b.shared_out.  With adapters and token_adapter the shared expert runs
    as a call of its own."""
    moe_route(x, L.w_router, L.E, L.k, b.topk_idx, b.topk_w, b.offsets, b.perm, b.active, b.ws_route, bias=L.bias,
              logits=b.logits, stream=stream)
    if token_adapter is None:
        moe_expert_ffn(desc or L.desc, x, b.topk_idx, b.offsets, b.perm, b.active, b.slot_out, b.shared_out, b.ws_ffn,
                       stream=stream)
        return
    moe_expert_ffn(L.routed_desc(desc), x, b.topk_idx, b.offsets, b.perm, b.active, b.slot_out, None, b.ws_ffn,
                   stream=stream)
    moe_shared_ffn(desc or L.desc, x, b.shared_out, b.ws_shared, L.adapters, token_adapter, stream=stream)


def forward_block(L: DeviceLayer, x: torch.Tensor, residual: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor,
                  eps: float, b: LayerBuffers, y: torch.Tensor, y_scale=None, token_adapter=None, stream=None):
    """The layer between its two norms, on a residual stream that is updated in place:

        residual += x;  xn = norm(residual) * w_in;  residual += layer(xn);  y = norm(residual) * w_out

    x [T][H] fp32 or bf16 (the attention's output) with the T of the buffers b, y in any type of moe_add_rms_norm.  A call
    that is refused for its shapes, types or adapters leaves the residual as it was."""
    if tuple(x.shape) != (b.T, L.H):
        raise ValueError(f"x has shape {tuple(x.shape)}, the buffers and the layer take {(b.T, L.H)}")
    _check_adapters(L, b, token_adapter)
    _norm_output(x.get_device(), b.T, L.H, residual, residual, w_out, y, y_scale)
    xn = b.block_rows(L, stream)
    moe_add_rms_norm(x, residual, residual, w_in, eps, xn, stream=stream)
    _route_and_experts(L, xn, b, None, token_adapter, stream)
    moe_combine_norm(b.slot_out, b.topk_w, b.shared_out, residual, residual, w_out, eps, y, y_scale,
                     steer_v=L.steer_v, steer_f=L.steer_f, stream=stream)
    return y


def forward(L: DeviceLayer, x: torch.Tensor, b: LayerBuffers, desc: LayerDesc | None = None, stream=None,
            token_adapter: torch.Tensor | None = None):
    """route -> expert FFN -> combine (+ steering, when the layer has a direction) for x [T][H] (bf16 or fp32)
    into b.y.  token_adapter (int32 [T]): each token's adapter of the shared expert (L.set_adapters)."""
    T = x.shape[0]
    assert T == b.T
    _check_adapters(L, b, token_adapter)
    _route_and_experts(L, x, b, desc, token_adapter, stream)
    if L.steer_v is None:
        moe_combine(b.slot_out, b.topk_w, b.shared_out, T, L.k, L.H, b.y, stream=stream)
    else:
        moe_combine_steer(b.slot_out, b.topk_w, b.shared_out, T, L.k, L.H, L.steer_v, L.steer_f, b.y, stream=stream)
    return b.y


def forward_layer(L: DeviceLayer, x: torch.Tensor, b: LayerBuffers, desc: LayerDesc | None = None, stream=None):
    """The same layer as forward() through the single moe_layer call (one routing launch fewer at one token)."""
    assert x.shape[0] == b.T
    moe_layer(desc or L.desc, x, L.w_router, b.topk_idx, b.topk_w, b.offsets, b.perm, b.active, b.slot_out,
              b.shared_out, b.y, b.ws, bias=L.bias, logits=b.logits, steer_v=L.steer_v, steer_f=L.steer_f,
              stream=stream)
    return b.y
