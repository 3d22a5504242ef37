"""Cases of the products over rows grouped by expert, with bf16 and with 4-bit weights.

  grouped_linear   out[row] = W_e x[row] for the rows of each expert e, or silu(Wg x) * (Wu x) with W_e = [Wg; Wu]
  grouped_dgrad    dx[row] = W_e^T dy[row]
  grouped_wgrad    dW_e = sum over the rows of e of dy[row] x[row]^T
  q4_linear        grouped_linear with 4-bit weights: W[n][k] = (code[n][k] - zero[n][k / group]) * scale[n][k / group]

Rows are the (token, choice) slots s = t * k + j of a top-k router, sorted by expert; x may be the tokens themselves (slot s
reads row s / k), and what stands on the output's side may be in slot order.  Without a router (k = 0) one matrix takes
every token.  Each case is one call on synthetic inputs of seeded draws.  `run` computes it with elementary torch operations
in fp32, or with the library's entry points where `own` is set; `exact` computes it in binary64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _case(name, op, T, k, E, n_in, n_out, out, src="tokens", dst="sorted", act="none", skew=0.0, **more):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "n_in": n_in, "n_out": n_out, "out": out, "src": src, "dst": dst,
            "act": act, "skew": skew, **more}


def listed():
    return [
        # one decode token through its 8 of 256 unquantized experts: gate, up and SwiGLU
        _case("linear 1 token", "grouped_linear", 1, 8, 256, 4096, 2048, "bf16", act="swiglu"),
        # a small layer and a ragged batch: sizes that are no multiples of a tile
        _case("linear 300x4 1000x520", "grouped_linear", 300, 4, 16, 1000, 520, "bf16", src="sorted", skew=0.5),
        # a 2048-token prefill chunk over 256 experts, some 64 rows each: gate, up and SwiGLU
        _case("linear 2048 tokens", "grouped_linear", 2048, 8, 256, 4096, 2048, "bf16", act="swiglu"),
        # the whole 11,709-token prompt over 32 experts
        _case("linear 11709 tokens", "grouped_linear", 11709, 8, 32, 4096, 2048, "bf16", act="swiglu", skew=0.25),
        # a ragged batch of a small layer: the gradient of its input
        _case("dgrad 131x4 1000x520", "grouped_dgrad", 131, 4, 16, 1000, 520, "f32", src="sorted", dst="slots"),
        # a training step of 2048 tokens: the gradient that the down projection hands back to the SwiGLU
        _case("dgrad 2048 tokens", "grouped_dgrad", 2048, 8, 32, 2048, 4096, "bf16", src="sorted", dst="slots", skew=0.25),
        # weight gradients of a small layer, experts with few rows and with none
        _case("wgrad 77x2 512x1000", "grouped_wgrad", 77, 2, 32, 512, 1000, "bf16", skew=1.0),
        # a training step of 2048 tokens: gradients of the stacked gate and up projections
        _case("wgrad 2048 tokens", "grouped_wgrad", 2048, 8, 32, 4096, 4096, "f32", skew=0.25),
        # one decode token through a dense projection
        _case("q4 1 token", "q4_linear", 1, 0, 1, 4096, 4096, "bf16", group=32, zero=False, scale="f16"),
        # one decode step of 24 requests through an output projection
        _case("q4 24 requests", "q4_linear", 24, 0, 1, 4096, 32768, "f32", group=128, zero=True, scale="bf16"),
        # a verify step of 3 tokens, each through its 8 of 256 experts: gate, up and SwiGLU
        _case("q4 3 tokens experts", "q4_linear", 3, 8, 256, 4096, 2048, "bf16", act="swiglu", group=64, zero=False, scale="f16"),
        # a skewed 512-token chunk through the experts' down projections, back to slot order
        _case("q4 512 tokens experts", "q4_linear", 512, 8, 256, 2048, 4096, "f32", src="sorted", dst="slots", skew=0.5,
              group=32, zero=True, scale="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped_linear", "grouped_dgrad", "grouped_wgrad", "q4_linear"])
    c = {"op": op, "out": rng.choice(["bf16", "f32"]), "skew": rng.choice([0.0, 0.25, 0.5, 1.0])}
    if op == "q4_linear":
        c["group"] = rng.choice([32, 64, 128])
        c["zero"] = rng.random() < 0.5
        c["scale"] = rng.choice(["f16", "bf16", "f32"])
        c["n_in"] = c["group"] * _log(rng, 4, 4096 // c["group"])
        c["n_out"] = _log(rng, 64, 8192)
    else:
        c["n_in"], c["n_out"] = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 512)
    c["E"], c["k"] = _log(rng, 1, 128), rng.choice([1, 2, 4, 6, 8])
    c["k"] = min(c["k"], c["E"])
    if op == "q4_linear" and rng.random() < 0.5:
        c["E"], c["k"] = 1, 0
    c["src"] = rng.choice(["tokens", "sorted"]) if c["k"] else "tokens"
    c["dst"] = rng.choice(["slots", "sorted"]) if c["k"] else "sorted"
    c["act"] = "swiglu" if op in ("grouped_linear", "q4_linear") and rng.random() < 0.4 else "none"
    # no more products than a 2048-token chunk of 8 choices, 4096 x 4096
    most = 2048 * 8 * 4096 * 4096 // (max(c["k"], 1) * c["n_in"] * c["n_out"] * (2 if c["act"] == "swiglu" else 1))
    c["T"] = _log(rng, 1, min(2048 if op == "q4_linear" else 8192, most))
    return c


def _rows(case):
    return case["T"] * max(case["k"], 1)


def _weight_rows(case):
    return case["n_out"] * (2 if case["act"] == "swiglu" else 1)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _route(case, g, s):
    """A router's choices: k different experts per token, skewed by a per-expert bias; slots sorted by expert."""
    T, k, E = case["T"], case["k"], case["E"]
    if not k:
        s["counts"], s["perm"], s["offsets"] = [T], None, None
        return
    score = torch.randn(T, E, generator=g, device="cuda") + case["skew"] * torch.randn(E, generator=g, device="cuda")
    expert = score.topk(k, dim=1).indices.reshape(-1)
    perm = torch.sort(expert, stable=True).indices
    counts = torch.bincount(expert, minlength=E)
    s["counts"] = counts.tolist()
    s["perm"] = perm.to(torch.int32)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _quantize(w, group, zero, dtype):
    """Codes (two to a byte, the even column low), scales and zero points of the rows of one matrix."""
    N, K = w.shape
    v = w.view(N, K // group, group)
    if zero:
        lo, hi = v.amin(dim=2).clamp_max(0), v.amax(dim=2).clamp_min(0)
        scale = ((hi - lo) / 15).clamp_min(1e-8).to(dtype)
        z = torch.round(-lo / scale.float()).clamp(0, 15)
    else:
        scale = (v.abs().amax(dim=2) / 7).clamp_min(1e-8).to(dtype)
        z = torch.full_like(scale, 8, dtype=torch.float32)
    q = (torch.round(v / scale.float()[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8).view(N, K // 2, 2)
    return q[..., 0] | (q[..., 1] << 4), scale, z.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, n_in, n_out, E, R = case["op"], case["n_in"], case["n_out"], case["E"], _rows(case)
    N, bf = _weight_rows(case), torch.bfloat16

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=bf).mul_(std)

    s = {"case": case}
    _route(case, g, s)
    if op != "grouped_dgrad":
        s["x"] = normal(case["T"] if case["src"] == "tokens" else R, n_in)
    if op in ("grouped_dgrad", "grouped_wgrad"):
        s["dy"] = normal(R, n_out, std=0.1)
    if op == "q4_linear":
        G = case["group"]
        s["codes"] = torch.empty(E, N, n_in // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(E, N, n_in // G, dtype=DTYPES[case["scale"]], device="cuda")
        s["zero"] = torch.empty(E, N, n_in // G, dtype=torch.uint8, device="cuda")
        for e in range(E):
            w = torch.randn(N, n_in, generator=g, device="cuda") * 0.02
            s["codes"][e], s["scale"][e], s["zero"][e] = _quantize(w, G, case["zero"], s["scale"].dtype)
        if not case["zero"]:
            s["zero"] = None
    elif op != "grouped_wgrad":
        s["w"] = normal(E, N, n_in, std=0.02)
    shape = {"grouped_dgrad": (R, n_in), "grouped_wgrad": (E, n_out, n_in)}.get(op, (R, n_out))
    s["out"] = torch.empty(shape, dtype=DTYPES[case["out"]], device="cuda")
    if own:                         # what a program keeps beside a router's result and its weights: their descriptions
        import bit_quantized_moe_permute_amd as m
        s["m"] = m
        tokens = case["src"] == "tokens" and case["k"]
        s["groups"] = m.RowGroups(R, offsets=s["offsets"], in_index=s["perm"] if tokens else None,
                                  in_div=case["k"] if tokens and op != "grouped_dgrad" else 1,
                                  out_index=s["perm"] if case["dst"] == "slots" else None)
        if op == "q4_linear":
            s["q4"] = m.Q4Weights(s["codes"], s["scale"], s["zero"])
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    m, op = s["m"], s["case"]["op"]
    act = m.ACT_SWIGLU if s["case"]["act"] == "swiglu" else m.ACT_NONE
    if op == "grouped_linear":
        m.moe_grouped_linear(s["groups"], s["x"], s["w"], s["out"], act)
    elif op == "grouped_dgrad":
        m.moe_grouped_dgrad(s["groups"], s["dy"], s["w"], s["out"])
    elif op == "grouped_wgrad":
        m.moe_grouped_wgrad(s["groups"], s["x"], s["dy"], s["out"])
    else:
        m.moe_q4_linear(s["groups"], s["q4"], s["x"], s["out"], act)
    return s["out"]


def _in_rows(s, b, e):
    """Rows of x (of dx for the input's gradient) that the sorted slots b .. e - 1 have."""
    c = s["case"]
    if c["src"] == "sorted" or not c["k"]:
        return slice(b, e)
    p = s["perm"][b:e].long()
    return p if c["op"] == "grouped_dgrad" else p // c["k"]


def _out_rows(s, b, e):
    return s["perm"][b:e].long() if s["case"]["dst"] == "slots" else slice(b, e)


def _weights(s, e):
    """Matrix e in fp32."""
    if "w" in s:
        return s["w"][e].float()
    c, codes = s["case"], s["codes"][e]
    q = torch.stack([codes & 15, codes >> 4], dim=2).reshape(codes.shape[0], -1, c["group"]).float()
    z = 8.0 if s["zero"] is None else s["zero"][e].float()[..., None]
    return ((q - z) * s["scale"][e].float()[..., None]).view(codes.shape[0], -1)


def _plain(s):
    c, out, b = s["case"], torch.empty_like(s["out"]), 0
    for e, n in enumerate(s["counts"]):
        rows, b = (b, b + n), b + n
        if c["op"] == "grouped_wgrad":
            out[e] = s["dy"][_out_rows(s, *rows)].float().T @ s["x"][_in_rows(s, *rows)].float()
            continue
        if n == 0:
            continue
        if c["op"] == "grouped_dgrad":
            out[_in_rows(s, *rows)] = (s["dy"][_out_rows(s, *rows)].float() @ _weights(s, e)).to(out.dtype)
            continue
        y = s["x"][_in_rows(s, *rows)].float() @ _weights(s, e).T
        if c["act"] == "swiglu":
            gate, up = y[:, :c["n_out"]], y[:, c["n_out"]:]
            y = gate / (1 + torch.exp(-gate)) * up
        out[_out_rows(s, *rows)] = y.to(out.dtype)
    return out


# ----------------------------------------------------------------------------
# binary64
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f64, R, k = torch.float64, _rows(case), case["k"]
    # for every slot in sorted order: its expert, and the rows on either side
    slot = torch.arange(R, device="cuda") if s["perm"] is None else s["perm"].long()
    expert = torch.repeat_interleave(torch.arange(case["E"], device="cuda"), torch.tensor(s["counts"], device="cuda"))
    here = torch.arange(R, device="cuda")
    near = here if case["src"] == "sorted" else slot // k if k and case["op"] != "grouped_dgrad" else slot
    far = slot if case["dst"] == "slots" else here
    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    for e in range(case["E"]):
        mine = torch.nonzero(expert == e).flatten()
        if mine.numel() == 0:
            continue
        i, o = near[mine], far[mine]
        if case["op"] == "grouped_wgrad":
            out[e] = torch.matmul(s["dy"].index_select(0, o).to(f64).t(), s["x"].index_select(0, i).to(f64))
            continue
        if case["op"] == "q4_linear":
            packed, group = s["codes"][e], case["group"]
            w = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=f64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (packed % 16).to(f64), (packed // 16).to(f64)
            w -= torch.repeat_interleave(s["zero"][e].to(f64), group, dim=1) if case["zero"] else 8
            w *= torch.repeat_interleave(s["scale"][e].to(f64), group, dim=1)
        else:
            w = s["w"][e].to(f64)
        if case["op"] == "grouped_dgrad":
            out.index_copy_(0, i, torch.matmul(s["dy"].index_select(0, o).to(f64), w))
            continue
        y = torch.matmul(s["x"].index_select(0, i).to(f64), w.t())
        if case["act"] == "swiglu":
            gate, up = torch.chunk(y, 2, dim=1)
            y = gate * torch.sigmoid(gate) * up
        out.index_copy_(0, o, y)
    return out


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    R, E, n_in, n_out, N = _rows(case), case["E"], case["n_in"], case["n_out"], _weight_rows(case)
    used = E * (1 - (1 - max(case["k"], 1) / E) ** case["T"])            # experts with a row, expected (without skew)
    size = 4 if case["out"] == "f32" else 2
    flops, index = 2 * R * N * n_in, 4 * R * ((case["src"] == "tokens") + (case["dst"] == "slots")) if case["k"] else 0
    x = 2 * n_in * (case["T"] if case["src"] == "tokens" else R)
    if case["op"] == "grouped_wgrad":
        return {"bytes": x + 2 * R * n_out + size * E * n_out * n_in + index, "flops": flops}
    if case["op"] == "grouped_dgrad":
        return {"bytes": 2 * used * n_out * n_in + 2 * R * n_out + size * R * n_in + index, "flops": flops}
    if case["op"] == "q4_linear":
        per_group = {"f32": 4, "bf16": 2, "f16": 2}[case["scale"]] + case["zero"]
        weights = used * N * n_in * (0.5 + per_group / case["group"])
    else:
        weights = 2 * used * N * n_in
    return {"bytes": weights + x + size * R * n_out + index, "flops": flops}
