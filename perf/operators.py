"""Cases of the operators around the routed experts: the residual norm, the combine that ends in it, and the shared
expert with low-rank adapters.

  add_rms_norm   s = x + residual, stored in the residual's type; y = s / sqrt(mean(s^2) + eps) * weight, in bf16,
                 fp32 or 8 bits (e4m3 with a power-of-two scale per 32 columns, or with one fp32 scale per row)
  combine_norm   the same norm of residual + sum_j w[t][j] o[t*k+j] + shared[t] (optionally steered along v first)
  shared_ffn     Wd' (silu(Wg' x) * (Wu' x)) with W' = W + scale_a B_a A_a, a the token's adapter (or none)

Each case is one call on synthetic inputs of seeded draws.  `run` computes it with elementary torch operations in
fp32, or with the library's entry points where `own` is set; `exact` computes it in binary64.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _norm(name, T, H, x, res, w, y):
    return {"name": name, "op": "add_rms_norm", "T": T, "H": H, "x": x, "res": res, "w": w, "y": y}


def _combine(name, T, k, H, shared, steer, res, y):
    return {"name": name, "op": "combine_norm", "T": T, "k": k, "H": H, "shared": shared, "steer": steer, "res": res,
            "w": "bf16", "y": y}


def _shared(name, T, H, I, n, R, mix, out, x="bf16"):
    return {"name": name, "op": "shared_ffn", "T": T, "H": H, "I": I, "n": n, "R": R, "mix": mix, "x": x, "out": out}


def listed():
    return [
        # one decode token: the fp32 layer output joins a bf16 residual stream
        _norm("norm 1x4096", 1, 4096, "f32", "bf16", "bf16", "bf16"),
        # a batch of odd length over an odd, unaligned row length
        _norm("norm 515x2055", 515, 2055, "bf16", "bf16", "bf16", "bf16"),
        # the whole 11,709-token prompt, rows leaving in 8 bits with block scales for an 8-bit projection
        _norm("norm 11709x4096 mx8", 11709, 4096, "bf16", "bf16", "bf16", "mx8"),
        # a prefill chunk with an fp32 residual stream and 8-bit rows with row scales
        _norm("norm 1469x4096 row8", 1469, 4096, "f32", "f32", "f32", "row8"),
        # end of the layer at one decode token: top-8 combine, shared expert, residual, norm
        _combine("combine 1x8x4096", 1, 8, 4096, True, False, "bf16", "bf16"),
        # a ragged batch of a smaller top-4 layer with steering and an fp32 residual stream
        _combine("combine 131x4x1024 steer", 131, 4, 1024, True, True, "f32", "f32"),
        # end of the layer for a 2048-token prefill chunk
        _combine("combine 2048x8x4096", 2048, 8, 4096, True, False, "bf16", "mx8"),
        # shared expert at one decode token of one request with an adapter
        _shared("shared 1 token", 1, 4096, 2048, 8, 16, "each", "f32"),
        # one decode step of 24 requests, nearly each with an adapter of its own, of mixed ranks
        _shared("shared 24 requests", 24, 4096, 2048, 32, 64, "each", "f32"),
        # a small layer with fp32 activations and sizes that are no multiples of a tile
        _shared("shared 333x1000x520", 333, 1000, 520, 5, 24, "each", "f32", x="f32"),
        # a 512-token chunk holding the prompts of several requests
        _shared("shared 512 tokens", 512, 4096, 2048, 16, 16, "runs", "f32"),
        # a 2048-token chunk, bf16 result
        _shared("shared 2048 tokens", 2048, 4096, 2048, 8, 32, "runs", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_rms_norm", "combine_norm", "shared_ffn"])
    if op == "add_rms_norm":
        H = rng.choice([_log(rng, 64, 8192), 32 * _log(rng, 2, 256), 64 * _log(rng, 1, 128)])
        T = _log(rng, 1, min(16384, 11709 * 4096 // H))
        return {"op": op, "T": T, "H": H, "x": rng.choice(["f32", "bf16"]), "res": rng.choice(["f32", "bf16", "bf16", "none"]),
                "w": rng.choice(["f32", "bf16"]), "y": rng.choice(["bf16", "f32", "mx8", "row8"])}
    if op == "combine_norm":
        H = rng.choice([_log(rng, 64, 8192), 64 * _log(rng, 1, 128)])
        k = rng.choice([1, 2, 4, 6, 8, 8, 16])
        T = _log(rng, 1, min(4096, 2048 * 8 * 4096 // (k * H)))
        return {"op": op, "T": T, "k": k, "H": H, "shared": rng.random() < 0.75, "steer": rng.random() < 0.25,
                "res": rng.choice(["f32", "bf16"]), "w": rng.choice(["f32", "bf16"]),
                "y": rng.choice(["bf16", "f32", "mx8", "row8"])}
    H, I = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 256)
    T = _log(rng, 1, 2048)
    return {"op": op, "T": T, "H": H, "I": I, "n": _log(rng, 1, 48), "R": 8 * _log(rng, 1, 8),
            "mix": rng.choice(["each", "runs", "one", "none"]), "x": rng.choice(["bf16", "bf16", "f32"]),
            "out": rng.choice(["f32", "bf16"])}


def _ranks(case):
    """Ranks of the adapters in the pool: the full rank, half of it, and odd ones below it, in turn."""
    R = case["R"]
    return [max(1, [R, R // 2, R, R - 3][a % 4]) for a in range(case["n"])]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, H = case["T"], case["H"]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "shared_ffn":
        return _prepare_shared(case, g, normal, s)
    if case["op"] == "add_rms_norm":
        s["x"] = normal(T, H, dtype=DTYPES[case["x"]])
    else:
        k = case["k"]
        s["slot_out"] = normal(T * k, H)
        s["topk_w"] = torch.softmax(normal(T, k), dim=1)
        s["shared_out"] = normal(T, H) if case["shared"] else None
        s["steer_v"] = normal(H, std=1.0 / math.sqrt(H)) if case["steer"] else None
    res = None if case["res"] == "none" else DTYPES[case["res"]]
    s["residual"] = None if res is None else normal(T, H, std=2.0, dtype=res)
    s["residual_out"] = None if res is None else torch.empty(T, H, dtype=res, device="cuda")
    s["weight"] = normal(H, std=0.1, mean=1.0, dtype=DTYPES[case["w"]])
    y = case["y"]
    s["y"] = torch.empty(T, H, dtype=DTYPES.get(y, E4M3), device="cuda")
    s["y_scale"] = (torch.empty(T, (H + 31) // 32, dtype=E8M0, device="cuda") if y == "mx8" else
                    torch.empty(T, device="cuda") if y == "row8" else None)
    return s


def _prepare_shared(case, g, normal, s):
    T, H, I, n, R = (case[c] for c in ("T", "H", "I", "n", "R"))
    b = torch.bfloat16
    s["x"] = normal(T, H, dtype=DTYPES[case["x"]])
    s["gate"], s["up"], s["down"] = (normal(I, H, std=0.02, dtype=b), normal(I, H, std=0.02, dtype=b),
                                     normal(H, I, std=0.02, dtype=b))
    for p, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
        s[p + "_a"], s[p + "_b"] = normal(n, R, cols, std=0.02, dtype=b), normal(n, rows, R, std=0.02, dtype=b)
    s["rank"] = torch.tensor(_ranks(case), dtype=torch.int32, device="cuda")
    s["scale"] = 1.0 + torch.rand(n, generator=g, device="cuda")
    if case["mix"] == "each":       # every token its own request: adapters spread evenly, some tokens without one
        ids = (torch.arange(T, device="cuda") + int(torch.randint(n + 1, (1,), generator=g, device="cuda"))) % (n + 1) - 1
        ids = ids[torch.randperm(T, generator=g, device="cuda")]
    elif case["mix"] == "runs":     # prompts of several requests one after another
        cut = torch.sort(torch.randint(T + 1, (min(n, T),), generator=g, device="cuda")).values
        ids = torch.searchsorted(cut, torch.arange(T, device="cuda"), right=True) - 1
    elif case["mix"] == "one":
        ids = torch.full((T,), int(torch.randint(n, (1,), generator=g, device="cuda")), device="cuda")
    else:
        ids = torch.full((T,), -1, device="cuda")
    s["ids"] = ids.to(torch.int32)
    s["out"] = torch.empty(T, H, dtype=DTYPES[case["out"]], device="cuda")
    if own:                         # what a serving program keeps: the layer's and the pool's descriptions, a workspace
        import bit_quantized_moe_permute_amd as m
        s["m"] = m
        s["desc"] = m.LayerDesc(hidden=H, shared_inter=I, shared_gate=s["gate"].data_ptr(),
                                shared_up=s["up"].data_ptr(), shared_down=s["down"].data_ptr())
        s["pool"] = m.AdapterPool(H, I, rank=s["rank"], scale=s["scale"],
                                  **{p: (s[p + "_a"], s[p + "_b"]) for p in ("gate", "up", "down")})
        s["ws"] = torch.empty(m.moe_shared_ffn_workspace(s["desc"], T, s["pool"]), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"add_rms_norm": _own_norm, "combine_norm": _own_combine, "shared_ffn": _own_shared}[op](s)
    return {"add_rms_norm": _plain_norm, "combine_norm": _plain_combine, "shared_ffn": _plain_shared}[op](s)


def _own_norm(s):
    import bit_quantized_moe_permute_amd as m
    m.moe_add_rms_norm(s["x"], s["residual"], s["residual_out"], s["weight"], EPS, s["y"], s["y_scale"])
    return [s["residual_out"], s["y"], s["y_scale"]]


def _own_combine(s):
    import bit_quantized_moe_permute_amd as m
    m.moe_combine_norm(s["slot_out"], s["topk_w"], s["shared_out"], s["residual"], s["residual_out"], s["weight"], EPS,
                       s["y"], s["y_scale"], steer_v=s["steer_v"], steer_f=0.75)
    return [s["residual_out"], s["y"], s["y_scale"]]


def _own_shared(s):
    s["m"].moe_shared_ffn(s["desc"], s["x"], s["out"], s["ws"], s["pool"], s["ids"])
    return s["out"]


def _plain_tail(s, v):
    """Residual addition, norm and output rounding of the fp32 rows v."""
    stored = None
    if s["residual"] is not None:
        stored = (v + s["residual"].float()).to(s["residual"].dtype)
        v = stored.float()
    y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    return [stored, *_plain_round(y, s["case"]["y"])]


def _plain_round(y, kind):
    if kind in DTYPES:
        return y.to(DTYPES[kind]), None
    if kind == "row8":
        scale = y.abs().amax(dim=1).clamp_min(448 * 2.0**-126) / 448
        return (y / scale[:, None]).to(E4M3), scale
    T, H = y.shape
    y = torch.nn.functional.pad(y, (0, -H % 32)).reshape(T, -1, 32)
    m, p = torch.frexp(y.abs().amax(dim=2))              # amax = m 2^p: the least e with amax <= 448 2^e
    e = torch.where(m == 0, -127, torch.where(m > 0.875, p - 8, p - 9)).clamp(-127, 127)
    q = torch.ldexp(y, -e[..., None]).to(E4M3)
    return q.reshape(T, -1)[:, :H].contiguous(), (e + 127).to(torch.uint8).view(E8M0)


def _plain_norm(s):
    return _plain_tail(s, s["x"].float())


def _plain_combine(s):
    case = s["case"]
    v = (s["slot_out"].reshape(case["T"], case["k"], case["H"]) * s["topk_w"][:, :, None]).sum(dim=1)
    if s["shared_out"] is not None:
        v = v + s["shared_out"]
    if s["steer_v"] is not None:
        v = v - 0.75 * (v * s["steer_v"]).sum(dim=1, keepdim=True) * s["steer_v"]
    return _plain_tail(s, v)


def _plain_project(s, x, p):
    """x W^T + scale (x A^T) B^T of projection p: every adapter's products at once, kept where they are the token's."""
    w, a, b, ids = s[p], s[p + "_a"], s[p + "_b"], s["ids"]
    n, R, _ = a.shape
    col = torch.arange(n * R, device="cuda")
    used = col % R < s["rank"][col // R]
    keep = (ids[:, None] == col // R) & used
    u = torch.where(keep, (x @ a.reshape(n * R, -1).float().T) * s["scale"][col // R], 0.0)
    return x @ w.float().T + u @ b.permute(0, 2, 1).reshape(n * R, -1).float()


def _plain_shared(s):
    x = s["x"].float()
    gate, up = _plain_project(s, x, "gate"), _plain_project(s, x, "up")
    return _plain_project(s, gate / (1 + torch.exp(-gate)) * up, "down").to(s["out"].dtype)


# ----------------------------------------------------------------------------
# binary64
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "shared_ffn":
        return _exact_shared(case, s)
    if case["op"] == "combine_norm":
        o = s["slot_out"].view(case["T"], case["k"], -1)
        v = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            v += o[:, j].double() * s["topk_w"][:, j, None].double()
        if case["shared"]:
            v += s["shared_out"]
        if case["steer"]:
            d = s["steer_v"].double()
            v -= 0.75 * torch.outer(v @ d, d)
    else:
        v = s["x"].double()
    stored = None
    if s["residual"] is not None:
        stored = (v + s["residual"].double()).to(s["residual"].dtype)
        v = stored.double()
    rms = torch.sqrt(torch.square(v).sum(dim=1) / case["H"] + EPS)
    y = s["weight"].double()[None] * v / rms[:, None]
    if case["y"] in DTYPES:
        return [stored, y, None]
    if case["y"] == "row8":
        scale = torch.maximum(y.abs().max(dim=1).values / 448, torch.tensor(2.0**-126, dtype=torch.float64, device="cuda"))
        return [stored, (y / scale[:, None]).to(E4M3), scale.float()]
    blocks = torch.split(y, 32, dim=1)
    big = torch.stack([c.abs().max(dim=1).values for c in blocks], dim=1)
    e = torch.ceil(torch.log2(big / 448)).clamp(-127, 127)
    e = torch.where(big > 448 * torch.exp2(e), e + 1, torch.where(big <= 224 * torch.exp2(e), e - 1, e)).clamp(-127, 127)
    q = y / torch.repeat_interleave(torch.exp2(e), 32, dim=1)[:, :case["H"]]
    return [stored, q.to(E4M3), torch.exp2(e).to(E8M0)]


def _exact_shared(case, s):
    def project(x, p):
        out = x @ s[p].double().t()
        for a, r in enumerate(_ranks(case)):
            rows = (s["ids"] == a).nonzero().flatten()
            if len(rows):
                low = x[rows] @ s[p + "_a"][a, :r].double().t()
                out[rows] += float(s["scale"][a]) * (low @ s[p + "_b"][a, :, :r].double().t())
        return out

    x = s["x"].double()
    gate = project(x, "gate")
    h = gate * torch.sigmoid(gate) * project(x, "up")
    return project(h, "down")


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    T, H = case["T"], case["H"]
    size = {"f32": 4, "bf16": 2, "none": 0, "mx8": 1 + 1 / 32, "row8": 1}
    if case["op"] == "shared_ffn":
        I, n = case["I"], case["n"]
        with_one = {"each": T * n // (n + 1), "none": 0}.get(case["mix"], T)
        used = {"each": min(n, T), "runs": min(n, T), "one": 1, "none": 0}[case["mix"]]
        rank = sum(_ranks(case)) / n
        low = rank * 3 * (H + I)                         # values of one adapter's six matrices
        return {"bytes": 2 * (3 * H * I + used * low) + T * H * (size[case["x"]] + size[case["out"]]) + 4 * T,
                "flops": 6 * T * H * I + 2 * with_one * low}
    rows = T * H * (2 * size[case["res"]] + size[case["y"]]) + H * size[case["w"]] + (4 * T if case["y"] == "row8" else 0)
    if case["op"] == "add_rms_norm":
        return {"bytes": T * H * size[case["x"]] + rows, "flops": 6 * T * H}
    k = case["k"]
    return {"bytes": 4 * T * H * (k + case["shared"]) + 4 * T * k + rows + (4 * H if case["steer"] else 0),
            "flops": (2 * k + 6 + 4 * case["steer"]) * T * H}
