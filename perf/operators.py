"""The expert operators around the layer: cases, inputs, plain forms and 64-bit values.

Tokens sorted by expert and back (dispatch, combine) with their gradients, the block
quantisers to 8-bit floating point, the grouped 8-bit product with one scale per block of
128 (forward, both gradients, and fused with the activation), and the activation between
an expert's two products.

A case names its operator in ``op`` and gives M tokens of H values, K slots a token, E
experts, and where it matters N (output features) or I (intermediate features).  ``skew``
is the Zipf exponent of the expert choice, ``drop`` the share of slots that were dropped
(a capacity limit), ``type`` the type of the rows, ``fp8`` the 8-bit type.
"""
import math

import torch

own = False  # True: run() calls the package's operators; False: their plain form

BLOCK = 128
FLOOR = 2.0 ** -96  # smallest block maximum a scale is made from
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}


def _case(name, op, M, H, K, E, **kw):
    c = {"name": name, "op": op, "M": M, "H": H, "K": K, "E": E, "skew": 0.3, "drop": 0.0, "type": "bf16",
         "fp8": "e4m3"}
    c.update(kw)
    return c


def listed():
    return [
        # One decoded token of the H=2048, E=256, top-8 layer: the rows of its 8 experts, as
        # 8-bit rows and scales.  Latency alone.
        _case("dispatch_fp8_M1", "dispatch_quantize", 1, 2048, 8, 256),
        # A training batch of the E=512, top-10 layer with a capacity limit that drops slots.
        _case("dispatch_M8192_drop", "dispatch", 8192, 2560, 10, 512, skew=0.5, drop=0.08),
        # Prefill of the H=2048 layer: the experts' outputs weighted and summed per token.
        _case("combine_M4096", "combine", 4096, 2048, 8, 256),
        # The same step's gradient in FP32 at an odd number of tokens (H=2688, top-6).
        _case("combine_bwd_M2047_f32", "combine_backward", 2047, 2688, 6, 128, type="f32"),
        # Activations of the weight gradient: 128-row blocks inside each expert, ragged ends,
        # I=1856 (14.5 blocks of 128).
        _case("quant_cols_M4095", "quantize_columns", 4095, 1856, 6, 128, skew=0.5, fp8="e5m2"),
        # One layer's FC1 weights (E=128 experts of [1856, 2688]) to 8 bits, once a step.
        _case("quant_blocks_E128", "quantize_blocks", 1, 2688, 1, 128, N=1856),
        # Decode of 16 sequences: FC1 of the H=2048 layer, about one row an expert; the bytes of
        # the touched experts' weights are the work.
        _case("product_M16", "product", 16, 2048, 8, 256, N=1024),
        # Prefill: FC1 over 65536 rows, 256 a expert on average.
        _case("product_M8192", "product", 8192, 2048, 8, 256, N=1024),
        # The input gradient of an FC1 with ragged blocks both ways (N=1856, H=2688).
        _case("input_grad_M4096", "product_input_grad", 4096, 2688, 6, 128, N=1856, fp8="e5m2"),
        # The weight gradient of the H=2560, I=640 layer's FC2 (N=2560 outputs of 640 inputs).
        _case("weight_grad_M4096", "product_weight_grad", 4096, 640, 10, 512, N=2560, skew=0.5, out="f32"),
        # Serving: FC1, SwiGLU and the quantiser of FC2's input in one call.
        _case("product_act_M2048", "product_activation", 2048, 2560, 10, 512, I=640, act="swiglu"),
        # Training: the gradient through SwiGLU.
        _case("act_bwd_M4096", "activation_backward", 4096, 0, 8, 256, I=512, act="swiglu"),
    ]


OPS = ("dispatch", "dispatch_backward", "dispatch_quantize", "combine", "combine_backward", "quantize_rows",
       "quantize_columns", "quantize_blocks", "product", "product_activation", "product_input_grad",
       "product_weight_grad", "activation", "activation_quantize", "activation_backward")


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(OPS)
    E = _log(rng, 1, 256)
    K = rng.randint(1, min(8, E))
    M = _log(rng, 1, 8192)
    if rng.random() < 0.5:
        M |= 1
    H, N, I = _log(rng, 256, 2688, 16), _log(rng, 128, 2048, 16), _log(rng, 64, 1856, 16)
    c = {"op": op, "M": M, "H": H, "K": K, "E": E, "skew": rng.choice((0.0, 0.3, 0.6)), "drop": 0.0,
         "type": "bf16", "fp8": "e4m3"}
    if op in ("dispatch", "dispatch_backward", "dispatch_quantize", "combine", "combine_backward"):
        c["drop"] = rng.choice((0.0, 0.0, 0.1))
        c["type"] = rng.choice(("bf16", "bf16", "f32"))
    if op.startswith("quantize"):
        c["type"] = rng.choice(("bf16", "f32"))
    if "quantize" in op or op in ("product_input_grad", "product_weight_grad"):
        c["fp8"] = rng.choice(("e4m3", "e5m2"))
    if op == "quantize_blocks":
        c.update(M=1, K=1, N=N)
        c["E"] = max(1, min(E, 2 ** 28 // (N * H)))
    if op in ("product", "product_input_grad", "product_weight_grad"):
        c["N"] = N
        c["out"] = rng.choice(("bf16", "f32"))
    if op in ("product_activation", "activation", "activation_quantize", "activation_backward"):
        c.update(I=I, act=rng.choice(("swiglu", "relu2")))
    feats = c.get("N", 2 * I if "I" in c else 1)
    while c["M"] > 64 and (2.0 * c["M"] * K * feats * H > 2.0e11 or c["M"] * K * max(H, feats) > 6e7):
        c["M"] = c["M"] // 2 + 1
    return c


# ---------------------------------------------------------------- inputs
def _route(c, g):
    """Expert choice of M tokens: rows sorted by expert (inv, offsets) and host counts."""
    M, K, E, dev = c["M"], c["K"], c["E"], "cuda"
    ranks = torch.randperm(E, generator=g, device=dev).double() + 1.0
    u = torch.rand((M, E), generator=g, device=dev, dtype=torch.float64).clamp_(min=1e-300)
    ids = (-c["skew"] * ranks.log() - (-u.log()).log()).topk(K, dim=1).indices
    flat = ids.reshape(-1)
    P = M * K - int(M * K * c["drop"])
    if P < M * K:
        flat[torch.randperm(M * K, generator=g, device=dev)[P:]] = E
    order = flat.argsort(stable=True)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0)
    kept = order[:P]
    inv = torch.full((M * K,), -1, dtype=torch.int32, device=dev)
    inv[(kept % K) * M + kept // K] = torch.arange(P, dtype=torch.int32, device=dev)
    host = counts.tolist()
    return {"inv": inv, "offsets": offsets, "P": P, "cap": max(host), "blocks": P // BLOCK + min(E, P)}


def _randn(shape, g, dtype, scale=1.0):
    """Normal values whose rows differ in size, as activations and gradients do."""
    t = torch.randn(shape, generator=g, device="cuda")
    if len(shape) == 2:
        t *= torch.exp(torch.randn((shape[0], 1), generator=g, device="cuda"))
    return (t * scale).to(dtype)


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "fp8": FP8[c["fp8"]], "fmax": FP8_MAX[c["fp8"]]}
    s.update(_route(c, g))
    M, H, K, E, P, dt = c["M"], c["H"], c["K"], c["E"], s["P"], TYPES[c["type"]]
    if op in ("combine", "combine_backward"):
        w = torch.rand((M, K), generator=g, device="cuda") + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
    if op in ("dispatch", "dispatch_quantize"):
        s["x"] = _randn((M, H), g, dt)
    elif op in ("dispatch_backward", "combine"):
        s["ys"] = _randn((P, H), g, dt)
    elif op == "combine_backward":
        s["dy"], s["ys"] = _randn((M, H), g, dt), _randn((P, H), g, dt)
    elif op in ("quantize_rows", "quantize_columns"):
        s["x"] = _randn((P, H), g, dt)
        if op == "quantize_columns":  # room for the worst split; what no expert fills stays zero
            s["room"] = (torch.zeros((s["blocks"] * BLOCK, H), dtype=torch.uint8, device="cuda").view(s["fp8"]),
                         torch.zeros((s["blocks"], H), device="cuda"))
    elif op == "quantize_blocks":
        s["w"] = _randn((E, c["N"], H), g, dt, H ** -0.5)
    elif op.startswith("product"):
        N = 2 * c["I"] if c.get("act") == "swiglu" else c.get("I", 0) or c["N"]
        s["out"] = TYPES[c.get("out", "bf16")]
        if op == "product_weight_grad":
            s["dy_q"], s["dy_s"] = _plain_quantize_columns(s, _randn((P, N), g, torch.bfloat16, 1e-3), c["fp8"])
            s["x_q"], s["x_s"] = _plain_quantize_columns(s, _randn((P, H), g, torch.bfloat16), "e4m3")
        else:
            w = _randn((E, N, H), g, torch.bfloat16, H ** -0.5)
            s["w_q"], s["w_s"] = _plain_quantize_blocks(w, "e4m3")
            del w
            cols, size = (N, 1e-3) if op == "product_input_grad" else (H, 1.0)
            s["x_q"], s["x_s"] = _plain_quantize_rows(_randn((P, cols), g, torch.bfloat16, size), c["fp8"])
    else:  # the activation alone
        s["y"] = _randn((P, c["I"] * (2 if c["act"] == "swiglu" else 1)), g, dt)
        if op == "activation_backward":
            s["dh"] = _randn((P, c["I"]), g, dt, 1e-3)
    return s


# ---------------------------------------------------------------- plain forms
def _scales(amax, fp8):
    """Scale and factor of blocks whose largest magnitudes are ``amax``."""
    a = amax.clamp(min=FLOOR)
    top = torch.full_like(a, FP8_MAX[fp8])
    return a / top, top / a


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _plain_quantize_rows(x, fp8):
    R, C = x.shape
    b = torch.nn.functional.pad(x.float(), (0, _padded(C) - C)).view(R, -1, BLOCK)
    s, f = _scales(b.abs().amax(2), fp8)
    return (b * f[:, :, None]).view(R, -1)[:, :C].to(FP8[fp8]), s


def _plain_quantize_blocks(w, fp8):
    E, N, H = w.shape
    p = torch.nn.functional.pad(w.float(), (0, _padded(H) - H, 0, _padded(N) - N))
    p = p.view(E, _padded(N) // BLOCK, BLOCK, -1, BLOCK)
    s, f = _scales(p.abs().amax((2, 4)), fp8)
    q = (p * f[:, :, None, :, None]).to(FP8[fp8]).view(E, _padded(N), _padded(H))
    return q[:, :N, :H].contiguous(), s


def _groups(s):
    """Expert of each row, and the row's place inside it."""
    off = s["offsets"].long()
    rows = torch.arange(s["P"], device=off.device)
    e = torch.searchsorted(off, rows, right=True) - 1
    return e, rows - off[e]


def _plain_quantize_columns(s, x, fp8):
    """128-row blocks inside each expert; every expert starts a new block, its last is padded with zeros.
    Blocks behind the last expert's are zero, and so are their scales."""
    off, n = s["offsets"].long(), s["blocks"]
    first = torch.nn.functional.pad(((off[1:] - off[:-1] + BLOCK - 1) // BLOCK).cumsum(0), (1, 0))
    e, j = _groups(s)
    p = torch.zeros((n * BLOCK, x.shape[1]), device=x.device)
    p[first[e] * BLOCK + j] = x.float()
    p = p.view(n, BLOCK, -1)
    sc, f = _scales(p.abs().amax(1), fp8)
    sc = torch.where(torch.arange(n, device=x.device)[:, None] < first[-1], sc, 0)
    return (p * f[:, None, :]).to(FP8[fp8]).view(n * BLOCK, -1), sc


def _rows_value(q, sc):
    return q.float() * sc.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _weights_value(s):
    q, sc = s["w_q"], s["w_s"]
    return q.float() * sc.repeat_interleave(BLOCK, 1)[:, :q.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :q.shape[2]]


def _grouped(s, x, w):
    """x [P, c] times w [E, c, n], each row with its expert's matrix."""
    e, j = _groups(s)
    p = torch.zeros((s["case"]["E"], s["cap"], x.shape[1]), device=x.device)
    p[e, j] = x
    return torch.bmm(p, w)[e, j]


def _plain_activation(y, act):
    if act == "relu2":
        return y.relu().square()
    g, u = y.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def _slots(s, rows):
    """rows[inv] as [K, M, H], zero where the slot was dropped, and which slots were kept."""
    c = s["case"]
    inv = s["inv"].view(c["K"], c["M"]).long()
    kept = (inv >= 0)[:, :, None]
    return torch.where(kept, rows[inv.clamp(min=0)], 0), kept


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    dt = TYPES[c["type"]]
    if op in ("dispatch", "dispatch_quantize", "combine_backward"):
        inv = s["inv"].long()  # the slot of each row; dropped slots go to a place behind the last row
        src = torch.empty(s["P"] + 1, dtype=torch.long, device="cuda")
        src[torch.where(inv < 0, s["P"], inv)] = torch.arange(len(inv), device="cuda")
        src = src[:-1]
        m = src % c["M"]
    if op == "dispatch":
        return s["x"][m]
    if op == "dispatch_quantize":
        q, sc = _plain_quantize_rows(s["x"], c["fp8"])
        return q.view(torch.uint8)[m].view(q.dtype), sc[m]
    if op == "dispatch_backward":
        return _slots(s, s["ys"].float())[0].sum(0).to(dt)
    if op == "combine":
        return (_slots(s, s["ys"].float())[0] * s["w"].t()[:, :, None]).sum(0).to(dt)
    if op == "combine_backward":
        dy = s["dy"].float()
        dw = (_slots(s, s["ys"].float())[0] * dy).sum(2).t()
        return (dy[m] * s["w"][m, src // c["M"]][:, None]).to(dt), dw.contiguous()
    if op == "quantize_rows":
        return _plain_quantize_rows(s["x"], c["fp8"])
    if op == "quantize_columns":
        return _plain_quantize_columns(s, s["x"], c["fp8"])
    if op == "quantize_blocks":
        return _plain_quantize_blocks(s["w"], c["fp8"])
    if op == "product":
        return _grouped(s, _rows_value(s["x_q"], s["x_s"]), _weights_value(s).transpose(1, 2)).to(s["out"])
    if op == "product_input_grad":
        return _grouped(s, _rows_value(s["x_q"], s["x_s"]), _weights_value(s)).to(s["out"])
    if op == "product_activation":
        y = _grouped(s, _rows_value(s["x_q"], s["x_s"]), _weights_value(s).transpose(1, 2))
        return _plain_quantize_rows(_plain_activation(y, c["act"]), c["fp8"])
    if op == "product_weight_grad":
        off = s["offsets"].long()
        blocks = (off[1:] - off[:-1] + BLOCK - 1) // BLOCK
        first = blocks.cumsum(0) - blocks
        b = torch.arange(-(-s["cap"] // BLOCK), device="cuda")
        have = (b < blocks[:, None])[:, :, None, None]
        at = torch.where(b < blocks[:, None], first[:, None] + b, 0)
        dy = (s["dy_q"].float().view(s["blocks"], BLOCK, -1) * s["dy_s"][:, None, :])[at]
        x = (s["x_q"].float().view(s["blocks"], BLOCK, -1) * s["x_s"][:, None, :])[at]
        dy = torch.where(have, dy, 0).flatten(1, 2)
        return torch.bmm(dy.transpose(1, 2), x.flatten(1, 2)).to(s["out"])
    y = s["y"].float()
    if op == "activation":
        return _plain_activation(y, c["act"]).to(dt)
    if op == "activation_quantize":
        return _plain_quantize_rows(_plain_activation(y, c["act"]), c["fp8"])
    dh = s["dh"].float()
    if c["act"] == "relu2":
        return (2 * y.relu() * dh).to(dt)
    g, u = y.chunk(2, 1)
    sg = torch.sigmoid(g)
    return torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], 1).to(dt)


def _own(s):
    from mixture_experts_layer_35_b200 import experts
    c, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        return experts.dispatch(s["x"], s["inv"], s["P"])
    if op == "dispatch_quantize":
        return experts.dispatch_quantize(s["x"], s["inv"], s["P"], s["fp8"])
    if op == "dispatch_backward":
        return experts.dispatch_backward(s["ys"], s["inv"], c["M"])
    if op == "combine":
        return experts.combine(s["ys"], s["inv"], s["w"])
    if op == "combine_backward":
        return experts.combine_backward(s["dy"], s["ys"], s["inv"], s["w"])
    if op == "quantize_rows":
        return experts.quantize_rows(s["x"], s["fp8"])
    if op == "quantize_columns":
        return experts.quantize_columns(s["x"], s["offsets"], s["fp8"], out=s["room"])
    if op == "quantize_blocks":
        return experts.quantize_blocks(s["w"], s["fp8"])
    if op == "product":
        return experts.product(s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["offsets"], s["out"])
    if op == "product_activation":
        return experts.product_activation(s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["offsets"], c["act"])
    if op == "product_input_grad":
        return experts.product_input_grad(s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["offsets"], s["out"])
    if op == "product_weight_grad":
        return experts.product_weight_grad(s["dy_q"], s["dy_s"], s["x_q"], s["x_s"], s["offsets"], s["out"])
    if op == "activation":
        return experts.activation(s["y"], c["act"])
    if op == "activation_quantize":
        return experts.activation_quantize(s["y"], c["act"], s["fp8"])
    return experts.activation_backward(s["y"], s["dh"], c["act"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- floors
def work(case):
    """Bytes read and written once, and operations.  Experts that get rows: at most min(E, M K);
    weights of the others are not read."""
    c, op = case, case["op"]
    M, H, K, E = c["M"], c["H"], c["K"], c["E"]
    P = M * K - int(M * K * c["drop"])
    el = 4 if c["type"] == "f32" else 2
    nb = lambda n: -(-n // BLOCK)  # noqa: E731
    hit = E * (1 - (1 - 1 / E) ** P) if E > 1 else 1  # expected, for an even choice
    idx = 4 * M * K
    if op == "dispatch":
        return {"bytes": (M + P) * H * el + idx, "flops": 0}
    if op == "dispatch_quantize":
        return {"bytes": M * H * el + P * (H + 4 * nb(H)) + idx, "flops": 3 * M * H}
    if op == "dispatch_backward":
        return {"bytes": (M + P) * H * el + idx, "flops": P * H}
    if op == "combine":
        return {"bytes": (M + P) * H * el + 2 * idx, "flops": 2 * P * H}
    if op == "combine_backward":
        return {"bytes": (M + 2 * P) * H * el + 3 * idx, "flops": 3 * P * H}
    if op == "quantize_rows":
        return {"bytes": P * (H * (el + 1) + 4 * nb(H)), "flops": 3 * P * H}
    if op == "quantize_columns":
        return {"bytes": P * H * (el + 1) + 4 * nb(P) * H, "flops": 3 * P * H}
    if op == "quantize_blocks":
        return {"bytes": E * c["N"] * H * (el + 1), "flops": 3 * E * c["N"] * H}
    if op == "product":
        N, out = c["N"], 4 if c.get("out") == "f32" else 2
        return {"bytes": hit * N * H + P * (H + 4 * nb(H) + N * out), "flops": 2 * P * N * H}
    if op == "product_input_grad":
        N, out = c["N"], 4 if c.get("out") == "f32" else 2
        return {"bytes": hit * N * H + P * (N + 4 * nb(N) + H * out), "flops": 2 * P * N * H}
    if op == "product_weight_grad":
        N, out = c["N"], 4 if c.get("out") == "f32" else 2
        return {"bytes": E * N * H * out + P * (N + H), "flops": 2 * P * N * H}
    I = c["I"]
    W = 2 * I if c["act"] == "swiglu" else I
    if op == "product_activation":
        return {"bytes": hit * W * H + P * (H + 4 * nb(H) + I + 4 * nb(I)), "flops": 2 * P * W * H}
    if op == "activation":
        return {"bytes": P * (W + I) * el, "flops": 6 * P * I}
    if op == "activation_quantize":
        return {"bytes": P * (W * el + I + 4 * nb(I)), "flops": 9 * P * I}
    return {"bytes": P * (2 * W + I) * el, "flops": 12 * P * I}


# ---------------------------------------------------------------- 64-bit values
def _exact_blocks(t, fp8, rows, cols):
    """Scales and rounded 8-bit values of a 64-bit matrix in blocks of rows x cols."""
    R, C = t.shape
    q = torch.empty_like(t)
    sc = torch.empty((-(-R // rows), -(-C // cols)), dtype=torch.float64, device=t.device)
    for j in range(sc.shape[1]):
        c0, c1 = j * cols, min(C, j * cols + cols)
        part = t[:, c0:c1]
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.nn.functional.pad(top, (0, sc.shape[0] * rows - R)).view(-1, rows).amax(1)
        top = torch.maximum(top, torch.tensor(FLOOR, dtype=torch.float64, device=t.device))
        sc[:, j] = top / FP8_MAX[fp8]
        f = (FP8_MAX[fp8] / top).repeat_interleave(rows)[:R]
        q[:, c0:c1] = part * f[:, None]
    return q.to(FP8[fp8]).double(), sc


def _exact_act(y, act):
    if act == "relu2":
        return torch.where(y > 0, y * y, torch.zeros_like(y))
    g, u = y[:, :y.shape[1] // 2], y[:, y.shape[1] // 2:]
    return g / (1 + torch.exp(-g)) * u


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    M, K, E, P = c["M"], c["K"], c["E"], s["P"]
    off = s["offsets"].tolist()
    d = lambda t: t.double()  # noqa: E731
    if op in ("dispatch", "dispatch_quantize", "dispatch_backward", "combine", "combine_backward"):
        inv = s["inv"].long().view(K, M)
        keep = [torch.nonzero(inv[k] >= 0).view(-1) for k in range(K)]
    if op in ("dispatch", "dispatch_quantize"):
        x = d(s["x"])
        q, sc = _exact_blocks(x, c["fp8"], 1, BLOCK) if op == "dispatch_quantize" else (x, x)
        oq, os = q.new_empty((P, q.shape[1])), sc.new_empty((P, sc.shape[1]))
        for k in range(K):
            oq[inv[k, keep[k]]], os[inv[k, keep[k]]] = q[keep[k]], sc[keep[k]]
        return (oq, os) if op == "dispatch_quantize" else oq
    if op in ("dispatch_backward", "combine"):
        y = torch.zeros((M, c["H"]), dtype=torch.float64, device="cuda")
        for k in range(K):
            r = d(s["ys"][inv[k, keep[k]]])
            y[keep[k]] += r * d(s["w"][keep[k], k])[:, None] if op == "combine" else r
        return y
    if op == "combine_backward":
        dys = torch.empty((P, c["H"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((M, K), dtype=torch.float64, device="cuda")
        for k in range(K):
            m, p = keep[k], inv[k, keep[k]]
            dys[p] = d(s["dy"][m]) * d(s["w"][m, k])[:, None]
            dw[m, k] = torch.einsum("mh,mh->m", d(s["dy"][m]), d(s["ys"][p]))
        return dys, dw
    if op == "quantize_rows":
        return _exact_blocks(d(s["x"]), c["fp8"], 1, BLOCK)
    if op == "quantize_columns":
        qs, scs, b = torch.zeros(s["room"][0].shape, dtype=torch.float64, device="cuda"), d(s["room"][1]), 0
        for e in range(E):
            t = d(s["x"][off[e]:off[e + 1]])
            if len(t):
                q, sc = _exact_blocks(torch.nn.functional.pad(t, (0, 0, 0, -len(t) % BLOCK)), c["fp8"], BLOCK, 1)
                qs[b * BLOCK:b * BLOCK + len(q)], scs[b:b + len(sc)] = q, sc
                b += len(sc)
        return qs, scs
    if op == "quantize_blocks":
        per = [_exact_blocks(d(s["w"][e]), c["fp8"], BLOCK, BLOCK) for e in range(E)]
        return torch.stack([p[0] for p in per]), torch.stack([p[1] for p in per])
    if op in ("product", "product_input_grad", "product_activation"):
        out = []
        for e in range(E):
            if off[e + 1] > off[e]:
                w = d(s["w_q"][e])
                for i in range(s["w_s"].shape[1]):
                    for j in range(s["w_s"].shape[2]):
                        w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= d(s["w_s"][e, i, j])
                x = d(s["x_q"][off[e]:off[e + 1]])
                for j in range(s["x_s"].shape[1]):
                    x[:, j * BLOCK:(j + 1) * BLOCK] *= d(s["x_s"][off[e]:off[e + 1], j])[:, None]
                out.append(x @ w if op == "product_input_grad" else x @ w.t())
        y = torch.cat(out)
        return _exact_blocks(_exact_act(y, c["act"]), c["fp8"], 1, BLOCK) if op == "product_activation" else y
    if op == "product_weight_grad":
        dw, b = [], 0
        for e in range(E):
            t = torch.zeros((c["N"], c["H"]), dtype=torch.float64, device="cuda")
            for _ in range(-(-(off[e + 1] - off[e]) // BLOCK)):
                r = slice(b * BLOCK, b * BLOCK + BLOCK)
                t += (d(s["dy_q"][r]) * d(s["dy_s"][b])).t() @ (d(s["x_q"][r]) * d(s["x_s"][b]))
                b += 1
            dw.append(t)
        return torch.stack(dw)
    y = d(s["y"])
    if op == "activation":
        return _exact_act(y, c["act"])
    if op == "activation_quantize":
        return _exact_blocks(_exact_act(y, c["act"]), c["fp8"], 1, BLOCK)
    dh = d(s["dh"])
    if c["act"] == "relu2":
        return torch.where(y > 0, 2 * y * dh, torch.zeros_like(y))
    I = c["I"]
    g, u = y[:, :I], y[:, I:]
    sg = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * (sg + g * sg * (1 - sg)), dh * (g * sg)], 1)
