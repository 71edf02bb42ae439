"""The expert layer's further operators as a program calls them, beside the same mathematics in plain torch.

  product   iq4_g4_qmv            Y = X W^T for few rows of X, W in 4 bits with group scales
  experts   iq4_g4_grouped_qmv    the same product with one matrix per expert, rows sorted by expert
  dispatch  iq4_moe_dispatch      tokens' rows into the experts' order; its gradient (iq4_moe_combine without weights)
  combine   iq4_moe_combine       the experts' rows back to their tokens, weighted and summed; its gradient (iq4_moe_combine_grad)
  swiglu    iq4_swiglu            h = silu(g) u between the two expert products, quantised in the same pass; its gradient
                                  (iq4_swiglu_grad)

The weights.  `group` consecutive weights of a row (32, 64 or 128) share a scale s and a whole zero point z (8 without
zero points): w = s (q - z), q one of 0 .. 15.

The pairs.  Token t's slot j is pair p = t top + j.  slot_row[p] is the pair's row in the experts' order, or -1 where an
expert had no room for it (a dropped pair adds nothing); pairs[] is the inverse, offsets[] each expert's first row.

The gradients.  combine: O[t] = sum_j w[p] R[slot_row[p]] + A[t], so dR = w[p] dO[t] and dw[p] = <dO[t], R>.  swiglu, with
s = 1 / (1 + e^-g): du = dh g s, dg = dh u s (1 + g (1 - s)).

Where `own` is false, `run` is elementary torch in 32 bits.  What is held in 8 or 4 bits is returned as the values it
stands for, in bfloat16.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token against a square projection of a decode step: the weights are read once
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 4096, "group": 128, "zeros": True, "type": "f16", "scale": "f16"},
        # a verify window of four float rows, small groups, no zero points
        {"name": "product_window", "op": "product", "m": 4, "n": 2560, "k": 6144, "group": 32, "zeros": False, "type": "f32", "scale": "f16"},
        # the wide projection for a batch of requests that each decode one token; an odd number of rows
        {"name": "product_batch", "op": "product", "m": 47, "n": 14336, "k": 4096, "group": 64, "zeros": True, "type": "bf16", "scale": "bf16"},
        # a decode step's gate and up products, side by side: four tokens, eight of 128 experts each
        {"name": "experts_window", "op": "experts", "tokens": 4, "top": 8, "experts": 128, "n": 1536, "k": 2048, "group": 32, "zeros": True,
         "type": "f32", "scale": "f16", "gather": True},
        # a batch's down products: most experts get rows, some many; rows already in the experts' order
        {"name": "experts_batch", "op": "experts", "tokens": 61, "top": 8, "experts": 128, "n": 2048, "k": 768, "group": 128, "zeros": False,
         "type": "bf16", "scale": "bf16", "gather": False},
        # a prompt's rows into the experts' order
        {"name": "dispatch_prompt", "op": "dispatch", "tokens": 3256, "top": 8, "experts": 128, "hidden": 2048, "type": "bf16", "kept": 1.0, "grad": False},
        # the gradient of that in a training step, odd sizes, full experts
        {"name": "dispatch_grad", "op": "dispatch", "tokens": 1023, "top": 6, "experts": 96, "hidden": 2592, "type": "f32", "kept": 0.9, "grad": True},
        # a verify window's float rows back to its four tokens, the shared expert's row added
        {"name": "combine_window", "op": "combine", "tokens": 4, "top": 8, "experts": 128, "hidden": 2048, "type": "f32", "kept": 1.0, "add": True, "grad": False},
        # a prompt's rows back to its tokens
        {"name": "combine_prompt", "op": "combine", "tokens": 3256, "top": 8, "experts": 128, "hidden": 2048, "type": "f16", "kept": 1.0, "add": False,
         "grad": False},
        # the gradient of that: the experts' rows and the router's weights
        {"name": "combine_grad", "op": "combine", "tokens": 3256, "top": 8, "experts": 128, "hidden": 2048, "type": "bf16", "kept": 1.0, "add": False,
         "grad": True},
        # a prompt's gate|up rows into the 8-bit rows of the down product
        {"name": "swiglu_prompt", "op": "swiglu", "m": 26048, "k": 768, "type": "f16", "fmt": "mxfp8", "grad": False},
        # a training step's wide hidden layer
        {"name": "swiglu_grad", "op": "swiglu", "m": 3256, "k": 14336, "type": "bf16", "fmt": "", "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "experts", "dispatch", "combine", "swiglu"])
    if op in ("product", "experts"):
        group = rng.choice([32, 64, 128])
        case = {"op": op, "group": group, "zeros": rng.random() < 0.5, "type": rng.choice(list(TYPES)), "scale": rng.choice(["f16", "bf16"])}
        if op == "product":
            n, k = _log(rng, 64, 14336), group * _log(rng, 128 // group, 14336 // group)
            return case | {"m": _log(rng, 1, 64), "n": min(n, 14336 * 4096 // k), "k": k}
        experts = _log(rng, 4, 128)
        return case | {"tokens": _log(rng, 1, 64), "top": rng.randint(1, min(8, experts)), "experts": experts, "n": _log(rng, 64, 2048),
                       "k": group * _log(rng, 128 // group, 2048 // group), "gather": rng.random() < 0.5}
    t, grad = rng.choice(list(TYPES)), rng.random() < 0.5
    if op == "swiglu":
        k = 32 * _log(rng, 4, 448)
        m = min(_log(rng, 1, 26048), 3256 * 14336 // k)
        return {"op": op, "m": m, "k": k, "type": t, "fmt": "" if grad else rng.choice(["", "mxfp8", "mxfp4", "q8_1"]), "grad": grad}
    experts = _log(rng, 4, 128)
    top, hidden = rng.randint(1, min(8, experts)), _log(rng, 64, 8192)
    tokens = min(_log(rng, 1, 13056), max(1, 3256 * 8 * 2048 // (top * hidden)))
    case = {"op": op, "tokens": tokens, "top": top, "experts": experts, "hidden": hidden, "type": t,
            "kept": 0.9 if tokens >= 16 and rng.random() < 0.5 else 1.0, "grad": grad}
    return case | {"add": rng.random() < 0.5 and not grad} if op == "combine" else case


# ---- the plain forms ---------------------------------------------------------------------------


def _decoded(codes, scales, zeros, group):
    """Float32 weights of codes [..., k / 2] (the first of a byte in its low half) and scales, zeros [..., k / group]."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, group))
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).flatten(-2)


def _experts(s):
    x = s["x"].float()
    if s["gather"]:
        x = x[(s["pairs"] // s["top"]).long()]
    e = s["expert_of"]
    if x.shape[0] <= s["experts"]:  # few rows: each with its expert's matrix
        w = _decoded(s["codes"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e], s["group"])
        return torch.bmm(w, x.unsqueeze(-1)).squeeze(-1).to(s["t"])
    rows = torch.zeros(s["experts"], s["most"], x.shape[1], device=x.device)  # the experts' rows, padded to the longest
    rows[e, s["place"]] = x
    w = _decoded(s["codes"], s["scales"], s["zeros"], s["group"])
    return torch.bmm(rows, w.transpose(1, 2).contiguous())[e, s["place"]].to(s["t"])


def _token_rows(s, rows):
    """[tokens, top, hidden] float32: each pair's row, zero where it has none."""
    slot = s["slot_row"].long().reshape(-1, s["top"])
    return torch.where((slot >= 0).unsqueeze(-1), rows.float()[slot.clamp(min=0)], 0.0)


def _dispatch(s):
    if s["grad"]:
        return {"dx": _token_rows(s, s["rows"]).sum(1).to(s["t"])}
    return {"rows": s["x"][(s["pairs"] // s["top"]).long()]}


def _combine(s):
    w = s["w"]
    if not s["grad"]:
        out = (_token_rows(s, s["rows"]) * w.unsqueeze(-1)).sum(1)
        return {"out": (out if s["add"] is None else out + s["add"].float()).to(s["t"])}
    p, do = s["pairs"].long(), s["do"].float()
    return {"drows": (w.reshape(-1)[p].unsqueeze(-1) * do[p // s["top"]]).to(s["t"]),
            "dw": (do.unsqueeze(1) * _token_rows(s, s["rows"])).sum(-1)}


def _power(e):
    """2^(e - 127) in float32 for a biased exponent 0 .. 254, the subnormal 2^-127 included."""
    return torch.where(e > 0, (e << 23), torch.full_like(e, 1 << 22)).view(torch.float32)


def _exponent(x):
    return (x.view(torch.int32) >> 23) & 255


def _held(y, fmt):
    """The values that float32 rows have after they were held in `fmt`, blocks of 32."""
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "q8_1":
        d = top / 127
        kept = d.half()
        t = b * torch.where(kept == 0, torch.zeros_like(d), 1 / d)
        w = torch.trunc(t)
        q = torch.where((t - w).abs() >= 0.5, w + torch.sign(t), w).clamp(-127, 127)
        return (q * kept.float()).reshape(y.shape)
    s = (_exponent(top) - (2 if fmt == "mxfp4" else 8)).clamp(min=0)
    v = b * _power(254 - s)
    a = v.abs()
    if fmt == "mxfp4":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    else:
        step = _power((_exponent(a) - 3).clamp(min=127 - 9))
    q = (torch.round(a / step) * step).clamp(max=6.0 if fmt == "mxfp4" else 448.0)
    return (torch.copysign(q, v) * _power(s)).reshape(y.shape)


def _swiglu(s):
    k = s["k"]
    g, u = s["gu"][:, :k].float(), s["gu"][:, k:].float()
    if s["grad"]:
        dh, e = s["dh"].float(), 1 / (1 + torch.exp(-g))
        return {"dgu": torch.cat((dh * u * (e * (1 + g * (1 - e))), dh * (g * e)), 1).to(s["t"])}
    h = g / (1 + torch.exp(-g)) * u
    return {"held": _held(h, s["fmt"]).bfloat16()} if s["fmt"] else {"h": h.to(s["t"])}


# ---- inputs ------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _acts(g, m, k):
    """Activations: normal, every row with its own size, one channel in 64 some ten times larger."""
    x = _randn(g, m, k) * torch.exp(0.5 * _randn(g, m, 1))
    return torch.where(torch.rand(k, device=DEV, generator=g) < 1 / 64, 10 * x, x)


def _weights(g, case, rows):
    """4-bit weights as a checkpoint has them: codes around the zero points, scales of weights N(0, 0.02)."""
    k, group = case["k"], case["group"]
    z = torch.randint(6, 11, (rows, k // group), device=DEV, generator=g, dtype=torch.uint8) if case["zeros"] else None
    codes = []
    for at in range(0, rows, 1 << 15):  # in parts: the float rows need not fit at once
        n = min(1 << 15, rows - at)
        zero = 8 if z is None else z[at:at + n].unsqueeze(-1).float()
        q = (2.6 * _randn(g, n, k // group, group) + zero).round().clamp(0, 15).to(torch.uint8).reshape(n, k // 2, 2)
        codes.append(q[..., 0] | (q[..., 1] << 4))
    scales = (0.0077 * torch.exp(0.2 * _randn(g, rows, k // group))).to(TYPES[case["scale"]])
    return torch.cat(codes), scales, z


def _routed(g, case, s):
    """Pairs by expert, as iq4_moe_gather orders them: Zipf loads, the pairs past an expert's room dropped."""
    tokens, top, experts = case["tokens"], case["top"], case["experts"]
    gumbel = -torch.log(-torch.log(torch.rand(tokens, experts, device=DEV, generator=g, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
    ids = (_share(experts).log().to(DEV) + gumbel).topk(top, -1).indices.reshape(-1)
    ids[torch.rand(tokens * top, device=DEV, generator=g) >= case.get("kept", 1.0)] = experts
    expert_of, pairs = torch.sort(ids, stable=True)
    counts = torch.bincount(ids, minlength=experts + 1)[:experts]
    n = int(counts.sum())
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    slot = torch.full((tokens * top,), -1, dtype=torch.int32, device=DEV)
    slot[pairs[:n]] = torch.arange(n, dtype=torch.int32, device=DEV)
    s |= {"n_rows": n, "offsets": offsets, "pairs": pairs[:n].int(), "slot_row": slot, "expert_of": expert_of[:n], "most": int(counts.max()),
          "place": torch.arange(n, device=DEV) - offsets[expert_of[:n]].long()}


def _share(experts):
    """Zipf weights of the experts."""
    p = torch.arange(1, experts + 1, dtype=torch.float64) ** -1.1
    return p / p.sum()


def prepare(case, seed):
    g = _gen(seed)
    t = TYPES[case["type"]]
    s = dict(case) | {"t": t}
    op = case["op"]
    if op == "swiglu":
        s["gu"] = (1.5 * _randn(g, case["m"], 2 * case["k"])).to(t)
        if case["grad"]:
            s["dh"] = _acts(g, case["m"], case["k"]).to(t)
    elif op == "product":
        s["codes"], s["scales"], s["zeros"] = _weights(g, case, case["n"])
        s["x"] = _acts(g, case["m"], case["k"]).to(t)
    else:
        _routed(g, case, s)
        if op == "experts":
            e, n = case["experts"], case["n"]
            s["codes"], s["scales"], s["zeros"] = (None if v is None else v.reshape(e, n, -1) for v in _weights(g, case, e * n))
            s["x"] = _acts(g, case["tokens"] if case["gather"] else s["n_rows"], case["k"]).to(t)
        elif op == "dispatch" and not case["grad"]:
            s["x"] = _acts(g, case["tokens"], case["hidden"]).to(t)
        else:
            s["rows"] = _acts(g, s["n_rows"], case["hidden"]).to(t)
        if op == "combine":
            s["w"] = torch.softmax(_randn(g, case["tokens"], case["top"]), -1)
            s["add"] = _acts(g, case["tokens"], case["hidden"]).to(t) if case["add"] else None
            if case["grad"]:
                s["do"] = _acts(g, case["tokens"], case["hidden"]).to(t)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program of the framework keeps: packed weights, its output buffers."""
    import dequant_matmul_iq4_amd as iq4

    types = {torch.float32: iq4.IQ4_F32, torch.float16: iq4.IQ4_F16, torch.bfloat16: iq4.IQ4_BF16}
    op, t = s["op"], s["t"]
    new = lambda *shape, dtype=t: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    s |= {"iq4": iq4, "type": types[t]}
    if op == "swiglu":
        m, k = s["m"], s["k"]
        s["f"] = {"": 0, "q8_1": iq4.IQ4_ROWS_Q8_1, "mxfp8": iq4.IQ4_ROWS_MXFP8, "mxfp4": iq4.IQ4_ROWS_MXFP4}[s["fmt"]]
        if s["grad"]:
            s["dgu"] = new(m, 2 * k)
        elif s["fmt"]:
            s["ldq"], s["lds"] = iq4.iq4_rows_bytes(s["f"], k)
            s |= {"q": new(m, s["ldq"], dtype=torch.uint8), "d": new(m, s["lds"], dtype=torch.uint8), "held": new(m, k, dtype=torch.bfloat16)}
        else:
            s["h"] = new(m, k)
    elif op in ("product", "experts"):
        n, k, e = s["n"], s["k"], s.get("experts", 1)
        each = iq4.iq4_g4_packed_bytes(n, k, s["group"], s["zeros"] is not None)
        s["packed"] = torch.empty(e * each, dtype=torch.uint8, device=DEV)
        codes, scales, zeros = (None if s[v] is None else s[v].reshape(e, n, -1) for v in ("codes", "scales", "zeros"))
        for i in range(e):
            iq4.iq4_g4_pack_weights(codes[i], k // 2, scales[i], k // s["group"], None if zeros is None else zeros[i], k // s["group"], n, k,
                                    s["group"], s["packed"][i * each:])
        s |= {"scale_type": types[s["scales"].dtype], "y": new(s["m"] if op == "product" else s["n_rows"], n)}
    elif op == "dispatch":
        s["out"] = new(s["tokens"] if s["grad"] else s["n_rows"], s["hidden"])
    elif s["grad"]:
        s |= {"drows": new(s["n_rows"], s["hidden"]), "dw": new(s["tokens"], s["top"], dtype=torch.float32)}
    else:
        s["out"] = new(s["tokens"], s["hidden"])


def _run_own(s):
    iq4, op, t = s["iq4"], s["op"], s["type"]
    if op == "product":
        iq4.iq4_g4_qmv(s["packed"], s["n"], s["k"], s["group"], s["scale_type"], s["zeros"] is not None, s["x"], t, s["k"], s["m"], s["y"], t, s["n"])
        return {"y": s["y"]}
    if op == "experts":
        iq4.iq4_g4_grouped_qmv(s["packed"], s["experts"], s["n"], s["k"], s["group"], s["scale_type"], s["zeros"] is not None, s["x"], t, s["k"],
                               s["x"].shape[0], s["offsets"], s["pairs"] if s["gather"] else None, s["top"], s["n_rows"], s["y"], t, s["n"])
        return {"y": s["y"]}
    if op == "swiglu":
        m, k, gu = s["m"], s["k"], s["gu"]
        if s["grad"]:
            iq4.iq4_swiglu_grad(s["dh"], t, k, gu, 2 * k, gu[:, k:], 2 * k, t, m, k, s["dgu"], 2 * k, s["dgu"][:, k:], 2 * k)
            return {"dgu": s["dgu"]}
        if not s["fmt"]:
            iq4.iq4_swiglu(gu, 2 * k, gu[:, k:], 2 * k, t, m, k, s["h"], t, k)
            return {"h": s["h"]}
        iq4.iq4_swiglu(gu, 2 * k, gu[:, k:], 2 * k, t, m, k, None, t, 0, s["f"], s["q"], s["ldq"], s["d"], s["lds"])
        iq4.iq4_dequant_rows(s["q"], s["ldq"], s["d"], s["lds"], s["f"], m, k, iq4.IQ4_BF16, s["held"], k)
        return {"held": s["held"]}
    h, rows = s["hidden"], s["n_rows"]
    if op == "dispatch" and not s["grad"]:
        iq4.iq4_moe_dispatch(s["x"], t, h, s["tokens"], h, s["slot_row"], None, s["top"], rows, s["out"], t, h)
        return {"rows": s["out"]}
    if op == "dispatch":
        iq4.iq4_moe_combine(s["rows"], t, h, rows, s["slot_row"], None, s["tokens"], s["top"], h, None, 0, s["out"], t, h)
        return {"dx": s["out"]}
    if s["grad"]:
        iq4.iq4_moe_combine_grad(s["do"], t, h, s["rows"], t, h, rows, s["slot_row"], s["w"], s["tokens"], s["top"], h, s["drows"], h, s["dw"])
        return {"drows": s["drows"], "dw": s["dw"]}
    iq4.iq4_moe_combine(s["rows"], t, h, rows, s["slot_row"], s["w"], s["tokens"], s["top"], h, s["add"], h, s["out"], t, h)
    return {"out": s["out"]}


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "product":
        w = _decoded(s["codes"], s["scales"], s["zeros"], s["group"])
        return {"y": torch.matmul(s["x"].float(), w.t()).to(s["t"])}
    if s["op"] == "experts":
        return {"y": _experts(s)}
    return {"dispatch": _dispatch, "combine": _combine, "swiglu": _swiglu}[s["op"]](s)


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _exact_weights(codes, scales, zeros, group):
    """Float64 weights of one matrix, each number by itself: w = s (q - z)."""
    n, half = codes.shape
    c = codes.long()
    w = torch.empty(n, 2 * half, dtype=torch.float64, device=codes.device)
    w[:, 0::2], w[:, 1::2] = c.remainder(16).double(), c.div(16, rounding_mode="floor").double()
    z = torch.full_like(scales, 8.0) if zeros is None else zeros
    w -= z.double().repeat_interleave(group, 1)
    return w.mul_(scales.double().repeat_interleave(group, 1))


def _two(e):
    """2^e in float64 for whole e, -1022 .. 1023 (a power function need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_held(y, fmt):
    """Float64 rows (each value one of binary32) -> the values after `fmt`, by the formats' grids."""
    b = y.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "q8_1":
        d = (top / 127).float().double()
        kept = d.half().double()
        r = torch.where(kept > 0, (1 / d.clamp(min=1e-300)).float().double(), 0.0)
        t = (b * r).float().double()
        return (t.sign() * (t.abs() + 0.5).floor().clamp(max=127) * kept).flatten(-2)
    most, low, bits, above = (6.0, 0, 1, 2) if fmt == "mxfp4" else (448.0, -6, 3, 8)
    e = torch.frexp(top)[1] - 1 - above
    scale = _two(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
    v = b / scale
    grid = _two((torch.frexp(v)[1] - 1).clamp(min=low) - bits)
    return (torch.round(v / grid) * grid).clamp(-most, most).mul(scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "product":
        return {"y": s["x"].double() @ _exact_weights(s["codes"], s["scales"], s["zeros"], s["group"]).t()}
    if op == "experts":
        x, at, y = s["x"].double(), s["offsets"].tolist(), []
        if s["gather"]:
            x = x[torch.div(s["pairs"], s["top"], rounding_mode="floor").long()]
        for e in range(s["experts"]):
            if at[e + 1] > at[e]:
                z = None if s["zeros"] is None else s["zeros"][e]
                y.append(x[at[e]:at[e + 1]] @ _exact_weights(s["codes"][e], s["scales"][e], z, s["group"]).t())
        return {"y": torch.cat(y)}
    if op == "swiglu":
        out = []
        for rows in torch.arange(s["m"], device=DEV).split(4096):  # in parts: 64 bits of the whole need not fit
            g, u = s["gu"][rows].double().chunk(2, 1)
            if not s["grad"]:
                h = g * torch.sigmoid(g) * u
                out.append(_exact_held(h.float().double(), s["fmt"]) if s["fmt"] else h)
                continue
            dh, e = s["dh"][rows].double(), torch.sigmoid(g)
            out.append(torch.cat((dh * u * (e + g * e * torch.sigmoid(-g)), dh * g * e), 1))
        return {"dgu" if s["grad"] else "held" if s["fmt"] else "h": torch.cat(out)}
    tokens, top, hidden = s["tokens"], s["top"], s["hidden"]
    pairs, token = s["pairs"].long(), torch.div(s["pairs"].long(), top, rounding_mode="floor")
    if op == "dispatch" and not s["grad"]:
        return {"rows": s["x"].double().index_select(0, token)}
    rows = s["rows"].double()
    if op == "dispatch":
        return {"dx": torch.zeros(tokens, hidden, dtype=torch.float64, device=DEV).index_add_(0, token, rows)}
    w = s["w"].double().flatten()[pairs].unsqueeze(1)
    if s["grad"]:
        do = s["do"].double().index_select(0, token)
        dw = torch.zeros(tokens * top, dtype=torch.float64, device=DEV)
        dw[pairs] = (do * rows).sum(1)
        return {"drows": w * do, "dw": dw.reshape(tokens, top)}
    out = torch.zeros(tokens, hidden, dtype=torch.float64, device=DEV) if s["add"] is None else s["add"].double()
    return {"out": out.index_add(0, token, w * rows)}


def work(case):
    op, size = case["op"], SIZE[case["type"]]
    if op == "swiglu":
        each = case["m"] * case["k"]
        if case["grad"]:
            return {"bytes": 5 * size * each, "flops": 12 * each}
        # g and u, and h; or what holds h, and the values that stands for
        held = {"": size, "q8_1": 1 + 1 / 16 + 2, "mxfp8": 1 + 1 / 32 + 2, "mxfp4": 1 / 2 + 1 / 32 + 2}[case["fmt"]]
        return {"bytes": int(each * (2 * size + held)), "flops": 6 * each}
    if op in ("product", "experts"):
        n, k = case["n"], case["k"]
        matrix = n * (k // 2) + n * (k // case["group"]) * (2.5 if case["zeros"] else 2)
        if op == "product":
            m, rows, matrices = case["m"], case["m"], 1
        else:
            m = case["tokens"] * case["top"]
            rows = case["tokens"] if case["gather"] else m
            matrices = min(case["experts"], float((1 - (1 - _share(case["experts"])) ** m).sum()))  # experts that get a row
        return {"bytes": int(matrices * matrix + rows * k * size + m * n * size), "flops": 2 * m * n * k}
    token = case["tokens"] * case["hidden"] * size
    pairs = case["tokens"] * case["top"]
    rows = int(pairs * case["kept"]) * case["hidden"] * size
    if op == "dispatch":
        return {"bytes": token + rows + 4 * pairs, "flops": rows // size if case["grad"] else 0}
    if case["grad"]:
        return {"bytes": token + 2 * rows + 12 * pairs, "flops": 3 * rows // size}
    return {"bytes": token * (2 if case["add"] else 1) + rows + 8 * pairs, "flops": 2 * rows // size}
