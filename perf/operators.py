"""The row-format operators as a program calls them, beside the same mathematics in plain torch.

Four operators around rows of activations that are held in 4 or 8 bits with a scale per 32
elements, and weights held in 4 bits the same way:

  norm      iq4_rmsnorm         residual + RMS norm, the row quantised in the same pass
  rows      iq4_quantize_rows   rows of floats -> codes and scales, and back (iq4_dequant_rows)
  product   iq4_mx_gemm         Y = X W^T, W in MXFP4, X in MXFP4 or MXFP8 rows
  grouped   iq4_mx_grouped_gemm the same product with one matrix per expert, rows sorted by expert

The formats.  MXFP4 and MXFP8 (OCP microscaling): 32 elements share a power of two
2^(s - 127), s = max(E - 2, 0) for E2M1 and max(E - 8, 0) for E4M3, E the biased binary32
exponent of the block's largest magnitude; an element is x / 2^(s - 127) rounded to nearest
even, clamped to the format's largest value (6, 448).  Q8_1: d = f32(max|x|) / 127, an element
is round(f32(x * f32(1 / d))), halves away from zero, clamped to [-127, 127], d kept in binary16.

The norm.  h = x + residual, rounded to the rows' type; u = f32(1 / sqrt(mean(h^2) + eps)) with
the mean in 64 bits; y = f32(f32(h * u) * gain).  What is quantised is y.

Where `own` is false, `run` is elementary torch in 32 bits (the mean square in 64).  What is held
in 4 or 8 bits is returned as the values it stands for.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's row before the attention projections of a decode step; 8-bit blocks feed the
        # matvec on 8-bit activations, the sum is the residual stream
        {"name": "norm_token_q8", "op": "norm", "m": 1, "k": 4096, "type": "f32", "fmt": "q8_1", "plain": False},
        # a verify window of four tokens, odd number of blocks; the plain row goes to the router
        {"name": "norm_window_mx8", "op": "norm", "m": 4, "k": 2592, "type": "bf16", "fmt": "mxfp8", "plain": True},
        # a long prompt's rows before the 4-bit projection
        {"name": "norm_prompt_mx4", "op": "norm", "m": 13056, "k": 4096, "type": "bf16", "fmt": "mxfp4", "plain": False},
        # four tokens' rows quantised on their own, as before an output projection
        {"name": "rows_window_mx4", "op": "rows", "m": 4, "k": 4096, "type": "f32", "fmt": "mxfp4"},
        # a prompt's hidden rows before the down projection
        {"name": "rows_prompt_mx8", "op": "rows", "m": 3256, "k": 14336, "type": "f16", "fmt": "mxfp8"},
        # one token against a square projection: the weights are read once
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 4096, "fmt": "mxfp4", "out": "f32"},
        # a verify window with 8-bit activations
        {"name": "product_window", "op": "product", "m": 4, "n": 2560, "k": 6144, "fmt": "mxfp8", "out": "f32"},
        # a short ragged prompt against a matrix of odd sizes
        {"name": "product_ragged", "op": "product", "m": 333, "n": 5000, "k": 2592, "fmt": "mxfp8", "out": "bf16"},
        # the long prompt's projection
        {"name": "product_prompt", "op": "product", "m": 13056, "n": 14336, "k": 4096, "fmt": "mxfp4", "out": "bf16"},
        # a decode step's gate and up products, side by side: four tokens, eight of 128 experts each
        {"name": "grouped_window", "op": "grouped", "tokens": 4, "top": 8, "experts": 128, "n": 1536, "k": 2048, "fmt": "mxfp8", "out": "f32",
         "gather": True},
        # a prompt's gate and up products: rows gathered by expert, loads skewed, some experts empty
        {"name": "grouped_prompt_up", "op": "grouped", "tokens": 3256, "top": 8, "experts": 128, "n": 1536, "k": 2048, "fmt": "mxfp4", "out": "f16",
         "gather": True},
        # its down products: rows already in the experts' order
        {"name": "grouped_prompt_down", "op": "grouped", "tokens": 3256, "top": 8, "experts": 128, "n": 2048, "k": 768, "fmt": "mxfp8", "out": "f16",
         "gather": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rows", "product", "grouped"])
    if op in ("norm", "rows"):
        k = 32 * _log(rng, 4, 448)
        m = min(_log(rng, 1, 13056), 13056 * 4096 // k)
        case = {"op": op, "m": m, "k": k, "type": rng.choice(list(TYPES))}
        if op == "norm":
            return case | {"fmt": rng.choice(["q8_1", "mxfp8", "mxfp4"]), "plain": rng.random() < 0.5}
        return case | {"fmt": rng.choice(["mxfp8", "mxfp4"])}
    if op == "product":
        n, k = _log(rng, 64, 14336), 32 * _log(rng, 4, 448)
        m = max(1, min(_log(rng, 1, 13056), 13056 * 14336 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "fmt": rng.choice(["mxfp8", "mxfp4"]), "out": rng.choice(list(TYPES))}
    experts = _log(rng, 4, 128)
    return {"op": op, "tokens": _log(rng, 1, 3256), "top": rng.randint(1, min(8, experts)), "experts": experts, "n": _log(rng, 64, 2048),
            "k": 32 * _log(rng, 4, 64), "fmt": rng.choice(["mxfp8", "mxfp4"]), "out": rng.choice(list(TYPES)), "gather": rng.random() < 0.5}


# ---- the plain forms ---------------------------------------------------------------------------


def _exponent(amax):
    """Biased binary32 exponent of float32 values (0 for zero and subnormals)."""
    return (amax.view(torch.int32) >> 23) & 255


def _power(e):
    """2^(e - 127) in float32 for a biased exponent 0 .. 254, the subnormal 2^-127 included."""
    return torch.where(e > 0, (e << 23), torch.full_like(e, 1 << 22)).view(torch.float32)


def _to_mx(x, fmt):
    """Float32 rows -> (codes as element values, biased scale exponents), block by block."""
    b = x.reshape(x.shape[0], -1, 32)
    s = (_exponent(b.abs().amax(-1, keepdim=True)) - (2 if fmt == "mxfp4" else 8)).clamp(min=0)
    v = b * _power(254 - s)
    a = v.abs()
    if fmt == "mxfp4":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = (torch.round(a / step) * step).clamp(max=6.0)
    else:
        step = _power((_exponent(a) - 3).clamp(min=127 - 9))
        q = (torch.round(a / step) * step).clamp(max=448.0)
    return torch.copysign(q, v), s


def _bits_of(q, fmt):
    """Element values -> stored bytes: two 4-bit codes a byte (the first one low), or one code."""
    a = q.abs()
    sign = torch.signbit(q).to(torch.uint8)
    if fmt == "mxfp4":
        c = torch.where(a <= 2, a * 2, torch.where(a <= 4, a + 2, torch.full_like(a, 7.0))).to(torch.uint8) | (sign << 3)
        c = c.reshape(c.shape[0], -1)
        return c[:, 0::2] | (c[:, 1::2] << 4)
    e = (_exponent(a) - 120).clamp(min=1)
    c = torch.round((a / _power(e + 120) - 1) * 8).to(torch.int32) + (e << 3)
    return ((c.to(torch.uint8)) | (sign << 7)).reshape(c.shape[0], -1)


def _values(codes, fmt):
    """Stored bytes -> element values, float32, 32 to a block."""
    if fmt == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        pairs = torch.stack((codes & 15, codes >> 4), -1)
        return table[pairs.int()].reshape(*codes.shape[:-1], -1, 32)
    c = torch.arange(256, device=codes.device, dtype=torch.int32)
    e, f = (c >> 3) & 15, (c & 7).float()
    table = torch.where(e > 0, (8 + f) * _power(e + 117), f * 2.0**-9) * torch.where(c > 127, -1.0, 1.0)
    return table[codes.int()].reshape(*codes.shape[:-1], -1, 32)


def _decoded(codes, scales, fmt):
    """Float32 rows that codes [..., k] and biased scale exponents [..., k / 32] stand for."""
    v = _values(codes, fmt) * _power(scales.int()).unsqueeze(-1)
    return v.reshape(*v.shape[:-2], -1)


def _held(y, fmt):
    """The values that float32 rows have after they were held in `fmt`."""
    if fmt != "q8_1":
        q, s = _to_mx(y, fmt)
        return (q * _power(s)).reshape(y.shape)
    b = y.reshape(y.shape[0], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127
    d16 = d.half()
    r = torch.where(d16 == 0, torch.zeros_like(d), 1 / d)
    t = b * r
    w = torch.trunc(t)
    q = torch.where((t - w).abs() >= 0.5, w + torch.sign(t), w).clamp(-127, 127)
    return (q * d16.float()).reshape(y.shape)


def _norm(s):
    h = (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    f = h.float()
    u = (1 / torch.sqrt(f.double().square().mean(-1, keepdim=True) + s["eps"])).float()
    y = (f * u) * s["gain"]
    out = {"h": h, "held": _held(y, s["fmt"])}
    if s["plain"]:
        out["y"] = y.to(s["x"].dtype)
    return out


def _grouped(s):
    rows = _decoded(s["codes"], s["scales"], s["fmt"])
    if s["pairs"] is not None:
        rows = rows[(s["pairs"] // s["top"]).long()]
    if rows.shape[0] <= s["experts"]:  # few rows: each with its expert's matrix
        w = _decoded(s["w_codes"][s["expert_of"]], s["w_scales"][s["expert_of"]], "mxfp4")
        y = torch.bmm(w, rows.unsqueeze(-1)).squeeze(-1)
    else:  # the experts' rows side by side, padded to the longest
        x = torch.zeros(s["experts"], s["most"], rows.shape[1], device=rows.device)
        x[s["expert_of"], s["place"]] = rows
        w = _decoded(s["w_codes"], s["w_scales"], "mxfp4")
        y = torch.bmm(x, w.transpose(1, 2).contiguous())[s["expert_of"], s["place"]]
    return y.to(s["out"])


# ---- inputs ------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _acts(g, m, k):
    """Activations: normal, every row with its own size, one channel in 64 some ten times larger."""
    x = torch.randn(m, k, device=DEV, generator=g) * torch.exp(0.5 * torch.randn(m, 1, device=DEV, generator=g))
    big = torch.rand(k, device=DEV, generator=g) < 1 / 64
    return torch.where(big, 10 * x, x)


def _weights(g, shape, k):
    """Weights N(0, 0.02) in MXFP4, as a checkpoint has them: codes [..., k / 2], scales [..., k / 32]."""
    codes, scales = [], []
    rows = math.prod(shape)
    for at in range(0, rows, 1 << 15):  # in parts: the float rows need not fit at once
        q, s = _to_mx(0.02 * torch.randn(min(1 << 15, rows - at), k, device=DEV, generator=g), "mxfp4")
        codes.append(_bits_of(q, "mxfp4"))
        scales.append(s.reshape(s.shape[0], -1).to(torch.uint8))
    return torch.cat(codes).reshape(*shape, k // 2), torch.cat(scales).reshape(*shape, k // 32)


def _stored(x, fmt):
    q, s = _to_mx(x, fmt)
    return _bits_of(q, fmt), s.reshape(s.shape[0], -1).to(torch.uint8)


def _padded(t, width):
    """Rows of bytes, each followed by zeros up to `width`, as the library lays rows out."""
    p = torch.zeros(t.shape[0], width, dtype=torch.uint8, device=t.device)
    p[:, : t.shape[1]] = t
    return p


def _share(experts):
    """Zipf weights of the experts."""
    p = torch.arange(1, experts + 1, dtype=torch.float64) ** -1.1
    return p / p.sum()


def prepare(case, seed):
    g = _gen(seed)
    op, k, fmt = case["op"], case["k"], case["fmt"]
    s = {"op": op, "fmt": fmt, "k": k}
    if op in ("norm", "rows"):
        m, t = case["m"], TYPES[case["type"]]
        s |= {"m": m, "x": _acts(g, m, k).to(t)}
        if op == "norm":
            s |= {"res": _acts(g, m, k).to(t), "gain": 1 + 0.2 * torch.randn(k, device=DEV, generator=g), "eps": 1e-6, "plain": case["plain"]}
    else:
        s |= {"n": case["n"], "out": TYPES[case["out"]]}
        if op == "product":
            s["m"] = case["m"]
            s["w_codes"], s["w_scales"] = _weights(g, (case["n"],), k)
            s["codes"], s["scales"] = _stored(_acts(g, case["m"], k), fmt)
        else:
            tokens, top, experts = case["tokens"], case["top"], case["experts"]
            s["w_codes"], s["w_scales"] = _weights(g, (experts, case["n"]), k)
            gumbel = -torch.log(-torch.log(torch.rand(tokens, experts, device=DEV, generator=g, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
            ids = (_share(experts).log().to(DEV) + gumbel).topk(top, -1).indices.reshape(-1)
            expert_of, pairs = torch.sort(ids, stable=True)
            counts = torch.bincount(ids, minlength=experts)
            offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
            offsets[1:] = counts.cumsum(0)
            s |= {"m": ids.numel(), "experts": experts, "top": top, "offsets": offsets, "expert_of": expert_of, "most": int(counts.max()),
                  "place": torch.arange(ids.numel(), device=DEV) - offsets[expert_of].long(), "pairs": pairs.int() if case["gather"] else None}
            s["codes"], s["scales"] = _stored(_acts(g, tokens if case["gather"] else ids.numel(), k), fmt)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program of the framework keeps: packed weights, rows in the library's strides, its output buffers."""
    import dequant_matmul_iq4_amd as iq4

    fmt = {"q8_1": iq4.IQ4_ROWS_Q8_1, "mxfp8": iq4.IQ4_ROWS_MXFP8, "mxfp4": iq4.IQ4_ROWS_MXFP4}[s["fmt"]]
    types = {torch.float32: iq4.IQ4_F32, torch.float16: iq4.IQ4_F16, torch.bfloat16: iq4.IQ4_BF16}
    k, m = s["k"], s["m"]
    ldq, lds = iq4.iq4_rows_bytes(fmt, k)
    s |= {"iq4": iq4, "f": fmt, "ldq": ldq, "lds": lds}
    if s["op"] in ("norm", "rows"):
        s |= {"type": types[s["x"].dtype], "q": torch.empty(m, ldq, dtype=torch.uint8, device=DEV),
              "d": torch.empty(m, lds, dtype=torch.uint8, device=DEV), "held": torch.empty(m, k, device=DEV)}
        if s["op"] == "norm":
            s |= {"h": torch.empty_like(s["x"]), "y": torch.empty_like(s["x"]) if s["plain"] else None}
        return
    e, n = s.get("experts", 1), s["n"]
    each = iq4.iq4_mx_packed_bytes(n, k)
    packed = torch.empty(e * each, dtype=torch.uint8, device=DEV)
    for i in range(e):
        c, d = (s["w_codes"][i], s["w_scales"][i]) if "experts" in s else (s["w_codes"], s["w_scales"])
        iq4.iq4_mx_pack_weights(c, k // 2, d, k // 32, n, k, packed[i * each:])
    s |= {"packed": packed, "q": _padded(s["codes"], ldq), "d": _padded(s["scales"], lds), "y_type": types[s["out"]],
          "y": torch.empty(m, n, dtype=s["out"], device=DEV)}


def run(s):
    if own:
        iq4 = s["iq4"]
        if s["op"] == "norm":
            iq4.iq4_rmsnorm(s["x"], s["k"], s["res"], s["k"], s["type"], s["m"], s["k"], s["gain"], s["eps"], s["h"], s["k"], s["y"], s["type"],
                            s["k"], s["f"], s["q"], s["ldq"], s["d"], s["lds"])
        if s["op"] == "rows":
            iq4.iq4_quantize_rows(s["x"], s["type"], s["m"], s["k"], s["k"], s["f"], s["q"], s["ldq"], s["d"], s["lds"])
        if s["op"] in ("norm", "rows"):
            iq4.iq4_dequant_rows(s["q"], s["ldq"], s["d"], s["lds"], s["f"], s["m"], s["k"], iq4.IQ4_F32, s["held"], s["k"])
            return {name: s[name] for name in ("h", "held", "y") if s.get(name) is not None}
        if s["op"] == "product":
            iq4.iq4_mx_gemm(s["packed"], s["n"], s["k"], s["f"], s["q"], s["ldq"], s["d"], s["lds"], s["m"], s["y"], s["y_type"], s["n"])
        else:
            iq4.iq4_mx_grouped_gemm(s["packed"], s["experts"], s["n"], s["k"], s["f"], s["q"], s["ldq"], s["d"], s["lds"], s["q"].shape[0],
                                    s["offsets"], s["pairs"], s["top"], s["m"], s["y"], s["y_type"], s["n"])
        return {"y": s["y"]}
    if s["op"] == "norm":
        return _norm(s)
    if s["op"] == "rows":
        return {"held": _held(s["x"].float(), s["fmt"])}
    if s["op"] == "product":
        w = _decoded(s["w_codes"], s["w_scales"], "mxfp4")
        return {"y": torch.matmul(_decoded(s["codes"], s["scales"], s["fmt"]), w.t()).to(s["out"])}
    return {"y": _grouped(s)}


# ---- the definitions in 64 bits ------------------------------------------------------------------


def _two(e):
    """2^e in float64 for whole e, -1022 .. 1023 (a power function need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_bytes(codes, scales, fmt):
    """Float64 rows of stored bytes, from the formats' fields: sign, exponent, fraction."""
    c = codes.long()
    if fmt == "mxfp4":
        c = torch.stack((c.remainder(16), c.div(16, rounding_mode="floor")), -1).flatten(-2)
        sign, e, f, bias, bits = c // 8, c // 2 % 4, c % 2, 1, 1
    else:
        sign, e, f, bias, bits = c // 128, c // 8 % 16, c % 8, 7, 3
    power = _two(e.clamp(min=1) - bias)
    v = (1 - 2 * sign) * power * ((e > 0).double() + f.double() / 2**bits)
    return v * _two(scales.long() - 127).repeat_interleave(32, -1)


def _exact_held(y, fmt):
    """Float64 rows (each value one of binary32) -> the values after `fmt`, by the formats' grids."""
    b = y.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "q8_1":
        d = (top / 127).float().double()
        kept = d.half().double()
        r = torch.where(kept > 0, (1 / d.clamp(min=1e-300)).float().double(), 0.0)
        t = (b * r).float().double()
        return (t.sign() * (t.abs() + 0.5).floor().clamp(max=127) * kept).float().double().flatten(-2)
    most, low, bits, above = (6.0, 0, 1, 2) if fmt == "mxfp4" else (448.0, -6, 3, 8)
    e = torch.frexp(top)[1] - 1 - above
    scale = _two(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
    v = b / scale
    grid = _two((torch.frexp(v)[1] - 1).clamp(min=low) - bits)
    return (torch.round(v / grid) * grid).clamp(-most, most).mul(scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rows":
        return {"held": _exact_held(s["x"].double(), s["fmt"])}
    if s["op"] == "norm":
        h = (s["x"].double() + s["res"].double()).to(s["x"].dtype)
        f = h.double()
        u = torch.rsqrt((f * f).sum(-1, keepdim=True) / s["k"] + s["eps"]).float().double()
        y = ((f * u).float().double() * s["gain"].double()).float().double()
        out = {"h": h.double(), "held": _exact_held(y, s["fmt"])}
        return out | {"y": y} if s["plain"] else out
    rows = _exact_bytes(s["codes"], s["scales"], s["fmt"])
    if s["op"] == "product":
        return {"y": rows @ _exact_bytes(s["w_codes"], s["w_scales"], "mxfp4").t()}
    if s["pairs"] is not None:
        rows = rows[torch.div(s["pairs"], s["top"], rounding_mode="floor").long()]
    at, y = s["offsets"].tolist(), []
    for e in range(s["experts"]):
        if at[e + 1] > at[e]:
            y.append(rows[at[e]:at[e + 1]] @ _exact_bytes(s["w_codes"][e], s["w_scales"][e], "mxfp4").t())
    return {"y": torch.cat(y)}


def _row_bytes(k, fmt):
    return {"q8_1": k + k // 16, "mxfp8": k + k // 32, "mxfp4": k // 2 + k // 32}[fmt]


def work(case):
    op, k = case["op"], case["k"]
    if op in ("norm", "rows"):
        m, t = case["m"], SIZE[case["type"]]
        moved = m * (k * t + _row_bytes(k, case["fmt"]) + 4 * k)  # the rows, what holds them, the values they stand for
        if op == "rows":
            return {"bytes": moved, "flops": 4 * m * k}
        return {"bytes": moved + m * k * t * (3 if case["plain"] else 2) + 4 * k, "flops": 8 * m * k}
    matrix = case["n"] * _row_bytes(k, "mxfp4")
    if op == "product":
        m, rows, matrices = case["m"], case["m"], 1
    else:
        m = case["tokens"] * case["top"]
        rows = case["tokens"] if case["gather"] else m
        matrices = min(case["experts"], float((1 - (1 - _share(case["experts"])) ** m).sum()))  # experts that get a row
    return {"bytes": int(matrices * matrix + rows * _row_bytes(k, case["fmt"]) + m * case["n"] * SIZE[case["out"]]), "flops": 2 * m * case["n"] * k}
