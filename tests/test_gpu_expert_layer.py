"""The experts' operators in a run, as a layer has them: route, gather, products by expert, SwiGLU,
combine, and back.

Each step is held to the oracle on what the device had as its input, so that its own bound counts and no
other: whole-number products exactly; real ones by their additions, a whole step of binary32 (2^-23) of
the magnitudes each; SwiGLU by 2^-20 and half a step of its type; combined rows bit for bit.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import dev, host, note
from rows_util import FMT, HALF_STEP, TYPES, floats, packed, row_buffers, rounder, split_rows
from test_gpu_g4 import bank
from test_gpu_slots import combined

pytestmark = pytest.mark.gpu
F = np.float32


def _dims(tokens, experts, top, hidden, inter):
    return {"tokens": tokens, "experts": experts, "top": top, "hidden": hidden, "inter": inter}


class Layer:
    """One layer's weights and buffers; `run` enqueues it whole."""

    def __init__(self, seed, d, t):
        self.d, self.t = d, t
        self.gu, self.w_gu = bank(seed, d["experts"], 2 * d["inter"], d["hidden"], 32, True, "f16")
        self.down, self.w_down = bank(seed + 50, d["experts"], d["hidden"], d["inter"], 32, False, "bf16")
        pairs = d["tokens"] * d["top"]
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        typed = lambda *s: torch.zeros(*s, dtype=TYPES[t][1], device="cuda")  # noqa: E731
        self.x, self.logits = typed(d["tokens"], d["hidden"]), torch.zeros(d["tokens"], d["experts"], device="cuda")
        self.work = lambda: {"ids": i32(d["tokens"], d["top"]), "w": torch.zeros(d["tokens"], d["top"], device="cuda"), "counts": i32(d["experts"]),
                             "offsets": i32(d["experts"] + 1), "pairs": i32(pairs), "slot_row": i32(pairs), "gu": typed(pairs, 2 * d["inter"]),
                             "h": typed(pairs, d["inter"]), "rows": torch.zeros(pairs, d["hidden"], device="cuda"),
                             "out": typed(d["tokens"], d["hidden"])}

    def set(self, seed):
        rng = np.random.default_rng(seed)
        self.xs = rng.integers(-4, 5, (self.d["tokens"], self.d["hidden"])) / 32.0
        self.x.copy_(floats(self.xs, self.t))
        self.logits.copy_(dev(rng.standard_normal(tuple(self.logits.shape)).astype(F)))

    def run(self, b, stream=None):
        d, (code, _) = self.d, TYPES[self.t]
        T, E, top, H, I = (d[k] for k in ("tokens", "experts", "top", "hidden", "inter"))
        iq4.iq4_route_topk(self.logits, T, E, top, b["ids"], b["w"], stream=stream)
        iq4.iq4_moe_gather(b["ids"], T * top, E, b["counts"], b["offsets"], b["pairs"], b["slot_row"], stream=stream)
        iq4.iq4_g4_grouped_qmv(self.gu, E, 2 * I, H, 32, iq4.IQ4_F16, 1, self.x, code, H, T, b["offsets"], b["pairs"], top, T * top, b["gu"], code,
                               2 * I, stream=stream)
        iq4.iq4_swiglu(b["gu"], 2 * I, b["gu"][:, I:], 2 * I, code, T * top, I, b["h"], code, I, stream=stream)
        iq4.iq4_g4_grouped_qmv(self.down, E, H, I, 32, iq4.IQ4_BF16, 0, b["h"], code, I, T * top, b["offsets"], None, top, T * top, b["rows"],
                               iq4.IQ4_F32, H, stream=stream)
        iq4.iq4_moe_combine(b["rows"], iq4.IQ4_F32, H, T * top, b["slot_row"], b["w"], T, top, H, self.x, H, b["out"], code, H, stream=stream)

    def check(self, b):
        d, t = self.d, self.t
        I, top = d["inter"], d["top"]
        ids, w = host(b["ids"]), host(b["w"])
        pairs, slot = host(b["pairs"]), host(b["slot_row"]).reshape(ids.shape)
        assert np.array_equal(pairs[slot.reshape(-1)], np.arange(ids.size))
        of = ids.reshape(-1)[pairs]
        gu, h, rows = (host(b[k].double()) for k in ("gu", "h", "rows"))
        want = np.stack([oracle.g4_product(self.w_gu[e], self.xs[p // top][None])[0] for e, p in zip(of, pairs)])
        # whole numbers of 2^-6; what bfloat16 or binary16 hold of them is one rounding
        assert np.array_equal(gu, rounder(t)(want))
        want = oracle.swiglu(gu[:, :I], gu[:, I:])
        fine = abs(want) < float(torch.finfo(TYPES[t][1]).max)
        small = float(torch.finfo(TYPES[t][1]).smallest_normal) * HALF_STEP[t] * 2
        bound = (2.0**-20 + HALF_STEP[t]) * abs(want) + 2.0**-125 * abs(gu[:, :I] * gu[:, I:]) + small
        assert fine.all() and np.all(abs(h - want) <= bound)
        want = np.stack([oracle.g4_product(self.w_down[e], v[None])[0] for e, v in zip(of, h)])
        # bfloat16: terms of up to 31 |s h| (16 + q and 16 + z); s is at most 2.  What binary32's two
        # parts miss, 2^-23 |w h| and 2^-39 of the largest h, is far less than that allows
        mags = abs(h).sum(1, keepdims=True) * 2 * 31
        assert np.all(abs(rows - want) <= (I + 2 * I / 32 + 64) * 2.0**-23 * mags)
        want = combined(rows.astype(F), slot, w, self.xs.astype(F), len(rows))
        assert np.array_equal(host(b["out"].double()), rounder(t)(want.astype(np.float64)))


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("dims", [(1, 4, 2, 128, 32), (4, 16, 4, 256, 160), (33, 5, 3, 160, 96), (70, 8, 1, 288, 416)], ids=str)
def test_a_decode_layer(dims, t):
    note(f"layer: {dims} {t}")
    layer = Layer(3, _dims(*dims), t)
    layer.set(4)
    b = layer.work()
    layer.run(b)
    layer.check(b)


def test_a_layer_captured_and_replayed():
    """A graph of the layer, its inputs changed between replays, with eager layers between them."""
    note("layer: graph")
    layer = Layer(5, _dims(6, 8, 2, 256, 96), "bf16")
    b, c = layer.work(), layer.work()
    layer.set(1)
    layer.run(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(b)
    for i in range(5):
        layer.set(10 + i)
        graph.replay()
        layer.check(b)
        layer.run(c)
        assert all(torch.equal(b[k], c[k]) for k in b)


def test_two_layers_at_once():
    """Two streams with a layer each, nothing between them."""
    note("layer: two streams")
    layers = [Layer(7 + i, _dims(20, 8, 2, 256, 96), "f16") for i in range(2)]
    works = [[x.work() for _ in range(3)] for x in layers]
    for i, x in enumerate(layers):
        x.set(i)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for j in range(3):
        for x, s, b in zip(layers, streams, works):
            x.run(b[j], s)
    torch.cuda.synchronize()
    for x, bs in zip(layers, works):
        for b in bs:
            x.check(b)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_a_layer_of_mx_rows(fmt):
    """MXFP4 weights: rows quantised, the gate and up products, SwiGLU straight to rows, the down product, combine."""
    note(f"layer: {fmt} rows")
    T, E, top, H, I = 9, 4, 2, 256, 96
    rng = np.random.default_rng(2)
    wq = [[oracle.quantize_rows(rng.standard_normal((n, k)).astype(F), "mxfp4") for _ in range(E)] for n, k in ((2 * I, H), (H, I))]
    gu, down = (torch.cat([packed(*q, n, k) for q in ws]) for ws, (n, k) in zip(wq, ((2 * I, H), (H, I))))
    deq = [[oracle.dequant_rows(*q, "mxfp4") for q in ws] for ws in wq]
    x = floats(rng.standard_normal((T, H)), "bf16")
    ids = dev(np.stack([rng.permutation(E)[:top] for _ in range(T)]).astype(np.int32))
    w = dev(rng.random((T, top)).astype(F))
    counts, offsets, pairs, slot = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, T * top, T * top))
    iq4.iq4_moe_gather(ids, T * top, E, counts, offsets, pairs, slot)
    q, d, ldq, lds = row_buffers(fmt, T, H)
    iq4.iq4_quantize_rows(x, iq4.IQ4_BF16, T, H, H, FMT[fmt], q, ldq, d, lds)
    y = torch.zeros(T * top, 2 * I, device="cuda")
    iq4.iq4_mx_grouped_gemm(gu, E, 2 * I, H, FMT[fmt], q, ldq, d, lds, T, offsets, pairs, top, T * top, y, iq4.IQ4_F32, 2 * I)
    h = torch.zeros(T * top, I, device="cuda")
    q2, d2, ldq2, lds2 = row_buffers(fmt, T * top, I)
    iq4.iq4_swiglu(y, 2 * I, y[:, I:], 2 * I, iq4.IQ4_F32, T * top, I, h, iq4.IQ4_F32, I, FMT[fmt], q2, ldq2, d2, lds2)
    rows = torch.zeros(T * top, H, dtype=torch.bfloat16, device="cuda")
    iq4.iq4_mx_grouped_gemm(down, E, H, I, FMT[fmt], q2, ldq2, d2, lds2, T * top, offsets, None, top, T * top, rows, iq4.IQ4_BF16, H)
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    iq4.iq4_moe_combine(rows, iq4.IQ4_BF16, H, T * top, slot, w, T, top, H, x, H, out, iq4.IQ4_BF16, H)
    of, ps = host(ids).reshape(-1)[host(pairs)], host(pairs)
    xs = oracle.dequant_rows(*split_rows(fmt, H, q, d), fmt)
    got = host(y)
    for i, (e, p) in enumerate(zip(of, ps)):
        want, mags = oracle.mx_product(deq[0][e], xs[p // top][None])[0], oracle.mx_product(abs(deq[0][e]), abs(xs[p // top])[None])[0]
        assert np.all(abs(got[i] - want) <= H * 2.0**-24 * mags)
    want = oracle.swiglu(got[:, :I], got[:, I:])
    assert np.all(abs(host(h) - want) <= 2.0**-20 * abs(want) + 2.0**-120)
    codes = oracle.quantize_rows(host(h), fmt)
    assert all(np.array_equal(a, b) for a, b in zip(split_rows(fmt, I, q2, d2), codes))
    hs, got = oracle.dequant_rows(*codes, fmt), host(rows.double())
    for i, e in enumerate(of):
        want, mags = oracle.mx_product(deq[1][e], hs[i][None])[0], oracle.mx_product(abs(deq[1][e]), abs(hs[i])[None])[0]
        assert np.all(abs(got[i] - want) <= I * 2.0**-24 * mags + HALF_STEP["bf16"] * (abs(want) + I * 2.0**-24 * mags))
    want = combined(got.astype(F), host(slot).reshape(T, top), host(w), host(x.float()), T * top)
    assert np.array_equal(host(out.double()), rounder("bf16")(want.astype(np.float64)))


# ---- training ------------------------------------------------------------------------------


def _forward64(x, slot, w, n_rows, inter):
    rows = oracle.moe_dispatch(x, slot, None, np.zeros((n_rows, x.shape[1])))
    h = oracle.swiglu(rows[:, :inter], rows[:, inter:])
    return rows, h, oracle.moe_combine(h, slot, w)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("tokens,top,inter", [(1, 1, 5), (9, 3, 40), (70, 8, 33)])
def test_a_training_step(tokens, top, inter, captured):
    """Rows out, SwiGLU, rows back with weights, and the gradients of all three, some pairs dropped (rows
    that no pair has hold zeros): against the formulas in 64 bits and against differences."""
    note(f"layer: training {tokens} x {top}, {inter}, captured {captured}")
    rng = np.random.default_rng(tokens)
    n_rows, H = tokens * top + 3, 2 * inter
    slot = rng.permutation(n_rows)[: tokens * top].reshape(tokens, top).astype(np.int32)
    slot[rng.random(slot.shape) < 0.2] = -1
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    x, w, do = z(tokens, H), z(tokens, top), z(tokens, inter)
    rows, h, out, dh, dgu, dx, dw = z(n_rows, H), z(n_rows, inter), z(tokens, inter), z(n_rows, inter), z(n_rows, H), z(tokens, H), z(tokens, top)
    s = dev(slot)

    def step():
        iq4.iq4_moe_dispatch(x, 0, H, tokens, H, s, None, top, n_rows, rows, 0, H)
        iq4.iq4_swiglu(rows, H, rows[:, inter:], H, 0, n_rows, inter, h, 0, inter)
        iq4.iq4_moe_combine(h, 0, inter, n_rows, s, w, tokens, top, inter, None, 0, out, 0, inter)
        iq4.iq4_moe_combine_grad(do, 0, inter, h, 0, inter, n_rows, s, w, tokens, top, inter, dh, inter, dw)
        iq4.iq4_swiglu_grad(dh, 0, inter, rows, H, rows[:, inter:], H, 0, n_rows, inter, dgu, H, dgu[:, inter:], H)
        iq4.iq4_moe_combine(dgu, 0, H, n_rows, s, None, tokens, top, H, None, 0, dx, 0, H)

    run = step
    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    for _ in range(4 if captured else 1):
        xs, ws, dos = (rng.standard_normal(v.shape).astype(F).astype(np.float64) for v in (x, w, do))
        for v, a in ((x, xs), (w, ws), (do, dos)):
            v.copy_(dev(a.astype(F)))
        run()
        r64, h64, o64 = _forward64(xs, slot, ws, n_rows, inter)
        drows, dw64 = oracle.moe_combine_grad(dos, h64, slot, ws)
        drows = np.nan_to_num(drows)
        dg64, du64 = oracle.swiglu_grad(drows, r64[:, :inter], r64[:, inter:])
        dgu64 = np.concatenate([dg64, du64], 1)
        dx64 = oracle.moe_combine(dgu64, slot, None)
        # each value is off by 2^-20 (dg's by 2^-19 of (2 + |g|) / 2 times its size without the bracket), each
        # sum by half a step an addition and a product: all below 2^-17 of the magnitudes
        e = 2.0**-17
        g = abs(r64[:, :inter])
        mags = np.concatenate([abs(drows * r64[:, inter:]) * (2 + g), abs(du64)], 1)
        assert np.all(abs(host(out) - o64) <= e * oracle.moe_combine(abs(h64), slot, abs(ws)))
        assert np.all(abs(host(dw) - dw64) <= e * oracle.moe_combine_grad(abs(dos), abs(h64), slot, None)[1])
        assert np.all(abs(host(dgu) - dgu64) <= e * mags)
        assert np.all(abs(host(dx) - dx64) <= e * oracle.moe_combine(mags, slot, None))
        # differences, along a random direction of everything at once
        vx, vw, eps = rng.standard_normal(xs.shape), rng.standard_normal(ws.shape), 1e-6
        f = lambda a: (_forward64(xs + a * vx, slot, ws + a * vw, n_rows, inter)[2] * dos).sum()  # noqa: E731
        slope = (f(eps) - f(-eps)) / (2 * eps)
        mine = (host(dx) * vx).sum() + (host(dw) * vw).sum()
        size = np.abs(host(dx) * vx).sum() + np.abs(host(dw) * vw).sum() + abs(f(0.0)) * 1e-9 / eps
        assert abs(mine - slope) <= 1e-5 * size
