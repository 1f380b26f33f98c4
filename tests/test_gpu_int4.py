"""4-bit KV cache on a B200 against the oracle: cache bytes bit for bit (every
finite half, constant rows, rows with infinities and NaN, strided inputs, slots
that are skipped or out of range), the read-back, decode over the cache for every
head layout, length and split, whole-block copies and swaps, and the calls around
them (streams, graphs, pools past 2^32 bytes, bad block ids).

Tolerance of a decode element, from the arithmetic of the kernel (all sums in
fp32): with X the largest sum of absolute terms of a score,
  scores   8 chained products of 16 terms and 6 more operations, each within 2^-23
           of the absolute sum: dx = X (8 * 17 + 6) 2^-23; a weight is off by at
           most e_p = 2 dx + 2^-20 of itself (exp2 and its argument included)
  weights  rounded to half, 2^-11 (bf16 outputs), or kept to 2^-21 by the residual
           (half outputs), acting on the centred codes: at most 7.5 scale
  sums     over N tokens, N / 16 + 32 rounded additions of terms up to 15 scale + |mid|
  output   half a step of its type
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from oracle import cache_ops as OC
from oracle import int4 as I4
from oracle.fpbits import bits_to_f64
from tests.parity import out_to_f64, tensor_bits
from workloads import gen

pytestmark = pytest.mark.gpu

TDT = {"f16": torch.float16, "bf16": torch.bfloat16}


def dev16(bits, dt):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(TDT[dt]).cuda()


def f32(bits, dt):
    return bits_to_f64(bits, dt).astype(np.float32)


def caches(nb, hkv, d, fill=0xFF):
    """Device caches full of `fill` (0xFF: NaN parameters in every unwritten slot)."""
    k = torch.full((nb, hkv, 16, d // 2 + 4), fill, dtype=torch.uint8, device="cuda")
    return k, torch.full_like(k, fill)


def tolerance(ref, q, k, v, kpar, vpar, scale, dt):
    """Elementwise bound for one (sequence, head): q [d], k/v [n, d], parameters [n, 2]."""
    n = len(k)
    qa = np.abs(q).sum()
    X = abs(scale) * float((np.abs(kpar[:, 0]) * 15 * qa + np.abs(kpar[:, 1]) * qa).max())
    dx = X * (8 * 17 + 6) * 2.0 ** -23
    e_p = 2 * dx + 2.0 ** -20
    e_w = 2.0 ** -11 if dt == "bf16" else 2.0 ** -20
    s, top = float(np.abs(vpar[:, 0]).max()), float(np.abs(v).max())
    term = 15 * s + float(np.abs(vpar[:, 1]).max())
    return (2 * e_p * top + e_w * 7.5 * s + (n / 16 + 32) * 2.0 ** -23 * term +
            torch.finfo(TDT[dt]).eps / 2 * np.abs(ref) + 2.0 ** -25)


def params(cache):
    nb, hkv, _, row = cache.shape
    d = 2 * (row - 4)
    return cache.reshape(nb, hkv, -1)[:, :, 8 * d:].copy().view(np.float16).astype(
        np.float64).reshape(nb, hkv, 16, 2)


def check_decode(out, q_bits, kc, vc, tables, ctx, scale, dt, rows=None):
    """Every (sequence, head) row of `out` (or the listed sequences) against the oracle."""
    got = out_to_f64(out, dt)
    q = bits_to_f64(q_bits, dt)
    kv, vv = I4.dequantize_cache(kc, False), I4.dequantize_cache(vc, True)
    kp, vp = params(kc), params(vc)
    G = q.shape[1] // kc.shape[1]
    for s in rows if rows is not None else range(len(ctx)):
        n = int(ctx[s])
        if n == 0:
            assert not got[s].any()
            continue
        blocks = tables[s][:-(-n // 16)]
        for h in range(q.shape[1]):
            cut = lambda x: np.concatenate([x[b, h // G] for b in blocks])[:n]
            k, v = cut(kv), cut(vv)
            ref = I4.softmax_attention(q[s, h], k, v, scale)
            tol = tolerance(ref, q[s, h], k, v, cut(kp), cut(vp), scale, dt)
            err = np.abs(got[s, h] - ref)
            assert (err <= tol).all(), (s, h, n, float(err.max()), float(tol[err.argmax()]))


class Batch:
    """A seeded batch over 4-bit caches: rows written by the library (bit-exact against the
    oracle, tested below), NaN parameters in every unused slot."""

    def __init__(self, ctx, hq, hkv, d, dt, seed, kscale=1.0, vscale=1.0, qscale=1.0):
        self.ctx = np.asarray(ctx, np.int32)
        self.hq, self.hkv, self.d, self.dt = hq, hkv, d, dt
        blocks = [-(-int(c) // 16) for c in ctx]
        self.nb = sum(blocks) + 3
        perm = np.random.default_rng([seed, 9]).permutation(self.nb).astype(np.int32)
        self.tables = np.full((len(ctx), max(max(blocks), 1)), -1, np.int32)
        used = 0
        for s, n in enumerate(blocks):
            self.tables[s, :n] = perm[used:used + n]
            used += n
        T = int(self.ctx.sum())
        slots = np.array([int(self.tables[s, p // 16]) * 16 + p % 16
                          for s in range(len(ctx)) for p in range(int(self.ctx[s]))], np.int64)
        self.key = gen.normal_bits([seed, 1], (T, hkv, d), dt, kscale)
        self.value = gen.normal_bits([seed, 2], (T, hkv, d), dt, vscale)
        self.q = gen.normal_bits([seed, 3], (len(ctx), hq, d), dt, qscale)
        self.kc, self.vc = caches(self.nb, hkv, d)
        if T:
            pa.pa_reshape_and_cache_int4(dev16(self.key, dt), dev16(self.value, dt), self.kc,
                                         self.vc, torch.from_numpy(slots).cuda())
        self.scale = 1 / math.sqrt(d)
        self.t = torch.from_numpy(self.tables).cuda()
        self.c = torch.from_numpy(self.ctx).cuda()
        self.qd = dev16(self.q, dt)
        self.max_ctx = int(self.ctx.max())

    def run(self, part=0, order=False, err=None, ws=None, out=None, q=None, stream=None):
        out = torch.full_like(self.qd, float("nan")) if out is None else out
        if ws is None:
            ws = pa.decode_workspace(len(self.ctx), self.hq, self.hkv, self.d, self.max_ctx, part)
        o = torch.from_numpy(pa.pa_longest_first_order(self.ctx)).cuda() if order else None
        pa.pa_paged_decode_int4(out, self.qd if q is None else q, self.kc, self.vc, self.t, self.c,
                                self.max_ctx, self.scale, part, ws, err, stream, o)
        return out

    def check(self, out, rows=None):
        check_decode(out, self.q, self.kc.cpu().numpy(), self.vc.cpu().numpy(), self.tables,
                     self.ctx, self.scale, self.dt, rows)


# ---- the write and the read-back --------------------------------------------------

def oracle_write(nb, hkv, d, key, value, slots, fill=0x55):
    k = np.full((nb, hkv, 16, d // 2 + 4), fill, np.uint8)
    v = np.full_like(k, fill)
    I4.reshape_and_cache_int4(k, v, key, value, slots)
    return k, v


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_write_bytes(dt, d):
    hkv, T, nb = 3, 61, 9
    key = gen.normal_bits([71, d], (T, hkv, d), dt)
    value = gen.normal_bits([72, d], (T, hkv, d), dt, 3.0)
    top = 0x7BFF if dt == "f16" else 0x7F7F
    key[0, 0] = 0                                   # all zero: scale 0
    key[1, 0] = 0x3C00 if dt == "f16" else 0x3F80   # constant
    key[2, 1, 5] = top                              # largest finite (clamped for bf16)
    key[3, 1, 0], key[3, 1, 7] = top, top | 0x8000
    key[4, 2] = np.arange(d)                        # subnormals
    value[5, 0, :] = 0x8000                         # -0
    slots = np.random.default_rng(3).permutation(nb * 16)[:T].astype(np.int64)
    slots[::13] = -1
    kc, vc = caches(nb, hkv, d, 0x55)
    pa.pa_reshape_and_cache_int4(dev16(key, dt), dev16(value, dt), kc, vc,
                                 torch.from_numpy(slots).cuda())
    ok, ov = oracle_write(nb, hkv, d, f32(key, dt), f32(value, dt), slots)
    assert np.array_equal(kc.cpu().numpy(), ok)
    assert np.array_equal(vc.cpu().numpy(), ov)
    # and back: value = mid + (code - 7.5) scale, rounded once; skipped rows stay
    kb = torch.full((T, hkv, d), 7.0, dtype=TDT[dt], device="cuda")
    vb = torch.full_like(kb, 7.0)
    pa.pa_read_slots_int4(kb, vb, kc, vc, torch.from_numpy(slots).cuda())
    for back, cache, values in ((kb, ok, False), (vb, ov, True)):
        ref = I4.dequantize_cache(cache, values)
        want = np.full((T, hkv, d), 7.0)
        for t, s in enumerate(slots):
            if s >= 0:
                want[t] = ref[s // 16, :, s % 16]
        want = torch.from_numpy(want.astype(np.float32)).to(TDT[dt])  # exact in fp32: 2 halves
        assert np.array_equal(tensor_bits(back), tensor_bits(want))


def test_write_every_finite_half():
    """Every finite half appears once in a row: rows of neighbouring values and shuffled ones."""
    hkv, d = 4, 128
    pos = np.arange(0, 0x7C00, dtype=np.uint16)
    vals = np.concatenate([pos, pos | 0x8000])
    vals = np.concatenate([vals, np.zeros((-len(vals)) % (hkv * d), np.uint16)])
    key = vals.reshape(-1, hkv, d)
    value = np.random.default_rng(4).permutation(vals).reshape(-1, hkv, d)
    T = len(key)
    nb = -(-T // 16)
    slots = np.arange(T, dtype=np.int64)
    kc, vc = caches(nb, hkv, d, 0)
    pa.pa_reshape_and_cache_int4(dev16(key, "f16"), dev16(value, "f16"), kc, vc,
                                 torch.from_numpy(slots).cuda())
    ok, ov = oracle_write(nb, hkv, d, f32(key, "f16"), f32(value, "f16"), slots, 0)
    assert np.array_equal(kc.cpu().numpy(), ok) and np.array_equal(vc.cpu().numpy(), ov)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_write_infinities_and_nan(dt):
    """Infinities are clamped to the halves' range; a row with a NaN reads back as NaN, and so
    does the attention over it, while its neighbours are untouched."""
    hkv, d, nb = 2, 64, 2
    inf, nan = (0x7C00, 0x7E01) if dt == "f16" else (0x7F80, 0x7FC1)
    key = gen.normal_bits([81], (16, hkv, d), dt)
    value = gen.normal_bits([82], (16, hkv, d), dt)
    key[2, 0, 9], key[2, 0, 11] = inf, inf | 0x8000
    value[4, 1, 63] = nan
    slots = np.arange(16, dtype=np.int64)
    kc, vc = caches(nb, hkv, d, 0)
    pa.pa_reshape_and_cache_int4(dev16(key, dt), dev16(value, dt), kc, vc,
                                 torch.from_numpy(slots).cuda())
    ok, ov = oracle_write(nb, hkv, d, f32(key, dt), f32(value, dt), slots, 0)
    assert np.array_equal(kc.cpu().numpy(), ok)
    got = vc.cpu().numpy()
    assert np.isnan(params(got)[0, 1, 4]).all()
    got[0, 1].reshape(-1)[8 * d + 16:8 * d + 20] = ov[0, 1].reshape(-1)[8 * d + 16:8 * d + 20]
    assert np.array_equal(got, ov)                 # every code, the NaN row's (0) included
    q = dev16(gen.normal_bits([83], (1, hkv, d), dt), dt)
    out = torch.empty_like(q)
    tables = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for n, bad in ((4, False), (5, True)):
        ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
        pa.pa_paged_decode_int4(out, q, kc, vc, tables, ctx, 16, 0.125)
        assert bool(torch.isfinite(out[0, 0]).all())
        assert bool(torch.isnan(out[0, 1]).all()) == bad


def test_write_strides_slots_and_empty():
    hkv, d, nb = 2, 64, 4
    wide = dev16(gen.normal_bits([84], (9, 3 * hkv, d), "f16"), "f16")   # a fused qkv projection
    key, value = wide[:, hkv:2 * hkv], wide[:, 2 * hkv:]
    slots = torch.tensor([0, -1, 17, 64, 5, 63, 1 << 40, 2, 3], dtype=torch.int64, device="cuda")
    kc, vc = caches(nb, hkv, d, 0x33)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_int4(key, value, kc, vc, slots, err)
    assert err.item() == pa.PA_DEVERR_SLOT_RANGE
    s = slots.cpu().numpy()
    s[s >= 64] = -1
    b = tensor_bits(wide)
    ok, ov = oracle_write(nb, hkv, d, f32(b[:, hkv:2 * hkv], "f16"), f32(b[:, 2 * hkv:], "f16"), s,
                          0x33)
    assert np.array_equal(kc.cpu().numpy(), ok) and np.array_equal(vc.cpu().numpy(), ov)
    err.zero_()
    back = torch.full((9, 3 * hkv, d), 5.0, dtype=torch.float16, device="cuda")
    pa.pa_read_slots_int4(back[:, :hkv], back[:, hkv:2 * hkv], kc, vc, slots, err)
    assert err.item() == pa.PA_DEVERR_SLOT_RANGE
    assert bool((back[:, 2 * hkv:] == 5).all())
    assert bool((back[torch.from_numpy(s < 0).cuda()] == 5).all())
    before = kc.clone()
    pa.pa_reshape_and_cache_int4(key[:0], value[:0], kc, vc, slots[:0])
    pa.pa_read_slots_int4(back[:0, :hkv], back[:0, :hkv], kc, vc, slots[:0])
    assert torch.equal(kc, before)


# ---- decode ------------------------------------------------------------------------

@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_decode_layouts(G, d, dt):
    b = Batch([1, 0, 15, 16, 17, 33, 250, 1100], G * 3, 3, d, dt, 100 * G + d)
    for part in (0, 16, 64, 512):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = b.run(part, order=part == 64, err=err)
        assert err.item() == 0
        b.check(out)


@pytest.mark.parametrize("G", [1, 8])
def test_decode_warp_partitions(G):
    """Enough sequences of short partitions for one warp per partition and a merge launch."""
    ctx = np.random.default_rng(5).integers(1000, 2100, 64)
    ctx[3], ctx[7] = 0, 1
    b = Batch(ctx, 4 * G, 4, 64, "bf16", 7)
    assert pa.pa_paged_decode_plan(64, 4 * G, 4, 64, b.max_ctx, 64)[2] == 2
    b.check(b.run(64), rows=[0, 3, 7, 31, 63])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("part", [65536, 0])
def test_decode_long_context_mean(dt, part):
    """60000 tokens, in one partition and in the library's: the output is a mean of thousands of
    values, a hundredth of one of them, and has to stay within the type's rounding of it. Bound
    of the relative norm: half a step of the type (its root mean square is below) plus the
    weights' share, 2^-11 rounded to bf16's operands (sqrt(1/3) of it in the mean, over the
    centred codes), plus 64 additions of the matrix instruction at 2^-24 of 7.5 scale each."""
    b = Batch([60000], 4, 1, 128, dt, 43)
    out = b.run(part)
    kc, vc = b.kc.cpu().numpy(), b.vc.cpu().numpy()
    blocks = b.tables[0]
    k = np.concatenate([x for x in I4.dequantize_cache(kc, False)[blocks, 0]])[:60000]
    v = np.concatenate([x for x in I4.dequantize_cache(vc, True)[blocks, 0]])[:60000]
    scale = float(params(vc)[blocks, 0].reshape(-1, 2)[:60000, 0].max())
    got = out_to_f64(out[0], dt)
    for h in range(4):
        ref = I4.softmax_attention(bits_to_f64(b.q, dt)[0, h], k, v, b.scale)
        rms = float(np.sqrt((ref ** 2).mean()))
        step = torch.finfo(TDT[dt]).eps / 2
        bound = step + (2.0 ** -11 if dt == "bf16" else 2.0 ** -20) + 64 * 2.0 ** -24 * 7.5 * scale / rms
        assert np.linalg.norm(got[h] - ref) <= bound * np.linalg.norm(ref), (
            h, np.linalg.norm(got[h] - ref) / np.linalg.norm(ref), bound)


def test_decode_value_scales_of_every_size():
    """Value rows whose scales differ by 2^20, rising, falling and zero: the reference of the
    weights moves, and small rows keep their share when the large ones carry no weight."""
    ctx, d, hkv = [200, 333], 128, 2
    b = Batch(ctx, 4, hkv, d, "f16", 11)
    v = f32(b.value, "f16")
    rng = np.random.default_rng(6)
    grow = 2.0 ** np.concatenate([np.linspace(-14, 6, 200), rng.uniform(-14, 6, 333)])
    v *= grow[:, None, None].astype(np.float32)
    v[::17] = 0.25                                  # constant rows: scale 0
    b.value = v.astype(np.float16).view(np.uint16)
    slots = np.array([int(b.tables[s, p // 16]) * 16 + p % 16
                      for s in range(2) for p in range(ctx[s])], np.int64)
    pa.pa_reshape_and_cache_int4(dev16(b.key, "f16"), dev16(b.value, "f16"), b.kc, b.vc,
                                 torch.from_numpy(slots).cuda())
    b.check(b.run())
    b.check(b.run(32))
    # all values tiny: nothing is lost to the reference
    tiny = (v * np.float32(0) + 2.0 ** -13 * rng.standard_normal(v.shape)).astype(np.float16)
    pa.pa_reshape_and_cache_int4(dev16(b.key, "f16"), dev16(tiny.view(np.uint16), "f16"), b.kc,
                                 b.vc, torch.from_numpy(slots).cuda())
    out = b.run()
    b.check(out)
    assert out.abs().max() > 0


@pytest.mark.parametrize("dt,mag", [("f16", 0.0), ("f16", 2.0 ** -20), ("f16", 1000.0),
                                    ("bf16", 2.0 ** -120), ("bf16", 1e5), ("bf16", 2.0 ** 60)])
def test_decode_query_magnitudes(dt, mag):
    """Queries far outside half's range, and zero: the softmax scale brings the scores back."""
    b = Batch([40, 100], 8, 2, 64, dt, 13)
    bits = b.q
    qf = f32(bits, dt) * np.float32(mag)
    b.q = gen.f32_to_bits(qf, dt)
    b.qd = dev16(b.q, dt)
    b.scale = 0.125 / max(mag, 2.0 ** -10)
    b.check(b.run())


def test_decode_bad_ids_and_contexts():
    b = Batch([50, 40, 30, 70], 4, 2, 64, "f16", 17)
    ref = b.run(16)
    b.t[1, 1] = b.nb                                   # one block of sequence 1
    b.c[2] = 16 * b.tables.shape[1] + 1                # longer than the table
    b.c[3] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.run(16, err=err)
    assert err.item() == pa.PA_DEVERR_BLOCK_RANGE | pa.PA_DEVERR_CONTEXT_RANGE
    assert torch.equal(out[0], ref[0]) and not out[2:].any()
    # the bad block is left out of sequence 1: attention over the rest of its tokens
    kv, vv = (I4.dequantize_cache(c.cpu().numpy(), v) for c, v in ((b.kc, False), (b.vc, True)))
    q = bits_to_f64(b.q, "f16")
    rows = [x for x in range(40) if x // 16 != 1]
    for h in range(4):
        k, v = (np.stack([x[b.tables[1, p // 16], h // 2, p % 16] for p in rows]) for x in (kv, vv))
        want = I4.softmax_attention(q[1, h], k, v, b.scale)
        assert np.abs(out_to_f64(out[1, h], "f16") - want).max() < 4e-3
    b.t[0, :] = -1
    assert not b.run(16)[0].any()                      # no readable block: a zero row


def test_decode_placement_and_repeat_are_bit_identical():
    ctx = [3, 64, 500, 1000]
    b = Batch(ctx, 16, 4, 128, "bf16", 19)
    first = b.run()
    assert torch.equal(first, b.run())
    perm = torch.randperm(b.nb)
    k2, v2 = b.kc.clone(), b.vc.clone()
    k2[perm.cuda()], v2[perm.cuda()] = b.kc, b.vc
    b.kc, b.vc = k2, v2
    b.t = torch.where(b.t >= 0, perm.to(torch.int32).cuda()[b.t.clamp(min=0).long()], b.t)
    assert torch.equal(first, b.run())


def test_decode_streams_and_graph():
    """A side stream, a captured graph replayed with new queries, and two graphs at once on
    workspaces of their own."""
    b = Batch([700, 1500, 16], 8, 1, 128, "f16", 23)
    want = b.run(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run(64)
    side.synchronize()
    assert torch.equal(want, got)
    graphs = []
    for _ in range(2):
        ws = pa.decode_workspace(3, 8, 1, 128, b.max_ctx, 64)
        q, out = b.qd.clone(), torch.empty_like(b.qd)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(64, ws=ws, out=out, q=q)
        graphs.append((g, ws, q, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs[1][2].copy_(b.qd.flip(0))
    torch.cuda.synchronize()
    for (g, *_), st in zip(graphs, streams):
        with torch.cuda.stream(st):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][3], want)
    b.q, b.qd = b.q[::-1].copy(), b.qd.flip(0).contiguous()
    assert torch.equal(graphs[1][3], b.run(64))
    b.check(graphs[1][3])


def test_decode_pool_past_4_gib():
    """Blocks whose byte offset passes 2^32 in each pool."""
    hkv, d = 8, 128
    tile = hkv * 16 * (d // 2 + 4)
    nb = (1 << 32) // tile + 40
    kc = torch.zeros(nb, hkv, 16, d // 2 + 4, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    n = 300
    blocks = np.arange(nb - 19, nb, dtype=np.int32)[::-1].copy()
    slots = np.array([int(blocks[p // 16]) * 16 + p % 16 for p in range(n)], np.int64)
    key, value = (gen.normal_bits([91, i], (n, hkv, d), "bf16") for i in (1, 2))
    pa.pa_reshape_and_cache_int4(dev16(key, "bf16"), dev16(value, "bf16"), kc, vc,
                                 torch.from_numpy(slots).cuda())
    qb = gen.normal_bits([91, 3], (1, hkv, d), "bf16")
    q = dev16(qb, "bf16")
    out = torch.empty_like(q)
    pa.pa_paged_decode_int4(out, q, kc, vc, torch.from_numpy(blocks[None]).cuda(),
                            torch.tensor([n], dtype=torch.int32, device="cuda"), n, 0.09)
    low = nb - 19
    check_decode(out, qb, kc[low:].cpu().numpy(), vc[low:].cpu().numpy(), (blocks - low)[None],
                 [n], 0.09, "bf16")
    kb = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    vb = torch.empty_like(kb)
    pa.pa_read_slots_int4(kb, vb, kc, vc, torch.from_numpy(slots).cuda())
    ref = I4.dequantize_cache(kc[low:].cpu().numpy(), False)
    want = np.stack([ref[s // 16 - low, :, s % 16] for s in slots])
    assert np.array_equal(tensor_bits(kb),
                          tensor_bits(torch.from_numpy(want.astype(np.float32)).bfloat16()))


def test_copy_and_swap_blocks():
    rng = np.random.default_rng(12)
    shape = (12, 3, 16, 68)
    k, v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
    kc, vc = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    pairs = [(0, 5), (3, 1), (3, 11)]
    pa.pa_copy_blocks(kc, vc, pairs)
    OC.copy_blocks(k, v, pairs)
    assert np.array_equal(kc.cpu().numpy(), k) and np.array_equal(vc.cpu().numpy(), v)
    hk, hv = (torch.zeros(4, *shape[1:], dtype=torch.uint8).pin_memory() for _ in range(2))
    pa.pa_swap_blocks(kc, vc, hk, hv, [(5, 2), (11, 0)])
    torch.cuda.synchronize()
    assert np.array_equal(hk.numpy()[[2, 0]], k[[5, 11]])
    assert np.array_equal(hv.numpy()[[2, 0]], v[[5, 11]])
    assert not hk[1].any() and not hk[3].any()


def test_stall_request_is_left_to_the_other_decodes():
    """The 4-bit decode has no on-chip barrier waits: the library's test hook does not touch it
    and stays armed for the next decode that has."""
    from paged_kv_cache_352_b200 import _lib as L
    b = Batch([200, 90], 4, 2, 64, "f16", 29)
    want = b.run(64)
    assert L.lib().pa_test_stall_next_decode(200000) == 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(want, b.run(64, err=err)) and err.item() == 0
    kc = torch.zeros(b.nb, 2, 16, 64, dtype=torch.float16, device="cuda")
    ws = pa.decode_workspace(2, 4, 2, 64, b.max_ctx, 64)
    pa.pa_paged_decode(torch.empty_like(b.qd), b.qd, kc, kc, b.t, b.c, b.max_ctx, 0.1, 64, ws, err)
    assert err.item() & pa.PA_DEVERR_WAIT_TIMEOUT


@pytest.mark.parametrize("mode,host,cascade", [("swap", 400, None), ("recompute", 0, None),
                                               ("swap", 400, pa.PA_SCHED_CASCADE_ON)])
def test_serving_loop_over_a_4_bit_cache(mode, host, cascade):
    """The scheduler's executor attached to 4-bit pools: admissions, copy-on-write, preemption by
    swap or recomputation, every step's pool bytes and outputs against the oracle; the cascade
    stays off whatever its mode."""
    hq, hkv, d, dt, nb, cap = 8, 2, 64, "f16", 18, 10
    swap = mode == "swap"
    order = np.random.default_rng(61).permutation(nb)
    pm = pa.PA_PREEMPT_SWAP if swap else pa.PA_PREEMPT_RECOMPUTE
    c = pa.Scheduler(nb, 16, order, max_num_seqs=cap, num_host_blocks=host, preempt_mode=pm)
    rng = np.random.default_rng(62)
    trace = [(i, int(rng.integers(1, 60)), int(rng.integers(1, 25)),
              int(rng.integers(1, 4)) if swap else 1, int(rng.integers(0, 6))) for i in range(24)]
    for t in trace:
        c.submit(*t)
    c.attach(hq, hkv, d, torch.float16, 90, int4=True)
    if cascade is not None:
        c.set_cascade(cascade)
    kc, vc = caches(nb, hkv, d, 0)
    ok, ov = kc.cpu().numpy(), vc.cpu().numpy()
    hk, hv = (torch.zeros(max(host, 1), hkv, 16, d // 2 + 4, dtype=torch.uint8).pin_memory()
              for _ in range(2))
    sk, sv = hk.numpy().copy(), hv.numpy().copy()
    toks = gen.RequestTokens(63, {t[0]: t[1] for t in trace}, hkv, d, dt,
                             prompt_tokens={t[0]: None for t in trace})
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    seen = {"swap_out": 0, "swap_in": 0, "copies": 0, "preempted": 0}
    step = 0
    while not c.idle():
        c.step()
        p = c.plan()
        for k in seen:
            seen[k] += len(p[k])

        def rows(ws):
            got = [toks.row(r, s, pos) for r, s, pos, _ in ws]
            pick = lambda i: np.array([x[i] for x in got], np.uint16).reshape(-1, hkv, d)
            return pick(0), pick(1), [int(w[3]) for w in ws]

        pk, pv, ps = rows(p["prefill"])
        wk, wv, ws = rows(p["writes"])
        q = gen.normal_bits([64, step], (len(p["batch"]), hq, d), dt)
        out = torch.empty(len(p["batch"]), hq, d, dtype=torch.float16, device="cuda")
        c.execute(kc, vc, hk if host else None, hv if host else None, dev16(pk, dt), dev16(pv, dt),
                  dev16(wk, dt), dev16(wv, dt), dev16(q, dt), out, 0.125, dev_error=err)
        torch.cuda.synchronize()
        assert c.last_cascade()[0] == 0
        for a, b in p["swap_out"]:
            sk[b], sv[b] = ok[a], ov[a]
        for a, b in p["swap_in"]:
            ok[b], ov[b] = sk[a], sv[a]
        I4.reshape_and_cache_int4(ok, ov, f32(pk, dt), f32(pv, dt), ps)
        for a, b in p["copies"]:
            ok[b], ov[b] = ok[a], ov[a]
        I4.reshape_and_cache_int4(ok, ov, f32(wk, dt), f32(wv, dt), ws)
        assert np.array_equal(kc.cpu().numpy(), ok) and np.array_equal(vc.cpu().numpy(), ov)
        ctx = [int(x[2]) for x in p["batch"]]
        check_decode(out, q, ok, ov, np.asarray(p["tables"]), ctx, 0.125, dt)
        step += 1
    assert err.item() == 0 and seen["preempted"] > 0, seen
    assert not swap or (seen["swap_in"] > 0 and seen["copies"] > 0), seen


def test_refusals_on_device_tensors():
    b = Batch([20], 2, 2, 64, "f16", 31)
    with pytest.raises(pa.PAError):                     # an E4M3-shaped pool
        bad = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda")
        pa.pa_paged_decode_int4(b.qd, b.qd, bad, bad, b.t, b.c, 20, 0.1)
    with pytest.raises(pa.PAError):                     # other types for q and out
        pa.pa_paged_decode_int4(b.qd.bfloat16(), b.qd, b.kc, b.vc, b.t, b.c, 20, 0.1)
    with pytest.raises(pa.PAError):                     # a split without a workspace
        pa.pa_paged_decode_int4(b.qd, b.qd, b.kc, b.vc, b.t, b.c, 20, 0.1, 16)
    with pytest.raises(pa.PAError):
        pa.pa_paged_decode_int4(b.qd, b.qd[:, :1], b.kc, b.vc, b.t, b.c, 20, 0.1)
    with pytest.raises(pa.PAError):
        pa.pa_reshape_and_cache_int4(b.qd, b.qd, b.kc, b.vc,
                                     torch.zeros(1, dtype=torch.int32, device="cuda"))
