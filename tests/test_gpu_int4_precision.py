"""What the 4-bit decode's weights and sums lose, against the oracle, with a bound that follows
each token's share of the output.

With p_t the softmax weights, s_t and mid_t the value rows' parameters, P = sum p_t:
  scores   as in test_gpu_int4: a weight is off by at most e_p = 2 dx + 2^-20 of itself,
           dx = X 142 2^-23, so an output by 2 e_p sum p_t |v_t| / P
  weights  w_t = p_t s_t is kept to 2^-20 of itself and to 2^-30 of the largest one
           (a half and the half of what that rounds off), and acts on centred codes of at most 7.5
  sums     of a step (two blocks) the matrix instruction cuts its addends at 2^-23 of the largest,
           a code's operand counting as 2^9 of it, so at 2^-14 of the step's largest w: the running
           sum in each of at most 8 products, and of the weights' products those of an eighth of
           the largest and less (others end above that: 11 bits), at most 4 a token. The sum that
           the codes are centred by: 34 additions at 2^-23 of it, times 7.5. Steps add up in fp32,
           rounded to nearest: n / 128 + 64 additions a warp at 2^-24 of the centred sums
  output   half a step of its type."""

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from oracle import int4 as I4
from oracle.fpbits import bits_to_f64
from tests.parity import out_to_f64
from tests.test_gpu_int4 import TDT, Batch, dev16, f32, params
from workloads import gen

pytestmark = pytest.mark.gpu


def half_step(x, dt):
    """Half a step of type dt at magnitudes x (and what a rounding just above them takes)."""
    info = torch.finfo(TDT[dt])
    e = np.floor(np.log2(np.maximum(np.abs(x) * (1 + 2.0 ** -12), info.tiny)))
    return info.eps / 2 * 2.0 ** e


def rows_of(b, s, h):
    """(q, k, v, key parameters, value parameters) of one sequence's head in float64."""
    n = int(b.ctx[s])
    g = h // (b.hq // b.hkv)
    blocks = b.tables[s][:-(-n // 16)]
    kc, vc = (c[torch.from_numpy(blocks).long().cuda()][:, g:g + 1].cpu().numpy()
              for c in (b.kc, b.vc))
    cut = lambda x: x[:, 0].reshape(-1, x.shape[-1])[:n]
    return (bits_to_f64(b.q, b.dt)[s, h], cut(I4.dequantize_cache(kc, False)),
            cut(I4.dequantize_cache(vc, True)), cut(params(kc)), cut(params(vc)))


def cut_in_steps(w):
    """What the steps' products may lose, in codes times weights. A step is at most a block and a
    neighbour of it, however the blocks pair up."""
    blocks = np.pad(w, (0, -len(w) % 16)).reshape(-1, 16)
    m = np.pad(blocks.max(1), 1)
    m = np.maximum(np.maximum(m[:-2], m[1:-1]), m[2:])
    small = ((blocks > 0) & (blocks < m[:, None] / 8)).sum(1)
    return 2.0 ** -14 * float((m * (4 + 4 * small)).sum())


def bound(b, s, h):
    """(reference, elementwise bound) of one row."""
    q, k, v, kp, vp = rows_of(b, s, h)
    qa, n = np.abs(q).sum(), len(k)
    X = abs(b.scale) * float(((np.abs(kp[:, 0]) * 15 + np.abs(kp[:, 1])) * qa).max())
    e_p = 2 * X * 142 * 2.0 ** -23 + 2.0 ** -20
    z = k @ q * b.scale
    p = np.exp(z - z.max())
    P = p.sum()
    ref = p @ v / P
    w = p * np.abs(vp[:, 0])
    centred = p @ np.abs(v - vp[:, 1:]) / P
    lost = (2 * e_p * (p @ np.abs(v)) / P + 7.5 * (2.0 ** -20 * w.sum() + n * 2.0 ** -30 * w.max()) / P
            + (cut_in_steps(w) + 255 * 2.0 ** -23 * w.sum()) / P
            + (n / 128 + 64) * 2.0 ** -24 * centred)
    return ref, lost + half_step(np.abs(ref) + lost, b.dt) + 2.0 ** -25


def check(b, out, rows=None):
    got = out_to_f64(out, b.dt)
    for s in range(len(b.ctx)) if rows is None else rows:
        for h in range(b.hq):
            ref, tol = bound(b, s, h)
            err = np.abs(got[s, h] - ref)
            assert (err <= tol).all(), (s, h, float(err.max()), float(tol[(err / tol).argmax()]))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_weights_lose_nothing_that_the_output_keeps(G, d, dt):
    """Flat scores over value rows of different ranges: an output is within half a step of its
    type and a hundredth of that."""
    b = Batch([2, 9, 40, 100, 333], 2 * G, 2, d, dt, 300 + 10 * G + d, qscale=2.0 ** -9)
    v = f32(b.value, dt) * np.random.default_rng(G).uniform(0.2, 3, b.value.shape[:2])[..., None]
    write_values(b, v.astype(np.float32))
    for part in (0, 32):
        check(b, b.run(part))


def write_values(b, v, k=None):
    b.value = gen.f32_to_bits(v, b.dt)
    if k is not None:
        b.key = gen.f32_to_bits(k, b.dt)
    slots = np.array([int(b.tables[s, p // 16]) * 16 + p % 16
                      for s in range(len(b.ctx)) for p in range(int(b.ctx[s]))], np.int64)
    pa.pa_reshape_and_cache_int4(dev16(b.key, b.dt), dev16(b.value, b.dt), b.kc, b.vc,
                                 torch.from_numpy(slots).cuda())


def directed(b, offsets):
    """Keys that give sequence 0's tokens the scores `offsets` (head 0's KV head; q one-hot)."""
    q = np.zeros((1, b.hq, b.d), np.float32)
    q[:, :, 0] = 8.0
    b.q = gen.f32_to_bits(q, b.dt)
    b.qd = dev16(b.q, b.dt)
    k = np.zeros((len(offsets), b.hkv, b.d), np.float32)
    k[:, :, 0] = (np.asarray(offsets) / (8.0 * b.scale))[:, None]
    return k


@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lead", [32, 500])
def test_small_values_behind_constant_rows(dt, G, lead):
    """Tokens of high scores and constant value rows (scale 0), then thousands of low scores and
    small values: what the latter add is all there is, and no weight of theirs may underflow."""
    n = 3000
    b = Batch([n], G, 1, 64, dt, 51)
    off = np.where(np.arange(n) < lead, 0.0, -8.0)
    k = directed(b, off)
    v = f32(b.value, dt) * np.float32(2.0 ** -3 if dt == "f16" else 2.0 ** -9)
    v[:lead] = 0.0
    write_values(b, v, k)
    for part in (0, 4096, 128):
        out = b.run(part)
        check(b, out)
        assert out.abs().max() > 0


@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_small_values_beside_a_large_row_of_no_weight(dt, G):
    """A value row of thousands whose softmax weight is e^-40, first or last, beside rows a
    millionth as large and smaller: the large row's scale must not cost the small ones their weights' bits."""
    for place in (0, 40, 89):
        b = Batch([90], G, 1, 128, dt, 52)
        off = np.zeros(90)
        off[place] = -40.0
        k = directed(b, off)
        small, ratio = (-8, 22) if dt == "f16" else (-13, 28)
        v = f32(b.value, dt) * np.float32(2.0 ** small)
        v[place] *= np.float32(2.0 ** ratio)
        write_values(b, v, k)
        for part in (0, 32):
            check(b, b.run(part))


def test_references_at_both_ends():
    """Constant rows alone, constant rows of far higher scores after others, scores that rise by
    hundreds, and the smallest scale a row can have."""
    b = Batch([256], 2, 1, 64, "bf16", 53)
    for off, rows in ((np.zeros(256), slice(0, 256)), (np.arange(256) * 3.0, slice(64, 128)),
                      (np.arange(256) * -3.0, slice(0, 64)),
                      (np.where(np.arange(256) < 128, 0.0, 300.0), slice(128, 256))):
        k = directed(b, off)
        v = f32(b.value, "bf16").copy()
        v[rows] = 0.5
        write_values(b, v, k)
        check(b, b.run())
        v[:] = 2.0 ** -24 * np.random.default_rng(1).integers(-7, 9, v.shape)
        write_values(b, v, k)
        assert params(b.vc.cpu().numpy())[b.tables[0], 0, :, 0].max() <= 2.0 ** -23
        check(b, b.run())


@pytest.mark.parametrize("dt,G", [("f16", 1), ("f16", 8), ("bf16", 4)])
@pytest.mark.parametrize("part", [65536, 8192, 0])
def test_long_tail_beside_large_rows(dt, G, part):
    """65536 tokens of equal weights: a row thousands of times as large as the others at the front,
    its negative at the end, and what is left, a mean of all the small ones, must not be cut at
    the large row's size all the way."""
    n = 65536
    b = Batch([n], G, 1, 128, dt, 54)
    b.q = np.zeros_like(b.q)
    b.qd = dev16(b.q, dt)
    v = f32(b.value, dt) * np.float32(0.25)
    v[:32] = v[-32:] = 0.0                      # no others in the large rows' steps
    v[0] = np.random.default_rng(2).uniform(-4000, 4000, 128)
    v[-1] = -v[0]
    write_values(b, v)
    check(b, b.run(part))


@pytest.mark.parametrize("G", [1, 4, 8])
def test_means_are_as_good_as_half(G):
    """131072 tokens with scores of unit variance: the outputs, a 140th of a value, take no more
    error from weights and sums than a quarter of half precision's half step, beside the rounding
    itself (which the reference tells exactly). Sums of 32 bits rounded to nearest leave 2^-21."""
    b = Batch([131072], G, 1, 128, "f16", 43)
    got = out_to_f64(b.run(2048)[0], "f16")
    err, rounding, norm = 0.0, 0.0, 0.0
    for h in range(G):
        q, k, v, _, _ = rows_of(b, 0, h)
        ref = I4.softmax_attention(q, k, v, b.scale)
        err += ((got[h] - ref) ** 2).sum()
        rounding += ((ref.astype(np.float16) - ref) ** 2).sum()
        norm += (ref ** 2).sum()
    assert err <= rounding + 2.0 ** -26 * norm, ((err / norm) ** 0.5, (rounding / norm) ** 0.5)
