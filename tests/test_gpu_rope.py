"""Rotary cache writes on a B200 against the oracle, bit for bit: the rotation is
defined operation by operation in fp32 and rounded once per stored element, so
queries, 16-bit caches, E4M3 codes and 4-bit rows all have to match exactly."""

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from oracle import fp8 as F8
from oracle import int4 as I4
from oracle import rope as R
from oracle.fpbits import bits_to_f64
from tests.parity import tensor_bits
from workloads import gen

pytestmark = pytest.mark.gpu

TDT = {"f16": torch.float16, "bf16": torch.bfloat16}
SCALES = (0.03, 0.02)


def dev16(bits, dt):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(TDT[dt]).cuda()


def to_bits(x, dt):
    return gen.f32_to_bits(x, dt)


class Case:
    def __init__(self, T, hq, hkv, d, rot, interleaved, dt, cache, seed=0, positions=None):
        self.T, self.hq, self.hkv, self.d, self.dt, self.cache = T, hq, hkv, d, dt, cache
        self.interleaved = interleaved
        self.q = gen.normal_bits([seed, 1], (T, hq, d), dt)
        self.k = gen.normal_bits([seed, 2], (T, hkv, d), dt)
        self.v = gen.normal_bits([seed, 3], (T, hkv, d), dt)
        self.nb = -(-T // 16) + 2
        rng = np.random.default_rng([seed, 4])
        self.slots = rng.permutation(self.nb * 16)[:T].astype(np.int64)
        self.P = 300
        self.pos = rng.integers(0, self.P, T) if positions is None else np.asarray(positions)
        self.table = pa.pa_rope_table(self.P, rot, 10000.0)
        self.fill = 0x5A
        if cache == "int4":
            self.kc = torch.full((self.nb, hkv, 16, d // 2 + 4), self.fill, dtype=torch.uint8,
                                 device="cuda")
        elif cache == "e4m3":
            self.kc = torch.full((self.nb, hkv, 16, d), self.fill, dtype=torch.uint8, device="cuda")
        else:
            self.kc = torch.full((self.nb, hkv, 16, 2 * d), self.fill, dtype=torch.uint8,
                                 device="cuda").view(TDT[dt])
        self.vc = self.kc.clone()

    def call(self, q=None, q_out=None, key=None, value=None, err=None, stream=None):
        q = dev16(self.q, self.dt) if q is None else q
        q_out = torch.empty_like(q) if q_out is None else q_out
        key = dev16(self.k, self.dt) if key is None else key
        value = dev16(self.v, self.dt) if value is None else value
        a = [q_out, q, key, value, torch.from_numpy(self.pos.astype(np.int64)).cuda(),
             torch.from_numpy(self.table).cuda(), self.kc, self.vc,
             torch.from_numpy(self.slots).cuda()]
        kw = dict(interleaved=self.interleaved, dev_error=err, stream=stream)
        if self.cache == "int4":
            pa.pa_rope_and_cache_int4(*a, **kw)
        elif self.cache == "e4m3":
            pa.pa_rope_and_cache_fp8(*a, *SCALES, **kw)
        else:
            pa.pa_rope_and_cache(*a, **kw)
        return q_out

    def check(self, q_out, skip=()):
        """skip: tokens whose position was refused (nothing of them is written)."""
        live = np.array([t for t in range(self.T) if t not in skip], int)
        f = lambda b: bits_to_f64(b, self.dt).astype(np.float32)
        rot = lambda b: R.rotate(f(b[live]), self.table, self.pos[live], self.interleaved)
        got = tensor_bits(q_out)
        assert np.array_equal(got[live], to_bits(rot(self.q), self.dt))
        k, v = rot(self.k), f(self.v[live])
        slots = np.where(self.slots >= self.nb * 16, -1, self.slots)[live]
        if self.cache == "int4":
            ek = np.full(self.kc.shape, self.fill, np.uint8)
            ev = ek.copy()
            I4.reshape_and_cache_int4(ek, ev, k, v, slots)
        elif self.cache == "e4m3":
            ek = np.full(self.kc.shape, self.fill, np.uint8)
            ev = ek.copy()
            for t, s in enumerate(slots):
                if s >= 0:
                    ek[s // 16, :, s % 16] = F8.encode_e4m3_array(k[t] / np.float32(SCALES[0]))
                    ev[s // 16, :, s % 16] = F8.encode_e4m3_array(v[t] / np.float32(SCALES[1]))
        else:
            ek = np.full(self.kc.shape, 0x5A5A, np.uint16)
            ev = ek.copy()
            for t, s in enumerate(slots):
                if s >= 0:
                    ek[s // 16, :, s % 16] = to_bits(k[t], self.dt)
                    ev[s // 16, :, s % 16] = self.v[live[t]]
        raw = (lambda x: x.cpu().numpy()) if self.cache != "same" else tensor_bits
        assert np.array_equal(raw(self.kc), ek)
        assert np.array_equal(raw(self.vc), ev)


@pytest.mark.parametrize("cache", ["same", "e4m3", "int4"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 48), (128, 128), (128, 32), (128, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_and_write(cache, dt, d, rot, interleaved):
    c = Case(21, 6, 3, d, rot, interleaved, dt, cache, seed=d + rot)
    c.check(c.call())


@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (1, 32, 8), (2, 5, 3), (17, 64, 1), (333, 7, 2)])
@pytest.mark.parametrize("cache", ["same", "int4"])
def test_token_counts_and_heads(T, hq, hkv, cache):
    """One token over many warps, one warp over a token's rows, head counts that end inside a
    warp's row group."""
    c = Case(T, hq, hkv, 128, 128, False, "bf16", cache, seed=T)
    c.check(c.call())


def test_many_tokens():
    """Enough tokens that a warp keeps all rows of a token."""
    c = Case(2500, 3, 1, 64, 64, False, "f16", "e4m3", seed=5)
    c.check(c.call())


def test_in_place_and_strides():
    """q_out is q, and the rows come out of one fused projection."""
    c = Case(40, 4, 2, 64, 64, False, "f16", "int4", seed=6)
    wide = torch.cat([dev16(x, "f16") for x in (c.q, c.k, c.v)], 1)
    q, k, v = wide[:, :4], wide[:, 4:6], wide[:, 6:]
    out = c.call(q=q, q_out=q, key=k, value=v)
    assert out.data_ptr() == wide.data_ptr()
    c.check(out)
    assert np.array_equal(tensor_bits(k), c.k) and np.array_equal(tensor_bits(v), c.v)
    one = Case(1, 4, 2, 64, 64, False, "f16", "same", seed=7)
    one.check(one.call(q=dev16(one.q, "f16")[:, :].expand(1, 4, 64)))


def test_slots_and_positions_out_of_range():
    c = Case(30, 4, 2, 64, 32, True, "bf16", "same", seed=8)
    c.slots[3], c.slots[9], c.slots[11] = -1, c.nb * 16, 1 << 50
    c.pos[[5, 9, 20]] = [-1, c.P, 1 << 40]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = dev16(c.q, "bf16")
    q_out = torch.full_like(q, 3.0)
    c.call(q=q, q_out=q_out, err=err)
    assert err.item() == pa.PA_DEVERR_SLOT_RANGE | pa.PA_DEVERR_POSITION
    c.check(q_out, skip=(5, 9, 20))
    assert bool((q_out[[5, 9, 20]] == 3).all())


def test_special_values():
    """Infinities and NaN pass through the rotation as IEEE arithmetic has it; elements past
    rotary_dim and values keep their bits."""
    c = Case(4, 2, 1, 64, 32, False, "f16", "same", seed=9)
    c.k[0, 0, 3], c.k[1, 0, 40], c.v[2, 0, 5], c.q[3, 1, 50] = 0x7C00, 0x7E00, 0x7E55, 0xFC00
    q_out = c.call()
    k = tensor_bits(c.kc)
    at = lambda t: (c.slots[t] // 16, 0, c.slots[t] % 16)
    x = bits_to_f64(k[at(0)], "f16")
    with np.errstate(invalid="ignore"):
        want = R.rotate(bits_to_f64(c.k[:1], "f16").astype(np.float32), c.table, c.pos[:1], False)
    assert np.array_equal(x, want[0, 0].astype(np.float16).astype(np.float64), equal_nan=True)
    assert not np.isfinite(x[3]) and not np.isfinite(x[19])
    assert k[at(1)][40] == 0x7E00 and tensor_bits(c.vc)[at(2)][5] == 0x7E55
    assert tensor_bits(q_out)[3, 1, 50] == 0xFC00


def test_stream_and_graph():
    c = Case(64, 8, 2, 128, 128, False, "bf16", "int4", seed=10)
    q, k, v = (dev16(x, "bf16") for x in (c.q, c.k, c.v))
    q_out = torch.empty_like(q)
    a = (q_out, q, k, v, torch.from_numpy(c.pos).cuda(), torch.from_numpy(c.table).cuda(), c.kc,
         c.vc, torch.from_numpy(c.slots).cuda())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_rope_and_cache_int4(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    c.check(q_out)


def test_far_positions():
    """Angles of positions up to a million: the table is computed in double precision."""
    P = 1 << 20
    t = pa.pa_rope_table(P, 32, 500000.0)
    for p in (0, 1, 65535, P - 1):
        f = 500000.0 ** (-np.arange(16) * 2.0 / 32)
        want = np.concatenate([np.cos(p * f), np.sin(p * f)])
        assert np.abs(t[p] - want).max() <= 2.0 ** -24 + 1e-9
    c = Case(3, 2, 2, 64, 32, False, "f16", "same", seed=12, positions=[0, 65535, P - 1])
    c.table = t
    c.check(c.call())


def test_refusals_on_device_tensors():
    c = Case(4, 2, 2, 64, 64, False, "f16", "same", seed=13)
    q, k, v = (dev16(x, "f16") for x in (c.q, c.k, c.v))
    pos, tab = torch.from_numpy(c.pos).cuda(), torch.from_numpy(c.table).cuda()
    slots = torch.from_numpy(c.slots).cuda()
    good = [torch.empty_like(q), q, k, v, pos, tab, c.kc, c.vc, slots]

    def refused(i, x):
        a = list(good)
        a[i] = x
        with pytest.raises(pa.PAError):
            pa.pa_rope_and_cache(*a)

    refused(0, torch.empty_like(q, dtype=torch.bfloat16))
    refused(0, torch.empty(4, 3, 64, dtype=torch.float16, device="cuda"))
    refused(4, pos.int())
    refused(4, pos[:3])
    refused(5, tab[:, :24].contiguous())           # not a multiple of 16
    refused(5, tab.half())
    refused(5, torch.zeros(10, 80, device="cuda"))  # wider than the head
    refused(6, c.kc.bfloat16())
    refused(8, slots.int())
    refused(1, q.cpu())
    refused(1, q.transpose(1, 2).contiguous().transpose(1, 2))
