"""Rotary writes and the 4-bit cache without a GPU: the oracles pinned to the format's and the
rotation's definitions, the host table, and the host-side refusals of the C interface."""

import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from oracle import int4 as I4
from oracle import rope as R
from paged_kv_cache_352_b200 import _lib as L

FAKE = ctypes.c_void_p(4096)   # never dereferenced: every call fails validation first
ODD = ctypes.c_void_p(4104)    # 8-byte aligned only


# ---- the oracles ---------------------------------------------------------------------

def test_code_places_cover_a_tile_once():
    for d in (64, 128):
        for values in (False, True):
            places = {I4.code_place(d, t, x, values) for t in range(16) for x in range(d)}
            assert len(places) == 16 * d and max(b for b, _ in places) == 8 * d - 1


def test_value_places_by_hand():
    # d = 128: a 16-byte chunk holds 16 dimensions of a token pair, four dimensions a word,
    # token 2p in its low half; chunks go by (pair / 4, dimensions / 16, pair % 4)
    assert I4.code_place(128, 0, 0, True) == (0, 0)
    assert I4.code_place(128, 0, 1, True) == (0, 1)
    assert I4.code_place(128, 1, 2, True) == (3, 0)
    assert I4.code_place(128, 0, 4, True) == (4, 0)
    assert I4.code_place(128, 2, 0, True) == (16, 0)
    assert I4.code_place(128, 8, 0, True) == (512, 0)
    assert I4.code_place(128, 0, 16, True) == (64, 0)
    assert I4.code_place(64, 0, 8, True) == (32, 0)
    assert I4.code_place(64, 15, 63, True) == (511, 1)
    assert I4.code_place(64, 3, 10, False) == (101, 0)


def test_quantize_row_by_hand():
    n, s, m = I4.quantize_row(np.arange(16, dtype=np.float32))       # exact: 0 .. 15
    assert (s, m) == (1.0, 7.5) and list(n) == list(range(16))
    n, s, m = I4.quantize_row(np.full(8, -3.0, np.float32))
    assert (s, m) == (0.0, -3.0)
    n, s, m = I4.quantize_row(np.array([np.inf, -np.inf, 0], np.float32))
    assert m == 0 and s == np.float16(2 * 65504 / 15) and list(n[:2]) == [15, 0]
    n, s, m = I4.quantize_row(np.array([1, np.nan], np.float32))
    assert np.isnan(s) and np.isnan(m) and not n.any()


def test_quantization_error_is_half_a_step():
    x = np.random.default_rng(0).standard_normal((200, 64)).astype(np.float32)
    for row in x:
        n, s, m = I4.quantize_row(row)
        back = float(m) + (n - 7.5) * float(s)
        # half a step inside; the ends may miss by what rounding scale and mid moved them
        assert np.abs(back - row).max() <= 0.5 * float(s) * (1 + 2e-3) + 8 * 2.0 ** -11 * abs(
            row).max()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_against_complex_products(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 64)).astype(np.float32)
    pos = [0, 1, 7, 99, 255]
    tab = R.table(256, 32, 10000.0)
    y = R.rotate(x, tab, pos, interleaved)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0], x[0])
    lo, hi = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    f = 10000.0 ** (-np.arange(16) * 2.0 / 32)
    w = np.exp(1j * np.outer(pos, f))[:, None]
    z = (x[..., lo].astype(float) + 1j * x[..., hi]) * w
    # three fp32 roundings of products up to |x|, and the table's own
    assert np.abs(y[..., lo] - z.real).max() < 8 * 2.0 ** -24 * np.abs(x).max()
    assert np.abs(y[..., hi] - z.imag).max() < 8 * 2.0 ** -24 * np.abs(x).max()


def test_rope_table_matches_the_oracle():
    for rot, theta in ((16, 10000.0), (128, 500000.0), (48, 100.0)):
        a, b = pa.pa_rope_table(70, rot, theta), R.table(70, rot, theta)
        # both are double computations of angles up to 69, rounded to fp32
        assert np.abs(a - b).max() <= 2.0 ** -24
    assert pa.pa_rope_table(0, 16).shape == (0, 16)
    for bad in ((5, 24, 1e4), (5, 0, 1e4), (5, 144, 1e4)):
        with pytest.raises(pa.PAError) as e:
            pa.pa_rope_table(*bad)
        assert e.value.code == L.PA_ERR_UNSUPPORTED
    for theta in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(pa.PAError):
            pa.pa_rope_table(5, 16, theta)


# ---- host-side refusals ---------------------------------------------------------------

def rope(lib, name="pa_rope_and_cache", **kw):
    a = dict(q_out=FAKE, q=FAKE, key=FAKE, value=FAKE, sqo=512, sq=512, sk=256, sv=256, pos=FAKE,
             table=FAKE, P=100, rot=64, inter=0, kc=FAKE, vc=FAKE, slots=FAKE, T=4, hq=4, hkv=2,
             d=128, bs=16, nb=8, dt=L.PA_F16)
    a.update(kw)
    extra = (kw.pop("ks", 1.0), a.pop("vs", 1.0)) if name.endswith("fp8") else ()
    a.pop("ks", None)
    return getattr(lib, name)(*a.values(), *extra, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), L.PA_ERR_UNSUPPORTED), (dict(bs=32), L.PA_ERR_UNSUPPORTED),
    (dict(dt=L.PA_FP8_E4M3), L.PA_ERR_UNSUPPORTED), (dict(dt=L.PA_INT4), L.PA_ERR_UNSUPPORTED),
    (dict(rot=24), L.PA_ERR_UNSUPPORTED), (dict(rot=0), L.PA_ERR_UNSUPPORTED),
    (dict(rot=144), L.PA_ERR_UNSUPPORTED), (dict(rot=80, d=64, sq=256, sqo=256),
                                            L.PA_ERR_UNSUPPORTED),
    (dict(inter=2), L.PA_ERR_INVALID_ARG), (dict(P=0), L.PA_ERR_INVALID_ARG),
    (dict(hq=0), L.PA_ERR_INVALID_ARG), (dict(hkv=0), L.PA_ERR_INVALID_ARG),
    (dict(nb=0), L.PA_ERR_INVALID_ARG), (dict(T=-1), L.PA_ERR_INVALID_ARG),
    (dict(sq=504), L.PA_ERR_INVALID_ARG), (dict(sqo=516), L.PA_ERR_INVALID_ARG),
    (dict(sk=248), L.PA_ERR_INVALID_ARG), (dict(sv=260), L.PA_ERR_INVALID_ARG),
    (dict(q_out=None), L.PA_ERR_INVALID_ARG), (dict(pos=None), L.PA_ERR_INVALID_ARG),
    (dict(table=None), L.PA_ERR_INVALID_ARG), (dict(key=None), L.PA_ERR_INVALID_ARG),
    (dict(vc=None), L.PA_ERR_INVALID_ARG), (dict(slots=None), L.PA_ERR_INVALID_ARG),
    (dict(q=ODD), L.PA_ERR_INVALID_ARG), (dict(table=ODD), L.PA_ERR_INVALID_ARG),
    (dict(value=ODD), L.PA_ERR_INVALID_ARG), (dict(kc=ODD), L.PA_ERR_INVALID_ARG),
    (dict(sqo=520), L.PA_ERR_INVALID_ARG),           # in place with other strides
])
@pytest.mark.parametrize("name", ["pa_rope_and_cache", "pa_rope_and_cache_fp8",
                                  "pa_rope_and_cache_int4"])
def test_rope_refusals(name, kw, code):
    assert rope(L.lib(), name, **kw) == code and L.last_error()


def test_rope_fp8_scales_and_empty():
    for bad in (0.0, -1.0, math.nan, math.inf):
        st = L.lib().pa_rope_and_cache_fp8(
            FAKE, FAKE, FAKE, FAKE, 512, 512, 256, 256, FAKE, FAKE, 100, 64, 0, FAKE, FAKE, FAKE, 4,
            4, 2, 128, 16, 8, L.PA_F16, bad, 1.0, None, None)
        assert st == L.PA_ERR_INVALID_ARG and "k_scale" in L.last_error()
    assert rope(L.lib(), T=0, q=None, key=None) == L.PA_OK


@pytest.mark.parametrize("name", ["pa_reshape_and_cache_int4", "pa_read_slots_int4"])
def test_int4_row_calls_refuse(name):
    f = getattr(L.lib(), name)
    base = [FAKE, FAKE, 256, 256, FAKE, FAKE, FAKE, 4, 2, 128, 16, 8, L.PA_F16, None, None]

    def st(**kw):
        a = list(base)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert st(_9=96) == L.PA_ERR_UNSUPPORTED and st(_10=8) == L.PA_ERR_UNSUPPORTED
    assert st(_12=L.PA_INT4) == L.PA_ERR_UNSUPPORTED
    for kw in (dict(_0=None), dict(_5=None), dict(_6=None), dict(_2=248), dict(_3=258),
               dict(_0=ODD), dict(_4=ODD), dict(_7=-1), dict(_8=0), dict(_11=0)):
        assert st(**kw) == L.PA_ERR_INVALID_ARG, kw
    assert st(_7=0, _0=None) == L.PA_OK


def test_int4_decode_refuses():
    f = L.lib().pa_paged_decode_int4
    base = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, None, 2, 64, 8, 2, 128, 16, 32, 0.1, 0, None, 0,
            None, L.PA_F16, None]

    def st(**kw):
        a = list(base)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert st(_12=32) == L.PA_ERR_UNSUPPORTED and st(_13=32) == L.PA_ERR_UNSUPPORTED
    assert st(_10=6) == L.PA_ERR_UNSUPPORTED                       # ratio 3
    assert st(_10=7) == L.PA_ERR_INVALID_ARG
    assert st(_20=L.PA_INT4) == L.PA_ERR_UNSUPPORTED
    assert st(_16=24) == L.PA_ERR_INVALID_ARG                      # not a multiple of 16
    assert st(_16=16) == L.PA_ERR_INVALID_ARG                      # split without a workspace
    assert st(_15=float("nan")) == L.PA_ERR_INVALID_ARG
    assert st(_0=None) == L.PA_ERR_INVALID_ARG and st(_2=ODD) == L.PA_ERR_INVALID_ARG
    assert st(_14=1 << 29) == L.PA_ERR_UNSUPPORTED                 # places beyond 2^38 bytes
    assert st(_8=0) == L.PA_OK


def test_copy_blocks_takes_the_4_bit_type():
    assert L.lib().pa_copy_blocks(FAKE, FAKE, None, 0, 8, 128, 16, 64, L.PA_INT4, None) == L.PA_OK
    assert L.lib().pa_copy_blocks(FAKE, FAKE, None, 0, 8, 128, 16, 64, 4, None) == \
        L.PA_ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors_and_other_pools():
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    pool = torch.zeros(3, 2, 16, 36, dtype=torch.uint8)
    slots = torch.zeros(2, dtype=torch.int64)
    for bad in (pool, torch.zeros(3, 2, 16, 64, dtype=torch.uint8), pool.view(torch.int8)):
        with pytest.raises(pa.PAError) as e:
            pa.pa_reshape_and_cache_int4(x, x, bad, bad, slots)
        assert e.value.code in (L.PA_ERR_INVALID_ARG, L.PA_ERR_UNSUPPORTED)
    with pytest.raises(pa.PAError):
        pa.pa_read_slots_int4(x[:, :1], x, pool, pool, slots)


@pytest.mark.parametrize("last", [64, 128])
def test_swap_refuses_pools_of_other_formats(last):
    """An 8-bit and a 4-bit pool of one head_dim are both bytes, with blocks of other sizes."""
    codes = torch.zeros(3, 2, 16, last, dtype=torch.uint8)
    int4 = torch.zeros(3, 2, 16, last // 2 + 4, dtype=torch.uint8)
    for src, dst in ((codes, int4), (int4, codes)):
        with pytest.raises(pa.PAError, match="differ in layout"):
            pa.pa_swap_blocks(src, src, dst, dst, [(0, 1)])


def test_scheduler_refuses_4_bit_pools_of_other_sizes():
    s = pa.Scheduler(4, 16, num_host_blocks=2)
    # what attach() leaves: it allocates on the device, which this test does without
    s.int4, s.fp8, s._int4_pool = True, False, (2, 16, 64)
    pool = lambda n, h, d: torch.zeros(n, h, 16, d // 2 + 4, dtype=torch.uint8)
    x = torch.zeros(1, 2, 64, dtype=torch.float16)
    run = lambda k, hk: s.execute(k, k, hk, hk, None, None, x, x, x, x, 1.0)
    for k, hk in ((pool(3, 2, 64), None), (pool(4, 1, 64), None), (pool(4, 2, 128), None),
                  (pool(4, 2, 64), pool(1, 2, 64)), (pool(4, 2, 64), pool(2, 2, 128))):
        with pytest.raises(pa.PAError, match="attached sizes"):
            run(k, hk)
