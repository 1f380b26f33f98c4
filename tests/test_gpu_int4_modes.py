"""The 4-bit decode's three ways to merge a split: by each sequence's last CTA, in a second launch
over warps' partitions, and in a second launch over CTAs' partitions cut into four."""

import pytest
import torch

import paged_kv_cache_352_b200 as pa
from tests.test_gpu_int4 import Batch, dev16

pytestmark = pytest.mark.gpu

# the three modes: (contexts, KV heads, partition)
MODES = {"last CTA": ([700, 100, 513], 2, 64), "warps": ([1024] * 64, 4, 64),
         "quartered": ([1040] * 8, 4, 16), "one partition": ([300, 20], 2, 0)}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dt,G", [("f16", 1), ("bf16", 4), ("f16", 8)])
def test_nan_and_inf_queries_show_in_every_mode(mode, dt, G):
    """A query with a NaN or an infinity gives NaN in its own row. Other KV heads and sequences
    keep their bits; heads of the same KV head share its softmax references' moves and stay
    within their own bound."""
    ctx, hkv, part = MODES[mode]
    b = Batch(ctx, G * hkv, hkv, 64, dt, 3)
    want = b.run(part)
    assert bool(torch.isfinite(want).all())
    q = b.qd.clone()
    q[0, 0, 5], q[1, G * hkv - 1, 63], q[0, G * hkv - 1] = float("nan"), float("inf"), -float("inf")
    out = b.run(part, q=q)
    bad = torch.zeros(want.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, -1] = bad[0, -1] = True
    assert bool(torch.isnan(out[bad]).all())
    shared = bad.view(len(ctx), hkv, G).any(2, keepdim=True).expand(-1, -1, G).reshape(bad.shape)
    assert torch.equal(out[~shared], want[~shared])
    out[bad] = want[bad]
    b.check(out, rows=[0, 1])


@pytest.mark.parametrize("mode", MODES)
def test_nan_rows_show_in_every_mode(mode):
    """A cached key or value with a NaN reaches the outputs that attend to it."""
    ctx, hkv, part = MODES[mode]
    for which in ("key", "value"):
        b = Batch(ctx, hkv, hkv, 64, "f16", 4)
        want = b.run(part)
        rows = getattr(b, which)
        rows[17, 0, 3] = 0x7E00                         # sequence 0, KV head 0
        slot = torch.tensor([int(b.tables[0, 1]) * 16 + 1], device="cuda")
        pa.pa_reshape_and_cache_int4(dev16(b.key[17:18], "f16"), dev16(b.value[17:18], "f16"),
                                     b.kc, b.vc, slot)
        out = b.run(part)
        assert bool(torch.isnan(out[0, 0]).all())
        assert torch.equal(out[1:], want[1:]) and torch.equal(out[0, 1:], want[0, 1:])
