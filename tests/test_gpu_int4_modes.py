"""The 4-bit decode's three ways to merge a split: by each sequence's last CTA, in a second launch
over warps' partitions, and in a second launch over CTAs' partitions cut into four."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from tests.test_gpu_int4 import Batch, dev16

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# (sequences, KV heads, longest context, partition): the second launch over CTAs' partitions takes
# fewer than 128 (sequence, KV head) pairs that give 2048 partitions and more
QUARTERED = [(8, 4, 1040, 16), (8, 4, 2100, 32), (8, 4, 3120, 48), (8, 4, 7200, 112),
             (4, 8, 5200, 80)]


def contexts(n, longest, part):
    """Long, short, empty and ragged ones."""
    ctx = [longest, 0, 1, part, part + 1, longest - 1, 16 * ((longest - part) // 16), 5 * part - 7]
    return ctx[:n]


@pytest.mark.parametrize("dt,G,d", [("f16", 1, 64), ("bf16", 8, 128), ("f16", 8, 64)])
@pytest.mark.parametrize("seqs,hkv,longest,part", QUARTERED)
def test_quartered_partitions(seqs, hkv, longest, part, dt, G, d):
    ctx = contexts(seqs, longest, part)
    b = Batch(ctx, G * hkv, hkv, d, dt, part)
    parts, launches = pa.pa_paged_decode_plan(seqs, G * hkv, hkv, d, b.max_ctx, part)[1:]
    assert seqs * hkv * parts >= 2048 and launches == 1     # the rule of the 4-bit decode alone
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.run(part, err=err)
    assert err.item() == 0
    b.check(out)
    assert torch.equal(out, b.run(part, order=True))


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


FORCED = """
import sys
import torch
import paged_kv_cache_352_b200 as pa
from tests.test_gpu_int4 import Batch
b = Batch([1040, 1033, 900, 1040, 17, 1000, 999, 1040], 16, 4, 64, "f16", 8)
out = b.run(16)
for s in range(8):
    one = torch.empty_like(out[s:s + 1])
    ws = pa.decode_workspace(1, 16, 4, 64, b.max_ctx, 16)
    pa.pa_paged_decode_int4(one, b.qd[s:s + 1].clone(), b.kc, b.vc, b.t[s:s + 1].clone(),
                            b.c[s:s + 1].clone(), b.max_ctx, b.scale, 16, ws)
    assert torch.equal(one[0], out[s]), s
print("alike")
"""


def test_forced_merge_by_the_last_cta():
    """PA_DECODE_SPLIT=cta holds for this decode too: a batch gives the bits that its sequences
    give alone, where nothing else than the merge by the last CTA is chosen."""
    env = dict(os.environ, PA_DECODE_SPLIT="cta", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", FORCED], capture_output=True, text=True, env=env,
                       cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "alike" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("seqs,hkv", [(40, 8), (159, 8), (160, 8), (161, 8), (320, 4), (256, 8)])
def test_sizes_around_the_partition_rule(seqs, hkv):
    """Longest first, partitions of the library's choice, on both sides of 1280 (sequence, KV head)
    pairs: workspaces of the plan's size hold, and the rows are the oracle's."""
    ctx = np.random.default_rng(seqs).integers(1, 60, seqs)
    ctx[[0, seqs // 2, seqs - 1]] = 5000, 4097, 2049
    b = Batch(ctx, 2 * hkv, hkv, 64, "f16", seqs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.run(0, order=True, err=err)
    assert err.item() == 0
    b.check(out, rows=[0, 1, seqs // 2, seqs - 1])
