"""One split-KV workspace for calls of different sizes, zero-filled once: batches that grow and
shrink, every merge (by a sequence's last CTA, and in a second launch over warps' or over CTAs'
partitions), every cache type, and an executor whose batch grows over contexts that split.

Every call has to give the bits that it gives on a workspace of its own (results depend on logical
positions alone), and to leave zeros where another size's merge counters lie: a split batch of U
(sequence, KV head) pairs needs at least 532 U bytes, 4 of them for the pair's counter, so counters
lie in the first 1/133 of a buffer."""

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from tests.test_gpu_int4 import Batch, caches, check_decode, dev16
from workloads import gen

pytestmark = pytest.mark.gpu

# (contexts, partition_tokens): growing and shrinking numbers of sequences; with 4 KV heads the
# third and the sixth merge in a second launch
SIZES = [
    ([900, 1500, 33], 64), ([700] * 40 + [65, 64, 1, 0], 512), ([1024] * 64, 64),
    ([600] * 70, 512), ([1100], 16), ([1040, 1024, 5, 0, 1030, 1040, 17, 900], 16),
    ([530] * 90, 512), ([2000, 64, 65], 32), ([513] * 130, 512), ([100] * 3, 0), ([1500] * 20, 0)]


def _sizes(G, hkv, d):
    return max(pa.pa_paged_decode_workspace_size(len(c), G * hkv, hkv, d, max(c), 16, p)
               for c, p in SIZES)


class Plain:
    """A seeded batch over a 16-bit or an E4M3 cache."""

    def __init__(self, ctx, hq, hkv, d, fp8, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        blocks = [-(-int(c) // 16) for c in ctx]
        nb = sum(blocks) + 1
        perm = torch.randperm(nb, generator=g, device="cuda").int()
        self.t = torch.full((len(ctx), max(blocks)), -1, dtype=torch.int32, device="cuda")
        used = 0
        for s, n in enumerate(blocks):
            self.t[s, :n] = perm[used:used + n]
            used += n
        shape = (nb, hkv, 16, d)
        if fp8:
            self.kc, self.vc = (torch.randint(0, 120, shape, generator=g, device="cuda").byte()
                                for _ in range(2))
        else:
            self.kc, self.vc = (torch.randn(shape, generator=g, device="cuda").bfloat16()
                                for _ in range(2))
        self.q = torch.randn(len(ctx), hq, d, generator=g, device="cuda").bfloat16()
        self.c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.max_ctx, self.fp8 = max(ctx), fp8

    def run(self, part, ws):
        out = torch.full_like(self.q, float("nan"))
        if self.fp8:
            pa.pa_paged_decode_fp8(out, self.q, self.kc, self.vc, self.t, self.c, self.max_ctx,
                                   0.01, 0.02, 0.02, part, ws)
        else:
            pa.pa_paged_decode(out, self.q, self.kc, self.vc, self.t, self.c, self.max_ctx, 0.09,
                               part, ws)
        return out


def _own(ctx, G, hkv, d, max_ctx, part):
    return pa.decode_workspace(len(ctx), G * hkv, hkv, d, max_ctx, part)


@pytest.mark.parametrize("spare", [0, 1 << 20])
@pytest.mark.parametrize("kind,G,d", [("int4", 1, 64), ("int4", 8, 128), ("bf16", 2, 64),
                                      ("bf16", 8, 128), ("fp8", 4, 64), ("fp8", 1, 128)])
def test_batches_of_other_sizes(kind, G, d, spare):
    hkv = 4
    ws = torch.zeros(_sizes(G, hkv, d) + spare, dtype=torch.uint8, device="cuda")
    order = list(range(len(SIZES))) + [0, 8, 1, 2, 8, 5, 6]
    for step, i in enumerate(order):
        ctx, part = SIZES[i]
        if kind == "int4":
            b = Batch(ctx, G * hkv, hkv, d, "f16", 100 + i)
            got = b.run(part, ws=ws)
            want = b.run(part, ws=_own(ctx, G, hkv, d, b.max_ctx, part))
        else:
            b = Plain(ctx, G * hkv, hkv, d, kind == "fp8", 100 + i)
            got, want = b.run(part, ws), b.run(part, _own(ctx, G, hkv, d, b.max_ctx, part))
        assert bool(torch.isfinite(want).all())
        same = (got == want).flatten(1).all(1)
        assert bool(same.all()), (step, i, torch.nonzero(~same).flatten().tolist())
        assert not ws[:ws.numel() // 133].any(), (step, i)
        if kind == "int4" and step < len(SIZES) and sum(ctx) < 20000:
            b.check(got, rows=[0, len(ctx) // 2, len(ctx) - 1])


def test_types_share_a_workspace():
    """The same buffer under decodes of different caches, heads and dimensions in turn."""
    shapes = [("int4", 8, 128), ("bf16", 2, 64), ("fp8", 4, 128), ("int4", 1, 64)]
    ws = torch.zeros(max(_sizes(G, 4, d) for _, G, d in shapes), dtype=torch.uint8, device="cuda")
    for i in (5, 0, 8, 2, 3):
        for kind, G, d in shapes:
            ctx, part = SIZES[i]
            b = Batch(ctx, G * 4, 4, d, "f16", 7) if kind == "int4" else \
                Plain(ctx, G * 4, 4, d, kind == "fp8", 7)
            got = b.run(part, ws=ws)
            assert torch.equal(got, b.run(part, ws=_own(ctx, G, 4, d, b.max_ctx, part))), (i, kind)


def test_executor_over_a_4_bit_cache_with_split_contexts():
    """A batch that grows from one sequence to dozens while contexts pass 512 tokens, so that
    nearly every step merges partitions with other counters than the one before."""
    hq, hkv, d, dt, nb, cap = 8, 4, 64, "f16", 1500, 40
    c = pa.Scheduler(nb, 16, np.arange(nb), max_num_seqs=cap)
    rng = np.random.default_rng(5)
    trace = [(i, int(rng.integers(480, 800)), int(rng.integers(4, 30)), 1, i // 3)
             for i in range(40)]
    for t in trace:
        c.submit(*t)
    c.attach(hq, hkv, d, torch.float16, 900, int4=True)
    kc, vc = caches(nb, hkv, d, 0)
    toks = gen.RequestTokens(63, {t[0]: t[1] for t in trace}, hkv, d, dt,
                             prompt_tokens={t[0]: None for t in trace})
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    widest = split = step = 0
    while not c.idle():
        c.step()
        p = c.plan()

        def rows(ws):
            got = [toks.row(r, s, pos) for r, s, pos, _ in ws]
            pick = lambda i: np.array([x[i] for x in got], np.uint16).reshape(-1, hkv, d)
            return pick(0), pick(1)

        (pk, pv), (wk, wv) = rows(p["prefill"]), rows(p["writes"])
        n = len(p["batch"])
        q = gen.normal_bits([64, step], (n, hq, d), dt)
        out = torch.full((n, hq, d), float("nan"), dtype=torch.float16, device="cuda")
        c.execute(kc, vc, None, None, dev16(pk, dt), dev16(pv, dt), dev16(wk, dt), dev16(wv, dt),
                  dev16(q, dt), out, 0.125, dev_error=err)
        ctx = [int(x[2]) for x in p["batch"]]
        tables = torch.from_numpy(np.asarray(p["tables"], np.int32)).cuda()
        want = torch.full_like(out, float("nan"))
        if n:
            pa.pa_paged_decode_int4(want, dev16(q, dt), kc, vc, tables,
                                    torch.tensor(ctx, dtype=torch.int32, device="cuda"), max(ctx),
                                    0.125, workspace=pa.decode_workspace(n, hq, hkv, d, max(ctx)),
                                    seq_order=torch.from_numpy(
                                        pa.pa_longest_first_order(ctx)).cuda())
            same = (out == want).flatten(1).all(1)
            assert bool(same.all()), (step, n, torch.nonzero(~same).flatten().tolist())
            if step % 8 == 0:
                check_decode(out, q, kc.cpu().numpy(), vc.cpu().numpy(), np.asarray(p["tables"]),
                             ctx, 0.125, dt, rows=[0, n // 2, n - 1])
        widest, split = max(widest, n), split + (n > 0 and max(ctx) > 512)
        step += 1
    assert err.item() == 0 and widest > 25 and split > 20, (widest, split)
