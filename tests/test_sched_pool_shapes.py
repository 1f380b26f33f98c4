"""The executor's pools: 16- and 8-bit ones are taken in any shape of the right type (a flat buffer,
K and V of different numbers of blocks), 4-bit ones in the attached shape alone."""

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa

HQ, HKV, D, NB = 4, 2, 64, 12


def _refusal(s, k, v):
    with pytest.raises(pa.PAError) as e:
        s.execute(k, v, None, None, *[torch.zeros(1, HKV, D, dtype=torch.float16)] * 4,
                  *[torch.zeros(1, HQ, D, dtype=torch.float16)] * 2, 0.1)
    return str(e.value)


def test_shapes_are_not_what_is_refused():
    """Without a GPU the first refusal of a good pool is that it is not CUDA memory."""
    for dt, fp8 in ((torch.float16, False), (torch.uint8, True)):
        s = pa.Scheduler(NB, 16, np.arange(NB), max_num_seqs=2)
        s.fp8 = fp8
        pool = torch.zeros(NB, HKV, 16, D, dtype=dt)
        for k, v in ((pool, pool), (pool.view(-1), pool.view(-1)), (pool, pool[:9]),
                     (pool.view(NB, -1), pool)):
            assert "CUDA" in _refusal(s, k, v)
        assert "element type" in _refusal(s, pool.to(torch.bfloat16) if fp8 else pool.byte(), pool)
        four = torch.zeros(NB, HKV, 16, D // 2 + 4, dtype=torch.uint8)
        assert "element type" in _refusal(s, four, four)


@pytest.mark.gpu
def test_a_flat_pool_runs_as_its_blocks():
    outs = []
    for flat in (False, True):
        s = pa.Scheduler(NB, 16, np.arange(NB), max_num_seqs=2)
        s.submit(0, 37, 3, 1, 0)
        s.attach(HQ, HKV, D, torch.float16, 64)
        pool = [torch.zeros(NB, HKV, 16, D, dtype=torch.float16, device="cuda") for _ in range(2)]
        g = torch.Generator(device="cuda").manual_seed(1)
        rows = lambda n, h: torch.randn(n, h, D, generator=g, device="cuda").half()
        got = []
        while not s.idle():
            s.step()
            p = s.plan()
            n = len(p["batch"])
            out = torch.zeros(n, HQ, D, dtype=torch.float16, device="cuda")
            k, v = (x.view(-1) if flat else x for x in pool)
            s.execute(k, v, None, None, rows(len(p["prefill"]), HKV), rows(len(p["prefill"]), HKV),
                      rows(len(p["writes"]), HKV), rows(len(p["writes"]), HKV), rows(n, HQ), out,
                      0.125)
            got.append(out)
        outs.append(torch.cat(got))
    assert outs[0].abs().sum() > 0 and torch.equal(*outs)
