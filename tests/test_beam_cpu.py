"""Beam selection and reordering without a GPU: the oracle pinned by hand, the C interface's
refusals, and pa_bm_reorder against the oracle's block manager over random streams."""

import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_352_b200 as pa
from oracle import beam as OB
from oracle import block_manager as OBM
from paged_kv_cache_352_b200 import _lib as L

FAKE = ctypes.c_void_p(4096)   # never dereferenced: every call fails validation first


def test_oracle_selection_by_hand():
    # two beams over three tokens with probabilities 1/2, 1/4, 1/4 and 1/8, 1/8, 3/4
    x = np.log(np.array([[2, 1, 1], [1, 1, 6.0]]))
    s, p, t = OB.select(x, [math.log(0.5), math.log(0.5)], 4)
    # 3/8, 1/4, then 1/8 twice: beam 0's tokens 1 and 2 tie, the lower index first
    assert np.allclose(np.exp(s), [3 / 8, 1 / 4, 1 / 8, 1 / 8])
    assert list(zip(p, t)) == [(1, 2), (0, 0), (0, 1), (0, 2)]
    s, p, t = OB.select(np.array([[0.0, -math.inf]]), [0.0], 3)
    assert list(s) == [0.0, -math.inf, -math.inf] and list(p) == [0, -1, -1] and t[0] == 0
    s, p, t = OB.select(np.array([[0.0, math.nan], [1.0, 1.0]]), [0.0, -1.0], 2)
    assert list(p) == [1, 1] and OB.all_scores(np.array([[0.0, math.nan]]), [0.0])[1]


def test_selection_refusals():
    f = L.lib().pa_beam_select
    base = [FAKE, FAKE, FAKE, FAKE, 1000, FAKE, 2, 4, 1000, 8, FAKE, 1 << 30, None, L.PA_F32, None]

    def st(**kw):
        a = list(base)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 1, 2, 3, 5, 10):
        assert st(**{f"_{i}": None}) == L.PA_ERR_INVALID_ARG
    assert st(_4=999) == L.PA_ERR_INVALID_ARG and st(_4=1002) == L.PA_ERR_INVALID_ARG
    assert st(_4=1004, _13=L.PA_BF16) == L.PA_ERR_INVALID_ARG       # 16-byte rows: 8 halves
    assert st(_3=ctypes.c_void_p(4100)) == L.PA_ERR_INVALID_ARG
    assert st(_10=ctypes.c_void_p(4224)) == L.PA_ERR_INVALID_ARG    # workspace alignment
    assert st(_11=64) == L.PA_ERR_INVALID_ARG and "workspace" in L.last_error()
    assert st(_6=-1) == L.PA_ERR_INVALID_ARG
    for kw in (dict(_7=0), dict(_7=65), dict(_9=0), dict(_9=65), dict(_8=0), dict(_8=(1 << 24) + 1),
               dict(_13=L.PA_INT4), dict(_13=L.PA_FP8_E4M3)):
        assert st(**kw) == L.PA_ERR_UNSUPPORTED, kw
    assert st(_6=2 ** 31 - 1, _8=1 << 24) == L.PA_ERR_UNSUPPORTED   # beyond the grid
    assert st(_6=0, _0=None) == L.PA_OK


def test_workspace_size():
    n = pa.pa_beam_select_workspace_size
    base = n(0, 4, 1000, 8)                   # counters
    assert base <= 2048 and n(1, 1, 1, 1) <= base + 3 * 256   # maxima, sums, keys
    # per (row, tile): a maximum, a sum and `select` 8-byte keys; tiles of at least 2048 logits
    for b, k, v, s in ((1, 4, 32000, 8), (64, 8, 131072, 16), (7, 3, 50257, 64)):
        tiles = -(-v // 2048)
        assert 0 < n(b, k, v, s) <= b * k * tiles * (8 + 8 * s) + base + 3 * 256
    with pytest.raises(pa.PAError):
        n(1, 65, 10, 1)
    assert L.lib().pa_beam_select_workspace_size(1, 1, 1, 1, L.PA_F32, None) == L.PA_ERR_INVALID_ARG


# ---- pa_bm_reorder -----------------------------------------------------------------------

def test_reorder_by_hand():
    bm = pa.BlockManager(8, 16)
    bm.add_seq(1, 20)              # blocks 0, 1
    bm.add_seq(2, 40)              # blocks 2, 3, 4
    bm.add_seq(3, 5)               # block 5
    bm.reorder([1, 2, 3], [1, 1, -1])
    assert bm.table(1) == bm.table(2) == [2, 3, 4] and bm.seq_len(1) == 40
    assert bm.refcount(2) == 2 and bm.refcount(5) == 1 and bm.num_free() == 4
    assert bm.free_list()[:2] == [0, 1]                 # last block released first
    bm.reorder([1, 2, 3], [2, 0, 0])                    # at once: 2 keeps what 1 was
    assert bm.table(1) == [5] and bm.table(2) == bm.table(3) == [2, 3, 4]
    slots, cow = bm.append_slots(2, 1)                  # shared, partly filled: copied
    assert len(cow) == 1 and cow[0][0] == 4
    bm.reorder([], [])


def test_reorder_refusals_change_nothing():
    bm = pa.BlockManager(8, 16)
    bm.set_host_pool(4)
    bm.add_seq(1, 20)
    bm.add_seq(2, 3)
    before = (bm.table(1), bm.table(2), bm.free_list())
    for ids, par, code in (([1, 9], [0, 0], L.PA_ERR_UNKNOWN_SEQ),
                           ([1, 1], [0, 0], L.PA_ERR_INVALID_ARG),
                           ([1, 2], [0, 2], L.PA_ERR_INVALID_ARG),
                           ([1, 2], [-2, 0], L.PA_ERR_INVALID_ARG)):
        with pytest.raises(pa.PAError) as e:
            bm.reorder(ids, par)
        assert e.value.code == code
    with pytest.raises(pa.PAError):
        bm.reorder([1, 2], [0])
    assert (bm.table(1), bm.table(2), bm.free_list()) == before
    bm.swap_out(2)
    with pytest.raises(pa.PAError) as e:
        bm.reorder([1, 2], [1, 0])
    assert e.value.code == L.PA_ERR_SEQ_SWAPPED
    assert L.lib().pa_bm_reorder(None, None, None, 1) == L.PA_ERR_INVALID_ARG
    assert L.lib().pa_bm_reorder(bm._h, None, None, 1) == L.PA_ERR_INVALID_ARG
    assert L.lib().pa_bm_reorder(bm._h, None, None, -1) == L.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("seed", range(6))
def test_reorder_matches_the_oracle(seed):
    """Random beams: appends, reorderings, frees and forks, with prefix-cached prompts among them."""
    rng = np.random.default_rng(seed)
    nb = 60
    order = rng.permutation(nb)
    c, o = pa.BlockManager(nb, 16, order), OBM.BlockManager(nb, 16, order)
    live, nid = [], 0
    prompt = rng.integers(0, 9, 48).tolist()
    for it in range(600):
        op = int(rng.integers(0, 6))
        if op == 0 or len(live) < 2:
            args = ("add_seq_cached", nid, prompt[:int(rng.integers(0, 49))])
        elif op == 1:
            args = ("fork", live[int(rng.integers(len(live)))], nid)
        elif op == 2:
            args = ("append_slots", live[int(rng.integers(len(live)))], int(rng.integers(0, 12)))
        elif op == 3 and len(live) > 6:
            args = ("free_seq", live[int(rng.integers(len(live)))])
        else:
            ids = rng.permutation(live)[:int(rng.integers(1, len(live) + 1))].tolist()
            args = ("reorder", ids, rng.integers(-1, len(ids), len(ids)).tolist())
        codes = []
        for m, err in ((o, OBM.BlockManagerError), (c, pa.PAError)):
            try:
                getattr(m, args[0])(*args[1:])
                codes.append(None)
            except err as e:
                codes.append(e.code)
        assert codes[0] == codes[1], (it, args, codes)
        if codes[0] is None:
            if args[0] in ("add_seq_cached", "fork"):
                live.append(nid)
                nid += 1
            elif args[0] == "free_seq":
                live.remove(args[1])
        assert c.free_list() == o.free_list() and c.evictable_list() == o.evictable_list()
        for s in live:
            assert c.table(s) == o.table(s) and c.seq_len(s) == o.seq_len(s)
        assert [c.refcount(b) for b in range(nb)] == [o.refcount(b) for b in range(nb)]
    for s in list(live):
        c.free_seq(s)
    assert c.num_free() == nb
