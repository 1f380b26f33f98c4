"""Beam selection on a B200 against the oracle, and a beam search over a paged
4-bit cache: rotate and append, attend, select, reorder, copy on write.

A score's tolerance: the exponentials of a row are within 26 steps of fp32 (26 2^-23)
for terms that count (exponents above -20), a thread adds up at most 64 of them in
fp32 (64 2^-24), the rest is double precision and one rounding to float: 8e-6 +
2^-24 |score|. (Where CTAs walk many chunks a thread adds 17 steps a chunk and one for each
of at most 16 chunks, 33 2^-24; each move of its reference may add 2 2^-23, and a row of
random logits moves it a few times.) Tokens and parents have to be the oracle's, except
that candidates of different beams whose scores lie closer than that may change places."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from oracle import beam as OB
from oracle import block_manager as OBM
from oracle import int4 as I4
from oracle import rope as R
from oracle.fpbits import bits_to_f64
from tests.parity import tensor_bits

pytestmark = pytest.mark.gpu

TDT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def tol(score):
    return 8e-6 + 2.0 ** -24 * np.abs(score)


def run(logits, beam_scores, n, ws=None, err=None, stream=None):
    B, K = beam_scores.shape
    out = (torch.full((B, n), 7.0, device="cuda"),
           torch.full((B, n), 7, dtype=torch.int32, device="cuda"),
           torch.full((B, n), 7, dtype=torch.int32, device="cuda"))
    ws = pa.beam_workspace(B, K, logits.shape[1], n) if ws is None else ws
    pa.pa_beam_select(*out, logits, beam_scores, ws, err, stream)
    return out


def check(out, logits, beam_scores, n):
    B, K = beam_scores.shape
    x = logits.float().cpu().numpy().reshape(B, K, -1)
    scores, parents, tokens = (t.cpu().numpy() for t in out)
    for b in range(B):
        want = OB.select(x[b], beam_scores[b].cpu().numpy(), n)
        every, _ = OB.all_scores(x[b], beam_scores[b].cpu().numpy())
        live = want[0] > -math.inf
        assert np.array_equal(scores[b] > -math.inf, live)
        assert (parents[b][~live] == -1).all() and (tokens[b][~live] == -1).all()
        assert np.all(np.abs(scores[b][live] - want[0][live]) <= tol(want[0][live]))
        seen = set()
        for i in np.flatnonzero(live):
            got = (int(parents[b, i]), int(tokens[b, i]))
            assert got not in seen
            seen.add(got)
            if got != (want[1][i], want[2][i]):
                assert got[0] != want[1][i], (b, i, got, want[1][i], want[2][i])
                assert abs(every[got] - want[0][i]) <= 2 * tol(want[0][i])


def make(B, K, V, dt, seed, spread=3.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = 4 if dt == "f32" else 8
    width = -(-V // per) * per + pad
    x = (torch.randn(B * K, width, generator=g, device="cuda") * spread).to(TDT[dt])
    s = -torch.rand(B, K, generator=g, device="cuda") * 8
    return x[:, :V], s


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,K,V,n", [
    (1, 1, 1, 1), (2, 3, 1, 4), (3, 4, 5, 16), (1, 4, 100, 8), (2, 2, 4095, 4), (2, 2, 4096, 4),
    (1, 5, 4097, 10), (1, 4, 32000, 8), (5, 3, 50257, 7), (40, 8, 16385, 16), (3, 16, 20011, 33),
    (1, 64, 3001, 64), (300, 2, 517, 3), (2, 1, 131075, 2)])
def test_selection(dt, B, K, V, n):
    x, s = make(B, K, V, dt, B * 131 + V)
    check(run(x, s, n), x, s, n)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_ties_go_to_the_lowest_index(dt):
    """Equal logits everywhere (more ties than are ranked at once), few distinct values, beams
    that are copies of each other, and zeros of both signs."""
    for V in (4000, 40000):
        x = torch.zeros(3 * 4, V, dtype=TDT[dt], device="cuda")
        s = torch.zeros(3, 4, device="cuda")
        sc, pr, tk = run(x, s, 9)
        assert (pr == 0).all() and torch.equal(tk.cpu(), torch.arange(9).repeat(3, 1).int())
        check((sc, pr, tk), x, s, 9)
        x[:, 1::2] = -0.0
        assert torch.equal(run(x, s, 9)[2], tk)
        x, s = make(3, 4, V, dt, V)
        x = x.round().contiguous()
        check(run(x, s, 24), x, s, 24)
        x[1::4] = x[0::4]
        s[:, 1] = s[:, 0] = 0.0
        out = run(x, s, 24)
        check(out, x, s, 24)
        for b in range(3):                      # of two equal candidates the first beam's leads
            got = [(int(p), int(t)) for p, t in zip(out[1][b], out[2][b])]
            for p, t in got:
                if p == 1:
                    assert (0, t) in got and got.index((0, t)) < got.index((1, t))


def test_masks_dead_beams_and_few_candidates():
    x, s = make(6, 4, 5000, "bf16", 77)
    x = x.clone()
    x[torch.rand(x.shape, device="cuda") < 0.7] = -math.inf
    s[0, 1:] = -math.inf                       # a first step: one live beam
    s[1] = -math.inf                           # no beam left
    x[2 * 4:3 * 4] = -math.inf                 # everything masked ...
    x[2 * 4 + 1, 4321] = 1.0                   # ... but one token of beam 1
    x[3 * 4 + 2] = -math.inf                   # one beam without tokens
    x[4 * 4:5 * 4, 8:] = -math.inf             # 8 tokens a beam: fewer than select
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(x, s, 40, err=err)
    check(out, x, s, 40)
    assert err.item() == 0
    assert int((out[1][2] >= 0).sum()) == 1 and abs(out[0][2, 0] - s[2, 1]) < 1e-5


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_nan_and_inf_rows_are_refused(dt):
    x, s = make(4, 3, 9000, dt, 5)
    x = x.clone()
    x[0, 8999], x[4, 17] = math.nan, math.inf
    s[2, 1], s[3, 0] = math.nan, math.inf
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(x, s, 6, err=err)
    assert err.item() == pa.PA_DEVERR_LOGITS
    check(out, x, s, 6)
    assert 0 not in out[1][0] and 1 not in out[1][1] and 1 not in out[1][2] and 0 not in out[1][3]


def test_extreme_logits_and_scores():
    """Logits of +-60000 (a distribution of one token), rows of large equal values, scores far
    apart."""
    x, s = make(2, 3, 6000, "f16", 9)
    x = x.clone()
    x[0, 5], x[1, 7], x[2] = 60000.0, -60000.0, 60000.0
    s = torch.tensor([[0.0, -1e4, -20.0], [-1e6, -1e6, -1e-3]], device="cuda")
    check(run(x, s, 12), x, s, 12)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_masks_of_the_lowest_value(dt):
    """Tokens masked with the type's lowest value instead of -inf, a row of nothing else, one of
    the largest, and a beam score that low."""
    x, s = make(3, 3, 4500, dt, 15)
    low, top = torch.finfo(TDT[dt]).min, torch.finfo(TDT[dt]).max
    x[0:3][torch.rand(3, 4500, device="cuda") < 0.9] = low
    x[3:6] = low                               # uniform: every token at -log V
    x[6], x[7, :9] = top, top
    s[0, 1] = torch.finfo(torch.float32).min
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(x, s, 9, err=err)
    assert err.item() == 0
    check(out, x, s, 9)
    assert abs(float(out[0][1, 0] - s[1].max()) + math.log(4500)) < 1e-5


def test_padded_rows_stream_graph_and_two_calls_at_once():
    x, s = make(4, 4, 20000, "bf16", 21, pad=64)
    assert x.stride(0) == 20064
    x.as_strided((16, 64), (20064, 1), 20000).fill_(1e4)      # the padding is not part of a row
    want = run(x, s, 8)
    check(want, x, s, 8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for k in range(2):
        xk = x.clone() if k == 0 else x.flip(0).contiguous()
        sk = s if k == 0 else s.flip(0).flip(1).contiguous()
        ws = pa.beam_workspace(4, 4, 20000, 8)
        out = (torch.zeros(4, 8, device="cuda"),
               torch.zeros(4, 8, dtype=torch.int32, device="cuda"),
               torch.zeros(4, 8, dtype=torch.int32, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_beam_select(*out, xk, sk, ws)
        graphs.append((g, xk, sk, ws, out))
    for _ in range(4):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(graphs[0][4], want):
        assert torch.equal(a, b)
    check(graphs[1][4], graphs[1][1], graphs[1][2], 8)


def test_one_workspace_for_calls_of_other_sizes():
    ws = pa.beam_workspace(64, 8, 40000, 16)
    for B, K, V, n in ((1, 1, 100, 1), (64, 8, 40000, 16), (200, 1, 64, 4), (2, 4, 30000, 8),
                       (290, 1, 10, 2), (1, 64, 5000, 16), (3, 2, 100, 5), (200, 1, 64, 4)):
        x, s = make(B, K, V, "bf16", B + V)
        check(run(x, s, n, ws=ws), x, s, n)


@pytest.mark.parametrize("dt,B,K,V,n", [
    ("f16", 80, 4, 50257, 12), ("bf16", 600, 1, 24577, 5), ("f32", 24, 9, 33000, 18),
    ("bf16", 2, 64, 131080, 64), ("f32", 700, 1, 90, 3), ("f32", 530, 1, 90, 3),
    ("f16", 150, 4, 8192, 8)])
def test_shares_that_cross_rows(dt, B, K, V, n):
    """Enough work for every SM: CTAs walk several chunks, of one row or of several, with rows
    of ties, masked rows, dead beams and refused ones among them."""
    x, s = make(B, K, V, dt, B + K + V)
    x[1::7] = x[1::7].round()
    x[2::11] = 0.5                             # more ties than a piece ranks at once
    x[3::13, : V - 40] = -math.inf
    x[4::17] = -math.inf
    x[5::19, -1] = math.nan
    s[::5, 0] = -math.inf
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.beam_workspace(B, K, V, n)
    out = run(x, s, n, ws=ws, err=err)
    assert err.item() == pa.PA_DEVERR_LOGITS
    check(out, x, s, n)
    for a, b in zip(run(x, s, n, ws=ws), out):
        assert torch.equal(a, b)


def test_refusals_on_device_tensors():
    x, s = make(2, 2, 1000, "f32", 3)
    out = [torch.zeros(2, 4, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda"),
           torch.zeros(2, 4, dtype=torch.int32, device="cuda")]
    ws = pa.beam_workspace(2, 2, 1000, 4)
    bad = [
        (out[0].double(), *out[1:], x, s, ws), (out[0], out[1].long(), out[2], x, s, ws),
        (*out, x.double(), s, ws), (*out, x[:3], s, ws), (*out, x, s.half(), ws),
        (*out, x, s, ws[:256]), (*out, x, s, None), (*out, x.t().contiguous().t(), s, ws),
        (*out, x.cpu(), s, ws), (*out, x[:, 1:], s, ws),        # rows that start off 16 bytes
    ]
    for a in bad:
        with pytest.raises(pa.PAError):
            pa.pa_beam_select(*a)
    pa.pa_beam_select(torch.zeros(0, 4, device="cuda"), out[1][:0], out[2][:0], x[:0], s[:0], ws)


# ---- the operators together ------------------------------------------------------------

def test_beam_search_over_a_4_bit_cache():
    """Two prompts with four beams each, 24 steps: every step's rotation and append, attention,
    selection, reordering and copies, each held to the oracle on the same inputs. Beams share
    their prompt's blocks, part copy on write, and drop out."""
    hq, hkv, d, rot, V, K, NB = 8, 2, 64, 32, 500, 4, 96
    rng = np.random.default_rng(99)
    emb = {n: torch.from_numpy(rng.standard_normal((V, h, d)).astype(np.float16)).cuda()
           for n, h in (("q", hq), ("k", hkv), ("v", hkv))}
    head = torch.from_numpy(rng.standard_normal((hq * d, V)).astype(np.float32) * 0.2).cuda()
    table = torch.from_numpy(pa.pa_rope_table(256, rot)).cuda()
    kc = torch.zeros(NB, hkv, 16, d // 2 + 4, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ok, ov = kc.cpu().numpy(), vc.cpu().numpy()
    bm, ob = pa.BlockManager(NB), OBM.BlockManager(NB, 16, list(range(NB)))
    scale = 1 / math.sqrt(d)
    seqs = [[0, 1, 2, 3], [4, 5, 6, 7]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def f32(t):
        return bits_to_f64(tensor_bits(t), "f16").astype(np.float32)

    def append(tokens, positions, slots):
        q = emb["q"][tokens]
        q_out = torch.empty_like(q)
        key, value = emb["k"][tokens], emb["v"][tokens]
        pos, sl = torch.tensor(positions).cuda(), torch.from_numpy(np.asarray(slots)).cuda()
        pa.pa_rope_and_cache_int4(q_out, q, key, value, pos, table, kc, vc, sl, dev_error=err)
        tab = table.cpu().numpy()
        want = R.rotate(f32(q), tab, positions, False)
        assert np.array_equal(f32(q_out), want.astype(np.float16).astype(np.float32))
        I4.reshape_and_cache_int4(ok, ov, R.rotate(f32(key), tab, positions, False), f32(value),
                                  slots)
        return q_out

    prompts = [rng.integers(0, V, 37), rng.integers(0, V, 20)]
    for ids, prompt in zip(seqs, prompts):
        slots = bm.add_seq(ids[0], len(prompt))
        assert list(slots) == ob.add_seq(ids[0], len(prompt))
        append(torch.from_numpy(prompt).cuda(), list(range(len(prompt))), slots)
        for child in ids[1:]:
            bm.fork(ids[0], child)
            ob.fork(ids[0], child)
    tokens = torch.tensor([int(p[-1]) for p in prompts for _ in range(K)]).cuda()
    beam_scores = torch.full((2, K), -math.inf, device="cuda")
    beam_scores[:, 0] = 0.0
    ws_beam = pa.beam_workspace(2, K, V, K)
    out3 = (torch.empty(2, K, device="cuda"), torch.empty(2, K, dtype=torch.int32, device="cuda"),
            torch.empty(2, K, dtype=torch.int32, device="cuda"))
    copies = moves = 0
    for step in range(24):
        flat = [s for ids in seqs for s in ids]
        pairs, slots, positions = [], [], []
        for s in flat:
            positions.append(bm.seq_len(s))
            sl, cow = bm.append_slots(s, 1)
            osl, ocow = ob.append_slots(s, 1)
            assert list(sl) == osl and [tuple(p) for p in cow.tolist()] == [tuple(p) for p in ocow]
            slots.append(int(sl[0]))
            pairs += ocow
        if pairs:
            pa.pa_copy_blocks(kc, vc, pairs)
            for a, b in pairs:
                ok[b], ov[b] = ok[a], ov[a]
            copies += len(pairs)
        q = append(tokens, positions, np.asarray(slots, np.int64))
        ctx = np.asarray(positions, np.int32) + 1
        tables = bm.block_tables(flat, 8)
        out = torch.empty_like(q)
        ws = pa.decode_workspace(len(flat), hq, hkv, d, int(ctx.max()))
        pa.pa_paged_decode_int4(out, q, kc, vc, torch.from_numpy(tables).cuda(),
                                torch.from_numpy(ctx).cuda(), int(ctx.max()), scale, 0, ws, err)
        assert np.array_equal(kc.cpu().numpy(), ok) and np.array_equal(vc.cpu().numpy(), ov)
        want = I4.paged_decode_int4(tensor_bits(q), ok, ov, tables, ctx, scale, "f16")
        # |V| <= 5 here: half a step of half precision of that, and the scores' 2^-12
        assert np.abs(f32(out) - want).max() < 5 * (2.0 ** -11 + 2.0 ** -11)
        logits = out.float().reshape(len(flat), -1) @ head
        pa.pa_beam_select(*out3, logits, beam_scores, ws_beam, err)
        check(out3, logits, beam_scores, K)
        parents = out3[1].cpu().numpy()
        for ids, par in zip(seqs, parents):
            bm.reorder(ids, par)
            ob.reorder(ids, par.tolist())
            moves += int((par != np.arange(K)).sum())
        assert bm.num_free() == ob.num_free() and bm.free_list() == ob.free_list()
        tokens = out3[2].reshape(-1).long()
        beam_scores = out3[0].clone()
    assert err.item() == 0 and copies > 10 and moves > 10
    for s in [s for ids in seqs for s in ids]:
        bm.free_seq(s)
    assert bm.num_free() == NB
