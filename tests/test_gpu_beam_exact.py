"""Beam selection where candidates of different beams lie closer than fp32 sums of exponentials
tell apart: order, parents and tokens have to be the float64 oracle's, without tolerance."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_352_b200 as pa
from oracle import beam as OB
from tests.test_gpu_beam import TDT, check, make, run

pytestmark = pytest.mark.gpu


def exact(out, logits, beam_scores, n, seqs=None):
    """Parents and tokens equal to the oracle's, scores to a rounding of its float64 values."""
    B, K = beam_scores.shape
    scores, parents, tokens = (t.cpu().numpy() for t in out)
    for b in range(B) if seqs is None else seqs:
        x = logits[b * K:(b + 1) * K].float().cpu().numpy()
        want = OB.select(x, beam_scores[b].cpu().numpy(), n)
        assert np.array_equal(parents[b], want[1]), (b, parents[b], want[1])
        assert np.array_equal(tokens[b], want[2]), (b, tokens[b], want[2])


@pytest.mark.parametrize("dt,B,K,V,n", [
    ("f32", 3, 4, 3000, 16), ("bf16", 5, 8, 50257, 16), ("bf16", 64, 8, 131072, 16),
    ("f16", 80, 4, 50257, 12), ("f32", 24, 9, 33000, 18)])
def test_beams_that_are_copies(dt, B, K, V, n):
    """Beams with the same logits and scores, wherever a CTA's share of the rows ends: every tie
    goes to the smaller beam."""
    x, s = make(B, K, V, dt, 31)
    x = x.contiguous() if V % 8 == 0 else x
    for k in range(1, K, 2):
        x[k::K] = x[k - 1::K]
        s[:, k] = s[:, k - 1]
    exact(run(x, s, n), x, s, n, range(0, B, max(1, B // 16)))


@pytest.mark.parametrize("dt,B,K,V,n", [
    ("f32", 200, 2, 1500, 6), ("bf16", 120, 3, 5000, 8), ("f16", 70, 2, 131072, 6),
    ("f32", 40, 8, 40000, 12)])
def test_candidates_closer_than_fp32(dt, B, K, V, n):
    """Beam scores set so that the beams' best candidates lie within 1e-7 of each other."""
    x, s = make(B, K, V, dt, 77)
    xs = x.float().cpu().numpy().astype(np.float64)
    top = xs.max(1)
    lp = (top - top) - np.log(np.exp(xs - top[:, None]).sum(1))      # the best log-probability
    lp = lp.reshape(B, K)
    goal = -0.75 + np.random.default_rng(3).uniform(-1, 1, (B, K)) * 1e-7
    s.copy_(torch.from_numpy((goal - lp).astype(np.float32)))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(x, s, n, err=err)
    assert err.item() == 0
    exact(out, x, s, n)
    check(out, x, s, n)


def test_close_candidates_beside_dead_and_masked_beams():
    """The same with ended beams, masked tokens, refused rows and more ties than are ranked at
    once among the close ones."""
    B, K, V, n = 30, 4, 9000, 20
    x, s = make(B, K, V, "f32", 5)
    x = x.clone()
    for k in (1, 3):
        x[k::K] = x[k - 1::K]
        s[:, k] = s[:, k - 1]
    x[0:4, ::2] = -math.inf
    s[1, :2] = -math.inf
    x[8:12] = 0.25                             # every candidate of the sequence ties
    s[2] = torch.tensor([-1.0, -1.0000001, -1.0, -0.9999999])
    x[13, 5] = math.nan
    x[16:18] = -math.inf
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(x, s, n, err=err)
    assert err.item() == pa.PA_DEVERR_LOGITS
    exact(out, x, s, n)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [504, 40000])
def test_scores_past_the_largest_float(dt, V):
    """A beam score of the lowest float and logits masked with the type's lowest value add up past
    it: such tokens stay candidates and their score is the lowest float; -inf goes with -1."""
    low = torch.finfo(torch.float32).min
    x = torch.full((40 * 3, V), torch.finfo(TDT[dt]).min, dtype=TDT[dt], device="cuda")
    x[:, :2] = 1.0
    s = torch.full((40, 3), low, device="cuda")
    s[:, 1] = -math.inf
    out = run(x, s, 9)
    exact(out, x, s, 9, range(0, 40, 13))
    assert bool((out[1] >= 0).all()) and bool((out[0] == low).all())
    x[:, 2:] = -math.inf
    scores, parents, _ = (t.cpu().numpy() for t in run(x, s, 9))
    assert (parents == [0, 0, 2, 2, -1, -1, -1, -1, -1]).all()
    assert np.array_equal(np.isinf(scores), parents < 0)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_beam_score_is_reported_whatever_its_logits(bad):
    x, s = make(2, 3, 700, "f32", 6)
    x = x.clone()
    x[1] = -math.inf                           # every token of the beam is masked
    s[0, 1] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(x, s, 5, err=err)
    assert err.item() == pa.PA_DEVERR_LOGITS
    check(out, x, s, 5)
