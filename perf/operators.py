"""What is measured of the rotary cache writes, the 4-bit cache and the beam selection.

With ``own`` false every operator runs in its plain form: elementary torch
operations in 32 bits (64 for the log-probabilities of the beam selection, whose
ranks decide between close scores), rounded once at the end. With ``own`` true
``run`` makes the library's calls.

Operators (key ``op`` of a case):
  rope   rotate queries and keys by their positions, append keys and values to a
         paged cache of 16-bit elements or E4M3 codes
  write  the same into a cache of 4-bit codes, then the written rows read back
  decode attention of one query token a sequence over a 4-bit cache
  step   one serving step over a 4-bit cache: rotate, append, attend
  beam   selection of the best continuations over beams and vocabulary
"""

import math

import numpy as np
import torch

own = False

BS = 16  # tokens of a cache block
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FP8_SCALES = (0.02, 0.015)  # key and value scale of the E4M3 cases


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one sequence: pure latency
        {"name": "rope_one_token", "op": "rope", "cache": "same", "tokens": 1, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16"},
        # a batch of prompts at once: pure bandwidth
        {"name": "rope_prompts_16k", "op": "rope", "cache": "same", "tokens": 16384, "hq": 32,
         "hkv": 8, "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16"},
        # partial rotation with adjacent pairs, odd token count, 8-bit cache
        {"name": "rope_fp8_partial", "op": "rope", "cache": "e4m3", "tokens": 1237, "hq": 12,
         "hkv": 12, "d": 64, "rot": 32, "interleaved": True, "dtype": "f16"},
        # prompts into a 4-bit cache, and the rows read back (as a later chunk's attention would)
        {"name": "write_int4_prompts", "op": "write", "tokens": 4096, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "dtype": "bf16"},
        # the smallest decode: a handful of short sequences
        {"name": "decode_int4_tiny", "op": "decode", "batch": 4, "hq": 4, "hkv": 4, "d": 64,
         "ctx": "uniform", "lo": 1, "hi": 70, "dtype": "f16"},
        # multi-head attention of a 7B-like shape
        {"name": "decode_int4_mha", "op": "decode", "batch": 64, "hq": 32, "hkv": 32, "d": 128,
         "ctx": "uniform", "lo": 128, "hi": 2048, "dtype": "f16"},
        # a large serving batch with grouped heads and ragged contexts
        {"name": "decode_int4_gqa", "op": "decode", "batch": 256, "hq": 32, "hkv": 8, "d": 128,
         "ctx": "lognormal", "lo": 16, "hi": 4096, "dtype": "bf16"},
        # few long sequences: work split over the context
        {"name": "decode_int4_long", "op": "decode", "batch": 8, "hq": 64, "hkv": 8, "d": 128,
         "ctx": "uniform", "lo": 32768, "hi": 131072, "dtype": "bf16"},
        # a whole step of a serving loop: the new tokens' rotation and append, then attention
        {"name": "step_int4", "op": "step", "batch": 128, "hq": 32, "hkv": 8, "d": 128,
         "ctx": "lognormal", "lo": 16, "hi": 4096, "rot": 128, "interleaved": False,
         "dtype": "bf16"},
        # one request with four beams
        {"name": "beam_one_request", "op": "beam", "batch": 1, "beams": 4, "vocab": 32000,
         "select": 8, "dtype": "f32", "masked": False},
        # odd vocabulary, padded rows, a dead beam and masked tokens
        {"name": "beam_masked_odd", "op": "beam", "batch": 5, "beams": 3, "vocab": 50257,
         "select": 7, "dtype": "f16", "masked": True},
        # a serving batch of beams over a large vocabulary
        {"name": "beam_batch", "op": "beam", "batch": 64, "beams": 8, "vocab": 131072,
         "select": 16, "dtype": "bf16", "masked": False},
    ]


def draw(rng):
    def logint(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rope", "write", "decode", "decode", "step", "beam", "beam"])
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        vocab = logint(1000, 131072)
        batch = min(64, logint(1, max(1, 64 * 8 * 131072 // (beams * vocab * 2))))
        return {"op": "beam", "batch": batch, "beams": beams, "vocab": vocab,
                "select": rng.randint(1, min(32, 2 * beams + 3)),
                "dtype": rng.choice(["f16", "bf16", "f32"]), "masked": rng.random() < 0.4}
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 6, 8, 16])
    group = rng.choice([1, 2, 4, 8])
    heads = {"hq": hkv * group, "hkv": hkv, "d": d, "dtype": rng.choice(["f16", "bf16"])}
    rot = {"rot": rng.choice([16, 32, 48, 64] if d == 64 else [16, 32, 64, 80, 96, 112, 128]),
           "interleaved": rng.random() < 0.4}
    if op in ("rope", "write"):
        tokens = logint(1, max(1, min(16384, 16384 * 48 * 128 // (hkv * (group + 2) * d * 2))))
        c = {"op": op, "tokens": tokens, **heads, **rot}
        if op == "rope":
            c["cache"] = rng.choice(["same", "e4m3"])
        return c
    hi = logint(16, 65536)
    batch = max(1, min(256, logint(1, max(1, 2000000 // (hkv * hi)))))
    c = {"op": op, "batch": batch, "ctx": rng.choice(["uniform", "lognormal"]), "lo": 1, "hi": hi,
         **heads}
    if op == "step":
        c.update(rot)
    return c


def contexts(case):
    """Context lengths of the batch: the same for every seed, so that work() can count them."""
    rng = np.random.default_rng([case["batch"], case["lo"], case["hi"]])
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    if case["ctx"] == "uniform":
        c = rng.integers(lo, hi + 1, n)
    else:
        c = np.clip(np.rint(rng.lognormal(math.log(max(2.0, hi / 6)), 0.8, n)), lo, hi)
    c = c.astype(np.int64)
    c[0] = hi
    return c


def work(case):
    if case["op"] == "beam":
        rows = case["batch"] * case["beams"]
        n = rows * case["vocab"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * size + rows * 4 + case["batch"] * case["select"] * 12, "flops": 4 * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    kv4 = 2 * hkv * (d // 2 + 4)  # bytes of a token in the 4-bit caches
    if case["op"] in ("rope", "write"):
        t = case["tokens"]
        kv = {"same": 4 * hkv * d, "e4m3": 2 * hkv * d}[case["cache"]] if case["op"] == "rope" \
            else kv4 + kv4 + 4 * hkv * d  # written, read back, and the rows read back
        return {"bytes": t * (4 * hq * d + 4 * hkv * d + kv + 16 + 4 * case["rot"]),
                "flops": t * 3 * (hq + hkv) * case["rot"]}
    ctx = contexts(case)
    total, b = int(ctx.sum()), case["batch"]
    w = {"bytes": total * kv4 + b * 4 * hq * d + 4 * int((-(-ctx // BS)).sum()) + 4 * b,
         "flops": 4 * total * hq * d}
    if case["op"] == "step":
        w["bytes"] += b * (4 * hq * d + 4 * hkv * d + 16 + 4 * case["rot"])
        w["flops"] += b * 3 * (hq + hkv) * case["rot"]
    return w


# ---------------------------------------------------------------------------
# the 4-bit format, in plain form
# ---------------------------------------------------------------------------

def quantize(x):
    """Rows of 32-bit floats -> (codes 0..15, scale, mid): one half-precision scale and midpoint a
    row; a code n stands for mid + (n - 7.5) scale. Every step is rounded to 32 bits."""
    x = x.clamp(-65504.0, 65504.0)
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    scale = ((hi - lo) / torch.full_like(hi, 15.0)).half()
    mid = ((hi + lo) * 0.5).half()
    s = scale.float()
    inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
    code = torch.round((x - mid.float()) * inv + 7.5).clamp(0, 15).to(torch.uint8)
    return code, scale, mid


def pack(code, scale, mid, values):
    """Tiles of a 4-bit cache. code [..., 16, d] -> bytes [..., 16, d/2 + 4]: 16 d/2 bytes of codes,
    then (scale, mid) of the 16 tokens. Keys: token rows of d/2 bytes, dimension 2i in the low
    nibble of byte i. Values: the bytes of two tokens interleaved by pairs, in the order in which a
    matrix instruction's lanes take them."""
    lead, d = code.shape[:-2], code.shape[-1]
    b = code[..., 0::2] | (code[..., 1::2] << 4)  # [..., 16, d/2]
    if values:
        w = d // 32
        b = b.reshape(*lead, 2, 4, 2, 8, w, 2)  # token = 8 h + 2 p + e, byte = (g w + quad) 2 + half
        n = len(lead)
        b = b.permute(*range(n), n, n + 3, n + 1, n + 4, n + 2, n + 5)
    b = b.reshape(*lead, 8 * d)
    par = torch.cat([scale, mid], -1).contiguous().view(torch.uint8).reshape(*lead, 64)
    return torch.cat([b, par], -1).reshape(*lead, BS, d // 2 + 4)


def unpack(tile, values):
    """The 32-bit values of tiles [..., 16, d/2 + 4] -> [..., 16, d]."""
    lead, d = tile.shape[:-2], (tile.shape[-1] - 4) * 2
    flat = tile.reshape(*lead, 8 * d + 64)
    par = flat[..., 8 * d:].contiguous().view(torch.float16).reshape(*lead, BS, 2).float()
    b = flat[..., :8 * d]
    if values:
        w, n = d // 32, len(lead)
        b = b.reshape(*lead, 2, 8, 4, w, 2, 2)
        b = b.permute(*range(n), n, n + 2, n + 4, n + 1, n + 3, n + 5)
    b = b.reshape(*lead, BS, d // 2)
    code = torch.stack([b & 15, b >> 4], -1).reshape(*lead, BS, d).float()
    return par[..., 1:] + (code - 7.5) * par[..., :1]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def rope_table(rows, rot):
    """cos and sin of position x frequency, in 64 bits, rounded to 32: [rows, rot]."""
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] == "beam":
        b, k, v, n = case["batch"], case["beams"], case["vocab"], case["select"]
        width = v if v % 8 == 0 else v + 8 - v % 8  # rows padded as a sharded head leaves them
        logits = torch.empty(b * k, width, dtype=dt, device="cuda")
        logits.copy_(randn(b * k, width) * 3.0)
        s["beam_scores"] = -(randn(b, k).abs() * 4.0 + 2.0)
        if case["masked"]:  # a grammar's mask, and a beam that has ended
            logits[torch.rand(b * k, width, generator=g, device="cuda") < 0.3] = -math.inf
            s["beam_scores"][:, k - 1] = -math.inf if k > 1 else -1.0
        s["logits"] = logits[:, :v]
        s["scores"] = torch.empty(b, n, device="cuda")
        s["parents"] = torch.empty(b, n, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty(b, n, dtype=torch.int32, device="cuda")
        if own:
            import paged_kv_cache_352_b200 as pa
            s["ws"] = pa.beam_workspace(b, k, v, n)
        return s

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    bias = randn(hkv, d) * 1.5  # keys have channels with a mean of their own
    if case["op"] in ("rope", "write"):
        t = case["tokens"]
        nb = -(-t // BS) + 3
        order = torch.randperm(nb, generator=g, device="cuda")
        at = torch.arange(t, device="cuda")
        s["slots"] = order[at // BS] * BS + at % BS
        s["positions"] = at % 4096 + int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        s["table"] = rope_table(8192, case["rot"])
        s["q"] = randn(t, hq, d).to(dt)
        s["key"] = (randn(t, hkv, d) + bias).to(dt)
        s["value"] = randn(t, hkv, d).to(dt)
        s["q_out"] = torch.empty_like(s["q"])
        if case["op"] == "write":
            s["k_cache"] = torch.zeros(nb, hkv, BS, d // 2 + 4, dtype=torch.uint8, device="cuda")
            s["k_back"], s["v_back"] = torch.empty_like(s["key"]), torch.empty_like(s["value"])
        else:
            ct = dt if case["cache"] == "same" else torch.float8_e4m3fn
            s["k_cache"] = torch.zeros(nb, hkv, BS, d, device="cuda").to(ct)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        return s

    ctx = contexts(case)
    b, blocks = case["batch"], -(-ctx // BS)
    nb, width = int(blocks.sum()) + 2, int(blocks.max())
    order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    ends = torch.from_numpy(np.cumsum(blocks)).cuda()
    first = ends - torch.from_numpy(blocks).cuda()
    at = first[:, None] + torch.arange(width, device="cuda")
    s["tables"] = torch.where(at < ends[:, None], order[at.clamp(max=nb - 1)],
                              torch.full_like(order[:1], -1))
    s["k_cache"] = torch.empty(nb, hkv, BS, d // 2 + 4, dtype=torch.uint8, device="cuda")
    s["v_cache"] = torch.empty_like(s["k_cache"])
    step = max(1, (1 << 27) // (hkv * BS * d))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        x = randn(n, hkv, BS, d)
        s["v_cache"][i:i + n] = pack(*quantize(x), True)
        s["k_cache"][i:i + n] = pack(*quantize(randn(n, hkv, BS, d) + bias[:, None]), False)
    s["ctx"] = torch.from_numpy(ctx).to(torch.int32).cuda()
    s["order"] = torch.from_numpy(np.argsort(-ctx, kind="stable").astype(np.int32)).cuda()
    s["max_ctx"], s["scale"] = int(ctx.max()), 1.0 / math.sqrt(d)
    s["q"] = randn(b, hq, d).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if case["op"] == "step":
        last = s["ctx"].long() - 1
        s["positions"] = last
        s["slots"] = s["tables"].long().gather(1, (last // BS)[:, None])[:, 0] * BS + last % BS
        s["table"] = rope_table(case["hi"] + 1, case["rot"])
        s["key"] = (randn(b, hkv, d) + bias).to(dt)
        s["value"] = randn(b, hkv, d).to(dt)
        s["q_out"] = torch.empty_like(s["q"])
    if own:
        import paged_kv_cache_352_b200 as pa
        s["ws"] = pa.decode_workspace(b, hq, hkv, d, s["max_ctx"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return run_own(s)
    op = s["op"]
    if op == "beam":
        return plain_beam(s)
    if op == "decode":
        return plain_decode(s, s["q"])
    dt = s["q"].dtype
    q = rotate(s["q"], s).to(dt)
    k, v = rotate(s["key"], s), s["value"].float()
    at = (s["slots"] // BS, slice(None), s["slots"] % BS)
    if op == "rope":
        if s["cache"] == "e4m3":
            k = (k / torch.full_like(k, FP8_SCALES[0])).clamp(-448.0, 448.0)
            v = (v / torch.full_like(v, FP8_SCALES[1])).clamp(-448.0, 448.0)
            kc, vc = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
            kc[at] = k.to(torch.float8_e4m3fn).view(torch.uint8)
            vc[at] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            s["k_cache"][at], s["v_cache"][at] = k.to(dt), s["value"]
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "write":
        back = []
        for x in (k, v):
            code, scale, mid = quantize(x)
            back.append((mid.float() + (code.float() - 7.5) * scale.float()).to(dt))
        return {"q": q, "key": back[0], "value": back[1]}
    put(s["k_cache"], s["slots"], quantize(k), False)
    put(s["v_cache"], s["slots"], quantize(v), True)
    return {"q": q, "out": plain_decode(s, q)}


def run_own(s):
    import paged_kv_cache_352_b200 as pa
    op = s["op"]
    if op == "beam":
        pa.pa_beam_select(s["scores"], s["parents"], s["tokens"], s["logits"], s["beam_scores"],
                          s["ws"])
        return {"scores": s["scores"], "parents": s["parents"], "tokens": s["tokens"]}
    if op == "decode":
        pa.pa_paged_decode_int4(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"],
                                s["max_ctx"], s["scale"], workspace=s["ws"], seq_order=s["order"])
        return s["out"]
    a = (s["q_out"], s["q"], s["key"], s["value"], s["positions"], s["table"], s["k_cache"],
         s["v_cache"], s["slots"])
    if op == "rope":
        if s["cache"] == "e4m3":
            pa.pa_rope_and_cache_fp8(*a, *FP8_SCALES, interleaved=s["interleaved"])
        else:
            pa.pa_rope_and_cache(*a, interleaved=s["interleaved"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    pa.pa_rope_and_cache_int4(*a, interleaved=s["interleaved"])
    if op == "write":
        pa.pa_read_slots_int4(s["k_back"], s["v_back"], s["k_cache"], s["v_cache"], s["slots"])
        return {"q": s["q_out"], "key": s["k_back"], "value": s["v_back"]}
    pa.pa_paged_decode_int4(s["out"], s["q_out"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"],
                            s["max_ctx"], s["scale"], workspace=s["ws"], seq_order=s["order"])
    return {"q": s["q_out"], "out": s["out"]}


def rotate(x, s):
    """Rows rotated by their positions, in 32 bits: [T, H, d]."""
    rot, x = s["rot"], x.float()
    cs = s["table"][s["positions"]][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def put(cache, slots, parts, values):
    """New rows into the tiles that hold their slots (every slot in a block of its own)."""
    blocks, at = slots // BS, slots % BS
    code, scale, mid = parts
    n, h, d = code.shape
    # a tile with the new rows in every token's place, and which of its bytes are the row's
    tile = pack(code[:, :, None].expand(n, h, BS, d).contiguous(),
                scale[:, :, None].expand(n, h, BS, 1), mid[:, :, None].expand(n, h, BS, 1), values)
    token = torch.arange(BS, device=code.device) == at[:, None]
    mask = torch.where(token, 255, 0).to(torch.uint8)[:, None, :, None]
    half = mask.view(torch.int8).to(torch.int16).view(torch.float16)  # all bits of the token's
    mine = pack((mask & 15).expand(n, h, BS, d).contiguous(), half.expand(n, h, BS, 1),
                half.expand(n, h, BS, 1), values)
    cache[blocks] = (cache[blocks] & ~mine) | (tile & mine)


def plain_decode(s, q):
    tables, ctx = s["tables"].long().clamp(min=0), s["ctx"].long()
    b, hq, d = q.shape
    hkv = s["hkv"]

    def rows(cache, values):  # [B, Hkv, tokens, d]
        x = unpack(cache[tables], values)
        return x.transpose(1, 2).reshape(b, hkv, -1, d)

    x = q.float().reshape(b, hkv, hq // hkv, d)
    score = (x @ rows(s["k_cache"], False).transpose(-1, -2)) * s["scale"]
    inside = torch.arange(score.shape[-1], device=q.device) < ctx[:, None]
    score = score.masked_fill(~inside[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp()
    v = rows(s["v_cache"], True).masked_fill(~inside[:, None, :, None], 0.0)
    return ((p @ v) / p.sum(-1, keepdim=True)).reshape(b, hq, d).to(q.dtype)


def plain_beam(s):
    b, k, v, n = s["batch"], s["beams"], s["vocab"], s["select"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    logp = x - (top + (x - top).exp().sum(-1, keepdim=True).log())
    score = (s["beam_scores"].double()[:, :, None] + logp.reshape(b, k, v)).reshape(b, k * v)
    best, at = score.sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    dead = best == -math.inf
    return {"scores": best.float(),
            "parents": (at // v).masked_fill(dead, -1).to(torch.int32),
            "tokens": (at % v).masked_fill(dead, -1).to(torch.int32)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def turned(x, s):
    """The rotation of one row at a time as a complex product, in 64 bits."""
    rot = s["rot"]
    half = rot // 2
    cs = s["table"].double()[s["positions"]]
    w = torch.complex(cs[:, :half], cs[:, half:])[:, None]
    y = x.double().clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else \
        (slice(0, half), slice(half, rot))
    z = torch.complex(y[..., first], y[..., second]) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def held(x):
    """What a 4-bit row holds of 64-bit rows: scale and midpoint as halves, codes to the nearest."""
    x = x.clamp(-65504.0, 65504.0)
    hi, lo = x.max(-1, keepdim=True).values, x.min(-1, keepdim=True).values
    scale, mid = ((hi - lo) / 15).half().double(), ((hi + lo) / 2).half().double()
    n = ((x - mid) / torch.where(scale > 0, scale, math.inf) + 7.5).round().clamp(0, 15)
    return mid + (n - 7.5) * scale


def elements(cache, block, values):
    """The values of whole tiles, element by element from the byte that holds each: [n, Hkv, 16, d]."""
    d = (cache.shape[-1] - 4) * 2
    tile = cache[block].flatten(2)
    t = torch.arange(BS, device=cache.device)[:, None]
    x = torch.arange(d, device=cache.device)
    w = d // 32
    if values:
        pair = t // 2
        chunk = (pair // 4) * 32 + (x // (4 * w)) * 4 + pair % 4
        byte = (chunk * w + x // 4 % w) * 4 + t % 2 * 2 + x % 4 // 2
    else:
        byte = t * (d // 2) + x // 2
    code = (tile[:, :, byte] >> (x % 2 * 4).to(torch.uint8)) & 15
    par = tile[:, :, 8 * d:].contiguous().view(torch.float16).double()
    return par[:, :, 1::2, None] + (code.double() - 7.5) * par[:, :, 0::2, None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "beam":
        b, k, n = case["batch"], case["beams"], case["select"]
        logp = torch.log_softmax(s["logits"].double(), -1).reshape(b, k, -1)
        score = (logp + s["beam_scores"].double()[..., None]).reshape(b, -1)
        return {"scores": torch.topk(score, n, -1).values, "parents": None, "tokens": None}
    if op in ("rope", "write"):
        q, k, v = turned(s["q"], s), turned(s["key"], s), s["value"].double()
        if op == "write":
            return {"q": q, "key": held(k), "value": held(v)}
        kc, vc = (torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
                  for _ in range(2))
        if case["cache"] == "e4m3":
            k, v = (k / FP8_SCALES[0]).clamp(-448, 448), (v / FP8_SCALES[1]).clamp(-448, 448)
        kc[s["slots"] // BS, :, s["slots"] % BS] = k
        vc[s["slots"] // BS, :, s["slots"] % BS] = v
        return {"q": q, "k_cache": kc, "v_cache": vc}
    q = s["q"].double()
    new = None
    if op == "step":
        turned_q = turned(s["q"], s)
        q = turned_q.to(s["q"].dtype).double()
        new = held(turned(s["key"], s)), held(s["value"].double())
    hkv = case["hkv"]
    outs = []
    for i, n in enumerate(contexts(case)):
        block = s["tables"][i, :-(-n // BS)].long()
        k, v = (elements(s[c], block, c == "v_cache").transpose(0, 1).flatten(1, 2)[:, :n]
                for c in ("k_cache", "v_cache"))
        if new is not None:
            k, v = k.clone(), v.clone()
            k[:, n - 1], v[:, n - 1] = new[0][i], new[1][i]
        x = q[i].reshape(hkv, -1, k.shape[-1])
        p = torch.softmax(torch.einsum("hgd,htd->hgt", x, k) * s["scale"], -1)
        outs.append(torch.einsum("hgt,htd->hgd", p, v).flatten(0, 1))
    out = torch.stack(outs)
    return out if op == "decode" else {"q": turned_q, "out": out}
