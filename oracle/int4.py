"""4-bit KV cache, oracle side.

Test infrastructure: only the tests and the smoke check may use this module. It
shares no code with the CUDA-side library.

The pages name KV-cache quantization as the next lever on a bandwidth-bound
path ("PagedAttention: The vLLM Paper", "Impact and Follow-Ups" and
"Limitations") but fix no format. Reading taken: every row (one token, one KV
head, of K or of V) keeps 4-bit codes n with a half-precision scale and midpoint
of its own, and a code stands for mid + (n - 7.5) * scale.

  * storing a row: x in float32, clamped to +-65504; scale = half((max - min) /
    15), mid = half((max + min) * 0.5), inv = float32(1) / scale (0 for scale 0),
    n = clamp(rint((x - mid) * inv + 7.5), 0, 15), every operation a single
    float32 operation rounded to nearest, rint with ties to even. A row with a
    NaN gets NaN scale and mid, and codes 0;
  * a cache is bytes [num_blocks][Hkv][16][d/2 + 4]; a (block, KV head) tile holds
    8 d bytes of codes, then the 16 pairs (scale, mid). Key rows lie one after
    the other, two codes a byte, the even dimension low; the bytes of the value
    rows 2p and 2p + 1 interleave two by two and are ordered by (p / 4, dimension
    / (d/8), p % 4, dimension).
"""

import numpy as np

from oracle.attention import softmax_attention
from oracle.fpbits import bits_to_f64

BLOCK = 16


def quantize_row(x):
    """One row of float32 values -> (codes, scale, mid)."""
    x = np.asarray(x, np.float32)
    if np.isnan(x).any():
        return np.zeros(len(x), np.uint8), np.float16("nan"), np.float16("nan")
    x = np.clip(x, np.float32(-65504), np.float32(65504))
    hi, lo = x.max(), x.min()
    scale = np.float16((hi - lo) / np.float32(15))
    mid = np.float16((hi + lo) * np.float32(0.5))
    inv = np.float32(1) / np.float32(scale) if scale > 0 else np.float32(0)
    u = (x - np.float32(mid)) * inv + np.float32(7.5)
    return np.clip(np.rint(u), 0, 15).astype(np.uint8), scale, mid


def code_place(d, token, dim, values):
    """(byte, nibble) of a code inside its tile."""
    if not values:
        return token * (d // 2) + dim // 2, dim % 2
    words = d // 32                      # 32-bit words of one (pair of tokens, d/8 dimensions)
    pair, odd = divmod(token, 2)
    eighth, rest = divmod(dim, 4 * words)
    word, inner = divmod(rest, 4)
    chunk = (pair // 4) * 32 + eighth * 4 + pair % 4
    return (chunk * words + word) * 4 + 2 * odd + inner // 2, inner % 2


def write_row(tile, d, token, x, values):
    """Quantize row x into the flat tile (uint8 [16 (d/2 + 4)])."""
    codes, scale, mid = quantize_row(x)
    for dim in range(d):
        byte, nibble = code_place(d, token, dim, values)
        keep = 0x0F if nibble else 0xF0
        tile[byte] = (int(tile[byte]) & keep) | (int(codes[dim]) << (4 * nibble))
    tile[8 * d + 4 * token:8 * d + 4 * token + 4] = np.array([scale, mid], np.float16).view(np.uint8)


def read_tile(tile, d, values):
    """The 16 rows of a flat tile in float64."""
    par = tile[8 * d:].copy().view(np.float16).astype(np.float64).reshape(BLOCK, 2)
    out = np.empty((BLOCK, d))
    for t in range(BLOCK):
        for dim in range(d):
            byte, nibble = code_place(d, t, dim, values)
            out[t, dim] = par[t, 1] + (((int(tile[byte]) >> (4 * nibble)) & 15) - 7.5) * par[t, 0]
    return out


def reshape_and_cache_int4(k_cache, v_cache, key, value, slots):
    """key/value float32 [T, Hkv, d] into uint8 caches [nb, Hkv, 16, d/2 + 4]."""
    d = key.shape[-1]
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        b, o = divmod(int(slot), BLOCK)
        for h in range(key.shape[1]):
            write_row(k_cache[b, h].reshape(-1), d, o, key[t, h], False)
            write_row(v_cache[b, h].reshape(-1), d, o, value[t, h], True)


def dequantize_cache(cache, values):
    """float64 [nb, Hkv, 16, d] of a cache."""
    nb, hkv, _, row = cache.shape
    d = 2 * (row - 4)
    out = np.empty((nb, hkv, BLOCK, d))
    # the places are the same in every tile: take them once
    place = np.array([[code_place(d, t, x, values) for x in range(d)] for t in range(BLOCK)])
    flat = cache.reshape(nb, hkv, -1)
    codes = (flat[:, :, place[..., 0]] >> (4 * place[..., 1]).astype(np.uint8)) & 15
    par = flat[:, :, 8 * d:].copy().view(np.float16).astype(np.float64).reshape(nb, hkv, BLOCK, 2)
    with np.errstate(invalid="ignore"):
        out[:] = par[..., 1:] + (codes - 7.5) * par[..., :1]
    return out


def paged_decode_int4(q_bits, k_cache, v_cache, block_tables, context_lens, scale, dtype):
    """out[s][h] in float64 from 16-bit query patterns and 4-bit caches."""
    q = bits_to_f64(q_bits, dtype)
    B, hq, d = q.shape
    hkv = k_cache.shape[1]
    k, v = dequantize_cache(k_cache, False), dequantize_cache(v_cache, True)
    out = np.zeros((B, hq, d))
    for s in range(B):
        n = int(context_lens[s])
        if n == 0:
            continue
        blocks = [int(x) for x in block_tables[s][:-(-n // BLOCK)]]
        for h in range(hq):
            g = h // (hq // hkv)
            ks = np.concatenate([k[b, g] for b in blocks])[:n]
            vs = np.concatenate([v[b, g] for b in blocks])[:n]
            out[s, h] = softmax_attention(q[s, h], ks, vs, scale)
    return out
