"""Where the parts of a split-KV workspace lie when calls of different sizes share one buffer: the
merge counters of any call that fits stay clear of the accumulators that any other leaves."""

import random

import paged_kv_cache_352_b200 as pa


def up(x):
    return (x + 255) // 256 * 256


def parts(units, nparts, group, d, buffer):
    """(bytes needed, end of the counters, start of the accumulators) in a buffer."""
    ml_off = up(4 * units)
    acc_off = up(ml_off + units * nparts * group * 2 * 4)
    need = up(acc_off + units * nparts * group * d * 4)
    return need, 4 * units, acc_off + (buffer - need) // 256 * 256


def test_counters_stay_clear_of_accumulators():
    rng = random.Random(5)

    def draw():
        units = int(2 ** rng.uniform(0, 16))
        nparts = 2 + int(2 ** rng.uniform(0, rng.choice([1, 4, 9])))
        return units, rng.choice([2, nparts]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])

    for _ in range(20000):
        a, b = draw(), draw()
        needs = [parts(*x, 0)[0] for x in (a, b)]
        buffer = max(needs) + rng.choice([0, 0, 1, 255, 256, rng.randrange(1 << 22)])
        for x, y in ((a, b), (b, a)):
            assert parts(*y, buffer)[1] <= parts(*x, buffer)[2], (x, y, buffer)
            assert parts(*y, buffer)[1] <= buffer / 133
            assert parts(*x, buffer)[2] + 4 * x[0] * x[1] * x[2] * x[3] <= buffer


def test_the_same_sizes_as_the_library():
    for seqs, hkv, group, d, ctx, part in ((3, 2, 4, 128, 1500, 64), (70, 4, 1, 64, 600, 512),
                                           (1, 1, 8, 64, 33, 16), (8, 8, 8, 128, 131072, 512)):
        nparts = -(-(-(-ctx // 16)) // (part // 16))
        assert parts(seqs * hkv, nparts, group, d, 0)[0] == pa.pa_paged_decode_workspace_size(
            seqs, group * hkv, hkv, d, ctx, 16, part)
