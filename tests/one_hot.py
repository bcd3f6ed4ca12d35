"""Histories on which every token can be told from every other, for the tests of attention over pools.

V of token t is zero but in channel (t + 5 g) % D of KV head g, K in channel (7 t + g) % D.  A score is then one
product, which binary16 and bfloat16 operands give exactly, and an output channel the sum of a few tokens' weights,
all of one sign: what a kernel leaves out, counts twice or rounds shows at its full size, where in sums of random
values it would be lost among the others' roundings."""
import numpy as np

from tests import window_ref as R


# Cases whose histories are long enough for bounds that grow with their length to hide something; the CPU tests show
# that a single token left out of them or counted twice is seen.
# Partitions of 4-bit decode: lens, Hq, Hkv, D, block, type, partition size (odd numbers of 16 tokens among them).
PARTITIONS = [([40000, 17, 0, 1008, 1009, 2016], 8, 2, 128, 16, "bf16", 1008), ([30000, 29000], 2, 2, 128, 32, "f16", 1008),
              ([60000, 1007], 6, 2, 64, 64, "f16", 1008), ([50000, 70], 5, 1, 128, 32, "bf16", 528),
              ([60000], 4, 1, 64, 16, "f16", 16), ([120000, 3000], 4, 1, 128, 64, "bf16", 48),
              ([30000, 31, 900], 16, 2, 128, 64, "f16", 240), ([30000, 30001], 14, 2, 128, 16, "f16", 1008),
              ([60000], 16, 2, 64, 32, "bf16", 496), ([3000 + 37 * (i % 7) for i in range(40)], 8, 4, 64, 16, "bf16", 128)]
# Windows: bits of the pools, sequences, length, window.
WINDOWS = [(bits, S, L, w) for bits in (4, 16) for S, L, w in ((1, 9000, 8000), (40, 3000, 2000), (3, 30000, 29000))]
# Prompts: new tokens, past, query and KV heads, D.
PROMPTS = [([1], [5000], 4, 1, 128), ([37], [2000], 4, 1, 128), ([7], [20000], 4, 1, 128), ([200], [900], 4, 1, 64),
           ([5], [8000], 8, 2, 64), ([6000, 2100], [100, 0], 8, 2, 128), ([3000], [6000], 8, 1, 64)]
PROMPT_TYPES = [("f16", None), ("f16", "f32"), ("bf16", "f32")]  # pools, output


def partition_chain(L, size):
    """A partition's tokens, and the join's 16 warps over the partitions, which count as eight tokens each."""
    return size + -(-L // size) // 2


def prompt_part(dt, out):
    """What the types that hold a prompt's weight leave of it: one of the pools' type, or two for float32 outputs."""
    f16 = dt == "f16"
    return (2.0 ** -22 if f16 else 2.0 ** -17) if out == "f32" else (2.0 ** -11 if f16 else 2.0 ** -8)


def histories(lens, tables, NB, B, Hkv, D, rng):
    """k and v float32 [NB, B, Hkv, D] of sequences of `lens` tokens in the blocks of `tables`; zero elsewhere."""
    k, v = (np.zeros((NB, B, Hkv, D), np.float32) for _ in range(2))
    for i, L in enumerate(lens):
        t = np.arange(L)
        blk, off = tables[i, t // B], t % B
        for g in range(Hkv):
            k[blk, off, g, (7 * t + g) % D] = rng.uniform(-1, 1, L)
            v[blk, off, g, (t + 5 * g) % D] = rng.uniform(0.9, 1.1, L)
    return k, v


def queries(S, Hq, D, rng):
    """Magnitudes from a half to one: with a scale of 1, scores from -1 to 1."""
    return (rng.uniform(0.5, 1, (S, Hq, D)) * rng.choice([-1, 1], (S, Hq, D))).astype(np.float32)


def bound(want, chain, part, out_step, floor):
    """How far a row may be from its value, in units of the value.  Scores are at most S = 2 (in units of a factor of
    two; head scales are powers of two): the product is exact, its factor is rounded three times, the shift twice and
    their sum once, each by 2^-24 of at most S + 8, so a weight is off by 6 (S + 8) 2^-24 < 2^-18 and the sum of
    weights as much; an exponential by 2^-22, twice.  `part`: what the types that hold a weight leave of it.  An
    accumulator that takes up `chain` tokens does so 8 or more at a time, losing 2^-23 each; the meeting of the parts
    adds 32 roundings at the most.  `floor`: half a step of the smallest f16 that holds a weight, in units of the
    row's largest, for all the tokens of a channel."""
    rel = 2.0 ** -17 + 2.0 ** -21 + part + 2 * (chain / 8 + 32) * 2.0 ** -23 + out_step
    return np.abs(want) * rel + floor + 1e-30


def attend(q, k, v, scale, see):
    """window_ref's row of one query [Hq, D] over k, v [n, Hkv, D] float64."""
    return R.attend(q, k, v, scale, see)[0]
