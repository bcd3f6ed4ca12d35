"""Plain statements of the 4-bit pools and of attention over windows and
prompts, for the tests: numpy, 64 bits but where the definition says float32.
Nothing here shares code with the library."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6] + [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
E4M3 = np.array([np.nan if c == 127 else c * 2.0 ** -9 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7)
                 for c in range(128)])
HALF_STEP = {np.dtype("float32"): 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def nearest(a, grid):
    """Index of the grid value nearest to a >= 0 (ascending grid; ties to the even index; the last one beyond it)."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, a, side="left")
    at = np.minimum(i, len(mid) - 1)
    return i + ((i < len(mid)) & (a == mid[at]) & (i % 2 == 1))


def quantise(x, head_scale=None):
    """x float32 [..., H, D]: codes uint8 [..., D] (0..15) and scale bytes uint8 [..., D / 16]; float32 as defined."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if head_scale is not None:
            x = x * (np.float32(1) / np.asarray(head_scale, np.float32))[:, None]
        z = x.reshape(*x.shape[:-1], -1, 16)
        top = np.abs(z).max(-1)  # NaN where there is one
        scale = nearest(np.where(np.isnan(top), 0, top / np.float32(6)).astype(np.float64), E4M3[:127])
        scale = np.where(np.isnan(top), 127, scale)
        s = np.where(np.isnan(top), 0, E4M3[np.minimum(scale, 126)]).astype(np.float32)[..., None]
        quot = np.where(s > 0, np.abs(z) / s, 0)
        code = nearest(np.where(np.isnan(quot), 0, quot).astype(np.float64), E2M1[:8]) + 8 * np.signbit(z)
    return code.reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def unpack(pool, D):
    """Pool bytes [NB, H, tiles, 9 D]: codes [NB, H, 16 tiles, D] and scale bytes [NB, H, 16 tiles, D / 16]."""
    NB, H, T, _ = pool.shape
    b = pool[..., :8 * D].reshape(NB, H, T * 16, D // 2)
    return np.stack([b & 15, b >> 4], -1).reshape(NB, H, T * 16, D), pool[..., 8 * D:].reshape(NB, H, T * 16, D // 16)


def pack(codes, scales):
    """The reverse of unpack."""
    NB, H, B, D = codes.shape
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return np.concatenate([b.reshape(NB, H, B // 16, 8 * D), scales.reshape(NB, H, B // 16, D)], -1)


def values(pool, D, head_scale=None):
    """[NB, B, H, D] float64."""
    codes, scales = unpack(pool, D)
    x = E2M1[codes] * np.where(scales & 128, -1.0, 1.0).repeat(16, -1) * E4M3[scales & 127].repeat(16, -1)
    if head_scale is not None:
        x = x * np.asarray(head_scale, np.float64)[None, :, None, None]
    return x.transpose(0, 2, 1, 3)


def visible(p, n, window, sinks):
    """Of tokens 0 .. n - 1, those that the query at position p sees (window 0: none beside causality)."""
    t = np.arange(n)
    m = t <= p
    return m & ((t > p - window) | (t < sinks)) if window else m


def attend(q, k, v, scale, see):
    """One query row q [Hq, D] over k, v [n, H, D] float64, tokens `see` alone: (out [Hq, D], bound): `bound`
    holds, per element, sum_t p_t |v_t| and sum_t |v_t| and, per head, the magnitudes of the scores' terms (largest
    over tokens)."""
    Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mass, total, terms = np.zeros((Hq, D)), np.zeros((Hq, D)), np.zeros((Hq, D)), np.zeros(Hq)
    idx = np.nonzero(see)[0]
    if len(idx):
        for h in range(Hq):
            kk, vv = k[idx, h // G], v[idx, h // G]
            s = kk @ q[h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[h], mass[h], total[h] = p @ vv, p @ np.abs(vv), np.abs(vv).sum(0)
            terms[h] = (np.abs(kk) @ np.abs(q[h])).max() * abs(scale)
    return out, (mass, total, terms)


def bound(out, extra, D, n, weights, out_step, floor=2.0 ** -39):
    """How far a kernel's row may be from `attend`'s: its scores are off by at most (D + 8) 2^-23 of the terms
    (sums of D products on the tensor cores, each addition cut off at 2^-23 at the most, and the scale), a weight
    by twice that relative to the row's sum, by 2^-21 for its exponential and by `weights` for the type that holds
    it; sums of n tokens lose at most n 2^-23 (and the rows' merging as much again); the row is rounded once.
    Where f16 holds the weights, times 2^14, its subnormals' half step of 2^-25 is 2^-39 of the largest weight: a
    weight far below the largest is off by that absolutely, which matters where the largest one's value is 0 (`floor`:
    prompts hold them times 2^7, 2^-32; 4-bit pools times 2^8, 2^-33)."""
    mass, total, terms = extra
    rel = 4 * (D + 8) * 2.0 ** -23 * terms[:, None] + 2.0 ** -20 + weights + 4 * (n + 64) * 2.0 ** -23
    return mass * rel + total * floor + np.abs(out) * out_step + 1e-30
