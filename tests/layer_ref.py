"""Plain float64 statements of the layer operators (norm + rotation + write,
block summaries, block selection, sparse decode), for the tests.  Values come
in as float64 arrays; nothing here shares code with the library."""
import numpy as np

E4M3 = np.array([(-1.0 if c & 0x80 else 1.0) *
                 (np.nan if c & 0x7F == 0x7F else
                  (c & 7) * 2.0 ** -9 if not (c >> 3) & 15 else (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7))
                 for c in range(256)])


def norm_rope(x, weight, eps, angles, interleaved):
    """x [T, H, D]; angles [T, rot] (cosines, then sines) or None.  Returns (y, m): the values and, per
    element, the sum of magnitudes that meet in it (for error bounds)."""
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight
    y, m = x.copy(), np.abs(x)
    if angles is not None:
        rot = angles.shape[1]
        c, s = angles[:, None, :rot // 2], angles[:, None, rot // 2:]
        ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        m[..., ia], m[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, m


def step_exponent(top):
    """The smallest e >= -126 with top <= 127 * 2^e; 0 for top = 0."""
    if not top > 0:
        return 0
    e = -126
    while top > 127 * 2.0 ** e:
        e += 1
    return e


def summarize(keys, most):
    """keys [B, D] of one block and head: (codes int8 [2, D], scale)."""
    lo, hi = np.zeros(keys.shape[1]), np.zeros(keys.shape[1])
    for d in range(keys.shape[1]):
        col = keys[:, d][~np.isnan(keys[:, d])]
        if col.size:
            lo[d], hi[d] = np.clip([col.min(), col.max()], -most, most)
    unit = 2.0 ** step_exponent(max(np.abs(lo).max(), np.abs(hi).max()))
    return np.stack([np.floor(lo / unit), np.ceil(hi / unit)]).astype(np.int8), unit


def scores(q, codes, scale, most):
    """q [G, D], codes [n, 2, D], scale [n]: the best bound over the group's heads, [n]."""
    q = np.clip(np.nan_to_num(q, nan=0.0, posinf=most, neginf=-most), -most, most)
    best = np.full(codes.shape[0], -np.inf)
    for row in q:
        unit = 2.0 ** step_exponent(np.abs(row).max())
        c = np.rint(row / unit)  # ties to even
        dot = np.maximum(c * codes[:, 0].astype(np.float64), c * codes[:, 1]).sum(1)
        best = np.maximum(best, dot * unit * scale)
    return best


def select(score, n, keep, first, last):
    """The chosen blocks of [0, n), ascending."""
    if n <= keep:
        return list(range(n))
    want = keep - first - last
    middle = sorted(range(first, n - last), key=lambda b: (-score[b], b))[:want]
    return sorted(list(range(first)) + middle + list(range(n - last, n)))


def attend(q, k, v, scale):
    """q [G, D], k and v [t, D]: softmax(scale q k) v; zeros for t = 0."""
    if not k.shape[0]:
        return np.zeros_like(q)
    s = scale * q @ k.T
    p = np.exp(s - s.max(1, keepdims=True))
    return p @ v / p.sum(1, keepdims=True)


def attend_bound(q, k, v, scale, split):
    """Largest error of a float32 computation of attend() whose weights carry a relative error of
    `split`: a dot product of D terms is off by at most D * 2^-23 times the sum of its magnitudes (each
    addition loses at most one unit in the last place, the accumulator may truncate), a score by
    |scale| times that (a negative scale makes no error negative), a weight by twice its score's error and
    its own rounding, the sums by one rounding a token."""
    if not k.shape[0]:
        return 0.0
    eps_s = q.shape[1] * 2.0 ** -23 * abs(scale) * (np.abs(q) @ np.abs(k).T).max()
    return np.abs(v).max() * (2 * eps_s + 2 * split + (k.shape[0] + 64) * 2.0 ** -23)
