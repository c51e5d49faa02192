"""Plain 64-bit forms of what a step does around the cache: rotation, the
latent's norm, the rows of each kind, and attention over page-scaled rows.
Written from the definitions in include/mla.h; shares no code with the library."""
import math

import numpy as np

TURN = 1 << 64


def steps_of(freq):
    """int64 steps of frequencies in radians a position."""
    t = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % TURN for f in freq]
    return np.array([x - TURN if x >= TURN // 2 else x for x in t], dtype=np.int64)


def angles(pos, steps):
    """Radians [T, P], the product taken modulo a turn in whole numbers."""
    with np.errstate(over="ignore"):
        turn = np.asarray(pos, dtype=np.int64)[:, None] * np.asarray(steps, dtype=np.int64)[None]  # wraps modulo 2^64
    return turn.astype(np.float64) / 2.0 ** 64 * (2 * math.pi)


def rope(x, pos, steps, interleaved, mscale=1.0):
    """x [T, H, R] float64."""
    a = angles(pos, steps)[:, None, :]
    c, s = np.cos(a) * mscale, np.sin(a) * mscale
    out = np.empty_like(x)
    h = x.shape[-1] // 2
    ia, ib = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, h), slice(h, None))
    out[..., ia] = x[..., ia] * c - x[..., ib] * s
    out[..., ib] = x[..., ia] * s + x[..., ib] * c
    return out


def norm(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def page_scale(top):
    """The least power of two s with top <= 448 s, not below 2^-40."""
    s = 2.0 ** -40
    while top > 448 * s and s < 2.0 ** 40:
        s *= 2
    return s


def e4m3_off(x, scale):
    """How far the e4m3 code of x / scale, times scale, may be from x: half a step."""
    return np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)


def decode_page(q, rows, scale, q_len, Hq):
    """One request: q [q_len * Hq, 576], rows [T, 576] (codes times their page's
    scale), float64. out [q_len * Hq, 512], lse."""
    T = rows.shape[0]
    out, lse = np.zeros((q.shape[0], 512)), np.full(q.shape[0], -np.inf)
    for r in range(q.shape[0]):
        see = T - q_len + r // Hq + 1
        if see <= 0:
            continue
        z = rows[:see] @ q[r] * scale
        top = z.max()
        p = np.exp(z - top)
        out[r] = p @ rows[:see, :512] / p.sum()
        lse[r] = top + math.log(p.sum())
    return out, lse
