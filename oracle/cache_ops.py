"""fp64 oracle of the operators around the window attention: rotary positions, key weights,
eviction and draft verification. Plain loops over sequences and heads, no code shared with the
CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

from .pbd import _f64


# -------------------------------------------------------------------------- rotary positions
def rope_angles(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_max=1, low_turns=1.0,
                high_turns=32.0):
    """Angle per position of each of the rotary_dim / 2 pairs."""
    rd = rotary_dim
    if scaling == "base" and rd > 2:
        base = base * factor ** (rd / (rd - 2.0))
    out = []
    for i in range(rd // 2):
        w = math.exp(-2.0 * i / rd * math.log(base))
        if scaling == "linear":
            w /= factor
        elif scaling == "turns":
            n = original_max * w / (2 * math.pi)
            k = min(1.0, max(0.0, (n - low_turns) / (high_turns - low_turns)))
            w = k * w + (1 - k) * w / factor
        elif scaling == "pairs":
            def pair(turns):
                return rd * math.log(original_max / (2 * math.pi * turns)) / (2 * math.log(base))
            lo = max(0, math.floor(pair(high_turns)))
            hi = min(rd - 1, math.ceil(pair(low_turns)))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = (1 - r) * w + r * w / factor
        out.append(w)
    return np.array(out)


def rotate(x, positions, angles, layout="half", out_scale=1.0, inverse=False):
    """x [..., H, D] turned by positions [...]."""
    x = _f64(x)
    y = x.copy()
    half = len(angles)
    a = np.asarray(positions, dtype=np.float64)[..., None, None] * angles
    c, s = out_scale * np.cos(a), (-out_scale if inverse else out_scale) * np.sin(a)
    first, second = ((slice(0, half), slice(half, 2 * half)) if layout == "half"
                     else (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


# -------------------------------------------------------------------------- key weights
def key_weights(q, k_cache, seq_lens, window_lens, scale, weights_in=None, decay=1.0, mask="pbd"):
    """Attention weight per key, summed over the rows that share its KV head: [B, Hkv, S]; NaN where
    nothing is written."""
    q, k = _f64(q), _f64(k_cache)
    B, _, Hq, _ = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = np.full((B, Hkv, S), np.nan)
    for b in range(B):
        P, W = int(seq_lens[b]), int(window_lens[b])
        n = P + W
        for h in range(Hkv):
            total = np.zeros(n)
            for i in range(W):
                see = P + i + 1 if mask == "causal" else n
                for g in range(G):
                    s = scale * (k[b, h, :see] @ q[b, i, h * G + g])
                    e = np.exp(s - s.max())
                    total[:see] += e / e.sum()
            if weights_in is not None:
                total[:P] += decay * _f64(weights_in)[b, h, :P]
            out[b, h, :n] = total
    return out


# -------------------------------------------------------------------------- eviction
def evict(weights, positions, n, next_pos, budget, sink, recent):
    """Slots that stay for one (sequence, KV head) of n keys: source slot of each slot below
    min(n, budget)."""
    weights = np.asarray(weights, dtype=np.float64)[:n]
    keep = min(n, budget)

    def order(j):
        t = int(positions[j])
        safe = t < sink or t >= next_pos - recent
        w = weights[j] if not math.isnan(weights[j]) else -math.inf
        return (not safe, 0.0 if safe else -w, j)

    stay = set(sorted(range(n), key=order)[:keep])
    movers = iter(sorted(j for j in stay if j >= keep))
    return [j if j in stay else next(movers) for j in range(keep)]


# -------------------------------------------------------------------------- draft verification
def verify(p, q, drafts, u, sample_u):
    """One sequence: p [k + 1, V], q [k, V] or None, drafts [k]. Returns (tokens, accepted)."""
    p = _f64(p)
    V = p.shape[1]
    q = None if q is None else _f64(q)
    n = 0
    while n < len(drafts):
        x = int(drafts[n])
        qx = 1.0 if q is None else (q[n, x] if 0 <= x < V else 1.0)
        if not (0 <= x < V and float(u[n]) * qx < p[n, x]):
            break
        n += 1
    row = np.where(p[n] > 0, p[n], 0.0)
    if n < len(drafts):
        if q is None:
            rest = row.copy()
            if 0 <= int(drafts[n]) < V:
                rest[int(drafts[n])] = 0.0
        else:
            with np.errstate(invalid="ignore"):
                rest = p[n] - q[n]
            rest = np.where(rest > 0, rest, 0.0)
        if rest.sum() > 0:
            row = rest
    total = row.sum()
    if not (total > 0 and math.isfinite(total)):
        token = -1
    else:
        cum = np.cumsum(row)
        above = np.nonzero(cum > float(sample_u) * cum[-1])[0]
        token = int(above[0]) if len(above) else int(np.nonzero(row)[0][-1])
    return [int(x) for x in drafts[:n]] + [token], n
