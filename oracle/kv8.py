"""8-bit K/V cache with a scale for each block of tokens and head, fp64 reference.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Source: HLA summary, "Conclusion / Future directions" (latent caches combined
with quantisation and token eviction); the pages give no format.  Reading:

* Quantisation of a block of tokens of one head: s = amax / top (top = 127 for
  int8, 448 for e4m3) and code = x / s rounded to nearest-even, both quotients
  in binary32.  All zeros: s = 0, zero codes.  An infinity or a NaN in it:
  s = NaN, zero codes.
* Attention: one softmax over the cached tokens and the exact tokens that a
  query sees; no token: zeros.
* Eviction: the first and the last blocks stay, and of the others those whose
  weights sum highest (fp64 sum, rounded to binary32; NaN lowest; ties: the
  lowest block), in order.
"""

import math

import numpy as np

from .quant import to_e4m3

TOP = {"e4m3": 448.0, "i8": 127.0}


def quantise_block(x, code):
    """x [tokens, d] float32 -> codes (as values, fp64) [tokens, d], scale (float32)."""
    x = np.asarray(x, dtype=np.float32)
    if x.size == 0:
        return np.zeros(x.shape), np.float32(0)
    if not np.all(np.isfinite(x)):
        return np.zeros(x.shape), np.float32(np.nan)
    s = np.float32(np.max(np.abs(x)) / np.float32(TOP[code]))
    if s == 0:
        return np.zeros(x.shape), np.float32(0)
    with np.errstate(over="ignore"):
        y = (x / s).astype(np.float32).astype(np.float64)
    if code == "i8":
        return np.clip(np.round(y), -127, 127), s
    return to_e4m3(np.clip(y, -448, 448)), s


def write(x, block, code):
    """x [n, d] float32 of one head -> codes [n, d], scales [ceil(n / block)]."""
    codes, scales = [], []
    for t in range(0, len(x), block):
        c, s = quantise_block(x[t:t + block], code)
        codes.append(c)
        scales.append(s)
    return (np.concatenate(codes) if codes else np.zeros(x.shape)), np.array(scales, dtype=np.float32)


def values(codes, scales, block):
    """The values that codes [n, d] under scales [>= ceil(n / block)] stand for."""
    n = codes.shape[0]
    return np.asarray(codes, dtype=np.float64) * np.asarray(scales, dtype=np.float64)[np.arange(n) // block, None]


def attend(q, k, v, scale=0.0):
    """q [d], k, v [n, d] -> (o [d], weights [n])."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), np.zeros(0)
    s = k @ q * (scale if scale > 0 else 1.0 / math.sqrt(len(q)))
    a = np.exp(s - s.max())
    a = a / a.sum()
    return a @ v, a


def ring_rows(ring, ctx, tail):
    """Rows of the last `tail` positions of a context of ctx tokens: [tail, ...], oldest first."""
    return ring[[(ctx - tail + i) % len(ring) for i in range(tail)]]


def attn(q, k, v, win_k, win_v, scale=0.0):
    """One sequence.  q [nq, H, G, d]; k, v [H, n, d] cached values; win_k, win_v [tail, H, d] exact rows, oldest
    first, the last of them at the last query's position -> out [nq, H, G, d], weights [H, n] summed over queries."""
    nq, H, G, d = q.shape
    n, tail = k.shape[1], len(win_k)
    out, weights = np.zeros((nq, H, G, d)), np.zeros((H, n))
    for p in range(nq):
        see = max(0, tail - (nq - 1 - p))
        for h in range(H):
            kk, vv = np.concatenate([k[h], win_k[:see, h]]), np.concatenate([v[h], win_v[:see, h]])
            for g in range(G):
                out[p, h, g], a = attend(q[p, h, g], kk, vv, scale)
                weights[h] += a[:n]
    return out, weights


def choose(weights, length, block, keep, first, last):
    """Source blocks that one head keeps, in order; weights [>= length] float32."""
    nb = -(-length // block)
    if nb <= keep:
        return list(range(nb))
    mass = []
    for i in range(first, nb - last):
        s = np.float32(math.fsum(float(x) for x in weights[i * block:(i + 1) * block])) \
            if not np.any(np.isnan(weights[i * block:(i + 1) * block])) else np.float32(-np.inf)
        mass.append((-float(s), i))
    best = sorted(mass)[:keep - first - last]
    return sorted(list(range(first)) + [i for _, i in best] + list(range(nb - last, nb)))
