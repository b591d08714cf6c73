"""CPU oracle of the text side's attention, numpy fp64: causal attention of
packed prompts with grouped heads, the paged 4-bit key/value cache, attention
over it, and eviction by summed weight. Plain and slow; shares no code with the
GPU path. The quantisation recipe is vlm_oracle.quantize_nvfp4.
"""
from __future__ import annotations

import numpy as np

from oracle import vlm_oracle as O

PAGE = 64
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def attend(q, k, v, scale, first):
    """q [m, d], k and v [n, d]: query i sees the keys j <= first + i. Returns
    (o [m, d], p [m, n], a [m, d]) with a = sum_j p_ij |v_j|, the size that
    rounding errors of P are relative to. A query that sees no key gives 0, and
    what a query does not see is not read."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    m, n = q.shape[0], k.shape[0]
    o, p, a = np.zeros((m, v.shape[1])), np.zeros((m, n)), np.zeros((m, v.shape[1]))
    see = np.arange(n)[None, :] <= first + np.arange(m)[:, None]
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(see, (q @ np.where(np.isfinite(k), k, 0.0).T) * scale, -np.inf)
    odd = ~np.isfinite(k).all(1) | ~np.isfinite(v).all(1)
    for i in range(m):
        c = int(np.clip(first + i + 1, 0, n))
        if c == 0:
            continue
        if odd[:c].any():
            with np.errstate(invalid="ignore", over="ignore"):
                row = (k[:c] @ q[i]) * scale
                e = np.exp(row - row.max())
                p[i, :c] = e / e.sum()
                o[i], a[i] = p[i, :c] @ v[:c], p[i, :c] @ np.abs(v[:c])
            continue
        e = np.exp(s[i, :c] - s[i, :c].max())
        p[i, :c] = e / e.sum()
        o[i], a[i] = p[i, :c] @ v[:c], p[i, :c] @ np.abs(v[:c])
    return o, p, a


def prompt_attention(q, k, v, q_lens, kv_lens, scale):
    """q [T, H, d], k and v [Tk, Hk, d] packed. Returns (o, a) [T, H, d]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    group = q.shape[1] // k.shape[1]
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    q0 = k0 = 0
    for m, n in zip(q_lens, kv_lens):
        for h in range(q.shape[1]):
            o[q0:q0 + m, h], _, a[q0:q0 + m, h] = attend(q[q0:q0 + m, h], k[k0:k0 + n, h // group],
                                                         v[k0:k0 + n, h // group], scale, n - m)
        q0, k0 = q0 + m, k0 + n
    return o, a


# ---------------------------------------------------------------------------
# The paged cache: a page of one head is key codes [64][d/2], value codes,
# key scales [64][d/16], value scales
# ---------------------------------------------------------------------------

def page_bytes(dim: int) -> int:
    return PAGE * (dim + dim // 8)


def _parts(dim: int):
    c, s = PAGE * dim // 2, PAGE * dim // 16
    return (0, c, dim // 2), (c, c, dim // 2), (2 * c, s, dim // 16), (2 * c + s, s, dim // 16)


def e4m3_bytes(x) -> np.ndarray:
    """Codes of non-negative E4M3 values."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    e = np.clip(e - 1, -6, 8)
    sub = x < 2.0 ** -6
    man = np.where(sub, x * 512.0, (x / np.ldexp(1.0, e) - 1.0) * 8.0)
    return (np.where(sub, 0, e + 7).astype(np.int64) * 8 + np.rint(man).astype(np.int64)).astype(np.uint8)


def e4m3_values(b) -> np.ndarray:
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, np.exp2(e - 7.0) * (1.0 + m / 8.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def quantise(x, sg):
    """Rows x [n, d] -> (code bytes [n, d/2], scale bytes [n, d/16])."""
    q, sb = O.quantize_nvfp4(np.asarray(x, np.float32), np.float32(sg))
    code = np.searchsorted(MAGNITUDES, np.abs(q)).astype(np.uint8) | (np.signbit(q) * 8).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), e4m3_bytes(sb)


def write(pages, table, s, first, k, v, k_sg, v_sg):
    """Rows k, v [n, Hk, d] into the places from `first` on of sequence s (pages modified in place)."""
    dim = k.shape[2]
    for h in range(k.shape[1]):
        rows = [quantise(k[:, h], k_sg), quantise(v[:, h], v_sg)]
        for t in range(k.shape[0]):
            page, r = pages[table[s, (first + t) // PAGE], h], (first + t) % PAGE
            for which in (0, 1):
                for part, data in ((which, rows[which][0]), (2 + which, rows[which][1])):
                    at, _, w = _parts(dim)[part]
                    page[at + r * w:at + (r + 1) * w] = data[t]


def read(pages, table, s, h, n, dim):
    """Places [0, n) of sequence s, key head h: (keys, values) [n, d] as code * scale."""
    out = []
    ids = np.asarray(table)[s, :-(-n // PAGE)]
    for which in (0, 1):
        at, c, w = _parts(dim)[which]
        codes = pages[ids, h, at:at + c].reshape(-1, w)[:n]
        nib = np.stack([codes & 15, codes >> 4], 2).reshape(n, dim)
        at, c, w = _parts(dim)[2 + which]
        sc = e4m3_values(pages[ids, h, at:at + c].reshape(-1, w)[:n])
        mag = MAGNITUDES[nib & 7]
        out.append(np.where(nib & 8, -mag, mag) * np.repeat(sc, 16, axis=1))
    return out


def cache_attention(pages, table, lens, q, q_len, k_sg, v_sg, scale):
    """q [S * q_len, H, d]. Returns (o, a [S * q_len, H, d], w [S, Hk, max_pages * 64], logit_err)
    where w sums each place's weights over the new tokens and the head's queries,
    and a is sum_j p |v_j|."""
    q = np.asarray(q, np.float64)
    S, kvh, dim = len(lens), pages.shape[1], q.shape[2]
    group = q.shape[1] // kvh
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    w = np.zeros((S, kvh, np.asarray(table).shape[1] * PAGE))
    ks, vs = np.float64(np.float32(k_sg)), np.float64(np.float32(v_sg))
    for s, n in enumerate(lens):
        for h in range(kvh):
            k, v = read(pages, table, s, h, n, dim)
            for g in range(group):
                rows = slice(s * q_len, (s + 1) * q_len)
                o[rows, h * group + g], p, a[rows, h * group + g] = attend(q[rows, h * group + g], k * ks, v * vs, scale,
                                                                           n - q_len)
                w[s, h, :n] += p.sum(0)
    return o, a, w


def keep(weights, n, budget, sinks, recent):
    """The places of one (sequence, head) that stay, in order."""
    if n <= budget:
        return np.arange(n)
    w = np.where(np.isnan(weights[:n]), -np.inf, np.asarray(weights[:n], np.float64) + 0.0)
    mid = np.arange(sinks, n - recent)
    nan = np.isnan(weights[mid])
    order = mid[np.lexsort((mid, -w[mid], nan))]  # numbers before NaN, larger first, lower place first
    best = order[:budget - sinks - recent]
    return np.sort(np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)]).astype(np.int64))
