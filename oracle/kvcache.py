"""The paged NVFP4 key/value cache, the attention over it and rotary positions.

Oracle module (test infrastructure only, see ``oracle/__init__``).

[TRACE] "Le problème", "Résultats": the rollout keeps weights, activations
and the KV cache in FP4.  The pages describe neither the cache nor the
attention; these are the plainest readings: values on the NVFP4 grid with one
decode scale per head, softmax attention with grouped query heads over a
sequence's cached tokens, rotary positions in pairs.

Caches are dicts of arrays: k_codes, v_codes [pages, heads, page_size, D]
(one code each), k_scales, v_scales [pages, heads, page_size, D / 16], g_k,
g_v [heads].
"""
import numpy as np

from . import nvfp4 as Q


def row_positions(row_off, kv_len):
    """(sequence, position) of every row of a call, in row order."""
    out = []
    for b in range(len(kv_len)):
        n = int(row_off[b + 1]) - int(row_off[b])
        out += [(b, int(kv_len[b]) - n + i) for i in range(n)]
    return out


def place(cache, table, b, pos):
    """(page, place in it) of a position, or None where it has no page."""
    n_pages, _, ps, _ = cache["k_codes"].shape
    if pos < 0 or pos // ps >= table.shape[1]:
        return None
    page = int(table[b, pos // ps])
    return (page, pos % ps) if 0 <= page < n_pages else None


def write(cache, k, v, row_off, kv_len, table):
    """Quantize k, v [rows, heads, D] into the cache (a copy is returned)."""
    c = {name: a.copy() for name, a in cache.items()}
    for r, (b, pos) in enumerate(row_positions(row_off, kv_len)):
        at = place(c, table, b, pos)
        if at is None:
            continue
        for x, name in ((k, "k"), (v, "v")):
            for h in range(x.shape[1]):
                codes, scales = Q.quantize_with_scale(x[r, h][None], c["g_" + name][h])
                c[name + "_codes"][at[0], h, at[1]] = codes[0]
                c[name + "_scales"][at[0], h, at[1]] = scales[0]
    return c


def token(cache, name, at, h):
    """float64 values of one cached key or value (zeros without a page)."""
    D = cache["k_codes"].shape[-1]
    if at is None:
        return np.zeros(D)
    return Q.dequant(cache[name + "_codes"][at[0], h, at[1]][None], cache[name + "_scales"][at[0], h, at[1]][None],
                     cache["g_" + name][h])[0]


def read(cache, row_off, table, start=None):
    """(k, v) float64 [rows, heads, D] of positions start[b] + i."""
    n, heads = int(row_off[-1]), cache["k_codes"].shape[1]
    out = [np.zeros((n, heads, cache["k_codes"].shape[-1])) for _ in range(2)]
    for b in range(len(row_off) - 1):
        for i in range(int(row_off[b + 1]) - int(row_off[b])):
            at = place(cache, table, b, (0 if start is None else int(start[b])) + i)
            for o, name in zip(out, "kv"):
                for h in range(heads):
                    o[int(row_off[b]) + i, h] = token(cache, name, at, h)
    return out[0], out[1]


def attention(q, cache, row_off, kv_len, table, scale, window=0):
    """By the definition, over the positions with a page up to a row's own and
    inside the window: out [rows, heads_q, D], lse [rows, heads_q], and what
    error bounds need: vabs, the softmax average of |v|, sabs, the largest scale *
    sum |q_i k_i| of a row, and vsum, the plain sum of |v|."""
    rows, hq, D = q.shape
    heads = cache["k_codes"].shape[1]
    out, lse, vabs = np.zeros((rows, hq, D)), np.full((rows, hq), -np.inf), np.zeros((rows, hq, D))
    sabs, vsum = np.zeros((rows, hq)), np.zeros((rows, hq, D))
    memo = {}
    for r, (b, pos) in enumerate(row_positions(row_off, kv_len)):
        js = [j for j in range(max(0, pos - window + 1) if window else 0, pos + 1)
              if place(cache, table, b, j) is not None]
        if not js:
            continue
        for h in range(heads):
            for j in js:
                if (b, j, h) not in memo:
                    at = place(cache, table, b, j)
                    memo[b, j, h] = token(cache, "k", at, h), token(cache, "v", at, h)
            k = np.stack([memo[b, j, h][0] for j in js])
            v = np.stack([memo[b, j, h][1] for j in js])
            for i in range(h * (hq // heads), (h + 1) * (hq // heads)):
                s = k @ q[r, i] * scale
                m = s.max()
                e = np.exp(s - m)
                out[r, i] = e @ v / e.sum()
                vabs[r, i] = e @ np.abs(v) / e.sum()
                lse[r, i] = m + np.log(e.sum())
                sabs[r, i] = (np.abs(k) @ np.abs(q[r, i])).max() * abs(scale)
                vsum[r, i] = np.abs(v).sum(0)
    return out, lse, vabs, sabs, vsum


def rope(x, positions, freq, interleaved=False, mscale=1.0, inverse=False):
    """x [rows, heads, D] with the first 2 * len(freq) elements of each head
    turned by positions * freq; float64."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(freq)
    for f in range(half):
        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        t = np.asarray(positions, dtype=np.float64) * freq[f] * (-1.0 if inverse else 1.0)
        c, s = mscale * np.cos(t)[:, None], mscale * np.sin(t)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y
