"""Float64 statements of the rotation, the paged e4m3 cache and attention over
it, and sliding-window attention with its gradient.

Written from the definitions in include/fa.h, in plain NumPy; nothing of the
CUDA path is used. ``rotate_f32`` and ``append_f32`` follow the one place where
the interface fixes 32-bit arithmetic: products and sums of the rotation are
rounded one by one, so that codes and scales can be compared for equality.
"""

from __future__ import annotations

import numpy as np

E_MIN, E_MAX = -100, 120


def pair_columns(rot: int, interleaved: bool):
    half = rot // 2
    i = np.arange(half)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + half)


def cos_sin(table, positions, sections):
    """Cosine and sine of each token's pairs: table [rows, rot], positions [axes, T]."""
    half = table.shape[1] // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    assert axis.size == half
    rows = positions[axis].T  # [T, half]
    i = np.arange(half)
    return table[rows, i], table[rows, i + half]


def rotate(x, table, positions, sections, interleaved=False, inverse=False, dtype=np.float64):
    """x [T, H, d] rotated in ``dtype`` arithmetic, one rounding per operation."""
    x = x.astype(dtype)
    c, s = cos_sin(table, positions, sections)
    c, s = c.astype(dtype)[:, None], s.astype(dtype)[:, None]
    if inverse:
        s = -s
    a, b = pair_columns(table.shape[1], interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def e4m3_values():
    """The value of each of the 256 e4m3 codes (bias 7, no infinities)."""
    v = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        e, m = (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            v[code] = np.nan
        elif e == 0:
            v[code] = sign * m * 2.0 ** -9
        else:
            v[code] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return v


VALUES = e4m3_values()


def encode_e4m3(x):
    """Nearest e4m3 code of |x| <= 448 (ties to the even code), as uint8."""
    x = np.asarray(x, dtype=np.float64)
    grid = VALUES[:127]  # 0 .. 448, ascending
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def block_exponent(amax: float) -> int:
    """The least e with amax <= 448 * 2^e, within the range of a scale."""
    if not amax > 0:
        return E_MIN
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(x, codes, scale, page_table, cu, lens, page_size):
    """New rows x [T, Hkv, d] (already rotated) into codes [P, Hkv, page, d] and scale [P, Hkv], in
    place: block by block, token order."""
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        start = lens[b] - n
        done = 0
        while done < n:
            blk, lo = divmod(start + done, page_size)
            count = min(page_size - lo, n - done)
            new = x[cu[b] + done: cu[b] + done + count]
            pg = page_table[b, blk]
            for h in range(x.shape[1]):
                s = 2.0 ** block_exponent(float(np.abs(new[:, h]).max()))
                if lo > 0:
                    old = float(scale[pg, h])
                    s = max(s, old)
                    if s > old:
                        codes[pg, h, :lo] = encode_e4m3(VALUES[codes[pg, h, :lo]] * (old / s))
                codes[pg, h, lo: lo + count] = encode_e4m3(new[:, h].astype(np.float64) / s)
                scale[pg, h] = s
            done += count


def visible(n, m, window, sinks):
    """[n, m] mask of n queries at the end of m keys."""
    p = np.arange(n)[:, None] + (m - n)
    j = np.arange(m)[None, :]
    seen = j <= p
    if window > 0:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attend(q, k, v, scale, window, sinks):
    """One head: (o, lse, weights); rows that see nothing give 0 and -inf."""
    seen = visible(q.shape[0], k.shape[0], window, sinks)
    s = np.where(seen, (q @ k.T) * scale, -np.inf)
    top = s.max(1, keepdims=True) if s.shape[1] else np.full((s.shape[0], 1), -np.inf)
    ref = np.where(np.isneginf(top), 0.0, top)
    p = np.exp(s - ref)
    l = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (ref + np.log(l))[:, 0]
    w = p / np.where(l > 0, l, 1.0)
    # A weight of zero contributes nothing, whatever the value is.
    o = w @ np.where(seen.any(0)[:, None], v, 0.0)
    return o, lse, w


def paged(q, k_codes, v_codes, k_scale, v_scale, page_table, cu, lens, scale, window=0, sinks=0):
    """q [T, H, d] over the cache: (o [T, H, d], lse [H, T], a [T, H, d] = sum of weight * |value|)."""
    T, H, d = q.shape
    Hkv, page = k_codes.shape[1], k_codes.shape[2]
    o, lse, a = np.zeros((T, H, d)), np.full((H, T), np.nan), np.zeros((T, H, d))
    for b in range(len(lens)):
        pages = page_table[b, : -(-lens[b] // page)]
        for h in range(H):
            c = h // (H // Hkv)
            k = (VALUES[k_codes[pages, c]] * k_scale[pages, c].astype(np.float64)[:, None, None]).reshape(-1, d)[: lens[b]]
            v = (VALUES[v_codes[pages, c]] * v_scale[pages, c].astype(np.float64)[:, None, None]).reshape(-1, d)[: lens[b]]
            rows = slice(cu[b], cu[b + 1])
            oo, ll, w = attend(q[rows, h].astype(np.float64), k, v, scale, window, sinks)
            o[rows, h], lse[h, rows], a[rows, h] = oo, ll, w @ np.nan_to_num(np.abs(v))
    return o, lse, a


def window_forward(q, k, v, scale, window, sinks):
    """q [B, H, N, d], k and v [B, Hkv, M, d]: (o, lse)."""
    B, H = q.shape[:2]
    g = H // k.shape[1]
    o, lse = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        for h in range(H):
            o[b, h], lse[b, h], _ = attend(q[b, h], k[b, h // g], v[b, h // g], scale, window, sinks)
    return o, lse


def window_backward(q, k, v, dout, scale, window, sinks):
    """(dq, dk, dv) of sum(o * dout); the gradients of a shared head are summed over its group."""
    B, H = q.shape[:2]
    g = H // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        for h in range(H):
            c = h // g
            o, _, w = attend(q[b, h], k[b, c], v[b, c], scale, window, sinks)
            do = dout[b, h]
            ds = w * (do @ v[b, c].T - (do * o).sum(1, keepdims=True))
            dq[b, h] = ds @ k[b, c] * scale
            dk[b, c] += ds.T @ q[b, h] * scale
            dv[b, c] += w.T @ do
    return dq, dk, dv


def packed_forward(q, k, v, cu_q, cu_k, scale, window=0, sinks=0):
    """q [T, H, d], k and v [S, Hkv, d], sequences at cu_q and cu_k: (o, lse [H, T], a = sum of weight * |value|)."""
    T, H, d = q.shape
    g = H // k.shape[1]
    o, lse, a = np.zeros((T, H, d)), np.full((H, T), -np.inf), np.zeros((T, H, d))
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(H):
            o[rows, h], lse[h, rows], w = attend(q[rows, h], k[keys, h // g], v[keys, h // g], scale, window, sinks)
            a[rows, h] = w @ np.abs(v[keys, h // g])
    return o, lse, a


def packed_backward(q, k, v, dout, cu_q, cu_k, scale, window=0, sinks=0):
    """(dq, dk, dv) of sum(o * dout); the gradients of a shared head are summed over its group."""
    g = q.shape[1] // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(q.shape[1]):
            c = h // g
            o, _, w = attend(q[rows, h], k[keys, c], v[keys, c], scale, window, sinks)
            do = dout[rows, h]
            ds = w * (do @ v[keys, c].T - (do * o).sum(1, keepdims=True))
            dq[rows, h] = ds @ k[keys, c] * scale
            dk[keys, c] += ds.T @ q[rows, h] * scale
            dv[keys, c] += w.T @ do
    return dq, dk, dv


def read(codes, scale, page_table, starts, lengths, page_size):
    """Cached values [T, Hkv, d] of tokens starts[b] .. starts[b] + lengths[b] - 1 of each sequence b, one behind the other."""
    rows = []
    for b, (s, n) in enumerate(zip(starts, lengths)):
        for j in range(s, s + n):
            pg = page_table[b, j // page_size]
            rows.append(VALUES[codes[pg, :, j % page_size]] * scale[pg].astype(np.float64)[:, None])
    return np.array(rows).reshape(len(rows), codes.shape[1], codes.shape[3])
