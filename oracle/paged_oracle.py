"""float64 restatement of the uncompressed attention layers over a paged e4m3
cache: the page plan, the cache write, attention over packed prompts and
attention of single tokens over the cache. Plain loops over requests, pages,
heads and rows; nothing fused. Arrays are numpy; results are not rounded
(except to the cache's codes), so tests bound the kernels' roundings themselves.
"""

from __future__ import annotations

import numpy as np

from .cslc_oracle import e4m3_decode, e4m3_encode

F64 = np.float64
E_MIN, E_MAX = -40, 60


def page_plan(old_len, new_len, free_pages, table, page: int, n_pages: int, max_tokens: int):
    """(table, slots, cu, seq_len, status) after handing out pages; table is copied."""
    table = np.array(table, dtype=np.int32)
    width = table.shape[1]
    slots = np.full(max_tokens, -1, dtype=np.int32)
    cu, seq_len, used, lost = [0], [], 0, 0
    real = lambda p: 0 <= p < n_pages  # noqa: E731
    for b in range(len(old_len)):
        o, n = max(int(old_len[b]), 0), max(int(new_len[b]), 0)
        for j in range(-(-o // page), min(-(-(o + n) // page), width)):
            p = int(free_pages[used]) if used < len(free_pages) else -1
            table[b, j] = p if real(p) else -1
            used += 1
        for i in range(n):
            j, t = (o + i) // page, cu[-1] + i
            if j < width and real(table[b, j]):
                if t < max_tokens:
                    slots[t] = table[b, j] * page + (o + i) % page
            else:
                lost += 1
        cu.append(cu[-1] + n)
        seq_len.append(o + n)
    return (table, slots, np.array(cu, dtype=np.int32), np.array(seq_len, dtype=np.int32),
            np.array([used, lost], dtype=np.int32))


def scale_exponent(amax: float) -> int:
    """The smallest e in [-40, 60] with amax <= 448 * 2^e (60 when there is none)."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def encode(x):
    """e4m3 codes, round to nearest even; infinities saturate, NaN stays NaN."""
    x = np.asarray(x, dtype=F64)
    codes = e4m3_encode(np.nan_to_num(x, nan=0.0, posinf=1e30, neginf=-1e30))
    return np.where(np.isnan(x), (codes & 0x80) | 0x7F, codes).astype(np.uint8)


def page_write(x, slots, cache, scale):
    """One cache (keys or values) after the write: (codes, scales), both copies.
    x [T, Hkv, 128] (float64 of bf16), cache [n_pages, Hkv, P, 128], scale [n_pages, Hkv]."""
    cache, scale = np.array(cache), np.array(scale, dtype=F64)
    n_pages, Hkv, P, _ = cache.shape
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if not 0 <= s < n_pages * P:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % P != 0:
            n += 1
        p, o = divmod(s, P)
        for h in range(Hkv):
            run = np.asarray(x[t:t + n, h], dtype=F64)
            fin = np.abs(run[np.isfinite(run)])
            e = scale_exponent(float(fin.max()) if fin.size else 0.0)
            if o > 0:
                e_old = int(round(np.log2(scale[p, h])))
                if e > e_old:
                    cache[p, h, :o] = encode(e4m3_decode(cache[p, h, :o]) * 2.0 ** (e_old - e))
                e = max(e, e_old)
            cache[p, h, o:o + n] = encode(run * 2.0 ** -e)
            scale[p, h] = 2.0 ** e
        t += n
    return cache, scale


def attend_rows(q, k, v, scale: float):
    """One head: q [n, D], k / v [m, D], all of them visible. Returns (o, lse,
    a, s): a = the same average of |v|, s = the largest scale * sum |q||k| of a
    row (what a kernel's roundings are bounded by)."""
    s = scale * (q @ k.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(axis=1, keepdims=True)
    return (p @ v / l, (m + np.log(l))[:, 0], p @ np.abs(v) / l, scale * (np.abs(q) @ np.abs(k).T).max(axis=1))


def _empty(shape):
    o = np.zeros(shape)
    return o, np.full(shape[:-1], -np.inf), np.zeros(shape), np.zeros(shape[:-1])


def prompt_attention(q, k, v, cu_q, cu_k, scale: float, window: int = 0, rows=None):
    """q [Tq, H, D], k, v [Tk, Hkv, D]: (o, lse, a, s) as attend_rows, rows of no
    sequence NaN. `rows`: the packed rows to compute (others NaN)."""
    Tq, H, D = q.shape
    G = H // k.shape[1]
    out = [np.full((Tq, H, D), np.nan), np.full((Tq, H), np.nan), np.full((Tq, H, D), np.nan), np.full((Tq, H), np.nan)]
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            t = cu_q[b] + i
            if rows is not None and t not in rows:
                continue
            hi = i + nk - nq + 1
            lo = max(0, hi - window) if window else 0
            for h in range(H):
                if hi <= lo:
                    got = _empty((1, D))
                else:
                    j = slice(cu_k[b] + lo, cu_k[b] + hi)
                    got = attend_rows(q[t:t + 1, h], k[j, h // G], v[j, h // G], scale)
                for dst, x in zip(out, got):
                    dst[t, h] = x[0]
    return tuple(out)


def page_decode_attention(q, k_cache, v_cache, k_scale, v_scale, table, seq_len, scale: float, window: int = 0):
    """q [B, H, D]: (o, lse, a, s) as attend_rows over the stored values."""
    B, H, D = q.shape
    n_pages, Hkv, P, _ = k_cache.shape
    out = _empty((B, H, D))
    for b in range(B):
        n = min(max(int(seq_len[b]), 0), table.shape[1] * P)
        x = np.arange(max(0, n - window) if window else 0, n)
        p = table[b][x // P] if len(x) else np.zeros(0, dtype=np.int64)
        ok = (p >= 0) & (p < n_pages)
        x, p = x[ok], p[ok]
        if not len(x):
            continue
        for h in range(H):
            hk = h // (H // Hkv)
            k = e4m3_decode(k_cache[p, hk, x % P]) * k_scale[p, hk][:, None]
            v = e4m3_decode(v_cache[p, hk, x % P]) * v_scale[p, hk][:, None]
            for dst, y in zip(out, attend_rows(q[b:b + 1, h], k, v, scale)):
                dst[b, h] = y[0]
    return out
