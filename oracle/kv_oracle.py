"""Plain numpy implementation of the INT8 key/value cache: appending to it and
attention over it (include/pdq.h, pdq_kv_append and pdq_kv_attention).

Shares no code with the HIP path.  Where floating point decides an integer (the
codes) the steps are taken in binary32, one rounding an operation, as the
definition says; attention is computed in binary64.

A cache here is a dict: k, v int8 [pages, heads, page, dim] (both plain: the
device's order of v is plain_v / device_v), k_scale, v_scale float32 [pages, heads].
"""
import numpy as np

F = np.float32
MIN_SCALE = F(2.0 ** -64)


def device_v(v):
    """[pages, heads, page, dim] -> [pages, heads, page / 4, dim, 4]."""
    p, h, t, d = v.shape
    return np.ascontiguousarray(v.reshape(p, h, t // 4, 4, d).transpose(0, 1, 2, 4, 3))


def plain_v(v):
    p, h, t, d, _ = v.shape
    return np.ascontiguousarray(v.transpose(0, 1, 2, 4, 3).reshape(p, h, 4 * t, d))


def rotate(x, pos, cos, sin, interleaved):
    """x float32 [heads, dim] at position pos: the first 2 * cos.shape[1] channels rotated."""
    x = np.array(x, F)
    half = cos.shape[1]
    if not 0 <= pos < cos.shape[0]:
        x[:, :2 * half] = np.nan
        return x
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    u, w, c, s = x[:, a].copy(), x[:, b].copy(), cos[pos], sin[pos]
    x[:, a] = u * c - w * s
    x[:, b] = w * c + u * s
    return x


def rows_of(seq_len, cu_q, tokens):
    """(sequence, row, position) of every new row."""
    for s, n in enumerate(seq_len):
        lo, hi = (s, s + 1) if cu_q is None else (cu_q[s], cu_q[s + 1])
        for t in range(lo, min(hi, tokens)):
            yield s, t, int(n) - (hi - t)


def append(cache, table, seq_len, cu_q, k, v, q=None, cos=None, sin=None, interleaved=False, q_out=None):
    """In place on cache (and q_out, the rotated queries in float32)."""
    pages, heads, page, dim = cache["k"].shape
    touched = {}
    with np.errstate(invalid="ignore", over="ignore"):
        for s, t, pos in rows_of(seq_len, cu_q, len(k)):
            kr, vr = np.array(k[t], F), np.array(v[t], F)
            if cos is not None:
                kr = rotate(kr, pos, cos, sin, interleaved)
                if q is not None:
                    q_out[t] = rotate(q[t], pos, cos, sin, interleaved)
            j = pos // page
            if 0 <= pos < table.shape[1] * page and 0 <= table[s, j] < pages:
                touched.setdefault((s, int(table[s, j])), []).append((pos % page, kr, vr))
        for (_, p), new in touched.items():
            first = new[0][0]
            for name, which in (("k", 1), ("v", 2)):
                codes, scale = cache[name], cache[name + "_scale"]
                for h in range(heads):
                    x = np.stack([n[which][h] for n in new])
                    held = scale[p, h] if first > 0 else F(0)
                    if not np.isfinite(x).all() or not np.isfinite(held):
                        scale[p, h] = np.nan
                        codes[p, h, first:first + len(new)] = 0
                        continue
                    now = max(held, max(np.abs(x).max() * (F(1) / F(127)), MIN_SCALE))
                    if first > 0 and now > held:
                        codes[p, h, :first] = np.rint(codes[p, h, :first].astype(F) * (held / now))
                    codes[p, h, first:first + len(new)] = np.clip(np.rint(x / now), -127, 127)
                    scale[p, h] = now


def attention(cache, table, seq_len, cu_q, q, scale, softcap=0.0, window=0, slopes=None, prefix=None):
    """float64 (y [tokens, hq, dim], lse [tokens, hq], what |y| would be with every value's magnitude, the
    largest sum of |scale q k| of a row); rows of no sequence are NaN."""
    pages, heads, page, dim = cache["k"].shape
    tokens, hq, _ = q.shape
    y, mag = np.full((tokens, hq, dim), np.nan), np.full((tokens, hq, dim), np.nan)
    lse, big = np.full((tokens, hq), np.nan), np.zeros((tokens, hq))
    known = {}
    for s, t, pos in rows_of(seq_len, cu_q, tokens):
        if s not in known:
            n = min(int(seq_len[s]), table.shape[1] * page)
            ids = table[s, :(n + page - 1) // page].astype(np.int64)
            ok = np.repeat((ids >= 0) & (ids < pages), page)[:n]
            safe = np.where((ids >= 0) & (ids < pages), ids, 0)
            kv = []
            for name in ("k", "v"):
                c = cache[name][safe].astype(np.float64) * cache[name + "_scale"][safe].astype(np.float64)[..., None, None]
                kv.append(c.transpose(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n])
            known[s] = (n, ok, *kv)
        n, ok, k, v = known[s]
        key = np.arange(n)
        last = pos if prefix is None else max(pos, int(prefix[s]) - 1)
        seen = ok & (key <= last)
        if window:
            seen &= key > pos - window
        for h in range(hq):
            g = h // (hq // heads)
            kk, vv = k[g][seen], v[g][seen]
            if not len(kk):
                y[t, h], mag[t, h], lse[t, h] = 0, 0, -np.inf
                continue
            qq = q[t, h].astype(np.float64)
            z = kk @ qq * scale
            big[t, h] = (np.abs(kk) @ np.abs(qq)).max() * abs(scale)
            if softcap:
                z = softcap * np.tanh(z / softcap)
            if slopes is not None:
                z = z + float(slopes[h]) * (key[seen] - pos)
                big[t, h] += np.abs(float(slopes[h]) * (key[seen] - pos)).max()
            top = z.max()
            e = np.exp(z - top)
            lse[t, h] = top + np.log(e.sum())
            y[t, h] = e @ vv / e.sum()
            mag[t, h] = e @ np.abs(vv) / e.sum()
    return y, lse, mag, big
