"""Plain numpy implementation of the 8-bit floating-point products, the routing to experts and the
experts' layer (include/pdq.h).

Shares no code with the HIP path.  Codes and scales follow from exact steps (powers of two, one
rounding to e4m3), everything else is computed in binary64.
"""
import numpy as np

GROUP = 128


def e4m3(v):
    """v (|v| <= 448) rounded to the nearest e4m3 value, ties to even, as float64."""
    v = np.asarray(v, np.float64)
    exponent = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (exponent - 3)
    return np.rint(v / step) * step


def e4m3_bits(v):
    """The codes (uint8) of e4m3 values; a zero's sign is kept."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    exponent = np.floor(np.log2(np.maximum(a, 2.0 ** -6))).astype(int)
    small = a < 2.0 ** -6
    mant = np.where(small, np.rint(a * 512), np.rint((a / 2.0 ** exponent - 1) * 8)).astype(int)
    bits = np.where(small, mant, ((exponent + 7) << 3) + mant)
    return (bits | (np.signbit(v).astype(int) << 7)).astype(np.uint8)


def scale_byte(top):
    """The e8m0 byte of groups whose largest magnitude is `top` (NaN or infinite: 255)."""
    top = np.asarray(top, np.float64)
    m, e = np.frexp(np.where(np.isfinite(top), top, 1.0))
    p = e - 9 + (m > 0.875)
    b = np.clip(p + 127, 0, 254)
    return np.where(~np.isfinite(top), 255, np.where(top == 0, 127, b)).astype(np.uint8)


def scale_value(b):
    b = np.asarray(b)
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))


def _coded(v, b):
    s = scale_value(b)
    with np.errstate(invalid="ignore"):
        return np.where(b == 255, 0.0, e4m3(np.where(b == 255, 0.0, v) / np.where(b == 255, 1.0, s)))


def quantize(x):
    """x [rows, k] -> (code values [rows, k], scale bytes [rows, k / 128])."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    g = -(-k // GROUP)
    v = np.zeros((rows, g * GROUP))
    v[:, :k] = x
    v = v.reshape(rows, g, GROUP)
    b = scale_byte(np.abs(v).max(2))
    return _coded(v, b[..., None]).reshape(rows, -1)[:, :k], b


def quantize_weight(w):
    """w [n, k] -> (code values [n, k], scale bytes [n / 128, k / 128])."""
    w = np.asarray(w, np.float64)
    n, k = w.shape
    nb, g = -(-n // GROUP), -(-k // GROUP)
    v = np.zeros((nb * GROUP, g * GROUP))
    v[:n, :k] = w
    v = v.reshape(nb, GROUP, g, GROUP)
    b = scale_byte(np.abs(v).max((1, 3)))
    return _coded(v, b[:, None, :, None]).reshape(nb * GROUP, -1)[:n, :k], b


def spread(scale, n, k, rows=GROUP):
    """Block scales as a full matrix."""
    return np.repeat(np.repeat(np.asarray(scale, np.float64), rows, 0), GROUP, 1)[:n, :k]


def values(x):
    """What x's codes and scales stand for."""
    q, b = quantize(x)
    return q * spread(scale_value(b), *q.shape, rows=1)


def linear(x, wq, w_scale, bias=None):
    """x [m, k]; wq code values [n, k], w_scale [n / 128, k / 128] -> (y, the products' magnitudes summed, the
    largest magnitude of each eight neighbouring K values summed)."""
    v = values(x)
    w = np.asarray(wq, np.float64) * spread(w_scale, *np.shape(wq))
    y = v @ w.T
    size = np.abs(v) @ np.abs(w).T
    aligned = np.zeros_like(y)
    for a in range(0, v.shape[1], 8):
        aligned += np.max([np.abs(np.outer(v[:, j], w[:, j])) for j in range(a, a + 8)], 0)
    return (y, size, aligned) if bias is None else (y + bias, size + np.abs(bias), aligned)


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_score=1, renormalize=True, scale=1.0):
    """-> ids [tokens, k], weights [tokens, k], offsets, rows."""
    z = np.asarray(logits, np.float64)
    tokens, experts = z.shape
    size = experts // groups
    ids = np.full((tokens, k), -1, np.int64)
    weights = np.zeros((tokens, k))
    for t in range(tokens):
        row = z[t]
        nan = np.isnan(row).any()
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                p = 1 / (1 + np.exp(-row))
            else:
                top = np.max(np.where(np.isnan(row), -np.inf, row))
                p = np.where(row == top, 1.0, np.exp(row - top))
                p[row == -np.inf] = 0.0
                p = p / p.sum()
            c = row if bias is None else p + np.asarray(bias, np.float64)
        there = (row != -np.inf) & (c != -np.inf)
        number = there & ~np.isnan(c)
        if groups > 1:
            by = p if bias is None else c
            best = []
            for g in range(groups):
                v = sorted((by[e] for e in range(g * size, (g + 1) * size) if number[e]), reverse=True)[:group_score]
                best.append(sum(v) if v else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            there &= np.isin(np.arange(experts) // size, kept)
        order = sorted((e for e in range(experts) if there[e]), key=lambda e: (not number[e], -c[e] if number[e] else 0.0, e))
        chosen = order[:k]
        w = p[chosen]
        if renormalize and len(chosen):
            total = w.sum()
            w = w / total if total > 0 else np.zeros_like(w) if total == 0 else np.full_like(w, np.nan)
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = np.nan if nan else w * scale
    return (ids, weights, *sort_rows(ids, experts))


def sort_rows(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    rows = np.concatenate([np.flatnonzero(flat == e) for e in range(experts)])
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])])
    return offsets, np.concatenate([rows, np.full(flat.size - rows.size, -1)]).astype(np.int64)


def silu_mul(gate, up):
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up


def experts(x, ids, weights, gate_up, gate_up_scale, down, down_scale):
    """gate_up code values [experts, 2, inner, hidden], down [experts, hidden, inner] with their block
    scales -> (y [tokens, hidden], the sum of magnitudes that its error is counted in)."""
    v = values(x)
    y, size = np.zeros_like(v), np.zeros_like(v)
    for t in range(v.shape[0]):
        for e, w in zip(ids[t], weights[t]):
            if e < 0:
                continue
            gate, up = (gate_up[e, i] * spread(gate_up_scale[e, i], *gate_up.shape[2:]) for i in range(2))
            d = down[e] * spread(down_scale[e], *down.shape[1:])
            h = values(silu_mul(v[t] @ gate.T, v[t] @ up.T)[None])[0]
            y[t] += w * (d @ h)
            size[t] += np.abs(w) * (np.abs(d) @ np.abs(h))
    return y, size
