"""Plain float64 references of the few-row product, the paged MXFP4 cache and
the attention over it, with numpy on the host.  Codes are read through the
oracle (mx_dequant, mx_quantize_f32)."""
import numpy as np

from oracle import oracle as O


def dequant(q, s):
    """float64 values of codes [..., d/2] and scales [..., d/32]."""
    q, s = np.asarray(q), np.asarray(s)
    d = q.shape[-1] * 2
    return O.mx_dequant(np.ascontiguousarray(q.reshape(-1, d // 2)),
                        np.ascontiguousarray(s.reshape(-1, d // 32))).reshape(*q.shape[:-1], d)


def quantize(x):
    """MXFP4 codes [..., d/2] and scales [..., d/32] of float32 values [..., d]."""
    x = np.ascontiguousarray(x, np.float32)
    d = x.shape[-1]
    q, s = O.mx_quantize_f32(x.reshape(-1, d))
    return q.reshape(*x.shape[:-1], d // 2), s.reshape(*x.shape[:-1], d // 32)


def slots(page_table, row_start, lengths, rows, pages, page_size):
    """(page, offset) of every row, or None for a row without a slot."""
    out = [None] * rows
    for i, length in enumerate(lengths):
        a, e = int(row_start[i]), int(row_start[i + 1])
        if a < 0 or e > rows or e <= a:
            continue
        for r in range(a, e):
            p = int(length) - e + r
            if 0 <= p < page_table.shape[1] * page_size:
                page = int(page_table[i, p // page_size])
                if 0 <= page < pages:
                    out[r] = (page, p % page_size)
    return out


def attention(q, kq, ks, vq, vs, page_table, row_start, lengths, scale, window=0, sinks=0):
    """(out, room), float64 [rows, q_heads, dim]: the attention of q (float64)
    over the cache, and how far a kernel may be from it that sums scores and
    outputs in fp32 and rounds the weights and the result to bf16.  Rows of no
    sequence are NaN.

    room = 2^-8 |o| (half a step of the result) + A (2^-8 + 2 e + n 2^-22),
    A = sum_j w_j |v_j|: half a step of each bf16 weight; e the error of a
    score as an exponent, (dim + 8) 2^-23 scale max_j sum_d |q_d k_jd|, which
    enters the weight and the sum it is divided by; n fp32 additions of each
    sum, an exp2 of about one step of 2^-23 among them.  Underflow: a weight
    below fp32's normal range (2^-126 before the division) may be flushed, and
    the largest weight, by which the sum is at least bounded, may be scaled to
    2^-8 only, so each v_j adds at most 2^-118 |v_j|."""
    rows, q_heads, dim = q.shape
    pages, heads, size, _ = kq.shape
    group = q_heads // heads
    out, room = np.full(q.shape, np.nan), np.zeros(q.shape)
    for i, length in enumerate(lengths):
        a, e = int(row_start[i]), int(row_start[i + 1])
        if a < 0 or e > rows or e <= a:
            continue
        span = min(max(int(length), 0), page_table.shape[1] * size)
        j = np.arange(span)
        pg = page_table[i, j // size].astype(np.int64)
        there = (pg >= 0) & (pg < pages)
        k, v = np.zeros((span, heads, dim)), np.zeros((span, heads, dim))
        if there.any():
            at, of = pg[there], (j % size)[there]
            k[there] = dequant(kq[at, :, of], ks[at, :, :, of])
            v[there] = dequant(vq[at, :, of], vs[at, :, :, of])
        for r in range(a, e):
            p = int(length) - e + r
            seen = there & (j <= p)
            if window:
                seen &= (p - j < window) | (j < sinks)
            at = np.flatnonzero(seen)
            if not at.size:
                out[r] = 0.0
                continue
            for h in range(heads):
                qs = q[r, h * group:(h + 1) * group]
                with np.errstate(invalid="ignore"):
                    s = scale * (qs @ k[at, h].T)
                    w = np.exp(s - s.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    o, big = w @ v[at, h], w @ np.abs(v[at, h])
                    err = (dim + 8) * 2.0 ** -23 * scale * (np.abs(qs) @ np.abs(k[at, h]).T).max(1, keepdims=True)
                out[r, h * group:(h + 1) * group] = o
                room[r, h * group:(h + 1) * group] = (2.0 ** -8 * np.abs(o)
                                                      + big * (2.0 ** -8 + 2 * err + at.size * 2.0 ** -22)
                                                      + 2.0 ** -118 * np.abs(v[at, h]).sum(0))
    return out, room
