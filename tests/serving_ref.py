"""Plain float64 references of the few-row product, the paged MXFP4 cache and
the attention over it, with numpy on the host.  Codes are read through the
oracle (oracle.mx_dequant, oracle.mx_quantize_f32)."""
import numpy as np

from oracle import oracle as O


def bf16_round(a):
    """float64 -> the nearest bf16 value (ties to even), as float64."""
    flat = np.asarray(a, np.float64).reshape(-1)
    bits = np.array([O.lib().oracle_double_to_bf16(float(v)) for v in flat], np.uint16)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(np.shape(a))


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


def cache_values(codes, scales, page, off):
    """float64 [heads, dim] of one position."""
    return dequant(codes[page, :, off], scales[page, :, :, off])


def attention(q, kq, ks, vq, vs, page_table, row_start, lengths, scale, window, sinks):
    """float64 [rows, q_heads, dim]; rows of no sequence are NaN.  q is
    float64 [rows, q_heads, dim].  The scores and sums of one row at a time."""
    rows, q_heads, dim = q.shape
    pages, heads, size, _ = kq.shape
    group = q_heads // heads
    out = np.full(q.shape, np.nan)
    for i, length in enumerate(lengths):
        a, e = int(row_start[i]), int(row_start[i + 1])
        if a < 0 or e > rows or e <= a:
            continue
        span = min(max(int(length), 0), page_table.shape[1] * size)
        where = [(int(page_table[i, p // size]), p % size) for p in range(span)]
        there = np.array([0 <= pg < pages for pg, _ in where], bool)
        k = np.zeros((span, heads, dim))
        v = np.zeros((span, heads, dim))
        if there.any():
            pg = np.array([w[0] for w in where])[there]
            of = np.array([w[1] for w in where])[there]
            k[there] = dequant(kq[pg, :, of], ks[pg, :, :, of])
            v[there] = dequant(vq[pg, :, of], vs[pg, :, :, of])
        j = np.arange(span)
        for r in range(a, e):
            p = int(length) - e + r
            seen = there & (j <= p)
            if window:
                seen &= (p - j < window) | (j < sinks)
            at = np.flatnonzero(seen)
            if not at.size:
                out[r] = 0.0
                continue
            for h in range(q_heads):
                s = scale * (k[at, h // group] @ q[r, h])
                with np.errstate(invalid="ignore"):
                    w = np.exp(s - s.max())
                    out[r, h] = (w / w.sum()) @ v[at, h // group]
    return out
