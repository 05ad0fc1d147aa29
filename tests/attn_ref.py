"""Plain 64-bit references of the attention operators (numpy on the CPU, no
code shared with the library): what the cache bytes stand for, attention with
a window and sinks, and the 4-bit insertion."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_values(codes):
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def e2m1_values(codes, sf):
    """codes [n, D/2], sf [n, D/32] -> [n, D] float64."""
    n = np.empty((codes.shape[0], codes.shape[1] * 2), dtype=np.int64)
    n[:, 0::2] = codes & 15
    n[:, 1::2] = codes >> 4
    v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    s = np.where(sf == 255, np.nan, 2.0 ** (sf.astype(np.float64) - 127.0))
    return v * np.repeat(s, 32, axis=1)


def visible(p, n, window, sinks):
    """[n] booleans: the keys that position p sees among n."""
    j = np.arange(n)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attention(q, rows, block_table, page_size, q_start, seq_lens, window, sinks, scale, bad_pages=()):
    """q [T, H, D] float64, rows [num_slots, D] float64 -> (out, lse, A, sabs): the output, the log
    denominators, A = sum_j w_j |k_j| (what the rounding of the weights scales with) and the largest
    sum_d |q_d k_d| * scale over the visible keys.  Masked rows are never touched."""
    T, H, D = q.shape
    out = np.zeros((T, H, D))
    A = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    sabs = np.zeros((T, H))
    for b in range(len(seq_lens)):
        t0, t1 = int(q_start[b]), int(q_start[b + 1])
        L = int(seq_lens[b])
        for t in range(t0, t1):
            p = L - (t1 - t0) + (t - t0)
            if p < 0:
                continue
            j = np.nonzero(visible(p, L, window, sinks))[0]
            pages = block_table[b, j // page_size].astype(np.int64)
            keep = ~np.isin(pages, np.array(list(bad_pages), dtype=np.int64))
            j, pages = j[keep], pages[keep]
            if len(j) == 0:
                continue
            k = rows[pages * page_size + j % page_size]
            s = scale * (q[t] @ k.T)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(-1, keepdims=True)
            out[t] = (e / l) @ k
            A[t] = (e / l) @ np.abs(k)
            lse[t] = (m + np.log(l))[:, 0]
            sabs[t] = (scale * (np.abs(q[t]) @ np.abs(k).T)).max(-1)
    return out, lse, A, sabs


def encode_e2m1(y):
    """y [n, D] float32 values -> (codes [n, D/2], sf [n, D/32]) by nearest value, ties to the even code."""
    n, D = y.shape
    g = y.astype(np.float64).reshape(n, D // 32, 32)
    top = np.abs(g).max(-1)
    e = np.full(top.shape, -127)
    for cand in range(-126, 128):  # the smallest exponent that holds the block
        e = np.where(top > 6.0 * 2.0 ** (cand - 1), cand, e)
    v = g * 2.0 ** -e[..., None].astype(np.float64)
    d = np.abs(np.abs(v)[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    cand = d == best
    odd_only = cand & (np.arange(8) % 2 == 0)
    code = np.where(odd_only.any(-1), odd_only.argmax(-1), cand.argmax(-1))
    code = (code | np.where(np.signbit(v), 8, 0)).astype(np.uint8).reshape(n, D // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).astype(np.uint8)


def rotate(x, cos, sin, R):
    """Forward rotation of the last R elements (rotate-half pairs) in float32, one rounding per value."""
    y = x.astype(np.float32).copy()
    D = x.shape[-1]
    a, b = y[..., D - R:D - R // 2].copy(), y[..., D - R // 2:].copy()
    while cos.ndim < a.ndim:
        cos, sin = cos[:, None], sin[:, None]
    y[..., D - R:D - R // 2] = (a.astype(np.float64) * cos - b.astype(np.float64) * sin).astype(np.float32)
    y[..., D - R // 2:] = (b.astype(np.float64) * cos + a.astype(np.float64) * sin).astype(np.float32)
    return y
