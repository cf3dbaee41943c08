"""Plain forms of the paged cache and of attention, in 64 bits on the host, and
the error bounds of the kernels' products. No library call is made here."""
import math

import numpy as np

U16 = 2.0 ** -11  # half a step of fp16, relative
UB16 = 2.0 ** -8  # of bf16


def page_map(S, n_rows, max_pages, ps, n_pages, ctx, new, table, free, used):
    """kvq_page_map on lists; returns what the call writes."""
    table = [list(r) for r in table]
    cu, kv, seq, pos, slot = [0], [], [-1] * n_rows, [-1] * n_rows, [-1] * n_rows
    at, lacking, without = max(0, used), 0, 0
    for s in range(S):
        c, n = max(0, ctx[s]), max(0, new[s])
        for k in range(-(-c // ps), min(-(-(c + n) // ps), max_pages)):
            table[s][k] = free[at] if at < len(free) else -1
            lacking += at >= len(free)
            at += 1
        held = [k for k in range(-(-c // ps), max_pages) if k * ps < c + n and table[s][k] != -1]
        for i in range(n):
            p, r = c + i, cu[-1] + i
            k = p // ps
            new_page = k >= -(-c // ps)
            if k >= max_pages or (new_page and k not in held):
                without += 1
            if r < n_rows:
                seq[r], pos[r] = s, p
                page = table[s][k] if k < max_pages else -1
                slot[r] = page * ps + p % ps if 0 <= page < n_pages else -1
        cu.append(cu[-1] + n)
        kv.append(c + n)
    return dict(cu_rows=cu, kv_len=kv, block_table=table, seq=seq, pos=pos, slot=slot,
                report=[cu[-1], min(at, len(free)), without, lacking])


def hadamard(D):
    h = np.ones((1, 1))
    while h.shape[0] < D:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(D)


def rope(x, m, mode, table):
    """Rows x [..., D] turned to position m by the fp32 (cos, sin) table."""
    D = x.shape[-1]
    c, s = (table[m, :, i].astype(np.float64) for i in (0, 1))
    y = np.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if mode == 1 else (x[..., :D // 2], x[..., D // 2:])
    p, q = a * c - b * s, a * s + b * c
    if mode == 1:
        y[..., 0::2], y[..., 1::2] = p, q
    else:
        y[..., :D // 2], y[..., D // 2:] = p, q
    return y


def unpack(codes, D, bits):
    b = np.unpackbits(codes.reshape(-1, D * bits // 8), axis=1, bitorder="little").reshape(-1, D, bits)
    return (b * (1 << np.arange(bits))).sum(-1).astype(np.float64).reshape(*codes.shape[:-1], D)


def dequantized(codes, sz, D, bits, group):
    """Rotated rows y = Z + c S of records codes [..., RB], sz int16 [..., ng, 2]."""
    f = sz.view(np.float16).astype(np.float64)
    y = unpack(codes, D, bits).reshape(*codes.shape[:-1], D // group, group)
    return (f[..., 1:] + y * f[..., :1]).reshape(*codes.shape[:-1], D)


def softmax_rows(s, seen):
    """Weights of the scores s over the keys that `seen` allows; zeros in an empty row."""
    s = np.where(seen, s, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    p = np.where(seen, p, 0.0)
    total = p.sum(-1, keepdims=True)
    return p / np.where(total > 0, total, 1.0)
