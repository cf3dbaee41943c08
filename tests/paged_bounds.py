"""Attention over pages in 64 bits with the kernels' own roundings, and a bound of what is left.

Of the roundings to few bits, those that do not depend on the order of the work are made here as the kernels make
them, so they cost no tolerance: the query row turned in fp32 (each butterfly is one sum and one difference, the same
in any order of lanes) and rounded to fp16 after a scaling by a power of two, and the records dequantized to fp16. The
few-rows kernel makes neither: it takes codes as they are and every query value as two fp16 terms.

What is left, per query row and head, as a bound of the 2-norm of the output's error (an orthonormal turn of the output
keeps it). With p the weights, y the value rows, o the output, F = 2^-23 (a step of fp32; a product of the tensor cores
may truncate, so a whole step and not half is charged for each sum):
  scores     16 products at once, D / 16 of them in a chain, a few more steps to the exponent: (20 + D / 16) F of the
             score's magnitudes sum |q'||y|, and 8 F of the largest score's own size for the exponent's argument;
             the exponential itself 2^-22. A score's error d_n moves the weight by expm1(d_n), and by its mean the
             total: sum p (d_n + mean d) |y_n - o|.
  weights    one rounding to fp16: sum p 2^-11 |y_n|; weights below fp16's normal range: 2^-25 of the largest each.
             Two terms in the few-rows kernel: 2^-22.
  sums       16 keys at once and a chain over the rest: (24 + n / 16) F sum p |y_n|; the total (40 + n / 128) F;
             the parts' join 40 F; the turn of the output 16 F |o|.
  output     its rounding to fp16, 2^-11 |o|.
The few-rows kernel sums c S and Z apart, so there |y| is replaced by c |S| + |Z|."""
import numpy as np

import paged_ref as R

F = 2.0 ** -23


def turned_fp32(q):
    """FWHT of fp16 rows in fp32, strides ascending, and 1 / sqrt(D) as the library rounds it."""
    x = q.astype(np.float32)
    D = x.shape[-1]
    h = 1
    while h < D:
        y = x.reshape(*x.shape[:-1], D // (2 * h), 2, h)
        a, b = y[..., 0, :], y[..., 1, :]
        x = np.stack([a + b, a - b], -2).reshape(x.shape)
        h *= 2
    return x * np.float32(1.0 / np.sqrt(float(D)))


def query_rows(q, perm, rot, few):
    """fp16 query rows [m, D] of one head as the products take them, in 64 bits."""
    x = (q if perm is None else q[:, perm]).astype(np.float32)
    if rot:
        x = turned_fp32(x)
    if few:
        return x.astype(np.float64)
    top = np.abs(x).max(-1, keepdims=True)
    e = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))), 0.0)
    return (x.astype(np.float64) * 2.0 ** -e).astype(np.float16).astype(np.float64) * 2.0 ** e


def back_turned(o, perm, rot):
    """Rotated rows [m, D] of one head in the channels' own basis."""
    y = o @ R.hadamard(o.shape[-1]) if rot else o
    if perm is None:
        return y
    x = np.empty_like(y)
    x[:, perm] = y
    return x


class Head:
    """One head's keys and values: rows of sinks [a, D] in their own basis and records [b, D] in the rotated one."""

    def __init__(self, sink_k, sink_v, y_k, y_v, mag_k, mag_v, perm_v, rot, few):
        self.sink_k, self.sink_v, self.rot, self.few, self.perm_v = sink_k, sink_v, rot, few, perm_v
        self.y_k, self.y_v = (y_k, y_v) if few else tuple(y.astype(np.float16).astype(np.float64) for y in (y_k, y_v))
        self.mag_k, self.mag_v = (mag_k, mag_v) if few else (np.abs(self.y_k), np.abs(self.y_v))

    def attend(self, q, qr, seen, scale):
        """(output, bound of the error's 2-norm) of rows q (their own basis) and qr (rotated); seen [m, a + b]."""
        scale = float(np.float32(scale))
        a, n, D = len(self.sink_k), seen.shape[1], q.shape[1]
        s = scale * np.concatenate([q @ self.sink_k.T, qr @ self.y_k.T], 1)
        p = R.softmax_rows(s, seen)
        own = p[:, :a] @ self.sink_v
        rec = back_turned(p[:, a:] @ self.y_v, self.perm_v, self.rot)
        o = own + rec
        # all value rows in the channels' own basis, for |y_n - o|
        v = np.concatenate([self.sink_v, back_turned(self.y_v, self.perm_v, self.rot)], 0)
        apart = np.sqrt(np.maximum((v * v).sum(1)[None] - 2 * o @ v.T + (o * o).sum(1)[:, None], 0.0))
        mag = scale * np.concatenate([np.abs(q) @ np.abs(self.sink_k).T, np.abs(qr) @ self.mag_k.T], 1)
        top = np.abs(s).max(-1, where=p > 0, initial=0.0)[:, None]
        d = np.expm1((20 + D / 16) * F * mag + 8 * F * top + (2.0 ** -22 * mag if self.few else 0.0)) + 2.0 ** -22
        err = (p * (d + (p * d).sum(-1, keepdims=True)) * apart).sum(-1)
        size = np.concatenate([np.linalg.norm(self.sink_v, axis=1), np.linalg.norm(self.mag_v, axis=1)])
        at = p @ size
        live = seen.sum(-1)
        err += at * ((24 + live / 16) * F + (40 + live / 128) * F + 40 * F)
        if self.few:
            err += at * 2.0 ** -22 + live * 2.0 ** -32 * p.max(-1) * size.max(initial=0.0)
        else:
            err += at * R.U16 + live * 2.0 ** -25 * p.max(-1) * size.max(initial=0.0)
        norm = np.linalg.norm(o, axis=1)
        return o, err + (R.U16 + 16 * F) * norm + 2.0 ** -25 * np.sqrt(D)
