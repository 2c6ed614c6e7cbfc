"""64-bit references and error bounds for the operators around attention (norm + rotation of queries
and keys, its gradient, page bookkeeping, decode behind shared prefixes).

Bounds.  u = 2^-24 is half a step of fp32, and an output of type t is off by at most
torch.finfo(t).eps / 2 of its value from its one rounding.  What the arithmetic before it adds is
counted beside each bound.
"""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- norm + rotation ---------------------------------------------------------------------------
def rope_table(max_pos, rot, base=10000.0):
    """fp32 [max_pos, rot]: cosines, then sines (angles in 64 bits)."""
    pairs = max(rot // 2, 1)
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(rot // 2) / pairs)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).reshape(max_pos, rot)


def pair_columns(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(rope, positions, sections):
    """cos, sin [..., N, pairs] for positions [N] / [B, N], or with sections [axes, ...]; a position
    outside the table leaves its pairs unrotated."""
    table, pos = f64(rope), positions.cpu().numpy().astype(np.int64)
    pairs = table.shape[1] // 2
    if sections is None:
        pos, axis = pos[None], np.zeros(pairs, dtype=int)
    else:
        axis = np.repeat(np.arange(len(sections)), sections)
    at = np.moveaxis(pos[axis], 0, -1)  # [..., N, pairs]
    inside = (at >= 0) & (at < table.shape[0])
    row = np.where(inside, at, 0)
    col = np.arange(pairs)
    return np.where(inside, table[row, col], 1.0), np.where(inside, table[row, col + pairs], 0.0)


def rotate(y, cos, sin, rot, interleaved, back=False):
    """y [..., N, d] with cos, sin [..., N, pairs]: (rotated, sum of the magnitudes added up)."""
    z, mag = y.copy(), np.abs(y)
    lo, hi = pair_columns(rot, interleaved)
    s = -sin if back else sin
    z[..., lo] = y[..., lo] * cos - y[..., hi] * s
    z[..., hi] = y[..., hi] * cos + y[..., lo] * s
    mag[..., lo] = np.abs(y[..., lo] * cos) + np.abs(y[..., hi] * s)
    mag[..., hi] = np.abs(y[..., hi] * cos) + np.abs(y[..., lo] * s)
    return z, mag


def norm_rope(x, w, rope, positions, sections=None, interleaved=False, eps=1e-6):
    """x [B, H, N, d] (or [H, N, d]): (z, bound on the error before the output's rounding).

    The sum of squares has at most 12 roundings (half of them reach r), the mean, eps and rsqrt add
    6, the weight times the angle 1, the two products and the outer product 3: 20 u of the
    magnitudes that are added up."""
    x = f64(x)
    cos, sin = angles(rope, positions, sections)
    if cos.ndim == 3:  # [B, N, pairs]
        cos, sin = cos[:, None], sin[:, None]
    y = x
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(w)
    z, mag = rotate(y, cos, sin, rope.shape[1], interleaved)
    return z, 20 * U * mag


def norm_rope_bwd(x, dz, w, rope, positions, sections=None, interleaved=False, eps=1e-6):
    """(dx, bound on dx before its rounding, dw, sum of the magnitudes of dw's terms).

    dy has 2 roundings, times w 3; the row's dot product adds 12, r^2 (r: 11) 22, three products 3,
    and the outer difference and product 13: at most 60 u of r (|dy w| + |x| r^2 mean|dy w x|)."""
    x, dz = f64(x), f64(dz)
    cos, sin = angles(rope, positions, sections)
    if cos.ndim == 3:
        cos, sin = cos[:, None], sin[:, None]
    dy, mag = rotate(dz, cos, sin, rope.shape[1], interleaved, back=True)
    if w is None:
        return dy, 3 * U * mag, None, None
    w = f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dy * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    gm = mag * np.abs(w)
    bound = 60 * U * r * (gm + np.abs(x) * r * r * (gm * np.abs(x)).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, bound, (dy * x * r).sum(axes), (mag * np.abs(x) * r).sum(axes)


def dw_bound(mag_sum, rows):
    """A weight gradient's terms have 14 roundings; a thread adds at most rows / (888 blocks x 4
    warps) + 8 of them in turn (as many blocks as there are heads allow: two thirds at least), its block 16
    more, the last sum 7 + 7."""
    return (14 + rows / 2368 + 8 + 16 + 14) * U * mag_sum


def assert_within(got, ref, bound, dtype, what):
    got, bound = f64(got), bound + half_step(dtype) * (np.abs(ref) + bound)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.all(np.isfinite(got)), what + ": not finite"
    err = np.abs(got - ref)
    worst = (err - bound).max(initial=-1.0)
    assert np.all(err <= bound), "%s: off by %.3g more than its bound (max error %.3g)" % (what, worst, err.max())


# ---- page bookkeeping --------------------------------------------------------------------------
def page_update(table, old, new, free, ring, page, max_tokens, offset=None):
    """(table, free, ring_out, cu_seqlens, slots, positions) after one step, request by request."""
    table, free = table.copy(), free.copy()
    B, width = table.shape
    cap = len(free)
    head, tail = int(ring[0]), int(ring[1])
    need = [[-(-int(n) // page) for n in lens] for lens in (old, new)]
    tokens = sum(max(int(b) - int(a), 0) for a, b in zip(old, new))
    grow = sum(max(b - a, 0) for a, b in zip(*need))
    shrink = sum(max(a - b, 0) for a, b in zip(*need))
    bad = any(n < 0 or n > width * page for lens in (old, new) for n in lens) or tokens > max_tokens
    bad = bad or head < 0 or not 0 <= tail - head <= cap or tail - head + shrink > cap
    missing = -1 if bad else max(grow - (tail - head), 0)
    cu = np.zeros(B + 1, dtype=np.int32)
    slots = np.full(max_tokens, -1, dtype=np.int32)
    positions = np.zeros(max_tokens, dtype=np.int32)
    if missing:
        return table, free, np.array([head, tail, missing]), cu, slots, positions
    t = 0
    for b in range(B):
        a, n = int(old[b]), int(new[b])
        for i in range(need[0][b], need[1][b]):
            table[b, i] = free[head % cap]
            head += 1
        for i in range(need[1][b], need[0][b]):
            free[tail % cap] = table[b, i]
            tail += 1
        for p in range(a, n):
            slots[t] = table[b, p // page] * page + p % page
            positions[t] = p + (int(offset[b]) if offset is not None else 0)
            t += 1
        cu[b + 1] = t
    return table, free, np.array([head, tail, 0]), cu, slots, positions


# ---- decode behind shared prefixes --------------------------------------------------------------
def decode_reference(q, keys, values, scale):
    """q [Hq, d], keys and values [n, Hkv, d] (64 bits): (o [Hq, d], lse [Hq], bound of o before its
    rounding, bound of lse).

    A score is a sum of 128 products in fp32, off by at most 130 u of the sum of their magnitudes,
    and that is a relative error d of its weight.  Weights are rounded to bf16 for the product with V
    (2^-8 of each), 2^x adds 2^-22, the sums (16 in a thread's chain, 8 chains, one per 128 keys, one
    per part) fewer than 64 + n / 128 roundings."""
    Hq, d = q.shape
    n, Hkv, _ = keys.shape
    if n == 0:
        return np.zeros((Hq, d)), np.full(Hq, -np.inf), np.zeros((Hq, d)), np.zeros(Hq)
    g = Hq // Hkv
    qh = q.reshape(Hkv, g, d)
    x = np.einsum("hgd,nhd->hgn", qh, keys) * scale
    mag = np.einsum("hgd,nhd->hgn", np.abs(qh), np.abs(keys)).max(-1) * abs(scale)
    delta = 130 * U * mag + 2.0 ** -22 + (64 + n / 128) * U
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(-1, keepdims=True)
    p = e / z
    o = np.einsum("hgn,nhd->hgd", p, values)
    a = np.einsum("hgn,nhd->hgd", p, np.abs(values))
    lse = (m + np.log(z))[..., 0]
    return (o.reshape(Hq, d), lse.reshape(Hq), ((2.0 ** -8 + 3 * delta[..., None]) * a).reshape(Hq, d),
            (delta + 4 * U * np.abs(lse)).reshape(Hq))


def assert_decode(o, lse, ref, what):
    """o [Hq, d] bf16, lse [Hq] fp32 against decode_reference's answer."""
    ro, rl, bo, bl = ref
    assert_within(o, ro, bo, torch.bfloat16, what)
    lse = f64(lse)
    empty = rl == -math.inf
    assert np.all(lse[empty] == -math.inf), what + ": LSE of a row without keys"
    assert np.all(f64(o)[empty] == 0), what + ": O of a row without keys"
    err = np.abs(lse[~empty] - rl[~empty])
    assert np.all(err <= bl[~empty]), "%s: LSE off by %.3g" % (what, err.max(initial=0.0))
