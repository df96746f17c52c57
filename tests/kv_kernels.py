"""Checks of omq_kv_attn by the kernel that a request runs on, each with the bound of its own
arithmetic: the row kernel's operands are exact (its weights lose what is below 2^-40 of the
largest), the tile kernel rounds k, v and the weights to float16. A call in which some request
has more than 512 query rows per kv head (rows = tokens x Hq / Hkv) gives every request of more
than 64 rows to the tile kernel and the others to the row kernel; a call of one such request is
the tile kernel's alone."""
from __future__ import annotations

import numpy as np
import torch

from tests import kv_common as kc

FEW, MOST = 64, 512


def encode(x):
    """kc.encode of the rows of x, and the documented form of a constant row whose zero point is
    beyond 2^30: c = 0, z = -2^20 or 2^20 and h = |z h| 2^-20 (kc.encode cuts z there)."""
    c, h, z = kc.encode(x)
    with np.errstate(all="ignore"):
        full = -np.rint(x.astype(np.float32).min(-1, keepdims=True) / h)
        far = np.abs(full) > np.float32(2.0 ** 30)
        value = np.abs((full * h).astype(np.float32)) * np.float32(2.0 ** -20)
    return np.where(far, np.float32(0), c), np.where(far, value, h), np.where(far, np.sign(full) * np.float32(2.0 ** 20), z)


def tile_kernel(s, b):
    """Whether request b of a Setup runs on the tile kernel, where that does not depend on the
    sizes' estimate: no request has more than 64 rows, or some has more than 512."""
    rows = [int(n) * s.G for n in s.new]
    assert max(rows) <= FEW or max(rows) > MOST, "the estimate decides"
    return max(rows) > FEW and (rows[b] > FEW or len(rows) == 1)


def attend_tiles(q, k, v, scale, out_half_step):
    """One query row in binary64 against the keys it sees, k and v [N, D]. Returns (o, lse, bound
    of |o|'s error, bound of lse's error) of the tile kernel:
      operands  k' = scale log2(e) k and v, rounded to float16: 2^-11 of their size (and 2^-20 for
                the two parts of their step), and 2^-25; q, float16 or within its range: 2^-25
      score     D products of the rounded operands summed in float32, the matrix unit's partial
                sums to 2^-22; 2^x to 2^-22 of |x| + 1 in the exponent: e, in binary digits
      weights   every p by 2 e ln 2 (numerator and sum); as float16, at least 2^7 for the largest:
                2^-11 of each, or 2^-32 of the largest
      sums      N / 16 + 64 float32 additions, the matrix unit's to 2^-22
      output    half a step of its type (float16 subnormals: 2^-25)"""
    n, d = k.shape
    if n == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    log2e = 1.4426950408889634
    part = 2.0 ** -11 + 2.0 ** -20
    x = k @ q * scale
    top = x.max()
    p = np.exp(x - top)
    total = p.sum()
    lse = top + np.log(total)
    p /= total
    o = p @ v
    kq = np.abs(k * scale * log2e)
    e = (kq @ np.abs(q) * (part + (d + 8) * 2.0 ** -22)).max() + 2.0 ** -25 * np.abs(q).sum()
    e += 2.0 ** -25 * kq.sum(1).max() + 2.0 ** -22 * (np.abs(x).max() * log2e + 1)
    e_p = 2 * e * np.log(2)
    sums = (n / 16 + 64) * 2.0 ** -22
    bound = (part + 2.0 ** -11 + e_p + sums) * (p @ np.abs(v)) + 2.0 ** -32 * p.max() * np.abs(v).sum(0) + 2.0 ** -25
    bound += out_half_step * (np.abs(o) + bound) + 2.0 ** -25
    return o, lse, bound, e_p + sums + 2.0 ** -22 * abs(lse)


def check(s, out, lse=None, causal=True, scale=None, every=1, hidden=(), tiles=None):
    """Every row (or every `every`-th of a request) of every head of a Setup. hidden: (request, page
    index) pairs that are not pages. tiles: the kernel of each request, if the estimate decides."""
    scale = s.D ** -0.5 if scale is None else scale
    half = torch.finfo(out.dtype).eps / 2
    got = out.double().cpu().numpy()
    got_l = None if lse is None else lse.double().cpu().numpy()
    for b in range(len(s.lens)):
        n, m = int(s.lens[b]), int(s.new[b])
        if m == 0:
            continue
        there = np.ones(n, bool)
        for rb, pg in hidden:
            if rb == b:
                there[pg * s.page:(pg + 1) * s.page] = False
        on_tiles = tile_kernel(s, b) if tiles is None else tiles[b]
        (a, ah, az), (c, ch, cz) = s.kv[b]
        for i in sorted({0, m - 1, *range(0, m, every)}):
            seen = there & (np.arange(n) <= n - m + i) if causal else there
            t = int(s.cu[b]) + i
            for h in range(s.Hkv * s.G):
                j = h // s.G
                q = s.q[t, h].double().numpy()
                if on_tiles:
                    o, l, tol, ltol = attend_tiles(q, kc.values(a, ah, az)[seen, j], kc.values(c, ch, cz)[seen, j], scale, half)
                else:
                    o, l, tol, ltol = kc.attend(q, a[:, j], ah[:, j], az[:, j], c[:, j], ch[:, j], cz[:, j], seen, scale,
                                                half, 0.0, 64, -40)
                err = np.abs(got[t, h] - o)
                assert np.all(err <= tol), (b, i, h, float((err - tol).max()), float(err.max()))
                if got_l is not None:
                    assert (got_l[t, h] == l) if np.isinf(l) else abs(got_l[t, h] - l) <= ltol, (b, i, h)
