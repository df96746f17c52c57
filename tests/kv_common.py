"""Plain statements of the 4-bit paged cache for its tests: the step's plan as a loop over the
requests, the quantizer in numpy binary32, the pool's layout byte by byte, and the attention in
binary64 with the error bound its float32 / float16 arithmetic is allowed."""
from __future__ import annotations

import numpy as np

CELL = 16
F = np.float32


def cell_bytes(D):
    return CELL * D + 256


# ------------------------------------------------------------------------------ plan

def plan(lens, new, table, free, n_free, page, capacity):
    """The documented rules, request by request. Returns the state and the rows after it."""
    n_req, width = table.shape
    table, free = table.copy(), free.copy()
    n_pages = len(free)
    lens = [min(max(int(x), 0), width * page) for x in lens]
    top = min(max(int(n_free[0]), 0), n_pages)
    for b in range(n_req):
        if new[b] < 0:
            for j in range(-(-lens[b] // page)):
                if top < n_pages:
                    free[top] = table[b, j]
                    top += 1
    avail, asked, tokens = top, 0, 0
    out_lens, cu, rows = [], [0], []
    for b in range(n_req):
        n = int(new[b])
        if n < 0:
            out_lens.append(0)
            cu.append(cu[-1])
            continue
        held = -(-lens[b] // page)
        after = -(-(lens[b] + n) // page)
        grant = lens[b] + n <= width * page
        need = after - held if grant and n else 0
        asked += need
        if need and asked > avail:
            grant = False
        if grant and n:
            tokens += n
            grant = tokens <= capacity
        if not grant:
            n = 0
        elif need:
            for j in range(held, after):
                top -= 1
                table[b, j] = free[top]
        for i in range(n):
            pos = lens[b] + i
            rows.append((int(table[b, pos // page]) * page + pos % page, pos, b))
        out_lens.append(lens[b] + n)
        cu.append(cu[-1] + n)
    rows += [(-1, -1, -1)] * (capacity - len(rows))
    slots, positions, requests = (np.array([r[i] for r in rows], np.int32) for i in range(3))
    return dict(lens=np.array(out_lens, np.int32), n_free=np.array([top], np.int32),
                cu=np.array(cu, np.int32), slots=slots, positions=positions, requests=requests,
                table=table, free=free)


# ------------------------------------------------------------------------------ store

def encode(x, top=15):
    """(codes, h, z) of the rows of x (float32), one binary32 rounding per operation."""
    x = x.astype(F)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        h = (hi - lo).astype(F) / F(top)
        h = np.where(h >= F(1e-8), h, F(1e-8))
        z = -np.rint(lo / h)
        c = np.clip(np.rint(x / h) + z, F(0), F(top))
        z = np.clip(z, -F(2.0 ** 30), F(2.0 ** 30))
    return c, h, z


def values(c, h, z, dtype=np.float64):
    return (c.astype(dtype) - z.astype(dtype)) * h.astype(dtype)


def rope_rows(positions, D, base=10000.0):
    ang = np.asarray(positions, np.float64)[:, None] * base ** (-2.0 * np.arange(D // 2) / D)
    return np.cos(ang).astype(F), np.sin(ang).astype(F)


def rotate(x, cos, sin):
    """x [T, heads, D] float32; cos, sin [T, D/2]."""
    half = x.shape[-1] // 2
    a, b = x[..., :half].astype(F), x[..., half:].astype(F)
    c, s = cos[:, None], sin[:, None]
    return np.concatenate(((a * c).astype(F) - (b * s).astype(F),
                           (b * c).astype(F) + (a * s).astype(F)), -1).astype(F)


def put(pool, page, slots, which, c, h, z):
    """Write codes [T, Hkv, D] with h, z [T, Hkv, 1] into the pool bytes (which: 0 K, 1 V)."""
    D = c.shape[-1]
    half = CELL * D // 2
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        p, off = divmod(int(slot), page)
        cell, r = divmod(off, CELL)
        for head in range(c.shape[1]):
            b = pool[p, head, cell]
            code = c[t, head].astype(np.uint8)
            b[which * half + r * D // 2: which * half + (r + 1) * D // 2] = \
                code[0::2] | (code[1::2] << 4)
            at = 2 * half + 128 * which + 4 * r
            b[at:at + 4] = np.frombuffer(F(h[t, head, 0]).tobytes(), np.uint8)
            b[at + 64:at + 68] = np.frombuffer(np.int32(z[t, head, 0]).tobytes(), np.uint8)


def get(pool, page, slots, which):
    """(codes, h, z) [T, Hkv, D], [T, Hkv, 1] x 2 of the slots (all inside the pool)."""
    D = (pool.shape[-1] - 256) // CELL
    half = CELL * D // 2
    c = np.zeros((len(slots), pool.shape[1], D), F)
    h = np.zeros((len(slots), pool.shape[1], 1), F)
    z = np.zeros_like(h)
    for t, slot in enumerate(slots):
        p, off = divmod(int(slot), page)
        cell, r = divmod(off, CELL)
        b = pool[p, :, cell]
        byte = b[:, which * half + r * D // 2: which * half + (r + 1) * D // 2]
        c[t, :, 0::2], c[t, :, 1::2] = byte & 15, byte >> 4
        at = 2 * half + 128 * which + 4 * r
        h[t, :, 0] = np.ascontiguousarray(b[:, at:at + 4]).view(F)[:, 0]
        z[t, :, 0] = np.ascontiguousarray(b[:, at + 64:at + 68]).view(np.int32)[:, 0]
    return c, h, z


# ------------------------------------------------------------------------------ attention

def attend(q, kc, kh, kz, vc, vh, vz, seen, scale, out_half_step, operand_half_step=0.0, far=None, tiny=-25):
    """One query row in binary64 against N keys (codes [N, D], h, z [N, 1]; seen [N] booleans).
    Returns (o, lse, bound of |o|'s error, bound of lse's error).

    The bound. With p the weights and v the values, in the order of the arithmetic:
      score   products of an exact code and an exact q, summed in float32 over D terms (each
              partial sum rounded, the matrix unit's by at most 2^-22 of the largest), z's part
              subtracted, two more products: (D + 8) 2^-22 of h scale sum |q| (c + |z|) =: e_s;
              2^x and log2 h are off by 2^-22 of |x| + |log2 h| + 1 in the exponent
      weights relative change e_p = 2 (max over keys of those) of every p, numerator and sum
      float16 rounding of w = p h, largest 1: relative 2^-11, or 2^-25 absolute
      operands (many rows) k and v themselves rounded to float16: relative 2^-11 of each and, for
              k, of scale sum |q| |k| in the score (2^-25 absolute, times 2^-22 of a second part)
      sums    N/16 + 64 float32 additions (the matrix unit's by 2^-22) of terms p h (c + |z|)
      tiny    exponent of that absolute error: with the largest weight 2^15 instead of 1, -40;
              with 2^7 (many rows) -32
      far     zero points beyond this are weighed by the float32 weight, so that the float16
              rounding meets only the code there
      output  half a step of its type."""
    N, D = kc.shape
    if not seen.any():
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    q = q.astype(np.float64)
    kc, kh, kz, vc, vh, vz = (a.astype(np.float64)[seen] for a in (kc, kh, kz, vc, vh, vz))
    n = kc.shape[0]
    s = (((kc - kz) * kh) @ q) * scale
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    lse = top + np.log(total)
    p /= total
    v = (vc - vz) * vh
    o = p @ v
    mag = (kh * scale * ((kc + np.abs(kz)) @ np.abs(q))[:, None])[:, 0]
    x = np.abs(s) * 1.4427 + np.abs(np.log2(vh[:, 0])) + 1
    e_s = (D + 8) * 2.0 ** -22 * mag.max() + 2.0 ** -21 * x.max()
    e_s += operand_half_step * (scale * (np.abs((kc - kz) * kh) @ np.abs(q))).max()
    if operand_half_step:
        e_s += 2.0 ** -24 * np.abs(q).sum()
    e_p = 2 * e_s
    w = p * vh[:, 0]
    # the largest weight is scaled to 1: absolute float16 error 2^-25 of it
    met = np.abs(vc - vz)
    if far is not None:
        met = np.where(np.abs(vz) > far, vc, met)
    sub = 2.0 ** tiny * w.max() * met.sum(0)
    acc = (n / 16 + 64) * 2.0 ** -22 * (w @ (vc + np.abs(vz)))
    bound = (2.0 ** -11 + operand_half_step + e_p) * (p @ np.abs(v)) + sub + acc
    if operand_half_step:
        bound = bound + 2.0 ** -24
    bound = bound + out_half_step * (np.abs(o) + bound) + 2.0 ** -25
    return o, lse, bound, e_p + (n / 64 + 64) * 2.0 ** -22 + 2.0 ** -22 * abs(lse)
