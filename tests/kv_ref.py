"""Plain references of the cache operators (numpy / torch on the CPU, 64 bits)
and the inputs of their tests.

Tolerances, per element (half a bf16 step is 2^-8 of the value, half an fp16 step
2^-11, half an fp32 step 2^-24):

  norm + rotation   2^-8 |y| for the rounding of the output, and 2^-20 of
                    |a cos| + |b sin| for fp32: the mean of squares (D / 8 + 5
                    additions, then a square root: 25 half steps at D = 256), two
                    products, the rotation's two products and one addition, the
                    table's own rounding: under 16 = 2^4 fp32 steps in all.
  attention         2^-8 |o| for the output, and relative to A = sum p |v| / sum p:
                    2^-11 for the fp16 weights, 2 ds for the scores, 2^-20 for
                    exp2 and the division, n 2^-23 for n keys' fp32 sums (a tensor
                    core may truncate: a whole step each), where ds, the error of
                    a score, is (D + 8) 2^-23 max_t scale |q|.|k_t|; then what fp16
                    leaves of the smallest weights: the largest weight is held as 2^10 at
                    least (the lazy maximum of the many-row kernel), the smallest
                    fp16 step is 2^-24, half of it 2^-35 of the largest weight:
                    2^-35 sum |v| / sum p.  INT4 adds 2^-11 A (values rounded to
                    fp16 in the many-row kernel) and, as weights meet scales
                    relative to the largest scale, 2^-25 max |v| (values below it) and
                    n 2^-36 max |v| / sum p (weights: 2^-39 each, codes up to 7).
  lse               ds + 2^-20 (1 + |lse|) + n 2^-23 (its sum is taken in fp32, before the
                    weights are rounded).
"""
import numpy as np
import torch

import oracle as O

GROUP = {"nvfp4": 16, "fp4g32": 32, "int4": 64}


def quantize(fmt, x):
    """(packed codes [..., D/2] uint8, scale bytes [..., w] uint8, values [..., D] float64) of bf16 x."""
    bits = x.contiguous().view(torch.int16).numpy().view(np.uint16)
    D = bits.shape[-1]
    flat = bits.reshape(-1, D)
    if flat.shape[0] == 0:
        width = D // GROUP[fmt] * (2 if fmt == "int4" else 1)
        return tuple(np.zeros(bits.shape[:-1] + (n,), t) for n, t in ((D // 2, np.uint8), (width, np.uint8), (D, np.float64)))
    got = O.act_quant(fmt, flat, None, None)
    codes, scales = got[0], got[1]
    vals = O.dequant(fmt, codes, scales).astype(np.float64)
    lead = bits.shape[:-1]
    sb = np.ascontiguousarray(scales).view(np.uint8).reshape(flat.shape[0], -1)
    return codes.reshape(*lead, -1), sb.reshape(*lead, -1), vals.reshape(*lead, D)


def pieces(fmt, D, page):
    """Byte offsets of a block: key scales, value codes, value scales, end."""
    c = page * D // 2
    s = page * (D // GROUP[fmt]) * (2 if fmt == "int4" else 1)
    return c, c + s, 2 * c + s, 2 * c + 2 * s


def store(pool, fmt, D, page, slots, k, v):
    """Append to a numpy pool [pages, heads, block]; returns the values (k, v) held there."""
    ks, vc, vs, end = pieces(fmt, D, page)
    out = []
    for x, c0, s0, s1 in ((k, 0, ks, vc), (v, vc, vs, end)):
        codes, sb, vals = quantize(fmt, x)
        w = sb.shape[-1]
        for r, slot in enumerate(slots):
            if slot < 0 or slot >= pool.shape[0] * page:
                continue
            p, o = divmod(int(slot), page)
            pool[p, :, c0 + o * D // 2:c0 + (o + 1) * D // 2] = codes[r]
            pool[p, :, s0 + o * w:s0 + (o + 1) * w] = sb[r]
        out.append(vals)
    return out


def attention(q, keys, values, scale, causal, window, int4=False):
    """One request: q [n, Hq, D], keys / values [kv, Hk, D] float64 -> out, lse, tolerances of both."""
    n, hq, D = q.shape
    kv, hk, _ = keys.shape
    rep = hq // hk
    out, lse = np.zeros((n, hq, D)), np.full((n, hq), -np.inf)
    tol_o, tol_l = np.full((n, hq, D), 1e-30), np.full((n, hq), 1e-30)
    pos = kv - n + np.arange(n)[:, None]
    t = np.arange(kv)[None, :]
    seen = np.ones((n, kv), bool)
    if causal:
        seen &= t <= pos
    if window:
        seen &= t > pos - window
    any_ = seen.any(1)
    if not any_.any():
        return out, lse, tol_o, tol_l
    for h in range(hq):
        k, v = keys[:, h // rep], values[:, h // rep]
        s = np.where(seen, q[:, h] @ k.T * scale, -np.inf)
        big = np.where(seen, np.abs(q[:, h]) @ np.abs(k).T * abs(scale), 0).max(1)
        top = np.where(any_, s.max(1), 0)
        w = np.exp(s - top[:, None])
        total = np.where(any_, w.sum(1), 1)
        out[:, h] = w @ v / total[:, None]
        lse[any_, h] = (top + np.log(total))[any_]
        A = w @ np.abs(v) / total[:, None]
        ds = (D + 8) * 2.0 ** -23 * big
        tol_o[:, h] += 2.0 ** -8 * np.abs(out[:, h]) + (2.0 ** -11 + 2 * ds + 2.0 ** -20 + kv * 2.0 ** -23)[:, None] * A
        tol_o[:, h] += 2.0 ** -35 * (seen @ np.abs(v)) / total[:, None]
        if int4:
            most = np.abs(v).max()
            tol_o[:, h] += 2.0 ** -11 * A + (2.0 ** -25 * most + 2.0 ** -36 * most * seen.sum(1) / total)[:, None]
        tol_l[:, h] += ds + 2.0 ** -20 * (1 + np.abs(np.where(any_, lse[:, h], 0))) + kv * 2.0 ** -23
    return out, lse, tol_o, tol_l


def plan(q_lens, kv_lens, table, free, rows, page):
    """(cu_q, total, positions, slots, used, table) and whether anything was out of range."""
    table, bad, used, cu = table.copy(), False, 0, [0]
    pos, slots, total = np.full(rows, -1), np.full(rows, -1, np.int64), []
    W = table.shape[1]
    for b, (q, n) in enumerate(zip(q_lens, kv_lens)):
        q, n = int(q), int(n)
        if q < 0 or n < 0 or q + n > 2 ** 31 - 1:
            bad, q, n = True, 0, max(n, 0)
        if cu[-1] + q > rows:
            bad, q = True, rows - cu[-1]
        held, want = -(-n // page), -(-(n + q) // page)
        bad |= want > W
        need = max(min(want, W), held)
        for c in range(held, need):
            bad |= used >= len(free)
            table[b, c] = free[used] if used < len(free) else -1
            used += 1
        for t in range(q):
            r = cu[-1] + t
            pos[r] = n + t
            col = pos[r] // page
            pg = table[b, col] if col < W else -1
            if pg >= 0:
                slots[r] = int(pg) * page + pos[r] % page
            else:
                bad = True
        cu.append(cu[-1] + q)
        total.append(n + q)
    return np.array(cu), np.array(total), pos, slots, min(used, len(free)), table, bad


def norm_rope(x, weight, table, positions, eps, norm, interleaved):
    """x [rows, heads, D] float64 -> (y, tolerance)."""
    D = x.shape[-1]
    if norm:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight
    y, size = x.copy(), np.abs(x)
    rot = 0 if table is None else table.shape[1]
    if rot:
        half = rot // 2
        row = table[positions].astype(np.float64)[:, None]
        cos, sin = row[..., :half], row[..., half:]
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
        ya, yb = a * cos - b * sin, b * cos + a * sin
        sa, sb = np.abs(a * cos) + np.abs(b * sin), np.abs(b * cos) + np.abs(a * sin)
        if interleaved:
            y[..., 0:rot:2], y[..., 1:rot:2], size[..., 0:rot:2], size[..., 1:rot:2] = ya, yb, sa, sb
        else:
            y[..., :half], y[..., half:rot], size[..., :half], size[..., half:rot] = ya, yb, sa, sb
    return y, 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * size + 1e-37


def rotation(rows, rot, base=10000.0):
    i = np.arange(rot // 2)
    a = np.arange(rows)[:, None] * base ** (-2.0 * i / max(rot, 1))
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


class Batch:
    """Requests with cached keys and values, scattered over a pool of random bytes."""

    def __init__(self, fmt, D, page, hq, hk, lens, seed, outlier=True, spare_rows=0, k_scale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.D, self.page, self.hq, self.hk, self.lens = fmt, D, page, hq, hk, lens
        need = [-(-kv // page) for _, kv in lens]
        npages = sum(need) + 3
        self.pool = rng.integers(0, 256, (npages, hk, pieces(fmt, D, page)[3]), dtype=np.uint8)
        ids = rng.permutation(npages)
        self.table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
        self.keys, self.values, at = [], [], 0
        for b, (_, kv) in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            t = np.arange(kv)
            slots = self.table[b, t // page].astype(np.int64) * page + t % page
            k = torch.randn(kv, hk, D, generator=g) * k_scale
            v = torch.randn(kv, hk, D, generator=g)
            if outlier and kv:
                k[..., 3] *= 8
            kq, vq = store(self.pool, fmt, D, page, slots, k.to(torch.bfloat16), v.to(torch.bfloat16))
            self.keys.append(kq)
            self.values.append(vq)
        self.rows = sum(n for n, _ in lens) + spare_rows
        self.cu = np.concatenate(([0], np.cumsum([n for n, _ in lens]))).astype(np.int32)
        self.q = torch.randn(self.rows, hq, D, generator=g).to(torch.bfloat16)

    def expected(self, scale, causal, window):
        parts = []
        for b, (n, kv) in enumerate(self.lens):
            q = self.q[self.cu[b]:self.cu[b + 1]].double().numpy()
            parts.append(attention(q, self.keys[b], self.values[b], scale, causal, window, self.fmt == "int4"))
        return [np.concatenate([p[i] for p in parts]) for i in range(4)]
