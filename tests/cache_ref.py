"""Plain 64-bit NumPy implementations of the paged 8-bit cache's operators, and
the error bounds that the GPU tests hold the kernels to.  Shares no code with
the library."""
from __future__ import annotations

import math

import numpy as np

MIN_EXP = -64


def _e4m3_table() -> np.ndarray:
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f is NaN, no infinity."""
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = math.nan if c & 127 == 127 else v
        if c & 128:
            t[c] = -t[c]
    return t


E4M3 = _e4m3_table()


def encode(x: np.ndarray) -> np.ndarray:
    """Codes of 64-bit values: to nearest, ties to even; NaN and infinities to NaN (|x| <= 448 otherwise)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    mag = E4M3[:127]
    hi = np.clip(np.searchsorted(mag, a, side="left"), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - mag[lo], mag[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.isfinite(x), code | (np.signbit(x).astype(np.uint8) << 7), 0x7F)
    return code.astype(np.uint8)


def page_scale(values: np.ndarray) -> float:
    """2^max(-64, ceil(log2(amax / 448))) over the finite values."""
    f = np.abs(values[np.isfinite(values)])
    amax = float(f.max()) if f.size else 0.0
    if amax == 0.0:
        return 2.0 ** MIN_EXP
    m, e = math.frexp(amax / 448.0)  # m in [0.5, 1): m = 0.5 is a power of two
    return 2.0 ** max(MIN_EXP, e - 1 if m == 0.5 else e)


def plan(held, add, ring, state, table, page, tokens):
    """(lens, starts, slots, ring, state, table) after a step; a step that does not fit changes nothing."""
    held, add = [int(x) for x in held], [int(x) for x in add]
    ring, table = np.array(ring), np.array(table)
    num, (n, wide) = len(ring), table.shape
    head, count = int(state[0]), int(state[1])
    pages = lambda t: -(-t // page)
    bad = not (0 <= head < num and 0 <= count <= num)
    for i in range(n):
        bad |= held[i] < 0 or held[i] > wide * page or add[i] < -1 or held[i] + max(add[i], 0) > wide * page
    if not bad:
        for i in range(n):
            if add[i] > 0 and held[i] % page:
                bad |= not 0 <= table[i, pages(held[i]) - 1] < num
        opened = sum(pages(held[i] + max(add[i], 0)) - pages(held[i]) for i in range(n))
        back = sum(pages(held[i]) for i in range(n) if add[i] < 0)
        bad |= sum(max(a, 0) for a in add) > tokens or opened > count or count + back > num
    slots = np.full(tokens, -1, np.int32)
    if bad:
        return np.array(held, np.int32), np.zeros(n + 1, np.int32), slots, ring, np.array([head, count, 0, -13]), table
    lens, starts, t, taken, put = np.zeros(n, np.int32), np.zeros(n + 1, np.int32), 0, 0, 0
    old, status = ring.copy(), 0
    for i in range(n):
        starts[i] = t
        if add[i] < 0:
            for j in range(pages(held[i])):
                ring[(head + count + put) % num] = table[i, j]
                put += 1
            continue
        lens[i] = held[i] + add[i]
        for pos in range(held[i], held[i] + add[i]):
            j = pos // page
            if pos % page == 0:
                p = old[(head + taken) % num]
                taken += 1
                if not 0 <= p < num:
                    p, status = -1, -13
                table[i, j] = p
            if table[i, j] >= 0:
                slots[t] = table[i, j] * page + pos % page
            t += 1
    starts[n] = t
    return lens, starts, slots, ring, np.array([(head + taken) % num, count - taken + put, 0, status]), table


def store(x, slots, codes, scales, page):
    """New (codes [num_pages, hkv, page, 128], scales) after storing x [T, hkv, 128] (64-bit values)."""
    codes, scales = codes.copy(), scales.astype(np.float64)
    by_page = {}
    for t, s in enumerate(slots):
        if s >= 0:
            by_page.setdefault(int(s) // page, []).append((int(s) % page, t))
    for pg, cells in by_page.items():
        off = min(o for o, _ in cells)
        for h in range(codes.shape[1]):
            new = np.stack([x[t, h] for _, t in cells])
            s = page_scale(new)
            if off > 0:
                s = max(s, float(scales[pg, h]))
                if s > scales[pg, h]:
                    codes[pg, h, :off] = encode(E4M3[codes[pg, h, :off]] * (scales[pg, h] / s))
            scales[pg, h] = s
            for (o, t), row in zip(cells, new):
                codes[pg, h, o] = encode(row / s)
    return codes, scales


def attention(q, kc, vc, ks, vs, table, lens, starts, page, mask=None, scale=None):
    """(O, bound) of every row of the requests, NaN elsewhere.

    bound, per output value, of kernels that multiply in 8-bit terms (few rows) or
    in 8-bit terms and fp16 (many rows) and accumulate in 32 bits:
      q      two e4m3 terms of q / s, s the power of two that brings the row's
             largest |q| into (224, 448]: the first leaves at most 2^-4 of a
             value (half a step of 4 significant bits), the second 2^-4 of
             that, which the 8 bits of a bf16 value do not exceed, or half its
             smallest step, 2^-10 <= 2^-17 max|q| / s  ->  |dq| <= 2^-17 max|q|
      S      |dS| <= scale (2^-17 max|q| sum|k| + 2^-20 sum|q k|): the second
             part is 128 products and 8 partial sums in 32 bits
      P      P v = (p s) code for a page scale s: three e4m3 terms of p s, each
             leaving 2^-4: 2^-12, or half the third's smallest step, 2^-10.  The
             terms are scaled by 2^6, 2^10 and 2^14 against a reference that the
             largest p s is at least: 2^-24 max(p s), for every token's |code|.
             Many rows: p s in fp16, one rounding, 2^-11, or half its smallest
             step, 2^-25, scaled by 2^7: 2^-32 max(p s).  The larger of each;
             the exponential 2^-20, and the factor |dS| on both sides of the
             quotient: 2 |dS|
      O      partial sums in 32 bits: 2^-18 sum p|v|;  one rounding to bf16: 2^-8 |O|
    """
    T, hq, D = q.shape
    hkv = ks.shape[1]
    g = hq // hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    O, B = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    num = len(ks)
    for i, total in enumerate(lens):
        a, b = int(starts[i]), int(starts[i + 1])
        if a == b:
            continue
        total = max(int(total), 0)
        pos = np.arange(total)
        pg = np.asarray(table[i])[pos // page] if total else np.zeros(0, int)
        there = (pg >= 0) & (pg < num)
        pgc = np.clip(pg, 0, num - 1)
        for h in range(hkv):
            K = E4M3[kc[pgc, h, pos % page]] * ks[pgc, h][:, None].astype(np.float64)
            V = E4M3[vc[pgc, h, pos % page]] * vs[pgc, h][:, None].astype(np.float64)
            for j in range(h * g, h * g + g):
                keep = there.copy()
                if mask is not None:
                    w = mask[i, j].astype(np.int64) & 0xFFFFFFFF
                    keep &= ((w[pos // 4096] >> (pos // 128 % 32)) & 1).astype(bool)
                for t in range(a, b):
                    see = keep & (pos <= total - (b - a) + (t - a))
                    if not see.any():
                        O[t, j] = 0.0
                        B[t, j] = 0.0
                        continue
                    qq, Kq, Vq = q[t, j], K[see], V[see]
                    s = Kq @ qq * scale
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    dS = scale * (2.0 ** -17 * np.abs(qq).max() * np.abs(Kq).sum(1) +
                                  2.0 ** -20 * (np.abs(Kq) @ np.abs(qq))).max()
                    O[t, j] = p @ Vq
                    pv = p @ np.abs(Vq)
                    sv = vs[pgc, h][see].astype(np.float64)
                    low = 2.0 ** -24 * (p * sv).max() * (np.abs(Vq) / sv[:, None]).sum(0)
                    B[t, j] = 2.0 ** -8 * np.abs(O[t, j]) + (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -20 + 2 * dS) * 1.01 * pv + \
                        1.01 * low + 1e-38
    return O, B
