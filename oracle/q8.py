"""Oracle of the paged append (position rotation) and of the 8-bit cache: plain numpy, one sequence, head and block at a
time.  Test infrastructure; shares no code with the library.

The write path is defined in single fp32 operations, so it is restated in numpy float32 and compared bit for bit; the
attention is in fp64.
"""

from __future__ import annotations

import numpy as np

BLOCK = 16
F = np.float32


def e4m3_values():
    """The 256 values of the e4m3 code (NaN at 0x7f and 0xff): sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


_E4M3 = e4m3_values()
_POS = _E4M3[:127]  # the non-negative codes, increasing


def to_e4m3(y):
    """Nearest e4m3 code, ties to the even code, clamped at 448; NaN to 0.  y float32."""
    y = np.asarray(y, np.float32)
    a = np.minimum(np.abs(np.where(np.isnan(y), 0, y)).astype(np.float64), 448.0)
    hi = np.minimum(np.searchsorted(_POS, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    neg = np.signbit(np.where(np.isnan(y), 0, y))
    return (code | np.where(neg, 128, 0)).astype(np.uint8)


def values(codes, kind):
    """fp64 values of uint8 codes."""
    codes = np.asarray(codes, np.uint8)
    return codes.view(np.int8).astype(np.float64) if kind == "i8" else _E4M3[codes]


def rotate(x, cos_sin, pos, interleaved):
    """x [..., d] float32 rotated at position pos: one rounding per product and sum."""
    x = np.asarray(x, F).copy()
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    h = rot // 2
    c, s = cos_sin[pos, :h], cos_sin[pos, h:]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(h)
    ib = ia + (1 if interleaved else h)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = F(a * c) - F(b * s)
    x[..., ib] = F(b * c) + F(a * s)
    return x


def need(amax, kind):
    amax = F(amax)
    if not amax >= F(2.0 ** -100):
        return F(0)
    if kind == "i8":
        return F(amax / F(127))
    s = 2.0 ** -200
    while s * 448.0 < float(amax):
        s *= 2.0
    return F(s)


def round_codes(y, kind):
    if kind == "i8":
        y = np.where(np.isnan(y), F(0), y)
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    return to_e4m3(y)


def append(x, codes, scales, table, lens, counts, bt, kind):
    """New rows x (list per sequence of [count, Hkv, d] float32, already rotated) into pools codes [blocks, Hkv, bt, d]
    and scales [blocks, Hkv, bt / 16], in place."""
    for b, n in enumerate(counts):
        p0 = int(lens[b]) - n
        for blk in range(max(p0, 0) // BLOCK, -(-int(lens[b]) // BLOCK) if n else 0):
            page, off = table[b][blk * BLOCK // bt], blk * BLOCK % bt
            new = [p for p in range(blk * BLOCK, (blk + 1) * BLOCK) if max(p0, 0) <= p < lens[b]]
            old = [p for p in range(blk * BLOCK, (blk + 1) * BLOCK) if p < p0]
            if not new:
                continue
            for h in range(codes.shape[1]):
                rows = np.stack([x[b][p - p0, h] for p in new])
                mag = np.abs(rows)
                amax = F(np.max(np.where(np.isfinite(mag), mag, 0)))
                s_old = F(scales[page, h, off // BLOCK]) if old else F(0)
                s = max(s_old, need(amax, kind))
                inv = F(F(1) / s) if s > 0 else F(0)
                with np.errstate(invalid="ignore", over="ignore"):
                    for p, r in zip(new, rows):
                        codes[page, h, p % bt] = round_codes(F(r * inv), kind)
                if s != s_old:
                    ratio = F(s_old * inv)
                    for p in old:
                        v = values(codes[page, h, p % bt], kind).astype(F)
                        codes[page, h, p % bt] = round_codes(F(v * ratio), kind)
                scales[page, h, off // BLOCK] = s


def attend(q, kcodes, kscales, vcodes, vscales, table, lens, counts, bt, kind, scale, T=None):
    """Causal attention in fp64.  q list per sequence of [count, Hq, d].  Keys at or past position T (None: no bound) are
    seen by no token, whose own positions stay what they are.  Returns lists of (out [count, Hq, d], the magnitude
    sum_t p_t |v_t| of each output coordinate, the largest score error scale of each (token, head):
    scale * max_t sum_j |q_j k_tj|)."""
    Hkv, d = kcodes.shape[1], kcodes.shape[3]
    outs, mags, errs = [], [], []
    for b, n in enumerate(counts):
        L = int(lens[b])
        Hq = q[b].shape[1]
        G = Hq // Hkv
        o, mg, er = np.zeros((n, Hq, d)), np.zeros((n, Hq, d)), np.zeros((n, Hq))
        for h in range(Hkv):
            keys = L if T is None else min(L, T)
            k, v = np.zeros((keys, d)), np.zeros((keys, d))
            for t in range(keys):
                page, off = table[b][t // bt], t % bt
                k[t] = values(kcodes[page, h, off], kind) * np.float64(kscales[page, h, off // BLOCK])
                v[t] = values(vcodes[page, h, off], kind) * np.float64(vscales[page, h, off // BLOCK])
            for i in range(n):
                last = min(L - n + i, keys - 1)
                if last < 0:
                    continue
                for g in range(G):
                    qq = np.asarray(q[b][i, h * G + g], np.float64)
                    s = scale * (k[:last + 1] @ qq)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o[i, h * G + g] = p @ v[:last + 1]
                    mg[i, h * G + g] = p @ np.abs(v[:last + 1])
                    er[i, h * G + g] = abs(scale) * np.max(np.abs(k[:last + 1]) @ np.abs(qq))
        outs.append(o)
        mags.append(mg)
        errs.append(er)
    return outs, mags, errs
