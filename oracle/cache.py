"""CPU fp64 definitions of the rotary positions, the 8-bit cache and the attention over
it, in NumPy. Test infrastructure: written from the formulas, with no code of the package.
"""
from __future__ import annotations

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (4 exponent bits of bias 7, 3 mantissa bits, no
    infinities, NaN at S.1111.111)."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = np.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[code] = -mag if code & 128 else mag
    return out


_E4M3 = e4m3_values()
_POS = _E4M3[:127]  # ascending, 0 .. 448
_MID = (_POS[1:] + _POS[:-1]) / 2


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Values of uint8 bit patterns."""
    return codes.view(np.int8).astype(np.float64) if fmt == "int8" else _E4M3[codes]


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 bit patterns of the nearest codes, ties to even, saturating; NaN to NaN (int8: 0)."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(np.nan_to_num(x, nan=0.0, posinf=127.0, neginf=-127.0)), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    lo = np.searchsorted(_MID, a, side="left")      # first code whose upper midpoint is >= a
    tie = (lo < 126) & (a == _MID[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7f), code)


def scale_for(amax: float, fmt: str) -> float:
    """The smallest power of two s >= 2^-126 with amax <= s * QMAX; 0 for 0."""
    if amax == 0:
        return 0.0
    e = -126
    while amax > 2.0 ** e * QMAX[fmt]:
        e += 1
    return 2.0 ** e


def write(codes, scale, x, table, start, count, page, fmt):
    """Writes x [B, H, N, d] (fp64) into one of K and V in place: codes uint8 [P, H, page, d],
    scale fp64 [P, H]."""
    P = codes.shape[0]
    for b in range(x.shape[0]):
        first, end = start[b], min(start[b] + count[b], table.shape[1] * page)
        for i in range(first // page, -(-end // page) if end > first else 0):
            p = int(table[b, i])
            if not 0 <= p < P:
                continue
            t0, t1 = max(first, i * page), min(end, (i + 1) * page)
            held = max(0, first - i * page)
            for h in range(x.shape[1]):
                new = x[b, h, t0 - first:t1 - first]
                a = np.abs(new[np.isfinite(new)])
                old = scale[p, h] if held else 0.0
                power = 2.0 ** np.ceil(np.log2(old)) if old > 0 else 0.0
                s = max(power, scale_for(a.max() if a.size else 0.0, fmt))
                inv = 1 / s if s > 0 else 1.0  # scale 0: zeros, infinities (the largest code) and NaN
                if held and s > old:
                    codes[p, h, :held] = encode(decode(codes[p, h, :held], fmt) * (old * inv), fmt)
                with np.errstate(invalid="ignore"):
                    codes[p, h, t0 - i * page:t1 - i * page] = encode(new * inv, fmt)
                scale[p, h] = s


def sequence(codes, scale, table_row, page, fmt, first, n):
    """Rows [first, first + n) of a sequence, [H, n, d]; bad pages give NaN rows."""
    P, H, _, d = codes.shape
    out = np.full((H, n, d), np.nan)
    for t in range(n):
        p = int(table_row[(first + t) // page])
        if 0 <= p < P:
            out[:, t] = decode(codes[p, :, (first + t) % page], fmt) * scale[p][:, None]
    return out


def attend(q, k, v, scale, see):
    """q [H, N, d], k, v [HK, L, d], see [N, L] -> O, LSE, sum p |v|, and the largest sum |q k| scale of
    a row: the last two for error bounds. Rows that see nothing: 0 and -inf."""
    H, N, d = q.shape
    HK, L, _ = k.shape
    o, lse = np.zeros((H, N, d)), np.full((H, N), -np.inf)
    mag, big = np.zeros((H, N, d)), np.zeros((H, N))
    for h in range(H):
        kh, vh = k[h * HK // H], v[h * HK // H]
        for i in range(N):
            j = np.nonzero(see[i])[0]
            if not j.size:
                continue
            s = kh[j] @ q[h, i] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            lse[h, i] = m + np.log(l)
            o[h, i] = p @ vh[j] / l
            mag[h, i] = p @ np.abs(vh[j]) / l
            big[h, i] = (np.abs(kh[j]) @ np.abs(q[h, i])).max() * scale
    return o, lse, mag, big


def rotate(x, angles, positions, factor, interleaved, back=False):
    """x [B, H, N, d] with the first 2 * len(angles) channels turned by positions [B, N] times angles."""
    r = 2 * len(angles)
    th = positions[:, None, :, None].astype(np.float64) * np.asarray(angles, np.float64) * (-1 if back else 1)
    z = factor * np.exp(1j * th)
    y = np.array(x, np.float64)
    if interleaved:
        w = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * z
        y[..., 0:r:2], y[..., 1:r:2] = w.real, w.imag
    else:
        w = (x[..., :r // 2] + 1j * x[..., r // 2:r]) * z
        y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
    return y
