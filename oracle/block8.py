"""fp64 oracle of the 8-bit block format, the 8-bit product and the layer's
gradients -- TEST INFRASTRUCTURE ONLY (as the rest of this package).

numpy only. e4m3 values come from a table built from the format's definition
(sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent 0 subnormal;
0x7f and 0xff NaN; no infinities), roundings from a search in that table.
Every product also returns its tolerance scale: the sum of the magnitudes of
its terms.
"""
from __future__ import annotations

import numpy as np

# top exponent of a scale for each input type: 256 * 2^n overflows it there
TOP_EXP = {"f16": 8, "bf16": 120, "f32": 120}


def e4m3_table() -> np.ndarray:
    """The 256 values of e4m3, indexed by code."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            x = np.nan
        elif e == 0:
            x = m * 2.0 ** -9
        else:
            x = (8 + m) * 2.0 ** (e - 10)
        v[c] = -x if s else x
    return v


_TABLE = e4m3_table()
_POS = _TABLE[:127]          # 0 .. 448, ascending with the code


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values (ties to the even code), |x| <= 448; NaN -> 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(_POS[hi] == a, hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def _grid(rows: int, block_rows: int) -> int:
    return -(-rows // block_rows)


def pack8(x: np.ndarray, block_rows: int, dtype: str):
    """(codes uint8 [rows, K], scales float64 [ceil(rows / block_rows), K / 128])."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    codes = np.empty((rows, K), dtype=np.uint8)
    scales = np.empty((_grid(rows, block_rows), K // 128))
    for i in range(scales.shape[0]):
        for g in range(K // 128):
            r, c = slice(i * block_rows, min(rows, (i + 1) * block_rows)), slice(128 * g, 128 * g + 128)
            b = x[r, c]
            fin = np.isfinite(b)
            top = np.abs(b[fin]).max(initial=0.0)
            n = 0
            if top > 0:
                n = -126
                # the smallest n >= -126 with top <= 448 * 2^n
                m, e = np.frexp(top)
                n = max(n, int(e) - 12)
                while top > 448 * 2.0 ** n:
                    n += 1
            cap = 240.0 if n >= TOP_EXP[dtype] else 448.0
            v = np.where(fin, np.clip(np.where(fin, b, 0.0) / 2.0 ** n, -cap, cap), np.nan)
            codes[r, c] = e4m3_codes(v)
            scales[i, g] = 2.0 ** n
    return codes, scales


def unpack8(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    """code * scale, unrounded."""
    rows, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, dtype=np.float64), 128, axis=1), block_rows, axis=0)[:rows]
    return _TABLE[codes] * s


def _product(a: np.ndarray, b: np.ndarray):
    return a @ b, np.abs(a) @ np.abs(b)


def gemm8(w, w_scales, x, x_scales):
    """(Y [T, M], tolerance scale)."""
    return _product(unpack8(x, x_scales, 1), unpack8(w, w_scales, 128).T)


def wgrad(dy: np.ndarray, x: np.ndarray):
    """dW = dY^T X and its tolerance scale; x is the unpacked checkpoint."""
    return _product(np.asarray(dy, dtype=np.float64).T, x)


def weight(planes: np.ndarray, alpha: np.ndarray) -> np.ndarray:
    """W^ = sum_k alpha_k (.) B_k from row-major words [N, M, K/32] and scales [N, M, K/G]."""
    bits = np.unpackbits(np.ascontiguousarray(planes, dtype="<u4").view(np.uint8), axis=-1, bitorder="little")
    N, M = planes.shape[:2]
    signs = 2.0 * bits.reshape(N, M, -1) - 1.0
    K = signs.shape[2]
    a = np.repeat(np.asarray(alpha, dtype=np.float64), K // alpha.shape[2], axis=2)
    return (signs * a).sum(0)


def dgrad(dy: np.ndarray, planes: np.ndarray, alpha: np.ndarray):
    """dX = dY W^ and its tolerance scale."""
    return _product(np.asarray(dy, dtype=np.float64), weight(planes, alpha))
