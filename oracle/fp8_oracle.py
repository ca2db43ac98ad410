"""float64 definitions of the norm in front of the layer, its backward, and the products in 8 bits (NumPy).

e4m3 values are tried one by one (``levels``), scales found by doubling and halving: nothing is shared with
the library's bit arithmetic."""
from __future__ import annotations

import numpy as np

__all__ = ["e4m3_levels", "e4m3_decode", "fp8_scale_exponent", "fp8_quantize_rows", "fp8_row_values",
           "fp8_quantize_weights", "fp8_weight_values", "fp8_pack_weights", "rms_norm", "rms_norm_backward", "fp8_linear", "fp8_ffn"]

BLOCK = 128


def e4m3_levels() -> np.ndarray:
    """The 127 magnitudes by code: 8 subnormal steps of 2^-9, then eight values an octave up to 448."""
    out = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        out += [(1 + m / 8) * 2.0 ** (e - 7) for m in range(8)]
    return np.array(out[:127])


def e4m3_decode(codes) -> np.ndarray:
    lv = np.append(e4m3_levels(), np.nan)
    codes = np.asarray(codes)
    return np.where(codes >= 128, -1.0, 1.0) * lv[codes & 127]


def fp8_scale_exponent(top: float) -> int:
    """The least e >= -126 with top <= 448 * 2^e; 0 for zero."""
    if top == 0:
        return 0
    e = 0
    while top > 448 * 2.0 ** e:
        e += 1
    while e > -126 and top <= 448 * 2.0 ** (e - 1):
        e -= 1
    return e


def _nearest_codes(share: np.ndarray) -> np.ndarray:
    """Codes of values already divided by their scale: nearest level, ties to the even code; not finite: NaN."""
    lv = e4m3_levels()
    a = np.abs(share)
    with np.errstate(invalid="ignore"):
        hi = np.clip(np.searchsorted(lv, a), 1, 126)
        lo = hi - 1
        dl, dh = a - lv[lo], lv[hi] - a
        code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isfinite(share), code, 127)
    return (code | np.where(np.signbit(share), 128, 0)).astype(np.uint8)


def _largest(block) -> float:
    a = np.abs(block[np.isfinite(block)])
    return float(a.max()) if a.size else 0.0


def fp8_quantize_rows(x):
    """codes [rows, K up to whole blocks] (zeros behind K), exponents [rows, blocks]."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    nb = -(-K // BLOCK)
    codes = np.zeros((rows, nb * BLOCK), dtype=np.uint8)
    e = np.zeros((rows, nb), dtype=np.int64)
    for r in range(rows):
        for b in range(nb):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            e[r, b] = fp8_scale_exponent(_largest(v))
            codes[r, b * BLOCK:b * BLOCK + len(v)] = _nearest_codes(v / 2.0 ** e[r, b])
    return codes, e


def fp8_row_values(codes, e, K) -> np.ndarray:
    return (e4m3_decode(codes) * np.repeat(2.0 ** e.astype(np.float64), BLOCK, axis=1))[:, :K]


def fp8_quantize_weights(w):
    """codes [N, K] and exponents [N / 128, K / 128] (up to whole blocks) of one matrix."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    codes = np.zeros((N, K), dtype=np.uint8)
    e = np.zeros((-(-N // BLOCK), -(-K // BLOCK)), dtype=np.int64)
    for i in range(e.shape[0]):
        for j in range(e.shape[1]):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            e[i, j] = fp8_scale_exponent(_largest(w[at]))
            codes[at] = _nearest_codes(w[at] / 2.0 ** e[i, j])
    return codes, e


def fp8_weight_values(codes, e) -> np.ndarray:
    scale = np.repeat(np.repeat(2.0 ** e.astype(np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return e4m3_decode(codes) * scale[:codes.shape[0], :codes.shape[1]]


def fp8_pack_weights(matrices):
    """The library's layout of one group, byte by byte from its description: `matrices` holds (codes, exponents) of the one
    matrix, or of the gate and of the up rows."""
    N, K = matrices[0][0].shape
    H, nt, kt, nb = len(matrices), -(-N // 16), -(-K // BLOCK), -(-N // BLOCK)
    ks, blocks = -(-kt // 4) * 4, nt * H
    out = np.zeros(blocks * kt * 2048, dtype=np.uint8)
    scale = np.full((nb, H, ks), 127, dtype=np.uint8)
    for h, (codes, e) in enumerate(matrices):
        for n in range(N):
            for k in range(K):
                block = n // 16 * H + h
                tile, b = block // 16, min(16, blocks - block // 16 * 16)
                piece = (k // 64) * b + block % 16
                out[tile * 16 * kt * 2048 + piece * 1024 + 256 * (k % 64 // 16) + 16 * (n % 16) + k % 16] = codes[n, k]
        scale[:, h, :kt] = e + 127
    return out, scale.reshape(-1)


def rms_norm(x, residual, weight, eps, held=lambda a: a):
    """h (rounded by `held`, the layer's type), rstd, y."""
    h = held(np.asarray(x, dtype=np.float64) + (0 if residual is None else np.asarray(residual, dtype=np.float64)))
    with np.errstate(all="ignore"):
        rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
        return h, rstd, h * rstd[:, None] * np.asarray(weight, dtype=np.float64)


def rms_norm_backward(dy, h, weight, rstd, dh=None):
    g, xhat = dy * weight, h * rstd[:, None]
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * xhat).sum(axis=0)


def fp8_linear(rows, w):
    """Rows of values times one matrix (codes, exponents)."""
    return rows @ fp8_weight_values(*w).T


def fp8_ffn(rows, gate, up, down):
    """One group's FFN: y, and the H it was formed from, before and after its rounding to 8 bits."""
    g, u = fp8_linear(rows, gate), fp8_linear(rows, up)
    h = g / (1 + np.exp(-g)) * u
    held = fp8_row_values(*fp8_quantize_rows(h), h.shape[1])
    return fp8_linear(held, down), h, held
