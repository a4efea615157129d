"""The 8-bit cache's number format and the appends' arithmetic in float64 numpy, written from their definitions
(include/pkv.h) and independent of the library: the references of the 8-bit cache's tests."""
from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -80, 100
NAN_CODE = 0x7F


def _grid() -> np.ndarray:
    """Values of the e4m3 codes 0x00 .. 0x7e (exponent bias 7, subnormals of 2^-9)."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e > 0, np.ldexp(1.0 + m / 8.0, e - 7), m * 2.0 ** -9)


GRID = _grid()
CODE_VALUES = np.concatenate([GRID, [np.nan], -GRID, [np.nan]])  # of the codes 0 .. 255


def to_codes(y: np.ndarray) -> np.ndarray:
    """float64 values as the nearest e4m3 codes, ties to the even code, saturating; NaN to the NaN code."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), E4M3_MAX)
    hi = np.searchsorted(GRID, a)  # first grid value >= a
    lo = np.maximum(hi - 1, 0)
    below, above = a - GRID[lo], GRID[hi] - a
    pick_hi = (above < below) | ((above == below) & (hi % 2 == 0))
    code = np.where(pick_hi, hi, lo).astype(np.uint8)
    code = code | np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(y), NAN_CODE | np.where(np.signbit(y), 0x80, 0), code).astype(np.uint8)


def row_exponent(x: np.ndarray) -> np.ndarray:
    """e of the rows (last axis) of x: the least integer with max |finite x_i| <= 448 * 2^e, clamped."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=-1)
    m, e = np.frexp(a / 256.0)  # a = m 2^(e + 8), m in [0.5, 1); 448 * 2^k = 0.875 * 2^(k + 9)
    k = np.where(m <= 0.875, e - 1, e)
    return np.where(a == 0, EXP_MIN, np.clip(k, EXP_MIN, EXP_MAX)).astype(np.int64)


def quantise(x: np.ndarray):
    """Rows of x (float64) as (e4m3 codes, scale bytes)."""
    e = row_exponent(x)
    with np.errstate(invalid="ignore"):
        return to_codes(np.ldexp(x, -e[..., None])), (e + 127).astype(np.uint8)


def dequantise(codes: np.ndarray, scale_bytes: np.ndarray) -> np.ndarray:
    return np.ldexp(CODE_VALUES[codes], (scale_bytes.astype(np.int64) - 127)[..., None])


def codes_of(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def random_cache(seed, num_pages, hkv, d, *, spread=0.5):
    """A seeded 8-bit cache of quantised normal rows, rows and channels of different sizes: (k codes, v codes, scale
    bytes) with scales [pages, hkv, 2, 16]."""
    rng = np.random.default_rng(seed)
    ch = np.exp(spread * rng.standard_normal((hkv, 1, d)))
    rows = np.exp(spread * rng.standard_normal((num_pages, hkv, 16, 1)))
    kc, ks = quantise(rng.standard_normal((num_pages, hkv, 16, d)) * ch)
    vc, vs = quantise(rng.standard_normal((num_pages, hkv, 16, d)) * rows)
    return kc, vc, np.stack([ks, vs], axis=2)


def cache_to(kc, vc, sc, device):
    put = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(device).view(t)  # noqa: E731
    return put(kc, torch.float8_e4m3fn), put(vc, torch.float8_e4m3fn), put(sc, torch.float8_e8m0fnu)


def rotate64(x, weight, cos_sin, eps):
    """q or k rows [n, heads, d] (float64): y of include/pkv.h and, elementwise, (|u1| + |u2|) * norm, the size that
    fp32's errors are relative to. weight [d] or None, cos_sin [n, d] (the tokens' table rows) or None."""
    d = x.shape[-1]
    u = x if weight is None else x * weight
    norm = 1.0 if weight is None else 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    if cos_sin is None:
        return u * norm, np.abs(u) * norm
    c, s = cos_sin[:, None, : d // 2], cos_sin[:, None, d // 2:]
    u1, u2 = u[..., : d // 2], u[..., d // 2:]
    y = np.concatenate([u1 * c - u2 * s, u2 * c + u1 * s], axis=-1)
    size = np.concatenate([np.abs(u1) + np.abs(u2)] * 2, axis=-1)
    return y * norm, size * norm


def fp32_noise(d, size):
    """Bound on the fp32 error of y: the sum of squares (d terms and the shuffles, halved by the square root), the
    reciprocal square root, the products and the sum of a pair, the norm's product -- each at most 2^-24 relative to
    `size`."""
    return (d / 2 + 16) * 2.0 ** -24 * size


def attention64(q, k, v, scale):
    """One request: q [hq, d], k and v [n, hkv, d] (float64) -> (out, sum_j p_j |v_j|, the largest sum |q| |k_j|
    per head), in 64 bits."""
    hq, d = q.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    qg = q.reshape(hkv, g, d)
    kk, vv = k.transpose(1, 0, 2), v.transpose(1, 0, 2)
    s = np.einsum("hgd,hnd->hgn", qg, kk) * scale
    p = np.exp(s - s.max(axis=-1, keepdims=True))
    p /= p.sum(axis=-1, keepdims=True)
    out = np.einsum("hgn,hnd->hgd", p, vv).reshape(hq, d)
    absolute = np.einsum("hgn,hnd->hgd", p, np.abs(vv)).reshape(hq, d)
    size = np.einsum("hgd,hnd->hgn", np.abs(qg), np.abs(kk)).max(axis=-1).reshape(hq)
    return out, absolute, size


def decode_bound(out, absolute, size, scale, d, n, vmax):
    """Elementwise bound on |got - out| of the decode call over the 8-bit cache, from its roundings:
    bf16 output 2^-8; the fp16 weights 2^-11; the approximate exponentials, their arguments' last bits and the split
    records' 16 significant bits, 2^-14 together; the fp32 score sums over d products, (d + 8) 2^-24 of
    scale * sum |q||k|, which moves numerator and denominator; fp16's smallest weight, 2^-38 of the largest, n times."""
    ds = (d + 8) * 2.0 ** -24 * scale * size[:, None]
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -14 + 2 * ds) * absolute + n * 2.0 ** -38 * vmax + 1e-37
