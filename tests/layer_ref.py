"""Plain 64-bit references of the operators that run a calibrated layer, for their tests.

The quantisation itself is the oracle's (max scaling, packed export); products and sums are taken in FP64 from decoded
codes. Nothing here calls the library.
"""
from __future__ import annotations

import numpy as np

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3_table() -> np.ndarray:
    t = np.array([oracle.e4m3_value(c) if c < 127 else np.nan for c in range(128)], np.float64)
    return np.concatenate([t, -t])


def route(ids: np.ndarray, n_experts: int):
    """(offsets, order, pos) of a stable sort of the flat ids; ids outside [0, n_experts) have no place."""
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < n_experts)
    valid = np.nonzero(ok)[0]
    srt = valid[np.argsort(flat[valid], kind="stable")]
    order = np.full(flat.size, -1, np.int32)
    order[:srt.size] = srt
    pos = np.full(flat.size, -1, np.int32)
    pos[srt] = np.arange(srt.size)
    offsets = np.zeros(n_experts + 1, np.int64)
    offsets[1:] = np.cumsum(np.bincount(flat[ok], minlength=n_experts))
    return offsets, order, pos


def quantize_tokens(x: np.ndarray, amax=None):
    """(packed u8 [n, c/2], codes u8 [n, c/16], g f32 [n], values f32 [n, c]) of f32 tokens, by the oracle: one
    "matrix" per token when the scale is the token's, else one matrix."""
    x = np.ascontiguousarray(x, np.float32)
    n, c = x.shape
    if n == 0 or c == 0:
        return np.zeros((n, c // 2), np.uint8), np.zeros((n, c // 16), np.uint8), np.zeros(n, np.float32), x
    w = x.reshape(n, 1, c) if amax is None else x.reshape(1, n, c)
    am = np.abs(x).max(1).astype(np.float32) if amax is None else np.array([amax], np.float32)
    codes, _ = oracle.baseline_scales(w, am, 0)
    packed, _, gs = oracle.pack_nvfp4(w, am, codes)
    values = oracle.fake_quant(w, am, codes)
    g = gs if amax is None else np.repeat(gs, n)
    return packed.reshape(n, c // 2), codes.reshape(n, c // 16), g.astype(np.float32), values.reshape(n, c)


def tile(codes: np.ndarray, first_row: int = 0, group: int = 0, out: np.ndarray | None = None) -> np.ndarray:
    """Scale bytes [n, J] into tiles (u8, flat), byte by byte from the definition of the order."""
    n, J = codes.shape
    steps = -(-J // 4)
    t0 = first_row // 128 + group
    if out is None:
        out = np.zeros((t0 + -(-n // 128)) * steps * 512, np.uint8)
    r, j = np.meshgrid(np.arange(n), np.arange(J), indexing="ij")
    at = ((t0 + r // 128) * steps + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4
    out[at] = codes
    return out


def untile(tiles: np.ndarray, n: int, J: int, first_row: int = 0, group: int = 0) -> np.ndarray:
    """The inverse: scale bytes [n, 4 * ceil(J / 4)] of a group's rows, padding blocks included."""
    steps = -(-J // 4)
    r, j = np.meshgrid(np.arange(n), np.arange(4 * steps), indexing="ij")
    t0 = first_row // 128 + group
    return tiles[((t0 + r // 128) * steps + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4]


def decode(packed: np.ndarray, codes: np.ndarray) -> np.ndarray:
    """q * v in FP64 [..., c] (without the global scale)."""
    nib = np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[:-1] + (-1,))
    return E2M1[nib] * np.repeat(e4m3_table()[codes], 16, -1)


def product(xv: np.ndarray, wv: np.ndarray, xg: np.ndarray, wg: float):
    """(Y, S) in FP64: the product, and the sum of the absolute terms that its rounding is measured by."""
    s = np.asarray(xg, np.float64)[:, None] * float(wg)
    return (xv @ wv.T) * s, (np.abs(xv) @ np.abs(wv).T) * np.abs(s)


def product_tolerance(y: np.ndarray, s: np.ndarray, c: int, bf16: bool) -> np.ndarray:
    """Each term of the sum is exact in FP32 (2 + 2 bits of E2M1 times 4 + 4 of E4M3). Adding them rounds, or cuts, at
    most c times, each by at most one unit (2^-23) of a partial sum that S bounds; the two scalings round three times
    by 2^-24; the output by half a step of its type."""
    t = s * (c * 2.0 ** -23 + 3 * 2.0 ** -24)
    return t + (np.abs(y) + t) * 2.0 ** -8 if bf16 else t + (np.abs(y) + t) * 2.0 ** -24
