"""CPU oracle for the MXFP4 quantizers (E2M1 elements, E8M0 scales per 32).

TEST INFRASTRUCTURE ONLY, like the rest of this package: plain numpy in fp64,
sharing no code with the HIP path.

The format is the MX format of mxfp8.py with 4-bit elements: the scale byte is
clamp(floor(log2 amax) - 2, -127, 127) + 127 (0x00 for zeros, 0xFF when the
block holds a NaN or an Inf), the element is the E2M1 number nearest to
value * 2^(127 - byte) (a value halfway between two goes to the even code),
saturated to +-6, sign kept; the elements of a NaN/Inf block are code 0.
Codes are packed two to a byte, the even element low.
"""

from __future__ import annotations

import numpy as np

from .mxfp8 import BLOCK, E8M0_NAN, _as3d, bf16_to_f64, e8m0_value, group_bounds

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(codes: np.ndarray) -> np.ndarray:
    c = np.asarray(codes, dtype=np.uint8)
    v = E2M1[c & 7]
    return np.where(c & 8, -v, v)


def e2m1_encode(y: np.ndarray) -> np.ndarray:
    """Nearest code of every value, by distance to all eight magnitudes; of two
    equally near ones the even code."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), 6.0)
    code = np.zeros(a.shape, dtype=np.int64)
    best = np.full(a.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):              # even codes first: they win ties
        d = np.abs(a - E2M1[c])
        code = np.where(d < best, c, code)
        best = np.minimum(d, best)
    return (code | (np.signbit(y).astype(np.int64) << 3)).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    """[..., C] codes -> [..., C/2] bytes."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    q = np.asarray(q, dtype=np.uint8)
    return np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def _blocks(v: np.ndarray):
    """fp64 [..., nblocks, 32] -> (codes, scale bytes [..., nblocks])."""
    bad = ~np.isfinite(v).all(axis=-1)
    amax = np.max(np.abs(np.where(np.isfinite(v), v, 0.0)), axis=-1)
    byte = np.zeros(amax.shape, dtype=np.int64)
    pos = amax > 0
    _, p = np.frexp(amax[pos])
    byte[pos] = np.clip(p.astype(np.int64) - 1 - 2, -127, 127) + 127
    q = e2m1_encode(np.where(bad[..., None], 0.0, v) * np.exp2(127.0 - byte)[..., None])
    q[np.broadcast_to(bad[..., None], q.shape)] = 0
    byte[bad] = E8M0_NAN
    return q, byte.astype(np.uint8)


def quantize_rowwise_fp4(x_bits: np.ndarray):
    """bf16 bits [..., C] -> packed codes [..., C/2], scale bytes [..., C/32]."""
    v = bf16_to_f64(x_bits)
    q, s = _blocks(v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK))
    return pack(q.reshape(v.shape)), s


def quantize_colwise_fp4(x_bits: np.ndarray):
    """bf16 bits [B?, R, C] -> blocks along R, stored transposed: packed codes
    [B?, C, R/2], scale bytes [B?, C, R/32]."""
    squeeze = np.asarray(x_bits).ndim == 2
    q, s = quantize_rowwise_fp4(np.ascontiguousarray(np.swapaxes(_as3d(x_bits), 1, 2)))
    return (q[0], s[0]) if squeeze else (q, s)


def dequant_rowwise_fp4(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return e2m1_decode(unpack(q)) * np.repeat(e8m0_value(s), BLOCK, axis=-1)


def to_gemm_layout(s: np.ndarray) -> np.ndarray:
    """Row-major scale bytes [B?, R, KB] -> [B?, KB/4, R, 4]."""
    t = s.reshape(*s.shape[:-1], s.shape[-1] // 4, 4)
    return np.ascontiguousarray(np.swapaxes(t, -3, -2))


def grouped_product(X: np.ndarray, Y: np.ndarray, offs, absolute: bool = False) -> np.ndarray:
    """out[g_e] = X[g_e] @ Y[e]^T of dequantized fp64 operands X [I, K], Y
    [E, J, K]; rows of no group stay zero.  absolute=True sums |x| |y|."""
    f = np.abs if absolute else (lambda v: v)
    out = np.zeros((X.shape[0], Y.shape[1]), dtype=np.float64)
    for e, (a, b) in enumerate(group_bounds(offs, X.shape[0])):
        if b > a:
            out[a:b] = f(X[a:b]) @ f(Y[e]).T
    return out
