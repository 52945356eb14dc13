"""CPU oracle of the gated MoE layer, with a bound on how far fp32 may be off.

TEST INFRASTRUCTURE ONLY: numpy in fp64, no code shared with the HIP path.

    g, u = MX8(x) W13[e]^T;  h = MX8(silu(g) * u);  out = sum_j c_j (h W2[e_j]^T)

MX8 is the MXFP8 quantization along the contraction; the weights are given as
values (their codes already decoded).  h is rounded to 3 mantissa bits, so an
fp32 h a hair beside the exact one may round to the neighbouring code: the
bound counts, for every element of h, the codes that its error interval
reaches, through |W2|.
"""

from __future__ import annotations

import numpy as np

from .compare import ulp_bf16
from .mxfp8 import BLOCK, dequant_rowwise, e4m3_decode, e4m3_encode, e8m0_from_amax, quantize_blocks, quantize_rowwise


def _silu(g):
    return g / (1.0 + np.exp(-g))


def _quantize_h(h, d):
    """(values of MX8(h), largest distance to the values that h +- d may give)."""
    b, db = h.reshape(-1, BLOCK), d.reshape(-1, BLOCK)
    q, s = quantize_blocks(b)
    v = e4m3_decode(q) * np.exp2(s.astype(np.float64) - 127)[:, None]
    far = np.zeros_like(v)
    a = np.abs(b)
    ok = np.zeros(len(b), dtype=bool)
    for top in ((a + db).max(1), np.maximum(a - db, 0).max(1)):
        sc = e8m0_from_amax(top, ok).astype(np.float64)[:, None]
        for y in (b - db, b, b + db):
            far = np.maximum(far, np.abs(e4m3_decode(e4m3_encode(y * np.exp2(127 - sc))) * np.exp2(sc - 127) - v))
    return v.reshape(h.shape), far.reshape(h.shape)


def moe_layer(x_bits, ids, combine, w13, w2, u_mfma, u_down=None):
    """(out fp64 [T, K], bound on |bf16 result - out|).  w13 [E, 2N, K] and w2
    [E, K, N] fp64 values; u_mfma: error of a matrix sum per unit of the sum of
    its absolute products (u_down, where given: of the down projection's)."""
    u_down = u_mfma if u_down is None else u_down
    T, k = ids.shape
    E, N = w13.shape[0], w2.shape[2]
    x = dequant_rowwise(*quantize_rowwise(x_bits))
    out = np.zeros((T, w2.shape[1]))
    tol = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            gu = w13[e] @ x[t]
            # matrix sum, then seven fp32 additions of partial sums
            dgu = (u_mfma + 2.0 ** -21) * (np.abs(w13[e]) @ np.abs(x[t]))
            g, u, dg, du = gu[:N], gu[N:], dgu[:N], dgu[N:]
            h = _silu(g) * u
            # |silu'| < 1.1; expf, one addition, a division and a product in fp32
            d = np.abs(u) * 1.1 * dg + np.abs(_silu(g)) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(h)
            hq, far = _quantize_h(h, d)
            c = float(combine[t, j])
            out[t] += c * (w2[e] @ hq)
            aw = np.abs(w2[e])
            tol[t] += abs(c) * (aw @ far + (u_down + 2.0 ** -20) * (aw @ (np.abs(hq) + far)))
    return out, tol + 0.5 * ulp_bf16(np.abs(out) + tol)
