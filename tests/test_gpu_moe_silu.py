"""The hidden layer of the few-token layer, code by code: SiLU at the ends of its
range.  The down weights are an identity and the combine weights one, so the
output shows the codes of h = silu(g) * u themselves (four significant bits:
exact in bf16)."""

import numpy as np
import pytest

import oracle
from oracle import moe, mxfp4
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, to_dev_u8, bf16_host_bits, log

pytestmark = pytest.mark.gpu


def _quantized(W, fmt):
    """bf16 bits [E, J, C] -> (values, the layer's operand)."""
    quantize, restore = ((mxfp4.quantize_rowwise_fp4, mxfp4.dequant_rowwise_fp4) if fmt == "mxfp4" else
                         (oracle.quantize_rowwise, oracle.dequant_rowwise))
    q, s = quantize(W)
    return restore(q, s), (to_dev_u8(q), to_dev_u8(mxfp4.to_gemm_layout(s)))


def _identity(n, fmt):
    return _quantized(inp.f32_to_bf16_bits(np.eye(n, dtype=np.float32)[None]), fmt)[1]


def _hidden(x, w13, n, fmt):
    """MX8(silu(g) * u) of every token, read through identity down weights."""
    import torch
    import mxfp8_block_scaled_06_amd as mx
    T = x.shape[0]
    out = mx.mx_moe_few_tokens(to_dev_bf16(x), to_dev_i32(np.zeros(T, dtype=np.int32)),
                               torch.ones(T, device="cuda:0"), w13, _identity(n, fmt), weight_format=fmt)
    return oracle.bf16_to_f64(bf16_host_bits(out))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("gates,gate_exp,up_exp", [
    # gates to 1.5 * 2^127 = 2.6e38, past which -x log2 e overflows; -1.5 * 2^127 has a silu of 0
    ([1.5, 1.0, 0.5, -1.5, -1.0], 127, -122),
    # silu(-88) = -5.3e-37: the reciprocal of 1 + e^88 is subnormal, the result is not
    ([-5.5, -5.0, -5.5], 4, 120),
    # the same beside gates that outweigh it by e^80
    ([-5.5, -0.5, 0.5, 0.0], 4, 100),
])
def test_ends_of_the_range_of_silu(gates, gate_exp, up_exp, T, fmt):
    """Gate sums exact in fp32, as x[0] * W[n, 0] + x[1] * W[n, 1]; up sums a
    power of two, from another block of x and of W."""
    require_gpu()
    K = N = 128
    log(f"moe silu {gates} * 2^{gate_exp}, up 2^{up_exp}, T={T} {fmt}")
    a = gate_exp // 2                                # x[0] = x[1] = 2^a, x[32] = 2^b
    b = up_exp // 2
    x = np.zeros((T, K), dtype=np.float32)
    x[:, 0] = x[:, 1] = 2.0 ** a
    x[:, 32] = 2.0 ** b
    g = np.resize(np.array(gates), N)
    W = np.zeros((1, 2 * N, K), dtype=np.float32)
    # two parts that are E2M1 values in one block (5.5 = 4 + 1.5, 4.5 = 4 + 0.5, ...)
    whole = np.trunc(g / 2) * 2
    W[0, :N, 0] = np.where(np.abs(g) >= 4, np.sign(g) * 4, whole) * 2.0 ** (gate_exp - a)
    W[0, :N, 1] = np.where(np.abs(g) >= 4, g - np.sign(g) * 4, g - whole) * 2.0 ** (gate_exp - a)
    W[0, N:, 32] = 2.0 ** (up_exp - b)
    values, w13 = _quantized(inp.f32_to_bf16_bits(W), fmt)
    xv = oracle.dequant_rowwise(*oracle.quantize_rowwise(inp.f32_to_bf16_bits(x)))
    gu = xv @ values[0].T
    assert np.array_equal(gu[0, :N], g * 2.0 ** gate_exp) and (gu[:, N:] == 2.0 ** up_exp).all()
    with np.errstate(over="ignore"):
        h = moe._silu(gu[:, :N]) * gu[:, N:]
    # silu to 2^-20 of itself, as the layer's oracle allows, reaches one code only:
    # the result is then that code
    want, far = moe._quantize_h(h, 2.0 ** -20 * np.abs(h))
    assert not far.any() and want.any()
    if up_exp == 120:
        assert (want != 0).all()
    got = _hidden(inp.f32_to_bf16_bits(x), w13, N, fmt)
    assert np.array_equal(got, want), (got[0, :8], want[0, :8])
