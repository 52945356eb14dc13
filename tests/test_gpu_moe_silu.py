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


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_gate_and_up_sums_are_fp32_ones(fmt):
    """The codes of h of tokens with outliers, against 64 bits: fp32 sums move
    hardly one, sums through the block-scaled instruction (the grouped product of
    the same operands) many.

    The partial sums of an fp32 sum over the contraction are sums over runs of it,
    at most P = the greatest less the least prefix sum in magnitude.  K additions,
    each off by at most half a step of such a sum and independent, have a root
    mean square of 2^-24 sqrt(K/3) P at most: the codes that noise of that size
    moves are the limit.  (With the sum S of the absolute products for P, eleven
    times as large here, the limit would be above what block-scaled sums move.)"""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    K = N = 1024
    T = 64
    log(f"moe gate and up sums {fmt}")
    x = inp.random_bf16((T, K), seed=11, outliers=True)
    values, w13 = _quantized(inp.random_bf16((1, 2 * N, K), seed=12, std=0.05), fmt)
    xq, xs = oracle.quantize_rowwise(x)
    xv = oracle.dequant_rowwise(xq, xs)
    sums = xv @ values[0].T
    run, low, high = np.zeros((3, T, 2 * N))
    for k in range(K):
        run += xv[:, k:k + 1] * values[0][None, :, k]
        np.minimum(low, run, out=low)
        np.maximum(high, run, out=high)

    def codes(gu):
        h = moe._silu(gu[:, :N]) * gu[:, N:]
        return moe._quantize_h(h, np.zeros_like(h))[0]

    want = codes(sums)
    noise = 2.0 ** -24 * (K / 3) ** 0.5 * (high - low) * np.random.default_rng(13).standard_normal(sums.shape)
    limit = (codes(sums + noise) != want).sum()
    batch = (_hidden(x, w13, N, fmt) != want).sum()
    single = sum((_hidden(x[t:t + 1], w13, N, fmt) != want[t:t + 1]).sum() for t in range(T))
    product = mx.mx_grouped_gemm_mxfp4 if fmt == "mxfp4" else mx.mx_grouped_gemm_mx
    scaled = product(to_dev_u8(xq), to_dev_u8(mxfp4.to_gemm_layout(xs)), *w13, to_dev_i32(np.array([T])),
                     **({} if fmt == "mxfp4" else {"mode": 0}), out_dtype=torch.float32)
    instead = (codes(scaled.cpu().numpy().astype(np.float64)) != want).sum()
    log(f"codes of {T * N} moved: {batch} in a batch, {single} one by one; limit {limit}; block-scaled sums {instead}")
    assert batch <= limit and single <= limit
    assert instead > 2 * limit


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_tokens_of_subnormal_values(fmt):
    """Tokens around 2^-128, subnormal in bf16, against weights of about 2^120."""
    require_gpu()
    K = N = 128
    rng = np.random.default_rng(21)
    x = rng.integers(-64, 65, size=(5, K)).astype(np.float64) * 2.0 ** -133       # multiples of the least bf16
    W = rng.choice([-1.0, -0.5, 0.5, 1.0], size=(1, 2 * N, K)) * 2.0 ** 120
    bits = inp.f32_to_bf16_bits(x.astype(np.float32))
    values, w13 = _quantized(inp.f32_to_bf16_bits(W.astype(np.float32)), fmt)
    xv = oracle.dequant_rowwise(*oracle.quantize_rowwise(bits))
    assert xv.any()
    gu = xv @ values[0].T
    h = moe._silu(gu[:, :N]) * gu[:, N:]
    want, far = moe._quantize_h(h, 2.0 ** -20 * np.abs(h))
    got = _hidden(bits, w13, N, fmt)
    assert want.any() and (np.abs(got - want) <= far).all()
