"""GPU parity of the MXFP4 quantizers and dequantizer: codes and scale bytes
equal to the oracle's (every bf16 pattern among them), values exact."""

import numpy as np
import pytest

from mxfp8_block_scaled_06_amd import inputs as inp
from oracle import mxfp4
from gpu_util import require_gpu, to_dev_bf16, to_dev_u8, u8_host, log

pytestmark = pytest.mark.gpu


def _values(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("shape", [(1, 32), (1, 5120), (33, 5120), (7, 96), (2, 5, 128), (3, 129, 2048), (257, 160)])
@pytest.mark.parametrize("layout", ["rowmajor", "gemm"])
def test_rowwise_matches_oracle(shape, layout):
    require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    if layout == "gemm" and shape[-1] % 128:
        pytest.skip("the GEMM layout needs 128-multiples")
    log(f"fp4 rowwise {shape} {layout}")
    x = inp.random_bf16(shape, seed=sum(shape), outliers=True)
    x.reshape(-1)[::97] = 0
    q, s = mx.mx_quantize_rowwise_fp4(to_dev_bf16(x), scale_layout=layout)
    rq, rs = mxfp4.quantize_rowwise_fp4(x)
    assert np.array_equal(u8_host(q), rq)
    assert np.array_equal(u8_host(s), mxfp4.to_gemm_layout(rs) if layout == "gemm" else rs)
    v = mx.mx_dequantize_fp4(q, s, scale_layout=layout)
    assert np.array_equal(_values(v), mxfp4.dequant_rowwise_fp4(rq, rs))


def test_every_bf16_pattern():
    """Blocks of every exponent: each block holds 31 of the patterns and, so
    that the scale varies, one value of another binade (or none)."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    pats = inp.all_bf16_patterns()
    pats = pats[(pats & 0x7F80) != 0x7F80]          # finite
    n = -(-len(pats) // 31)
    body = np.resize(pats, n * 31).reshape(n, 31)
    cases = []
    for top in (0, 0x0001, 0x0080, 0x00FF, 0x0180, 0x0280, 0x3F80, 0x7F7F):
        cases.append(np.concatenate([body, np.full((n, 1), top, dtype=np.uint16)], axis=1))
    x = np.concatenate(cases).astype(np.uint16)
    q, s = mx.mx_quantize_rowwise_fp4(to_dev_bf16(x))
    rq, rs = mxfp4.quantize_rowwise_fp4(x)
    assert np.array_equal(u8_host(s), rs)
    assert np.array_equal(u8_host(q), rq)


def test_nonfinite_blocks_and_every_scale_byte():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x = inp.random_bf16((64, 256), seed=5)
    x[3, 40], x[9, 0], x[17, 255] = 0x7F80, 0xFF80, 0x7FC1
    q, s = mx.mx_quantize_rowwise_fp4(to_dev_bf16(x))
    rq, rs = mxfp4.quantize_rowwise_fp4(x)
    assert np.array_equal(u8_host(q), rq) and np.array_equal(u8_host(s), rs)
    v = _values(mx.mx_dequantize_fp4(q, s))
    assert np.array_equal(np.isnan(v), np.repeat(rs == 255, 32, axis=1)) and (rs == 255).sum() == 3
    # the dequantizer over all codes of all scale bytes, sign of zero included
    codes = np.tile(mxfp4.pack(np.resize(np.arange(16, dtype=np.uint8), 32))[None], (256, 1))
    sb = np.arange(256, dtype=np.uint8)[:, None]
    got = mx.mx_dequantize_fp4(to_dev_u8(codes), to_dev_u8(sb)).cpu().view(torch.int16).numpy().view(np.uint16)
    ref = mxfp4.dequant_rowwise_fp4(codes, sb)
    want = torch.from_numpy(ref).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    fine = ~np.isnan(ref)
    assert np.array_equal(got[fine], want[fine]) and (got[255] & 0x7FFF > 0x7F80).all()


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (2, 256, 384), (3, 384, 256), (1, 640, 1152), (2, 512, 768)])
def test_weights_match_oracle(E, N, K):
    require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"fp4 weights {E} {N} {K}")
    W = inp.random_bf16((E, N, K), seed=E + N + K, std=0.02, outliers=True)
    W[0, 5, 7], W[-1, 100, 64] = 0x7F80, 0xFFC0
    got = mx.mx_quantize_weights_fp4(to_dev_bf16(W))
    rq, rs = mxfp4.quantize_rowwise_fp4(W)
    cq, cs = mxfp4.quantize_colwise_fp4(W)
    for name, g, r in zip(("q", "s", "q_t", "s_t"), got, (rq, mxfp4.to_gemm_layout(rs), cq, mxfp4.to_gemm_layout(cs))):
        assert np.array_equal(u8_host(g), r), name


def test_caller_buffers_stream_and_odd_rows_stay():
    """Outputs go where the caller says, on the stream that is current, and
    nothing behind them is written."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x = to_dev_bf16(inp.random_bf16((37, 96), seed=3))
    qbuf = torch.full((38 * 48,), 0xAB, dtype=torch.uint8, device="cuda:0")
    sbuf = torch.full((38 * 3,), 0xCD, dtype=torch.uint8, device="cuda:0")
    q, s = qbuf[:37 * 48].view(37, 48), sbuf[:37 * 3].view(37, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.mx_quantize_rowwise_fp4(x, q=q, s=s)
        v = mx.mx_dequantize_fp4(q, s)
    side.synchronize()
    want = mx.mx_quantize_rowwise_fp4(x)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and torch.equal(v, mx.mx_dequantize_fp4(*want))
    assert (qbuf[37 * 48:] == 0xAB).all() and (sbuf[37 * 3:] == 0xCD).all()
    with pytest.raises(ValueError, match="contiguous"):
        mx.mx_quantize_rowwise_fp4(x.t())
    with pytest.raises(ValueError, match="shape"):
        mx.mx_dequantize_fp4(q, s[:30])
