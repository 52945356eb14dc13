"""The product with MXFP4 weights on the GPU against the fp64 oracle on the
same codes: both activation formats, ragged, empty and single-row groups, odd
column counts, row maps, fp32 and bf16 outputs, and the bf16 entry points.

Tolerances are those of the oracle's comparison (oracle/compare.py): the final
rounding, 2e-3 of the value and the matrix instruction's summation error; the
E2M1 products themselves are exact."""

import numpy as np
import pytest

import oracle
from oracle import mxfp4
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, to_dev_u8, bf16_host_bits, log

pytestmark = pytest.mark.gpu


def _act(x, fmt):
    """(codes, row-major scales, fp64 values) of activations."""
    if fmt == "mxfp4":
        q, s = mxfp4.quantize_rowwise_fp4(x)
        return q, s, mxfp4.dequant_rowwise_fp4(q, s)
    q, s = oracle.quantize_rowwise(x)
    return q, s, oracle.dequant_rowwise(q, s)


def _operands(counts, N, K, fmt, seed, outliers=True):
    x = inp.random_bf16((sum(counts), K), seed=seed, outliers=outliers)
    W = inp.random_bf16((len(counts), N, K), seed=seed + 1, std=0.02)
    return x, _act(x, fmt), W, mxfp4.quantize_rowwise_fp4(W)


CASES = [
    ([1], 8, 128), ([0, 1, 0], 16, 128), ([5, 0, 40, 19], 72, 384), ([64, 65, 63, 1], 264, 256), ([96, 160], 512, 256),
    ([300, 0, 513, 2], 520, 640), ([256, 257], 256, 1152), ([3] * 33, 136, 256), ([300, 400], 264, 128), ([700], 8, 384),
]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,N,K", CASES)
def test_product_matches_oracle(counts, N, K, fmt):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"fp4 product {counts} N={N} K={K} {fmt}")
    x, (qx, sx, vx), W, (qw, sw) = _operands(counts, N, K, fmt, seed=N + K)
    vw = mxfp4.dequant_rowwise_fp4(qw, sw)
    offs = inp.offsets_from_counts(counts)
    ref, ab = mxfp4.grouped_product(vx, vw, offs), mxfp4.grouped_product(vx, vw, offs, absolute=True)
    args = (to_dev_u8(qx), to_dev_u8(mxfp4.to_gemm_layout(sx)), to_dev_u8(qw), to_dev_u8(mxfp4.to_gemm_layout(sw)),
            to_dev_i32(offs))
    got = mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt)
    rep = oracle.r1_check(bf16_host_bits(got), ref, abs_terms=ab)
    assert rep["ok"], rep
    f = mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt, out_dtype=torch.float32)
    rep = oracle.r1_check(f.cpu().numpy(), ref, abs_terms=ab, f32=True)
    assert rep["ok"], rep
    assert torch.equal(f.bfloat16(), got)
    # from bf16, quantized on the way: the same codes, so the same bits
    mm = mx.mx_grouped_mm_fwd_fp4(to_dev_bf16(x), args[2], args[3], args[4], act_format=fmt)
    assert torch.equal(mm, got)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", [[7, 0, 90, 33], [300, 513]])
def test_row_map_drops_and_leaves_rows(counts, fmt):
    """Rows go where the map says, dropped rows nowhere, and what no entry
    names (and what lies behind the output) stays as it was."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    N, K = 136, 256
    x, (qx, sx, _), W, (qw, sw) = _operands(counts, N, K, fmt, seed=7)
    I = sum(counts)
    offs = inp.offsets_from_counts(counts)
    args = (to_dev_u8(qx), to_dev_u8(mxfp4.to_gemm_layout(sx)), to_dev_u8(qw), to_dev_u8(mxfp4.to_gemm_layout(sw)),
            to_dev_i32(offs))
    plain = mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt)
    rng = np.random.default_rng(3)
    c_rows = I + 20
    m = rng.permutation(c_rows)[:I].astype(np.int32)
    m[::9], m[4::17] = -1, c_rows
    for dtype in (torch.bfloat16, torch.float32):
        buf = torch.full((c_rows + 1, N), 7.0, dtype=dtype, device="cuda:0")
        mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt, row_map=to_dev_i32(m), out=buf[:c_rows])
        want = torch.full((c_rows + 1, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
        keep = torch.from_numpy((m >= 0) & (m < c_rows)).to("cuda:0")
        want[torch.from_numpy(m).to("cuda:0").long()[keep]] = plain[keep]
        assert torch.equal(buf.bfloat16(), want)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("total", [100, 700])
def test_offsets_that_end_early_or_go_wrong_stay_in_bounds(total, fmt):
    """Rows behind the last group are left as they were; decreasing or
    too-large offsets are clamped, so that nothing outside is touched."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    N, K = 64, 256
    x, (qx, sx, _), W, (qw, sw) = _operands([total // 2, total - total // 2], N, K, fmt, seed=11)
    args = [to_dev_u8(qx), to_dev_u8(mxfp4.to_gemm_layout(sx)), to_dev_u8(qw), to_dev_u8(mxfp4.to_gemm_layout(sw))]
    full = mx.mx_grouped_gemm_mxfp4(*args, to_dev_i32(np.array([40, total])), x_format=fmt)
    for offs, rows in (([40, total - 30], total - 30), ([40, 40], 40), ([40, 1 << 30], total), ([40, -5], 40), ([0, 0], 0)):
        buf = torch.full((total + 3, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
        mx.mx_grouped_gemm_mxfp4(*args, to_dev_i32(np.array(offs)), x_format=fmt, out=buf[:total])
        assert torch.equal(buf[:rows], full[:rows]) and (buf[rows:] == 7).all(), offs


def test_nan_rows_and_weights_stay_where_they_are():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    counts, N, K = [20, 33], 64, 256
    for fmt in ("mxfp8", "mxfp4"):
        x = inp.random_bf16((sum(counts), K), seed=21)
        W = inp.random_bf16((2, N, K), seed=22, std=0.02)
        x[5, 77] = 0x7F80
        W[1, 13, 200] = 0x7FC0
        qw, sw, qwt, swt = mx.mx_quantize_weights_fp4(to_dev_bf16(np.concatenate([W, W], axis=1)))
        out = mx.mx_grouped_mm_fwd_fp4(to_dev_bf16(x), qw, sw, to_dev_i32(inp.offsets_from_counts(counts)), act_format=fmt)
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[5] = True
        bad[20:, 13] = True
        bad[20:, 64 + 13] = True
        assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,N,K", [([1, 0, 30], 128, 8), ([33, 70], 384, 264), ([300, 280], 256, 520)])
def test_dgrad_matches_oracle(counts, N, K, fmt):
    """dOut [M, N] against the weights blocked along N: K any multiple of 8."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    g = inp.random_bf16((sum(counts), N), seed=31, std=1e-3)
    W = inp.random_bf16((len(counts), N, K), seed=32, std=0.02)
    qwt, swt = mxfp4.quantize_colwise_fp4(W)
    _, _, vg = _act(g, fmt)
    vw = mxfp4.dequant_rowwise_fp4(qwt, swt)
    offs = inp.offsets_from_counts(counts)
    got = mx.mx_grouped_mm_dgrad_fp4(to_dev_bf16(g), to_dev_u8(qwt), to_dev_u8(mxfp4.to_gemm_layout(swt)),
                                     to_dev_i32(offs), act_format=fmt)
    rep = oracle.r1_check(bf16_host_bits(got), mxfp4.grouped_product(vg, vw, offs),
                          abs_terms=mxfp4.grouped_product(vg, vw, offs, absolute=True))
    assert rep["ok"], rep
