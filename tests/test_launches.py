"""Launches of the MXFP4 operators and the few-token layer at sizes that no test
runs, seen without a GPU (launch_record.py)."""

import mxfp8_block_scaled_06_amd as mx
from launch_record import FAKE, record

P = FAKE
CU_LDS = 160 * 1024


def _layer(T, topk, E, K, N, fmt):
    need = 1 << 40
    return ("mx_moe_few_tokens", (P, P, P, P, P, P, P, fmt, T, topk, K, N, E, P, None, P, need, None))


def test_launches_are_seen():
    small, large, none = record([
        ("mx_grouped_gemm_mxfp4", (P, P, 0, P, P, mx.SCALES_GEMM, P, 64, 64, 128, 2, None, 0, P, 0, None)),
        ("mx_grouped_gemm_mxfp4", (P, P, 0, P, P, mx.SCALES_GEMM, P, 4096, 4096, 128, 2, None, 0, P, 0, None)),
        ("mx_grouped_gemm_mxfp4", (P, P, 0, P, P, mx.SCALES_GEMM, P, 0, 4096, 128, 2, None, 0, P, 0, None)),
    ])
    assert small.status == large.status == none.status == 0
    assert [len(c.launches) for c in (small, large, none)] == [1, 1, 0]
    assert "small" in small.launches[0].kernel and "small" not in large.launches[0].kernel
    assert large.limits == [(large.launches[0].kernel, large.launches[0].lds)]


def test_layers_of_all_shapes_share_one_lds_limit_per_kernel():
    """The limit of a kernel's LDS belongs to the process: a call that set it to
    its own need could lower it between another thread's setting and launch."""
    shapes = [(T, k, E, K, N) for T in (1, 7, 40, 128) for k in (1, 8, 32) for E in (2, 64, 1024)
              for K, N in ((128, 128), (7168, 2048), (65536, 128), (1024, 8192))]
    calls = record([_layer(*s, fmt) for s in shapes for fmt in (0, 1)])
    limits = {}
    for call in calls:
        assert call.status == 0, call.text
        assert len(call.launches) == 2
        for kernel, value in call.limits:
            limits.setdefault(kernel, set()).add(value)
    for call in calls:
        for launch in call.launches:
            assert launch.lds <= min(limits[launch.kernel]) and max(limits[launch.kernel]) <= CU_LDS
    assert all(len(v) == 1 for v in limits.values()), limits


def test_threads_of_a_launch_stay_below_the_limit_of_an_axis():
    """A launch takes fewer than 2^32 threads along an axis.  Up to the documented
    2^32 - 1 blocks of 32 the row quantizers, alone or in a product, need more."""
    rows, cols, tiny = (1 << 24) - 1, 1 << 13, 64      # 2^32 - 2^8 blocks
    need = 1 << 60
    calls = record([
        ("mx_quantize_rowwise", (P, 1, rows, cols, P, P, None)),
        ("mx_quantize_rowwise_gather", (P, 100, P, rows, cols, P, P, None)),
        ("mx_quantize_rowwise_fp4", (P, 1, rows, cols, P, P, mx.SCALES_ROWMAJOR, None)),
        ("mx_quantize_rowwise_fp4", (P, 1, rows, cols, P, P, mx.SCALES_GEMM, None)),
        ("mx_dequantize_fp4", (P, P, 1, rows, cols, mx.SCALES_ROWMAJOR, P, None)),
        ("mx_dequantize_fp4", (P, P, 1, rows, cols, mx.SCALES_GEMM, P, None)),
        ("mx_grouped_mm_fwd_q", (P, P, P, P, rows, tiny, cols, 1, P, P, need, None)),
        ("mx_grouped_mm_dgrad_q", (P, P, P, P, rows, cols, tiny, 1, P, P, need, None)),
        ("mx_grouped_mm_fwd_fp4", (P, P, P, P, rows, tiny, cols, 1, 0, P, P, need, None)),
        ("mx_grouped_mm_fwd_fp4", (P, P, P, P, rows, tiny, cols, 1, 1, P, P, need, None)),
        ("mx_grouped_mm_dgrad_fp4", (P, P, P, P, rows, cols, tiny, 1, 0, P, P, need, None)),
    ])
    for i, call in enumerate(calls):
        assert call.status == 0, (i, call.text)
        assert call.launches
        for launch in call.launches:
            assert max(launch.threads) < 1 << 32, (launch.kernel, launch.grid)
            assert launch.grid[1] <= 65535 and launch.grid[2] <= 65535, (launch.kernel, launch.grid)
    quantizer = calls[0].launches[0]
    assert quantizer.grid[0] * quantizer.grid[1] * quantizer.block[0] * 16 >= rows * cols      # 16 values a thread


def test_products_refuse_before_anything_is_launched():
    """A product that the multiplication would refuse does not quantize its rows
    first."""
    rows, need = (1 << 31) - 1, 1 << 60
    calls = record([("mx_grouped_mm_fwd_fp4", (P, P, P, P, rows, 256, 128, 1, fmt, P, P, need, None)) for fmt in (0, 1)]
                   + [("mx_grouped_mm_dgrad_fp4", (P, P, P, P, rows, 128, 256, 1, fmt, P, P, need, None)) for fmt in (0, 1)]
                   + [("mx_grouped_mm_fwd_fp4", (P, P, P, P, 1 << 20, 1 << 31, 128, 1, fmt, P, P, need, None)) for fmt in (0, 1)])
    calls += record([(f"mx_grouped_mm_{op}_fp4", (P, P, P + 2, P, 4096, 4096, 4096, 1, fmt, P, P, need, None))
                     for op in ("fwd", "dgrad") for fmt in (0, 1)])
    for i, call in enumerate(calls):
        assert call.status == (2 if i < 6 else 3), call.text
        assert not call.launches, call.launches[0].kernel
        assert "mx_grouped_mm" in call.text, call.text


def test_row_quantizer_refuses_misaligned_scale_dwords():
    """Scales in the GEMM layout are stored as dwords, row-major ones as bytes."""
    args = lambda s, layout: ("mx_quantize_rowwise_fp4", (P, 1, 64, 256, P, s, layout, None))  # noqa: E731
    bad, good, rowmajor = record([args(P + 2, mx.SCALES_GEMM), args(P + 4, mx.SCALES_GEMM), args(P + 1, mx.SCALES_ROWMAJOR)])
    assert bad.status == 3 and "4-byte" in bad.text and not bad.launches
    assert good.status == rowmajor.status == 0 and len(good.launches) == len(rowmajor.launches) == 1
