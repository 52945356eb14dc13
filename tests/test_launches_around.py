"""Launches of the operators around the experts' products at sizes that no test
runs, seen without a GPU (launch_record.py)."""

import mxfp8_block_scaled_06_amd as mx
from launch_record import FAKE, record

P = FAKE
BF16, F32 = 0, 1
MOST = (1 << 31) - 1


def _fits(launch):
    assert max(launch.threads) < 1 << 32, (launch.kernel, launch.grid)
    assert launch.grid[1] <= 65535 and launch.grid[2] <= 65535, (launch.kernel, launch.grid)
    assert launch.lds <= 64 * 1024


def test_threads_of_a_launch_stay_below_the_limit_of_an_axis():
    rows = 65534 * 128
    need = 1 << 60
    calls = record([
        ("mx_topk_router_fwd", (P, BF16, P, MOST, 32, 8, 0, 1, 1, 0, 1, 1.0, P, P, None)),
        ("mx_topk_router_fwd", (P, F32, P, MOST, 1024, 32, 1, 64, 8, 1, 1, 1.0, P, P, None)),
        ("mx_topk_router_fwd", (P, F32, P, MOST, 1022, 32, 1, 2, 1, 1, 1, 1.0, P, P, None)),
        ("mx_topk_router_bwd", (P, F32, P, P, P, MOST, 1024, 32, 0, 1, 1.0, P, None)),
        ("mx_topk_router_bwd", (P, BF16, P, P, P, MOST, 1, 1, 0, 1, 1.0, P, None)),
        ("mx_swiglu_fwd", (P, (1 << 27) - 1, 1024, P, P, P, None)),
        ("mx_swiglu_fwd", (P, (1 << 27) - 1, 1024, P, None, None, None)),
        ("mx_swiglu_bwd", (P, P, P, (1 << 27) - 1, 1024, P, None)),
        ("mx_swiglu_quantize", (P, P, MOST, rows, 16384, P, P, None)),
        ("mx_swiglu_quantize_fwd", (P, P, P, MOST, rows, 16384, rows, P, P, P, P, P, P, None)),
        ("mx_swiglu_quantize_bwd", (P, P, P, P, P, P, MOST, rows, 16384, rows, P, P, P, P, P, P, need, None)),
        ("mx_swiglu_quantize", (P, P, MOST, 128, (1 << 30) - 128, P, P, None)),
        ("mx_topk_combine_fwd", (P, BF16, P, P, MOST, 1024, 8192, P, None)),
        ("mx_topk_combine_fwd", (P, F32, P, P, MOST, 1, 8192, P, None)),
        ("mx_topk_combine_bwd", (P, BF16, P, P, P, MOST, 1024, 8192, P, P, None)),
        ("mx_topk_combine_bwd", (P, F32, P, P, P, MOST, 1, 8192, P, P, None)),
        ("mx_dequantize", (P, P, 1, (1 << 24) - 1, 1 << 13, mx.SCALES_ROWMAJOR, P, None)),
        ("mx_dequantize", (P, P, 1, (1 << 24) - 1, 1 << 13, mx.SCALES_GEMM, P, None)),
    ])
    for i, call in enumerate(calls):
        assert call.status == 0, (i, call.text)
        assert call.launches
        for launch in call.launches:
            _fits(launch)
    dequant = calls[-1].launches[0]
    assert dequant.grid[0] * dequant.grid[1] * dequant.block[0] * 8 >= ((1 << 24) - 1) << 13        # 8 codes a thread


def test_sizes_beyond_a_launch_are_refused():
    need = 1 << 60
    calls = record([
        ("mx_topk_router_fwd", (P, BF16, P, MOST + 1, 32, 8, 0, 1, 1, 0, 1, 1.0, P, P, None)),
        ("mx_swiglu_fwd", (P, 1 << 27, 1024, P, P, P, None)),
        ("mx_swiglu_quantize", (P, P, MOST, 128, 1 << 30, P, P, None)),
        ("mx_swiglu_quantize_fwd", (P, P, P, MOST, 65535 * 128, 128, 65535 * 128, P, P, P, P, P, P, None)),
        ("mx_swiglu_quantize_bwd", (P, P, P, P, P, P, MOST, 65535 * 128, 128, 65535 * 128, P, P, P, P, P, P, need, None)),
        ("mx_topk_combine_bwd", (P, BF16, P, P, P, MOST + 1, 8, 8192, P, P, None)),
    ])
    for call in calls:
        assert call.status == 2 and not call.launches, call.text


def test_nothing_to_do_launches_nothing():
    calls = record([
        ("mx_topk_router_fwd", (None, BF16, None, 0, 32, 8, 0, 1, 1, 0, 1, 1.0, None, None, None)),
        ("mx_topk_router_bwd", (None, BF16, None, None, None, 0, 32, 8, 0, 1, 1.0, None, None)),
        ("mx_swiglu_fwd", (None, 0, 1024, None, None, None, None)),
        ("mx_swiglu_fwd", (None, 4, 0, None, None, None, None)),
        ("mx_swiglu_bwd", (None, None, None, 0, 1024, None, None)),
        ("mx_swiglu_quantize", (None, None, 0, 0, 128, None, None, None)),
        ("mx_topk_combine_fwd", (None, BF16, None, None, 0, 8, 64, None, None)),
        ("mx_topk_combine_bwd", (P, BF16, P, None, P, 4, 8, 64, None, None, None)),
        ("mx_dequantize", (None, None, 1, 0, 128, mx.SCALES_GEMM, None, None)),
    ])
    for i, call in enumerate(calls):
        assert call.status == 0 and not call.launches, (i, call.text)


def test_slots_of_a_token_share_a_workgroup_up_to_eight():
    for k, slots in ((1, 1), (2, 1), (4, 1), (8, 1), (9, 2), (1024, 128)):
        call, = record([("mx_topk_combine_bwd", (P, BF16, P, P, P, 7, k, 128, P, P, None))])
        assert tuple(call.launches[0].grid) == (7, 1, slots)


def test_scales_from_which_no_score_comes_back_are_refused():
    for scale, status in ((2.0 ** -64, 0), (2.0 ** 64, 0), (2.0 ** -65, 2), (2.0 ** 65, 2), (1e-45, 2), (-1.0, 2), (float("nan"), 2)):
        for call in record([("mx_topk_router_fwd", (P, BF16, P, 4, 32, 8, 0, 1, 1, 0, 1, scale, P, P, None)),
                            ("mx_topk_router_bwd", (P, BF16, P, P, P, 4, 32, 8, 0, 1, scale, P, None))]):
            assert call.status == status and bool(call.launches) == (status == 0), (scale, call.text)


def test_rows_of_logits_may_start_at_any_token():
    """logits[t0:] and a gradient there: four elements' alignment where rows are multiples of four, else one's."""
    for kind, E, past, status in ((F32, 32, 16, 0), (F32, 32, 8, 3), (F32, 30, 4, 0), (F32, 30, 2, 3), (BF16, 32, 8, 0),
                                  (BF16, 20, 8, 0), (BF16, 20, 4, 3), (BF16, 30, 2, 0), (BF16, 30, 1, 3)):
        for call in record([("mx_topk_router_fwd", (P + past, kind, P, 4, E, 2, 0, 1, 1, 0, 1, 1.0, P, P, None)),
                            ("mx_topk_router_bwd", (P + past, kind, P, P, P, 4, E, 2, 0, 1, 1.0, P, None)),
                            ("mx_topk_router_bwd", (P, kind, P, P, P, 4, E, 2, 0, 1, 1.0, P + past, None))]):
            assert call.status == status and bool(call.launches) == (status == 0), (kind, E, past, call.text)
