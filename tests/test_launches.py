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
