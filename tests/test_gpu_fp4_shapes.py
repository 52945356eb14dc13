"""The MXFP4 operators and the few-token layer at the borders of their rules:
products on either side of the choice of tile, quantizers with one and several
steps per workgroup, layers whose work runs across experts and weight blocks,
random shapes, and all of them in one program (train, quantize, decode).

Tolerances are the oracle's (oracle/compare.py, oracle/moe.py)."""

import contextlib

import numpy as np
import pytest

import oracle
from oracle import moe, mxfp4
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, to_dev_u8, bf16_host_bits, u8_host, log

pytestmark = pytest.mark.gpu


def _act(x, fmt):
    if fmt == "mxfp4":
        q, s = mxfp4.quantize_rowwise_fp4(x)
        return q, s, mxfp4.dequant_rowwise_fp4(q, s)
    q, s = oracle.quantize_rowwise(x)
    return q, s, oracle.dequant_rowwise(q, s)


def _product(counts, N, K, fmt, seed):
    """Operands on the device (rows, weights, offsets) and the fp64 product."""
    x = inp.random_bf16((sum(counts), K), seed=seed, outliers=True)
    W = inp.random_bf16((len(counts), N, K), seed=seed + 1, std=0.02)
    qx, sx, vx = _act(x, fmt)
    qw, sw = mxfp4.quantize_rowwise_fp4(W)
    vw = mxfp4.dequant_rowwise_fp4(qw, sw)
    offs = inp.offsets_from_counts(counts)
    args = (to_dev_u8(qx), to_dev_u8(mxfp4.to_gemm_layout(sx)), to_dev_u8(qw), to_dev_u8(mxfp4.to_gemm_layout(sw)),
            to_dev_i32(offs))
    return x, args, mxfp4.grouped_product(vx, vw, offs), mxfp4.grouped_product(vx, vw, offs, absolute=True)


def _small(counts, N):
    """Whether the small workgroups take it: at most 640 cover the output."""
    I = sum(counts)
    return (I // 64 + min(len(counts), I)) * -(-N // 32) <= 640


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,N,K,small", [
    ([576], 2048, 640, True), ([640], 2048, 640, False), ([1], 20480, 128, True), ([1], 20488, 128, False),
    ([0, 300, 1, 513], 2056, 384, False), ([256, 257, 0, 40, 700], 1288, 1152, False), ([64] * 33, 600, 256, False),
    ([255, 1, 256, 2, 0, 511], 4104, 128, False), ([33] * 16, 640, 1408, True),
])
def test_product_on_both_sides_of_the_tile_rule(counts, N, K, small, fmt):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    assert _small(counts, N) is small
    log(f"fp4 product {counts} N={N} K={K} {fmt}")
    x, args, ref, ab = _product(counts, N, K, fmt, seed=N + K)
    got = mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt)
    rep = oracle.r1_check(bf16_host_bits(got), ref, abs_terms=ab)
    assert rep["ok"], rep
    f = mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt, out_dtype=torch.float32)
    rep = oracle.r1_check(f.cpu().numpy(), ref, abs_terms=ab, f32=True)
    assert rep["ok"], rep
    assert torch.equal(f.bfloat16(), got)
    assert torch.equal(mx.mx_grouped_mm_fwd_fp4(to_dev_bf16(x), *args[2:], act_format=fmt), got)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_large_tiles_with_maps_early_ends_and_nan(fmt):
    """The 256 x 256 tiles: rows scattered through a map with drops, offsets that
    end early or go wrong, rows behind the last group, NaN in one row and column."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    counts, N, K = [300, 0, 257, 143], 2056, 256
    assert not _small(counts, N)
    M = sum(counts)
    x, args, _, _ = _product(counts, N, K, fmt, seed=7)
    plain = mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt)
    m = np.random.default_rng(3).permutation(M + 50)[:M].astype(np.int32)
    m[::9] = -1
    buf = torch.full((M + 51, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
    mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt, row_map=to_dev_i32(m), out=buf[:M + 50])
    want = torch.full_like(buf, 7.0)
    keep = torch.from_numpy(m >= 0).to("cuda:0")
    want[torch.from_numpy(m).to("cuda:0").long()[keep]] = plain[keep]
    assert torch.equal(buf, want)
    for offs, rows in (([300, 300, 557, M - 30], M - 30), ([300, 300, 300, 300], 300), ([300, 300, 557, 1 << 30], M),
                       ([300, -7, -9, -9], 300), ([0, 0, 0, 0], 0)):
        buf = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
        mx.mx_grouped_gemm_mxfp4(*args[:4], to_dev_i32(np.array(offs)), x_format=fmt, out=buf[:M])
        assert torch.equal(buf[:rows], plain[:rows]) and (buf[rows:] == 7).all(), offs
    x = x.copy()
    x[5, 77] = 0x7F80
    W = inp.random_bf16((4, N, K), seed=22, std=0.02)
    W[2, 1301, 200] = 0x7FC0
    q, s = mxfp4.quantize_rowwise_fp4(W)
    out = mx.mx_grouped_mm_fwd_fp4(to_dev_bf16(x), to_dev_u8(q), to_dev_u8(mxfp4.to_gemm_layout(s)), args[4], act_format=fmt)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[5] = True
    bad[300:557, 1301] = True
    assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("counts,N", [([40, 90], 520), ([300, 513], 2056)])
def test_product_in_a_graph_and_on_another_stream(counts, N):
    """Captured with its own workspace and replayed on changed rows and offsets,
    with eager calls between the replays."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    K, M = 384, sum(counts)
    W = to_dev_bf16(inp.random_bf16((2, N, K), seed=61, std=0.02))
    w = mx.mx_quantize_weights_fp4(torch.cat((W, W[:, :1].expand(2, -N % 128, K)), 1).contiguous())[:2]
    A = to_dev_bf16(inp.random_bf16((M, K), seed=62))
    offs = to_dev_i32(inp.offsets_from_counts(counts))
    ws = torch.empty(mx.mx_grouped_mm_fp4_workspace_bytes(M, K), dtype=torch.uint8, device="cuda:0")
    out = torch.empty((M, w[0].shape[1]), dtype=torch.bfloat16, device="cuda:0")
    call = lambda: mx.mx_grouped_mm_fwd_fp4(A, *w, offs, out=out, ws=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    want = mx.mx_grouped_mm_fwd_fp4(A, *w, offs)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for r in range(4):
        A.copy_(to_dev_bf16(inp.random_bf16((M, K), seed=70 + r)))
        offs.copy_(to_dev_i32(np.array([counts[0] - 9 * r, M])))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, mx.mx_grouped_mm_fwd_fp4(A, *w, offs)), r


@pytest.mark.parametrize("shape", [(8200, 2176), (3, 2741, 2176), (2, 5, 128), (1, 70, 384), (9, 8, 640)])
def test_quantizer_steps_and_tails_in_both_layouts(shape):
    require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    torch = require_gpu()
    log(f"fp4 rowwise {shape}")
    x = inp.random_bf16(shape, seed=sum(shape), outliers=True)
    rq, rs = mxfp4.quantize_rowwise_fp4(x)
    q, s = mx.mx_quantize_rowwise_fp4(to_dev_bf16(x))
    qg, sg = mx.mx_quantize_rowwise_fp4(to_dev_bf16(x), scale_layout="gemm")
    assert np.array_equal(u8_host(q), rq) and np.array_equal(u8_host(s), rs)
    assert np.array_equal(u8_host(qg), rq) and np.array_equal(u8_host(sg), mxfp4.to_gemm_layout(rs))
    v, vg = mx.mx_dequantize_fp4(q, s), mx.mx_dequantize_fp4(qg, sg, scale_layout="gemm")
    assert torch.equal(v, vg)
    assert np.array_equal(oracle.bf16_to_f64(bf16_host_bits(v)), mxfp4.dequant_rowwise_fp4(rq, rs))


def _weights(W, fmt):
    q, s = (mxfp4.quantize_rowwise_fp4 if fmt == "mxfp4" else oracle.quantize_rowwise)(W)
    v = (mxfp4.dequant_rowwise_fp4 if fmt == "mxfp4" else oracle.dequant_rowwise)(q, s)
    return v, (to_dev_u8(q), to_dev_u8(mxfp4.to_gemm_layout(s)))


def _layer(T, k, E, K, N, fmt, seed, ids=None):
    import torch
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(seed)
    x = inp.random_bf16((T, K), seed=seed, outliers=True)
    v13, w13 = _weights(inp.random_bf16((E, 2 * N, K), seed=seed + 1, std=0.05), fmt)
    v2, w2 = _weights(inp.random_bf16((E, K, N), seed=seed + 2, std=0.05), fmt)
    if ids is None:
        ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    c = rng.random((T, k)).astype(np.float32)
    args = (to_dev_bf16(x), to_dev_i32(ids), torch.from_numpy(c).to("cuda:0"), w13, w2)
    out = mx.mx_moe_few_tokens(*args, weight_format=fmt)
    assert torch.equal(out, mx.mx_moe_few_tokens(*args, weight_format=fmt))     # a fixed order of additions
    ref, tol = moe.moe_layer(x, ids, c, v13, v2, oracle.compare.U_MFMA)
    err = np.abs(oracle.bf16_to_f64(bf16_host_bits(out)) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), int((~(err <= tol)).sum()))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,k,E,K,N", [
    (7, 2, 12, 128, 4096),        # 128 blocks an expert over 256 workgroups: runs across experts
    (40, 1, 2, 256, 9088),        # more than 16 tokens an expert, 284 blocks
    (50, 1, 2, 7168, 128),        # as many tokens of an expert as LDS holds x of
    (128, 32, 3, 128, 128),       # every token names an expert many times
    (3, 1, 2, 16384, 128), (100, 2, 70, 384, 640),
])
def test_layers_whose_work_crosses_experts_and_blocks(T, k, E, K, N, fmt):
    require_gpu()
    log(f"moe T={T} k={k} E={E} K={K} N={N} {fmt}")
    _layer(T, k, E, K, N, fmt, seed=T + K + N)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_longest_contraction(fmt):
    """K = 2^16, the documented limit: LDS holds x of two tokens."""
    require_gpu()
    log(f"moe K=65536 {fmt}")
    _layer(5, 1, 1, 65536, 128, fmt, seed=5, ids=np.zeros((5, 1), dtype=np.int32))


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(seed):
    require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(1000 + seed)
    fmt = ("mxfp8", "mxfp4")[seed % 2]
    E = int(rng.integers(1, 12))
    counts = [int(c) for c in rng.integers(0, 1 + int(rng.choice([3, 70, 400])), size=E)]
    N, K = 8 * int(rng.integers(1, 200)), 128 * int(rng.integers(1, 7))
    log(f"seed {seed}: product {counts} N={N} K={K} {fmt}")
    if sum(counts):
        x, args, ref, ab = _product(counts, N, K, fmt, seed)
        rep = oracle.r1_check(bf16_host_bits(mx.mx_grouped_gemm_mxfp4(*args, x_format=fmt)), ref, abs_terms=ab)
        assert rep["ok"], rep
    T, k, E = int(rng.integers(1, 129)), int(rng.integers(1, 9)), int(rng.integers(1, 40))
    K, N = 128 * int(rng.integers(1, 9)), 128 * int(rng.integers(1, 9))
    log(f"seed {seed}: moe T={T} k={k} E={E} K={K} N={N} {fmt}")
    _layer(T, k, E, K, N, fmt, seed)


def test_training_then_decoding():
    """The operators as a program uses them: MXFP4 products trained for some
    steps (one of them captured), then the weights quantized once and tokens
    decoded with the few-token layer, which equals the trained layer's own
    forward within the bound of its oracle on the same weights."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    E, K, N, T = 3, 256, 128, 24
    rng = np.random.default_rng(17)
    W13 = to_dev_bf16(inp.random_bf16((E, 2 * N, K), seed=201, std=0.05)).requires_grad_()
    W2 = to_dev_bf16(inp.random_bf16((E, K, N), seed=202, std=0.05)).requires_grad_()
    x = to_dev_bf16(inp.random_bf16((96, K), seed=203))
    grad = to_dev_bf16(inp.random_bf16((96, K), seed=204, std=0.1))
    offs = to_dev_i32(np.array([32, 32, 96]))

    def step():
        h = mx.mx_grouped_mm(x, W13, offs, check_offsets=False, weight_format="mxfp4")
        g, u = h.chunk(2, -1)
        a = (torch.nn.functional.silu(g) * u).contiguous()
        y = mx.mx_grouped_mm(a, W2, offs, check_offsets=False, weight_format="mxfp4")
        return torch.autograd.grad(y, (W13, W2), grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        with torch.no_grad():
            graph.replay()
            torch.cuda.synchronize()
            kept = [c.clone() for c in captured]
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
        assert not eager[0][1].any() and not eager[1][1].any()       # no tokens, no gradient
        with torch.no_grad():
            W13 -= 0.02 * eager[0]
            W2 -= 0.02 * eager[1]

    with torch.no_grad():
        w13, w2 = mx.mx_quantize_weights_fp4(W13)[:2], mx.mx_quantize_weights_fp4(W2)[:2]
        ids = rng.integers(0, E, size=(T, 2)).astype(np.int32)
        c = rng.random((T, 2)).astype(np.float32)
        out = mx.mx_moe_few_tokens(x[:T].contiguous(), to_dev_i32(ids), torch.from_numpy(c).to("cuda:0"), w13, w2)
    v = [mxfp4.dequant_rowwise_fp4(*mxfp4.quantize_rowwise_fp4(bf16_host_bits(w.detach()))) for w in (W13, W2)]
    assert np.array_equal(u8_host(w13[0]), mxfp4.quantize_rowwise_fp4(bf16_host_bits(W13.detach()))[0])
    ref, tol = moe.moe_layer(bf16_host_bits(x[:T].contiguous()), ids, c, v[0], v[1], oracle.compare.U_MFMA)
    err = np.abs(oracle.bf16_to_f64(bf16_host_bits(out)) - ref)
    assert (err <= tol).all(), float((err / tol).max())


def test_more_values_than_one_grid_axis_holds():
    """Past 2^35 values the quantizer's and dequantizer's threads exceed 2^32
    (the limit of a grid axis): the last rows come out like rows of their own."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rows, cols = (1 << 22) + 8, 8192
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GiB of free GPU memory")
    log("fp4 quantize and restore 2^35 + 2^16 values")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda:0")
    tail = to_dev_bf16(inp.random_bf16((8, cols), seed=77))
    x[-8:] = tail
    q, s = mx.mx_quantize_rowwise_fp4(x)
    del x
    tq, ts = mx.mx_quantize_rowwise_fp4(tail)
    assert torch.equal(q[-8:], tq) and torch.equal(s[-8:], ts) and not q[:-8:4099].any()
    v = mx.mx_dequantize_fp4(q, s)
    assert torch.equal(v[-8:], mx.mx_dequantize_fp4(tq, ts)) and not v[:-8:4099].any()
    del q, s, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,N,K", [([1], 8, 128), ([5, 0, 40, 19], 72, 384), ([16], 4096, 4096),
                                        ([3, 61, 2], 512, 896), ([0, 0], 64, 128)])
def test_rows_quantized_in_the_product_give_the_same_bits(counts, N, K, fmt):
    """Small products quantize their bf16 rows themselves: the same codes and
    scales as the quantizers', NaN blocks, zeros, subnormals and the largest
    values included, so the same bits as the two calls."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    M, E = sum(counts), len(counts)
    x = inp.random_bf16((M, K), seed=K, outliers=True)
    if M > 3:
        x[0, 5], x[1, 40], x[2, 100] = 0x7FC0, 0xFF80, 0x7F7F        # NaN, -Inf, the largest
        x[3, :64] = 0
        x[3, 64:96] = np.arange(32, dtype=np.uint16) | 0x8000        # subnormal, negative
    W = to_dev_bf16(inp.random_bf16((E, -(-N // 128) * 128, K), seed=9, std=0.02))
    qw, sw, _, _ = mx.mx_quantize_weights_fp4(W)
    qw, sw = qw[:, :N].contiguous(), sw[:, :, :N].contiguous()
    offs, xd = to_dev_i32(inp.offsets_from_counts(counts)), to_dev_bf16(x)
    if fmt == "mxfp8":
        q, s = mx.mx_quantize_rowwise(xd)
        s = mx.mx_scales_to_gemm_layout(s) if M else s.view(K // 128, 0, 4)
    else:
        q, s = mx.mx_quantize_rowwise_fp4(xd, scale_layout="gemm")
    want = mx.mx_grouped_gemm_mxfp4(q, s, qw, sw, offs, x_format=fmt)
    got = mx.mx_grouped_mm_fwd_fp4(xd, qw, sw, offs, act_format=fmt)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    if M > 3:
        assert torch.isnan(got[:2]).all() and not torch.isnan(got[2:]).any()
    # on another stream, twice in a graph, rows behind the last group left alone
    buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
    ws = torch.empty(max(1, mx.mx_grouped_mm_fp4_workspace_bytes(M, K, fmt)), dtype=torch.uint8, device="cuda:0")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_grouped_mm_fwd_fp4(xd, qw, sw, offs, act_format=fmt, out=buf[:M], ws=ws)
    for _ in range(3):
        buf.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf[:M].view(torch.int16), want.view(torch.int16)) and (buf[M:] == 7).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("ids,E,K,N", [
    ([3], 5, 128, 128), ([4, 1, 4, 0, 1], 6, 384, 640), ([-1, 7, 2, 9, 2], 8, 256, 256), ([-1], 2, 128, 128),
    (list(range(31, -1, -1)), 40, 128, 256), ([1023, 0, 512, 1 << 30], 1024, 128, 128), ([5, 3, 0, 2, 7, 6, 1, 4], 8, 256, 4096),
])
def test_one_token_finds_the_experts_that_a_batch_finds(ids, E, K, N, fmt):
    """A single token's experts are found in registers: the same bits as with a
    second token that names none, repeated and invalid ids included."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"moe one token {ids} E={E} K={K} N={N} {fmt}")
    x = to_dev_bf16(inp.random_bf16((2, K), seed=E + N, outliers=True))
    q = mx.mx_quantize_weights_fp4 if fmt == "mxfp4" else mx.mx_quantize_weights
    w13 = q(to_dev_bf16(inp.random_bf16((E, 2 * N, K), seed=1, std=0.05)))[:2]
    w2 = q(to_dev_bf16(inp.random_bf16((E, K, N), seed=2, std=0.05)))[:2]
    i = torch.full((2, len(ids)), -1, dtype=torch.int32, device="cuda:0")
    i[0] = torch.tensor(ids, dtype=torch.int32)
    c = torch.rand((2, len(ids)), device="cuda:0")
    two = mx.mx_moe_few_tokens(x, i, c, w13, w2, weight_format=fmt, check=False)
    one = mx.mx_moe_few_tokens(x[:1].contiguous(), i[:1].contiguous(), c[:1].contiguous(), w13, w2, weight_format=fmt,
                               check=False)
    assert torch.equal(one[0], two[0]) and not two[1].any()
    if any(0 <= e < E for e in ids):
        assert one.any()
    with pytest.raises(ValueError, match="outside") if any(not 0 <= e < E for e in ids) else contextlib.nullcontext():
        mx.mx_moe_few_tokens(x[:1].contiguous(), i[:1].contiguous(), c[:1].contiguous(), w13, w2, weight_format=fmt)
