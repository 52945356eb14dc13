"""The few-token MoE layer on the GPU against the fp64 oracle, within the
oracle's own bound (fp32 sums, the codes of h that an error interval reaches,
one bf16 rounding): both weight formats, 1 to 128 tokens, repeated, missing and
invalid experts, NaN in weights and tokens, graphs, streams and workspaces, and
the layer as the sum of the framework's other entry points."""

import numpy as np
import pytest

import oracle
from oracle import moe, mxfp4
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, to_dev_u8, bf16_host_bits, log

pytestmark = pytest.mark.gpu

# Error of a block-scaled matrix sum per unit of its absolute products.  The
# instruction aligns a block's products to the largest of them and drops what
# lies far below, so the coefficient goes by the range of the factors: E4M3
# spans 2^-9 .. 2^8 on the tokens' side whatever the weights' format, and every
# E2M1 number is an E4M3 number, so the oracle's coefficient for E4M3 x E4M3
# bounds both (measured on E4M3 x E2M1 sums, K = 128 .. 4096: at most 1.6e-4,
# a third of it).
U = oracle.compare.U_MFMA


def _quantized(W, fmt):
    if fmt == "mxfp4":
        q, s = mxfp4.quantize_rowwise_fp4(W)
        return mxfp4.dequant_rowwise_fp4(q, s), (to_dev_u8(q), to_dev_u8(mxfp4.to_gemm_layout(s)))
    q, s = oracle.quantize_rowwise(W)
    return oracle.dequant_rowwise(q, s), (to_dev_u8(q), to_dev_u8(mxfp4.to_gemm_layout(s)))


def _f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda:0")


def _routing(rng, T, k, E):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if k <= E else \
        rng.integers(0, E, size=(T, k)).astype(np.int32)
    c = rng.random((T, k)).astype(np.float32)
    return ids, (c / c.sum(1, keepdims=True)).astype(np.float32)


def _case(T, k, E, K, N, fmt, seed):
    rng = np.random.default_rng(seed)
    x = inp.random_bf16((T, K), seed=seed, outliers=True)
    v13, w13 = _quantized(inp.random_bf16((E, 2 * N, K), seed=seed + 1, std=0.05), fmt)
    v2, w2 = _quantized(inp.random_bf16((E, K, N), seed=seed + 2, std=0.05), fmt)
    ids, c = _routing(rng, T, k, E)
    return x, ids, c, v13, w13, v2, w2


def _check(out, ref, tol):
    got = oracle.bf16_to_f64(bf16_host_bits(out))
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float((err / tol).max()), int((~(err <= tol)).sum()))
    # Over all outputs less is left of the bound: a rounding error is spread evenly
    # over +- half a step, a root mean square of 1/sqrt(3) = 0.577 of the bound
    # (the other terms add errors up that in fact cancel, and leave less).  Of n >= 128
    # outputs the mean square scatters by sqrt(4/5/n) = 8%, its root by 4%: 0.7 is
    # five times that away.
    assert np.linalg.norm(got - ref) <= 0.7 * np.linalg.norm(tol)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,k,E,K,N", [
    (1, 1, 1, 128, 128), (1, 1, 5, 384, 256), (1, 4, 8, 256, 128), (3, 2, 40, 128, 384), (16, 2, 3, 640, 128),
    (17, 1, 2, 256, 256), (33, 3, 4, 128, 128), (65, 2, 5, 256, 128), (128, 1, 1, 128, 256), (128, 8, 9, 128, 128),
    (5, 32, 64, 128, 128), (2, 3, 1024, 128, 128),
])
def test_layer_matches_oracle(T, k, E, K, N, fmt):
    require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"moe T={T} k={k} E={E} K={K} N={N} {fmt}")
    x, ids, c, v13, w13, v2, w2 = _case(T, k, E, K, N, fmt, seed=T + 10 * k + E + K + N)
    out = mx.mx_moe_few_tokens(to_dev_bf16(x), to_dev_i32(ids), _f32(c), w13, w2, weight_format=fmt)
    _check(out, *moe.moe_layer(x, ids, c, v13, v2, U))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,k", [(1, 1), (40, 2)])
def test_exact_sums(T, k, fmt):
    """Gate and up sums that fp32 holds exactly (multiples of 2^-7, factors of
    few binades): what is left is the SwiGLU, the roundings and the down sums."""
    require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(T)
    E, K, N = 3, 256, 128
    pick = lambda vals, shape: inp.f32_to_bf16_bits(rng.choice(np.array(vals, dtype=np.float32), size=shape))  # noqa: E731
    x = pick([1, -1, 2, .5, 0], (T, K))
    v13, w13 = _quantized(pick([.5, -.5, .25, 0, .125], (E, 2 * N, K)), fmt)
    v2, w2 = _quantized(pick([1, -1, .5, 0], (E, K, N)), fmt)
    ids, c = _routing(rng, T, k, E)
    out = mx.mx_moe_few_tokens(to_dev_bf16(x), to_dev_i32(ids), _f32(c), w13, w2, weight_format=fmt)
    _check(out, *moe.moe_layer(x, ids, c, v13, v2, 0.0, U))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_repeated_and_invalid_experts(fmt):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    T, k, E, K, N = 19, 3, 4, 256, 128
    x, ids, c, v13, w13, v2, w2 = _case(T, k, E, K, N, fmt, seed=77)
    ids[3] = [2, 2, 2]                       # one expert three times
    ids[4] = [1, 0, 1]
    ids[5] = [-1, E, 1 << 30]                # none
    ids[6] = [7, 3, -5]                      # one of three
    args = (to_dev_bf16(x), to_dev_i32(ids), _f32(c), w13, w2)
    out = mx.mx_moe_few_tokens(*args, weight_format=fmt, check=False)
    _check(out, *moe.moe_layer(x, ids, c, v13, v2, U))
    assert not out[5].any()
    with pytest.raises(ValueError, match="outside"):
        mx.mx_moe_few_tokens(*args, weight_format=fmt)
    none = torch.full((T, k), -1, dtype=torch.int32, device="cuda:0")
    assert not mx.mx_moe_few_tokens(args[0], none, *args[2:], weight_format=fmt, check=False).any()
    assert mx.mx_moe_few_tokens(args[0][:0], none[:0], args[2][:0], w13, w2, weight_format=fmt).shape == (0, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_nan_reaches_only_its_own_tokens(fmt):
    """A NaN in a token or in an expert's weights reaches the tokens that have
    it and no other, whose results keep their bits."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    T, k, E, K, N = 20, 2, 4, 128, 128
    rng = np.random.default_rng(5)
    x = inp.random_bf16((T, K), seed=90)
    W13, W2 = inp.random_bf16((E, 2 * N, K), seed=91, std=0.05), inp.random_bf16((E, K, N), seed=92, std=0.05)
    ids, c = _routing(rng, T, k, E)
    run = lambda xx, a, b: mx.mx_moe_few_tokens(to_dev_bf16(xx), to_dev_i32(ids), _f32(c), _quantized(a, fmt)[1],  # noqa: E731
                                                _quantized(b, fmt)[1], weight_format=fmt)
    clean = run(x, W13, W2)
    xb = x.copy()
    xb[7, 3] = 0x7FC0
    got = run(xb, W13, W2)
    assert torch.isnan(got[7]).all() and torch.equal(torch.cat((got[:7], got[8:])), torch.cat((clean[:7], clean[8:])))
    has = torch.from_numpy((ids == 2).any(1)).to("cuda:0")
    for a, b in ((1, 0), (0, 1)):
        w13, w2 = W13.copy(), W2.copy()
        if a:
            w13[2, 5, 5] = 0x7F80
        else:
            w2[2, :, 9] = 0x7FC0
        got = run(x, w13, w2)
        assert torch.isnan(got[has]).all() and torch.equal(got[~has], clean[~has])


def test_equals_the_grouped_path():
    """The same layer from the framework's routing, grouped product and torch:
    the same operands, so only fp32 order and the bf16 rounding of the hidden
    layer differ there."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    T, k, E, K, N = 50, 2, 4, 256, 256
    x, ids, c, v13, w13, v2, w2 = _case(T, k, E, K, N, "mxfp4", seed=101)
    xd, idd, cd = to_dev_bf16(x), to_dev_i32(ids), _f32(c)
    out = mx.mx_moe_few_tokens(xd, idd, cd, w13, w2).double()
    offs, rows, _, _ = mx.mx_route(idd.reshape(-1), E)
    tokens = torch.where(rows >= 0, rows // k, rows)                 # grouped row -> token
    qx, sx = mx.mx_quantize_rowwise_gather(xd, tokens.int())
    gu = mx.mx_grouped_gemm_mxfp4(qx, sx, *w13, offs, row_map=rows, c_rows=T * k, out_dtype=torch.float32)
    g, u = gu.chunk(2, -1)
    h = torch.nn.functional.silu(g) * u
    qh, sh = mx.mx_quantize_rowwise_gather(h.bfloat16(), rows)
    y = mx.mx_grouped_gemm_mxfp4(qh, sh, *w2, offs, row_map=rows, c_rows=T * k, out_dtype=torch.float32)
    ref = (y.view(T, k, K) * cd[:, :, None]).sum(1).double()
    # h rounded to bf16 moves it by 2^-9 of itself at most half the time across
    # the border of an E4M3 code (steps of 2^-3 .. 2^-4): at most one element in
    # 2^-8 / 2^-4 = 1/16 by one step of at most 2^-3, an error of sqrt(1/16) / 8
    # relative to the norm
    assert (out - ref).norm() <= (1 / 32 + 2.0 ** -8) * ref.norm()


def test_workspace_output_and_what_lies_behind():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    T, k, E, K, N = 6, 2, 4, 256, 128
    x, ids, c, v13, w13, v2, w2 = _case(T, k, E, K, N, "mxfp4", seed=111)
    args = (to_dev_bf16(x), to_dev_i32(ids), _f32(c), w13, w2)
    want = mx.mx_moe_few_tokens(*args)
    need = mx.mx_moe_few_tokens_workspace_bytes(T, k, N)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda:0")    # not initialised
    buf = torch.full((T + 2, K), 7.0, dtype=torch.bfloat16, device="cuda:0")
    got = mx.mx_moe_few_tokens(*args, out=buf[:T], ws=ws[:need])
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)
    assert (buf[T:] == 7).all() and (ws[need:] == 0xFF).all()
    with pytest.raises(mx.MXError, match="workspace"):
        mx.mx_moe_few_tokens(*args, ws=ws[:need - 1])
    flat = mx.mx_moe_few_tokens(args[0], args[1][:, 0].contiguous(), args[2][:, 0].contiguous(), w13, w2)
    one = mx.mx_moe_few_tokens(args[0], args[1][:, :1].contiguous(), args[2][:, :1].contiguous(), w13, w2)
    assert torch.equal(flat, one)


def test_graph_replays_follow_their_inputs():
    """Captured once, replayed on changed tokens, experts and weights, with
    eager work between the replays."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    T, k, E, K, N = 9, 2, 5, 256, 256
    x, ids, c, v13, w13, v2, w2 = _case(T, k, E, K, N, "mxfp4", seed=121)
    xd, idd, cd = to_dev_bf16(x), to_dev_i32(ids), _f32(c)
    ws = torch.empty(mx.mx_moe_few_tokens_workspace_bytes(T, k, N), dtype=torch.uint8, device="cuda:0")
    out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda:0")
    call = lambda: mx.mx_moe_few_tokens(xd, idd, cd, w13, w2, check=False, out=out, ws=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    rng = np.random.default_rng(9)
    for r in range(4):
        ids2, c2 = _routing(rng, T, k, E)
        xd.copy_(to_dev_bf16(inp.random_bf16((T, K), seed=130 + r, outliers=True)))
        idd.copy_(to_dev_i32(ids2))
        cd.copy_(_f32(c2))
        if r == 2:
            w2[0].copy_(w2[0].flip(0))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, mx.mx_moe_few_tokens(xd, idd, cd, w13, w2)), r


def test_two_streams_with_their_own_workspaces():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    cases = [_case(T, 2, 6, 512, 512, "mxfp4", seed=140 + T) for T in (4, 30)]
    args = [(to_dev_bf16(x), to_dev_i32(ids), _f32(c), w13, w2) for x, ids, c, _, w13, _, w2 in cases]
    want = [mx.mx_moe_few_tokens(*a, check=False) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (s, a) in enumerate(zip(streams, args)):
            with torch.cuda.stream(s):
                got[i].append(mx.mx_moe_few_tokens(*a, check=False))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_inputs_that_want_a_gradient_are_refused():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, ids, c, v13, w13, v2, w2 = _case(2, 1, 2, 128, 128, "mxfp4", seed=150)
    xd = to_dev_bf16(x).requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        mx.mx_moe_few_tokens(xd, to_dev_i32(ids), _f32(c), w13, w2)
    with torch.no_grad():
        mx.mx_moe_few_tokens(xd, to_dev_i32(ids), _f32(c), w13, w2)
    with pytest.raises(ValueError, match="w2 codes"):
        mx.mx_moe_few_tokens(xd.detach(), to_dev_i32(ids), _f32(c), w13, w2[::-1])
    with pytest.raises(ValueError, match="expert_idx"):
        mx.mx_moe_few_tokens(xd.detach(), to_dev_i32(ids), _f32(c[:, 0]), w13, w2)
