"""The differentiable products with MXFP4 weights: output and both gradients
against the fp64 oracle of the formulas, against differences, in the routed
path (top-1 and top-k), and the treatment of caches and prequantized weights.
"""

import numpy as np
import pytest

import oracle
from oracle import mxfp4
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, bf16_host_bits, log

pytestmark = pytest.mark.gpu


def _vals(bits):
    q, s = oracle.quantize_rowwise(bits)
    return oracle.dequant_rowwise(q, s)


def _forms(A, W, G, offs):
    """{name: (value, sum of absolute terms)} of out, dA and dW in fp64."""
    vw = mxfp4.dequant_rowwise_fp4(*mxfp4.quantize_rowwise_fp4(W))
    vwt = mxfp4.dequant_rowwise_fp4(*mxfp4.quantize_colwise_fp4(W))
    r = {}
    for name, x, w in (("out", _vals(A), vw), ("dA", _vals(G), vwt)):
        r[name] = mxfp4.grouped_product(x, w, offs), mxfp4.grouped_product(x, w, offs, absolute=True)
    r["dW"] = oracle.grouped_mm_wgrad(G, A, offs), oracle.grouped_mm_wgrad(G, A, offs, absolute=True)
    return r


@pytest.mark.parametrize("counts,N,K", [([64, 0, 96], 256, 256), ([128], 384, 256), ([32, 160, 0], 256, 384),
                                        ([320, 288], 256, 384)])
def test_gradients_match_the_formulas(counts, N, K):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    M, E = sum(counts), len(counts)
    offs = inp.offsets_from_counts(counts)
    A = inp.random_bf16((M, K), seed=40, outliers=True)
    W = inp.random_bf16((E, N, K), seed=41, std=0.02)
    G = inp.random_bf16((M, N), seed=42, std=1e-3)
    log(f"fp4 autograd {counts} N={N} K={K}")
    a, w = to_dev_bf16(A).requires_grad_(), to_dev_bf16(W).requires_grad_()
    out = mx.mx_grouped_mm(a, w, to_dev_i32(offs), weight_format="mxfp4")
    out.backward(to_dev_bf16(G))
    for name, got in (("out", out.detach()), ("dA", a.grad), ("dW", w.grad)):
        ref, ab = _forms(A, W, G, offs)[name]
        rep = oracle.r1_check(bf16_host_bits(got), ref, abs_terms=ab)
        assert rep["ok"], (name, rep)
    for e, c in enumerate(counts):
        if c == 0:
            assert not w.grad[e].any()
    # only one gradient wanted: the same bits
    a2 = to_dev_bf16(A).requires_grad_()
    mx.mx_grouped_mm(a2, w.detach(), to_dev_i32(offs), weight_format="mxfp4").backward(to_dev_bf16(G))
    assert torch.equal(a2.grad, a.grad)
    w2 = w.detach().clone().requires_grad_()
    mx.mx_grouped_mm(a.detach(), w2, to_dev_i32(offs), weight_format="mxfp4").backward(to_dev_bf16(G))
    assert torch.equal(w2.grad, w.grad)


def test_input_gradient_against_differences():
    """Weights and steps that every format holds exactly (small powers of two),
    so that the product is linear in A and differences are exact: the gradient
    of sum(G * out) along a direction D is (f(A + D) - f(A - D)) / 2."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(7)
    counts, N, K = [64, 32], 128, 128
    M = sum(counts)
    offs = to_dev_i32(inp.offsets_from_counts(counts))
    A = rng.choice([1.0, 2.0, -1.0, -2.0], size=(M, K)).astype(np.float32)
    D = rng.choice([0.0, 0.5, -0.5], size=(M, K)).astype(np.float32)
    W = rng.choice([0.0, 0.5, 1.0, -1.0], size=(2, N, K)).astype(np.float32)
    G = rng.choice([1.0, -1.0, 0.25], size=(M, N)).astype(np.float32)
    dev = lambda v: to_dev_bf16(inp.f32_to_bf16_bits(v))  # noqa: E731
    # |out| <= 128 * 2.5: quarters up to 320 need 11 bits, so the sums are taken from the fp32 product
    def f(a):
        qa, sa, _, _ = mx.mx_quantize_dual(dev(a))
        qw, sw, _, _ = mx.mx_quantize_weights_fp4(dev(W))
        out = mx.mx_grouped_gemm_mxfp4(qa, sa, qw, sw, offs, out_dtype=torch.float32)
        return float((out.double().cpu() * torch.from_numpy(G).double()).sum())
    a = dev(A).requires_grad_()
    out = mx.mx_grouped_mm(a, dev(W), offs, weight_format="mxfp4")
    out.backward(dev(G))
    slope = (f(A + D) - f(A - D)) / 2
    # each gradient element is rounded to bf16 once (half a step, 2^-9 of it at most 2^-8), the rest is exact
    g = a.grad.double().cpu().numpy()
    assert abs(float((g * D).sum()) - slope) <= 2.0 ** -8 * float(np.abs(g * D).sum())


@pytest.mark.parametrize("topk", [1, 3])
def test_routed_experts(topk):
    """The routed path with 4-bit weights equals the grouped primitive on rows
    gathered by hand, dropped items included."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    T, E, N, K = 70, 4, 256, 384
    rng = np.random.default_rng(50 + topk)
    ids = rng.integers(0, E, size=(T, topk)).astype(np.int32)
    ids[ids == 2] = 0                                    # an expert without tokens
    ids[5, 0] = 9                                        # an id outside [0, E): dropped
    x, W = inp.random_bf16((T, K), seed=51, outliers=True), inp.random_bf16((E, N, K), seed=52, std=0.02)
    G = inp.random_bf16((T * topk, N), seed=53, std=1e-3)
    xd, wd = to_dev_bf16(x).requires_grad_(), to_dev_bf16(W).requires_grad_()
    idx = to_dev_i32(ids if topk > 1 else ids[:, 0])
    out = mx.mx_routed_experts(xd, idx, wd, check=False, weight_format="mxfp4")
    out.backward(to_dev_bf16(G).view(out.shape))
    offs, rows, _, _ = mx.mx_route(to_dev_i32(ids.reshape(-1)), E)
    end = int(offs[-1])
    r = rows[:end].long()
    real = r >= 0
    xg = torch.where(real[:, None], to_dev_bf16(x)[r.clamp(min=0) // topk], 0)
    gg = torch.where(real[:, None], to_dev_bf16(G)[r.clamp(min=0)], 0)
    xg, wg = xg.requires_grad_(), to_dev_bf16(W).requires_grad_()
    og = mx.mx_grouped_mm(xg, wg, offs, weight_format="mxfp4")
    og.backward(gg)
    want = torch.zeros_like(out).view(T * topk, N)
    want[r[real]] = og.detach()[real]
    assert torch.equal(out.detach().view(T * topk, N), want)
    assert torch.equal(wd.grad, wg.grad)
    if topk == 1:
        dx = torch.zeros_like(xd)
        dx[r[real]] = xg.grad[real]
        assert torch.equal(xd.grad, dx)
    else:
        # the items' fp32 gradients summed once: within half a bf16 step of the sum of rounded ones' bounds
        ref = torch.zeros((T, K), dtype=torch.float64, device="cuda:0").index_add_(0, r[real] // topk, xg.grad[real].double())
        ab = torch.zeros((T, K), dtype=torch.float64, device="cuda:0").index_add_(0, r[real] // topk, xg.grad[real].double().abs())
        assert ((xd.grad.double() - ref).abs() <= 2.0 ** -8 * (ab + ref.abs())).all()


def test_weights_and_caches():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    from mxfp8_block_scaled_06_amd.autograd import WeightCache, weight_cache
    counts, N, K = [32, 64], 128, 256
    offs = to_dev_i32(inp.offsets_from_counts(counts))
    A, W = to_dev_bf16(inp.random_bf16((96, K), seed=60)), to_dev_bf16(inp.random_bf16((2, N, K), seed=61, std=0.02))
    before = weight_cache().quantizations
    first = mx.mx_grouped_mm(A, W, offs, weight_format="mxfp4")
    assert weight_cache().quantizations == before        # nothing is kept unless the caller keeps it
    W.data.mul_(2)                                       # not even a change that no version counter sees goes unnoticed
    assert torch.equal(mx.mx_grouped_mm(A, W, offs, weight_format="mxfp4"), 2 * first)
    W.data.mul_(0.5)
    cache = WeightCache()
    for _ in range(2):
        assert torch.equal(mx.mx_grouped_mm(A, W, offs, cache=cache, weight_format="mxfp4"), first)
    assert cache.quantizations == 1
    mx.mx_grouped_mm(A, W, offs, cache=cache)            # the 8-bit copy is an entry of its own
    assert cache.quantizations == 2
    assert torch.equal(mx.mx_grouped_mm(A, W, offs, weights=mx.mx_quantize_weights_fp4(W), weight_format="mxfp4"), first)
    with pytest.raises(ValueError, match="prequantized"):
        mx.mx_grouped_mm(A, W, offs, weights=mx.mx_quantize_weights(W), weight_format="mxfp4")
    with pytest.raises(ValueError, match="weight_format"):
        mx.mx_grouped_mm(A, W, offs, weight_format="fp4")
    y = mx.mx_linear(A, W[0].contiguous(), weight_format="mxfp4")
    assert torch.equal(y, mx.mx_grouped_mm(A, W[:1].contiguous(), to_dev_i32(np.array([96])), weight_format="mxfp4"))
