"""The differentiable MoE layer on the GPU: bit for bit the chain of the entry
points it is made of, near the unquantized formula, and together with the router,
the few-token layer and graphs as a program uses them."""

import numpy as np
import pytest

from mxfp8_block_scaled_06_amd.autograd import WeightCache
from gpu_util import require_gpu, log

pytestmark = pytest.mark.gpu


def _case(T, k, E, K, N, seed=0, drop=0):
    import torch
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda:0") * std).bfloat16()  # noqa: E731
    ids = torch.stack([torch.randperm(E, generator=gen, device="cuda:0")[:k] for _ in range(T)]).int() if T else \
        torch.zeros((0, k), dtype=torch.int32, device="cuda:0")
    for i in range(drop):
        ids[(7 * i) % T, i % k] = (-1, E, 1 << 30)[i % 3]
    w = torch.rand((T, k), generator=gen, device="cuda:0")
    return r(T, K), ids, w / w.sum(1, keepdim=True) if T else w, r(E, 2 * N, K, std=0.05), r(E, K, N, std=0.05), r(T, K, std=1e-2)


def _grads(mx, x, ids, w, W13, W2, dout, **kw):
    import torch
    leaves = [t.clone().requires_grad_() for t in (x, w, W13, W2)]
    out = mx.mx_moe_layer(leaves[0], ids, *leaves[1:], **kw)
    return (out.detach(), *torch.autograd.grad(out, leaves, dout))


def _chain(mx, x, ids, w, W13, W2, dout, fmt):
    """The layer from entry points on explicitly grouped bf16 tensors."""
    import torch
    T, k = ids.shape
    K = x.shape[1]
    quantize = mx.mx_quantize_weights_fp4 if fmt == "mxfp4" else mx.mx_quantize_weights
    gemm = (lambda a, b, c, d, offs: mx.mx_grouped_gemm_mxfp4(a, b, c, d, offs)) if fmt == "mxfp4" else \
        (lambda a, b, c, d, offs: mx.mx_grouped_gemm_mx(a, b, c, d, offs, 0))
    gemm32 = (lambda a, b, c, d, offs: mx.mx_grouped_gemm_mxfp4(a, b, c, d, offs, out_dtype=torch.float32)) if fmt == "mxfp4" \
        else (lambda a, b, c, d, offs: mx.mx_grouped_gemm_mx_f32(a, b, c, d, offs, 0))
    q13, s13, q13t, s13t = quantize(W13)
    q2, s2, q2t, s2t = quantize(W2)
    offs, rows, pos, _ = mx.mx_route(ids.reshape(-1).contiguous(), W13.shape[0])
    live = (rows >= 0).unsqueeze(1)
    token = torch.div(rows.clamp(min=0), k, rounding_mode="floor").long()
    at, routed = pos.clamp(min=0).long(), (pos >= 0).view(T, k)

    def items(v):
        return torch.where(routed.reshape(-1, 1), v[at], 0)

    qx, sx, qxt, sxt = mx.mx_quantize_dual(torch.where(live, x[token], 0))
    gu = gemm(qx, sx, q13, s13, offs)
    qh, sh, qht, sht, kept, kept_s = mx.mx_swiglu_quantize_fwd(gu, rows, w)
    y = items(gemm(qh, sh, q2, s2, offs)).view(T, k, K)
    out = mx.mx_topk_combine_fwd(y, w)
    qg, sg, qgt, sgt = mx.mx_quantize_dual(torch.where(live, dout[token], 0))
    dW2 = mx.mx_grouped_gemm_mx(qgt, sgt, qht, sht, offs, 1)
    qd, sd, qdt, sdt, dw = mx.mx_swiglu_quantize_bwd(gemm(qg, sg, q2t, s2t, offs), kept, kept_s, rows, pos, w)
    dW13 = mx.mx_grouped_gemm_mx(qdt, sdt, qxt, sxt, offs, 1)
    dx = mx.mx_topk_sum_rows(items(gemm32(qd, sd, q13t, s13t, offs)).contiguous(), k)
    return out, dx, dw, dW13, dW2


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,k,E,K,N,drop", [(1, 1, 1, 128, 128, 0), (100, 2, 4, 256, 128, 0), (333, 1, 3, 128, 384, 0),
                                            (65, 8, 12, 384, 256, 0), (50, 3, 5, 128, 128, 9), (20, 1, 4, 256, 128, 5)])
def test_layer_is_the_chain_of_its_entry_points(T, k, E, K, N, drop, fmt):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"moe_layer T={T} k={k} E={E} K={K} N={N} drop={drop} {fmt}")
    args = _case(T, k, E, K, N, seed=T + K, drop=drop)
    got = _grads(mx, *args, check=drop == 0, weight_format=fmt)
    want = _chain(mx, *args, fmt)
    for a, b, name in zip(got, want, ("out", "dx", "dcombine", "dW13", "dW2")):
        assert torch.equal(a, b), name
    x, ids, w, W13, W2, _ = args
    with torch.no_grad():                                   # nothing kept: other quantizers, the same rows
        assert torch.equal(mx.mx_moe_layer(x, ids, w, W13, W2, check=drop == 0, weight_format=fmt), got[0])
    if drop:
        with pytest.raises(ValueError, match="expert id"):
            mx.mx_moe_layer(x, ids, w, W13, W2)
    if k == 1:
        flat = _grads(mx, x, ids[:, 0].contiguous(), w[:, 0].contiguous(), W13, W2, args[5], check=drop == 0, weight_format=fmt)
        assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(flat, got))


def test_layer_near_the_formula():
    """Against the unquantized formula in fp64.  Every MXFP8 rounding is off by at
    most 2^-4 of a value, 1/sqrt(3) of it in the mean: 3.6%.  Six of them meet in the
    gradients of x and of the gate and up weights (dout, W2, gate, up, their gradient,
    x or W13), four in the output: even if all added up, below 25%."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, ids, w, W13, W2, dout = _case(200, 3, 5, 512, 384, seed=5)
    got = _grads(mx, x, ids, w, W13, W2, dout)
    leaves = [t.double().cpu().requires_grad_() for t in (x, w, W13, W2)]
    i = ids.long().cpu()
    rows = []
    for t in range(200):
        for j in range(3):
            g, u = (leaves[2][i[t, j]] @ leaves[0][t]).chunk(2)
            rows.append(leaves[1][t, j] * (leaves[3][i[t, j]] @ (torch.nn.functional.silu(g) * u)))
    out = torch.stack(rows).view(200, 3, -1).sum(1)
    want = (out.detach(), *torch.autograd.grad(out, leaves, dout.double().cpu()))
    for a, b, name in zip(got, want, ("out", "dx", "dcombine", "dW13", "dW2")):
        assert (a.double().cpu() - b).norm() <= 0.25 * b.norm(), name


def test_only_what_is_needed():
    """Each gradient alone is the one of all together."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, ids, w, W13, W2, dout = _case(40, 2, 3, 128, 256, seed=6)
    all_ = _grads(mx, x, ids, w, W13, W2, dout)[1:]
    for i in range(4):
        leaves = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, w, W13, W2))]
        got, = torch.autograd.grad(mx.mx_moe_layer(leaves[0], ids, *leaves[1:]), leaves[i], dout)
        assert torch.equal(got, all_[i])


def test_weights_and_cache():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, ids, w, W13, W2, _ = _case(40, 2, 3, 128, 256, seed=7)
    cache = WeightCache()
    a = mx.mx_moe_layer(x, ids, w, W13, W2, cache=cache)
    b = mx.mx_moe_layer(x, ids, w, W13, W2, cache=cache)
    assert cache.quantizations == 2 and torch.equal(a, b)
    W13.mul_(2)
    c = mx.mx_moe_layer(x, ids, w, W13, W2, cache=cache)
    assert cache.quantizations == 3 and not torch.equal(a, c)
    d = mx.mx_moe_layer(x, ids, w, W13, W2, weights=(mx.mx_quantize_weights(W13), mx.mx_quantize_weights(W2)))
    assert torch.equal(c, d)
    for bad in ((mx.mx_quantize_weights(W13),), (mx.mx_quantize_weights(W2), mx.mx_quantize_weights(W13))):
        with pytest.raises(ValueError):
            mx.mx_moe_layer(x, ids, w, W13, W2, weights=bad)


def test_no_tokens():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    got = _grads(mx, *_case(0, 2, 3, 128, 256))
    assert [tuple(t.shape) for t in got] == [(0, 128), (0, 128), (0, 2), (3, 512, 128), (3, 128, 256)]
    assert not got[3].any() and not got[4].any()
    x, ids, w, W13, W2, _ = _case(0, 2, 3, 128, 256)
    assert tuple(mx.mx_moe_layer(x, ids, w, W13, W2).shape) == (0, 128)


def test_training_then_decoding():
    """The layer and the few-token layer compute one function.  The layer rounds the
    gate and up values to bf16 (2^-9 of a value), which moves a code of h by a step
    (2^-3) in up to 2^-9 * 2 / 2^-4 = 6% of the cases, and each expert's row (2^-9):
    sqrt(0.06) * 2^-3 / sqrt(3) + 2^-9 < 2^-5 in the norm.  The router's ids and weights feed both."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, _, _, W13, W2, _ = _case(60, 2, 8, 256, 384, seed=8)
    logits = torch.randn((60, 8), device="cuda:0").bfloat16()
    for fmt, quantize in (("mxfp8", mx.mx_quantize_weights), ("mxfp4", mx.mx_quantize_weights_fp4)):
        with torch.no_grad():
            ids, w = mx.mx_topk_router(logits, 2, score="sigmoid")
            a = mx.mx_moe_layer(x, ids, w, W13, W2, weight_format=fmt).double()
            b = mx.mx_moe_few_tokens(x, ids, w, quantize(W13)[:2], quantize(W2)[:2], weight_format=fmt).double()
        assert (a - b).norm() <= 2.0 ** -5 * b.norm()


def test_router_and_layer_train_together():
    """A training step as a program writes it: the router's projection, the layer, a
    dense gated layer beside it, one backward pass.  Its gradients are those of the
    steps taken one by one."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, _, _, W13, W2, dout = _case(96, 2, 8, 256, 128, seed=9)
    gate = (torch.randn((8, 256), device="cuda:0") * 0.05).requires_grad_()
    D13 = (torch.randn((256, 256), device="cuda:0") * 0.05).bfloat16().requires_grad_()
    D2 = (torch.randn((256, 128), device="cuda:0") * 0.05).bfloat16().requires_grad_()
    bias = torch.randn(8, device="cuda:0") * 0.01
    x, W13, W2 = (t.requires_grad_() for t in (x, W13, W2))
    logits = x.float() @ gate.t()
    ids, w = mx.mx_topk_router(logits, 2, "sigmoid", bias, groups=2, topk_groups=1, group_score="top2", scale=2.5)
    routed = mx.mx_moe_layer(x, ids, w, W13, W2)
    hidden = mx.mx_linear(x, D13)
    dense = mx.mx_linear(mx.mx_swiglu(hidden), D2)
    got = torch.autograd.grad(routed + dense, (x, gate, W13, W2, D13, D2), dout)
    # one by one
    dx1, dw, dW13, dW2 = _grads(mx, x.detach(), ids, w.detach(), W13.detach(), W2.detach(), dout)[1:]
    dl = mx.mx_topk_router_bwd(logits.detach(), ids, w.detach(), dw, "sigmoid", True, 2.5)
    assert torch.equal(got[2], dW13) and torch.equal(got[3], dW2)
    assert torch.allclose(got[1], dl.t() @ x.detach().float(), rtol=1e-4, atol=1e-6 * float(got[1].abs().max()))
    h, kept, kept_s = mx.mx_swiglu_fwd(hidden.detach())
    hh = h.requires_grad_()
    dh, dD2 = torch.autograd.grad(mx.mx_linear(hh, D2), (hh, D2), dout)
    x2 = x.detach().requires_grad_()
    dx2, dD13 = torch.autograd.grad(mx.mx_linear(x2, D13), (x2, D13), mx.mx_swiglu_bwd(dh, kept, kept_s))
    assert torch.equal(got[4], dD13) and torch.equal(got[5], dD2)
    # bf16 sums of three bf16 gradients: three roundings at 2^-9 of the magnitudes, and the product's
    parts = (dx1, dx2, (dl @ gate.detach()).bfloat16())
    assert ((got[0].double() - sum(p.double() for p in parts)).abs() <= 2.0 ** -7 * sum(p.double().abs() for p in parts)).all()


def test_decoding_step_in_a_graph():
    """Router and few-token layer captured together, replayed with new tokens."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x, _, _, W13, W2, _ = _case(1, 2, 8, 256, 384, seed=10)
    w13, w2 = mx.mx_quantize_weights_fp4(W13)[:2], mx.mx_quantize_weights_fp4(W2)[:2]
    for T in (1, 9):
        x, logits = torch.randn((T, 256), device="cuda:0").bfloat16(), torch.randn((T, 8), device="cuda:0")
        ids, w = mx.mx_topk_router_fwd(logits, 2)
        out, ws = torch.empty_like(x), torch.empty(mx.mx_moe_few_tokens_workspace_bytes(T, 2, 384), dtype=torch.uint8, device="cuda:0")

        def step():
            mx.mx_topk_router_fwd(logits, 2, expert_idx=ids, combine=w)
            mx.mx_moe_few_tokens(x, ids, w, w13, w2, check=False, out=out, ws=ws)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            x.copy_(torch.randn(x.shape, device="cuda:0"))
            logits.copy_(torch.randn(logits.shape, device="cuda:0"))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            step()
            torch.cuda.synchronize()
            assert torch.equal(got, out)


def test_layer_on_two_streams():
    """Two layers at once, each on a stream of its own, forward and backward."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    cases = [_case(300, 2, 4, 256, 256, seed=s) for s in (11, 12)]
    want = [_grads(mx, *c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(_grads(mx, *c, check=False))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_second_derivatives_are_refused():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    gu = torch.randn((32, 256), device="cuda:0").bfloat16().requires_grad_()
    g, = torch.autograd.grad(mx.mx_swiglu(gu).float().square().sum(), gu, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), gu)
