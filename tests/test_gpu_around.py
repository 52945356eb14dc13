"""The operators around the experts' products in the calls that programs make of
them together: captured training steps, two streams, checkpointing, saved tensors,
strides, and tensors of more than 2^31 elements."""

import pytest

from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

GIB = 1 << 30


def _ops(mx, torch):
    """(entry point, its differentiable inputs, its gradient) of each operator, each over leaves of its own."""
    g = torch.Generator(device="cuda:0").manual_seed(5)
    rand = lambda *shape: torch.randn(shape, device="cuda:0", generator=g)  # noqa: E731
    bias = rand(24) * 0.1
    yield (lambda l: mx.mx_topk_router(l, 3, "softmax", bias, 4, 2)[1], [rand(37, 24)], rand(37, 3))
    yield (lambda l: mx.mx_topk_router(l, 8, "sigmoid", renormalize=False)[1], [rand(65, 256).bfloat16()], rand(65, 8))
    yield (mx.mx_swiglu, [rand(33, 2 * 96).bfloat16()], rand(33, 96).bfloat16())
    yield (mx.mx_topk_combine, [rand(33, 5, 200).bfloat16(), rand(33, 5)], rand(33, 200).bfloat16())
    yield (mx.mx_topk_combine, [rand(9, 1, 1032), rand(9, 1)], rand(9, 1032).bfloat16())


def _step(torch, op, leaves, d):
    out = op(*leaves)
    return [out, *torch.autograd.grad(out, leaves, d)]


def _leaves(tensors):
    return [t.clone().requires_grad_() for t in tensors]


def test_captured_training_steps():
    """Forward and backward captured together and replayed on new values, against eager steps between the replays."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        leaves = _leaves(inputs)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _step(torch, op, leaves, d)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            static = [t.detach() for t in _step(torch, op, leaves, d)]
        for _ in range(3):
            with torch.no_grad():
                for leaf in leaves:
                    leaf.copy_(torch.randn(leaf.shape, device="cuda:0"))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in static]
            want = _step(torch, op, _leaves([t.detach() for t in leaves]), d)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_capture_beside_a_living_eager_graph_is_refused():
    """A leaf whose eager graph lives: refused in the capture, before anything is launched; taken once it is gone."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        leaves = _leaves(inputs)
        eager = op(*leaves)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(RuntimeError, match="graph of the same leaf"):
                op(*leaves)
            with torch.no_grad():
                static = op(*leaves)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, eager.detach())
        op(*leaves)
        del eager, graph
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            static = [t.detach() for t in _step(torch, op, leaves, d)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(static, _step(torch, op, _leaves(inputs), d)))


def test_layer_refuses_a_capture_beside_a_living_eager_graph():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    x = torch.randn((20, 128), device="cuda:0").bfloat16()
    W13 = torch.randn((2, 256, 128), device="cuda:0").bfloat16().requires_grad_()
    W2 = torch.randn((2, 128, 128), device="cuda:0").bfloat16().requires_grad_()
    ids = torch.randint(2, (20, 1), device="cuda:0", dtype=torch.int32)
    w = torch.ones((20, 1), device="cuda:0")
    eager = mx.mx_moe_layer(x, ids, w, W13, W2)
    scrap = torch.zeros(4, device="cuda:0")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scrap.add_(1)
        with pytest.raises(RuntimeError, match="graph of the same leaf"):
            mx.mx_moe_layer(x, ids, w, W13, W2, check=False)
    del eager


def test_two_streams_at_once():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    ops = list(_ops(mx, torch))
    want = [_step(torch, op, _leaves(inputs), d) for op, inputs, d in ops]
    gu = [torch.randn((256, 512), device="cuda:0").bfloat16() for _ in range(2)]
    w = [torch.rand(256, device="cuda:0") for _ in range(2)]
    dh = [torch.randn((256, 256), device="cuda:0").bfloat16() for _ in range(2)]

    def routed(i):
        a = mx.mx_swiglu_quantize_fwd(gu[i], None, w[i])
        b = mx.mx_swiglu_quantize_bwd(dh[i], a[4], a[5], None, None, w[i])
        return [*a, *b, mx.mx_dequantize(a[0], a[1], "gemm"), *mx.mx_swiglu_quantize(gu[i])]

    alone = [routed(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got, pairs = [], []
        for n, (op, inputs, d) in enumerate(ops):
            with torch.cuda.stream(streams[n % 2]):
                got.append(_step(torch, op, _leaves(inputs), d))
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                pairs.append(routed(i))
        torch.cuda.synchronize()
        for a, b in zip(got + pairs, want + alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_checkpointing_and_repeated_backwards():
    torch = require_gpu()
    from torch.utils.checkpoint import checkpoint
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        leaves = _leaves(inputs)
        out = op(*leaves)
        first = torch.autograd.grad(out, leaves, d, retain_graph=True)
        again = torch.autograd.grad(out, leaves, d)
        redone = torch.autograd.grad(checkpoint(op, *leaves, use_reentrant=False), leaves, d)
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, redone))


def test_saved_tensors_that_were_changed_are_refused():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    l = torch.randn((8, 16), device="cuda:0", requires_grad=True)
    _, w = mx.mx_topk_router(l, 2)
    w.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(w.sum(), l)
    y = torch.randn((8, 2, 64), device="cuda:0").bfloat16()
    c = torch.rand((8, 2), device="cuda:0", requires_grad=True)
    out = mx.mx_topk_combine(y, c)
    y.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(out.float().sum(), c)


def test_second_derivatives_of_each_are_refused():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        leaves = _leaves(inputs)
        grads = torch.autograd.grad(op(*leaves), leaves, d, create_graph=True)
        total = sum(g.float().square().sum() for g in grads)
        with pytest.raises(RuntimeError):         # not connected to the leaves
            torch.autograd.grad(total, leaves, retain_graph=True)
        with pytest.raises(RuntimeError, match="no derivative"):
            total.backward()


def test_strided_inputs_and_gradients():
    """Transposed, sliced and expanded tensors reach the kernels as copies."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        want = _step(torch, op, _leaves(inputs), d)
        for make in (lambda t: t.transpose(0, -1).contiguous().transpose(0, -1),
                     lambda t: torch.stack((t, t), dim=-1)[..., 1]):
            leaves = [make(t).detach().requires_grad_() for t in inputs]
            got = _step(torch, op, leaves, make(d))
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_and_pos_that_do_not_agree():
    """An item with several rows takes the sum of the one that pos names; one whose pos leads elsewhere gets 0."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    M, N, n = 64, 256, 6
    gu, dh = torch.randn((M, 2 * N), device="cuda:0").bfloat16(), torch.randn((M, N), device="cuda:0").bfloat16()
    rows = torch.full((M,), -1, dtype=torch.int32)
    rows[[0, 1, 2, 40, 63]] = torch.tensor([3, 0, 3, 1, 5], dtype=torch.int32)
    pos = torch.tensor([1, 40, -1, 2, 7, 1 << 30], dtype=torch.int32)      # 4: a row without an item; 5: no row
    rows, pos, w = rows.cuda(), pos.cuda(), torch.rand(n, device="cuda:0")
    kept, kept_s = mx.mx_swiglu_quantize_fwd(gu, rows, w)[4:]
    ones = torch.ones(M, device="cuda:0")
    each = mx.mx_swiglu_quantize_bwd(dh, *mx.mx_swiglu_quantize_fwd(gu)[4:], combine=ones)[4]
    for _ in range(3):
        dw = mx.mx_swiglu_quantize_bwd(dh, kept, kept_s, rows, pos, w)[4]
        want = torch.stack([each[1], each[40], 0 * each[0], each[2], 0 * each[0], 0 * each[0]])
        assert torch.equal(dw, want)


def _room(torch, gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * GIB:
        pytest.skip(f"needs {gib} GiB of free GPU memory")


def test_router_past_2_31_elements():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    _room(torch, 24)
    for T, E in (((1 << 23) + 77, 257), ((1 << 23) + 77, 256)):
        log(f"router {T} x {E}")
        l = torch.empty((T, E), dtype=torch.bfloat16, device="cuda:0").normal_()
        ids, w = mx.mx_topk_router_fwd(l, 2, renormalize=False)
        dw = torch.empty_like(w).normal_()
        dl = mx.mx_topk_router_bwd(l, ids, w, dw, renormalize=False)
        tail = l[-99:].clone()
        small = mx.mx_topk_router_fwd(tail, 2, renormalize=False)
        assert torch.equal(ids[-99:], small[0]) and torch.equal(w[-99:], small[1])
        assert torch.equal(dl[-99:], mx.mx_topk_router_bwd(tail, *small, dw[-99:].clone(), renormalize=False))
        del l, dl, ids, w, dw


def test_activation_past_2_31_elements():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    _room(torch, 48)
    M, N = 66 * 1024, 16384                       # gate and up 2^31 + 2^26
    log("swiglu 67584 x 16384")
    gu = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda:0").normal_()
    dh = torch.empty((M, N), dtype=torch.bfloat16, device="cuda:0").normal_()
    tail, dtail = gu[-128:].clone(), dh[-128:].clone()
    h, kept, kept_s = mx.mx_swiglu_fwd(gu)
    want = mx.mx_swiglu_fwd(tail)
    assert all(torch.equal(a[-128:], b) for a, b in zip((h, kept, kept_s), want))
    assert torch.equal(mx.mx_swiglu_bwd(dh, kept, kept_s)[-128:], mx.mx_swiglu_bwd(dtail, *want[1:]))
    del h, kept, kept_s
    log("routed activation 67584 x 16384")
    w = torch.rand(M, device="cuda:0")
    q, s, qt, st, kept, kept_s = mx.mx_swiglu_quantize_fwd(gu, None, w)
    want = mx.mx_swiglu_quantize_fwd(tail, None, w[-128:].clone())
    for a, b in zip((q[-128:], s[:, -128:], qt[:, -128:], st[-1:], kept[-128:], kept_s[:, -128:]), want):
        assert torch.equal(a, b)
    assert torch.equal(mx.mx_dequantize(kept, kept_s, "gemm")[-128:], mx.mx_dequantize(want[4], want[5], "gemm"))
    del q, s, qt, st
    q, s, qt, st, dw = mx.mx_swiglu_quantize_bwd(dh, kept, kept_s, None, None, w)
    want = mx.mx_swiglu_quantize_bwd(dtail, want[4], want[5], None, None, w[-128:].clone())
    for a, b in zip((q[-128:], s[:, -128:], qt[:, -128:], st[-1:], dw[-128:]), want):
        assert torch.equal(a, b)


def test_weighted_sum_past_2_31_elements():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    _room(torch, 48)
    T, k, N = 33 * 1024, 8, 8192                  # y 2^31 + 2^26
    log("weighted sum 33792 x 8 x 8192")
    y = torch.empty((T, k, N), dtype=torch.bfloat16, device="cuda:0").normal_()
    w = torch.rand((T, k), device="cuda:0")
    dout = torch.empty((T, N), dtype=torch.bfloat16, device="cuda:0").normal_()
    tail = (y[-3:].clone(), w[-3:].clone())
    assert torch.equal(mx.mx_topk_combine_fwd(y, w)[-3:], mx.mx_topk_combine_fwd(*tail))
    dy, dw = mx.mx_topk_combine_bwd(dout, y, w)
    want = mx.mx_topk_combine_bwd(dout[-3:].clone(), *tail)
    assert torch.equal(dy[-3:], want[0]) and torch.equal(dw[-3:], want[1])


def _shifted(torch, t):
    """t at an address one element past an aligned one."""
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    return room[1:].view(t.shape).copy_(t)


def test_operands_and_gradients_at_any_address():
    """Contiguous, but not where the kernels' wide loads could read them: a copy is made, as for strides."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        want = _step(torch, op, _leaves(inputs), d)
        leaves = [_shifted(torch, t).requires_grad_() for t in inputs]
        for got in (_step(torch, op, leaves, d), _step(torch, op, _leaves(inputs), _shifted(torch, d)),
                    _step(torch, op, leaves, _shifted(torch, d))):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        with torch.no_grad():
            assert torch.equal(op(*[_shifted(torch, t) for t in inputs]), want[0])
    # as autograd hands them over: the gradient of a part of a longer tensor
    gu = torch.randn((8, 192), device="cuda:0").bfloat16().requires_grad_()
    tail = torch.randn(1, device="cuda:0").bfloat16()
    d = torch.randn(8 * 96 + 1, device="cuda:0").bfloat16()
    got, = torch.autograd.grad(torch.cat((tail, mx.mx_swiglu(gu).reshape(-1))), gu, d)
    want, = torch.autograd.grad(mx.mx_swiglu(gu), gu, d[1:].clone().view(8, 96))
    assert torch.equal(got, want)


def test_layer_at_any_address():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    g = torch.Generator(device="cuda:0").manual_seed(6)
    rand = lambda *shape: torch.randn(shape, device="cuda:0", generator=g).bfloat16()  # noqa: E731
    ids = torch.randint(3, (40, 2), device="cuda:0", dtype=torch.int32, generator=g)
    w = torch.rand((40, 2), device="cuda:0", generator=g)
    inputs, d = [rand(40, 128), w, rand(3, 256, 128) * 0.05, rand(3, 128, 128) * 0.05], rand(40, 128)
    layer = lambda x, w, a, b: mx.mx_moe_layer(x, ids, w, a, b)  # noqa: E731
    want = _step(torch, layer, _leaves(inputs), d)
    for leaves, dout in (([_shifted(torch, t).requires_grad_() for t in inputs], d),
                         (_leaves(inputs), _shifted(torch, d))):
        got = _step(torch, layer, leaves, dout)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.no_grad():
        assert torch.equal(layer(*[_shifted(torch, t) for t in inputs]), want[0])


def test_products_at_any_address():
    """The differentiable products take operands and gradients that are contiguous anywhere."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    g = torch.Generator(device="cuda:0").manual_seed(7)
    rand = lambda *shape: torch.randn(shape, device="cuda:0", generator=g).bfloat16()  # noqa: E731
    offs = torch.tensor([32, 96], dtype=torch.int32, device="cuda:0")
    ids = torch.randint(2, (96, 2), device="cuda:0", dtype=torch.int32, generator=g)
    for fmt in ("mxfp8", "mxfp4"):
        for op, W, d in ((lambda x, W: mx.mx_grouped_mm(x, W, offs, weight_format=fmt), rand(2, 256, 128), rand(96, 256)),
                         (lambda x, W: mx.mx_linear(x, W, weight_format=fmt), rand(256, 128), rand(96, 256)),
                         (lambda x, W: mx.mx_routed_experts(x, ids[:, 0].contiguous(), W, weight_format=fmt),
                          rand(2, 256, 128), rand(96, 256)),
                         (lambda x, W: mx.mx_routed_experts(x, ids, W, weight_format=fmt), rand(2, 256, 128),
                          rand(96, 2, 256))):
            x = rand(96, 128)
            want = _step(torch, op, _leaves([x, W]), d)
            for leaves, dout in (([_shifted(torch, t).requires_grad_() for t in (x, W)], d),
                                 (_leaves([x, W]), _shifted(torch, d)),
                                 ([x.clone().requires_grad_(), W], _shifted(torch, d))):
                needed = [t for t in leaves if t.requires_grad]
                out = op(*leaves)
                got = [out, *torch.autograd.grad(out, needed, dout)]
                assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_forward_mode_is_refused():
    """No operator has a forward-mode derivative: operands with a tangent are refused, not taken for constants,
    with gradients enabled and without."""
    torch = require_gpu()
    import torch.autograd.forward_ad as fwd
    import mxfp8_block_scaled_06_amd as mx
    x = torch.randn((20, 128), device="cuda:0").bfloat16()
    W13 = torch.randn((2, 256, 128), device="cuda:0").bfloat16()
    W2 = torch.randn((2, 128, 128), device="cuda:0").bfloat16()
    ids = torch.randint(2, (20, 1), device="cuda:0", dtype=torch.int32)
    w = torch.ones((20, 1), device="cuda:0")
    l, bias = torch.randn((7, 24), device="cuda:0"), torch.randn(24, device="cuda:0")
    ops = [(op, inputs) for op, inputs, _ in _ops(mx, torch)]
    ops.append((lambda x, w, a, b: mx.mx_moe_layer(x, ids, w, a, b), [x, w, W13, W2]))
    ops.append((lambda b: mx.mx_topk_router(l, 3, "sigmoid", b), [bias]))
    for op, inputs in ops:
        for i in range(len(inputs)):
            for strided in (False, True):
                with fwd.dual_level():
                    args = [t.mT.contiguous().mT if strided and t.dim() > 1 else t for t in inputs]
                    args[i] = fwd.make_dual(args[i], torch.ones_like(args[i]))
                    for grad in (True, False):
                        with torch.set_grad_enabled(grad), pytest.raises((RuntimeError, ValueError)):
                            op(*args)
        op(*inputs)                       # without one they are taken as ever


def test_capture_of_a_copied_leaf_beside_its_eager_graph_is_refused():
    """Strided and unaligned leaves, which reach the kernels as copies, are looked at before the copy."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for op, inputs, d in _ops(mx, torch):
        for make in (lambda t: t.transpose(0, -1).contiguous().transpose(0, -1), lambda t: _shifted(torch, t)):
            leaves = [make(t).detach().requires_grad_() for t in inputs]
            eager = op(*leaves)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                with pytest.raises(RuntimeError, match="graph of the same leaf"):
                    op(*leaves)
                with torch.no_grad():
                    static = op(*leaves)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(static, eager.detach())
            del eager


def test_captured_training_step_of_router_and_layer():
    """The router and the layer captured together, forward and backward, with weights given; replayed on new tokens
    and logits against eager steps between the replays."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    g = torch.Generator(device="cuda:0").manual_seed(8)
    rand = lambda *shape: torch.randn(shape, device="cuda:0", generator=g)  # noqa: E731
    W13, W2 = ((rand(4, *shape) * 0.05).bfloat16() for shape in ((512, 256), (256, 256)))
    d = rand(96, 256).bfloat16()
    weights = mx.mx_quantize_weights(W13), mx.mx_quantize_weights(W2)

    def layer(x, logits, W13, W2):
        ids, w = mx.mx_topk_router(logits, 2)
        return mx.mx_moe_layer(x, ids, w, W13, W2, check=False, weights=weights)

    leaves = _leaves([rand(96, 256).bfloat16(), rand(96, 4), W13, W2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(torch, layer, leaves, d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = [t.detach() for t in _step(torch, layer, leaves, d)]
    for _ in range(3):
        with torch.no_grad():
            for leaf in leaves[:2]:
                leaf.copy_(rand(*leaf.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        want = _step(torch, layer, _leaves([t.detach() for t in leaves]), d)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
