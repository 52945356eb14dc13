"""Refusals of the router, the gated activation, the weighted sum and the MXFP8
dequantizer: status and text of the C ABI, errors of the binding.  No GPU, no
launch; the pointers are never followed."""

import pytest
import torch

import mxfp8_block_scaled_06_amd as mx
from test_abi import FAKE as P, _err, _lib

OK, NULL, SHAPE, ALIGN, WS, LAYOUT = 0, 1, 2, 3, 4, 6


def _router(lib, logits=P, kind=1, bias=None, T=4, E=8, k=2, score=0, groups=1, kg=1, gs=0, renorm=1, scale=1.0, ids=P,
            w=P):
    return lib.mx_topk_router_fwd(logits, kind, bias, T, E, k, score, groups, kg, gs, renorm, scale, ids, w, None)


@pytest.mark.parametrize("want,args", [
    (SHAPE, {"kind": 2}), (SHAPE, {"score": 2}), (SHAPE, {"T": -1}), (SHAPE, {"T": 1 << 31}), (SHAPE, {"E": 0}),
    (SHAPE, {"E": 1025}), (SHAPE, {"k": 0}), (SHAPE, {"k": 9}), (SHAPE, {"E": 64, "k": 33}), (SHAPE, {"scale": 0.0}),
    (SHAPE, {"scale": float("nan")}), (SHAPE, {"scale": float("inf")}), (SHAPE, {"scale": -1.0}),
    (SHAPE, {"groups": 3}), (SHAPE, {"groups": 0}), (SHAPE, {"E": 130, "groups": 65}), (SHAPE, {"groups": 4, "kg": 5}),
    (SHAPE, {"groups": 4, "kg": 0}), (SHAPE, {"groups": 4, "kg": 1, "k": 3}), (SHAPE, {"gs": 2}),
    (NULL, {"logits": None}), (NULL, {"ids": None}), (NULL, {"w": None}), (ALIGN, {"logits": P + 4}),
    (ALIGN, {"bias": P + 2}), (ALIGN, {"ids": P + 1}), (OK, {"T": 0, "logits": None, "ids": None, "w": None}),
])
def test_router_refusals(want, args):
    lib = _lib()
    assert _router(lib, **args) == want
    assert want == OK or "mx_topk_router_fwd" in _err(lib)


def test_router_backward_refusals():
    lib = _lib()

    def f(logits=P, kind=1, ids=P, w=P, dw=P, T=4, E=8, k=2, score=0, renorm=1, scale=1.0, dl=P):
        return lib.mx_topk_router_bwd(logits, kind, ids, w, dw, T, E, k, score, renorm, scale, dl, None)

    for want, args in ((SHAPE, {"k": 9}), (SHAPE, {"kind": -1}), (SHAPE, {"score": 5}), (SHAPE, {"scale": 0.0}),
                       (NULL, {"logits": None}), (NULL, {"ids": None}), (NULL, {"dw": None}), (NULL, {"dl": None}),
                       (ALIGN, {"dl": P + 8}), (ALIGN, {"dw": P + 2}), (OK, {"T": 0})):
        assert f(**args) == want, args


def test_activation_refusals():
    lib = _lib()
    f = lib.mx_swiglu_fwd
    assert f(P, 4, 48, P, P, P, None) == SHAPE and "multiple of 32" in _err(lib)
    assert f(P, -1, 64, P, P, P, None) == SHAPE
    assert f(P, 1 << 27, 1024, P, P, P, None) == SHAPE and "2^32" in _err(lib)
    assert f(P, 4, 64, P, P, None, None) == NULL and f(P, 4, 64, P, None, P, None) == NULL
    assert f(None, 4, 64, P, None, None, None) == NULL and f(P, 4, 64, None, None, None, None) == NULL
    assert f(P + 8, 4, 64, P, P, P, None) == ALIGN and f(P, 4, 64, P + 8, P, P, None) == ALIGN
    assert f(None, 0, 64, None, None, None, None) == OK and f(None, 4, 0, None, None, None, None) == OK
    b = lib.mx_swiglu_bwd
    assert b(P, P, P, 4, 40, P, None) == SHAPE and b(P, None, P, 4, 64, P, None) == NULL
    assert b(P, P + 8, P, 4, 64, P, None) == ALIGN and b(None, None, None, 0, 64, None, None) == OK
    q = lib.mx_swiglu_quantize
    assert q(P, None, 0, 4, 64, P, P, None) == SHAPE and "128" in _err(lib)
    assert q(P, P, -1, 4, 128, P, P, None) == SHAPE and q(P, P, 1 << 31, 4, 128, P, P, None) == SHAPE
    assert q(P, P, 4, 1 << 23, 128, P, P, None) == SHAPE and "rows" in _err(lib)
    assert q(P, P, 4, 4, 128, None, P, None) == NULL and q(P, P, 4, 4, 128, P, P + 2, None) == ALIGN


def test_activation_of_routed_rows_refusals():
    lib = _lib()

    def fwd(gu=P, rows=P, w=P, n=64, M=64, N=128, ldq=128, q=P, s=P, qt=P, st=P, kq=P, ks=P):
        return lib.mx_swiglu_quantize_fwd(gu, rows, w, n, M, N, ldq, q, s, qt, st, kq, ks, None)

    for want, args in ((SHAPE, {"M": 48}), (SHAPE, {"N": 64}), (SHAPE, {"ldq": 64}), (SHAPE, {"M": 160, "ldq": 128}),
                       (SHAPE, {"rows": None, "n": 63}), (SHAPE, {"n": 1 << 31}), (NULL, {"gu": None}), (NULL, {"kq": None}),
                       (NULL, {"st": None}), (ALIGN, {"kq": P + 8}), (ALIGN, {"st": P + 2}), (ALIGN, {"w": P + 2}),
                       (OK, {"N": 0}), (OK, {"M": 0, "ldq": 0})):
        assert fwd(**args) == want, args

    need = lib.mx_swiglu_quantize_workspace_bytes(64, 128)
    assert need >= 64 * 4
    assert lib.mx_swiglu_quantize_workspace_bytes(64, 64) == 0 and lib.mx_swiglu_quantize_workspace_bytes(-1, 128) == 0

    def bwd(dh=P, kq=P, ks=P, rows=P, pos=P, w=P, n=64, M=64, N=128, ldq=128, q=P, s=P, qt=P, st=P, dc=P, ws=P, b=need):
        return lib.mx_swiglu_quantize_bwd(dh, kq, ks, rows, pos, w, n, M, N, ldq, q, s, qt, st, dc, ws, b, None)

    for want, args in ((SHAPE, {"M": 48}), (SHAPE, {"ldq": 192}), (SHAPE, {"rows": None, "n": 65}), (NULL, {"pos": None}),
                       (NULL, {"dh": None}), (NULL, {"ks": None}), (NULL, {"qt": None}), (WS, {"ws": None}),
                       (WS, {"b": need - 1}), (ALIGN, {"ws": P + 128}), (ALIGN, {"dc": P + 2}), (ALIGN, {"q": P + 4})):
        assert bwd(**args) == want, args


def test_weighted_sum_refusals():
    lib = _lib()
    f, b = lib.mx_topk_combine_fwd, lib.mx_topk_combine_bwd
    assert f(P, 3, P, None, 4, 2, 64, P, None) == SHAPE and f(P, 0, P, None, 4, 0, 64, P, None) == SHAPE
    assert f(P, 0, P, None, 4, 1025, 64, P, None) == SHAPE and f(P, 0, P, None, 4, 2, 60, P, None) == SHAPE
    assert f(P, 0, P, None, -4, 2, 64, P, None) == SHAPE and f(P, 0, P, None, 1 << 31, 2, 64, P, None) == SHAPE
    assert f(None, 0, P, None, 4, 2, 64, P, None) == NULL and f(P, 0, P, None, 4, 2, 64, None, None) == NULL
    assert f(P + 8, 0, P, None, 4, 2, 64, P, None) == ALIGN and f(P, 0, P, P + 2, 4, 2, 64, P, None) == ALIGN
    assert f(None, 0, None, None, 0, 2, 64, None, None) == OK and f(None, 0, None, None, 4, 2, 0, None, None) == OK
    assert b(P, 0, P, None, P, 4, 2, 60, P, P, None) == SHAPE and b(None, 0, P, None, P, 4, 2, 64, P, P, None) == NULL
    assert b(P, 0, P, None, None, 4, 2, 64, P, P, None) == NULL and b(P, 0, P, None, P, 4, 2, 64, P + 8, P, None) == ALIGN
    assert b(P, 0, P, None, P, 4, 2, 64, None, None, None) == OK


def test_dequantizer_refusals():
    lib = _lib()
    f = lib.mx_dequantize
    assert f(P, P, 1, 4, 48, mx.SCALES_ROWMAJOR, P, None) == SHAPE and f(P, P, 1, 4, 64, mx.SCALES_GEMM, P, None) == SHAPE
    assert f(P, P, 1, 4, 64, 7, P, None) == LAYOUT and f(None, P, 1, 4, 64, 0, P, None) == NULL
    assert f(P + 8, P, 1, 4, 64, 0, P, None) == ALIGN and f(None, None, 1, 0, 64, 0, None, None) == OK


def test_binding_refuses():
    cpu, bf = torch.zeros(4, 64), torch.bfloat16
    for call in (lambda: mx.mx_topk_router(cpu, 2), lambda: mx.mx_swiglu(cpu.to(bf)),
                 lambda: mx.mx_topk_combine(torch.zeros(2, 2, 64, dtype=bf), torch.zeros(2, 2)),
                 lambda: mx.mx_swiglu_quantize(torch.zeros(4, 256, dtype=bf)),
                 lambda: mx.mx_dequantize(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        mx.mx_topk_router(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(TypeError):
        mx.mx_swiglu(cpu)
    x, W13, W2 = torch.zeros(4, 128, dtype=bf), torch.zeros(2, 256, 128, dtype=bf), torch.zeros(2, 128, 128, dtype=bf)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in ((x, ids.long(), w, W13, W2), (x, ids, w.to(bf), W13, W2), (x.float(), ids, w, W13, W2)):
        with pytest.raises(TypeError):
            mx.mx_moe_layer(*bad)
    for bad in ((x, ids[:3], w[:3], W13, W2), (x, ids, w[:, :1], W13, W2), (x, ids, w, W13[:, :128], W2),
                (x, ids, w, W13, W2[:1]), (x[:, :64], ids, w, W13, W2), (x, ids[:, :0], w[:, :0], W13, W2)):
        with pytest.raises(ValueError):
            mx.mx_moe_layer(*bad)
    bias = torch.zeros(8, requires_grad=True)
    with pytest.raises(ValueError, match="no gradient"):
        mx.mx_topk_router(torch.zeros(4, 8), 2, bias=bias)


def test_layer_refuses_empty_weights():
    bf = torch.bfloat16
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for E, K, N in ((0, 128, 128), (2, 0, 128), (2, 128, 0), (2, 128, 64)):
        with pytest.raises(ValueError, match="positive multiples"):
            mx.mx_moe_layer(torch.zeros(4, K, dtype=bf), ids, w, torch.zeros(E, 2 * N, K, dtype=bf), torch.zeros(E, K, N, dtype=bf))
