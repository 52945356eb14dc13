"""The MXFP4 oracle against hand-worked blocks, the refusals of the MXFP4
entry points (host-side checks, no kernel is launched) and of their binding."""

import numpy as np
import pytest

import mxfp8_block_scaled_06_amd as mx
from mxfp8_block_scaled_06_amd import inputs as inp
from oracle import mxfp4
from test_abi import FAKE, _err, _lib


def _bits(values):
    return inp.f32_to_bf16_bits(np.asarray(values, dtype=np.float32))


def test_element_codes_by_hand():
    # every magnitude, every midpoint (ties to the even code) and saturation
    y = [0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7.9, .26, .74, 2.51, 3.49, 4.99, 5.01]
    want = [0, 0, 1, 2, 2, 2, 3, 4, 4, 4, 5, 6, 6, 6, 7, 7, 1, 1, 5, 5, 6, 7]
    assert mxfp4.e2m1_encode(np.array(y)).tolist() == want
    assert mxfp4.e2m1_encode(-np.array(y)).tolist() == [w + 8 for w in want]
    assert mxfp4.e2m1_decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]


def test_blocks_by_hand():
    x = np.zeros((1, 4 * 32), dtype=np.float32)
    x[0, 32:36] = [7.0, -1.0, 0.5, -0.125]        # amax 7: exponent 2, byte 127: 7 saturates to 6, -0.125 rounds to -0
    x[0, 64] = 2.0 ** -120                        # exponent -122 would be -122: byte 5, code 4 = 6
    x[0, 96] = np.inf
    x[0, 97] = 1.0
    q, s = mxfp4.quantize_rowwise_fp4(_bits(x))
    assert s.tolist() == [[0, 127, 5, 255]]
    assert q[0, 16:18].tolist() == [0x7 | 0xA << 4, 0x1 | 0x8 << 4]
    assert q[0, 32] == 6 and not q[0, 48:].any() and not q[0, :16].any()
    v = mxfp4.dequant_rowwise_fp4(q, s)
    assert v[0, 32:36].tolist() == [6.0, -1.0, 0.5, -0.0] and v[0, 64] == 2.0 ** -120 and np.isnan(v[0, 96:]).all()


def test_quantizer_refusals():
    lib = _lib()
    R, G = mx.SCALES_ROWMAJOR, mx.SCALES_GEMM
    q = lib.mx_quantize_rowwise_fp4
    d = lambda x, b, r, c, qq, s, lay, st: lib.mx_dequantize_fp4(qq, s, b, r, c, lay, x, st)  # noqa: E731
    for f in (q, d):
        assert f(FAKE, 1, 4, 48, FAKE, FAKE, R, None) == 2
        assert "multiple of 32" in _err(lib)
        assert f(FAKE, 1, 4, 96, FAKE, FAKE, G, None) == 2
        assert "multiple of 128" in _err(lib)
        assert f(FAKE, 1, 4, 96, FAKE, FAKE, 2, None) == 6
        assert f(FAKE, 0, 4, 64, FAKE, FAKE, R, None) == 2
        assert f(FAKE, 1, -4, 64, FAKE, FAKE, R, None) == 2
        assert f(None, 1, 4, 64, FAKE, FAKE, R, None) == 1
        assert f(FAKE, 1, 4, 64, FAKE, None, R, None) == 1
        assert f(FAKE + 8, 1, 4, 64, FAKE, FAKE, R, None) == 3
        assert f(FAKE, 1, 4, 64, FAKE + 4, FAKE, R, None) == 3
        assert f(FAKE, 4, 1 << 25, 1024, FAKE, FAKE, R, None) == 2
        assert "2^32" in _err(lib)
        assert f(FAKE, 1 << 40, 1 << 40, 1024, FAKE, FAKE, R, None) == 2
        assert f(None, 1, 0, 64, None, None, R, None) == 0
    w = lib.mx_quantize_weights_fp4
    assert w(FAKE, 2, 256, 200, FAKE, FAKE, FAKE, FAKE, None) == 2
    assert w(FAKE, 2, 96, 256, FAKE, FAKE, FAKE, FAKE, None) == 2
    assert w(FAKE, 0, 128, 128, FAKE, FAKE, FAKE, FAKE, None) == 2
    assert w(FAKE, 1, 128, 128, FAKE, FAKE, None, FAKE, None) == 1
    assert w(FAKE, 1, 128, 128, FAKE, FAKE + 2, FAKE, FAKE, None) == 3
    assert w(None, 1, 0, 128, None, None, None, None, None) == 0


def test_binding_refusals():
    import torch
    _lib()
    with pytest.raises(ValueError, match="GPU tensor"):
        mx.mx_quantize_rowwise_fp4(torch.zeros((4, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="multiple of 32"):
        mx._scale_shape("rowmajor", (), 4, 48)
    with pytest.raises(ValueError, match="multiple of 128"):
        mx._scale_shape("gemm", (), 4, 96)
    with pytest.raises(ValueError, match="scale_layout"):
        mx._scale_shape("blocked", (), 4, 96)


def test_product_refusals():
    lib = _lib()
    g = lib.mx_grouped_gemm_mxfp4
    G = mx.SCALES_GEMM

    def call(X=FAKE, xf=0, Y=FAKE, lay=G, offs=FAKE, I=64, J=64, Kc=256, E=2, rm=None, cr=0, C=FAKE):
        return g(X, FAKE, xf, Y, FAKE, lay, offs, I, J, Kc, E, rm, cr, C, 0, None)

    assert call(lay=mx.SCALES_ROWMAJOR) == 6
    assert call(xf=2) == 2 and "x_format" in _err(lib)
    assert call(Kc=192) == 2 and call(Kc=0) == 2 and call(J=60) == 2 and call(I=-1) == 2
    assert call(E=0) == 2 and call(E=1025) == 2 and call(Kc=(1 << 23) + 128) == 2
    assert call(I=(1 << 31) - 1, J=1 << 20) == 2 and "tiles" in _err(lib)
    assert call(Y=None) == 1 and call(C=None) == 1 and call(offs=None) == 1
    assert call(X=FAKE + 8) == 3 and call(rm=FAKE + 2, cr=5) == 3
    assert call(rm=FAKE, cr=-1) == 2
    assert call(I=0) == 0 and call(J=0) == 0 and call(rm=FAKE, cr=0) == 0
    ws = lib.mx_grouped_mm_fp4_workspace_bytes
    assert ws(100, 256, 0) >= 100 * 264 > ws(100, 256, 1) >= 100 * 136
    assert ws(-1, 256, 0) == 0 and ws(100, 192, 0) == 0 and ws(100, 256, 2) == 0
    f, d = lib.mx_grouped_mm_fwd_fp4, lib.mx_grouped_mm_dgrad_fp4
    need = ws(256, 256, 0)
    assert f(FAKE, FAKE, FAKE, FAKE, 256, 512, 256, 2, 0, FAKE, FAKE, need - 1, None) == 4
    assert f(FAKE, FAKE, None, FAKE, 256, 512, 256, 2, 0, FAKE, FAKE, need, None) == 1
    assert f(FAKE, FAKE, FAKE, FAKE, 256, 512, 192, 2, 0, FAKE, FAKE, 1 << 40, None) == 2
    assert f(FAKE, FAKE, FAKE, FAKE, 256, 516, 256, 2, 0, FAKE, FAKE, 1 << 40, None) == 2
    assert f(FAKE, FAKE, FAKE, FAKE, 256, 512, 256, 2, 3, FAKE, FAKE, 1 << 40, None) == 2
    assert f(FAKE, FAKE, FAKE, FAKE, 256, 512, 256, 2, 0, FAKE, FAKE + 16, 1 << 40, None) == 3
    assert d(FAKE, FAKE, FAKE, FAKE, 256, 192, 256, 2, 0, FAKE, FAKE, 1 << 40, None) == 2


def test_product_binding_refusals():
    import torch
    _lib()
    with pytest.raises(ValueError, match="x_format"):
        mx.mx_grouped_gemm_mxfp4(*[None] * 5, x_format="fp4")
    with pytest.raises(ValueError, match="GPU tensor"):
        u8 = torch.zeros((4, 128), dtype=torch.uint8)
        mx.mx_grouped_gemm_mxfp4(u8, u8, u8, u8, u8)
    with pytest.raises(ValueError, match="act_format"):
        mx.mx_grouped_mm_fwd_fp4(*[None] * 4, act_format="bf16")


def test_moe_refusals():
    lib = _lib()
    need = lib.mx_moe_few_tokens_workspace_bytes(8, 2, 256)
    assert need >= 16 * 264 and need % 256 == 0
    assert lib.mx_moe_few_tokens_workspace_bytes(129, 2, 256) == 0
    assert lib.mx_moe_few_tokens_workspace_bytes(8, 33, 256) == 0
    assert lib.mx_moe_few_tokens_workspace_bytes(8, 2, 192) == 0

    def call(x=FAKE, ids=FAKE, c=FAKE, q=FAKE, s=FAKE, wf=1, T=8, k=2, K=256, N=256, E=4, out=FAKE, st=None, ws=FAKE,
             nb=need):
        return lib.mx_moe_few_tokens(x, ids, c, q, s, q, s, wf, T, k, K, N, E, out, st, ws, nb, None)

    assert call(wf=2) == 2
    assert call(T=129) == 2 and "grouped GEMMs" in _err(lib)
    assert call(T=-1) == 2 and call(k=0) == 2 and call(k=33) == 2 and call(E=0) == 2 and call(E=1025) == 2
    assert call(K=192) == 2 and call(N=0) == 2 and call(K=(1 << 16) + 128) == 2 and call(N=(1 << 20) + 128) == 2
    for name in ("x", "ids", "c", "q", "s", "out"):
        assert call(**{name: None}) == 1, name
    assert call(x=FAKE + 8) == 3 and call(q=FAKE + 8) == 3 and call(out=FAKE + 8) == 3 and call(ids=FAKE + 2) == 3
    assert call(st=FAKE + 2) == 3 and call(ws=FAKE + 16) == 3
    assert call(nb=need - 1) == 4 and call(ws=None) == 4
    assert call(x=None, T=0) == 0


def test_moe_oracle_by_hand():
    """One token, one expert, values that every format holds: g = 2, u = 3 in
    every row, h = MX8(silu(2) * 3), out = combine * N * h."""
    from oracle import moe
    K = N = 128
    x = _bits(np.concatenate([[1.0], np.zeros(K - 1)]))[None]
    w13 = np.zeros((1, 2 * N, K))
    w13[0, :N, 0], w13[0, N:, 0] = 2.0, 3.0
    out, tol = moe.moe_layer(x, np.array([[0]]), np.array([[0.5]], dtype=np.float32), w13, np.ones((1, K, N)), 0.0)
    h = 2 / (1 + np.exp(-2.0)) * 3                    # 5.28: on the grid of halves, 5.5 (step 0.5 in [4, 8))
    assert abs(h - 5.28) < 0.01 and np.allclose(out, 0.5 * N * 5.5) and (tol < 3).all()


def test_moe_refuses_hidden_layers_past_its_offsets():
    lib = _lib()
    assert lib.mx_moe_few_tokens_workspace_bytes(128, 32, 1 << 18) > 0
    assert lib.mx_moe_few_tokens_workspace_bytes(128, 32, (1 << 18) + 128) == 0
    assert lib.mx_moe_few_tokens(*[FAKE] * 7, 1, 128, 32, 256, (1 << 18) + 128, 4, FAKE, None, FAKE, 1 << 40, None) == 2
    assert "2^30" in _err(lib)


def test_sizes_past_one_launch_are_refused():
    lib = _lib()
    G = mx.SCALES_GEMM
    for f in (lib.mx_quantize_rowwise_fp4,
              lambda x, b, r, c, q, s, lay, st: lib.mx_dequantize_fp4(q, s, b, r, c, lay, x, st)):
        assert f(FAKE, 1, 1, (1 << 30) + 128, FAKE, FAKE, G, None) == 2
        assert "2^30" in _err(lib)
    g = lib.mx_grouped_gemm_mxfp4
    # one row, 2^23 column tiles: 2^32 threads
    assert g(FAKE, FAKE, 0, FAKE, FAKE, G, FAKE, 1, (1 << 31) - 8, 128, 1, None, 0, FAKE, 0, None) == 2
    assert "tiles" in _err(lib)
    assert g(FAKE, FAKE, 0, FAKE, FAKE, G, FAKE, 1 << 21, 1 << 20, 128, 1024, None, 0, FAKE, 0, None) == 2


def test_caches_refuse_unknown_formats():
    import torch
    from mxfp8_block_scaled_06_amd.autograd import WeightCache
    _lib()
    with pytest.raises(ValueError, match="weight_format"):
        WeightCache().get(torch.zeros((1, 128, 128), dtype=torch.bfloat16), weight_format="fp4")
