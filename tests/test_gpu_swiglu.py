"""The gated activation on the GPU against the fp64 oracle: bf16 forms, the 8-bit
checkpoint (bit for bit what the rowwise quantizer writes), gradients at the
values kept, and the form between two products with its codes, each within reach
of fp32's error; rows without an item, NaN, far values, graphs."""

import numpy as np
import pytest

import oracle
from oracle import around, ulp_bf16
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, u8_host, log

pytestmark = pytest.mark.gpu

# silu in fp32: the power at 2^-22, an addition, a reciprocal of an ulp, products:
# below 2^-20 of the value, and as much of the magnitudes that silu' is added from.
REL = 2.0 ** -20
TINY = 2.0 ** -126


def _f64(t):
    return t.detach().cpu().double().numpy()


def _rows_major(s):
    """GEMM-layout scales [C/128, R, 4] -> row-major [R, C/32]."""
    s = u8_host(s)
    return np.ascontiguousarray(s.transpose(1, 0, 2)).reshape(s.shape[1], -1)


def _bf16_close(got, ref, mag):
    tol = REL * mag + TINY
    tol = tol + 0.5 * ulp_bf16(np.abs(ref) + tol)
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / tol).max()


def _kept(gu_bits):
    q, s = oracle.quantize_rowwise(gu_bits)
    return q, s, oracle.dequant_rowwise(q, s)


@pytest.mark.parametrize("M,N", [(1, 32), (7, 8192), (3, 96), (129, 160), (4099, 64), (33, 2048)])
def test_activation_matches_oracle(M, N):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"swiglu M={M} N={N}")
    bits, dbits = inp.random_bf16((M, 2 * N), seed=M + N, outliers=True), inp.random_bf16((M, N), seed=M, std=1e-3)
    gu = to_dev_bf16(bits)
    h, kept, kept_s = mx.mx_swiglu_fwd(gu)
    x = oracle.bf16_to_f64(bits)
    ref = around.swiglu(x[:, :N], x[:, N:])
    _bf16_close(_f64(h), ref, np.abs(ref))
    q, s, v = _kept(bits)
    assert np.array_equal(u8_host(kept), q) and np.array_equal(u8_host(kept_s), s)
    assert torch.equal(mx.mx_swiglu_fwd(gu, keep=False)[0], h) and torch.equal(mx.mx_swiglu(gu), h)
    d = oracle.bf16_to_f64(dbits)
    dg, du, mag = around.swiglu_grad(d, v[:, :N], v[:, N:])
    leaf = gu.clone().requires_grad_()
    out = mx.mx_swiglu(leaf)
    assert torch.equal(out, h)
    got, = torch.autograd.grad(out, leaf, to_dev_bf16(dbits))
    _bf16_close(_f64(got)[:, :N], dg, mag)
    _bf16_close(_f64(got)[:, N:], du, np.abs(du))
    assert torch.equal(mx.mx_swiglu_bwd(to_dev_bf16(dbits), kept, kept_s), got)


def test_activation_over_the_whole_range():
    """Every bf16 gate value, ups of 1 and of a large number."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    g = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).reshape(-1, 64)
    for up in (1.0, 2.0 ** 60):
        u = np.full_like(g, inp.f32_to_bf16_bits(np.float32(up)))
        h = _f64(mx.mx_swiglu(to_dev_bf16(np.concatenate([g, u], 1))))
        x = oracle.bf16_to_f64(g)
        with np.errstate(invalid="ignore", over="ignore"):
            ref = around.swiglu(x, up)
        nan = np.isnan(x) | (x == -np.inf)
        assert np.isnan(h[nan]).all()
        top = 2.0 ** 127 * (2 - 2.0 ** -8)                 # from here on bf16 rounds to infinity
        big = np.isfinite(x) & (np.abs(ref) >= top)
        assert (np.abs(h[big]) == np.inf).all() and (h[x == np.inf] == np.inf).all()
        fine = ~nan & np.isfinite(ref) & ~big
        _bf16_close(h[fine], ref[fine], np.abs(ref[fine]))


def test_gradient_over_the_codes():
    """Every finite code as gate, at several scales, up and gradient 1."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    codes = np.concatenate([codes, codes[:2]]).reshape(8, 32)
    for byte in (0, 1, 90, 119, 121, 125, 127, 140, 200, 246):
        kept = np.concatenate([codes, np.full_like(codes, 0x38)], 1)           # 0x38: 1.0
        s = np.stack([np.full(8, byte), np.full(8, 127)], 1).astype(np.uint8)
        d = inp.f32_to_bf16_bits(np.ones((8, 32), np.float32))
        got = _f64(mx.mx_swiglu_bwd(to_dev_bf16(d), torch.from_numpy(kept).cuda(), torch.from_numpy(s).cuda()))
        g = oracle.e4m3_decode(codes) * 2.0 ** (byte - 127.0)
        dg, du, mag = around.swiglu_grad(1.0, g, 1.0)
        _bf16_close(got[:, :32], dg, mag)
        _bf16_close(got[:, 32:], du, np.abs(du))


def test_nan_blocks():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    bits = inp.random_bf16((6, 128), seed=9)
    bits[1, 3] = 0x7FC0
    bits[2, 70] = 0x7F80
    bits[4, 40] = 0xFF80
    q, s, _ = _kept(bits)
    h, kept, kept_s = mx.mx_swiglu_fwd(to_dev_bf16(bits))
    assert np.array_equal(u8_host(kept), q) and np.array_equal(u8_host(kept_s), s)
    dgu = mx.mx_swiglu_bwd(torch.ones((6, 64), dtype=torch.bfloat16, device="cuda:0"), kept, kept_s)
    bad = torch.isnan(dgu).cpu().numpy()
    want = np.zeros((6, 128), dtype=bool)
    want[1, :32] = want[1, 64:96] = want[2, :32] = want[4, 32:64] = want[4, 96:] = True
    want[2, 64:96] = False                       # the gradient of an up value has no up value in it
    assert np.array_equal(bad, want)


def _routing(rng, T, k, E, drop=0.0):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


def _grouped(rng, rows, cols, seed, std=1.0, outliers=False):
    """bf16 rows: of items random, padding zero, behind the last group NaN."""
    bits = inp.random_bf16((rows.shape[0], cols), seed=seed, std=std, outliers=outliers)
    bits[rows < 0] = 0
    last = np.flatnonzero(rows >= 0)
    bits[(last[-1] + 1 if last.size else 0):] = 0x7FC0
    return bits


def _check_codes(q, s, x, d):
    ok = around.codes_reached(q, s, x, d)
    assert ok.all(), (int((~ok).sum()), np.argwhere(~ok)[:4].tolist())


@pytest.mark.parametrize("T,k,E,N,drop", [(1, 1, 1, 128, 0), (100, 2, 4, 256, 0), (77, 3, 5, 384, 0.3), (300, 1, 2, 128, 0),
                                          (0, 2, 3, 128, 0), (40, 8, 32, 640, 0), (5, 2, 3, 128, 1.0)])
def test_activation_of_routed_rows(T, k, E, N, drop):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"swiglu_quantize T={T} k={k} E={E} N={N} drop={drop}")
    rng = np.random.default_rng(T + N)
    ids = _routing(rng, T, k, E, drop)
    cap = mx.route_capacity(T * k, E)
    _, rows, pos, _ = oracle.route_groups(ids.reshape(-1), E, cap)
    live = (rows >= 0)[:, None]
    w = rng.random((T, k)).astype(np.float32)
    if T:
        w[0, 0] = 0
    wr = np.where(rows >= 0, w.reshape(-1)[np.maximum(rows, 0)] if w.size else 0, 0).astype(np.float64)[:, None]
    bits = _grouped(rng, rows, 2 * N, seed=3, outliers=True)
    dbits = _grouped(rng, rows, N, seed=4, std=1e-3)
    d_rows, d_pos, d_w = to_dev_i32(rows), to_dev_i32(pos), torch.from_numpy(w).cuda()
    gu = to_dev_bf16(bits)
    q, s, qt, st, kept, kept_s = mx.mx_swiglu_quantize_fwd(gu, d_rows, d_w)
    x = np.where(live, np.nan_to_num(oracle.bf16_to_f64(bits)), 0.0)
    h = around.swiglu(x[:, :N], x[:, N:])
    _check_codes(u8_host(q), _rows_major(s), h, REL * np.abs(h))
    wh = wr * h
    _check_codes(u8_host(qt), _rows_major(st), np.ascontiguousarray(wh.T), REL * np.abs(wh.T) + TINY)
    rq, rs, v = _kept(np.where(live, bits, 0).astype(np.uint16))
    assert np.array_equal(u8_host(kept), rq) and np.array_equal(_rows_major(kept_s), rs)
    alone = mx.mx_swiglu_quantize(gu, d_rows)
    assert torch.equal(alone[0], q) and torch.equal(alone[1], s)

    dq, ds, dqt, dst, dc = mx.mx_swiglu_quantize_bwd(to_dev_bf16(dbits), kept, kept_s, d_rows, d_pos, d_w)
    dh = np.where(live, np.nan_to_num(oracle.bf16_to_f64(dbits)), 0.0)
    dg, du, mag = around.swiglu_grad(wr * dh, v[:, :N], v[:, N:])
    dgu, tol = np.concatenate([dg, du], 1), REL * np.concatenate([mag, np.abs(du)], 1) + TINY * live
    _check_codes(u8_host(dq), _rows_major(ds), dgu, tol)
    _check_codes(u8_host(dqt), _rows_major(dst), np.ascontiguousarray(dgu.T), np.ascontiguousarray(tol.T))
    # a row's sum: 8 + 4 additions within a tile and one per tile, at 2^-24 of the magnitudes
    p = dh * around.swiglu(v[:, :N], v[:, N:])
    routed = pos >= 0
    ref = np.where(routed, p.sum(1)[np.maximum(pos, 0)], 0.0)
    most = (REL + (13 + N // 128) * 2.0 ** -24) * np.abs(p).sum(1)[np.maximum(pos, 0)]
    err = np.abs(_f64(dc).reshape(-1) - ref)
    assert (err <= np.where(routed, most + TINY, 0)).all()


def test_rows_that_are_their_own_items():
    """Without rows: a dense layer's activation; M not a multiple of 128, a longer ldq."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    M, N = 160, 256
    bits, dbits = inp.random_bf16((M, 2 * N), seed=1), inp.random_bf16((M, N), seed=2)
    gu, dh = to_dev_bf16(bits), to_dev_bf16(dbits)
    rows = torch.arange(M, dtype=torch.int32, device="cuda:0")
    one = torch.ones(M, device="cuda:0")
    for ldq in (256, 512):
        a = mx.mx_swiglu_quantize_fwd(gu, ldq=ldq)
        b = mx.mx_swiglu_quantize_fwd(gu, rows, one, ldq=ldq)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert not a[2][:, M:].any() and not a[3].permute(0, 2, 1).reshape(ldq // 32, N)[M // 32:].any()
        c = mx.mx_swiglu_quantize_bwd(dh, a[4], a[5], ldq=ldq)
        d = mx.mx_swiglu_quantize_bwd(dh, a[4], a[5], rows, rows, one, ldq=ldq)
        e = mx.mx_swiglu_quantize_bwd(dh, a[4], a[5], combine=one, ldq=ldq)
        assert c[4] is None and torch.equal(d[4], e[4])
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(c[:4], d, e))
    # the bf16 form and the rowwise quantizer leave the same checkpoint
    h, kept, kept_s = mx.mx_swiglu_fwd(gu)
    assert torch.equal(kept, a[4]) and torch.equal(mx.mx_scales_to_gemm_layout(kept_s), a[5])
    # any number of rows without the columns
    q, s = mx.mx_swiglu_quantize(gu[:37].contiguous())
    assert torch.equal(q, a[0][:37]) and torch.equal(s, a[1][:, :37].contiguous())
    with pytest.raises(mx.MXError):
        mx.mx_swiglu_quantize_fwd(gu[:37].contiguous())
    with pytest.raises(ValueError):
        mx.mx_swiglu_quantize_bwd(dh, a[4], a[5], rows, None, one)
    with pytest.raises(ValueError):
        mx.mx_swiglu_quantize_fwd(gu, combine=one[:5])
    with pytest.raises(mx.MXError, match="WORKSPACE"):
        mx.mx_swiglu_quantize_bwd(dh, a[4], a[5], rows, rows, one, ws=torch.empty(16, dtype=torch.uint8, device="cuda:0"))


def test_entries_out_of_range_are_no_items():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    gu = to_dev_bf16(inp.random_bf16((32, 256), seed=5))
    w = torch.rand(8, device="cuda:0")
    rows = torch.full((32,), -1, dtype=torch.int32, device="cuda:0")
    rows[:4] = torch.tensor([7, 8, 1 << 30, 0], dtype=torch.int32)
    q = mx.mx_swiglu_quantize_fwd(gu, rows, w)[0]
    assert q[0].any() and q[3].any() and not q[1:3].any() and not q[4:].any()


def test_activation_in_a_graph():
    """Two graphs with workspaces of their own, replayed in turn with new inputs."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(8)
    T, k, E, N = 50, 2, 3, 256
    cap = mx.route_capacity(T * k, E)
    _, rows, pos, _ = oracle.route_groups(_routing(rng, T, k, E).reshape(-1), E, cap)
    rows, pos = to_dev_i32(rows), to_dev_i32(pos)
    w = torch.rand((T, k), device="cuda:0")
    steps = []
    for _ in range(2):
        gu = torch.randn((cap, 2 * N), device="cuda:0").bfloat16()
        dh = torch.randn((cap, N), device="cuda:0").bfloat16()
        ws = torch.empty(mx.mx_swiglu_quantize_workspace_bytes(cap, N), dtype=torch.uint8, device="cuda:0")
        first = mx.mx_swiglu_quantize_fwd(gu, rows, w)
        second = mx.mx_swiglu_quantize_bwd(dh, first[4], first[5], rows, pos, w, ws=ws)

        def step(gu=gu, dh=dh, ws=ws, a=first, b=second):
            mx.mx_swiglu_quantize_fwd(gu, rows, w, None, *a)
            mx.mx_swiglu_quantize_bwd(dh, a[4], a[5], rows, pos, w, None, *b, ws=ws)
            return (*a, *b)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        steps.append((gu, dh, step, graph))
    for _ in range(3):
        for gu, dh, step, graph in steps:
            gu.copy_(torch.randn(gu.shape, device="cuda:0"))
            dh.copy_(torch.randn(dh.shape, device="cuda:0"))
        for *_, graph in steps:
            graph.replay()
        torch.cuda.synchronize()
        for gu, dh, step, graph in steps:
            got = [t.clone() for t in step()]          # eager, over the replay's outputs
            graph.replay()
            torch.cuda.synchronize()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("layout", ["rowmajor", "gemm"])
def test_dequantizer(layout):
    """Every code at every scale byte; both layouts; batches."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    q = np.arange(256, dtype=np.uint8).reshape(1, 2, 128).repeat(256, 0)
    s = np.arange(256, dtype=np.uint8).reshape(256, 1, 1).repeat(2, 1).repeat(4, 2)
    ss = s if layout == "rowmajor" else s.reshape(256, 2, 1, 4).transpose(0, 2, 1, 3)
    out = _f64(mx.mx_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(np.ascontiguousarray(ss)).cuda(), layout))
    with np.errstate(invalid="ignore"):
        v = oracle.e4m3_decode(q) * np.where(s == 255, np.nan, np.exp2(s - 127.0)).repeat(32, 2)
    assert np.array_equal(np.isnan(out), np.isnan(v))
    normal = np.abs(v) >= 2.0 ** -126
    over = np.abs(v) >= 2.0 ** 128
    assert np.array_equal(out[normal & ~over], v[normal & ~over]) and (np.abs(out[over]) == np.inf).all()
    small = ~normal & ~np.isnan(v)
    assert (np.abs(out[small] - v[small]) <= 2.0 ** -134).all()
    # rows and blocks at their places
    x = inp.random_bf16((3, 37, 256), seed=6)
    d = to_dev_bf16(x)
    q, s = mx.mx_quantize_rowwise(d)
    sg = mx.mx_scales_to_gemm_layout(s)
    a, b = mx.mx_dequantize(q, s), mx.mx_dequantize(q, sg, "gemm")
    want = oracle.dequant_rowwise(*oracle.quantize_rowwise(x.reshape(-1, 256))).reshape(x.shape)
    assert torch.equal(a, b) and np.array_equal(_f64(a), want)


def test_replays_of_the_routed_activation():
    """Two graphs with workspaces of their own, replayed in turn on new values: each replay's outputs, kept before
    the buffers are filled with other bytes, are those of eager steps."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(8)
    T, k, E, N = 50, 2, 3, 256
    cap = mx.route_capacity(T * k, E)
    _, rows, pos, _ = oracle.route_groups(_routing(rng, T, k, E).reshape(-1), E, cap)
    rows, pos = to_dev_i32(rows), to_dev_i32(pos)
    steps = []
    for _ in range(2):
        w = torch.rand((T, k), device="cuda:0")
        gu = torch.randn((cap, 2 * N), device="cuda:0").bfloat16()
        dh = torch.randn((cap, N), device="cuda:0").bfloat16()
        ws = torch.empty(mx.mx_swiglu_quantize_workspace_bytes(cap, N), dtype=torch.uint8, device="cuda:0")
        outs = [*mx.mx_swiglu_quantize_fwd(gu, rows, w)]
        outs += mx.mx_swiglu_quantize_bwd(dh, outs[4], outs[5], rows, pos, w, ws=ws)

        def step(gu=gu, dh=dh, ws=ws, w=w, outs=outs):
            mx.mx_swiglu_quantize_fwd(gu, rows, w, None, *outs[:6])
            mx.mx_swiglu_quantize_bwd(dh, outs[4], outs[5], rows, pos, w, None, *outs[6:], ws=ws)

        def spoil(ws=ws, outs=outs):
            for t in (ws, *outs):
                t.fill_(77)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        steps.append(((gu, dh, w), outs, step, spoil, graph))
    before = None
    for _ in range(3):
        for inputs, _, _, spoil, _ in steps:
            for t in inputs:
                t.copy_(torch.randn(t.shape, device="cuda:0"))
            spoil()
        for *_, graph in steps:
            graph.replay()
        torch.cuda.synchronize()
        kept = [[t.clone() for t in outs] for _, outs, *_ in steps]
        assert before is None or not any(torch.equal(a[0], b[0]) for a, b in zip(kept, before))
        before = kept
        for (_, outs, step, spoil, _), got in zip(steps, kept):
            spoil()
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
