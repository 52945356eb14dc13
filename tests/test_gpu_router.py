"""The router on the GPU against the fp64 oracle: every choice equal, weights and
gradients within fp32's error; masks, ties, groups, NaN, odd expert counts,
single tokens, graphs, and the ids as they reach the few-token layer."""

import numpy as np
import pytest

from oracle import around, ulp_bf16
from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, log

pytestmark = pytest.mark.gpu

LOWEST = {"fp32": float(np.finfo(np.float32).min), "bf16": -2.0 ** 127 * (2 - 2.0 ** -7)}

# Weights: two powers at 2^-22 each (the hardware's at 2^-23, its argument's
# rounding put back), up to 16 + 6 additions of the sum, a division, a product
# at 2^-24: below 2^-19.  Results below fp32's normal range may be 0.
REL_W, TINY = 2.0 ** -19, 2.0 ** -126
# Gradients: of the magnitudes they are added from, the weights' error, the sum
# over the slots (five additions more) and three products: below 2^-18.
REL_D = 2.0 ** -18


def _logits(rng, T, E, dtype, std=1.5):
    l = rng.normal(size=(T, E)).astype(np.float32) * np.float32(std)
    return l if dtype == "fp32" else inp.bf16_bits_to_f32(inp.f32_to_bf16_bits(l))


def _dev(l, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(l, dtype=np.float32)).to("cuda:0").to(
        torch.float32 if dtype == "fp32" else torch.bfloat16)


def _check(l, dtype, k, rng, bias=None, grad=True, **kw):
    import torch
    import mxfp8_block_scaled_06_amd as mx
    T = l.shape[0]
    rids, rw = around.router(l, LOWEST[dtype], k, bias=bias, **kw)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).to("cuda:0")
    x = _dev(l, dtype).requires_grad_(grad)
    ids, w = mx.mx_topk_router(x, k, bias=b, **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    got = w.detach().cpu().double().numpy()
    assert (np.abs(got - rw) <= REL_W * rw + TINY).all(), np.abs(got - rw).max()
    if not grad:
        return
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dl, = torch.autograd.grad(w, x, torch.from_numpy(dw).to("cuda:0"))
    assert dl.dtype == x.dtype
    ref, mag = around.router_grad(l, LOWEST[dtype], rids, dw, kw.get("score", "softmax"), kw.get("renormalize", True),
                                  kw.get("scale", 1.0))
    tol = REL_D * mag + TINY
    if dtype == "bf16":
        tol = tol + 0.5 * ulp_bf16(np.abs(ref) + tol)
    err = np.abs(dl.cpu().double().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 16, 1), (7, 5, 5), (33, 64, 8), (9, 65, 6), (130, 128, 32), (5, 200, 3),
                                   (17, 256, 8), (4, 511, 7), (3, 1024, 32)])
def test_router_matches_oracle(T, E, k, score, dtype):
    require_gpu()
    log(f"router T={T} E={E} k={k} {score} {dtype}")
    rng = np.random.default_rng(T + E + k)
    l = _logits(rng, T, E, dtype)
    for renormalize in (True, False):
        for bias in (None, rng.normal(size=E).astype(np.float32) * np.float32(0.05)):
            _check(l, dtype, k, rng, bias, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("T,E,k,groups,kept", [(31, 256, 8, 8, 4), (6, 60, 4, 4, 1), (5, 66, 9, 3, 2), (3, 128, 8, 64, 7),
                                               (2, 1024, 16, 16, 16), (4, 8, 2, 8, 2)])
def test_groups(T, E, k, groups, kept, group_score):
    require_gpu()
    log(f"router groups T={T} E={E} k={k} groups={groups} kept={kept} {group_score}")
    rng = np.random.default_rng(E + groups)
    for score, bias in (("sigmoid", rng.normal(size=E).astype(np.float32) * np.float32(0.1)), ("softmax", None)):
        _check(_logits(rng, T, E, "fp32"), "fp32", k, rng, bias, score=score, groups=groups, topk_groups=kept,
               group_score=group_score)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score, dtype):
    """-inf and the lowest finite value mask alike; rows of nothing else give
    weights and gradients of 0 and distinct ids."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(3)
    l = _logits(rng, 40, 48, dtype)
    l[rng.random(l.shape) < 0.3] = -np.inf
    l[rng.random(l.shape) < 0.3] = LOWEST[dtype]
    l[7] = -np.inf
    l[8] = LOWEST[dtype]
    l[9] = np.where(np.arange(48) % 2 == 0, -np.inf, LOWEST[dtype])
    l[10] = -np.inf
    l[10, 30] = -1e4                                         # one expert alone
    bias = rng.normal(size=48).astype(np.float32)
    for kw in ({}, {"groups": 6, "topk_groups": 2, "group_score": "top2"}, {"groups": 6, "topk_groups": 2}):
        for b in (None, bias):
            for renormalize in (True, False):
                _check(l, dtype, 8, rng, b, score=score, renormalize=renormalize, **kw)
    ids, w = mx.mx_topk_router(_dev(l, dtype), 8, score=score)
    assert (w[7:10] == 0).all() and all(len(set(r)) == 8 for r in ids.cpu().numpy().tolist())
    assert float(w[10, 0]) == 1


@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lowest_index(bias):
    """Few distinct logits: nearly every choice is one among equals."""
    require_gpu()
    rng = np.random.default_rng(4)
    for E, k, groups in ((64, 8, 1), (200, 32, 1), (256, 8, 8), (96, 5, 4)):
        l = rng.integers(-2, 3, size=(50, E)).astype(np.float32)
        b = np.round(rng.normal(size=E)).astype(np.float32) if bias else None
        for gs in ("max", "top2"):
            _check(l, "bf16", k, rng, b, score="sigmoid", groups=groups, topk_groups=max(1, groups // 2), group_score=gs)


def test_choice_beyond_fp32():
    """Scores that fp32 holds equal and 64 bits do not: saturated sigmoids, small
    scores beside a bias of the same value."""
    require_gpu()
    rng = np.random.default_rng(5)
    l = 16 + np.arange(40, dtype=np.float32)[None, :] / 8 * rng.choice([-1, 1], size=(20, 40)).astype(np.float32)
    _check(l, "fp32", 9, rng, np.zeros(40, np.float32), score="sigmoid", grad=False)
    l = -rng.random((20, 300)).astype(np.float32) * 3 - 17
    _check(l, "fp32", 9, rng, np.full(300, 0.75, np.float32), score="sigmoid")
    # softmax scores 1e-9 apart
    l = rng.normal(size=(64, 256)).astype(np.float32) * np.float32(1e-6)
    _check(l, "fp32", 8, rng, np.full(256, -0.125, np.float32))


def test_far_logits():
    """Large logits, and weights whose scores lie below fp32's range."""
    require_gpu()
    rng = np.random.default_rng(6)
    for score in ("softmax", "sigmoid"):
        for shift in (-300.0, -95.0, 95.0, 3e4):
            l = (_logits(rng, 12, 70, "fp32") + np.float32(shift)).astype(np.float32)
            _check(l, "fp32", 6, rng, score=score, grad=shift > -300 or score == "softmax")


def test_nan_and_infinity():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(7)
    l = _logits(rng, 6, 100, "fp32")
    l[0, 3] = np.nan
    l[1] = np.nan
    l[2, 5] = np.inf
    l[3, [5, 6]] = np.inf
    for bias in (None, torch.full((100,), 0.5, device="cuda:0"), torch.full((100,), float("nan"), device="cuda:0")):
        for score in ("softmax", "sigmoid"):
            ids, w = mx.mx_topk_router(_dev(l, "fp32"), 8, score=score, bias=bias)
            got = ids.cpu().numpy()
            assert ((got >= 0) & (got < 100)).all() and all(len(set(r)) == 8 for r in got.tolist())
            if score == "softmax":
                assert torch.isnan(w[0:2]).all()
            if bias is None:
                assert got[2, 0] == 5 and got[3, :2].tolist() == [5, 6] and 3 not in got[0]
            # the other tokens do not notice
            clean, cw = mx.mx_topk_router(_dev(l[4:], "fp32"), 8, score=score, bias=bias)
            assert torch.equal(ids[4:], clean) and torch.equal(w[4:], cw)


def test_empty_and_given_outputs():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    ids, w = mx.mx_topk_router(torch.zeros((0, 8), device="cuda:0"), 2)
    assert tuple(ids.shape) == (0, 2) and tuple(w.shape) == (0, 2)
    l = torch.randn((5, 24), device="cuda:0")
    ids, w = torch.empty((5, 4), dtype=torch.int32, device="cuda:0"), torch.empty((5, 4), device="cuda:0")
    a, b = mx.mx_topk_router_fwd(l, 4, expert_idx=ids, combine=w)
    assert a is ids and b is w
    want = torch.topk(torch.softmax(l.double(), 1), 4)
    assert torch.equal(ids.long(), want.indices)
    # logits whose rows are not dense reach the kernel as a copy
    wide = torch.randn((5, 48), device="cuda:0")
    x, y = mx.mx_topk_router(wide[:, ::2], 4), mx.mx_topk_router(wide[:, ::2].contiguous(), 4)
    assert all(torch.equal(p, q) for p, q in zip(x, y))
    with pytest.raises(ValueError, match="contiguous"):
        mx.mx_topk_router_fwd(wide[:, ::2], 4)
    with pytest.raises(ValueError):
        mx.mx_topk_router_fwd(l, 4, bias=torch.zeros(23, device="cuda:0"))
    for bad in ({"score": "relu"}, {"group_score": "sum"}):
        with pytest.raises(ValueError):
            mx.mx_topk_router(l, 4, **bad)
    for bad in ({"groups": 5}, {"groups": 4, "topk_groups": 5}, {"scale": 0.0}):
        with pytest.raises(mx.MXError):
            mx.mx_topk_router(l, 4, **bad)
    with pytest.raises(mx.MXError):
        mx.mx_topk_router(l, 25)


def test_ids_that_are_not_the_forwards():
    """Ids out of range add nothing, a repeated one adds up."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    l = torch.randn((2, 70), device="cuda:0")
    ids = torch.tensor([[3, -1, 70, 1 << 30], [5, 5, 69, 5]], dtype=torch.int32, device="cuda:0")
    w, dw = torch.rand((2, 4), device="cuda:0"), torch.randn((2, 4), device="cuda:0")
    dl = mx.mx_topk_router_bwd(l, ids, w, dw, "sigmoid", False)
    part = (w * (1 - w) * dw).double()
    want = torch.zeros((2, 70), dtype=torch.float64, device="cuda:0")
    want[0, 3], want[1, 5], want[1, 69] = part[0, 0], part[1, 0] + part[1, 1] + part[1, 3], part[1, 2]
    assert (dl.double() - want).abs().max() <= 2.0 ** -20


def test_router_in_a_graph_and_on_a_stream():
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    bias = torch.randn(60, device="cuda:0") * 0.05
    l = torch.randn((9, 60), device="cuda:0", dtype=torch.bfloat16)
    ids, w = torch.empty((9, 4), dtype=torch.int32, device="cuda:0"), torch.empty((9, 4), device="cuda:0")
    dw, dl = torch.randn((9, 4), device="cuda:0"), torch.empty_like(l)

    def step():
        mx.mx_topk_router_fwd(l, 4, "sigmoid", bias, 4, 2, "top2", expert_idx=ids, combine=w)
        mx.mx_topk_router_bwd(l, ids, w, dw, "sigmoid", dlogits=dl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        l.copy_(torch.randn((9, 60), device="cuda:0"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (ids, w, dl)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, dl)))


def test_large_batch_is_deterministic():
    """More tokens than waves: every wave walks several.  Against the same call in pieces."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    l = torch.randn((40001, 32), device="cuda:0", dtype=torch.bfloat16)
    a = mx.mx_topk_router(l, 8, renormalize=False)
    parts = [mx.mx_topk_router(p.contiguous(), 8, renormalize=False) for p in l.split(1777)]
    assert torch.equal(a[0], torch.cat([p[0] for p in parts])) and torch.equal(a[1], torch.cat([p[1] for p in parts]))
    # a permutation of the tokens permutes the results
    at = torch.randperm(l.shape[0], device="cuda:0")
    b = mx.mx_topk_router(l[at], 8, renormalize=False)
    assert torch.equal(a[0][at], b[0]) and torch.equal(a[1][at], b[1])


@pytest.mark.parametrize("E,groups", [(32, 1), (64, 8), (100, 1), (128, 4), (256, 8), (256, 1), (500, 5), (512, 16), (1024, 1)])
def test_many_tokens_against_fp64(E, groups):
    """Enough tokens that some have experts, or groups, which fp32 would put in the
    wrong order: every choice that of the 64-bit scores, sorted with torch."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    gen = torch.Generator(device="cuda:0").manual_seed(E + groups)
    kept = max(1, groups // 2)
    for dtype in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            l = (torch.randn((20000, E), generator=gen, device="cuda:0") * 1.5).to(dtype)
            for bias, gs in ((None, "max"), (torch.randn(E, generator=gen, device="cuda:0") * 0.05, "top2")):
                k = min(8, kept * (E // groups))
                ids, _ = mx.mx_topk_router(l, k, score, bias, groups, kept, gs)
                d = l.double()
                c = d if bias is None else (torch.softmax(d, 1) if score == "softmax" else torch.sigmoid(d)) + bias.double()
                if groups > 1:
                    two = torch.sort(c.view(-1, groups, E // groups), dim=2, descending=True).values
                    value = two[..., 0] if gs == "max" else two[..., :2].sum(2)
                    best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :kept]
                    on = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
                    c = c.masked_fill(~on.repeat_interleave(E // groups, 1), -float("inf"))
                want = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
                assert torch.equal(ids.long(), want), (dtype, score, gs)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_zeros_of_either_sign_are_equal(dtype):
    """-0.0 beside +0.0, as logits times a mask of zeros and ones hold them: one value, so the lowest index,
    whichever lanes have them."""
    require_gpu()
    rng = np.random.default_rng(11)
    for E, k, groups in ((16, 1, 1), (40, 6, 1), (256, 8, 1), (256, 8, 8), (96, 5, 4), (60, 4, 4), (512, 8, 16), (1024, 32, 1)):
        l = -np.abs(_logits(rng, 40, E, dtype))
        at = rng.random(l.shape) < 0.5
        l[at] = rng.choice(np.array([-0.0, 0.0], np.float32), size=int(at.sum()))
        l[0] = np.where(np.arange(E) < E // 4, -0.0, 0.0)
        l[1] = np.where(np.arange(E) < E // 4, 0.0, -0.0)
        for score in ("softmax", "sigmoid"):
            _check(l, dtype, k, rng, score=score, groups=groups, topk_groups=max(1, groups // 2))


@pytest.mark.parametrize("E,groups", [(32, 8), (256, 8), (512, 16)])
def test_group_sums_that_cancel(E, groups):
    """A large positive c and a large negative one in every group: their sums lie far below what fp32 keeps of
    them.  Every choice that of the 64-bit sums."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    gen = torch.Generator(device="cuda:0").manual_seed(E)
    n = E // groups
    for big in (1e3, 1e5, 3e38):
        # (at 3e38 the two largest of every group add up to infinity in fp32)
        bias = torch.full((groups, n), -big, device="cuda:0")
        bias[:, 0] = big
        if big > 1e30:
            bias = -bias * (1 + torch.arange(groups, device="cuda:0") / 256).unsqueeze(1)
        bias = bias.reshape(-1)
        for score in ("softmax", "sigmoid"):
            l = torch.randn((40000, E), generator=gen, device="cuda:0") * 1.5
            ids, _ = mx.mx_topk_router(l, 1, score, bias, groups, 1, "top2")
            d = l.double()
            c = (torch.softmax(d, 1) if score == "softmax" else torch.sigmoid(d)) + bias.double()
            value = torch.sort(c.view(-1, groups, n), dim=2, descending=True).values[..., :2].sum(2)
            best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :1]
            c = c.view(-1, groups, n).gather(1, best.unsqueeze(2).expand(-1, 1, n)).squeeze(1)
            want = best * n + torch.sort(c, dim=1, descending=True, stable=True).indices[:, :1]
            assert torch.equal(ids.long(), want), (big, score, int((ids.long() != want).sum()))


def test_group_sums_below_fp32():
    """Biases of the lowest value: a group of such experts alone has a sum below fp32's range and comes before a
    group of masked ones."""
    require_gpu()
    rng = np.random.default_rng(12)
    l = _logits(rng, 9, 32, "fp32")
    l[:, :8] = -np.inf
    bias = np.zeros(32, np.float32)
    bias[8:24] = LOWEST["fp32"]
    for kept, k in ((1, 4), (2, 12), (3, 12)):
        _check(l, "fp32", k, rng, bias, score="sigmoid", groups=4, topk_groups=kept, group_score="top2")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gradient_of_sure_experts(dtype):
    """Sigmoid scores next to 1: their gradient is s (1 - s), of which fp32's 1 - s leaves nothing from a logit of
    17 on.  The weight at 2^-19, the logit's own sigmoid at 2^-21, two products at 2^-24: below REL_D of the value."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(13)
    for scale in (1.0, 2.5, 2.0 ** -20):
        l = (rng.random(size=(50, 24)).astype(np.float32) * 32 - 2).astype(np.float32)
        x = _dev(l, dtype).requires_grad_()
        v = x.detach().cpu().double().numpy()
        ids, w = mx.mx_topk_router(x, 6, "sigmoid", renormalize=False, scale=scale)
        dw = rng.normal(size=(50, 6)).astype(np.float32)
        dl, = torch.autograd.grad(w, x, torch.from_numpy(dw).to("cuda:0"))
        at = ids.cpu().numpy()
        p = np.take_along_axis(v, at, 1)
        want = np.zeros(v.shape)
        np.put_along_axis(want, at, scale * dw.astype(np.float64) / ((1 + np.exp(-p)) * (1 + np.exp(p))), 1)
        tol = REL_D * np.abs(want)
        if dtype == "bf16":
            tol = tol + 0.5 * ulp_bf16(np.abs(want) + tol)
        err = np.abs(dl.cpu().double().numpy() - want)
        assert (err <= tol + TINY).all(), (err / (tol + TINY)).max()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_experts_pass_no_gradient(score, renormalize, dtype):
    """Slots of masked experts, whose weights are 0: whatever comes in as their gradient (NaN and infinity of a
    padding token), the logits' gradient is that of zeros there, and 0 at the masked experts."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    rng = np.random.default_rng(14)
    l = _logits(rng, 12, 20, dtype)
    l[:, 5:] = np.where(rng.random((12, 15)) < 0.5, -np.inf, LOWEST[dtype])        # five left for six slots
    l[:3] = -np.inf                                                               # and none in padding tokens
    x = _dev(l, dtype)
    ids, w = mx.mx_topk_router_fwd(x, 6, score, renormalize=renormalize)
    dw = torch.from_numpy(rng.normal(size=(12, 6)).astype(np.float32)).to("cuda:0")
    off = torch.from_numpy(np.take_along_axis(l <= LOWEST[dtype], ids.cpu().numpy(), 1)).to("cuda:0")
    assert (w[off] == 0).all() and off[:3].all() and off[3:].sum() == 9
    want = mx.mx_topk_router_bwd(x, ids, w, dw.masked_fill(off, 0.0), score, renormalize)
    assert (want[x <= LOWEST[dtype]] == 0).all() and want[3:, :5].any()
    for bad in (float("nan"), float("inf"), -float("inf")):
        got = mx.mx_topk_router_bwd(x, ids, w, dw.masked_fill(off, bad), score, renormalize)
        assert torch.equal(got, want), bad
    # a gradient that is not finite where it counts stays in its token's experts
    dw[4, 0] = float("nan")
    got = mx.mx_topk_router_bwd(x, ids, w, dw, score, renormalize)
    assert torch.isnan(got[4, ids[4, 0]]) and (got[4, 5:] == 0).all() and torch.equal(got[5:], want[5:])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_logits_of_a_slice_of_tokens(dtype):
    """logits[t0:]: rows of any expert count, wherever they start, and a gradient written there."""
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    for E in (5, 20, 30, 37, 60, 130, 260, 1022):
        whole = _dev(_logits(np.random.default_rng(E), 9, E, dtype), dtype)
        dw = torch.randn((9, 3), device="cuda:0")
        for score, renormalize in (("softmax", False), ("sigmoid", True)):
            ids, w = mx.mx_topk_router_fwd(whole, 3, score, renormalize=renormalize)
            dl = mx.mx_topk_router_bwd(whole, ids, w, dw, score, renormalize)
            for t0 in (1, 2, 3, 7):
                got = mx.mx_topk_router_fwd(whole[t0:], 3, score, renormalize=renormalize)
                assert torch.equal(got[0], ids[t0:]) and torch.equal(got[1], w[t0:])
                out = torch.zeros_like(whole)
                mx.mx_topk_router_bwd(whole[t0:], *got, dw[t0:], score, renormalize, dlogits=out[t0:])
                assert torch.equal(out[t0:], dl[t0:]) and not out[:t0].any()
                leaf = whole[t0:].detach().requires_grad_()
                again, w2 = mx.mx_topk_router(leaf, 3, score, renormalize=renormalize)
                assert torch.equal(again, ids[t0:]) and torch.equal(torch.autograd.grad(w2, leaf, dw[t0:])[0], dl[t0:])
