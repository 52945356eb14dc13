"""The oracle of what surrounds the experts' products, on the CPU: its gradients
against differences, its choice of experts by hand, its code bounds."""

import numpy as np
import pytest

import oracle
from oracle import around

LOWEST = float(np.finfo(np.float32).min)


def test_choice_by_hand():
    l = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, 0.0]])
    ids, w = around.router(l, LOWEST, 3, renormalize=False)
    assert ids.tolist() == [[1, 2, 4]]                      # equal logits: the lower index first
    e = np.exp(l[0] - 3)
    assert np.allclose(w, e[[1, 2, 4]] / e.sum(), rtol=1e-14)
    # masked experts come last, by index
    ids, w = around.router(np.array([[-np.inf, 1.0, LOWEST, 2.0]]), LOWEST, 4)
    assert ids.tolist() == [[3, 1, 0, 2]] and w[0, 2:].tolist() == [0, 0]
    # a bias moves the choice and not the weights
    ids, w = around.router(np.array([[0.0, 1.0, 2.0]]), LOWEST, 1, "sigmoid", bias=[1.0, 0, 0], renormalize=False)
    assert ids.tolist() == [[0]] and w[0, 0] == 0.5
    # groups: [1, 0] with 1 against [.9, .9] with 1.8 by two, 1 against .9 by one
    l = np.log(np.array([[1.0, 1e-9, .9, .9]]))
    one, _ = around.router(l, LOWEST, 1, "sigmoid", groups=2, topk_groups=1, group_score="max")
    two, _ = around.router(l, LOWEST, 1, "sigmoid", groups=2, topk_groups=1, group_score="top2")
    assert one.tolist() == [[0]] and two.tolist() == [[2]]
    # nothing but masked experts
    ids, w = around.router(np.full((1, 4), -np.inf), LOWEST, 2, groups=2, topk_groups=1, group_score="top2")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0, 0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("k", [1, 3, 7])
def test_router_gradient_against_differences(score, renormalize, k):
    rng = np.random.default_rng(k)
    l = rng.normal(size=(4, 7))
    ids, w = around.router(l, LOWEST, k, score, renormalize=renormalize, scale=2.5)
    dw = rng.normal(size=(4, k))
    dl, _ = around.router_grad(l, LOWEST, ids, dw, score, renormalize, 2.5)
    for t in range(4):
        assert np.allclose(around.router_weights(l[t], ids[t], score, renormalize, 2.5), w[t], rtol=1e-13)
        for e in range(7):
            h = np.zeros(7)
            h[e] = 1e-5
            f = [around.router_weights(l[t] + x, ids[t], score, renormalize, 2.5) @ dw[t] for x in (h, -h)]
            # central differences: h^2/6 of a third derivative below 10, and 1e-16 / h of rounding
            assert abs((f[0] - f[1]) / 2e-5 - dl[t, e]) < 1e-9


def test_activation_gradient_against_differences():
    rng = np.random.default_rng(1)
    g, u, dh = rng.normal(size=(3, 200)) * np.array([[4.0], [1], [1]])
    dg, du, _ = around.swiglu_grad(dh, g, u)
    h = 1e-5
    assert np.abs(dh * (around.swiglu(g + h, u) - around.swiglu(g - h, u)) / (2 * h) - dg).max() < 1e-8
    assert np.abs(dh * (around.swiglu(g, u + h) - around.swiglu(g, u - h)) / (2 * h) - du).max() < 1e-8


def test_codes_reached():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(8, 128))
    q, s = oracle.quantize_blocks(x.reshape(8, 4, 32))
    q = q.reshape(8, 128)
    assert around.codes_reached(q, s, x, np.zeros_like(x)).all()
    far = q.copy()
    far[3, 5] ^= 1                                    # a neighbouring code
    ok = around.codes_reached(far, s, x, np.zeros_like(x))
    assert not ok[3, 5] and ok.sum() == ok.size - 1
    assert around.codes_reached(far, s, x, 0.2 * np.abs(x)).all()
    s2 = s.copy()
    s2[1, 2] += 1
    assert not around.codes_reached(q, s2, x, np.zeros_like(x))[1, 64:96].any()
