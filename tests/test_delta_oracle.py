"""Pins of the fp64 oracle of the gated delta rule and of rms norm, on the CPU:
closed forms, the product of transition matrices, and differences."""
import numpy as np
import pytest
import torch

import oracle


def problem(seed, T, B, H, Hk, Dk, Dv):
    r = np.random.default_rng(seed)
    p = {"q": r.normal(size=(T, B, Hk, Dk)), "k": r.normal(size=(T, B, Hk, Dk)), "v": r.normal(size=(T, B, H, Dv)),
         "log_decay": -np.exp(r.normal(size=(T, B, H)) - 1), "beta": r.uniform(size=(T, B, H))}
    p["k"] /= np.sqrt(np.square(p["k"]).sum(-1, keepdims=True))
    return p, r.normal(size=(B, H, Dk, Dv)), r.normal(size=(T, B, H, Dv)), r.normal(size=(B, H, Dk, Dv))


def test_one_token_is_the_formula():
    p, S0, _, _ = problem(0, 1, 1, 1, 1, 3, 2)
    o, S, _ = oracle.gated_delta_rule(**p, scale=0.5, S0=S0)
    k, v, a, b = p["k"][0, 0, 0], p["v"][0, 0, 0], np.exp(p["log_decay"][0, 0, 0]), p["beta"][0, 0, 0]
    want = a * (np.eye(3) - b * np.outer(k, k)) @ S0[0, 0] + b * np.outer(k, v)
    np.testing.assert_allclose(S[0, 0], want, rtol=1e-14, atol=1e-14)
    np.testing.assert_allclose(o[0, 0, 0], 0.5 * want.T @ p["q"][0, 0, 0], rtol=1e-14, atol=1e-14)


def test_final_state_is_the_product_of_transitions():
    p, S0, _, _ = problem(1, 9, 2, 4, 2, 5, 3)
    _, S, _ = oracle.gated_delta_rule(**p, S0=S0)
    for b in range(2):
        for h in range(4):
            M, N = np.eye(5), np.zeros((5, 3))
            for t in range(9):
                k = p["k"][t, b, h // 2]
                A = np.exp(p["log_decay"][t, b, h]) * (np.eye(5) - p["beta"][t, b, h] * np.outer(k, k))
                M, N = A @ M, A @ N + p["beta"][t, b, h] * np.outer(k, p["v"][t, b, h])
            np.testing.assert_allclose(S[b, h], M @ S0[b, h] + N, rtol=1e-12, atol=1e-13)


def test_full_correction_answers_with_the_value():
    """beta = 1, unit keys: a key that was just written finds its value, and
    orthogonal keys do not disturb each other."""
    k = np.eye(4)[[0, 1, 0, 2]][:, None, None]
    v = np.arange(8.0).reshape(4, 1, 1, 2)
    o, S, _ = oracle.gated_delta_rule(k, k, v, None, np.ones((4, 1, 1)), scale=1.0)
    np.testing.assert_allclose(o, v, atol=1e-15)
    np.testing.assert_allclose(S[0, 0], [[4, 5], [2, 3], [6, 7], [0, 0]], atol=1e-15)


def test_without_correction_it_is_linear_attention():
    """Orthogonal keys with beta = 1 find nothing: S sums k v^T with the decays."""
    r = np.random.default_rng(2)
    k = np.eye(6)[:, None, None]
    q, v = r.normal(size=(6, 1, 1, 6)), r.normal(size=(6, 1, 1, 3))
    o, S, _ = oracle.gated_delta_rule(q, k, v, np.full((6, 1, 1), -0.3), np.ones((6, 1, 1)))
    want, wantS = oracle.linear_attention(q, k, v, [-0.3])
    np.testing.assert_allclose(o, want, rtol=1e-13, atol=1e-14)
    np.testing.assert_allclose(S, wantS, rtol=1e-13, atol=1e-14)


@pytest.mark.parametrize("lengths", [None, [4, 0]])
def test_gradients_are_the_differences(lengths):
    p, S0, do, dS1 = problem(3, 6, 2, 4, 2, 4, 3)
    grads, _ = oracle.gated_delta_rule_backward(**p, do=do, scale=0.4, S0=S0, dS1=dS1, lengths=lengths)

    def loss(p, S0):
        o, S, _ = oracle.gated_delta_rule(**p, scale=0.4, S0=S0, lengths=lengths)
        return (o * do).sum() + (S * dS1).sum()

    r = np.random.default_rng(4)
    for name, g in zip(("q", "k", "v", "log_decay", "beta", "S0"), grads):
        at = S0 if name == "S0" else p[name]
        d, eps = r.normal(size=at.shape), 1e-5
        up, down = (loss(p, S0 + s * d) if name == "S0" else loss({**p, name: at + s * d}, S0) for s in (eps, -eps))
        assert abs((up - down) / (2 * eps) - (g * d).sum()) <= 1e-7 * (1 + np.abs(g * d).sum()), name


def test_rms_norm_and_its_differences():
    r = np.random.default_rng(5)
    x, res, w, dy, ds = (r.normal(size=s) for s in ((3, 7), (3, 7), (7,), (3, 7), (3, 7)))
    y, rstd, s = oracle.rms_norm(x, w, 1e-3, res)
    np.testing.assert_allclose(s, x + res)
    np.testing.assert_allclose(y, (x + res) / np.sqrt(((x + res) ** 2).mean(1) + 1e-3)[:, None] * w, rtol=1e-14)
    dx, dw = oracle.rms_norm_backward(dy, s, rstd, w, ds)
    d, eps = r.normal(size=x.shape), 1e-6
    loss = lambda x, w: (oracle.rms_norm(x, w, 1e-3, res)[0] * dy).sum() + ((x + res) * ds).sum()
    assert abs((loss(x + eps * d, w) - loss(x - eps * d, w)) / (2 * eps) - (dx * d).sum()) < 1e-7
    e = r.normal(size=7)
    assert abs((loss(x, w + eps * e) - loss(x, w - eps * e)) / (2 * eps) - (dw * e).sum()) < 1e-7


def test_e4m3_values_are_torch_s():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.e4m3_values(), codes)
