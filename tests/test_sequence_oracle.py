"""Pins of the linear-attention and layer-norm oracle (CPU): the sums over pairs
of tokens, closed forms, and gradients against differences."""
import numpy as np
import pytest

import oracle


def problem(T=7, B=2, H=4, Hkv=2, Dk=3, Dv=5, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((T, B, H, Dk)), k=r.standard_normal((T, B, Hkv, Dk)),
                v=r.standard_normal((T, B, Hkv, Dv)), log_decay=-r.uniform(0.0, 1.0, H)), \
        r.standard_normal((B, H, Dk, Dv))


def test_matches_the_sum_over_pairs_of_tokens():
    p, S0 = problem()
    T, B, H, Dk = p["q"].shape
    o, S = oracle.linear_attention(**p, scale=0.7, S0=S0)
    d = np.exp(p["log_decay"])
    for t in range(T):
        for b in range(B):
            for h in range(H):
                want = d[h] ** (t + 1) * (p["q"][t, b, h] @ S0[b, h])
                for j in range(t + 1):
                    want = want + d[h] ** (t - j) * (p["q"][t, b, h] @ p["k"][j, b, h // 2]) * p["v"][j, b, h // 2]
                np.testing.assert_allclose(o[t, b, h], 0.7 * want, rtol=1e-12, atol=1e-12)
    want = d[:, None, None] ** T * S0[0] + sum(
        d[:, None, None] ** (T - 1 - j) * np.repeat(p["k"][j, 0, :, :, None] * p["v"][j, 0, :, None, :], 2, axis=0)
        for j in range(T))
    np.testing.assert_allclose(S[0], want, rtol=1e-12, atol=1e-12)


def test_no_decay_is_a_running_sum_and_total_decay_one_token():
    p, _ = problem(H=2, Hkv=2)
    p["log_decay"] = np.array([0.0, -np.inf])
    o, S = oracle.linear_attention(**p, scale=1.0)
    kv = np.cumsum(p["k"][:, :, 0, :, None] * p["v"][:, :, 0, None, :], axis=0)
    np.testing.assert_allclose(o[:, :, 0], np.einsum("tbd,tbde->tbe", p["q"][:, :, 0], kv), rtol=1e-12, atol=1e-12)
    one = np.sum(p["q"][:, :, 1] * p["k"][:, :, 1], axis=-1, keepdims=True) * p["v"][:, :, 1]
    np.testing.assert_allclose(o[:, :, 1], one, rtol=1e-12, atol=1e-12)


def test_two_calls_with_a_carried_state_are_one():
    p, S0 = problem(T=9)
    o, S = oracle.linear_attention(**p, S0=S0)
    first = {n: (x[:4] if n != "log_decay" else x) for n, x in p.items()}
    last = {n: (x[4:] if n != "log_decay" else x) for n, x in p.items()}
    o1, S1 = oracle.linear_attention(**first, S0=S0)
    o2, S2 = oracle.linear_attention(**last, S0=S1)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, [0, 5]])
def test_gradients_match_differences(lengths):
    p, S0 = problem(T=6)
    r = np.random.default_rng(1)
    do = r.standard_normal((6, 2, 4, 5))
    dS1 = r.standard_normal(S0.shape)

    def loss(p, S0):
        o, S = oracle.linear_attention(**p, scale=0.6, S0=S0, lengths=lengths)
        return np.sum(o * do) + np.sum(S * dS1)

    grads = oracle.linear_attention_backward(**p, do=do, scale=0.6, S0=S0, dS1=dS1, lengths=lengths)
    for name, g in zip(("q", "k", "v", "S0"), grads):
        x = S0 if name == "S0" else p[name]
        for i in r.integers(0, x.size, 12):
            step = np.zeros(x.size)
            step[i] = 1e-5
            step = step.reshape(x.shape)
            hi, lo = (loss(p, S0 + s) if name == "S0" else loss({**p, name: x + s}, S0) for s in (step, -step))
            assert abs((hi - lo) / 2e-5 - g.reshape(-1)[i]) < 1e-7, (name, i)


def test_layer_norm_closed_forms_and_differences():
    r = np.random.default_rng(2)
    x, w, b, dy = r.standard_normal((5, 9)), r.standard_normal(9), r.standard_normal(9), r.standard_normal((5, 9))
    y, mean, rstd = oracle.layer_norm(x, w, b)
    n = (y - b) / w
    np.testing.assert_allclose(n.mean(1), 0, atol=1e-12)
    np.testing.assert_allclose(n.var(1), 1 / (1 + 1e-5 / x.var(1)), rtol=1e-12)
    np.testing.assert_allclose(oracle.layer_norm(np.full((2, 4), 3.0), w[:4], b[:4])[0], np.stack([b[:4]] * 2))
    dx, dw, db = oracle.layer_norm_backward(dy, x, w)

    def loss(x, w, b):
        return np.sum(oracle.layer_norm(x, w, b)[0] * dy)

    for which, g in ((0, dx), (1, dw), (2, db)):
        for i in range(g.size):
            args = [[x, w, b], [x, w, b]]
            for sign, a in zip((1, -1), args):
                step = np.zeros(g.size)
                step[i] = sign * 1e-5
                a[which] = a[which] + step.reshape(g.shape)
            assert abs((loss(*args[0]) - loss(*args[1])) / 2e-5 - g.reshape(-1)[i]) < 1e-7
