"""Pins of the operators' oracle: closed forms, library routines and differences (CPU)."""

import numpy as np
import pytest
from scipy.special import log_softmax
from scipy.stats import entropy as scipy_entropy

import oracle as O


def test_logprobs_closed_forms():
    V = 7
    r = O.token_logprobs(np.zeros((1, V)), [3], 0.5, top=3)   # uniform at any temperature
    assert np.isclose(r["logp"][0], -np.log(V)) and np.isclose(r["entropy"][0], np.log(V))
    assert r["top_idx"][0].tolist() == [0, 1, 2]              # ties: lowest index
    assert np.allclose(r["stats"][0], [0.0, np.log(V)])
    r = O.token_logprobs(np.array([[0.0, np.log(3.0)]]), [0], 1.0, top=4)
    assert np.allclose(r["logp"], np.log(0.25)) and r["top_idx"][0].tolist() == [1, 0, -1, -1]
    r = O.token_logprobs(np.array([[-np.inf, 2.0, -np.inf]]), [0], 1.0, top=2)
    assert r["logp"][0] == -np.inf and r["entropy"][0] == 0 and r["top_idx"][0].tolist() == [1, -1]
    r = O.token_logprobs(np.full((1, 3), -np.inf), [1], 1.0, top=1)
    assert r["logp"][0] == -np.inf and r["entropy"][0] == 0 and np.all(r["stats"] == -np.inf)


@pytest.mark.parametrize("T", [0.5, 1.0, 1.7])
def test_logprobs_match_library_routines(T):
    rng = np.random.default_rng(1)
    l = rng.normal(0, 3, (6, 200))
    t = rng.integers(0, 200, 6)
    r = O.token_logprobs(l, t, T, top=5)
    lp = log_softmax(l / T, axis=-1)
    assert np.allclose(r["logp"], lp[np.arange(6), t], atol=1e-13)
    assert np.allclose(r["entropy"], scipy_entropy(np.exp(lp), axis=-1), atol=1e-13)
    assert np.allclose(r["top_logp"], -np.sort(-lp, axis=-1)[:, :5], atol=1e-13)
    rows = np.array([3, 3, 9])
    q = O.token_logprobs(l, [1, 2, 0], T, rows=rows)
    assert np.allclose(q["logp"][:2], lp[3, [1, 2]]) and np.isnan(q["logp"][2])


def test_logprobs_gradient_by_differences():
    rng = np.random.default_rng(2)
    N, V, T, k = 4, 12, 0.8, 3
    l = rng.normal(0, 2, (N, V))
    t = np.array([5, 0, -1, 11])
    gl, gh, gt = rng.normal(size=N), rng.normal(size=N), rng.normal(size=(N, k))
    idx = O.token_logprobs(l, t, T, top=k)["top_idx"]
    live = t >= 0

    def f(x):
        lp = log_softmax(x / T, axis=-1)
        H = -(np.exp(lp) * lp).sum(-1)
        s = (gl * lp[np.arange(N), np.maximum(t, 0)] + gh * H)[live].sum()
        return s + (gt * np.take_along_axis(lp, np.maximum(idx, 0), 1))[live].sum()

    g = O.token_logprobs_grad(l, t, T, gl, gh, idx, gt)
    num = np.zeros_like(l)
    for i in np.ndindex(*l.shape):
        e = np.zeros_like(l)
        e[i] = 1e-5
        num[i] = (f(l + e) - f(l - e)) / 2e-5
    assert np.allclose(g, num, atol=1e-8) and np.all(g[2] == 0)


def test_quantisation_closed_forms():
    x = np.array([[127.0, -63.5, 1.0, 0.0], [0.0, 0.0, 0.0, 0.0], [1.0, np.inf, 0, 0], [np.nan, 1, 2, 3]])
    q, s = O.quantize_q8(x)
    assert q[0].tolist() == [127, -64, 1, 0] and s[0] == 1.0      # -63.5 rounds to even
    assert not q[1:].any() and s[1] == 0 and np.isnan(s[2:]).all()
    h = np.array([[3.0, -4.0]])                                   # root mean square 5 / sqrt(2)
    q, s = O.rmsnorm_q8(h, np.array([1.0, 0.5]), 0.0)
    assert q[0].tolist() == [127, -85]                            # v = (3, -2)
    assert np.isclose(s[0], 3 / (5 / np.sqrt(2)) / 127)


def test_quantisation_error_is_half_a_step():
    rng = np.random.default_rng(3)
    h, g = rng.normal(size=(20, 300)), 1 + 0.1 * rng.normal(size=300)
    q, s = O.rmsnorm_q8(h, g, 1e-6)
    h32, g32 = h.astype(np.float32).astype(np.float64), g.astype(np.float32).astype(np.float64)
    y = h32 * g32 / np.sqrt((h32 ** 2).mean(1, keepdims=True) + 1e-6)
    assert np.all(np.abs(q * s[:, None] - y) <= s[:, None] * (0.5 + 1e-4)) and np.abs(q).max() == 127


def test_matmul_q8_against_integers():
    rng = np.random.default_rng(4)
    q, w = rng.integers(-128, 128, (5, 64)), rng.integers(-128, 128, (7, 64))
    a, b = rng.random(5), rng.random(7)
    want = [[a[i] * b[j] * sum(int(x) * int(y) for x, y in zip(q[i], w[j])) for j in range(7)] for i in range(5)]
    assert np.allclose(O.matmul_q8(q, a, w, b), want, rtol=1e-15)
