"""NaN among the logits: every row that holds one has NaN log probabilities, entropy, statistics and
gradient, no alternatives, and the NONFINITE flag -- also where the NaN stands among masked values, alone
or throughout, whatever tile of the row it is in and however the row is split."""

import numpy as np
import pytest
import torch

from speculative_decoding_04_b200 import dspark as D
from tests.parity import dev, host
from tests.test_gpu_logprobs import as64, check, grad_check, strided

pytestmark = pytest.mark.gpu

INF = float("inf")


def nan_rows(V, rng):
    """Rows [K, V] and which of them hold a NaN."""
    fine = rng.normal(0, 2, V)
    rows, bad = [], []

    def add(l, is_bad):
        rows.append(np.array(l, dtype=np.float64))
        bad.append(is_bad)

    def with_nan(l, at):
        l = np.array(l, dtype=np.float64)
        l[at] = np.nan
        return l

    masked = np.full(V, -INF)
    add(fine, False)
    add(masked, False)
    add(np.full(V, np.nan), True)                          # what a broken hidden state gives
    for at in sorted({0, V // 2, V - 1}):                  # alone among masked values: head, middle, tail
        add(with_nan(masked, at), True)
    for at in sorted({0, V // 2, V - 1}):                  # among finite values
        add(with_nan(fine, at), True)
    if V > 1:
        for cut in sorted({1, max(1, V // 3), max(1, V // 2), max(1, V - 600), V - 1}):
            lead, tail = fine.copy(), fine.copy()
            lead[:cut] = -INF                              # masked up to `cut`: the NaN comes first or last of it
            add(lead, False)
            add(with_nan(lead, 0), True)
            add(with_nan(lead, cut - 1), True)
            tail[cut:] = -INF                              # and masked from there on
            add(tail, False)
            add(with_nan(tail, V - 1), True)
            add(with_nan(tail, cut), True)
            lead = lead.copy()
            lead[:cut] = np.nan                            # NaN throughout the leading part
            add(lead, True)
    if V > 1200:                                           # one finite value, in another tile than the NaN
        one = masked.copy()
        one[V - 700] = 1.0
        add(one, False)
        add(with_nan(one, 3), True)
        add(with_nan(one, V - 1), True)
    return np.stack(rows), np.array(bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 9, 300, 511, 1025, 5003, 20011])
def test_rows_with_nan(dtype, V):
    rng = np.random.default_rng(V)
    l, bad = nan_rows(V, rng)
    N = len(bad)
    tok = rng.integers(0, V, N).astype(np.int32)
    for ld, off, top in ((V, 0, 0), (V + 1, 1, 5), (V + 3, 3, 32)):
        t = strided(l, dtype, ld, off)
        flags = torch.zeros(N, dtype=torch.int32, device="cuda")
        got = D.token_logprobs(t, dev(tok), 0.9, top=top, flags=flags)
        assert np.array_equal(np.isnan(host(got[0])), bad)
        assert host(flags).tolist() == [D.FLAG_NONFINITE if b else 0 for b in bad]
        check(as64(t), tok, 0.9, top, got)
        gl, gh = rng.normal(size=N).astype(np.float32), rng.normal(size=N).astype(np.float32)
        g = D.token_logprobs_backward(t, dev(tok), 0.9, got[4], got[1], dev(gl), dev(gh))
        assert np.array_equal(np.isnan(as64(g)).all(-1), bad) and np.array_equal(np.isnan(as64(g)).any(-1), bad)
        grad_check(t, tok, 0.9, gl, gh, None, None, g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_with_nan_split_over_a_cluster(dtype):
    """One row a call: a cluster of CTAs has it, and each has masked tiles of its own."""
    rng = np.random.default_rng(1)
    V = 151936
    l, bad = nan_rows(V, rng)
    tok = np.array([V // 5], dtype=np.int32)
    for row, b in zip(l, bad):
        t = strided(row[None], dtype, V, 1)
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = D.token_logprobs(t, dev(tok), 1.0, top=4, flags=flags)
        assert bool(torch.isnan(got[0][0])) == b and int(flags[0]) == (D.FLAG_NONFINITE if b else 0)
        check(as64(t), tok, 1.0, 4, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_rows_with_nan(dtype):
    """As many rows as leave one CTA of few warps to each."""
    rng = np.random.default_rng(2)
    V = 7001
    l, bad = nan_rows(V, rng)
    l, bad = np.tile(l, (20, 1)), np.tile(bad, 20)
    t = strided(l, dtype, V + 1, 3)
    tok = rng.integers(0, V, len(bad)).astype(np.int32)
    flags = torch.zeros(len(bad), dtype=torch.int32, device="cuda")
    logp, ent, ti, tl, st = (host(x) for x in D.token_logprobs(t, dev(tok), 1.0, top=3, flags=flags))
    assert np.array_equal(host(flags) == D.FLAG_NONFINITE, bad) and not host(flags)[~bad].any()
    for x in (logp, ent, st[:, 0], st[:, 1]):
        assert np.array_equal(np.isnan(x), bad)
    assert np.array_equal(np.isnan(tl).all(-1), bad) and np.all(ti[bad] == -1)


@pytest.mark.parametrize("M", [5, 200])   # both forms of the product
def test_a_nan_hidden_state_reaches_the_flags(M):
    """Hidden states -> norm -> head -> log probabilities -> gradient: a NaN or an infinity in one token's
    hidden state marks that token and no other."""
    rng = np.random.default_rng(3)
    d, V = 256, 4000
    x = rng.normal(size=(M, d))
    x[1, 17], x[3, d - 1] = np.nan, np.inf
    bad = np.isin(np.arange(M), (1, 3))
    w, ws = D.quantize_q8(dev(rng.normal(size=(V, d)).astype(np.float32)))
    q, s, _ = D.rmsnorm_q8(dev(x.astype(np.float32)).bfloat16(), None, 1e-6)
    assert np.array_equal(np.isnan(host(s)), bad)
    logits = D.matmul_q8(q, s, w, ws)
    assert np.array_equal(np.isnan(host(logits)).all(-1), bad) and np.array_equal(np.isnan(host(logits)).any(-1), bad)
    tok = rng.integers(0, V, M).astype(np.int32)
    flags = torch.zeros(M, dtype=torch.int32, device="cuda")
    got = D.token_logprobs(logits, dev(tok), 1.0, top=2, flags=flags)
    assert host(flags).tolist() == [D.FLAG_NONFINITE if b else 0 for b in bad]
    check(as64(logits), tok, 1.0, 2, got)
    gl = np.ones(M, dtype=np.float32)
    g = D.token_logprobs_backward(logits, dev(tok), 1.0, got[4], got[1], dev(gl))
    grad_check(logits, tok, 1.0, gl, None, None, None, g, "f32")
    assert np.array_equal(np.isnan(host(g)).all(-1), bad)

