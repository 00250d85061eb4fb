"""Log probabilities of given tokens (entropy, top alternatives) and their gradient on the GPU
against the float64 oracle.

Tolerances.  u = 2^-24 is half an fp32 step.  The kernel forms d = (l - R) log2(e)/T in fp32 (three
roundings: 3u relative), 2^d with ex2.approx (2^-22 = 4u relative) and sums per lane in fp32: a lane
adds at most `terms` values to each accumulator, so a sum of non-negative terms is off by at most
(terms + 6) u relative (6: the packed halves and the warp's five additions); everything after is fp64.
An error of d by 3u|d| moves a term by 3u|d| ln 2 of itself, |d| in bits.  With D = sum p |d ln 2|
(nats from the reference, which is the running maximum and so at or above each term):
  ln S:      err_S = u (terms + 10 + 3 D)
  logp:      err_S + u |logp|                              (one rounding to fp32)
  entropy:   H = ln S - E/S with E <= D S:  err_S + D (2 (terms + 10) u) + 3 u (D + D2), plus u H;
             D2 = sum p (d ln 2)^2
The sums are written for the final maximum; a reference that grew on the way adds one more rounding
for each growth (at most a few dozen for shuffled rows, one a tile for ascending ones), counted in
`terms` as one per tile of the lane's warp.
"""


import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_04_b200 import dspark as D
from speculative_decoding_04_b200 import inputs
from tests.parity import dev, draw_tokens, host, pm

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def strided(a, dtype, ld=None, offset=0):
    """[N, V] on the GPU with row stride ld, its first element `offset` elements into an allocation;
    what lies between the rows is NaN, so that a read outside a row shows."""
    N, V = a.shape
    ld = V if ld is None else ld
    flat = torch.full((offset + N * ld + 64,), float("nan"), dtype=DT[dtype], device="cuda")
    t = flat[offset:offset + N * ld].view(N, ld)[:, :V]
    t.copy_(torch.from_numpy(np.array(a)).to(DT[dtype]).cuda())
    return t


def as64(t):
    return t.double().cpu().numpy()


def check(logits64, tokens, T, top, got, rows=None):
    logp, ent, ti, tl, stats = (None if x is None else host(x) for x in got)
    r = O.token_logprobs(logits64, tokens, T, top, rows)
    V = logits64.shape[-1]
    tiles = -(-V // 512) + 1
    per_warp = -(-tiles // 16)
    terms = per_warp * 16 + per_warp   # values a lane adds to one accumulator, plus one rescale a tile
    logp, ent, stats = logp.reshape(-1), ent.reshape(-1), stats.reshape(-1, 2)
    for n, p in enumerate(r["p"]):
        assert np.array_equal(np.isnan(logp[n]), np.isnan(r["logp"][n])), n
        if p is None:   # padding, unreadable, or fully masked
            for a, b in ((logp[n], r["logp"][n]), (ent[n], r["entropy"][n])):
                assert np.isnan(a) if np.isnan(b) else a == b, (n, a, b)
            assert np.array_equal(stats[n], r["stats"][n].astype(np.float32), equal_nan=True)
            continue
        m, logS = r["stats"][n]
        d = np.where(p > 0, -(np.log(np.maximum(p, 1e-320)) + logS), 0.0)
        Dn, D2 = float((p * d).sum()), float((p * d * d).sum())
        eS = U32 * (terms + 10 + 3 * Dn)
        if np.isfinite(r["logp"][n]):
            assert abs(logp[n] - r["logp"][n]) <= eS + U32 * abs(r["logp"][n]) + 1e-30, n
        elif not np.isnan(r["logp"][n]):
            assert logp[n] == r["logp"][n]
        eH = eS + Dn * 2 * (terms + 10) * U32 + 3 * U32 * (Dn + D2) + U32 * r["entropy"][n]
        assert abs(ent[n] - r["entropy"][n]) <= eH, (n, ent[n], r["entropy"][n])
        assert stats[n, 0] == np.float32(m)
        assert abs(stats[n, 1] - logS) <= eS + U32 * abs(logS)
    if top:
        ti, tl = ti.reshape(-1, top), tl.reshape(-1, top)
        assert np.array_equal(ti, r["top_idx"])
        fin = np.isfinite(r["top_logp"])
        assert np.array_equal(tl[~fin], r["top_logp"][~fin].astype(np.float32), equal_nan=True)
        bound = U32 * (terms + 10 + 3 * np.log(V) + 3 * 32 + np.abs(r["top_logp"][fin]))
        assert np.all(np.abs(tl[fin] - r["top_logp"][fin]) <= bound)
    return r


def rows_of(rng, N, V):
    prior = -1.1 * np.log(rng.permutation(V) + 1.0)
    return prior + rng.normal(0, 1.5, (N, V))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 511, 512, 513, 1025, 4099, 33000])
def test_logprobs_sizes(dtype, V):
    rng = np.random.default_rng(V)
    N = 5
    for ld, off, top, T in ((V, 0, 5, 1.0), (V + 1, 1, 1, 0.7), (V + 3, 3, 32, 1.6), (V + 64, 2, 0, 1.0)):
        t = strided(rows_of(rng, N, V), dtype, ld, off)
        tok = rng.integers(0, V, N).astype(np.int32)
        got = D.token_logprobs(t, dev(tok), T, top=top)
        check(as64(t), tok, T, top, got)


@pytest.mark.parametrize("N,V,dtype", [(1, 151936, "f32"), (3, 151936, "bf16"), (40, 50001, "f16"),
                                       (2, 262144, "f16"), (1, 1_000_003, "f32")])
def test_logprobs_few_rows_split_over_a_cluster(N, V, dtype):
    rng = np.random.default_rng(N + V)
    t = strided(rows_of(rng, N, V), dtype)
    tok = rng.integers(0, V, N).astype(np.int32)
    flags = torch.zeros(N, dtype=torch.int32, device="cuda")
    check(as64(t), tok, 0.9, 20, D.token_logprobs(t, dev(tok), 0.9, top=20, flags=flags))
    assert not host(flags).any()


def test_logprobs_many_rows_one_cta_each():
    rng = np.random.default_rng(5)
    N, V = 700, 3001
    t = strided(rows_of(rng, N, V), "bf16", V + 7)
    tok = rng.integers(-1, V, N).astype(np.int32)
    check(as64(t), tok, 1.0, 3, D.token_logprobs(t, dev(tok), 1.0, top=3))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_logprobs_masks(dtype):
    rng = np.random.default_rng(11)
    N, V = 12, 5003
    low = float(torch.finfo(DT[dtype]).min)
    l = rows_of(rng, N, V)
    l[0] = -np.inf                                  # nothing left
    l[1, rng.random(V) < 0.9] = -np.inf
    l[2] = -np.inf
    l[2, 4711] = 3.0                                # one token left
    l[3] = low                                      # the type's lowest value throughout: uniform
    l[4, ::2] = low
    l[5, :3000] = -np.inf                           # whole tiles masked before the first logit
    l[6, 77] = np.nan
    l[7, 5002] = np.inf
    l[8, 10] = -np.inf                              # the given token is masked
    l[9] = np.where(np.arange(V) == 0, 1.0, -np.inf)
    l[10] = np.where(np.arange(V) == V - 1, 1.0, -np.inf)
    tok = np.array([5, 7, 4711, 12, 1, 4000, 3, 9, 10, 1, V - 1, 8], dtype=np.int32)
    t = strided(l, dtype, V + 1)
    flags = torch.zeros(N, dtype=torch.int32, device="cuda")
    for top in (0, 4, 32):
        flags.zero_()
        check(as64(t), tok, 1.0, top, D.token_logprobs(t, dev(tok), 1.0, top=top, flags=flags))
        assert host(flags).tolist() == [D.FLAG_NONFINITE if n in (6, 7) else 0 for n in range(N)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 400])
def test_logprobs_ties_and_orders(dtype, N):
    """Constant, ascending, descending and heavily tied rows, -0 against +0, at one CTA and at a cluster per row."""
    V = 40_000
    rng = np.random.default_rng(3)
    kinds = [np.full(V, 1.25), np.arange(V) / 64.0, -np.arange(V) / 64.0, rng.integers(0, 3, V).astype(float),
             np.where(rng.random(V) < 0.5, -0.0, 0.0), np.where(np.arange(V) % 512 == 511, 2.0, 0.0),
             np.repeat(rng.normal(size=V // 8), 8)]
    for k, row in enumerate(kinds):
        l = np.broadcast_to(row, (N, V))
        t = strided(l, dtype)
        tok = np.full(N, 17, dtype=np.int32)
        got = D.token_logprobs(t, dev(tok), 1.0, top=32)
        if N > 1:   # equal rows: equal results, and the first against the oracle
            for x in got:
                assert torch.equal(x, x[:1].expand_as(x)), k
            got, t, tok = tuple(x[:1] for x in got), t[:1], tok[:1]
        check(as64(t), tok, 1.0, 32, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 150])
@pytest.mark.parametrize("top", [1, 20, 32])
def test_logprobs_large_values_in_every_few_tiles(dtype, N, top):
    """Rows whose large values lie in all tiles of 512 but those of every 32nd group onwards (the worst
    spread for a choice by lanes), in one tile of 32 only, and the same value in all tiles."""
    rng = np.random.default_rng(top)
    V = 300_000
    tile = np.arange(V) // 512
    l = rng.normal(0, 1, (N, V)).astype(np.float32)
    l[0] += np.where(tile % 32 < top - 1, 12.0, 0.0)
    for n in range(1, min(N, 4)):
        l[n] += [0.0, np.where(tile % 32 == 5, 12.0, 0.0), np.where(tile % 32 == 31, -30.0, 0.0),
                 np.where(np.arange(V) % 512 == 77, 40.0 - l[n], 0.0)][n]
    t = strided(l, dtype)
    tok = rng.integers(0, V, N).astype(np.int32)
    check(as64(t), tok, 0.9, top, D.token_logprobs(t, dev(tok), 0.9, top=top))


def test_logprobs_extremes_of_magnitude():
    V = 3000
    rng = np.random.default_rng(8)
    l = rng.normal(size=(4, V))
    l[0] *= 1e4
    l[1] = l[1] * 1e-30
    l[2] = 3e38 + l[2]
    l[3, 5], l[3, 6] = 3e38, -3e38
    t = strided(l, "f32")
    tok = np.array([1, 2, 3, 5], dtype=np.int32)
    check(as64(t), tok, 1.0, 3, D.token_logprobs(t, dev(tok), 1.0, top=3))


@pytest.mark.parametrize("dtype,N", [("f32", 1), ("bf16", 3), ("f32", 400)])
@pytest.mark.parametrize("gap", [0.0, 4.0, 10.0, 18.0, 28.0])
def test_logprobs_of_a_dominant_token_keep_their_digits(dtype, N, gap):
    """With p close to 1, -log p and the entropy are about the sum of the other tokens' exponentials, which
    is held apart from the dominant token's 1: its relative error is that of a sum of small terms --
    `terms` additions and 3u |d| for each term's exponent (d below 45 nats here), ex2's and the joins' --
    not u / (1 - p).  The entropy adds its terms' own factors d: twice that."""
    rng = np.random.default_rng(int(gap) + N)
    V = 20_011
    l = rng.normal(0, 1, (N, V))
    tok = rng.integers(0, V, N).astype(np.int32)
    l[np.arange(N), tok] = l.max(-1) + gap
    t = strided(l, dtype)
    logp, ent, _, _, _ = D.token_logprobs(t, dev(tok), 1.0)
    x = as64(t)
    z = x - x[np.arange(N), tok][:, None]
    e = np.exp(z)
    e[np.arange(N), tok] = 0
    S = e.sum(-1)
    rel = U32 * (17 * (-(-V // 512) + 1) + 20 + 3 * 45)   # 17 values a tile at most in one accumulator
    want = np.log1p(S)
    assert np.all(np.abs(host(logp) + want) <= rel * want)
    H = want - (e * z).sum(-1) / (1 + S)
    assert np.all(np.abs(host(ent) - H) <= 2 * rel * H)


def test_logprobs_tokens_and_rows():
    rng = np.random.default_rng(21)
    n_rows, V = 9, 2049
    t = strided(rows_of(rng, n_rows, V), "f32")
    rows = np.array([0, 8, 8, 3, -1, 9, 2 ** 40, 4, 5, 6, 6, 6], dtype=np.int64)
    tok = np.array([1, 2, 2, -1, 3, 4, 5, V, -2, 0, V - 1, 2 ** 31 - 1], dtype=np.int32)
    flags = torch.zeros(12, dtype=torch.int32, device="cuda")
    got = D.token_logprobs(t, dev(tok).view(3, 4), 1.0, top=2, rows=dev(rows).view(3, 4), flags=flags)
    assert got[0].shape == (3, 4) and got[2].shape == (3, 4, 2) and got[4].shape == (3, 4, 2)
    check(as64(t), tok, 1.0, 2, got, rows)
    R, K = D.FLAG_RAGGED_OFFSETS, D.FLAG_TOKEN_RANGE
    assert host(flags).tolist() == [0, 0, 0, 0, R, R, R, K, K, 0, 0, K]


def test_logprobs_offsets_beyond_32_bits():
    V, n_rows = 1 << 20, 2100   # 2.2e9 elements of bf16
    l = torch.zeros((n_rows, V), dtype=torch.bfloat16, device="cuda")
    l[2099, 1_000_000] = 9.0
    l[2098, 3] = 4.0
    tok = torch.tensor([1_000_000, 3, 0], dtype=torch.int32, device="cuda")
    rows = torch.tensor([2099, 2098, 2047], dtype=torch.int64, device="cuda")
    logp, ent, ti, tl, st = D.token_logprobs(l, tok, 1.0, top=1, rows=rows)
    want = [9.0 - np.log(V - 1 + np.exp(9.0)), 4.0 - np.log(V - 1 + np.exp(4.0)), -np.log(V)]
    # a lane adds 64 tiles / (16 warps * 16 CTAs) * 16 values: far below the 1e-5 of 160 steps
    assert np.allclose(host(logp), want, rtol=0, atol=1e-5) and host(ti).ravel().tolist() == [1_000_000, 3, 0]
    full = torch.arange(n_rows, device="cuda", dtype=torch.int32) % 7
    stats = torch.empty((n_rows, 2), device="cuda")
    e = torch.empty(n_rows, device="cuda")
    D.token_logprobs(l, full, 1.0, entropy=e, stats=stats)
    g = D.token_logprobs_backward(l, full, 1.0, stats, e, torch.ones(n_rows, device="cuda"), grad=l)   # in place
    assert g.data_ptr() == l.data_ptr()
    p = np.exp(9.0 - np.log(V - 1 + np.exp(9.0)))
    assert abs(float(g[2099, 1_000_000]) + p) <= p * (2.0 ** -8 + 1e-5)
    assert abs(float(g[2099, 2099 % 7]) - 1.0) <= 2.0 ** -8


# --------------------------------------------------------------------------- backward

def grad_check(t, tok, T, gl, gh, ti, gt, got, dtype):
    """p's relative error: 3 roundings of (l - m)/T - ln S (3u (|lp| + |ln S| + |d|)), the stats' own
    error in ln S (as in check: e_S), ex2's 4u and the products' 4u; one rounding to the dtype."""
    l64 = as64(t)
    V = l64.shape[-1]
    want = O.token_logprobs_grad(l64, tok, T, gl, gh, ti, gt)
    got = as64(got)
    tiles = -(-V // 512) + 1
    per_warp = -(-tiles // 16)
    for n in range(l64.shape[0]):
        if not 0 <= tok[n] < V or not np.isfinite(l64[n].max()):
            assert np.array_equal(got[n], want[n], equal_nan=True), n
            continue
        z = (l64[n] - l64[n].max()) / T
        S = np.log(np.exp(z).sum())
        lp = z - S
        p = np.exp(lp)
        a = np.abs(np.where(np.isfinite(lp), lp, 0.0))
        eS = U32 * (per_warp * 17 + 10 + 3 * np.log(V) + S)
        rel = 3 * U32 * (2 * a + S) + eS + 8 * U32
        H = -(p * np.where(p > 0, lp, 0)).sum()
        G = (0 if gl is None else abs(float(gl[n]))) + (0 if gt is None else np.abs(gt[n]).sum())
        h = 0 if gh is None else abs(float(gh[n]))
        mag = p * (G + h * (a + H)) / T
        # the entropy passed in carries its own error, below 2e-5 at these sizes
        bound = mag * rel + p * h * (2e-5 + eS) / T + 4 * U32 * (np.abs(want[n]) + G / T * (want[n] != 0))
        bound = bound + EPS[dtype] * np.abs(want[n]) * (1 + 1e-3)
        bound += {"f32": 1e-44, "bf16": 1e-40, "f16": 2.0 ** -25}[dtype]   # subnormals of the type
        assert np.all(np.abs(got[n] - want[n]) <= bound), (n, np.max(np.abs(got[n] - want[n]) - bound))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 9, 513, 4096, 4099, 20011])
def test_backward_matches_formula(dtype, V):
    rng = np.random.default_rng(V + 1)
    N = 6
    for ld, off, T, k in ((V, 0, 1.0, 0), (V + 1, 1, 0.7, 3), (V + 5, 3, 1.4, 32)):
        t = strided(rows_of(rng, N, V), dtype, ld, off)
        tok = rng.integers(0, V, N).astype(np.int32)
        tok[1] = -1
        gl, gh = rng.normal(size=N).astype(np.float32), rng.normal(size=N).astype(np.float32)
        logp, ent, ti, tl, st = D.token_logprobs(t, dev(tok), T, top=k)
        gt = rng.normal(size=(N, k)).astype(np.float32) if k else None
        g = D.token_logprobs_backward(t, dev(tok), T, st, ent, dev(gl), dev(gh), top_idx=ti,
                                      g_top=None if gt is None else dev(gt))
        assert g.stride() == t.stride() or N == 1
        grad_check(t, tok, T, gl, gh, None if ti is None else host(ti), gt, g, dtype)
        # a gradient of another alignment, and in place
        g2 = strided(np.zeros((N, V)), dtype, V + 3, 1)
        D.token_logprobs_backward(t, dev(tok), T, st, ent, dev(gl), dev(gh), top_idx=ti,
                                  g_top=None if gt is None else dev(gt), grad=g2)
        assert torch.equal(g, g2)
        D.token_logprobs_backward(t, dev(tok), T, st, ent, dev(gl), dev(gh), top_idx=ti,
                                  g_top=None if gt is None else dev(gt), grad=t)
        assert torch.equal(g, t)


def test_backward_repeated_indices_masks_and_missing_gradients():
    rng = np.random.default_rng(9)
    N, V, T = 7, 9000, 0.9
    l = rows_of(rng, N, V)
    l[0] = -np.inf
    l[1, rng.random(V) < 0.8] = -np.inf
    l[2, 100] = np.nan
    l[5, 8999] = np.inf
    t = strided(l, "f32", V + 2)
    tok = np.array([3, 4, 5, V, 17, 1, 8], dtype=np.int32)
    logp, ent, ti, tl, st = D.token_logprobs(t, dev(tok), T, top=1)
    idx = rng.integers(0, V, (N, 6)).astype(np.int32)
    idx[:, 1] = idx[:, 0]          # the same index twice
    idx[:, 2] = np.maximum(tok, 0)  # the given token among them
    idx[3, 2] = 0
    idx[:, 3] = -1                 # no alternative
    idx[:, 4] = [V, 2 ** 31 - 1, -7, V + 1, -2 ** 31, V, -1]   # outside the vocabulary: no alternatives either
    gl, gt = rng.normal(size=N).astype(np.float32), rng.normal(size=(N, 6)).astype(np.float32)
    g = D.token_logprobs_backward(t, dev(tok), T, st, ent, dev(gl), None, top_idx=dev(idx), g_top=dev(gt))
    grad_check(t, tok, T, gl, None, np.where((idx >= 0) & (idx < V), idx, -1), gt, g, "f32")
    gh = rng.normal(size=N).astype(np.float32)
    g = D.token_logprobs_backward(t, dev(tok), T, st, ent, None, dev(gh))
    grad_check(t, tok, T, None, gh, None, None, g, "f32")


def test_backward_of_the_types_lowest_value():
    """A row of the lowest value throughout is uniform: its statistics keep that (m = lowest, ln S = ln V)."""
    V = 600
    low = torch.finfo(torch.float32).min
    t = torch.full((1, V), low, device="cuda")
    tok = torch.tensor([5], dtype=torch.int32, device="cuda")
    logp, ent, _, _, st = D.token_logprobs(t, tok, 1.0)
    g = D.token_logprobs_backward(t, tok, 1.0, st, ent, torch.ones(1, device="cuda"))
    want = -np.full(V, 1.0 / V)
    want[5] += 1
    assert np.allclose(host(g)[0], want, rtol=64 * U32, atol=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gap", [2.0, 10.0, 25.0])
def test_backward_of_a_dominant_token_keeps_its_digits(dtype, gap):
    """g (1 - p) of a token with p close to 1: 1 - p comes from log p, whose relative error is that of the
    sum of the other tokens' exponentials (as for the forward call), passed on by a factor of at most 1, and
    some 12 roundings follow."""
    rng = np.random.default_rng(int(gap))
    N, V, T = 5, 20_011, 1.0
    l = rng.normal(0, 1, (N, V))
    tok = rng.integers(0, V, N).astype(np.int32)
    l[np.arange(N), tok] = l.max(-1) + gap
    t = strided(l, dtype)
    _, ent, _, _, st = D.token_logprobs(t, dev(tok), T)
    gl = rng.normal(size=N).astype(np.float32)
    g = D.token_logprobs_backward(t, dev(tok), T, st, ent, dev(gl)).double().cpu().numpy()[np.arange(N), tok]
    x = as64(t)
    e = np.exp(x - x[np.arange(N), tok][:, None])
    e[np.arange(N), tok] = 0
    S = e.sum(-1)
    want = gl * S / (1 + S)
    rel = U32 * (17 * (-(-V // 512) + 1) + 20 + 3 * 45 + 12)
    assert np.all(np.abs(g - want) <= (rel + EPS[dtype] * (1 + 1e-3)) * np.abs(want))


def test_backward_by_differences():
    """The gradient against central differences of the forward kernel itself: with h = 2^-3 the
    difference quotient of logp (fp32, error below 2e-5 of 10) is good to 2e-5 * 10 / h and the third
    derivative (below 1 for a log softmax at T = 1) to h^2 / 6."""
    rng = np.random.default_rng(4)
    V, h = 300, 2.0 ** -3
    l = rng.normal(0, 2, V).astype(np.float32)
    cols = rng.integers(0, V, 8)
    tok = torch.full((16,), int(cols[0]), dtype=torch.int32, device="cuda")
    base = np.repeat(l[None], 16, 0)
    for i, c in enumerate(cols):
        base[2 * i, c] += h
        base[2 * i + 1, c] -= h
    lp = host(D.token_logprobs(dev(base), tok, 1.0)[0]).astype(np.float64)
    x = dev(l[None])
    _, ent, _, _, st = D.token_logprobs(x, tok[:1], 1.0)
    g = host(D.token_logprobs_backward(x, tok[:1], 1.0, st, ent, torch.ones(1, device="cuda")))[0]
    num = (lp[0::2] - lp[1::2]) / (2 * h)
    assert np.all(np.abs(g[cols] - num) <= 2e-4 / h + h * h / 6)


# --------------------------------------------------------------------------- use

def test_streams_graphs_and_repeats():
    rng = np.random.default_rng(31)
    N, V = 33, 30011
    t = strided(rows_of(rng, N, V), "bf16", V + 5)
    tok = dev(rng.integers(0, V, N).astype(np.int32))
    gl, gh = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    fwd = D.token_logprobs(t, tok, 1.0, top=7)
    bwd = D.token_logprobs_backward(t, tok, 1.0, fwd[4], fwd[1], gl, gh, top_idx=fwd[2], g_top=fwd[3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f2 = D.token_logprobs(t, tok, 1.0, top=7, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fwd, f2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f3 = D.token_logprobs(t, tok, 1.0, top=7)
        b3 = D.token_logprobs_backward(t, tok, 1.0, f3[4], f3[1], gl, gh, top_idx=f3[2], g_top=f3[3])
    for _ in range(3):
        for x in f3:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(fwd, f3)) and torch.equal(b3, bwd)


def test_nothing_beside_the_outputs_is_written():
    rng = np.random.default_rng(41)
    N, V, k = 4, 1000, 3
    t = strided(rows_of(rng, N, V), "f16", V + 9, 3)
    before = t.clone()
    pad = torch.full((N * V + 64,), 7.0, dtype=torch.float16, device="cuda")
    grad = pad[5:5 + N * V].view(N, V)
    big = torch.full((N * (5 + 2 * k) + 64,), 7.0, device="cuda")
    logp, ent = big[2:2 + N], big[2 + N:2 + 2 * N]
    tok = dev(rng.integers(0, V, N).astype(np.int32))
    out = D.token_logprobs(t, tok, 1.0, top=k, logp=logp, entropy=ent)
    D.token_logprobs_backward(t, tok, 1.0, out[4], ent, torch.ones(N, device="cuda"), grad=grad)
    assert torch.all(big[:2] == 7) and torch.all(big[2 + 2 * N:] == 7)
    assert torch.all(pad[:5] == 7) and torch.all(pad[5 + N * V:] == 7)
    assert torch.equal(t, before)


def test_empty_batches():
    t = torch.zeros((3, 100), device="cuda")
    out = D.token_logprobs(t, torch.empty(0, dtype=torch.int32, device="cuda"), 1.0, top=2,
                           rows=torch.empty(0, dtype=torch.int64, device="cuda"))
    assert out[0].shape == (0,) and out[2].shape == (0, 2)
    g = D.token_logprobs_backward(t[:0], out[0].int(), 1.0, out[4], out[1], out[0])
    assert g.shape == (0, 100)


@pytest.mark.parametrize("ragged", [False, True])
def test_emitted_tokens_of_a_round(ragged):
    """verify's y with the log probabilities of what it emitted, padded and flattened."""
    wl = inputs.SINGLE_USER.with_(name="lp_round", B=6, gamma=4, V=5000, T=0.8, seed=91)
    ld, lt = inputs.logits(wl)
    u_draft, u_acc, u_res = inputs.uniforms(wl)
    x = draw_tokens(ld, u_draft, wl.T)
    L = np.array([4, 0, 3, 2, 4, 1], dtype=np.int32)
    B, G = x.shape
    if ragged:
        off, _ = D.ragged_layout(dev(L), G)
        flat = O.pack_ragged(lt, L)
        n, y, _, _ = D.verify_ragged(pm(ld), dev(flat), off, dev(x), dev(L), dev(u_acc), dev(u_res), wl.T)
        rows = off[:-1, None] + torch.arange(G + 1, device="cuda")
        got = D.token_logprobs(dev(flat), y, wl.T, top=3, rows=rows.contiguous())
        check(flat.astype(np.float64), host(y), wl.T, 3, got, host(rows).ravel())
    else:
        n, y, _, _ = D.verify(pm(ld), dev(lt), dev(x), dev(L), dev(u_acc), dev(u_res), wl.T)
        got = D.token_logprobs(dev(lt), y, wl.T, top=3)
        check(lt.reshape(-1, wl.V).astype(np.float64), host(y), wl.T, 3, got)
    assert np.all((host(got[0]) == 0) == (host(y) < 0))
    # the drafted tokens under the position-major draft logits: row k * B + b
    rows = (torch.arange(G, device="cuda") * B + torch.arange(B, device="cuda")[:, None]).contiguous()
    got = D.token_logprobs(pm(ld), dev(x), wl.T, rows=rows)
    check(ld.transpose(1, 0, 2).reshape(-1, wl.V).astype(np.float64), x, wl.T, 0, got, host(rows).ravel())


def test_refusals():
    t = torch.zeros((4, 64), device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    st, e = torch.zeros((4, 2), device="cuda"), torch.zeros(4, device="cuda")
    for kw in (dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(top=33), dict(top=-1)):
        with pytest.raises(D.DsparkError):
            D.token_logprobs(t, tok, **{"T": 1.0, **kw})
    with pytest.raises(D.DsparkError):
        D.token_logprobs(t[:3], tok, 1.0)                       # fewer rows than entries
    for bad in (t.double(), t.cpu(), t.t(), t[0]):
        with pytest.raises(ValueError):
            D.token_logprobs(bad, tok, 1.0)
    for bad in (tok.long(), tok.cpu()):
        with pytest.raises(ValueError):
            D.token_logprobs(t, bad, 1.0)
    with pytest.raises(ValueError):
        D.token_logprobs(t, tok, 1.0, rows=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        D.token_logprobs(torch.zeros((4, 4, 64), device="cuda")[:, :3], tok, 1.0)   # rows not evenly apart
    with pytest.raises(D.DsparkError):
        D.token_logprobs_backward(t, tok, 1.0, st, None, e, e)  # entropy's gradient without the entropy
    with pytest.raises(ValueError):
        D.token_logprobs_backward(t, tok, 1.0, st, e, e, top_idx=tok.view(4, 1))
    buf = torch.zeros(4 * 64 + 8, device="cuda")
    with pytest.raises(D.DsparkError) as err:
        D.token_logprobs_backward(buf[:256].view(4, 64), tok, 1.0, st, e, e, grad=buf[8:264].view(4, 64))
    assert "overlap" in str(err.value)
    with pytest.raises(ValueError):
        D.token_logprobs_backward(t, tok[:2], 1.0, st, e, e)
