"""The LM head in 8-bit integers on the GPU against the oracle: norm with 8-bit output, quantisation,
integer product with scales, and the chain of them into a round.

Tolerances (u = 2^-24, half an fp32 step): q is exact (it is defined on fp32 products).  The scale: a
thread adds at most ceil(d / 32) squares, then 10 additions join the threads: (ceil(d / 32) + 10) u,
halved by the square root, and 6 more roundings.  The product: the integer sum is exact, its rounding
and the two products are 3 u, and the output's own rounding is half a step of its type.
"""

import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_04_b200 import dspark as D
from speculative_decoding_04_b200 import inputs
from tests.parity import check_draft, check_verify, dev, draw_tokens, host, host_rm

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def strided(a, dtype, ld=None, offset=0, fill=float("nan")):
    M, d = a.shape
    ld = d if ld is None else ld
    dt = DT.get(dtype, dtype)
    flat = torch.full((offset + M * ld + 64,), fill, dtype=dt, device="cuda")
    t = flat[offset:offset + M * ld].view(M, ld)[:, :d]
    t.copy_(torch.from_numpy(np.array(a)).to(dt).cuda())
    return t


def f32(t):
    return t.float().cpu().numpy()


def check_norm(h32, gain, eps, q, scale):
    wq, ws = O.rmsnorm_q8(h32, gain, eps) if eps is not None else O.quantize_q8(h32)
    assert np.array_equal(host(q).reshape(wq.shape), wq)
    s = host(scale).reshape(-1)
    assert np.array_equal(np.isnan(s), np.isnan(ws))
    tol = ((-(-h32.shape[1] // 32) + 10) / 2 + 6) * U32
    ok = ~np.isnan(ws)
    assert np.all(np.abs(s[ok] - ws[ok]) <= tol * ws[ok] + 1e-45)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 64, 100, 129, 131, 255, 1000, 1003, 2048, 2501, 4095, 4097, 5120, 8200,
                               16383, 16384, 32801, 40000])
def test_norm_sizes(dtype, d):
    rng = np.random.default_rng(d)
    M = 5
    for ld, off, res, gdt in ((d, 0, True, dtype), (d + 8, 8, True, "f32"), (d + 1, 1, True, dtype), (d, 0, False, "f32"),
                              (d + 3, 3, False, dtype), (d + 5, 5, True, "f32")):
        x = strided(rng.normal(size=(M, d)), dtype, ld, off)
        r = strided(2 * rng.normal(size=(M, d)), dtype, ld, off) if res else None
        g = torch.from_numpy(1 + 0.2 * rng.normal(size=d)).to(DT[gdt]).cuda()
        x0, r0 = x.clone(), None if r is None else r.clone()
        q, s, h = D.rmsnorm_q8(x, g, 1e-5, residual=r)
        want = x0 if r is None else (x0.float() + r0.float()).to(DT[dtype])
        assert (h is None) == (r is None) and (h is None or torch.equal(h, want))
        check_norm(f32(want), f32(g), 1e-5, q, s)
        if res:   # in place over the residual and over x
            q2, s2, h2 = D.rmsnorm_q8(x, g, 1e-5, residual=r, h_out=r)
            # (another alignment of h may sum in another order: the scale is held to its tolerance)
            assert h2 is r and torch.equal(r, want) and torch.equal(q2, q)
            check_norm(f32(want), f32(g), 1e-5, q2, s2)
            r.copy_(r0)
            q2, s2, _ = D.rmsnorm_q8(x, g, 1e-5, residual=r, h_out=x)
            assert torch.equal(x, want) and torch.equal(q2, q)
            check_norm(f32(want), f32(g), 1e-5, q2, s2)
    x = strided(rng.normal(size=(M, d)), dtype)
    q, s = D.quantize_q8(x)
    check_norm(f32(x), None, None, q, s)
    q, s, _ = D.rmsnorm_q8(x, None, 1e-5)
    check_norm(f32(x), None, 1e-5, q, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [256, 1001])
def test_norm_special_rows(dtype, d):
    rng = np.random.default_rng(7)
    x = rng.normal(size=(8, d))
    big, tiny = {"f32": (1e30, 1e-37), "bf16": (1e30, 1e-37), "f16": (6e4, 6e-8)}[dtype]
    x[0] = 0
    x[1, 3] = np.nan
    x[2, d - 1] = np.inf
    x[3] *= 0
    x[3, 5] = -1
    x[4] *= big / 8      # squares overflow fp32
    x[5] = tiny          # below the grid's range (fp32, bf16): counts as zero
    x[6] = 1.0
    x[7] = np.where(np.arange(d) % 2, 0.5, 127.0)   # ties: 0.5 of a step
    t = strided(x, dtype, d + 8)
    g = torch.ones(d, dtype=DT[dtype], device="cuda")
    q, s, _ = D.rmsnorm_q8(t, g, 1e-6)
    check_norm(f32(t), f32(g), 1e-6, q, s)
    q, s = D.quantize_q8(t)
    check_norm(f32(t), None, None, q, s)
    gz = torch.zeros(d, dtype=DT[dtype], device="cuda")
    q, s, _ = D.rmsnorm_q8(t[6:], gz, 1e-6)
    assert not host(q).any() and not host(s).any()


def make_q(rng, M, K, ld=None, lo=-127, hi=128):
    ld = (K + 15) // 16 * 16 if ld is None else ld
    return strided(rng.integers(lo, hi, (M, K)), torch.int8, ld, 0, fill=99)


def check_matmul(q, qs, w, ws, out, dtype):
    want = O.matmul_q8(host(q), host(qs), host(w), host(ws))
    got = out.double().cpu().numpy().reshape(want.shape)
    tol = (3 * U32 + HALF[dtype] * (1 + 4 * U32)) * np.abs(want) + {"f32": 1e-45, "bf16": 1e-40, "f16": 2.0 ** -25}[dtype]
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 77, 128, 255, 256, 257, 520, 1088])
@pytest.mark.parametrize("N,K", [(1, 1), (15, 16), (130, 127), (1000, 129), (5003, 1000), (40000, 64)])
def test_matmul_sizes(M, N, K):
    rng = np.random.default_rng(M * N + K)
    for dtype, extra in (("f32", 0), ("bf16", 3), ("f16", 1)):
        q, w = make_q(rng, M, K), make_q(rng, N, K, (K + 15) // 16 * 16 + 16 * extra)
        qs, ws = torch.rand(M, device="cuda") * 0.01, torch.rand(N, device="cuda") * 0.001
        buf = torch.full((M * (N + extra) + 16,), 7.0, dtype=DT[dtype], device="cuda")
        out = buf[5:5 + M * (N + extra)].view(M, N + extra)[:, :N]
        flags = torch.zeros(M, dtype=torch.int32, device="cuda")
        D.matmul_q8(q, qs, w, ws, out=out, flags=flags)
        check_matmul(q, qs, w, ws, out, dtype)
        assert not host(flags).any()
        assert torch.all(buf[:5] == 7) and torch.all(buf[5 + M * (N + extra):] == 7)
        if extra:
            assert torch.all(buf[5:5 + M * (N + extra)].view(M, N + extra)[:, N:] == 7)
        assert torch.equal(D.matmul_q8(q, qs, w, ws, out_dtype=DT[dtype]), out)


@pytest.mark.parametrize("M", [79, 80, 81, 95, 96, 97, 112])
def test_matmul_sizes_about_the_change_of_form(M):
    rng = np.random.default_rng(M)
    for N, K in ((2000, 128), (40003, 300)):
        q, w = make_q(rng, M, K), make_q(rng, N, K)
        qs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        for dtype in ("f32", "bf16"):
            check_matmul(q, qs, w, ws, D.matmul_q8(q, qs, w, ws, out_dtype=DT[dtype]), dtype)


def test_matmul_extremes():
    """The largest sums int32 holds: K = 131071 of -128 * -128, and alternating signs."""
    K = 131071
    q = make_q(np.random.default_rng(0), 3, K)
    w = make_q(np.random.default_rng(1), 5, K)
    q.fill_(-128)
    w.fill_(-128)
    w[1].fill_(127)
    w[2, ::2] = 127
    one = torch.ones(5, device="cuda")
    out = D.matmul_q8(q, one[:3], w, one)
    check_matmul(q, one[:3], w, one, out, "f32")
    assert float(out[0, 0]) == np.float32(131071 * 16384)


def test_matmul_wide_k_many_tiles():
    rng = np.random.default_rng(5)
    q, w = make_q(rng, 300, 4096), make_q(rng, 60001, 4096)
    qs, ws = torch.rand(300, device="cuda"), torch.rand(60001, device="cuda")
    for dtype in ("f32", "bf16"):
        check_matmul(q, qs, w, ws, D.matmul_q8(q, qs, w, ws, out_dtype=DT[dtype]), dtype)


def test_matmul_scales_zero_nan_and_leading_dimensions():
    rng = np.random.default_rng(6)
    q, w = make_q(rng, 12, 200), make_q(rng, 500, 200)
    qs, ws = torch.rand(12, device="cuda"), torch.rand(500, device="cuda")
    qs[3], qs[5], ws[7] = 0.0, float("nan"), 0.0
    out = host(D.matmul_q8(q, qs, w, ws))
    assert not out[3].any() and np.isnan(out[5]).all() and not out[[0, 1, 2, 4], 7].any()
    q3 = q.as_strided((3, 4, 200), (4 * q.stride(0), q.stride(0), 1))
    out3 = D.matmul_q8(q3, qs.view(3, 4), w, ws)
    assert out3.shape == (3, 4, 500) and np.array_equal(host(out3).reshape(12, 500), out, equal_nan=True)


def test_streams_and_graphs():
    rng = np.random.default_rng(8)
    M, d, N = 40, 1024, 9000
    x, r = torch.randn(M, d, device="cuda").bfloat16(), torch.randn(M, d, device="cuda").bfloat16()
    g = torch.rand(d, device="cuda").bfloat16()
    w, ws = D.quantize_q8(torch.randn(N, d, device="cuda").bfloat16())

    def head():
        q, s, h = D.rmsnorm_q8(x, g, 1e-6, residual=r)
        return q, s, h, D.matmul_q8(q, s, w, ws)

    want = head()
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    q, s, h = D.rmsnorm_q8(x, g, 1e-6, residual=r, stream=s2)
    out = D.matmul_q8(q, s, w, ws, stream=s2)
    s2.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (q, s, h, out)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = head()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_quantised_rows_are_laid_out_for_the_product():
    for d, ld in ((100, 112), (511, 512), (512, 512), (513, 640), (4271, 4352)):
        q, s = D.quantize_q8(torch.randn(6, d, device="cuda"))
        assert q.shape == (6, d) and q.stride() == (ld, 1)
        n, s2, _ = D.rmsnorm_q8(torch.randn(2, 3, d, device="cuda"), None, 1e-6)
        assert n.shape == (2, 3, d) and n.stride() == (3 * ld, ld, 1)
        check_matmul(n.reshape(6, d), s2.view(-1), q, s, D.matmul_q8(n, s2, q, s), "f32")


def test_two_calls_at_once():
    """Two products on two streams: no scratch is shared."""
    rng = np.random.default_rng(12)
    jobs = []
    for M, N, K in ((64, 30000, 512), (600, 9001, 768)):
        q, w = make_q(rng, M, K), make_q(rng, N, K)
        qs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        jobs.append((q, qs, w, ws, D.matmul_q8(q, qs, w, ws)))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [D.matmul_q8(*j[:4], stream=s) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, j[4]) for o, j in zip(outs, jobs))


@pytest.mark.parametrize("M", [40, 300])   # one CTA a tile, and CTA pairs
def test_bounded_waits_return(M):
    """Accumulator barriers that expect one arrival more than will come: the call returns, its outputs
    are NaN and its flags say so, and the next call is right.  Nothing faults or hangs."""
    rng = np.random.default_rng(13)
    q, w = make_q(rng, M, 300), make_q(rng, 4000, 300)
    qs, ws = torch.rand(M, device="cuda"), torch.rand(4000, device="cuda")
    flags = torch.zeros(M, dtype=torch.int32, device="cuda")
    D.set_option("debug_wait_limit", 1 << 12)
    D.set_option("debug_unreachable_barrier", 3)
    out = D.matmul_q8(q, qs, w, ws, flags=flags)
    torch.cuda.synchronize()
    assert torch.isnan(out).all()
    assert np.all(host(flags).view(np.uint32) == np.uint32(D.FLAG_DEVICE_TIMEOUT))
    D.set_option("debug_unreachable_barrier", 0)
    D.set_option("debug_wait_limit", 0)
    flags.zero_()
    out = D.matmul_q8(q, qs, w, ws, flags=flags)
    check_matmul(q, qs, w, ws, out, "f32")
    assert not host(flags).any()


def test_empty_batches():
    x = torch.zeros((0, 64), device="cuda")
    q, s, h = D.rmsnorm_q8(x, None, 1e-6, residual=x)
    assert q.shape == (0, 64) and h.shape == (0, 64)
    w, ws = D.quantize_q8(torch.ones((10, 64), device="cuda"))
    assert D.matmul_q8(q, s, w, ws).shape == (0, 10)


@pytest.mark.parametrize("layout", ["position", "request"])
def test_head_into_a_round(layout):
    """Hidden states -> norm -> head -> draft -> verify -> log probabilities, in one run: every stage
    against the oracle on the device's own inputs to it."""
    wl = inputs.SINGLE_USER.with_(name="head_round", B=5, gamma=4, V=4096, r=64, T=0.9, seed=17, w_sigma=0.05)
    B, G, V, d = wl.B, wl.gamma, wl.V, 256
    rng = np.random.default_rng(17)
    lead = (G, B) if layout == "position" else (B, G)
    hid, res = (torch.from_numpy(rng.normal(size=lead + (d,))).bfloat16().cuda() for _ in range(2))
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    Wh, Ws = D.quantize_q8(torch.from_numpy(rng.normal(size=(V, d)) * 0.15).bfloat16().cuda())
    q, s, h = D.rmsnorm_q8(hid, gain, 1e-6, residual=res)
    check_norm(f32(h).reshape(-1, d), f32(gain), 1e-6, q, s)
    U = D.matmul_q8(q, s, Wh, Ws)
    check_matmul(q.reshape(-1, d), s.reshape(-1), Wh, Ws, U, "f32")
    data = inputs.full_inputs(wl)
    W1, W2 = dev(data["W1"], torch.bfloat16), dev(data["W2"], torch.bfloat16)
    x, ld, fl = D.markov_draft(U, W1, W2, dev(data["x0"]), dev(data["u_draft"]), wl.T, layout=layout)
    rm = (lambda t: host_rm(t)) if layout == "position" else host
    check_draft(rm(U), data["W1"], data["W2"], data["x0"], data["u_draft"], wl.T, host(x), rm(ld), host(fl))
    ht = torch.from_numpy(rng.normal(size=(B, G + 1, d))).bfloat16().cuda()
    qt, st, _ = D.rmsnorm_q8(ht, gain, 1e-6)
    lt = D.matmul_q8(qt, st, Wh, Ws)
    n, y, _, fl = D.verify(ld, lt, x, None, dev(data["u_acc"]), dev(data["u_res"]), wl.T, ld_layout=layout)
    check_verify(rm(ld), host(lt), host(x), None, data["u_acc"], data["u_res"], wl.T, host(n), host(y),
                 flags_gpu=host(fl))
    logp, ent, ti, tl, stats = D.token_logprobs(lt, y, wl.T, top=4)
    r = O.token_logprobs(host(lt).reshape(-1, V), host(y).ravel(), wl.T, 4)
    assert np.allclose(host(logp).ravel(), r["logp"], rtol=1e-6, atol=1e-5)
    assert np.array_equal(host(ti).reshape(-1, 4), r["top_idx"])


def test_refusals():
    x = torch.zeros((4, 64), device="cuda")
    g = torch.ones(64, device="cuda")
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(D.DsparkError):
            D.rmsnorm_q8(x, g, eps)
    for bad in (g[:63], g.double(), g.cpu()):
        with pytest.raises(ValueError):
            D.rmsnorm_q8(x, bad, 1e-6)
    with pytest.raises(ValueError):
        D.rmsnorm_q8(x, g, 1e-6, residual=x.bfloat16())
    with pytest.raises(ValueError):
        D.rmsnorm_q8(x.t(), g[:4], 1e-6)
    buf = torch.zeros(4 * 64 + 8, device="cuda")
    with pytest.raises(D.DsparkError) as e:
        D.rmsnorm_q8(buf[:256].view(4, 64), g, 1e-6, residual=x, h_out=buf[8:264].view(4, 64))
    assert "overlaps" in str(e.value)
    q, s = D.quantize_q8(x)
    w, ws = D.quantize_q8(torch.ones((10, 64), device="cuda"))
    with pytest.raises(ValueError):
        D.matmul_q8(q[:, :32], s, w, ws)
    with pytest.raises(ValueError):
        D.matmul_q8(q.float(), s, w, ws)
    with pytest.raises(ValueError):
        D.matmul_q8(q, s[:3], w, ws)
    with pytest.raises(ValueError):
        D.matmul_q8(q, s, w, ws, out_dtype=torch.float64)
    with pytest.raises(D.DsparkError) as e:   # rows not on 16 bytes
        D.matmul_q8(torch.zeros((4, 60), dtype=torch.int8, device="cuda"), s,
                    torch.zeros((10, 60), dtype=torch.int8, device="cuda"), ws)
    assert "multiples of 16" in str(e.value)
    flat = torch.zeros(4 * 64 + 1, dtype=torch.int8, device="cuda")
    with pytest.raises(D.DsparkError) as e:
        D.matmul_q8(flat[1:].view(4, 64), s, w, ws)
    assert "16-byte" in str(e.value)
