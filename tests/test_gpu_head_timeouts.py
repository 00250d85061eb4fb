"""Bounded waits of the 8-bit product that give up in some of a CTA's warps, or in calls of many tiles a CTA:
an output that could not be computed is NaN and its token's flags say so, every other output is right, and the
next call is right.  The options make a wait give up; nothing faults or hangs."""

import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_04_b200 import dspark as D
from tests.parity import host
from tests.test_gpu_head_q8 import DT, HALF, U32, check_matmul, make_q

pytestmark = pytest.mark.gpu


def problem(M, N, K=300):
    rng = np.random.default_rng(M + N)
    q, w = make_q(rng, M, K), make_q(rng, N, K)
    return q, 0.5 + torch.rand(M, device="cuda"), w, 0.5 + torch.rand(N, device="cuda")


def with_option(barrier, a, dtype):
    flags = torch.zeros(a[0].shape[0], dtype=torch.int32, device="cuda")
    D.set_option("debug_wait_limit", 1 << 12)
    D.set_option("debug_unreachable_barrier", barrier)
    try:
        out = D.matmul_q8(*a, out_dtype=DT[dtype], flags=flags)
        torch.cuda.synchronize()
    finally:
        D.set_option("debug_unreachable_barrier", 0)
        D.set_option("debug_wait_limit", 0)
    return out.double().cpu().numpy(), host(flags).view(np.uint32)


def check_partial(a, out, flags, dtype):
    lost = np.isnan(out)
    assert np.array_equal(flags, np.where(lost.any(-1), np.uint32(D.FLAG_DEVICE_TIMEOUT), np.uint32(0)))
    want = O.matmul_q8(*(host(t) for t in a))
    tol = (3 * U32 + HALF[dtype] * (1 + 4 * U32)) * np.abs(want) + 1e-40   # as check_matmul; |want| < 6e6
    assert np.all(np.abs(out - want)[~lost] <= tol[~lost])
    again = torch.zeros(out.shape[0], dtype=torch.int32, device="cuda")
    check_matmul(*a, D.matmul_q8(*a, out_dtype=DT[dtype], flags=again), dtype)
    assert not host(again).any()
    return lost


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(40, 37000), (20, 36999), (300, 4000), (200, 4001)])
def test_one_warp_gives_up(M, N, dtype):
    """One tile a CTA; the last epilogue warp's wait gives up, all others' are met."""
    a = problem(M, N)
    out, flags = with_option(4, a, dtype)
    lost = check_partial(a, out, flags, dtype)
    # 32 of a CTA's channels, for the tokens of that warp's chunks
    step = 32 if M <= 80 else 64
    tile = M if M <= 80 else (M // (1 + (M > 256)) + 31) // 32 * 32
    rows = (np.arange(M) % tile) % step >= step - 16
    assert np.array_equal(lost.any(-1), rows) and 0 < lost[rows].mean() < 0.5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(40, 150000), (7, 100001), (300, 60001), (600, 40000)])
def test_waits_give_up_in_calls_of_many_tiles(M, N, dtype):
    """More than two tiles a CTA: an accumulator's barrier is used again, and a parity waited for in vain at
    one tile is met at once two tiles on."""
    a = problem(M, N)
    out, flags = with_option(3, a, dtype)
    assert check_partial(a, out, flags, dtype).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(40, 150000), (300, 60001)])
def test_one_warp_gives_up_in_calls_of_many_tiles(M, N, dtype):
    """Without that warp's arrivals the third tile's products are not issued: its outputs are lost, the first
    two tiles' are right but for the warp's own."""
    a = problem(M, N)
    out, flags = with_option(4, a, dtype)
    lost = check_partial(a, out, flags, dtype)
    assert lost.any(-1).all() and 0 < lost.mean() < 1


@pytest.mark.parametrize("M", [3, 100])
@pytest.mark.parametrize("limit", [1 << 32, (1 << 33) + 1, 1 << 40])
def test_a_long_limit_is_not_cut_to_a_short_one(M, limit):
    a = problem(M, 5000, 2000)
    flags = torch.zeros(M, dtype=torch.int32, device="cuda")
    D.set_option("debug_wait_limit", limit)
    try:
        out = D.matmul_q8(*a, flags=flags)
        torch.cuda.synchronize()
    finally:
        D.set_option("debug_wait_limit", 0)
    assert not host(flags).any()
    check_matmul(*a, out, "f32")
