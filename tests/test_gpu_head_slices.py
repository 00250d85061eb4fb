"""The 8-bit product into columns of a wider buffer: nothing beside the output is written, whatever the output's
width, alignment and distance of rows."""

import numpy as np
import pytest
import torch

from speculative_decoding_04_b200 import dspark as D
from tests.test_gpu_head_q8 import DT, check_matmul, make_q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 40, 80, 81, 200, 300])
def test_columns_beside_the_output_stay(M, dtype):
    rng = np.random.default_rng(M)
    K = 130
    q, qs = make_q(rng, M, K), torch.rand(M, device="cuda") * 0.01
    for N in (1, 3, 8, 13, 125, 127, 128, 255, 257, 2045):
        w, ws = make_q(rng, N, K), torch.rand(N, device="cuda") * 0.01
        for ld in (N, N + 1, N + 2, N + 3, (N + 7) // 8 * 8, (N + 7) // 8 * 8 + 8, 2 * N + 5):
            for off in (0, 8, 3):
                buf = torch.full((off + M * ld + 64,), 7.0, dtype=DT[dtype], device="cuda")
                rows = buf[off:off + M * ld].view(M, ld)
                D.matmul_q8(q, qs, w, ws, out=rows[:, :N])
                check_matmul(q, qs, w, ws, rows[:, :N], dtype)
                assert torch.all(buf[:off] == 7) and torch.all(buf[off + M * ld:] == 7), (N, ld, off)
                assert torch.all(rows[:, N:] == 7), (N, ld, off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_heads_into_one_buffer(dtype):
    """Two products on two streams into neighbouring columns, rows on 16 bytes, the border within 16 bytes."""
    rng = np.random.default_rng(5)
    M, K, N = 300, 256, 4001
    q, qs = make_q(rng, M, K), torch.rand(M, device="cuda") * 0.01
    ws = [(make_q(rng, N, K), torch.rand(N, device="cuda") * 0.01) for _ in range(2)]
    buf = torch.zeros((M, 8008), dtype=DT[dtype], device="cuda")
    streams = [torch.cuda.Stream() for _ in ws]
    for _ in range(5):
        buf.fill_(7.0)
        torch.cuda.synchronize()
        for i, (w, s) in enumerate(ws):
            D.matmul_q8(q, qs, w, s, out=buf[:, i * N:(i + 1) * N], stream=streams[i])
        torch.cuda.synchronize()
        for i, (w, s) in enumerate(ws):
            check_matmul(q, qs, w, s, buf[:, i * N:(i + 1) * N], dtype)
        assert torch.all(buf[:, 2 * N:] == 7)
