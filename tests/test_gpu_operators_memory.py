"""Arguments that lie side by side in one buffer."""

import numpy as np
import pytest
import torch

from speculative_decoding_04_b200 import dspark as D
from tests.parity import dev, host
from tests.test_gpu_head_q8 import check_norm, f32
from tests.test_gpu_logprobs import grad_check, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 100, 1000, 4097])
def test_norm_into_the_columns_beside_its_input(d):
    buf = torch.randn(7, 2 * d + 3, device="cuda").bfloat16()
    x, h_out = buf[:, :d], buf[:, d:2 * d]
    r = torch.randn(7, d, device="cuda").bfloat16()
    want, rest = (x.float() + r.float()).bfloat16(), buf[:, 2 * d:].clone()
    x0 = x.clone()
    q, s, h = D.rmsnorm_q8(x, None, 1e-6, residual=r, h_out=h_out)
    assert h is h_out and torch.equal(h, want) and torch.equal(x, x0) and torch.equal(buf[:, 2 * d:], rest)
    check_norm(f32(want), None, 1e-6, q, s)
    with pytest.raises(D.DsparkError, match="overlaps"):
        D.rmsnorm_q8(x, None, 1e-6, residual=r, h_out=buf[:, d - 1:2 * d - 1])
    with pytest.raises(D.DsparkError, match="overlaps"):
        D.rmsnorm_q8(h_out, None, 1e-6, residual=r, h_out=buf[:, 1:d + 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_into_the_columns_beside_the_logits(dtype):
    rng = np.random.default_rng(1)
    N, V = 5, 1001
    buf = torch.zeros((N, 2 * V + 1), dtype=dtype, device="cuda")
    l, grad = buf[:, :V], buf[:, V:2 * V]
    l.copy_(dev(rows_of(rng, N, V)))
    l0 = l.clone()
    tok = rng.integers(0, V, N).astype(np.int32)
    _, ent, _, _, st = D.token_logprobs(l, dev(tok), 1.0)
    gl = np.ones(N, dtype=np.float32)
    g = D.token_logprobs_backward(l, dev(tok), 1.0, st, ent, dev(gl), grad=grad)
    assert g.data_ptr() == grad.data_ptr() and torch.equal(l, l0) and not buf[:, 2 * V:].any()
    grad_check(l, tok, 1.0, gl, None, None, None, g, "f32" if dtype == torch.float32 else "bf16")
    with pytest.raises(D.DsparkError, match="overlaps"):
        D.token_logprobs_backward(l, dev(tok), 1.0, st, ent, dev(gl), grad=buf[:, V - 1:2 * V - 1])
