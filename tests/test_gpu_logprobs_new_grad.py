"""The gradient that token_logprobs_backward allocates itself."""

import numpy as np
import pytest
import torch

from speculative_decoding_04_b200 import dspark as D
from tests.parity import dev
from tests.test_gpu_logprobs import grad_check, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_a_new_gradient_takes_no_more_memory_than_its_rows(dtype):
    """The last position of each request's logits: rows a whole request apart."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    rng = np.random.default_rng(2)
    B, S, V = 4, 40, 5003
    full = torch.zeros((B, S, V), dtype=dt, device="cuda")
    l = full[:, -1]
    l.copy_(dev(rows_of(rng, B, V)))
    tok = rng.integers(0, V, B).astype(np.int32)
    _, ent, _, _, st = D.token_logprobs(l, dev(tok), 1.0)
    gl, gh = rng.normal(size=B).astype(np.float32), rng.normal(size=B).astype(np.float32)
    g = D.token_logprobs_backward(l, dev(tok), 1.0, st, ent, dev(gl), dev(gh))
    assert g.shape == l.shape and g.untyped_storage().nbytes() <= B * (V + 8) * l.element_size()
    grad_check(l, tok, 1.0, gl, gh, None, None, g, dtype)
    g3 = D.token_logprobs_backward(full[:, -1:], dev(tok), 1.0, st, ent, dev(gl), dev(gh))
    assert g3.shape == (B, 1, V) and torch.equal(g3[:, 0], g)
    # rows with a little space behind them keep their stride
    p = full.view(B * S, V)[:, :V - 3]
    tok = np.zeros(B * S, dtype=np.int32)
    _, ent, _, _, st = D.token_logprobs(p, dev(tok), 1.0)
    g = D.token_logprobs_backward(p, dev(tok), 1.0, st, ent, dev(np.ones(B * S, dtype=np.float32)))
    assert g.stride() == p.stride()
