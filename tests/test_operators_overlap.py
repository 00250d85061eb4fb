"""What counts as an overlap of an output with an input (no GPU needed): the argument checks of the gradient and
of the norm, against a count of shared bytes."""

import pytest
import torch

from speculative_decoding_04_b200 import build

build.build()
from speculative_decoding_04_b200 import dspark as D  # noqa: E402

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers are only passed where no GPU exists")
FAKE = 4096 * 256


def shared(a, lda, b, ldb, rows, cols, es):
    def held(p, ld):
        return {p + r * ld * es + i for r in range(rows) for i in range(cols * es)}
    return bool(held(a, lda) & held(b, ldb))


@no_gpu
@pytest.mark.parametrize("rows", [1, 2, 3, 5])
@pytest.mark.parametrize("cols,ld", [(4, 4), (4, 7), (4, 8), (4, 9), (1, 2)])
def test_gradients_beside_the_logits(rows, cols, ld):
    """Every offset around the logits: refused where memory is shared, but for the logits themselves."""
    span = rows * ld + 3
    for off in range(-span, span + 1):
        st = D.lib.dspark_token_logprobs_backward(FAKE, D.F32, ld, FAKE, rows, cols, 1.0, FAKE, None, FAKE, None, 0, None,
                                                  None, FAKE + 4 * off, ld, None)
        refused = st == D.EINVAL and "overlaps" in D.last_error()
        assert refused == (off != 0 and shared(FAKE, ld, FAKE + 4 * off, ld, rows, cols, 4)), off


@no_gpu
@pytest.mark.parametrize("rows", [1, 2, 4])
def test_norm_outputs_beside_the_inputs(rows):
    d, ld = 6, 15
    for off in range(-rows * ld - 3, rows * ld + 4):
        # the residual far away, then the other way round
        for x, r in ((FAKE, FAKE + (1 << 20)), (FAKE + (1 << 20), FAKE)):
            h = FAKE + 2 * off
            st = D.lib.dspark_rmsnorm_q8(x, D.BF16, ld, r, ld, None, D.F32, rows, d, 1e-6, h, ld, FAKE, 16, FAKE, None)
            refused = st == D.EINVAL and "overlaps" in D.last_error()
            assert refused == (off != 0 and shared(FAKE, ld, h, ld, rows, d, 2)), off


@no_gpu
def test_other_strides_are_refused_where_the_ranges_cross():
    for ldg, off, want in ((9, 4, True), (9, 64, False), (16, 0, True), (8, 4, False)):
        st = D.lib.dspark_token_logprobs_backward(FAKE, D.F32, 8, FAKE, 4, 4, 1.0, FAKE, None, FAKE, None, 0, None, None,
                                                  FAKE + 4 * off, ldg, None)
        assert (st == D.EINVAL and "overlaps" in D.last_error()) == want, (ldg, off)
