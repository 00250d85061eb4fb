"""The error of the log probabilities and the entropy, bounded by the roundings that the kernel makes.

u = 2^-24 is half an fp32 step.  All sums are fp32.  A term 2^d of S (d <= 0, in bits) is rounded
  3 |d| ln 2  for its exponent: (l - R) c, c itself, and when the reference R rises by r, 2 |r| more, the
              rises adding up to what d lacks of the final exponent,
  4           for ex2,
  7 + t       by additions: in its tile of 16 values a lane (8 pairs), and one for each of the warp's t tiles,
  5 t         for rises of the reference: ex2's 4 and the product, at most one rise a tile,
  6           joining the two halves of a pair and 32 lanes,
  14 + 14     joining the warps and, where a cluster has the row, its CTAs.
The terms are not negative, so S is off by at most the largest of these relatively, and ln S absolutely by
  e_S = u (45 + 6 t + 3 D),   D = sum p |d| ln 2.
A CTA has at least 2, 4 or 8 warps for up to 32, 128 and more tiles (a tile: 512 values, and one more where the
row does not start on 16 bytes).  logp: e_S + u |logp|.  The entropy ln S - E / S, E = sum 2^d d ln 2 <= D S:
e_S, the same relative error twice over on E / S (E's own terms and S), 3 u D2 for the exponents in E's terms with
D2 = sum p (d ln 2)^2, and u of the result."""

import numpy as np
import pytest

import oracle as O
from speculative_decoding_04_b200 import dspark as D
from tests.parity import dev, host
from tests.test_gpu_logprobs import U32, as64, rows_of, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V", [(1, 151936), (3, 40001), (600, 3001), (200, 17001), (40, 70001), (5, 300)])
def test_errors_stay_within_the_roundings(dtype, N, V):
    rng = np.random.default_rng(N + V)
    l = rows_of(rng, N, V)
    if N > 2:
        l[1] = np.sort(l[1])            # the reference rises in every tile
        l[2] = -np.sort(-l[2])
    t = strided(l, dtype, V + 1, 1)
    tok = rng.integers(0, V, N).astype(np.int32)
    logp, ent, _, _, stats = (None if x is None else host(x) for x in D.token_logprobs(t, dev(tok), 1.0))
    r = O.token_logprobs(as64(t), tok, 1.0)
    tiles = -(-V // 512) + 1
    per_warp = -(-tiles // (2 if tiles <= 32 else 4 if tiles <= 128 else 8))
    k = 45 + 6 * per_warp
    for n, p in enumerate(r["p"]):
        logS = r["stats"][n, 1]
        d = np.where(p > 0, -(np.log(np.maximum(p, 1e-320)) + logS), 0.0)
        Dn, D2 = float((p * d).sum()), float((p * d * d).sum())
        eS = U32 * (k + 3 * Dn)
        assert abs(stats[n, 1] - logS) <= eS + U32 * abs(logS), n
        assert abs(logp[n] - r["logp"][n]) <= eS + U32 * abs(r["logp"][n]), n
        assert abs(ent[n] - r["entropy"][n]) <= eS + 2 * U32 * (k + 3) * Dn + 3 * U32 * D2 + U32 * r["entropy"][n], n
