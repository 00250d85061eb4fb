"""CPU oracle of the operators at the vocabulary-sized ends of a round (test infrastructure).

Plain float64 NumPy from the operators' definitions, sharing no code with the CUDA path:
  * token_logprobs, token_logprobs_grad -- log softmax at temperature T of given tokens, its entropy
    and largest entries, and the gradient with respect to the logits.
  * rmsnorm_q8, quantize_q8 -- root-mean-square norm (or none) on an 8-bit grid per row; the grid is
    defined on fp32 products, so q is reproduced exactly and the scale is fp64.
  * matmul_q8 -- integer product with a scale for each row of either side.
"""

from __future__ import annotations

import numpy as np


def token_logprobs(logits, tokens, T: float = 1.0, top: int = 0, rows=None):
    """dict(logp [N], entropy [N], top_idx [N, top], top_logp [N, top], stats [N, 2], p) of the entries.

    Entry n reads row rows[n] (n without rows).  Token -1: zeros and no alternatives, p is None.  A row
    index outside the array: NaN.  A row with NaN or +inf: NaN.  A token outside [0, V): logp NaN.  A
    row of -inf only: logp -inf, entropy 0, stats (-inf, -inf).  Alternatives: value descending, index
    ascending, -inf left out (-1, -inf in their places)."""
    logits = np.asarray(logits, dtype=np.float64)
    tokens = np.asarray(tokens).reshape(-1)
    N, V = tokens.size, logits.shape[-1]
    logp, ent, stats = np.zeros(N), np.zeros(N), np.zeros((N, 2))
    ti, tl, ps = np.full((N, top), -1, dtype=np.int64), np.full((N, top), -np.inf), []
    for n in range(N):
        r = n if rows is None else int(rows[n])
        t = int(tokens[n])
        ps.append(None)
        if t == -1:
            continue
        if not 0 <= r < logits.shape[0] or np.isnan(logits[r]).any() or np.isposinf(logits[r]).any():
            logp[n] = ent[n] = np.nan
            stats[n] = np.nan
            tl[n] = np.nan
            continue
        l = logits[r]
        m = l.max()
        ok = 0 <= t < V
        if m == -np.inf:
            logp[n], stats[n] = (-np.inf if ok else np.nan), -np.inf
            continue
        z = (l - m) / T
        logS = np.log(np.exp(z).sum())
        lp = z - logS
        p = np.exp(lp)
        ps[-1] = p
        logp[n] = lp[t] if ok else np.nan
        ent[n] = -np.sum(p[p > 0] * lp[p > 0])
        stats[n] = m, logS
        order = np.lexsort((np.arange(V), -l))[:top]
        order = order[l[order] > -np.inf]
        ti[n, :order.size], tl[n, :order.size] = order, lp[order]
    return dict(logp=logp, entropy=ent, top_idx=ti, top_logp=tl, stats=stats, p=ps)


def token_logprobs_grad(logits, tokens, T: float, g_logp=None, g_entropy=None, top_idx=None, g_top=None):
    """d(sum g_logp logp + sum g_entropy entropy + sum g_top top_logp) / d logits, entry n = row n."""
    logits = np.asarray(logits, dtype=np.float64)
    N, V = logits.shape
    out = np.zeros((N, V))
    for n in range(N):
        t, l = int(tokens[n]), logits[n]
        if not 0 <= t < V:
            continue
        if np.isnan(l).any() or np.isposinf(l).any():
            out[n] = np.nan
            continue
        if l.max() == -np.inf:
            continue
        z = (l - l.max()) / T
        lp = z - np.log(np.exp(z).sum())
        p = np.exp(lp)
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)
        w = np.zeros(V)   # weights of the log probabilities
        if g_logp is not None:
            w[t] += float(g_logp[n])
        if g_top is not None:
            for i, g in zip(top_idx[n], g_top[n]):
                if i >= 0:
                    w[int(i)] += float(g)
        d = w - p * w.sum()
        if g_entropy is not None:
            d -= float(g_entropy[n]) * (plp - p * plp.sum())
        out[n] = d / T
    return out


def rmsnorm_q8(h, gain, eps: float):
    """(q int8 [M, d], scale fp64 [M]) of rows h (already x + residual, rounded to their type).

    v = fp32(h * gain), A = max |v|, q = rint(fp32(v * fp32(127 / A))), scale = A / sqrt(mean h^2 + eps) / 127.
    A row with A < 2^-120: zeros.  A row with NaN or infinity: q 0, scale NaN."""
    h32 = np.asarray(h, dtype=np.float32)
    g = np.ones(h32.shape[1], np.float32) if gain is None else np.asarray(gain, dtype=np.float32)
    return _to_grid(h32, g, lambda r: 1 / np.sqrt(np.mean(h32[r].astype(np.float64) ** 2) + eps))


def quantize_q8(x):
    """(q int8, scale fp64) of rows: A = max |x|, q = rint(fp32(x * fp32(127 / A))), scale = A / 127."""
    x32 = np.asarray(x, dtype=np.float32)
    return _to_grid(x32, np.ones(x32.shape[1], np.float32), lambda r: 1.0)


def _to_grid(h, g, factor):
    q, scale = np.zeros(h.shape, np.int8), np.zeros(h.shape[0])
    for r in range(h.shape[0]):
        with np.errstate(all="ignore"):
            v = h[r] * g
            A = np.abs(v).max()
        if not np.isfinite(A) or not np.isfinite(h[r]).all():
            scale[r] = np.nan
        elif A >= 2.0 ** -120:
            q[r] = np.rint(v * (np.float32(127) / A)).astype(np.int8)
            scale[r] = float(A) * factor(r) / 127
    return q, scale


def matmul_q8(q, q_scale, w, w_scale):
    """[M, N] fp64: q_scale[m] w_scale[n] sum_k q[m, k] w[n, k] (products of 8-bit integers are exact in fp64)."""
    s = np.asarray(q, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    return s * np.asarray(q_scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)
