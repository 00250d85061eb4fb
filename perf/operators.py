"""Workloads of the operators at the two vocabulary-sized ends of a round: the LM head in 8-bit
integers (root-mean-square norm with an 8-bit output, integer product with scales) and the log
probabilities of given tokens with entropy and top alternatives, forward and backward.

`own` says which side `run` computes: False the plain form in elementary torch operations, True the
library's kernels through `speculative_decoding_04_b200.dspark`.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one user's stream, with the most alternatives a serving API returns: latency
        dict(name="logp_one_token", op="logp", N=1, V=151936, ld=151936, dtype="f32", top=20, T=1.0, mask=0.0, pad=0),
        # every row of a verified block at 64 requests of 16 drafts
        dict(name="logp_high_concurrency", op="logp", N=1088, V=151936, ld=151936, dtype="f32", top=8, T=0.8, mask=0.0,
             pad=0),
        # constrained decoding: an odd vocabulary, rows not aligned to 16 bytes, most of it masked, some rows padding
        dict(name="logp_masked_odd", op="logp", N=77, V=50001, ld=50001, dtype="f16", top=5, T=1.3, mask=0.9, pad=13),
        # scoring long texts with a large vocabulary
        dict(name="logp_scoring", op="logp", N=2048, V=262144, ld=262144, dtype="bf16", top=1, T=1.0, mask=0.0, pad=0),
        # a small training step of a draft head
        dict(name="logp_grad_small", op="grad", N=24, V=30000, ld=30000, dtype="f32", top=0, T=1.0, mask=0.0, pad=3),
        # a training step on a batch of texts, with an entropy bonus and a loss on the alternatives, padded rows
        dict(name="logp_grad_batch", op="grad", N=2048, V=151936, ld=152064, dtype="bf16", top=4, T=1.0, mask=0.0,
             pad=200),
        # the final norm of one token
        dict(name="norm_one_token", op="norm", M=1, d=4096, dtype="bf16", res=True),
        # the final norm over the positions of a long batch
        dict(name="norm_batch", op="norm", M=16384, d=5120, dtype="bf16", res=True),
        # the head for one token: one pass over the weights
        dict(name="head_one_token", op="head", M=1, N=151936, K=4096, out="f32"),
        # the head for the scheduled rows of a few users, odd sizes
        dict(name="head_ragged", op="head", M=77, N=50001, K=1000, out="bf16"),
        # the head for every row of a verified block at 64 requests of 16 drafts
        dict(name="head_high_concurrency", op="head", M=1088, N=151936, K=4096, out="f32"),
        # the head over a batch of texts
        dict(name="head_scoring", op="head", M=4096, N=129280, K=2048, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("logp", "grad", "norm", "head"))
    if op in ("logp", "grad"):
        dtype = rng.choice(("f32", "bf16", "f16"))
        V = _log_int(rng, 1000, 262144)
        most = (1 << 30 if op == "logp" else 600_000_000) // (V * _SIZE[dtype])
        N = max(1, min(_log_int(rng, 1, 4096), most))
        return dict(op=op, N=N, V=V, ld=V + rng.choice((0, 0, 1, 64)), dtype=dtype,
                    top=rng.choice((0, 1, 5, 20)) if op == "logp" else rng.choice((0, 0, 4)),
                    T=rng.choice((1.0, 0.7, 1.3)), mask=rng.choice((0.0, 0.0, 0.5)),
                    pad=rng.randrange(0, max(1, N // 3) + 1) if N > 1 else 0)
    if op == "norm":
        d = _log_int(rng, 64, 16384)
        return dict(op=op, M=max(1, min(_log_int(rng, 1, 16384), 80_000_000 // d)), d=d,
                    dtype=rng.choice(("bf16", "f16", "f32")), res=rng.random() < 0.7)
    K, N = _log_int(rng, 64, 8192), _log_int(rng, 1000, 262144)
    K = min(K, 600_000_000 // N)
    M = max(1, min(_log_int(rng, 1, 4096), 670_000_000_000 // (N * K), 300_000_000 // N))
    return dict(op=op, M=M, N=N, K=K, out=rng.choice(("f32", "bf16", "f16")))


# ------------------------------------------------------------------ inputs

def _logits(case, g):
    """Log-Zipf prior over a permutation of the vocabulary plus noise, as a language model's rows look."""
    N, V = case["N"], case["V"]
    prior = -1.1 * torch.log(torch.randperm(V, generator=g, device="cuda").float() + 1)
    full = torch.zeros((N, case["ld"]), dtype=_DT[case["dtype"]], device="cuda")
    l = full[:, :V]
    l.copy_(torch.randn((N, V), generator=g, device="cuda").mul_(1.5).add_(prior))
    tok = l.argmax(-1).int()
    some = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    tok = torch.where(torch.rand(N, generator=g, device="cuda") < 0.5, tok, some)
    if case["mask"]:
        hide = torch.rand((N, V), generator=g, device="cuda") < case["mask"]
        hide[torch.arange(N, device="cuda"), tok.long()] = False
        if N > 3:
            hide[1] = True   # a row whose mask leaves nothing
        l.masked_fill_(hide, -math.inf)
    if case["pad"]:   # rows that carry no token
        tok[torch.randperm(N, generator=g, device="cuda")[:case["pad"]]] = -1
    return l, tok


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda")  # noqa: E731
    if case["op"] in ("logp", "grad"):
        s["logits"], s["tokens"] = _logits(case, g)
    if case["op"] == "grad":   # what the forward pass left: each row's maximum and log sum, entropy, alternatives
        N, k = case["N"], case["top"]
        stats, ent = torch.zeros((N, 2), device="cuda"), torch.zeros(N, device="cuda")
        for a in range(0, N, 256):
            l = s["logits"][a:a + 256].double()
            m = l.amax(-1)
            z = (l - m[:, None]) / case["T"]
            stats[a:a + 256, 0], stats[a:a + 256, 1] = m, torch.logsumexp(z, -1)
            lp = torch.log_softmax(z, -1)
            ent[a:a + 256] = -(lp.exp() * lp.clamp(min=-1e300)).sum(-1).nan_to_num(0.0)
        s["stats"], s["entropy"] = stats, ent
        s["g_logp"], s["g_entropy"] = rnd(N), 0.1 * rnd(N)
        s["top_idx"] = torch.randint(0, case["V"], (N, k), generator=g, device="cuda", dtype=torch.int32) if k else None
        s["g_top"] = 0.2 * rnd(N, k) if k else None
    if case["op"] == "norm":
        dt = _DT[case["dtype"]]
        s["x"] = rnd(case["M"], case["d"]).to(dt)
        s["residual"] = (2.0 * rnd(case["M"], case["d"])).to(dt) if case["res"] else None
        s["gain"] = (1.0 + 0.1 * rnd(case["d"])).to(dt)
    if case["op"] == "head":
        M, N, K = case["M"], case["N"], case["K"]
        ld = -(-K // 16) * 16   # rows of 8-bit values start on 16 bytes
        q = torch.zeros((M, ld), dtype=torch.int8, device="cuda")
        w = torch.zeros((N, ld), dtype=torch.int8, device="cuda")
        q[:, :K] = (30.0 * rnd(M, K)).round_().clamp_(-127, 127)
        for a in range(0, N, 16384):
            n = min(16384, N - a)
            w[a:a + n, :K] = (30.0 * rnd(n, K)).round_().clamp_(-127, 127)
        s["q"], s["w"] = q[:, :K], w[:, :K]
        s["q_scale"] = 0.01 + 0.01 * torch.rand(M, generator=g, device="cuda")
        s["w_scale"] = 0.0005 + 0.001 * torch.rand(N, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def _ordered(x):
    """int32 with the order of fp32 values (-0 as +0)."""
    i = (x + 0.0).view(torch.int32)
    return i ^ ((i >> 31) & 0x7FFFFFFF)


def _plain_logp(s):
    l, tok, k, V = s["logits"].float(), s["tokens"], s["top"], s["V"]
    ml = l.amax(-1, keepdim=True)
    z, m = l * (1.0 / s["T"]), ml * (1.0 / s["T"])
    none = torch.isinf(m)[:, 0]   # no unmasked token in the row
    d = z - torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(d)
    S = e.sum(-1, dtype=torch.float64)
    logS = torch.log(S)
    ed = torch.where(e > 0, e * d, 0.0).sum(-1, dtype=torch.float64)
    live = tok >= 0
    ent = torch.where(live & ~none, (logS - ed / S).float(), 0.0)
    zt = l.gather(1, tok.clamp(min=0).long()[:, None])[:, 0] * (1.0 / s["T"])
    logp = torch.where(none, -math.inf, ((zt - m[:, 0]).double() - logS).float())
    logp = torch.where(live, logp, 0.0)
    stats = torch.where(live[:, None], torch.stack((ml[:, 0], logS.float()), 1), 0.0)
    out = {"logp": logp, "entropy": ent, "stats": stats}
    if k:
        key = (_ordered(l).long() << 32) | (V - 1 - torch.arange(V, device=l.device))
        idx = V - 1 - (torch.topk(key, k, -1).values & 0xFFFFFFFF)
        lt = l.gather(1, idx)
        gone = torch.isinf(lt) | ~live[:, None]
        out["top_idx"] = torch.where(gone, -1, idx).int()
        lp = ((lt * (1.0 / s["T"]) - m).double() - logS[:, None]).float()
        out["top_logp"] = torch.where(gone, -math.inf, lp)
    return out


def _plain_grad(s):
    l, tok = s["logits"], s["tokens"]
    m, logS = s["stats"][:, :1], s["stats"][:, 1:]
    fine = (tok >= 0) & torch.isfinite(m[:, 0])
    lp = (l.float() - m) * (1.0 / s["T"]) - logS
    p = torch.exp(lp)
    G = torch.where(fine, s["g_logp"] if s["g_top"] is None else s["g_logp"] + s["g_top"].sum(-1), 0.0)
    gH = torch.where(fine, s["g_entropy"], 0.0)
    d = -p * (G[:, None] + torch.where(p > 0, gH[:, None] * (lp + s["entropy"][:, None]), 0.0))
    one = torch.where(fine, s["g_logp"], 0.0)
    d.scatter_add_(1, tok.clamp(min=0).long()[:, None], one[:, None])
    if s["g_top"] is not None:
        d.scatter_add_(1, s["top_idx"].long(), torch.where(fine[:, None], s["g_top"], 0.0))
    d = torch.where(fine[:, None], d, 0.0)   # p of a row without a token is not defined
    return {"grad": (d * (1.0 / s["T"])).to(l.dtype)}


def _plain_norm(s):
    x, g = s["x"], s["gain"].float()
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    hf = h.float()
    inv = torch.rsqrt((hf * hf).mean(-1, keepdim=True) + 1e-6)
    v = hf * g
    A = v.abs().amax(-1, keepdim=True)
    q = torch.round(v * (torch.full_like(A, 127.0) / A))
    out = {"y": q * (A * inv * (1.0 / 127.0))}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_head(s):
    acc = s["q"].float() @ s["w"].float().t()
    return {"out": (acc * s["q_scale"][:, None] * s["w_scale"]).to(_DT[s["out"]])}


def _own(s):
    from speculative_decoding_04_b200 import dspark as D

    op = s["op"]
    if op == "logp":
        logp, ent, ti, tl, stats = D.token_logprobs(s["logits"], s["tokens"], s["T"], top=s["top"])
        out = {"logp": logp, "entropy": ent, "stats": stats}
        return {**out, "top_idx": ti, "top_logp": tl} if s["top"] else out
    if op == "grad":
        return {"grad": D.token_logprobs_backward(s["logits"], s["tokens"], s["T"], s["stats"], s["entropy"],
                                                  s["g_logp"], s["g_entropy"], top_idx=s["top_idx"],
                                                  g_top=s["g_top"])}
    if op == "norm":
        q, scale, h = D.rmsnorm_q8(s["x"], s["gain"], 1e-6, residual=s["residual"])
        out = {"y": q * scale[:, None]}
        return {**out, "h": h} if h is not None else out
    return {"out": D.matmul_q8(s["q"], s["q_scale"], s["w"], s["w_scale"], out_dtype=_DT[s["out"]])}


def run(state):
    if own:
        return _own(state)
    return {"logp": _plain_logp, "grad": _plain_grad, "norm": _plain_norm, "head": _plain_head}[state["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    """Each input read once, each output written once; the products' operations and, for the rest, the few
    operations an element takes. A row without a token need not be read (its gradient is written)."""
    if case["op"] == "logp":
        n, b = case["N"] - case["pad"], _SIZE[case["dtype"]]
        return {"bytes": n * case["V"] * b + case["N"] * (20 + 8 * case["top"]), "flops": 5 * n * case["V"]}
    if case["op"] == "grad":
        b = _SIZE[case["dtype"]]
        return {"bytes": (2 * case["N"] - case["pad"]) * case["V"] * b + case["N"] * (24 + 8 * case["top"]),
                "flops": 6 * (case["N"] - case["pad"]) * case["V"]}
    if case["op"] == "norm":
        b = _SIZE[case["dtype"]]
        per = b + 1 + (2 * b if case["res"] else 0)
        return {"bytes": case["M"] * case["d"] * per + 4 * case["M"] + b * case["d"], "flops": 6 * case["M"] * case["d"]}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": N * K + M * K + M * N * _SIZE[case["out"]] + 4 * (M + N), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logp":
        N, k = case["N"], case["top"]
        f = {n: [] for n in ("logp", "entropy", "stats", "top_logp")}
        for a in range(0, N, 256):
            t = s["tokens"][a:a + 256].long()
            z = s["logits"][a:a + 256].double() / case["T"]
            lse = torch.logsumexp(z, -1)
            lp = z - lse[:, None]
            dead, void = t < 0, torch.isinf(lse)
            lp[void] = -math.inf
            at = lp[torch.arange(len(t), device="cuda"), t.clamp(min=0)]
            p = lp.exp()
            H = -(p * lp.clamp(min=-1e300)).sum(-1)
            f["logp"].append(at.masked_fill(dead, 0))
            f["entropy"].append(H.masked_fill(dead | void, 0))
            m = s["logits"][a:a + 256].double().amax(-1)
            logS = torch.where(void, -math.inf, lse - m / case["T"])
            f["stats"].append(torch.stack((m, logS), 1).masked_fill(dead[:, None], 0))
            if k:
                f["top_logp"].append(torch.sort(lp, -1, descending=True).values[:, :k].masked_fill(dead[:, None], -math.inf))
        out = {n: torch.cat(v) for n, v in f.items() if v}
        if k:
            out["top_idx"] = None
        return out
    if case["op"] == "grad":
        parts = []
        for a in range(0, case["N"], 256):
            c = {n: v[a:a + 256] if torch.is_tensor(v) else v for n, v in s.items()}
            t = c["tokens"].long()
            z = c["logits"].double() / case["T"]
            p = torch.softmax(z, -1)
            lp = torch.log_softmax(z, -1).clamp(min=-1e300)
            gl, gh = c["g_logp"].double()[:, None], c["g_entropy"].double()[:, None]
            H = -(p * lp).sum(-1, keepdim=True)
            gr = -gl * p - gh * p * (lp + H)
            rows = torch.arange(len(t), device="cuda")
            gr[rows, t.clamp(min=0)] += gl[:, 0]
            if case["top"]:
                gt = c["g_top"].double()
                gr -= gt.sum(-1, keepdim=True) * p
                for j in range(case["top"]):
                    gr[rows, c["top_idx"][:, j].long()] += gt[:, j]
            gr /= case["T"]
            gr[(t < 0) | torch.isinf(z.amax(-1))] = 0
            parts.append(gr)
        return {"grad": torch.cat(parts)}
    if case["op"] == "norm":
        h = s["x"].double()
        if case["res"]:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        inv = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6)
        # the grid is defined on the fp32 products h*g and 127/max: which step a value takes is not rounding noise
        v = (h * s["gain"].double()).float()
        A = v.abs().amax(-1, keepdim=True).double()
        q = torch.round((v.double() * (127 / A).float().double()).float()).double()
        out = {"y": q * A * inv / 127}
        if case["res"]:
            out["h"] = h
        return out
    if case["M"] * case["N"] > 700_000_000:
        return None
    q = s["q"].double() * s["q_scale"].double()[:, None]
    parts = [q @ s["w"][a:a + 16384].double().t() for a in range(0, case["N"], 16384)]
    return {"out": torch.cat(parts, 1) * s["w_scale"].double()}
