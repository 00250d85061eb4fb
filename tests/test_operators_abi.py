"""Argument checks of the LM head and log-probability entry points (no GPU needed): every bad argument is
found on the host, before anything is launched."""

import ctypes

import pytest
import torch

from speculative_decoding_04_b200 import build

build.build()
from speculative_decoding_04_b200 import dspark as D  # noqa: E402

# a fake device address: only ever reaches argument checks that fail before any launch
FAKE = 4096 * 256
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers are only passed where no GPU exists")


def call(fn, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(D.lib, fn)(*a.values())


LP = dict(logits=FAKE, dtype=D.F32, ld=1000, n_rows=8, rows=None, tokens=FAKE, N=8, V=1000, T=1.0, top=4, logp=FAKE,
          entropy=None, top_idx=FAKE, top_logp=FAKE, stats=FAKE, flags=None, stream=None)
LB = dict(logits=FAKE, dtype=D.F32, ld=1000, tokens=FAKE, N=8, V=1000, T=1.0, stats=FAKE, entropy=FAKE, g_logp=FAKE,
          g_entropy=FAKE, top=2, top_idx=FAKE, g_top=FAKE, grad=FAKE + (1 << 24), ldg=1000, stream=None)
NQ = dict(x=FAKE, dtype=D.BF16, ldx=64, res=FAKE, ldr=64, gain=FAKE, gain_dtype=D.F32, M=4, d=64, eps=1e-6,
          h=FAKE + (1 << 24), ldh=64, q=FAKE, ldq=64, scale=FAKE, stream=None)
QQ = dict(x=FAKE, dtype=D.F16, ldx=64, M=4, d=64, q=FAKE, ldq=64, scale=FAKE, stream=None)
MM = dict(q=FAKE, ldq=64, q_scale=FAKE, w=FAKE, ldw=64, w_scale=FAKE, M=4, N=100, K=64, out=FAKE, out_dtype=D.F32,
          ldo=100, flags=None, stream=None)


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(dtype=7), "dtype"), (dict(N=-1), "N"), (dict(V=0), "V"), (dict(V=(1 << 21) + 1, ld=1 << 22), "2^21"),
    (dict(ld=999), "ld"), (dict(n_rows=7), "rows"), (dict(n_rows=-1, rows=FAKE), "rows"), (dict(ld=1 << 62), "large"),
    (dict(T=0.0), "T"), (dict(T=float("nan")), "T"), (dict(T=float("inf")), "T"), (dict(T=1e-7), "T"),
    (dict(top=33), "top"), (dict(top=-1), "top"), (dict(logits=None), "null"), (dict(tokens=None), "null"),
    (dict(logp=None), "null"), (dict(top_idx=None), "top_idx"), (dict(top_logp=None), "top_logp"),
    (dict(logits=FAKE + 2), "aligned"), (dict(stats=FAKE + 4), "8-byte"), (dict(N=1 << 27, n_rows=1 << 27), "2^26")])
def test_token_logprobs_refuses(kw, word):
    assert call("dspark_token_logprobs", LP, **kw) == D.EINVAL
    assert word in D.last_error()


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(dtype=-1), "dtype"), (dict(N=-2), "N"), (dict(V=0), "V"), (dict(ldg=999), "ldg"), (dict(ld=10), "ld"),
    (dict(T=-1.0), "T"), (dict(top=40), "top"), (dict(stats=None), "null"), (dict(grad=None), "null"),
    (dict(entropy=None), "entropy"), (dict(g_top=None), "g_top"), (dict(top_idx=None), "top_idx"),
    (dict(stats=FAKE + 4), "8-byte"), (dict(grad=FAKE + 4), "overlaps"), (dict(grad=FAKE, ldg=1001), "overlaps"),
    (dict(grad=FAKE + 8 * 4000 - 4), "overlaps"), (dict(grad=FAKE + 2), "aligned")])
def test_token_logprobs_backward_refuses(kw, word):
    assert call("dspark_token_logprobs_backward", LB, **kw) == D.EINVAL
    assert word in D.last_error()


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(dtype=5), "dtype"), (dict(gain_dtype=D.F16), "gain_dtype"), (dict(M=-1), "M"), (dict(d=0), "d"),
    (dict(ldx=63), "stride"), (dict(ldq=63), "stride"), (dict(ldr=63), "stride"), (dict(ldh=63), "stride"),
    (dict(eps=0.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(x=None), "null"),
    (dict(q=None), "null"), (dict(scale=None), "null"), (dict(h=None), "null"), (dict(x=FAKE + 1), "aligned"),
    (dict(gain=FAKE + 2), "aligned"), (dict(h=FAKE + 64), "overlaps"), (dict(h=FAKE, ldh=65), "overlaps")])
def test_rmsnorm_q8_refuses(kw, word):
    assert call("dspark_rmsnorm_q8", NQ, **kw) == D.EINVAL
    assert word in D.last_error()


@no_gpu
@pytest.mark.parametrize("kw,word", [(dict(dtype=9), "dtype"), (dict(d=0), "d"), (dict(ldx=3), "stride"),
                                     (dict(x=None), "null"), (dict(x=FAKE + 1), "aligned")])
def test_quantize_q8_refuses(kw, word):
    assert call("dspark_quantize_q8", QQ, **kw) == D.EINVAL
    assert word in D.last_error()


@no_gpu
@pytest.mark.parametrize("kw,word", [
    (dict(out_dtype=3), "out_dtype"), (dict(M=-1), "M"), (dict(N=0), "N"), (dict(K=0), "K"),
    (dict(K=131072, ldq=131072, ldw=131072), "131071"), (dict(ldq=48), "stride"), (dict(ldw=48), "stride"),
    (dict(ldo=99), "stride"), (dict(ldq=72), "multiples of 16"), (dict(ldw=65), "multiples of 16"),
    (dict(ldq=1 << 41), "large"), (dict(q=None), "null"), (dict(w_scale=None), "null"), (dict(out=None), "null"),
    (dict(q=FAKE + 8), "16-byte"), (dict(w=FAKE + 1), "16-byte"), (dict(out=FAKE + 2), "aligned"),
    (dict(M=1 << 30, N=1 << 30, ldo=1 << 30), "large")])
def test_matmul_q8_refuses(kw, word):
    assert call("dspark_matmul_q8", MM, **kw) == D.EINVAL
    assert word in D.last_error()


@no_gpu
def test_empty_batches_return_before_anything_is_launched():
    assert call("dspark_token_logprobs", LP, N=0, logits=None, tokens=None, logp=None) == D.OK
    assert call("dspark_token_logprobs_backward", LB, N=0, logits=None, grad=None) == D.OK
    assert call("dspark_rmsnorm_q8", NQ, M=0, x=None) == D.OK
    assert call("dspark_quantize_q8", QQ, M=0, x=None) == D.OK
    assert call("dspark_matmul_q8", MM, M=0, q=None) == D.OK


def test_new_symbols_are_declared():
    assert {"dspark_token_logprobs", "dspark_token_logprobs_backward", "dspark_rmsnorm_q8", "dspark_quantize_q8",
            "dspark_matmul_q8"} <= set(D.declared_functions())
    assert D.TOP_MAX == 32 and ctypes.sizeof(ctypes.c_int64) == 8


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 64))
    i8 = torch.zeros((4, 64), dtype=torch.int8)
    tok = torch.zeros(4, dtype=torch.int32)
    for f in (lambda: D.token_logprobs(x, tok), lambda: D.rmsnorm_q8(x, None, 1e-6), lambda: D.quantize_q8(x),
              lambda: D.matmul_q8(i8, x[:, 0], i8, x[:, 0]),
              lambda: D.token_logprobs_backward(x, tok, 1.0, x[:, :2], None, x[:, 0])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        D.token_logprobs(x.numpy(), tok)


@no_gpu
def test_rmsnorm_q8_refuses_an_eps_among_the_denormals():
    assert call("dspark_rmsnorm_q8", NQ, eps=1e-38) == D.EINVAL and "eps" in D.last_error()


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda:1")
    x = torch.zeros((4, 64))
    i8 = torch.zeros((4, 64), dtype=torch.int8)
    tok = torch.zeros(4, dtype=torch.int32)
    for f in (lambda **k: D.token_logprobs(x, tok, **k), lambda **k: D.rmsnorm_q8(x, None, 1e-6, **k),
              lambda **k: D.quantize_q8(x, **k), lambda **k: D.matmul_q8(i8, x[:, 0], i8, x[:, 0], **k),
              lambda **k: D.token_logprobs_backward(x, tok, 1.0, x[:, :2], None, x[:, 0], **k)):
        with pytest.raises(ValueError, match="stream"):
            f(stream=Stream())
