"""Refusals of the operators over rows of logits that need no GPU: the C ABI rejects invalid
arguments before it touches CUDA, the binding before it calls the library."""
import ctypes

import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
from layernorm_ln_fwd_gb300 import build as lnbuild

N = None


@pytest.fixture(scope="module")
def lib():
    lnbuild.build()
    return ln.lib()


P = ctypes.c_void_p(256)  # never dereferenced: validation fails first


def test_logprobs_arguments(lib):
    for f in (lib.ln_logprobs_f32, lib.ln_logprobs_bf16):
        def call(x=P, ld=8, tok=P, rows=4, V=8, scale=1.0, top=0, logp=P, ent=N, lse=N, ranks=N, ids=N, lp=N):
            return f(x, ld, tok, rows, V, scale, top, logp, ent, lse, ranks, ids, lp, N)
        assert call(x=N) == 1 and call(tok=N) == 1 and call(logp=N) == 1
        assert call(rows=-1) == 1 and call(V=0) == 1 and call(ld=7) == 1
        for bad in (0.0, -1.0, float("inf"), float("nan"), 3e38):  # (3e38 log2 e is not finite)
            assert call(scale=bad) == 1
        assert call(top=-1) == 1 and call(top=2) == 1 and call(top=2, ids=P) == 1 and call(top=2, lp=P) == 1
        assert call(ids=P, lp=P) == 1  # alternatives of none
        assert call(top=ln.MAX_TOP + 1, ids=P, lp=P) == 3
        assert call(V=(1 << 24) + 1, ld=1 << 25) == 3 and call(rows=2**31 - 2**16 + 1) == 3
        assert call(ld=2**62) == 1  # row addresses beyond 64 bits
        assert call(tok=N, logp=N, ranks=P) == 1
        assert call(x=N, tok=N, rows=0, logp=N) == 0


def test_logprobs_bwd_arguments(lib):
    for f in (lib.ln_logprobs_bwd_f32, lib.ln_logprobs_bwd_bf16):
        def call(x=P, ld=8, tok=P, lse=P, ent=N, dl=P, de=N, rows=4, V=8, scale=1.0, dx=P, ldd=8):
            return f(x, ld, tok, lse, ent, dl, de, rows, V, scale, dx, ldd, N)
        assert call(x=N) == 1 and call(tok=N) == 1 and call(lse=N) == 1 and call(dx=N) == 1
        assert call(dl=N) == 1 and call(de=P) == 1  # no upstream gradient; no entropy for it
        assert call(ld=7) == 1 and call(ldd=7) == 1 and call(scale=0.0) == 1
        assert call(ldd=9) == 1  # in place, but rows elsewhere
        assert call(V=(1 << 24) + 1, ld=1 << 25, ldd=1 << 25) == 3
        assert call(x=N, tok=N, lse=N, dl=N, rows=0, dx=N) == 0


def test_distill_arguments(lib):
    for f in (lib.ln_distill_f32, lib.ln_distill_bf16):
        def call(x=P, ld=8, ids=P, t=P, w=N, rows=4, V=8, K=3, scale=1.0, dloss=1.0, loss=P, dx=N, ldd=8):
            return f(x, ld, ids, t, w, rows, V, K, scale, dloss, loss, dx, ldd, N)
        assert call(x=N) == 1 and call(ids=N) == 1 and call(t=N) == 1 and call(loss=N) == 1
        assert call(K=0) == 1 and call(K=ln.MAX_TOP + 1) == 3
        assert call(scale=-1.0) == 1 and call(dloss=float("nan")) == 1
        assert call(ld=7) == 1 and call(dx=ctypes.c_void_p(512), ldd=7) == 1 and call(dx=P, ldd=9) == 1
        assert call(V=(1 << 24) + 1, ld=1 << 25) == 3
        assert call(x=N, ids=N, t=N, rows=0, loss=N) == 0
    assert lib.ln_last_launch_count() == 0


def test_binding_refuses_tensors_of_the_host():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    for call in (lambda: ln.logprobs(x, t), lambda: ln.logprobs_bwd(x, t, f, dlogp=f),
                 lambda: ln.distill(x, t[:, None], f[:, None])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        ln.logprobs(x.double(), t)
    with pytest.raises(ValueError):
        ln.logprobs(x.t(), t)
    with pytest.raises(ValueError):
        ln.logprobs(x[0], t)
    with pytest.raises(ValueError):
        ln.distill(x, t, f)
