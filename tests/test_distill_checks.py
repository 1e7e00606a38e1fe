"""Refusals of the distillation calls: the C ABI returns its documented status before any HIP call, the
binding raises before it enters the library, and without a device a call returns FAIRY2I_ERR_HIP.  No GPU
needed."""
import os

import pytest
import torch

import widely_linear_gemv_amd as f2

FAKE = 1 << 20          # a 16-byte aligned, never dereferenced address
Y, Z = 1 << 40, 1 << 41
ODD = FAKE + 2
S = None


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(f2.LIB_PATH):
        from widely_linear_gemv_amd import build
        build.build()
    return f2.lib()


def loss_args(**kw):
    a = dict(h=FAKE, W=FAKE, xd=1, N=4, V=100, K=64, ti=FAKE, tl=FAKE, td=0, top=8, T=1.0, loss=Y, lse=Z, ws=FAKE,
             wsb=1 << 40, st=S)
    a.update(kw)
    return list(a.values())


def grad_args(**kw):
    a = dict(h=FAKE, W=FAKE, xd=1, N=4, V=100, K=64, ti=FAKE, tl=FAKE, td=0, top=8, T=1.0, lse=FAKE, g=FAKE, dh=Y, dW=Z,
             ws=FAKE, wsb=1 << 40, st=S)
    a.update(kw)
    return list(a.values())


COMMON = [(dict(h=None), 1), (dict(W=None), 1), (dict(ti=None), 1), (dict(tl=None), 1), (dict(lse=None), 1),
          (dict(xd=2), 4), (dict(td=3), 4), (dict(td=-1), 4), (dict(N=0), 2), (dict(V=0), 2), (dict(K=96), 2), (dict(K=0), 2),
          (dict(N=1 << 20, V=(1 << 16) + 1), 2), (dict(top=0), 2), (dict(top=129), 2), (dict(top=-1), 2),
          (dict(T=0.0), 2), (dict(T=-1.0), 2), (dict(T=float("nan")), 2), (dict(T=float("inf")), 2), (dict(T=2.0 ** -21), 2),
          (dict(h=ODD), 5), (dict(W=FAKE + 8), 5), (dict(ti=FAKE + 4), 5), (dict(tl=ODD), 5), (dict(tl=FAKE + 1, td=1), 5),
          (dict(lse=ODD), 5), (dict(ws=None), 6), (dict(wsb=64), 6), (dict(ws=FAKE + 8), 5)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(loss=None), 1), (dict(loss=ODD), 5), (dict(lse=Y), 2), (dict(lse=Y + 12), 2), (dict(loss=FAKE), 2), (dict(ti=Y), 2),
    (dict(tl=Z), 2), (dict(h=Z), 2), (dict(W=Y), 2)])
def test_loss_errors(L, kw, status):
    assert L.fairy2i_distill(*loss_args(**kw)) == status
    assert f2.fairy2i_last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(g=None), 1), (dict(dh=None, dW=None), 1), (dict(dh=ODD), 5), (dict(dW=ODD), 5), (dict(g=ODD), 5), (dict(dh=FAKE), 2),
    (dict(ti=Y), 2), (dict(tl=Z + 16), 2), (dict(lse=Z), 2), (dict(g=Y), 2), (dict(dW=Y + 64), 2), (dict(h=Z), 2), (dict(W=Y), 2)])
def test_gradient_errors(L, kw, status):
    assert L.fairy2i_distill_backward(*grad_args(**kw)) == status
    assert f2.fairy2i_last_error()


def test_workspaces(L):
    """0 for sizes out of range; the lists are part of it; an untouched vocabulary loss needs none of them."""
    loss, grad = f2.fairy2i_distill_workspace_bytes, f2.fairy2i_distill_backward_workspace_bytes
    for bad in ((0, 100, 64, 1, 8), (4, 100, 65, 1, 8), (4, 100, 64, 1, 0), (4, 100, 64, 1, 129)):
        assert loss(*bad) == 0 and grad(*bad) == 0
    for code in (f2.F32, f2.BF16):
        assert loss(2048, 32000, 4096, code, 32) >= f2.fairy2i_vocab_loss_workspace_bytes(2048, 32000, 4096, code) + 2048 * 31 * 4
        assert grad(2048, 32000, 4096, code, 32) >= f2.fairy2i_vocab_loss_backward_workspace_bytes(2048, 32000, 4096, code) + 2048 * 32 * 8


def test_without_a_device(L):
    if torch.cuda.device_count() != 0:
        pytest.skip("a device is visible")
    assert L.fairy2i_distill(*loss_args()) == 7 and f2.fairy2i_last_error()
    assert L.fairy2i_distill_backward(*grad_args()) == 7 and f2.fairy2i_last_error()


def raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_binding_checks():
    h, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(100, 64, dtype=torch.bfloat16)
    index, logit = torch.zeros(4, 8, dtype=torch.int64), torch.zeros(4, 8)
    f = f2.fairy2i_distill
    raises("dtype", f, h.double(), W, index, logit)
    raises("dtype", f, h, W.float(), index, logit)
    raises("shape", f, h[0], W, index, logit)
    raises("shape", f, h, W[:, :32], index, logit)
    raises("dtype", f, h, W, index.int(), logit)
    raises("shape", f, h, W, index[:3], logit)
    raises("shape", f, h, W, index, logit[:, :7])
    raises("dtype", f, h, W, index, logit.half())
    raises("contiguous", f, h, W, torch.zeros(8, 4, dtype=torch.int64).t(), logit)
    raises("contiguous", f, h, W, index, torch.zeros(8, 4).t())
    raises("shape", f, h, W, index, logit, loss=torch.zeros(5))
    raises("dtype", f, h, W, index, logit, lse=torch.zeros(4).double())
    raises("GPU", f, h, W, index, logit)
    b, lse, g = f2.fairy2i_distill_backward, torch.zeros(4), torch.zeros(4)
    raises("dtype", b, h, W, index, logit, lse.double(), g)
    raises("shape", b, h, W, index, logit, lse, g[:3])
    raises("nothing", b, h, W, index, logit, lse, g, want_dh=False, want_dW=False)
    raises("not wanted", b, h, W, index, logit, lse, g, want_dh=False, dh=h)
    raises("shape", b, h, W, index, logit, lse, g, dW=W[:-1])
    raises("dtype", b, h, W, index, logit, lse, g, dh=h.float())
    raises("GPU", b, h, W, index, logit, lse, g)
