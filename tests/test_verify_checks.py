"""Refusals of the draft verification call: the C ABI returns its documented status before any HIP call, the
binding raises before it enters the library, and without a device the call returns FAIRY2I_ERR_HIP.  No GPU
needed."""
import os

import pytest
import torch

import widely_linear_gemv_amd as f2

FAKE = 1 << 20          # a 16-byte aligned, never dereferenced address
Y, Z = 1 << 44, 1 << 45
STREAM = None


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(f2.LIB_PATH):
        from widely_linear_gemv_amd import build
        build.build()
    return f2.lib()


def args(**kw):
    a = dict(p=FAKE, q=FAKE, dt=0, S=3, D=4, V=100, draft=FAKE, len=FAKE, u=FAKE, r=FAKE, tokens=Y, accepted=Z, ws=FAKE,
             wsb=1 << 40, st=STREAM)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(p=None), 1), (dict(draft=None), 1), (dict(u=None), 1), (dict(r=None), 1), (dict(tokens=None), 1), (dict(accepted=None), 1),
    (dict(dt=2), 4), (dict(dt=-1), 4), (dict(S=0), 2), (dict(S=(1 << 20) + 1, V=1), 2), (dict(D=0), 2), (dict(D=64), 2),
    (dict(V=0), 2), (dict(V=(1 << 24) + 1, S=1), 2), (dict(S=2049, V=1 << 24), 2),
    (dict(p=FAKE + 2), 5), (dict(q=FAKE + 1, dt=1), 5), (dict(draft=FAKE + 4), 5), (dict(len=FAKE + 2), 5), (dict(u=FAKE + 2), 5),
    (dict(r=FAKE + 1), 5), (dict(tokens=Y + 4), 5), (dict(accepted=Z + 2), 5), (dict(ws=FAKE + 8), 5),
    (dict(ws=None, V=131072), 6), (dict(wsb=16, V=131072), 6),
    (dict(p=Y), 2), (dict(q=Z), 2), (dict(draft=Y + 8), 2), (dict(len=Z + 4), 2), (dict(u=Y), 2), (dict(r=Z), 2),
    (dict(accepted=Y + 3 * 5 * 8 - 4), 2), (dict(p=Y - 3 * 5 * 100 * 4 + 4), 2)])
def test_errors(L, kw, status):
    assert L.fairy2i_verify_draft(*args(**kw)) == status
    assert f2.fairy2i_last_error()


def test_workspace(L):
    """None where a sequence has a workgroup to itself."""
    assert f2.fairy2i_verify_draft_workspace_bytes(3, 4, 4097) == 0
    assert f2.fairy2i_verify_draft_workspace_bytes(3, 4, 131072) == 3 * (64 + 2) * 8
    assert f2.fairy2i_verify_draft_workspace_bytes(3, 64, 4097) == 0


def test_without_a_device(L):
    if torch.cuda.device_count() != 0:
        pytest.skip("a device is visible")
    assert L.fairy2i_verify_draft(*args()) == 7 and f2.fairy2i_last_error()
    assert L.fairy2i_verify_draft(*args(q=None, len=None)) == 7


def raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_binding_checks():
    f = f2.fairy2i_verify_draft
    p, q, x, u, r = torch.zeros(3, 5, 100), torch.zeros(3, 4, 100), torch.zeros(3, 4, dtype=torch.int64), torch.zeros(3, 4), torch.zeros(3)
    raises("dtype", f, p.double(), q, x, u, r)
    raises("shape", f, p[0], q, x, u, r)
    raises("shape", f, p[:, :1].contiguous(), None, x, u, r)
    raises("contiguous", f, torch.zeros(5, 3, 100).transpose(0, 1), q, x, u, r)
    raises("dtype", f, p, q.bfloat16(), x, u, r)
    raises("shape", f, p, p, x, u, r)
    raises("dtype", f, p, q, x.int(), u, r)
    raises("shape", f, p, q, x[:, :3], u, r)
    raises("dtype", f, p, q, x, u.double(), r)
    raises("shape", f, p, q, x, u, u)
    raises("dtype", f, p, q, x, u, r, draft_len=torch.zeros(3, dtype=torch.int64))
    raises("shape", f, p, q, x, u, r, tokens=x)
    raises("dtype", f, p, q, x, u, r, accepted=torch.zeros(3))
    raises("GPU", f, p, q, x, u, r)
    raises("GPU", f, p, None, x, u, r)
    with pytest.raises(TypeError):
        f(p, q, None, u, r)
    with pytest.raises(TypeError):
        f(None, q, x, u, r)
