"""Refusals of the operators beside the packed layers (low-rank adapters, vocabulary loss, gradient
clipping): the C ABI returns its documented status before any HIP call, the binding raises before it
enters the library, and without a device every call returns FAIRY2I_ERR_HIP.  No GPU needed."""
import ctypes
import json
import math
import os
import subprocess
import sys

import pytest
import torch

import widely_linear_gemv_amd as f2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # a 16-byte aligned, never dereferenced address
ODD = FAKE + 2
Y, Z, Q = (FAKE + (k << 20) for k in (1, 2, 3))      # outputs, apart from the inputs
S = None


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(f2.LIB_PATH):
        from widely_linear_gemv_amd import build
        build.build()
    return f2.lib()


def lora_args(**kw):
    a = dict(x=FAKE, x_dtype=1, N=4, m=64, A=FAKE, B=FAKE, alpha=FAKE, L=2, r=8, n=32, ss=FAKE, sa=FAKE, S=2, base=Y,
             y=Y, y_dtype=0, ws=FAKE, wsb=1 << 30, st=S)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(alpha=None), 1), (dict(base=None), 1),
    (dict(y=None), 1), (dict(ss=None), 1), (dict(sa=None), 1),
    (dict(x_dtype=2), 4), (dict(y_dtype=3), 4), (dict(x_dtype=-1), 4),
    (dict(N=0), 2), (dict(N=(1 << 20) + 1), 2), (dict(m=32), 2), (dict(m=65), 2), (dict(m=(1 << 20) + 64), 2),
    (dict(n=0), 2), (dict(n=(1 << 20) + 1), 2), (dict(L=0), 2), (dict(L=4097), 2), (dict(r=0), 2), (dict(r=129), 2),
    (dict(S=0), 2), (dict(S=(1 << 20) + 1), 2),
    (dict(x=ODD), 5), (dict(A=ODD), 5), (dict(B=FAKE + 8), 5), (dict(base=ODD), 5), (dict(y=ODD), 5), (dict(ss=ODD), 5),
    (dict(ws=FAKE + 8), 5), (dict(ws=None), 6), (dict(wsb=8), 6),
    (dict(y=FAKE, base=FAKE), 2), (dict(y=Y + 16), 2),                          # y on x; y on part of base
])
def test_lora_errors(L, kw, status):
    assert L.fairy2i_lora(*lora_args(**kw)) == status
    assert f2.fairy2i_last_error()


def test_lora_grouped_errors(L):
    items = (f2.LoraItem * 2)(f2.LoraItem(FAKE, FAKE, FAKE, Y, Y, 32), f2.LoraItem(FAKE, FAKE, FAKE, Y, None, 32))
    call = lambda it, count: L.fairy2i_lora_grouped(it, count, FAKE, 1, 4, 64, 2, 8, FAKE, FAKE, 2, 0, FAKE, 1 << 30, S)
    assert call(None, 1) == 1
    assert call(items, 0) == 2
    assert call(items, 2) == 1 and "item 1" in f2.fairy2i_last_error()
    items[1].y, items[1].n = Y, 0
    assert call(items, 2) == 2
    items[1].n, items[1].B = 32, ODD
    assert call(items, 2) == 5
    items[1].B = FAKE
    assert call(items, 2) == 2 and "overlaps" in f2.fairy2i_last_error()       # both write one y
    items[1].base = items[1].y = Z
    items[0].base = items[0].y = Z + 64
    assert call(items, 2) == 2                                                  # some bytes in common
    items[0].base, items[0].y = Z, Y
    assert call(items, 2) == 2                                                  # item 1's y is item 0's base


def test_lora_refuses_y_over_the_adapters(L):
    """Workgroups that store y run beside others that still read A, B, alpha and the segments."""
    far, y_bytes = 1 << 30, 4 * 64 * 4
    size = {"A": 2 * 8 * 128 * 2, "B": 2 * 64 * 8 * 2, "alpha": 2 * 4, "ss": 3 * 4, "sa": 2 * 4}
    for name, nbytes in size.items():
        for at in (far, far - (nbytes - 1) // 16 * 16, far + y_bytes - 16):
            assert L.fairy2i_lora(*lora_args(y=far, **{name: at})) == 2, (name, at - far)
            assert "overlaps" in f2.fairy2i_last_error()
    # an item's y over another item's adapters
    for name in ("A", "B", "alpha"):
        items = (f2.LoraItem * 2)(f2.LoraItem(FAKE, FAKE, FAKE, Y, Y, 32), f2.LoraItem(FAKE, FAKE, FAKE, Z, Z, 32))
        setattr(items[1], name, Y)
        assert L.fairy2i_lora_grouped(items, 2, FAKE, 1, 4, 64, 2, 8, FAKE, FAKE, 2, 0, FAKE, 1 << 30, S) == 2, name
        items = (f2.LoraItem * 2)(f2.LoraItem(FAKE, FAKE, FAKE, Y, Y, 32), f2.LoraItem(FAKE, FAKE, FAKE, Z, Z, 32))
        setattr(items[0], name, Z)
        assert L.fairy2i_lora_grouped(items, 2, FAKE, 1, 4, 64, 2, 8, FAKE, FAKE, 2, 0, FAKE, 1 << 30, S) == 2, name


def back_args(**kw):
    a = dict(dy=FAKE, x=FAKE, x_dtype=1, N=4, m=64, A=FAKE, B=FAKE, alpha=FAKE, L=2, r=8, n=32, ss=FAKE, sa=FAKE, S=2,
             dxb=Y, dx=Y, dx_dtype=0, dA=Q, dB=Z, ws=FAKE, wsb=1 << 40, st=S)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(x=None), 1), (dict(dA=None), 1), (dict(dB=None), 1), (dict(dx=None), 1), (dict(dxb=None), 1),
    (dict(x_dtype=2), 4), (dict(dx_dtype=2), 4), (dict(N=0), 2), (dict(m=96), 2), (dict(n=0), 2), (dict(L=0), 2),
    (dict(r=129), 2), (dict(S=0), 2), (dict(dy=ODD), 5), (dict(dA=FAKE + 4), 5), (dict(dx=ODD), 5), (dict(ws=None), 6),
    (dict(wsb=64), 6), (dict(dx=FAKE, dxb=FAKE), 2), (dict(dx=Y + 64), 2), (dict(dy=Y), 2),
    (dict(dA=FAKE), 2), (dict(dB=FAKE), 2), (dict(dA=Z + 64), 2), (dict(dB=Y), 2),
])
def test_lora_backward_errors(L, kw, status):
    assert L.fairy2i_lora_backward(*back_args(**kw)) == status


def test_lora_backward_refuses_outputs_over_inputs(L):
    """dx is written while A, B, alpha and the segments may still be read, dA and dB while the segments are."""
    far, out_bytes = 1 << 30, {"dx": 4 * 128 * 4, "dA": 2 * 8 * 128 * 4, "dB": 2 * 64 * 8 * 4}
    size = {"A": 2 * 8 * 128 * 2, "B": 2 * 64 * 8 * 2, "alpha": 2 * 4, "ss": 3 * 4, "sa": 2 * 4}
    for out, nbytes in out_bytes.items():
        for name, have in size.items():
            for at in (far, far - (have - 1) // 16 * 16, far + nbytes - 16):
                kw = {out: far, name: at, **({"dxb": far} if out == "dx" else {})}
                assert L.fairy2i_lora_backward(*back_args(**kw)) == 2, (out, name, at - far)
                assert "overlaps" in f2.fairy2i_last_error()


def loss_args(**kw):
    a = dict(h=FAKE, W=FAKE, dt=1, N=4, V=100, K=64, t=FAKE, loss=Y, lse=Z, ws=FAKE, wsb=1 << 30, st=S)
    a.update(kw)
    return list(a.values())


def grad_args(**kw):
    a = dict(h=FAKE, W=FAKE, dt=1, N=4, V=100, K=64, t=FAKE, lse=FAKE, g=FAKE, dh=Y, dW=Z, ws=FAKE, wsb=1 << 40, st=S)
    a.update(kw)
    return list(a.values())


SIZES = [(dict(N=0), 2), (dict(V=0), 2), (dict(K=0), 2), (dict(K=96), 2), (dict(K=65600), 2), (dict(N=(1 << 20) + 1), 2),
         (dict(V=(1 << 24) + 1), 2), (dict(N=1 << 16, V=(1 << 20) + 1), 2), (dict(dt=2), 4), (dict(h=ODD), 5),
         (dict(W=ODD), 5), (dict(t=FAKE + 4), 5), (dict(ws=None), 6), (dict(wsb=16), 6)]


@pytest.mark.parametrize("kw,status", SIZES + [(dict(h=None), 1), (dict(W=None), 1), (dict(t=None), 1), (dict(loss=None), 1),
                                               (dict(lse=None), 1), (dict(loss=ODD), 5), (dict(loss=Z + 12), 2),
                                               (dict(lse=FAKE), 2), (dict(t=Y), 2)])
def test_vocab_loss_errors(L, kw, status):
    assert L.fairy2i_vocab_loss(*loss_args(**kw)) == status


@pytest.mark.parametrize("kw,status", SIZES + [(dict(lse=None), 1), (dict(g=None), 1), (dict(dh=None, dW=None), 1),
                                               (dict(dh=ODD), 5), (dict(dW=ODD), 5), (dict(g=ODD), 5),
                                               (dict(dh=FAKE), 2), (dict(dW=FAKE), 2), (dict(dh=Z + 64), 2)])
def test_vocab_loss_backward_errors(L, kw, status):
    assert L.fairy2i_vocab_loss_backward(*grad_args(**kw)) == status


def test_vocab_loss_backward_refuses_outputs_over_inputs(L):
    """target, lse and g are read for every piece of the vocabulary, after the first ones' dW is stored."""
    far = 1 << 30
    size = {"target": 4 * 8, "lse": 4 * 4, "g": 4 * 4}
    for out, nbytes in (("dh", 4 * 64 * 2), ("dW", 100 * 64 * 2)):
        for name, key in (("target", "t"), ("lse", "lse"), ("g", "g")):
            for at in (far, far - size[name] + 8, far + nbytes - 8):
                call = L.fairy2i_vocab_loss_backward(*grad_args(**{out: far, key: at}))
                assert call == 2 and "overlap" in f2.fairy2i_last_error(), (out, name, at - far)


def test_clip_errors(L):
    ptrs = lambda *v: (ctypes.c_void_p * len(v))(*v)
    num = lambda *v: (ctypes.c_int64 * len(v))(*v)
    dts = lambda *v: (ctypes.c_int * len(v))(*v)
    c = lambda count=2, g=ptrs(FAKE, FAKE), o=None, n=num(8, 8), d=dts(0, 1), mx=1.0, norm=FAKE, ws=FAKE, wsb=1 << 20: \
        L.fairy2i_clip_grads(count, g, o, n, d, mx, norm, ws, wsb, S)
    assert c(count=-1) == 2
    assert c(norm=None) == 1 and c(g=None) == 1 and c(n=None) == 1 and c(d=None) == 1
    assert c(mx=-1.0) == 2 and c(mx=math.nan) == 2
    assert c(n=num(8, -1)) == 2
    assert c(d=dts(0, 2)) == 4
    assert c(g=ptrs(FAKE, None)) == 1 and c(o=ptrs(FAKE, None)) == 1
    assert c(g=ptrs(FAKE + 2, FAKE)) == 5           # fp32 needs 4 bytes
    assert c(g=ptrs(FAKE, FAKE + 1)) == 5           # bf16 needs 2
    assert c(ws=None) == 6 and c(wsb=16) == 6
    # 8 fp32 and 8 bf16 values: 32 and 16 bytes
    assert c() == 2 and "twice" in f2.fairy2i_last_error()
    assert c(g=ptrs(FAKE, FAKE + 28)) == 2 and c(g=ptrs(FAKE + 12, FAKE)) == 2
    assert c(g=ptrs(FAKE, Z), o=ptrs(Y, Y)) == 2                    # one output for two gradients
    assert c(g=ptrs(FAKE, Z), o=ptrs(Z, Y)) == 2                    # written over the other gradient
    assert c(g=ptrs(FAKE, Z), o=ptrs(FAKE + 16, Y)) == 2            # over part of its own
    assert c(g=ptrs(FAKE, FAKE), o=ptrs(FAKE, Y)) == 2              # read by the second, clipped by the first


def test_workspace_sizes_of_refused_shapes_are_zero():
    assert f2.fairy2i_lora_workspace_bytes(1, 0, 64, 8, 1) == 0
    assert f2.fairy2i_lora_workspace_bytes(1, 4, 65, 8, 1) == 0
    assert f2.fairy2i_lora_backward_workspace_bytes(4, 64, 32, 0, 8, 1, f2.BF16) == 0
    assert f2.fairy2i_vocab_loss_workspace_bytes(4, 100, 63, f2.BF16) == 0
    assert f2.fairy2i_vocab_loss_backward_workspace_bytes(1 << 20, 1 << 20, 64, f2.F32) == 0
    assert f2.fairy2i_lora_workspace_bytes(3, 16, 2048, 16, 16) > 0
    assert f2.fairy2i_clip_grads_workspace_bytes([5, 0, 9000]) == 16 + 32 * 3 + 8 * 3


# ---- binding ----

def raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def adapters(dt=torch.bfloat16):
    x = torch.zeros((5, 128), dtype=dt)
    A, B = torch.zeros((3, 4, 128), dtype=dt), torch.zeros((3, 64, 4), dtype=dt)
    al = torch.ones(3)
    ss, sa = torch.tensor([0, 2, 5], dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32)
    return x, A, B, al, ss, sa, torch.zeros((5, 64))


def test_lora_binding():
    x, A, B, al, ss, sa, base = adapters()
    f = f2.fairy2i_lora
    raises("dtype", f, x.half(), A, B, al, ss, sa, base)
    raises("A: dtype", f, x, A.float(), B, al, ss, sa, base)
    raises("B: dtype", f, x, A, B.float(), al, ss, sa, base)
    raises("A: shape", f, x, A[:, :, :-2], B, al, ss, sa, base)
    raises("B: shape", f, x, A, B[:, :, :-1], al, ss, sa, base)
    raises("B: shape", f, x, A, B[:2], al, ss, sa, base)
    raises("contiguous", f, x, A, B.transpose(1, 2).contiguous().transpose(1, 2), al, ss, sa, base)
    raises("alpha", f, x, A, B, al[:2], ss, sa, base)
    raises("seg_start", f, x, A, B, al, ss[:2], sa, base)
    raises("seg_start", f, x, A, B, al, ss.long(), sa, base)
    raises("seg_adapter", f, x, A, B, al, ss, sa[:0], base)
    raises("base", f, x, A, B, al, ss, sa, base[:4])
    raises("y: dtype", f, x, A, B, al, ss, sa, base, y=base.bfloat16())
    big = torch.zeros(6 * 64)
    raises("overlaps", f, x, A, B, al, ss, sa, big[:320].view(5, 64), y=big[64:].view(5, 64))
    raises("workspace", f, x, A, B, al, ss, sa, base, workspace=torch.zeros(16, dtype=torch.uint8))
    raises("GPU", f, x, A, B, al, ss, sa, base)
    raises("no items", f2.fairy2i_lora_grouped, x, [], ss, sa)
    raises(r"items\[1\]", f2.fairy2i_lora_grouped, x, [(A, B, al, base, None), (A[:2], B[:2], al[:2], base, None)], ss, sa)


def test_lora_backward_binding():
    x, A, B, al, ss, sa, _ = adapters()
    dy, f = torch.zeros((5, 64), dtype=torch.bfloat16), f2.fairy2i_lora_backward
    raises("dy", f, dy.float(), x, A, B, al, ss, sa)
    raises("dy", f, dy[:4], x, A, B, al, ss, sa)
    raises("needs dx_base", f, dy, x, A, B, al, ss, sa, dx=torch.zeros((5, 128)))
    raises("dx: dtype", f, dy, x, A, B, al, ss, sa, dx_base=torch.zeros((5, 128)), dx=torch.zeros((5, 128)).bfloat16())
    raises("dA", f, dy, x, A, B, al, ss, sa, dA=torch.zeros((3, 4, 128), dtype=torch.bfloat16))
    raises("dB", f, dy, x, A, B, al, ss, sa, dB=torch.zeros((3, 4, 64)))
    raises("GPU", f, dy, x, A, B, al, ss, sa)


def test_vocab_binding():
    h, W, t = torch.zeros((3, 64)), torch.zeros((10, 64)), torch.zeros(3, dtype=torch.int64)
    f, b = f2.fairy2i_vocab_loss, f2.fairy2i_vocab_loss_backward
    raises("W: dtype", f, h, W.bfloat16(), t)
    raises("W: shape", f, h, W[:, :32].contiguous(), t)
    raises("contiguous", f, h, torch.zeros((64, 10)).t(), t)
    raises("target", f, h, W, t.int())
    raises("target", f, h, W, t[:2])
    raises("loss", f, h, W, t, loss=torch.zeros(4))
    raises("GPU", f, h, W, t)
    v = torch.zeros(3)
    raises("lse", b, h, W, t, v[:2], v)
    raises("g: dtype", b, h, W, t, v, v.double())
    raises("nothing", b, h, W, t, v, v, want_dh=False, want_dW=False)
    raises("not wanted", b, h, W, t, v, v, want_dW=False, dW=torch.zeros_like(W))
    raises("dh", b, h, W, t, v, v, dh=torch.zeros((3, 32)))
    raises("GPU", b, h, W, t, v, v)


def test_clip_binding():
    f, g = f2.fairy2i_clip_grads, torch.zeros(40)
    raises("no gradients", f, [], 1.0)
    raises("dtype", f, [g.double()], 1.0)
    raises("contiguous", f, [torch.zeros((4, 4)).t()], 1.0)
    raises("outputs", f, [g], 1.0, out=[])
    raises("dtype", f, [g], 1.0, out=[g.bfloat16()])
    raises("overlaps", f, [g[:20]], 1.0, out=[g[10:30]])
    raises("max_norm", f, [g], -1.0)
    raises("max_norm", f, [g], math.nan)
    raises("norm", f, [g], 1.0, norm=torch.zeros(2))
    raises("GPU", f, [g], 1.0)
    raises("GPU", f, grads=[g], max_norm=1.0)               # by name
    raises("max_norm", f, max_norm=-1.0, grads=[g])
    with pytest.raises(TypeError, match="grads"):
        f(max_norm=1.0)


CHILD = r'''
import ctypes, json, sys
sys.path.insert(0, ROOT)
import torch
if torch.cuda.device_count() != 0:
    print(json.dumps({"skipped": "a device is visible"}))
    sys.exit(0)
import widely_linear_gemv_amd as f2
L = f2.lib()
P, Q = 1 << 20, 1 << 21
W = 1 << 40
items = (f2.LoraItem * 1)(f2.LoraItem(P, P, P, Q, Q, 32))
one = lambda t, v: (t * 1)(v)
out = {}
for name, call in {
    "lora": lambda: L.fairy2i_lora(P, 1, 4, 64, P, P, P, 2, 8, 32, P, P, 2, Q, Q, 0, P, W, None),
    "grouped": lambda: L.fairy2i_lora_grouped(items, 1, P, 0, 4, 64, 2, 8, P, P, 2, 0, P, W, None),
    "backward": lambda: L.fairy2i_lora_backward(P, P, 1, 4, 64, P, P, P, 2, 8, 32, P, P, 2, Q, Q, 1, 2 * Q, 3 * Q, P, W, None),
    "loss": lambda: L.fairy2i_vocab_loss(P, P, 1, 4, 100, 64, P, Q, 2 * Q, P, W, None),
    "loss_backward": lambda: L.fairy2i_vocab_loss_backward(P, P, 0, 4, 100, 64, P, P, P, Q, 2 * Q, P, W, None),
    "clip": lambda: L.fairy2i_clip_grads(1, one(ctypes.c_void_p, P), None, one(ctypes.c_int64, 8), one(ctypes.c_int, 0), 1.0,
                                         P, P, W, None),
}.items():
    out[name] = [call(), f2.fairy2i_last_error()]
print(json.dumps(out))
'''


def test_without_a_device_every_call_returns_err_hip():
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    res = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + CHILD], env=env, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    out = json.loads(res.stdout.strip().splitlines()[-1])
    if "skipped" in out:
        pytest.skip(out["skipped"])
    assert len(out) == 6
    for name, (status, msg) in out.items():
        assert status == 7 and msg, (name, status, msg)
