"""Refusals of the four-bit calls: the C ABI returns its documented status before any HIP call, the
binding raises before it enters the library, and without a device a call returns FAIRY2I_ERR_HIP.  No GPU
needed."""
import os

import pytest
import torch

import widely_linear_gemv_amd as f2
from widely_linear_gemv_amd.stack import DecodeStep, PROJECTIONS

FAKE = 1 << 20          # a 16-byte aligned, never dereferenced address
FAR = 1 << 40
ODD = FAKE + 2
S = None


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(f2.LIB_PATH):
        from widely_linear_gemv_amd import build
        build.build()
    return f2.lib()


def pack_args(**kw):
    a = dict(codes=FAKE, scales=FAKE, sd=1, zeros=FAKE, rows=40, cols=200, group=64, packed=FAR, st=S)
    a.update(kw)
    return list(a.values())


def gemv_args(**kw):
    a = dict(packed=FAKE, rows=40, cols=200, group=64, sd=1, x=FAKE, xd=1, B=2, y=FAR, yd=0, st=S)
    a.update(kw)
    return list(a.values())


SIZES = [(dict(rows=0), 2), (dict(rows=(1 << 24) + 1, cols=1), 2), (dict(cols=0), 2), (dict(cols=(1 << 20) + 1, rows=1), 2),
         (dict(group=0), 2), (dict(group=16), 2), (dict(group=256), 2), (dict(rows=1 << 24, cols=(1 << 10) + 1), 2),
         (dict(sd=2), 4), (dict(sd=-1), 4)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(packed=None), 1), (dict(packed=FAR + 8), 5), (dict(scales=FAKE + 1), 5),
    (dict(scales=ODD, sd=0), 5), (dict(codes=FAR), 2), (dict(scales=FAR), 2), (dict(zeros=FAR), 2),
    (dict(codes=FAR - 40 * 200 + 1), 2), (dict(zeros=FAR - 40 * 4 + 1), 2), (dict(scales=FAR - 40 * 4 * 2 + 2), 2)])
def test_pack_errors(L, kw, status):
    assert L.fairy2i_pack_w4(*pack_args(**kw)) == status
    assert f2.fairy2i_last_error()


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(packed=None), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(xd=2), 4), (dict(yd=3), 4), (dict(B=0), 2), (dict(B=17), 2),
    (dict(packed=ODD), 5), (dict(x=ODD), 5), (dict(y=FAR + 4), 5), (dict(x=FAR), 2), (dict(packed=FAR), 2),
    (dict(y=FAKE + 2 * 200 * 2 - 16), 2)])
def test_gemv_errors(L, kw, status):
    assert L.fairy2i_gemv_w4(*gemv_args(**kw)) == status
    assert f2.fairy2i_last_error()


def test_bytes(L):
    """1 KB a tile and 128 columns; 16 scales and 16 bytes of zero points a tile and group."""
    assert f2.fairy2i_packed_bytes_w4(40, 200, 64, torch.bfloat16) == 3 * (2 * 1024 + 4 * (32 + 16))
    assert f2.fairy2i_packed_bytes_w4(16, 128, 128, torch.float32) == 1024 + 80
    assert f2.fairy2i_packed_bytes_w4(0, 128, 128) == 0 and f2.fairy2i_packed_bytes_w4(16, 128, 100) == 0
    assert L.fairy2i_packed_bytes_w4(16, 128, 128, 2) == 0


def test_without_a_device(L):
    if torch.cuda.device_count() != 0:
        pytest.skip("a device is visible")
    assert L.fairy2i_pack_w4(*pack_args()) == 7 and f2.fairy2i_last_error()
    assert L.fairy2i_gemv_w4(*gemv_args()) == 7 and f2.fairy2i_last_error()


def raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_binding_checks():
    codes, scales = torch.zeros(40, 200, dtype=torch.uint8), torch.zeros(40, 4, dtype=torch.bfloat16)
    zeros = torch.zeros(40, 4, dtype=torch.uint8)
    pack = f2.fairy2i_pack_w4
    raises("dtype", pack, codes.int(), scales, 64)
    raises("shape", pack, codes[0], scales, 64)
    raises("group", pack, codes, scales, 48)
    raises("shape", pack, codes, scales, 32)
    raises("dtype", pack, codes, scales.half(), 64)
    raises("contiguous", pack, codes.t(), scales, 64)
    raises("dtype", pack, codes, scales, 64, zeros.int())
    raises("shape", pack, codes, scales, 64, zeros[:-1])
    buf = torch.zeros(f2.fairy2i_packed_bytes_w4(40, 200, 64), dtype=torch.uint8)
    raises("bytes", pack, codes, scales, 64, zeros, packed=buf[:-16])
    raises("GPU", pack, codes, scales, 64, zeros, packed=buf)
    with pytest.raises(TypeError):
        pack(codes, None, 64)
    layer = f2.W4Layer(buf, 40, 200, 64)
    raises("out of range", f2.W4Layer, buf, 40, 0, 64)
    raises("scales_dtype", f2.W4Layer, buf, 40, 200, 64, torch.float16)
    x = torch.zeros(2, 200)
    gemv = f2.fairy2i_gemv_w4
    with pytest.raises(TypeError):
        gemv(buf, x)
    with pytest.raises(TypeError):
        gemv(layer, None)
    raises("dtype", gemv, layer, x.double())
    raises("shape", gemv, layer, x[:, :-1])
    raises("shape", gemv, layer, x[0])
    raises("contiguous", gemv, layer, torch.zeros(200, 2).t())
    raises("shape", gemv, layer, x, y=torch.zeros(2, 41))
    raises("dtype", gemv, layer, x, y=torch.zeros(2, 40, dtype=torch.float64))
    raises("contiguous", gemv, layer, x, y=torch.zeros(40, 2).t())
    raises("GPU", gemv, layer, x)


def test_decode_step_checks_the_shape():
    layer = f2.W4Layer(torch.zeros(f2.fairy2i_packed_bytes_w4(40, 200, 64), dtype=torch.uint8), 40, 200, 64)
    raises("at four bits", DecodeStep, [[layer] * len(PROJECTIONS)], [[torch.zeros(1, 4096)] * 4])
