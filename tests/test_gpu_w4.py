"""Layers kept at four bits (fairy2i_pack_w4, fairy2i_gemv_w4) against the formula in 64 bits.

Tolerance from the arithmetic, per output: with A = sum_j |s| (16 + c + 16 + z) |x_j| the size of the terms
that are summed, fp32 sums of at most 3 G + G (products of three parts, and x itself) and ceil(cols / G) + 8
terms give (4 G + groups + 40) 2^-24 A, and the result is rounded once (u, half a step of y's type)."""
import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2
from widely_linear_gemv_amd.stack import DecodeStep, GROUPS, PROJECTIONS

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def make(rows, cols, G, sdt, zeros, seed, dev, full_bytes=False):
    g = torch.Generator().manual_seed(seed)
    groups = -(-cols // G)
    codes = torch.randint(0, 256 if full_bytes else 16, (rows, cols), generator=g, dtype=torch.uint8)
    scales = (torch.randn(rows, groups, generator=g) * cols ** -0.5).to(sdt)
    zero = torch.randint(0, 256 if full_bytes else 16, (rows, groups), generator=g, dtype=torch.uint8) if zeros else None
    layer = f2.fairy2i_pack_w4(codes.to(dev), scales.to(dev), G, None if zero is None else zero.to(dev))
    return codes, scales, zero, layer


def reference(codes, scales, zero, G, x, ydt):
    """y and its bound, in 64 bits."""
    rows, cols = codes.shape
    wide = lambda t: t.double().repeat_interleave(G, 1)[:, :cols]
    c = (codes & 15).double()
    z = torch.full_like(c, 8.0) if zero is None else wide(zero)
    s, xd = wide(scales), x.double()
    y = xd @ (s * (c - z)).t()
    A = xd.abs() @ (s.abs() * (32 + c + z)).t()
    u = torch.finfo(ydt).eps / 2
    return y, (4 * G + -(-cols // G) + 40) * E24 * A + u * y.abs()


def check(layer, parts, G, x, ydt, dev, label):
    announce("w4", label)
    y = torch.full((x.shape[0], layer.rows), float("nan"), dtype=ydt, device=dev)
    got = f2.fairy2i_gemv_w4(layer, x.to(dev), y=y)
    assert got is y
    want, bound = reference(*parts, G, x, ydt)
    over = ((y.double().cpu() - want).abs() - bound).max().item()
    assert over <= 0, (label, over)
    return y


SIZES = [(1, 1), (1, 128), (16, 32), (17, 130), (5, 1405), (1003, 333), (64, 4096), (100, 11008), (40, 33000)]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_against_64_bits(size, G):
    dev = device()
    rows, cols = size
    for k, (sdt, zeros) in enumerate(((BF, True), (F32, True), (BF, False))):
        codes, scales, zero, layer = make(rows, cols, G, sdt, zeros, 7 + k, dev)
        g = torch.Generator().manual_seed(3)
        for B, xdt, ydt in ((1, BF, BF), (2, BF, F32), (5, F32, F32), (16, BF, BF), (16, F32, BF), (1, F32, F32)):
            x = torch.randn(B, cols, generator=g).to(xdt)
            check(layer, (codes, scales, zero), G, x, ydt, dev, (size, G, sdt, zeros, B, xdt, ydt))


# sizes on both sides of where waves and tiles of a workgroup change (256, 640 and 1024 tiles of 16 rows)
LARGE = [(4096, 300), (4100, 1405), (10240, 130), (10300, 2000), (16384, 129), (16500, 640)]


@pytest.mark.parametrize("xdt", [BF, F32])
@pytest.mark.parametrize("size", LARGE, ids=lambda s: "%dx%d" % s)
def test_many_rows(size, xdt):
    """The 64-bit reference runs on the GPU."""
    dev = device()
    rows, cols = size
    for G, sdt in ((32, F32), (64, BF), (128, BF)):
        codes, scales, zero, layer = make(rows, cols, G, sdt, True, 21, dev)
        parts = [t.to(dev) for t in (codes, scales, zero)]
        x = torch.randn(16, cols, generator=torch.Generator().manual_seed(4)).to(xdt).to(dev)
        announce("w4 many rows", size, xdt, G)
        want, bound = reference(*parts, G, x, F32)
        all16 = f2.fairy2i_gemv_w4(layer, x)
        assert ((all16.double() - want).abs() <= bound).all(), (size, G)
        for B in (1, 2, 4, 5):
            assert torch.equal(f2.fairy2i_gemv_w4(layer, x[:B].contiguous()), all16[:B]), (size, G, B)


def test_offsets_past_32_bits():
    """A layer of 2^33 codes: its last rows' blocks lie past 2^32 bytes.  All weights are 0 but some of theirs."""
    dev = device()
    rows, cols = (1 << 17) + 5, (1 << 16) + 100
    announce("w4 offsets")
    codes = torch.full((rows, cols), 8, dtype=torch.uint8, device=dev)
    codes[rows - 1, ::1000], codes[rows - 6, cols - 1], codes[3, 5] = 9, 0, 15
    scales = torch.ones((rows, -(-cols // 128)), dtype=BF, device=dev)
    layer = f2.fairy2i_pack_w4(codes, scales, 128)
    assert layer.buf.numel() > 1 << 32
    del codes
    x = torch.ones((2, cols), dtype=BF, device=dev)
    x[1] = 2.0
    y = f2.fairy2i_gemv_w4(layer, x)
    want = torch.zeros(rows, device=dev)
    want[rows - 1], want[rows - 6], want[3] = -(-cols // 1000), -8.0, 7.0
    assert torch.equal(y, torch.stack([want, 2 * want]))         # whole numbers under 2^24 are exact


def test_every_batch_is_the_same_sum():
    """A batch entry's outputs do not depend on the entries beside it, bit for bit."""
    dev = device()
    for cols, xdt in ((4096, BF), (11008, BF), (1405, F32), (9000, F32)):
        codes, scales, zero, layer = make(50, cols, 64, BF, True, 1, dev)
        x = torch.randn(16, cols, generator=torch.Generator().manual_seed(2)).to(xdt).to(dev)
        announce("w4 batches", cols, xdt)
        want = f2.fairy2i_gemv_w4(layer, x)
        for B in (1, 2, 3, 7, 15):
            for b0 in (0, 16 - B):
                part = x[b0:b0 + B].clone()
                assert torch.equal(f2.fairy2i_gemv_w4(layer, part), want[b0:b0 + B]), (cols, B, b0)


def test_high_bits_and_far_zero_points():
    """The codes' higher bits are ignored; a zero point may be any byte."""
    dev = device()
    codes, scales, zero, layer = make(33, 500, 32, F32, True, 5, dev, full_bytes=True)
    x = torch.randn(3, 500, generator=torch.Generator().manual_seed(1))
    check(layer, (codes, scales, zero), 32, x, F32, dev, "bytes")


def test_whole_numbers_are_exact():
    """Scales that are powers of two, whole x: every sum is exact in fp32."""
    dev = device()
    g = torch.Generator().manual_seed(9)
    codes = torch.randint(0, 16, (70, 999), generator=g, dtype=torch.uint8)
    zero = torch.randint(0, 16, (70, 32), generator=g, dtype=torch.uint8)
    scales = torch.full((70, 32), 0.25)
    x = torch.randint(-8, 9, (4, 999), generator=g).float()
    layer = f2.fairy2i_pack_w4(codes.to(dev), scales.to(dev), 32, zero.to(dev))
    want = reference(codes, scales, zero, 32, x, F32)[0]
    for xdt in (BF, F32):
        assert torch.equal(f2.fairy2i_gemv_w4(layer, x.to(xdt).to(dev)).double().cpu(), want)


@pytest.mark.parametrize("xdt", [BF, F32])
def test_wide_values(xdt):
    """Large means, outliers, tiny and huge x (fp32 x past the largest bf16 too)."""
    dev = device()
    codes, scales, zero, layer = make(48, 700, 64, BF, True, 11, dev)
    x = torch.randn(4, 700, generator=torch.Generator().manual_seed(4))
    x[0] += 100.0
    x[1, ::97] *= 1e4
    x[2] *= 1e-30
    x[3] *= 1e30
    check(layer, (codes, scales, zero), 64, x.to(xdt), F32, dev, xdt)
    big = torch.full((1, 700), 0.0)
    big[0, 5] = torch.finfo(F32).max                      # alone, with a scale that keeps it in range
    codes, scales = codes.clone(), torch.full_like(scales, 2.0 ** -10)
    small = f2.fairy2i_pack_w4(codes.to(dev), scales.to(dev), 64, zero.to(dev))
    if xdt == F32:
        # 16 + c times the largest fp32 leaves fp32's range before the scale: NaN or infinity, never a number
        assert not torch.isfinite(f2.fairy2i_gemv_w4(small, big.to(dev))).all()
        check(small, (codes, scales, zero), 64, big * 2.0 ** -10, F32, dev, "near the largest")


def test_a_nan_stays_in_its_entry():
    dev = device()
    codes, scales, zero, layer = make(40, 1000, 128, BF, True, 12, dev)
    x = torch.randn(6, 1000, generator=torch.Generator().manual_seed(5))
    clean = f2.fairy2i_gemv_w4(layer, x.to(dev))
    bad = x.clone()
    bad[2, 999], bad[4, 0] = float("nan"), float("inf")
    for dt in (F32, BF):
        announce("w4 nan", dt)
        want = f2.fairy2i_gemv_w4(layer, x.to(dt).to(dev))
        y = f2.fairy2i_gemv_w4(layer, bad.to(dt).to(dev))
        for b in (0, 1, 3, 5):
            assert torch.equal(y[b], want[b])
        assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[4]).any()
    # a row's scale does not reach other rows
    s2 = scales.clone()
    s2[7, 3] = float("nan")
    y = f2.fairy2i_gemv_w4(f2.fairy2i_pack_w4(codes.to(dev), s2.to(dev), 128, zero.to(dev)), x.to(dev))
    keep = torch.arange(40) != 7
    assert torch.equal(y[:, keep.to(dev)], clean[:, keep.to(dev)]) and torch.isnan(y[:, 7]).all()


def test_writes_its_outputs_only():
    """The bytes before and behind y and the packed form stay as they were."""
    dev = device()
    rows, cols = 19, 150
    codes = torch.randint(0, 16, (rows, cols), dtype=torch.uint8, device=dev)
    scales = torch.rand(rows, 5, device=dev)
    n = f2.fairy2i_packed_bytes_w4(rows, cols, 32, F32)
    buf = torch.full((n + 64,), 77, dtype=torch.uint8, device=dev)
    announce("w4 borders")
    layer = f2.fairy2i_pack_w4(codes, scales, 32, packed=buf[32:32 + n])
    assert (buf[:32] == 77).all() and (buf[32 + n:] == 77).all()
    for ydt in (F32, BF):
        for B in (1, 3, 16):
            out = torch.full((B * rows + 32,), 5.0, dtype=ydt, device=dev)
            y = out[16:16 + B * rows].view(B, rows)
            f2.fairy2i_gemv_w4(layer, torch.randn(B, cols, device=dev), y=y)
            assert (out[:16] == 5.0).all() and (out[16 + B * rows:] == 5.0).all() and not (y == 5.0).all()


def test_streams_and_graph():
    dev = device()
    codes, scales, zero, layer = make(200, 3000, 64, BF, True, 13, dev)
    x = torch.randn(4, 3000, generator=torch.Generator().manual_seed(6)).to(dev).bfloat16()
    want = f2.fairy2i_gemv_w4(layer, x)
    side = torch.cuda.Stream()
    announce("w4 side stream")
    again = f2.fairy2i_pack_w4(codes.to(dev), scales.to(dev), 64, zero.to(dev))
    side.wait_stream(torch.cuda.current_stream())
    y = f2.fairy2i_gemv_w4(again, x, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    announce("w4 graph")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = f2.fairy2i_gemv_w4(layer, x)
    x2 = x.flip(0).contiguous()
    for k in range(3):
        if k % 2:
            keep = x.clone()
            x.copy_(x2)
        y.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want.flip(0) if k % 2 else want), k
        if k % 2:
            x.copy_(keep)
        assert torch.equal(f2.fairy2i_gemv_w4(layer, x), want)


@pytest.mark.parametrize("B", [1, 8])
def test_decode_step_with_four_bit_projections(B):
    """A decode step whose down projection and one of q, k, v are kept at four bits: those outputs are the
    four-bit products, the others what the step gives without them, eagerly and in a graph."""
    dev = device()
    T = 2
    g = torch.Generator(device=dev).manual_seed(1)
    two_bit, mixed, xs = [], [], []
    for L in range(2):
        row = []
        for _, rows, cols, _ in PROJECTIONS:
            n, m = rows // 2, cols // 2
            packed = torch.randint(0, 256, (f2.fairy2i_packed_bytes(n, m, T),), generator=g, device=dev, dtype=torch.uint8)
            row.append((packed, torch.rand((n, T, 2, 2), generator=g, device=dev) * 0.02))
        two_bit.append(row)
        own = list(row)
        for p in (1, 6):
            _, rows, cols, _ = PROJECTIONS[p]
            codes = torch.randint(0, 16, (rows, cols), generator=g, device=dev, dtype=torch.uint8)
            own[p] = f2.fairy2i_pack_w4(codes, torch.rand((rows, cols // 64), generator=g, device=dev) * 0.02, 64)
        mixed.append(own)
        xs.append([torch.randn((B, next(c for _, _, c, grp in PROJECTIONS if grp == k)), generator=g, device=dev).bfloat16()
                   for k in range(GROUPS)])
    announce("decode step with four-bit projections", B)
    plain = DecodeStep(two_bit, xs).run()
    step = DecodeStep(mixed, xs)
    ys = step.run()

    def look():
        for L in range(2):
            for p, (name, _, _, grp) in enumerate(PROJECTIONS):
                if p in (1, 6):
                    assert torch.equal(ys[L][p], f2.fairy2i_gemv_w4(mixed[L][p], xs[L][grp])), (L, name)
                else:
                    # a group without one of its projections may be split over waves otherwise
                    err = (ys[L][p].double() - plain[L][p].double()).norm() / plain[L][p].double().norm()
                    assert err <= 1e-5, (L, name)
    look()
    graph = step.capture()
    for k in range(2):
        for row in ys:
            for y in row:
                y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        look()
