"""Four-bit products: what fp32 sums of exact products have to give to the last bits, beside test_gpu_w4.py, whose
bounds grow with the columns."""
import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(33, 1405), (4096, 300), (4100, 700), (10240, 130), (10300, 2000), (16384, 129), (16500, 640)]


def layer_of(rows, cols, G, sdt, seed, dev):
    """Codes 7..15 over zero points 0..3, some over 19 and more, and scales that are powers of two."""
    g = torch.Generator(device=dev).manual_seed(seed)
    groups = -(-cols // G)
    codes = torch.randint(7, 16, (rows, cols), generator=g, device=dev, dtype=torch.uint8)
    zero = torch.randint(0, 4, (rows, groups), generator=g, device=dev, dtype=torch.uint8)
    far = torch.rand(rows, groups, generator=g, device=dev) < 0.3
    zero[far] = torch.randint(19, 256, (int(far.sum()),), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.exp2(torch.randint(-6, 7, (rows, groups), generator=g, device=dev).float()).to(sdt)
    return codes, scales, zero, f2.fairy2i_pack_w4(codes, scales, G, zero)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_every_bit_of_fp32_x_counts(size, G):
    """One value a batch entry: y is s (c - z) x, off by the rounding of (16 + c) x / 16 in a sum (2^-24 of it;
    twice that allows for a matrix instruction that rounds once more) and that of the result.  x is 24 bits of
    which the second eight are 0x40..0x6f and the last 0x30..0x3f: cut into bf16 parts, the third is 48 2^-23 of x's
    power of two or more, and a product without it would be off by |c - z| 48 / (2 (16 + c + |c - z|)) times what is
    allowed here, 3.5 times at least (c - z >= 4, or <= -4)."""
    dev = device()
    rows, cols = size
    g = torch.Generator(device=dev).manual_seed(5)
    codes, scales, zero, layer = layer_of(rows, cols, G, BF if G == 64 else F32, 3, dev)
    every = torch.arange(cols, device=dev) if rows < 100 else torch.unique(torch.cat([
        torch.randint(0, cols, (40,), generator=g, device=dev), torch.tensor([0, 1, 31, 32, 127, 128, cols - 1], device=dev)]))
    announce("w4 every bit", size, G)
    for B in (16, 4, 1):
        for k in range(0, len(every) if B == 16 or rows < 100 else 3 * B, B):
            at = every[k:k + B]
            n = len(at)
            draw = lambda lo, hi: torch.randint(lo, hi, (n,), generator=g, device=dev)
            bits = 0x3F800000 | draw(0, 128) << 16 | draw(0x40, 0x70) << 8 | draw(0x30, 0x40)
            v = bits.to(torch.int32).view(F32) * torch.where(torch.arange(n, device=dev) % 2 == 0, 1.0, -1.0)
            x = torch.zeros((n, cols), device=dev)
            x[torch.arange(n, device=dev), at] = v
            y = f2.fairy2i_gemv_w4(layer, x).double()
            c, z, s = codes[:, at].t().double(), zero[:, at // G].t().double(), scales[:, at // G].t().double()
            want = s * (c - z) * v.double()[:, None]
            room = 2 * E24 * s * v.double().abs()[:, None] * (16 + c + (c - z).abs())
            assert ((y - want).abs() <= room).all(), (size, G, B, k, ((y - want).abs() / room).max())


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_weights_that_are_zero_give_zero(size, G):
    """fp32 x, codes that are their zero points: every product is 0, and so is y, whatever x is."""
    dev = device()
    rows, cols = size
    g = torch.Generator(device=dev).manual_seed(6)
    zero = torch.randint(0, 16, (rows, -(-cols // G)), generator=g, device=dev, dtype=torch.uint8)
    codes = zero.repeat_interleave(G, 1)[:, :cols].contiguous()
    layer = f2.fairy2i_pack_w4(codes, torch.rand(zero.shape, generator=g, device=dev), G, zero)
    announce("w4 zero weights", size, G)
    for B in (1, 3, 16):
        x = torch.randn((B, cols), generator=g, device=dev) * 10 + 3
        assert not f2.fairy2i_gemv_w4(layer, x).any()


@pytest.mark.parametrize("mean", [0.0, 3.0, 100.0])
@pytest.mark.parametrize("size", [(1003, 1405, 32), (4096, 4096, 128), (512, 11008, 64), (12000, 4096, 128), (6144, 2048, 64)],
                         ids=lambda s: "%dx%d-G%d" % s)
def test_no_less_exact_than_a_product_of_the_layer_written_out(size, mean):
    """fp32 x of any mean: y is no farther from 64 bits (2-norm) than the fp32 product with the matrix itself,
    whose entries s (c - z) fp32 holds exactly for bf16 scales.  Both have terms of size |s (c - z) x|; a matrix
    instruction sums 32 of them here where the other product rounds after one or a few."""
    dev = device()
    rows, cols, G = size
    g = torch.Generator(device=dev).manual_seed(7)
    groups = -(-cols // G)
    codes = torch.randint(0, 16, (rows, cols), generator=g, device=dev, dtype=torch.uint8)
    zero = torch.randint(5, 11, (rows, groups), generator=g, device=dev, dtype=torch.uint8)
    scales = (torch.rand(rows, groups, generator=g, device=dev) + 0.5).to(BF)
    layer = f2.fairy2i_pack_w4(codes, scales, G, zero)
    wide = lambda t: t.double().repeat_interleave(G, 1)[:, :cols]
    W = wide(scales) * (codes.double() - wide(zero))
    assert torch.equal(W.float().double(), W)
    announce("w4 exactness", size, mean)
    for B in (1, 5, 16):
        x = torch.randn((B, cols), generator=g, device=dev) + mean
        want = x.double() @ W.t()
        mine = (f2.fairy2i_gemv_w4(layer, x).double() - want).norm().item()
        plain = ((x @ W.float().t()).double() - want).norm().item()
        assert mine <= plain, (size, mean, B, mine / want.norm().item(), plain / want.norm().item())


@pytest.mark.parametrize("xdt", [BF, F32])
def test_the_most_rows_and_the_most_columns(xdt):
    """2^24 rows of one column: y = s (c - z) x, each factor a whole number or a power of two.  2^20 columns of five
    rows: all weights 0 but a few, whole sums."""
    dev = device()
    rows = 1 << 24
    announce("w4 most rows", xdt)
    codes = (torch.arange(rows, device=dev) % 16).to(torch.uint8).view(rows, 1)
    scales = torch.exp2((torch.arange(rows, device=dev) % 7 - 3).float()).view(rows, 1).to(BF)
    layer = f2.fairy2i_pack_w4(codes, scales, 128)
    x = torch.arange(1, 17, device=dev).view(16, 1).to(xdt)
    y = f2.fairy2i_gemv_w4(layer, x)
    want = (scales.float() * (codes.float() - 8))[:, 0]
    for b in range(16):
        assert torch.equal(y[b], want * (b + 1)), b
    del y, want, codes, scales, layer
    cols = 1 << 20
    announce("w4 most columns", xdt)
    codes = torch.full((5, cols), 8, dtype=torch.uint8, device=dev)
    codes[0, ::1000], codes[3, cols - 1], codes[4, cols // 2:] = 9, 0, 9
    layer = f2.fairy2i_pack_w4(codes, torch.ones((5, cols // 32), device=dev), 32)
    x = torch.ones((16, cols), dtype=xdt, device=dev)
    x[15] = 2.0
    want = torch.tensor([-(-cols // 1000), 0.0, 0.0, -8.0, cols // 2], device=dev).repeat(16, 1)
    want[15] *= 2
    if xdt == F32:
        assert torch.equal(f2.fairy2i_gemv_w4(layer, x), want)
    else:                                                 # sums of 1 + c / 16 of either sign, off by 2^-24 of 2^21 in all
        assert ((f2.fairy2i_gemv_w4(layer, x) - want).abs() <= 2.0 ** -3).all()
