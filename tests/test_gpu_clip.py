"""Global gradient norm and clipping (fairy2i_clip_grads) against 64 bits: the norm is off by one
fp32 rounding (2^-24) and fp64 noise, an output by the rounding of c (2^-24), the product (2^-24) and
its dtype's rounding."""
import math

import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu


def grads_of(sizes, dts, seed, dev, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dts[k % len(dts)]).to(dev) for k, n in enumerate(sizes)]


def check(grads, before, norm, max_norm):
    want = math.sqrt(sum(float((b.double() ** 2).sum()) for b in before))
    assert abs(norm.item() - want) <= 2.0 ** -23 * want
    c = min(1.0, max_norm / (want + 1e-6))
    for g, b in zip(grads, before):
        w = b.double() * c
        bound = w.abs() * (2.0 ** -22 + torch.finfo(g.dtype).eps / 2)
        assert ((g.double() - w).abs() <= bound).all()


@pytest.mark.parametrize("sizes", [[1], [8192], [8193, 3, 1], [5, 16384, 100, 40000, 7], [100] * 230, [300000]])
@pytest.mark.parametrize("dts", [[torch.float32], [torch.bfloat16], [torch.float32, torch.bfloat16]])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_norm_and_clip(sizes, dts, max_norm):
    dev = device()
    grads = grads_of(sizes, dts, 3, dev)
    before = [g.clone() for g in grads]
    announce("clip", sizes[:5], dts, max_norm)
    out = [torch.full_like(g, 5.0) for g in grads]
    norm = f2.fairy2i_clip_grads(grads, max_norm, out=out)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    check(out, before, norm, max_norm)
    again = f2.fairy2i_clip_grads(grads, max_norm)
    assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(grads, out))


def test_misaligned_views_and_empty_tensors():
    dev = device()
    flat = torch.randn(5000, generator=torch.Generator().manual_seed(4)).to(dev)
    half = flat.bfloat16()
    grads = [flat[1:1001], half[3:2003], flat[2000:2000], flat[2002:2003], half[4097:4098]]
    before, rest = [g.clone() for g in grads], (flat.clone(), half.clone())
    announce("clip misaligned")
    norm = f2.fairy2i_clip_grads(grads, 2.0)
    check(grads, before, norm, 2.0)
    assert torch.equal(flat[1001:2002], rest[0][1001:2002]) and flat[0] == rest[0][0]
    assert torch.equal(half[2003:4097], rest[1][2003:4097]) and torch.equal(half[:3], rest[1][:3])


def test_huge_and_tiny_values():
    dev = device()
    for scale in (1e30, 1e-30):
        grads = [torch.full((1000,), scale, device=dev), torch.full((77,), -scale, device=dev).bfloat16()]
        before = [g.clone() for g in grads]
        announce("clip scale", scale)
        norm = f2.fairy2i_clip_grads(grads, 1.0)
        check(grads, before, norm, 1.0)


def test_not_finite():
    dev = device()
    g = [torch.ones(10, device=dev), torch.ones(10, device=dev)]
    g[1][3] = float("inf")
    announce("clip infinity")
    norm = f2.fairy2i_clip_grads(g, 1.0)
    assert norm.item() == math.inf and not g[0].any() and torch.isnan(g[1][3])
    g = [torch.ones(10, device=dev)]
    g[0][0] = float("nan")
    announce("clip NaN")
    assert torch.isnan(f2.fairy2i_clip_grads(g, 1.0)).all() and torch.isnan(g[0]).all()


def test_norm_alone_and_zero():
    dev = device()
    g = [torch.randn(100, device=dev)]
    before = g[0].clone()
    announce("clip norm alone")
    norm = f2.fairy2i_clip_grads(g, math.inf)
    assert torch.equal(g[0], before) and abs(norm.item() - before.double().norm().item()) <= 2.0 ** -23 * norm.item()
    f2.fairy2i_clip_grads(g, 0.0)
    assert not g[0].any()
    assert f2.fairy2i_clip_grads(g, 1.0).item() == 0.0


def test_norm_alone_of_bad_gradients():
    """max_norm infinite changes nothing, whatever the norm is."""
    dev = device()
    for bad in (math.inf, -math.inf, math.nan):
        g = [torch.randn(9000, device=dev), torch.randn(33, device=dev).bfloat16()]
        g[1][7] = bad
        before = [t.clone() for t in g]
        announce("clip norm alone", bad)
        norm = f2.fairy2i_clip_grads(g, math.inf).item()
        assert not math.isfinite(norm)
        assert torch.equal(g[0], before[0]) and torch.equal(g[1].view(torch.int16), before[1].view(torch.int16))


def test_stream_and_graph():
    dev = device()
    grads = grads_of([9000, 77, 20000], [torch.float32, torch.bfloat16], 5, dev)
    out = [torch.empty_like(g) for g in grads]
    want_norm = f2.fairy2i_clip_grads(grads, 1.0, out=out).clone()
    want = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    announce("clip graph")
    n2 = f2.fairy2i_clip_grads((g for g in grads), 1.0, out=out, stream=side)
    side.synchronize()
    assert torch.equal(n2, want_norm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        norm = f2.fairy2i_clip_grads(grads, 1.0, out=out)
    for k in range(4):
        for o in out:
            o.zero_()
        norm.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want_norm) and all(torch.equal(a, b) for a, b in zip(out, want)), k
        f2.fairy2i_clip_grads(grads, 1.0, out=[torch.empty_like(x) for x in grads])


def test_norm_inside_a_gradient_is_refused():
    """norm is stored before the gradients are scaled: in one of them, or in an output, the call is refused
    and changes nothing."""
    dev = device()
    flat = torch.randn(40, generator=torch.Generator().manual_seed(6)).to(dev)
    other, before = torch.zeros(40, device=dev), flat.clone()
    for norm, out in ((flat[3:4], None), (flat[0:1], None), (flat[29:30], [other[:30]]), (other[7:8], [other[:30]])):
        announce("clip norm inside", norm.data_ptr() - flat.data_ptr(), out is None)
        with pytest.raises(f2.Fairy2iError, match="norm overlaps") as e:
            f2.fairy2i_clip_grads([flat[:30]], 1.0, out=out, norm=norm)
        assert e.value.status == 2
    torch.cuda.synchronize()
    assert torch.equal(flat, before) and not other.any()
    f2.fairy2i_clip_grads([flat[:30]], 1.0, norm=flat[30:31])                    # next to them: taken
    want = before[:30].double().norm().item()
    assert abs(flat[30].item() - want) <= 2.0 ** -23 * want and torch.equal(flat[31:], before[31:])


@pytest.mark.parametrize("size,max_norm", [(1e30, 1e-9), (3e38, 1e-20), (3e38, 1e-37), (1e38, 1.0), (1e-30, 1e-38)])
def test_coefficients_under_the_normal_range(size, max_norm):
    """c = max_norm / norm from 1e-40 to 1e-78 beside outputs that fp32 holds: as exact as any other."""
    dev = device()
    gen = torch.Generator().manual_seed(8)
    grads = [((torch.rand(n, generator=gen) + 0.1) * size / 1.1).to(dt).to(dev)
             for n, dt in ((9000, torch.float32), (77, torch.bfloat16), (5, torch.float32))]
    before = [g.clone() for g in grads]
    announce("clip small coefficient", size, max_norm)
    norm = f2.fairy2i_clip_grads(grads, max_norm)
    want = math.sqrt(sum(float((b.double() ** 2).sum()) for b in before))
    assert abs(norm.item() - want) <= 2.0 ** -23 * want or (norm.item() == math.inf and want > 3.4e38)
    c = min(1.0, torch.tensor(max_norm).double().item() / (want + 1e-6))        # max_norm enters as fp32
    for g, b in zip(grads, before):
        w = b.double() * c
        tiny = 2.0 ** -126 * (w < 2.0 ** -125).double()                          # outputs under the normal range
        assert ((g.double() - w).abs() <= w.abs() * (2.0 ** -22 + torch.finfo(g.dtype).eps / 2) + tiny).all()
