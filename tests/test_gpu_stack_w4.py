"""Decode steps some of whose groups are wholly at four bits."""
import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2
from widely_linear_gemv_amd.stack import DecodeStep, GROUPS, PROJECTIONS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("algo", [f2.GEMV_MFMA_F4, f2.GEMV_MFMA_I8])
def test_groups_at_four_bits_have_no_digit_forms(algo, given):
    """x's digit form is made where a two-bit projection reads it, and nowhere else; each output is that of its own
    call, also from the captured step."""
    dev = device()
    T, B = 2, 2
    g = torch.Generator(device=dev).manual_seed(2)
    layers, xs = [], []
    for L in range(2):
        row = []
        for _, rows, cols, grp in PROJECTIONS:
            if grp == 1 + L or grp == 3:
                codes = torch.randint(0, 16, (rows, cols), generator=g, device=dev, dtype=torch.uint8)
                row.append(f2.fairy2i_pack_w4(codes, torch.rand((rows, cols // 64), generator=g, device=dev) * 0.02, 64))
            else:
                n, m = rows // 2, cols // 2
                packed = torch.randint(0, 256, (f2.fairy2i_packed_bytes(n, m, T),), generator=g, device=dev, dtype=torch.uint8)
                row.append((packed, torch.rand((n, T, 2, 2), generator=g, device=dev) * 0.02))
        layers.append(row)
        xs.append([torch.randn((B, next(c for _, _, c, grp in PROJECTIONS if grp == k)), generator=g, device=dev).bfloat16()
                   for k in range(GROUPS)])
    announce("decode step with groups at four bits", algo, given)
    step = DecodeStep(layers, xs, algo=algo, digits_given=given)
    for L in range(2):
        assert [d is None for d in step.digits[L]] == [k == 1 + L or k == 3 for k in range(GROUPS)]
    ys = step.run()
    graph = step.capture()
    for again in (False, True):
        if again:
            for y in (y for row in ys for y in row):
                y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
        for L in range(2):
            for p, (name, _, _, grp) in enumerate(PROJECTIONS):
                if isinstance(layers[L][p], f2.W4Layer):
                    assert torch.equal(ys[L][p], f2.fairy2i_gemv_w4(layers[L][p], xs[L][grp])), (L, name)
                else:
                    want = f2.fairy2i_gemv(*layers[L][p], xs[L][grp]).double()
                    assert (ys[L][p].double() - want).norm() <= 1e-4 * want.norm(), (L, name)
