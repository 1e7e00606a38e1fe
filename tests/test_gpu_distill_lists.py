"""Distillation from lists that lie at the ends of what the calls allow, beside test_gpu_distill.py, whose
formulas and bounds these tests use."""
import math

import pytest
import torch

from gpu_util import announce, device
from test_gpu_distill import BF, F32, backward, close, forward, grad_reference, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tdt", [F32, BF])
@pytest.mark.parametrize("T", [2.0 ** -20, 0.5, 1.0, 4.0])
def test_logits_that_leave_fp32_over_the_temperature(T, tdt):
    """Finite logits of any size are logits: lists of the type's lowest or largest value throughout (equal
    probabilities), with a few of them among ordinary ones, and of values whose quotient by T is out of fp32's
    range.  The formula depends on their distances from the largest alone, so the reference takes those, and
    those under -1e30 as minus infinity (their exponentials are 0 in 64 bits)."""
    dev = device()
    N, V, K, top = 12, 300, 64, 9
    c, d = make(N, V, K, top, F32, 41, dev, T, ignored=0.0)
    c["h"] *= T                                            # the student's logits of ordinary size
    c["index"] = torch.stack([torch.randperm(V, generator=torch.Generator().manual_seed(i))[:top] for i in range(N)])
    low, high = torch.finfo(tdt).min, torch.finfo(tdt).max
    z = (torch.randn(N, top, generator=torch.Generator().manual_seed(2)) * T).to(tdt).double()
    z[0], z[1] = low, high
    z[2, ::2] = low
    z[3, 4] = high
    z[4, :3], z[4, 3:] = high, low
    z[5] = torch.where(torch.arange(top) % 3 == 0, 2.0 ** 120, -(2.0 ** 120))
    z[6] = 2.0 ** 125
    z[7, 1:] = -math.inf
    z[7, 0] = low
    c["logit"] = z.to(tdt)
    c["g"] = torch.rand(N, generator=torch.Generator().manual_seed(3))
    away = c["logit"].double() - c["logit"].double().amax(1, keepdim=True)
    shifted = dict(c, logit=torch.where(away < -1e30, torch.full_like(away, -math.inf), away))
    d.update({k: c[k].to(dev) for k in ("h", "index", "logit", "g")})
    announce("distill extreme logits", T, tdt)
    loss, lse = forward(d)
    r = reference(shifted)
    assert r["counts"].all()
    close(lse, r["lse"], r["dl"], "lse")
    close(loss, r["loss"], r["dloss"], "loss")
    dh, dW = backward(d, lse)
    wh, bh, wW, bW = grad_reference(shifted, r)
    close(dh, wh, bh, "dh")
    close(dW, wW, bW, "dW")
