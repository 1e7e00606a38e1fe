"""Distillation from lists that lie at the ends of what the calls allow, beside test_gpu_distill.py, whose
formulas and bounds these tests use."""
import math

import pytest
import torch

from gpu_util import announce, device
from test_gpu_distill import BF, F32, backward, close, forward, grad_reference, make, reference

import widely_linear_gemv_amd as f2

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


def two_entries(N, V, K, dev, seed):
    """Lists of two entries (their softmax is the same bit for bit wherever they stand) and equal g."""
    c, d = make(N, V, K, 2, BF, seed, dev, ignored=0.0)
    c["index"] = torch.stack([torch.randperm(V, generator=torch.Generator().manual_seed(i))[:2] for i in range(N)])
    c["logit"] = torch.randn(N, 2, generator=torch.Generator().manual_seed(seed)) * 0.3
    c["g"] = torch.full((N,), 1 / 261.0)
    d.update({k: c[k].to(dev) for k in ("index", "logit", "g")})
    return d


@pytest.mark.parametrize("places", [(0, 1), (1, 2), (5, 0), (70, 71), (127, 3), (126, 127), (40, 64)], ids=str)
def test_unused_slots_anywhere(places):
    """Where a list's used slots stand changes no bit of the gradient, equal g among all tokens (whose common
    factor costs h no rounding)."""
    dev = device()
    d = two_entries(300, 900, 256, dev, 8)
    announce("distill unused slots", places)
    _, lse = forward(d)
    dh, dW = backward(d, lse)
    wide = dict(d, index=torch.full((300, 128), -1, device=dev), logit=torch.full((300, 128), math.nan, device=dev))
    for k, place in enumerate(places):
        wide["index"][:, place], wide["logit"][:, place] = d["index"][:, k], d["logit"][:, k]
    _, lse2 = forward(wide)
    dh2, dW2 = backward(wide, lse2)
    assert torch.equal(lse2, lse) and torch.equal(dh2, dh) and torch.equal(dW2, dW)


@pytest.mark.parametrize("leading", [1, 20, 100])
@pytest.mark.parametrize("kind", ["minus infinity", "empty", "outside"])
def test_tokens_that_do_not_count_lend_no_factor(kind, leading):
    """In front, tokens that do not count, with other g than the rest's common one (some of them 0, infinite or
    NaN): the same gradient, bit for bit, as with the common g there."""
    dev = device()
    if kind == "minus infinity":
        leading = min(leading, 30)                         # further tokens with used slots are not looked at
    d = two_entries(300, 900, 256, dev, 9)
    if kind == "minus infinity":
        d["logit"][:leading] = -math.inf
    else:
        d["index"][:leading] = -1 if kind == "empty" else 900
    announce("distill tokens that do not count", kind, leading)
    _, lse = forward(d)
    dh, dW = backward(d, lse)
    assert not dh[:leading].any()
    g = d["g"].clone()
    g[:leading] = torch.linspace(0.3, 0.5, leading, device=dev)
    g[leading // 2] = torch.tensor([0.0, math.inf, math.nan])[leading % 3].item()
    dh2, dW2 = backward(dict(d, g=g), lse)
    assert torch.equal(dh2, dh) and torch.equal(dW2, dW)


@pytest.mark.parametrize("N", [50, 300])
def test_a_list_of_one_has_the_cross_entropys_roundings(N):
    """bf16, one listed entry, temperature 1: the products are those of the vocabulary loss, and so is every bit of
    the gradient."""
    dev = device()
    c, d = make(N, 700, 128, 1, BF, 3, dev, ignored=0.3)
    target = torch.where((d["index"] >= 0) & (d["index"] < 700), d["index"], torch.full_like(d["index"], -1))[:, 0].contiguous()
    announce("distill lists of one", N)
    _, lse = forward(d)
    dh, dW = backward(d, lse)
    _, lse2 = f2.fairy2i_vocab_loss(d["h"], d["W"], target)
    dh2, dW2 = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], target, lse2, d["g"])
    assert torch.equal(lse, lse2) and torch.equal(dh, dh2) and torch.equal(dW, dW2)


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("sure", [0.55, 0.9, 0.97, 1.0])
def test_an_entry_that_dominates_moves_no_whole_row(sure, T):
    """bf16, a teacher that gives one entry of each list the probability `sure` and more: that entry's p dominates
    the token's dh and its own row of dW, so that its rounding would move all their values together, by up to
    2^-8 of themselves.  Along each such row the error is at most what is left: the roundings of the row's own
    K values, of variance 2^-16 / 3 at most, six standard deviations 6 2^-8 (3 / K)^0.5 / 3^0.5 = 2^-11.4 for
    normal values; the other entries' roundings, u = 2^-8 of each at most; and 2^-14 for fp32's.  A row of dW has
    the roundings of m h too, with m in (1/2, 1] the token's own factor: one for each of the 128 significands that
    a bf16 h has, the largest with up to 1.5 / 128 of the row's square: 2^-8 (1.5 / 128 / 3)^0.5 = 2^-12 of
    standard deviation, or, with m within 2^-9 of 1, which is one token in 2^8, up to 2^-9 that is alike for all.
    So no row of dW more than 2^-9, and their root mean square (three of 64 such tokens: (3 2^-18 / 64 + 2^-24)^0.5)
    at most 2^-11."""
    dev = device()
    N, V, K, top = 64, 900, 4096, 6
    c, d = make(N, V, K, top, BF, 44, dev, T, ignored=0.0, near=False)
    c["index"] = torch.randperm(V, generator=torch.Generator().manual_seed(1))[:N * top].view(N, top)
    share = torch.rand(N, top, generator=torch.Generator().manual_seed(2)).double() + 0.1
    first = sure + (1 - sure) * torch.rand(N, generator=torch.Generator().manual_seed(3)).double()
    share[:, 0] = 0
    share = share / share.sum(1, keepdim=True) * (1 - first[:, None])
    share[:, 0] = first
    c["logit"] = (share.log() * T).float()
    c["index"][::3], c["logit"][::3] = c["index"][::3].flip(1), c["logit"][::3].flip(1)
    c["g"] = torch.rand(N, generator=torch.Generator().manual_seed(4)) + 0.5
    d.update({k: c[k].to(dev) for k in ("index", "logit", "g")})
    announce("distill dominating entry", sure, T)
    _, lse = forward(d)
    dh, dW = (t.double().cpu() for t in backward(d, lse))
    r = reference(c)
    wh, _, wW, _ = grad_reference(c, r)
    h, W = c["h"].double(), c["W"].double()
    at = c["index"].gather(1, c["logit"].argmax(1, keepdim=True))[:, 0]
    rows = torch.arange(N)
    p = (r["l"] - r["lse"][:, None]).exp().scatter_add_(1, r["at"], -r["t"]) * (c["g"].double() / T)[:, None]
    p[rows, at] = 0.0                                      # the others
    own, u = 6 * 2.0 ** -8 / K ** 0.5, 2.0 ** -8
    for err, want, left, room in ((dh - wh, wh, p.abs() * (wh @ W.t()).abs(), own),
                                  (dW[at] - wW[at], wW[at], (p.abs() * (h @ wW.t()).abs())[:, at].t(), own + 2.0 ** -9)):
        size = (want * want).sum(1)
        along, rest = ((err * want).sum(1) / size).abs(), u * left.sum(1) / size + 2.0 ** -14
        assert (along <= room + rest).all(), (along.max(), room)
        assert (along - rest).clamp(min=0).square().mean().sqrt() <= 2.0 ** -11


@pytest.mark.parametrize("kind", ["mean", "two", "random"])
def test_no_rounding_of_g_reaches_all_values(kind):
    """bf16, g that lie 2^-8 of themselves from the nearest bf16 value (both of `two` in the same direction): the
    part of dh's and dW's error along dh and dW themselves.  A g rounded to bf16 makes it 14.3 2^-12 (mean) and
    12.3 2^-12 (two; 14.3 and 11.2 2^-12 in the halves of dh); `random` g are rounded in all directions.  What may
    be there: the final roundings, six standard deviations 6 2^-8 (3 / (N K))^0.5 / 3^0.5 < 2^-14; those of p, of
    which each entry's share is p_iv <W_v, dh_i> / |dh|^2 (six deviations of their sum, computed below); 2^-13 for
    values of unequal size; and for dW the rounding of m h, one for each of the 128 significands of h, which is the
    same m for half of the tokens of `two`: six deviations of half of 2^-8 (1.5 / 128 / 3)^0.5, 3 2^-12."""
    dev = device()
    N, V, K = 300, 2000, 512
    c, d = make(N, V, K, 16, BF, 16, dev, ignored=0.1, near=False)
    one, other = 2.0 ** -8 * (1 + 0.9 * 2.0 ** -8), 1.25 * 2.0 ** -8 * (1 + 0.7 * 2.0 ** -8)
    g = {"mean": torch.full((N,), one), "two": torch.where(torch.arange(N) % 2 == 0, one, other), "random": c["g"]}[kind]
    c["g"], d["g"] = g, g.to(dev)
    announce("distill rounding of g", kind)
    _, lse = forward(d)
    dh, dW = (t.double().cpu() for t in backward(d, lse))
    r = reference(c)
    wh, _, wW, _ = grad_reference(c, r)
    h, W = c["h"].double(), c["W"].double()
    p = (r["l"] - r["lse"][:, None]).exp().scatter_add_(1, r["at"], -r["t"]) * torch.where(r["counts"], g.double(), 0.0)[:, None]
    along = lambda err, want: abs(((err * want).sum() / (want * want).sum()).item())
    for got, want, shares, more in ((dh, wh, p * (wh @ W.t()), 0.0), (dW, wW, p * (h @ wW.t()), 3 * 2.0 ** -12)):
        own = 6 * 2.0 ** -8 / 3 ** 0.5 * shares.square().sum().sqrt().item() / (want * want).sum().item()
        limit = 2.0 ** -12 + own + more
        assert limit < 10 * 2.0 ** -12                     # a rounded g is seen
        assert along(got - want, want) <= limit, (along(got - want, want), limit)
    if kind == "two":                                       # each half by itself
        for half in (0, 1):
            want = wh[half::2]
            own = 6 * 2.0 ** -8 / 3 ** 0.5 * (p * (wh @ W.t()))[half::2].square().sum().sqrt().item() / (want * want).sum().item()
            assert along((dh - wh)[half::2], want) <= 2.0 ** -12 + own < 10 * 2.0 ** -12


@pytest.mark.parametrize("dt", [BF, F32])
def test_the_most_tokens(dt):
    """2^20 tokens with lists of 128: rows from both ends and between, as in test_gpu_distill.py; the gradient of W
    of tokens that do not count but for those rows."""
    dev = device()
    N, V, K, top = 1 << 20, 70, 64, 128
    g = torch.Generator(device=dev).manual_seed(51)
    d = {"h": torch.randn(N, K, generator=g, device=dev).to(dt), "W": (torch.randn(V, K, generator=g, device=dev) / 8).to(dt),
         "index": torch.randint(-20, V + 20, (N, top), generator=g, device=dev),
         "logit": torch.randn(N, top, generator=g, device=dev), "g": torch.rand(N, generator=g, device=dev), "T": 1.0}
    rows = torch.cat([torch.arange(500), torch.arange(N // 2 - 250, N // 2 + 250), torch.arange(N - 500, N)]).to(dev)
    few = {k: v[rows] if k not in ("W", "T") else v for k, v in d.items()}
    announce("distill most tokens", dt)
    loss, lse = forward(d)
    r = reference(few)
    close(lse[rows], r["lse"], r["dl"], "lse")
    close(loss[rows], r["loss"], r["dloss"], "loss")
    dh, _ = backward(d, lse, want_dW=False)
    wh, bh, wW, bW = grad_reference(few, r)
    close(dh[rows], wh, bh, "dh")
    others = torch.ones(N, dtype=torch.bool, device=dev)
    others[rows] = False
    d["index"][others] = -1
    dh2, dW = backward(d, lse)
    assert not dh2[others].any()
    close(dh2[rows], wh, bh, "dh alone")
    close(dW, wW, bW, "dW")
