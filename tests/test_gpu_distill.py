"""Distillation from a teacher's top logits (fairy2i_distill) and its gradient against the formulas in 64 bits.

Tolerances from the arithmetic, with u the inputs' unit roundoff (finfo.eps / 2), T the temperature, t the
teacher's probabilities and z its listed logits over T:
  logit   d_iv = (K + 8) 2^-24 sum_k |h_ik W_vk| / T, for fp32 operands 2^-23 of the same sum more (products of
          their smallest parts left out), and 2^-23 |l_iv| (1 / T and the product with it are rounded)
  lse     max_v d_iv + 2^-18 + 2^-22 |lse|                        (exponentials and their sum: 64 roundings)
  t       relative e_i = 2^-21 max |z| + 2^-19                    (z is rounded twice; two exponentials, a sum
          of at most 128 and a quotient)
  loss    sum_k t (e_i (1 + |log t - l + lse|) + d) + lse's + 2^-20 + 2^-17 sum_k t (|log t| + |l|) / 2^3
          + 2^-22 (|lse| + |loss|)                                (two sums of at most 128 terms)
  p       |g| / T (softmax (d + lse's + 2^-20) + t (e_i + 2^-22)) + u |p|
  dh, dW  the p's errors through the product, (V + 16) or (N + 16) 2^-24 of the absolute terms for the fp32
          sums, and u of the result; for bf16 dW one rounding (u) of its other operand more, which is h times
          the g's own factor."""
import math

import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def make(N, V, K, top, dt, seed, dev, temperature=1.0, tdt=F32, ignored=0.2, spread=1.0, near=True):
    """Lists of different lengths in random order; every fifth token has an entry listed twice."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, K, generator=g).to(dt)
    W = (torch.randn(V, K, generator=g) * spread * K ** -0.5).to(dt)
    index = torch.stack([torch.randperm(V, generator=g)[:top] if V >= top else torch.randint(0, V, (top,), generator=g)
                         for _ in range(N)])
    logit = torch.randn(N, top, generator=g) * 2
    if near:                                              # a teacher that agrees with the student, mostly
        logit = logit + (h.float()[:, None, :] * W.float()[index]).sum(2) * 2
    length = torch.randint(1, top + 1, (N,), generator=g)
    length[torch.rand(N, generator=g) < ignored] = 0
    used = torch.arange(top)[None, :] < length[:, None]
    other = torch.tensor([-1, V, 1 << 40, -(1 << 35)])[torch.arange(N * top) % 4].view(N, top)
    index = torch.where(used, index, other)
    if top >= 2:
        index[::5, 1] = index[::5, 0]                    # listed twice
    logit[~used] = float("nan")                          # unused slots may hold anything
    if top >= 2:
        logit[::5, 1] = torch.where(length[::5] > 0, torch.randn(len(length[::5]), generator=g), logit[::5, 1])
    if top >= 4:
        logit[1::7, 3] = float("-inf")                   # probability 0
    c = {"h": h, "W": W, "index": index, "logit": logit.to(tdt), "g": torch.rand(N, generator=g) / N, "T": temperature}
    return c, {k: v.to(dev) if torch.is_tensor(v) else v for k, v in c.items()}


def reference(c):
    h, W, T = c["h"].double(), c["W"].double(), c["T"]
    N, K = h.shape
    V = W.shape[0]
    l = h @ W.t() / T
    size = h.abs() @ W.abs().t() / T
    d = (K + 8) * E24 * size + (2.0 ** -23 * size if c["h"].dtype == F32 else 0.0) + 2.0 ** -23 * l.abs()
    lse = torch.logsumexp(l, 1)
    dl = d.max(1).values + 2.0 ** -18 + 2.0 ** -22 * lse.abs()
    index = c["index"]
    used = (index >= 0) & (index < V)
    z = torch.where(used, c["logit"].double() / T, torch.full((), -math.inf, dtype=torch.float64, device=h.device))
    counts = (z > -math.inf).any(1)
    t = torch.where(counts[:, None], torch.softmax(torch.where(counts[:, None], z, torch.zeros_like(z)), 1), torch.zeros_like(z))
    log_t = torch.where(t > 0, t.log(), torch.zeros_like(t))
    at = index.clamp(0, V - 1)
    la = l.gather(1, at)
    terms = torch.where(t > 0, log_t - la + lse[:, None], torch.zeros_like(t))
    loss = (t * terms).sum(1)
    e = 2.0 ** -21 * torch.where(z > -math.inf, z.abs(), torch.zeros_like(z)).max(1).values + 2.0 ** -19
    bound = ((t * (e[:, None] * (1 + terms.abs()) + d.gather(1, at))).sum(1) + dl + 2.0 ** -20
             + 2.0 ** -20 * (t * (log_t.abs() + la.abs())).sum(1) + 2.0 ** -22 * (lse.abs() + loss.abs()))
    return {"l": l, "d": d, "lse": lse, "dl": dl, "t": t, "e": e, "at": at, "counts": counts, "loss": loss,
            "dloss": torch.where(counts, bound, torch.zeros_like(bound))}


def grad_reference(c, r=None):
    r = r or reference(c)
    h, W = c["h"].double(), c["W"].double()
    N, V = r["l"].shape
    u = torch.finfo(c["h"].dtype).eps / 2
    g = torch.where(r["counts"], c["g"].double(), torch.zeros_like(r["lse"])) / c["T"]
    soft = (r["l"] - r["lse"][:, None]).exp()
    teacher = torch.zeros_like(soft).scatter_add_(1, r["at"], r["t"])
    p = (soft - teacher) * g[:, None]
    ep = (g.abs()[:, None] * (soft * (r["d"] + r["dl"][:, None] + 2.0 ** -20) + teacher * (r["e"][:, None] + 2.0 ** -22))
          + u * p.abs())
    dh, dW = p @ W, p.t() @ h
    bh = ep @ W.abs() + (V + 16) * E24 * (p.abs() @ W.abs()) + u * dh.abs()
    bW = ep.t() @ h.abs() + ((N + 16) * E24 + (u if u > E24 else 0.0)) * (p.abs().t() @ h.abs()) + u * dW.abs()
    return dh, bh, dW, bW


def close(got, want, bound, label):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), label
    over = ((got - want.cpu()).abs() - bound.cpu()).max().item()
    assert over <= 0, (label, over)


def forward(d, **kw):
    return f2.fairy2i_distill(d["h"], d["W"], d["index"], d["logit"], d["T"], **kw)


def backward(d, lse, **kw):
    return f2.fairy2i_distill_backward(d["h"], d["W"], d["index"], d["logit"], lse, d["g"], d["T"], **kw)


def check(c, d, label):
    announce("distill", label)
    loss, lse = forward(d)
    r = reference(c)
    close(lse, r["lse"], r["dl"], ("lse", label))
    close(loss, r["loss"], r["dloss"], ("loss", label))
    assert not loss.cpu()[~r["counts"].cpu()].any()
    announce("distill gradient", label)
    nan = lambda t: torch.full_like(t, float("nan"))
    dh, dW = backward(d, lse, dh=nan(d["h"]), dW=nan(d["W"]))
    wh, bh, wW, bW = grad_reference(c, r)
    close(dh, wh, bh, ("dh", label))
    close(dW, wW, bW, ("dW", label))
    assert not dh.cpu()[~r["counts"].cpu()].any()
    return loss, lse, dh, dW


SIZES = [(1, 1, 64, 1), (1, 5000, 128, 128), (3, 17, 64, 5), (16, 257, 192, 7), (33, 1000, 256, 32), (65, 129, 64, 128),
         (130, 8193, 128, 3), (128, 128, 1088, 64), (257, 33, 320, 2), (300, 16500, 64, 19)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "N%d-V%d-K%d-top%d" % s)
def test_loss_and_gradient(size, dt):
    dev = device()
    for T, tdt in ((1.0, F32), (2.5, BF)):
        c, d = make(*size, dt, 5, dev, T, tdt)
        if size[0] == 1:
            c["index"][0, 0] = 0
            c["logit"][0, 0] = 1.0
            d["index"], d["logit"] = c["index"].to(dev), c["logit"].to(dev)
        _, lse, dh, dW = check(c, d, (size, dt, T, tdt))
        only_h, only_W = backward(d, lse, want_dW=False), backward(d, lse, want_dh=False)
        assert only_h[1] is None and only_W[0] is None
        assert torch.equal(only_h[0], dh) and torch.equal(only_W[1], dW)


# one size for each tile shape that the products may take, with two pieces among them
LARGE = [(2048, 16384, 64, 8), (2048, 9000, 192, 128), (1000, 8200, 256, 1), (600, 12000, 1024, 33), (2048, 2000, 4096, 16),
         (1024, 2000, 4096, 100), (256, 8192, 2048, 10), (64, 4000, 4096, 64), (4096, 1000, 4096, 12)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("size", LARGE, ids=lambda s: "N%d-V%d-K%d-top%d" % s)
def test_large_tiles(size, dt):
    """Sizes that fill the device with larger tiles; the 64-bit reference runs on the GPU."""
    dev = device()
    _, d = make(*size, dt, 15, dev, 1.7)
    check(d, d, ("large", size, dt))


def test_a_list_of_one_is_the_cross_entropy():
    """One listed entry has probability 1: the loss is the vocabulary loss, and so is the gradient, each
    within its own bounds of the formula."""
    dev = device()
    c, d = make(50, 700, 128, 1, F32, 3, dev, ignored=0.3)
    announce("distill top 1")
    loss, lse = forward(d)
    target = d["index"][:, 0].contiguous()
    l2, s2 = f2.fairy2i_vocab_loss(d["h"], d["W"], target)
    r = reference(c)
    assert torch.equal(lse, s2)
    assert ((loss - l2).abs().cpu() <= 2 * r["dloss"]).all()
    dh, dW = backward(d, lse)
    h2, W2 = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], target, s2, d["g"])
    _, bh, _, bW = grad_reference(c, r)
    assert ((dh - h2).abs().cpu() <= 2 * bh).all() and ((dW - W2).abs().cpu() <= 2 * bW).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_teacher_that_is_the_student(dt):
    """The whole vocabulary listed with the student's own logits: loss and gradient are what rounding leaves."""
    dev = device()
    N, V, K = 40, 100, 64
    c, d = make(N, V, K, 100, dt, 4, dev, 2.0, ignored=0.0)
    c["index"] = torch.arange(V).flip(0).repeat(N, 1)
    c["logit"] = (c["h"].double() @ c["W"].double().t()).float().flip(1)
    d.update(index=c["index"].to(dev), logit=c["logit"].to(dev))
    loss, _, dh, dW = check(c, d, ("self", dt))
    assert loss.abs().max() <= 2.0 ** -15 and dh.abs().max() <= 2.0 ** -15


def test_lists_of_every_kind():
    """An entry listed many times, in and out of tile borders; minus infinity everywhere; nothing listed;
    order of the list; a huge index."""
    dev = device()
    N, V, K, top = 9, 600, 64, 128
    c, d = make(N, V, K, top, F32, 6, dev, ignored=0.0)
    c["index"][0] = 127
    c["index"][1] = torch.tensor([127, 128, 255, 256, 511, 512, 599, 0]).repeat(16)
    c["logit"][0:2] = torch.randn(2, top, generator=torch.Generator().manual_seed(1))
    c["index"][2], c["logit"][2] = torch.arange(top), float("-inf")
    c["index"][3] = -1
    c["index"][4] = (1 << 32) + 5                        # not entry 5
    c["index"][5] = torch.arange(top) + 400
    c["logit"][5] = torch.randn(top, generator=torch.Generator().manual_seed(2))
    c["logit"][5, 60:] = float("-inf")
    c["index"][6], c["logit"][6] = c["index"][5].flip(0), c["logit"][5].flip(0)
    c["h"][6] = c["h"][5]
    d.update({k: c[k].to(dev) for k in ("index", "logit", "h")})
    loss, _, dh, _ = check(c, d, "kinds")
    assert loss[2] == 0 and loss[3] == 0 and loss[4] == 0 and not dh[2:5].any()


@pytest.mark.parametrize("dt", [BF, F32])
def test_wide_logits(dt):
    """Student's and teacher's logits hundreds apart."""
    dev = device()
    c, d = make(40, 700, 64, 20, dt, 6, dev, spread=150.0)
    announce("distill wide logits", dt)
    loss, lse = forward(d)
    r = reference(c)
    close(lse, r["lse"], r["dl"], "lse")
    close(loss, r["loss"], r["dloss"], "loss")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", [20, 300])
def test_padding_reaches_no_gradient(dt, N):
    """Whatever lies in rows of h that do not count (no list, or g = 0): dh and dW are the same."""
    dev = device()
    c, d = make(N, 700, 128, 16, dt, 23, dev, ignored=0.0)
    d["index"][N - 6:] = -1
    d["g"][3] = 0.0
    d["h"][N - 6:] = 0.0
    _, lse = forward(d)
    announce("distill padding", dt, N)
    dh, dW = backward(d, lse)
    bad = dict(d, h=d["h"].clone())
    bad["h"][N - 6:N - 3] = float("nan")
    bad["h"][N - 3:] = float("inf")
    bad["h"][3] = float("nan")
    loss2, lse2 = forward(bad)
    assert not loss2[N - 6:].any()
    dh2, dW2 = backward(bad, lse2)
    assert torch.equal(dh2, dh) and torch.equal(dW2, dW) and torch.isfinite(dW).all()


def test_bad_values_stay_apart():
    """NaN or plus infinity in a used slot: that token's loss and dh; a NaN row of h likewise."""
    dev = device()
    c, d = make(20, 300, 64, 8, BF, 8, dev, ignored=0.0)
    loss, lse = forward(d)
    dh, _ = backward(d, lse)
    for what, value in (("logit", float("nan")), ("logit", float("inf")), ("h", float("nan"))):
        bad = dict(d)
        bad[what] = d[what].clone()
        bad[what][4, 0] = value
        announce("distill bad values", what, value)
        loss2, lse2 = forward(bad)
        dh2, _ = backward(bad, lse2, want_dW=False)
        keep = [i for i in range(20) if i != 4]
        assert torch.isnan(loss2[4]) and torch.equal(loss2[keep], loss[keep])
        assert torch.isnan(dh2[4]).any() and torch.equal(dh2[keep], dh[keep])


@pytest.mark.parametrize("kind", ["mean", "two", "random"])
def test_rounding_is_not_common_to_all_values(kind):
    """bf16: the part of dh's and dW's error along dh and dW themselves, which a rounding shared by all values
    (of g, say) would make up to 2^-8.  Independent roundings of N K >= 2^17 values of at most 2^-8 each
    leave under 2^-8 * 6 / 2^8.5 along any fixed direction (six standard deviations); the p's entries are
    fewer, at least N top >= 2^11 of them that matter, 2^-8 * 6 / 2^5.5 if all were of one size; together with
    values of unequal size under 2^-10."""
    dev = device()
    N, V, K = 300, 2000, 512
    c, d = make(N, V, K, 16, BF, 16, dev, ignored=0.1, near=False)
    g = {"mean": torch.full((N,), 1 / 261.0), "two": torch.where(torch.arange(N) % 2 == 0, 1 / 261.0, 0.7 / 261.0),
         "random": c["g"]}[kind]
    c["g"], d["g"] = g, g.to(dev)
    announce("distill common rounding", kind)
    _, lse = forward(d)
    dh, dW = backward(d, lse)
    wh, _, wW, _ = grad_reference(c)
    for got, want, name in ((dh, wh, "dh"), (dW, wW, "dW")):
        err = got.double().cpu() - want
        along = ((err * want).sum() / (want * want).sum()).item()
        assert abs(along) <= 2.0 ** -10, (name, along)


def wide_weights(kind, N):
    g = torch.linspace(0.5, 1.5, N)
    if kind == "small first":
        g[0], g[1] = 1e-20, 1e20
    elif kind == "subnormal first":
        g[0] = 8e-40
    elif kind == "signs":
        g = torch.randn(N, generator=torch.Generator().manual_seed(4)) * 10.0 ** torch.linspace(-6, 6, N)
        g[0] = 0.0
    elif kind == "all of fp32":
        g = 10.0 ** torch.linspace(-37, 37, N, dtype=torch.float64)[torch.randperm(N, generator=torch.Generator().manual_seed(1))]
    return g.float()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["small first", "subnormal first", "signs", "all of fp32"])
def test_weights_of_any_size(kind, dt):
    """Finite weights give the formula's gradients however far apart they lie.  Beside the bounds above, a value
    under fp32's and bf16's normal range may be held as 0: an output (2^-126), a value of p (2^-126 times |W| or
    |h| and, for bf16, a factor under 4 that is applied afterwards), a term of dW's sums (2^-126, a factor
    under 2)."""
    dev = device()
    N, V, K = 60, 300, 128
    c, d = make(N, V, K, 12, dt, 37, dev, ignored=0.1)
    c["g"] = wide_weights(kind, N)
    d["g"] = c["g"].to(dev)
    announce("distill weights", kind, dt)
    _, lse = forward(d)
    dh, dW = backward(d, lse)
    wh, bh, wW, bW = grad_reference(c)
    tiny = 2.0 ** -126
    close(dh, wh, bh + tiny + 4 * tiny * c["W"].double().abs().sum(0), "dh")
    close(dW, wW, bW + (1 + 2 * N) * tiny + 4 * tiny * c["h"].double().abs().sum(0), "dW")


def test_long_padding_in_front():
    """The first token that counts lies past the ones that are searched for a common factor of g."""
    dev = device()
    N, V, K = 4400, 60, 64
    for kind in ("equal", "different"):
        c, d = make(N, V, K, 4, BF, 31, dev, ignored=0.0)
        c["index"][:4300] = -1
        if kind == "equal":
            c["g"] = torch.full((N,), 0.01)
        d["index"], d["g"] = c["index"].to(dev), c["g"].to(dev)
        check(c, d, ("padding in front", kind))


def test_gradient_against_differences():
    """Along random directions of h and W: central differences of the loss, whose curvature in the logits is
    lse's alone (the listed logits enter it linearly)."""
    dev = device()
    N, V, K, T = 12, 90, 64, 1.25
    c, d = make(N, V, K, 10, F32, 9, dev, T, ignored=0.0)
    loss, lse = forward(d)
    dh, dW = backward(d, lse)
    gsum = d["g"].double().sum().item()
    r = reference(c)
    noise = r["dloss"].max().item()
    for name, grad in (("h", dh), ("W", dW)):
        v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(3)).to(dev)
        v = v / (K ** 0.5 if name == "W" else 1.0)
        t, vals = 2.0 ** -5, []
        for sign in (1, -1):
            e = dict(d)
            e[name] = d[name] + sign * t * v
            announce("distill difference", name, sign)
            vals.append((forward(e)[0].double() * d["g"].double()).sum().item())
        want = (vals[0] - vals[1]) / (2 * t)
        got = (grad.double() * v.double()).sum().item()
        # a logit moves by at most `move` per unit of t; |third derivative of lse| <= 4 move^3
        move = ((v @ d["W"].t()) if name == "h" else (d["h"] @ v.t())).abs().max().item() / T
        bound = gsum * (t * t * 4 * move ** 3 / 6 + 2 * noise / (2 * t))
        assert abs(got - want) <= bound, (name, got, want, bound)
        assert bound <= abs(want), (name, bound, want)       # the comparison says something


def test_streams_graphs_and_shared_workspace():
    dev = device()
    N, V, K, top = 70, 3000, 128, 24
    c, d = make(N, V, K, top, BF, 10, dev, 2.0)
    loss, lse = (t.clone() for t in forward(d))
    dh, dW = (t.clone() for t in backward(d, lse))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    announce("distill on a side stream")
    l2, s2 = forward(d, stream=side)
    g2 = backward(d, s2, stream=side)
    side.synchronize()
    assert torch.equal(l2, loss) and torch.equal(g2[0], dh) and torch.equal(g2[1], dW)
    ws = torch.empty(max(f2.fairy2i_distill_workspace_bytes(N, V, K, f2.BF16, top),
                         f2.fairy2i_distill_backward_workspace_bytes(N, V, K, f2.BF16, top)), dtype=torch.uint8, device=dev)
    announce("distill graphs")
    graphs = []
    for _ in range(2):                                  # two graphs over one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            a = forward(d, workspace=ws)
            b = backward(d, a[1], workspace=ws)
        graphs.append((g, a, b))
    for k in range(4):
        for g, a, b in graphs:
            ws.fill_(255)
            a[0].zero_()
            b[0].fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a[0], loss) and torch.equal(a[1], lse) and torch.equal(b[0], dh) and torch.equal(b[1], dW), k


@pytest.mark.parametrize("dt", [BF, F32])
def test_vocabulary_offsets_past_32_bits(dt):
    """A vocabulary whose last rows lie past 2^32 bytes, listed entries at both ends: the answer in closed form."""
    dev = device()
    K = 1024
    V = (1 << 21) + 77 if dt == BF else (1 << 20) + 77
    announce("distill offsets", dt, V)
    W = torch.zeros((V, K), dtype=dt, device=dev)
    h = torch.zeros((2, K), dtype=dt, device=dev)
    h[:, 0] = 1.0
    W[V - 1, 0], W[5, 0] = 12.0, 3.0
    index = torch.tensor([[V - 1, 5], [V - 2, -1]], device=dev)
    logit = torch.tensor([[math.log(0.75), math.log(0.25)], [9.0, 0.0]], device=dev)
    loss, lse = f2.fairy2i_distill(h, W, index, logit)
    want = math.log(math.exp(12.0) + math.exp(3.0) + (V - 2))
    first = 0.75 * (math.log(0.75) - 12) + 0.25 * (math.log(0.25) - 3) + want
    for i, l in enumerate((first, want)):
        assert abs(lse[i].item() - want) <= 2.0 ** -17 * want and abs(loss[i].item() - l) <= 2.0 ** -17 * want
    dh, _ = f2.fairy2i_distill_backward(h, W, index, logit, lse, torch.ones(2, device=dev), want_dW=False)
    mean = (12 * math.exp(12.0) + 3 * math.exp(3.0)) / math.exp(want)
    u = torch.finfo(dt).eps / 2
    for i, l in enumerate((0.75 * 12 + 0.25 * 3, 0.0)):
        # two or three non-zero terms of size <= 12, each rounded once, and the result
        assert abs(dh[i, 0].item() - (mean - l)) <= 2 * u * 12 + u * abs(mean - l) + 2.0 ** -14
        assert not dh[i, 1:].any()
