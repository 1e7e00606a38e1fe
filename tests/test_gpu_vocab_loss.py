"""Vocabulary cross entropy (fairy2i_vocab_loss) and its gradient against the formulas in 64 bits.

Tolerances from the arithmetic, with u the inputs' unit roundoff (finfo.eps / 2):
  logit   d_iv = (K + 8) 2^-24 sum_k |h_ik W_vk|                  (fp32 sums of exact products), for fp32
          operands 2^-23 of the same sum more                    (products of their smallest parts left out)
  lse     max_v d_iv + 2^-18 + 2^-22 |lse|                        (exponentials and their sum: 64 roundings)
  loss    lse's + d_it + 2^-23 (|lse| + |loss|)
  p       |p| (u + d_iv + lse's + 2^-20) + 2^-23 |g| at the target (one rounding to the inputs' dtype)
  dh, dW  the p's errors through the product, (V + 16) or (N + 16) 2^-24 of the absolute terms for the
          fp32 sums, and u of the result; for bf16 dW one rounding (u) of its other operand more, which
          is h times the g's own factor."""
import math

import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24


def make(N, V, K, dt, seed, dev, ignored=0.2, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, K, generator=g).to(dt)
    W = (torch.randn(V, K, generator=g) * spread * K ** -0.5).to(dt)
    t = torch.randint(0, V, (N,), generator=g)
    skip = torch.rand(N, generator=g) < ignored
    t[skip] = torch.tensor([-100, V, -1, 1 << 40])[torch.arange(int(skip.sum())) % 4]
    gr = torch.rand(N, generator=g) / N
    c = {"h": h, "W": W, "t": t, "g": gr}
    return c, {k: v.to(dev) for k, v in c.items()}


def reference(c):
    h, W, t = c["h"].double(), c["W"].double(), c["t"]
    N, K = h.shape
    V = W.shape[0]
    z = h @ W.t()
    d = (K + 8) * E24 * (h.abs() @ W.abs().t()) + (2.0 ** -23 * (h.abs() @ W.abs().t()) if c["h"].dtype == torch.float32 else 0.0)
    lse = torch.logsumexp(z, 1)
    dl = d.max(1).values + 2.0 ** -18 + 2.0 ** -22 * lse.abs()
    ok = (t >= 0) & (t < V)
    at = t.clamp(0, V - 1)
    row = torch.arange(N, device=z.device)
    loss = torch.where(ok, lse - z[row, at], torch.zeros_like(lse))
    dloss = torch.where(ok, dl + d[row, at] + 2.0 ** -23 * (lse.abs() + loss.abs()), torch.zeros_like(lse))
    return z, d, lse, dl, loss, dloss, ok, at


def grad_reference(c):
    z, d, lse, dl, _, _, ok, at = reference(c)
    h, W = c["h"].double(), c["W"].double()
    N, V = z.shape
    u = torch.finfo(c["h"].dtype).eps / 2
    row = torch.arange(N, device=z.device)
    g = torch.where(ok, c["g"].double(), torch.zeros_like(lse))
    soft = (z - lse[:, None]).exp()
    p = soft.clone()
    p[row, at] -= 1.0
    p = p * g[:, None]
    ep = g.abs()[:, None] * soft * (d + dl[:, None] + 2.0 ** -20) + u * p.abs()
    ep[row, at] += 2.0 ** -23 * g.abs()
    dh, dW = p @ W, p.t() @ h
    bh = ep @ W.abs() + (V + 16) * E24 * (p.abs() @ W.abs()) + u * dh.abs()
    bW = ep.t() @ h.abs() + ((N + 16) * E24 + (u if u > E24 else 0.0)) * (p.abs().t() @ h.abs()) + u * dW.abs()
    return dh, bh, dW, bW


def close(got, want, bound, label):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), label
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, (label, over)


SIZES = [(1, 1, 64), (1, 5000, 128), (3, 17, 64), (16, 257, 192), (33, 1000, 256), (65, 129, 64), (130, 8193, 128),
         (128, 128, 1088), (257, 33, 320), (300, 16500, 64)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "N%d-V%d-K%d" % s)
def test_loss_and_gradient(size, dt):
    dev = device()
    c, d = make(*size, dt, 5, dev)
    N, V, K = size
    announce("vocab loss", size, dt)
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    _, _, wl, bl, wo, bo, ok, _ = reference(c)
    close(lse, wl, bl, "lse")
    close(loss, wo, bo, "loss")
    assert not loss.cpu()[~ok].any()
    announce("vocab gradient", size, dt)
    nan = lambda t: torch.full_like(t, float("nan"))
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"], dh=nan(d["h"]), dW=nan(d["W"]))
    wh, bh, wW, bW = grad_reference(c)
    close(dh, wh, bh, "dh")
    close(dW, wW, bW, "dW")
    assert not dh.cpu()[~ok].any()
    only_h = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"], want_dW=False)
    only_W = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"], want_dh=False)
    assert only_h[1] is None and only_W[0] is None
    assert torch.equal(only_h[0], dh) and torch.equal(only_W[1], dW)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_wide_logits(dt):
    """Logits hundreds apart: the running maximum keeps every exponential in range."""
    dev = device()
    c, d = make(40, 700, 64, dt, 6, dev, spread=150.0)
    announce("vocab wide logits", dt)
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    _, _, wl, bl, wo, bo, _, _ = reference(c)
    close(lse, wl, bl, "lse")
    close(loss, wo, bo, "loss")


# one size for each tile shape that the gradient's and the loss's products may take, with two pieces
LARGE = [(2048, 16384, 64), (2048, 9000, 192), (1000, 8200, 256), (600, 12000, 1024), (2048, 2000, 4096),
         (1024, 2000, 4096), (256, 8192, 2048), (64, 4000, 4096), (4096, 1000, 4096)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", LARGE, ids=lambda s: "N%d-V%d-K%d" % s)
def test_large_tiles(size, dt):
    """Sizes that fill the device with larger tiles; the 64-bit reference runs on the GPU."""
    dev = device()
    _, d = make(*size, dt, 15, dev)
    announce("vocab large", size, dt)
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    _, _, wl, bl, wo, bo, _, _ = (x.cpu() for x in reference(d))
    close(lse, wl, bl, "lse")
    close(loss, wo, bo, "loss")
    wh, bh, wW, bW = (x.cpu() for x in grad_reference(d))
    close(dh, wh, bh, "dh")
    close(dW, wW, bW, "dW")


@pytest.mark.parametrize("kind", ["mean", "two", "random"])
def test_rounding_is_not_common_to_all_values(kind):
    """bf16: the part of dh's and dW's error along dh and dW themselves, which a rounding shared by all
    values (of -g at the targets, say) would make up to 2^-8.  Independent roundings of N K >= 2^17
    values of at most 2^-8 each leave under 2^-8 * 6 / 2^8.5 along any fixed direction (six standard
    deviations); 2^-12 allows for values of unequal size.  The one rounding that is alike for all tokens
    is that of the target's entry, -(1 - p): -1 is a bf16 value, so the rounded entry is off by at most
    its distance from it, p, which adds at most sum_i |g_i| p_i |<W_t, dh_i>| / |dh|^2 along dh (with h
    and dW in their place along dW)."""
    dev = device()
    N, V, K = 300, 2000, 512
    c, d = make(N, V, K, torch.bfloat16, 16, dev, ignored=0.1)
    g = {"mean": torch.full((N,), 1 / 261.0), "two": torch.where(torch.arange(N) % 2 == 0, 1 / 261.0, 0.7 / 261.0),
         "random": c["g"]}[kind]
    c["g"], d["g"] = g, g.to(dev)
    announce("vocab common rounding", kind)
    _, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    wh, _, wW, _ = grad_reference(c)
    z, _, l64, _, _, _, ok, at = reference(c)
    h, W = c["h"].double(), c["W"].double()
    p = torch.where(ok, c["g"].double() * (z[torch.arange(N), at] - l64).exp(), torch.zeros(N, dtype=torch.float64))
    alike = {"dh": p * (W[at] * wh).sum(1).abs(), "dW": p * (h * wW[at]).sum(1).abs()}
    for got, want, name in ((dh, wh, "dh"), (dW, wW, "dW")):
        err = got.double().cpu() - want
        along = ((err * want).sum() / (want * want).sum()).item()
        assert abs(along) <= 2.0 ** -12 + (alike[name].sum() / (want * want).sum()).item(), (name, along)
    if kind == "two":                                       # each half by itself
        for half in (0, 1):
            err, want = (dh.double().cpu() - wh)[half::2], wh[half::2]
            room = 2.0 ** -12 + (alike["dh"][half::2].sum() / (want * want).sum()).item()
            assert abs(((err * want).sum() / (want * want).sum()).item()) <= room, half


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_weights_of_every_kind(dt):
    """g of both signs, zero, tiny and huge (zero in the first token), against the formula."""
    dev = device()
    N, V, K = 40, 500, 128
    c, d = make(N, V, K, dt, 17, dev, ignored=0.1)
    g = torch.randn(N, generator=torch.Generator().manual_seed(4)) * 10.0 ** torch.linspace(-6, 6, N)
    g[0] = 0.0
    c["g"], d["g"] = g, g.to(dev)
    announce("vocab weights", dt)
    _, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    wh, bh, wW, bW = grad_reference(c)
    close(dh, wh, bh, "dh")
    close(dW, wW, bW, "dW")
    d["h"][0] = float("nan")                                # g = 0: adds nothing
    dh2, _ = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"], want_dW=False)
    assert torch.equal(dh2, dh)


def test_long_padding_in_front():
    """The first token that counts lies past the ones that are searched for a common factor of g: the
    gradients of the others, equal g and different ones, are the formula's."""
    dev = device()
    N, V, K = 4400, 60, 64
    for kind in ("equal", "different"):
        c, d = make(N, V, K, torch.bfloat16, 31, dev, ignored=0.0)
        c["t"][:4300] = -100
        if kind == "equal":
            c["g"] = torch.full((N,), 0.01)
        d["t"], d["g"] = c["t"].to(dev), c["g"].to(dev)
        announce("vocab padding in front", kind)
        _, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
        dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
        wh, bh, wW, bW = grad_reference(c)
        close(dh, wh, bh, "dh")
        close(dW, wW, bW, "dW")


def test_no_token_counts():
    dev = device()
    c, d = make(9, 100, 64, torch.bfloat16, 7, dev)
    d["t"].fill_(-100)
    announce("vocab no token counts")
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    assert not loss.any() and not dh.any() and not dW.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [20, 300])
def test_padding_reaches_no_gradient(dt, N):
    """Whatever lies in rows of h that do not count (target -100, or g = 0): dh and dW are the same."""
    dev = device()
    c, d = make(N, 700, 128, dt, 23, dev, ignored=0.0)
    d["t"][N - 6:] = -100
    d["g"][3] = 0.0
    d["h"][N - 6:] = 0.0
    _, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    announce("vocab padding", dt, N)
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    bad = d["h"].clone()
    bad[N - 6:N - 3] = float("nan")
    bad[N - 3:] = float("inf")
    bad[3] = float("nan")
    loss2, lse2 = f2.fairy2i_vocab_loss(bad, d["W"], d["t"])
    assert not loss2[N - 6:].any()
    dh2, dW2 = f2.fairy2i_vocab_loss_backward(bad, d["W"], d["t"], lse2, d["g"])
    assert torch.equal(dh2, dh) and torch.equal(dW2, dW)


def test_bad_rows_stay_apart():
    """A NaN row and an infinite one: their own loss and dh only; NaN in a row that does not count
    reaches no gradient."""
    dev = device()
    c, d = make(20, 300, 64, torch.bfloat16, 8, dev, ignored=0.0)
    d["t"][4] = -100
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    bad = d["h"].clone()
    bad[4] = float("nan")
    announce("vocab NaN in an ignored row")
    loss2, lse2 = f2.fairy2i_vocab_loss(bad, d["W"], d["t"])
    keep = [i for i in range(20) if i != 4]
    assert loss2[4] == 0 and torch.isnan(lse2[4]) and torch.equal(lse2[keep], lse[keep]) and torch.equal(loss2[keep], loss[keep])
    dh2, _ = f2.fairy2i_vocab_loss_backward(bad, d["W"], d["t"], lse2, d["g"], want_dW=False)
    assert torch.equal(dh2, dh)
    bad[2] = float("inf")
    announce("vocab infinite row")
    loss3, lse3 = f2.fairy2i_vocab_loss(bad, d["W"], d["t"])
    keep = [i for i in range(20) if i not in (2, 4)]
    assert not torch.isfinite(lse3[2]) and torch.equal(lse3[keep], lse[keep]) and torch.equal(loss3[keep], loss[keep])


def test_gradient_against_differences():
    """Along random directions of h and W: central differences of the loss.  The loss is smooth with
    third derivatives under 2 |v|^3-like terms of the logits' change; with t = 2^-7 and unit-size
    logit directions the truncation is under t^2 of the gradient's own scale."""
    dev = device()
    N, V, K = 12, 90, 64
    c, d = make(N, V, K, torch.float32, 9, dev, ignored=0.0)
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    gsum = d["g"].double().sum().item()
    for name, grad in (("h", dh), ("W", dW)):
        v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(3)).to(dev)
        v = v / (K ** 0.5 if name == "W" else 1.0)
        t, vals = 2.0 ** -7, []
        for sign in (1, -1):
            e = dict(d)
            e[name] = d[name] + sign * t * v
            announce("vocab difference", name, sign)
            vals.append((f2.fairy2i_vocab_loss(e["h"], e["W"], e["t"])[0].double() * d["g"].double()).sum().item())
        want = (vals[0] - vals[1]) / (2 * t)
        got = (grad.double() * v.double()).sum().item()
        # a logit moves by q = <direction>, at most `move`; |third derivative of lse| <= 4 move^3
        move = ((v @ d["W"].t()) if name == "h" else (d["h"] @ v.t())).abs().max().item()
        bound = gsum * (t * t * 4 * move ** 3 / 6 + 2 * 2.0 ** -17 / (2 * t))
        assert abs(got - want) <= bound, (name, got, want, bound)


def test_streams_graphs_and_shared_workspace():
    dev = device()
    N, V, K = 70, 3000, 128
    c, d = make(N, V, K, torch.bfloat16, 10, dev)
    loss, lse = (t.clone() for t in f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"]))
    dh, dW = (t.clone() for t in f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    announce("vocab on a side stream")
    l2, s2 = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"], stream=side)
    g2 = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], s2, d["g"], stream=side)
    side.synchronize()
    assert torch.equal(l2, loss) and torch.equal(g2[0], dh) and torch.equal(g2[1], dW)
    bf = f2.BF16
    ws = torch.empty(max(f2.fairy2i_vocab_loss_workspace_bytes(N, V, K, bf),
                         f2.fairy2i_vocab_loss_backward_workspace_bytes(N, V, K, bf)), dtype=torch.uint8, device=dev)
    announce("vocab graphs")
    graphs = []
    for _ in range(2):                                  # two graphs over one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            a = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"], workspace=ws)
            b = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], a[1], d["g"], workspace=ws)
        graphs.append((g, a, b))
    for k in range(4):
        for g, a, b in graphs:
            ws.fill_(255)
            a[0].zero_()
            b[0].fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a[0], loss) and torch.equal(a[1], lse) and torch.equal(b[0], dh) and torch.equal(b[1], dW), k


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_vocabulary_offsets_past_32_bits(dt):
    """A vocabulary whose last rows lie past 2^32 bytes: tokens whose targets sit there, few hidden
    columns elsewhere zero, so that the whole answer is known in closed form."""
    dev = device()
    K = 1024
    V = (1 << 21) + 77 if dt == torch.bfloat16 else (1 << 20) + 77     # 2^32 bytes and more
    N = 3
    announce("vocab offsets", dt, V)
    W = torch.zeros((V, K), dtype=dt, device=dev)
    h = torch.zeros((N, K), dtype=dt, device=dev)
    h[:, 0] = 1.0
    W[V - 1, 0] = 12.0
    W[5, 0] = 3.0
    t = torch.tensor([V - 1, 5, V - 2], device=dev)
    loss, lse = f2.fairy2i_vocab_loss(h, W, t)
    want = math.log(math.exp(12.0) + math.exp(3.0) + (V - 2))
    for i, l in enumerate((12.0, 3.0, 0.0)):
        assert abs(lse[i].item() - want) <= 2.0 ** -17 * want and abs(loss[i].item() - (want - l)) <= 2.0 ** -17 * want
    dh, _ = f2.fairy2i_vocab_loss_backward(h, W, t, lse, torch.ones(N, device=dev), want_dW=False)
    mean = (12 * math.exp(12.0) + 3 * math.exp(3.0)) / math.exp(want)
    u = torch.finfo(dt).eps / 2
    for i, l in enumerate((12.0, 3.0, 0.0)):
        # two or three non-zero terms of size <= 12, each rounded once, and the result
        assert abs(dh[i, 0].item() - (mean - l)) <= 2 * u * 12 + u * abs(mean - l) + 2.0 ** -14
        assert not dh[i, 1:].any()


def wide_weights(kind, N):
    """Finite g whose quotients pass fp32's range or fall under it, the first counting one often tiny."""
    g = torch.linspace(0.5, 1.5, N)
    if kind == "small first":
        g[0], g[1] = 1e-20, 1e20
    elif kind == "subnormal first":
        g[0] = 8e-40
    elif kind == "decayed":
        g = 0.9 ** torch.arange(N - 1, -1, -1, dtype=torch.float64)
    elif kind == "large first":
        g[0], g[2], g[3] = 1e20, -1e-20, 1e-30
    elif kind == "all of fp32":
        g = 10.0 ** torch.linspace(-37, 37, N, dtype=torch.float64)[torch.randperm(N, generator=torch.Generator().manual_seed(1))]
    return g.float()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["small first", "subnormal first", "decayed", "large first", "all of fp32"])
def test_weights_of_any_size(kind, dt):
    """Finite weights give the formula's gradients however far apart they lie.  Beside the bounds above, a value
    under fp32's and bf16's normal range may be held as 0: an output (2^-126), a value of p (2^-126 times |W| or
    |h| and, for bf16, a factor under 4 that is applied afterwards), a term of dW's sums (2^-126, a factor
    under 2)."""
    dev = device()
    N, V, K = (1200 if kind == "decayed" else 60), 300, 128
    c, d = make(N, V, K, dt, 37, dev, ignored=0.0)
    c["g"] = wide_weights(kind, N)
    d["g"] = c["g"].to(dev)
    announce("vocab weights of any size", kind, dt)
    _, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    wh, bh, wW, bW = grad_reference(c)
    tiny = 2.0 ** -126
    close(dh, wh, bh + tiny + 4 * tiny * c["W"].double().abs().sum(0), "dh")
    close(dW, wW, bW + (1 + 2 * N) * tiny + 4 * tiny * c["h"].double().abs().sum(0), "dW")


@pytest.mark.parametrize("kind", ["equal", "different"])
def test_target_entry_shifts_no_row(kind):
    """bf16, target probabilities of 0.2 to 0.7 (a head that has learnt): dh_i is mostly the target's entry
    -g_i (1 - p) times W_t, and row t of dW the same times h_i, so a rounding of that entry would move a whole
    row by up to u = 2^-8 of itself.  The part of a row's error along W_t (h_i) is held to independent
    roundings of at most u each -- of the row's own values, of p's other entries, and for dW of m_i h_i --
    which together pass 6 times the root of their squares' sum with a probability under 2 e^-18, plus what
    fp32 costs the softmax and the sums."""
    dev = device()
    N, V, K, u = 256, 2000, 1024, 2.0 ** -8
    gen = torch.Generator().manual_seed(43)
    W = torch.randn(V, K, generator=gen) * K ** -0.5
    t = torch.randperm(V, generator=gen)[:N]
    prob = torch.rand(N, generator=gen) * 0.5 + 0.2
    h = W[t] / (W[t] ** 2).sum(1, keepdim=True) * (V * prob / (1 - prob)).log()[:, None]
    g = torch.full((N,), 1.0 / N) if kind == "equal" else (torch.rand(N, generator=gen) + 0.5) / N
    c = {"h": h.bfloat16(), "W": W.bfloat16(), "t": t, "g": g}
    d = {k: v.to(dev) for k, v in c.items()}
    announce("vocab target entry", kind)
    _, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    z, dz, lse64, dl, _, _, _, at = reference(c)
    h, W, row = c["h"].double(), c["W"].double(), torch.arange(N)
    soft = (z - lse64[:, None]).exp()
    assert 0.15 < soft[row, at].min() and soft[row, at].max() < 0.75
    p = soft.clone()
    p[row, at] -= 1.0
    p = p * g.double()[:, None]
    ep = g.double()[:, None] * soft * (dz + dl[:, None] + 2.0 ** -20)          # fp32's part of p's error
    ep[row, at] += 2.0 ** -23 * g.double()
    rest = p.clone()
    rest[row, at] = 0.0
    Wt = W[at]
    want = p @ W
    cross = (W @ Wt.t()).t()                                                    # <W_v, W_t> [N][V]
    got = ((dh.double().cpu() - want) * Wt).sum(1).abs()
    chance = ((u * want * Wt) ** 2).sum(1) + ((u * rest * cross) ** 2).sum(1)
    sums = (V + 16) * E24 * ((p.abs() @ W.abs()) * Wt.abs()).sum(1)
    over = (got - 6 * chance.sqrt() - (ep * cross.abs()).sum(1) - sums) / (Wt ** 2).sum(1) / g.double()
    assert over.max() <= 0, ("dh", over.max().item(), (over > 0).sum().item())
    want = (p.t() @ h)[at]                                                      # rows t of dW
    mine = p[row, at]
    cross = h @ h.t()                                                           # <h_j, h_i>
    others = rest.t()[at]                                                       # p_jt [row t][j]
    got = ((dW.double().cpu()[at] - want) * h).sum(1).abs()
    chance = ((u * want * h) ** 2).sum(1) + ((u * others * cross) ** 2).sum(1) \
        + ((u * mine[:, None] * h * h) ** 2).sum(1) + ((u * others) ** 2 @ (h * h) * (h * h)).sum(1)
    sums = (N + 16) * E24 * (((p.abs().t() @ h.abs())[at]) * h.abs()).sum(1)
    over = (got - 6 * chance.sqrt() - (ep.t()[at] * cross.abs()).sum(1) - sums) / (h ** 2).sum(1) / g.double()
    assert over.max() <= 0, ("dW", over.max().item(), (over > 0).sum().item())


@pytest.mark.parametrize("w", [1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -8 - 2.0 ** -23, 1.7, -0.6180339, 1.5 + 2.0 ** -8 + 2.0 ** -16])
def test_fp32_product_of_two_values(w):
    """One term and one vocabulary entry, so that lse is the product itself.  Parts rounded to bf16 leave
    |x2| <= 2^-8 and |x3| <= 2^-17 of x's power of two, so the three products left out are within
    (2 2^-25 + 2^-34) of |h W|; the five smaller products are under 2^-6 of it, their sums' roundings (2^-23
    each if the matrix cores cut instead of rounding) under 2^-27 together, and the last sum costs 2^-23."""
    dev = device()
    gen = torch.Generator().manual_seed(47)
    x = torch.cat([torch.tensor([1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -23, -1.0, 1 + 2.0 ** -16, 3.0e38, -3.4e38]),
                   torch.randn(4000, generator=gen), torch.rand(90, generator=gen) * 1e30])
    h = torch.zeros(len(x), 64)
    h[:, 5] = x
    W = torch.zeros(1, 64)
    W[0, 5] = w
    big = 2.0 ** -10 if abs(w) > 1 else 1.0                  # the products stay in range
    W *= big
    announce("vocab fp32 product", w)
    _, lse = f2.fairy2i_vocab_loss(h.to(dev), W.to(dev), torch.zeros(len(x), dtype=torch.int64, device=dev))
    want = x.double() * W[0, 5].double()
    close(lse, want, (2.0 ** -24 + 2.0 ** -33 + 2.0 ** -27 + 2.0 ** -23) * want.abs(), w)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_confident_targets(dt):
    """Targets whose probability leaves from 0.1 down to under 2^-20 of it to the rest (bf16: on both sides of
    where 1 - p_target stays in p), and tokens as sure of another entry: the formula's gradients."""
    dev = device()
    N, V, K = 96, 800, 512
    gen = torch.Generator().manual_seed(53)
    W = torch.randn(V, K, generator=gen) * K ** -0.5
    sure = torch.randperm(V, generator=gen)[:N]
    rest = 10.0 ** torch.linspace(-1, -8, N)
    h = W[sure] / (W[sure] ** 2).sum(1, keepdim=True) * (V / rest).log()[:, None]
    t = torch.where(torch.arange(N) % 3 == 2, (sure + 1) % V, sure)
    c = {"h": h.to(dt), "W": W.to(dt), "t": t, "g": torch.rand(N, generator=gen) + 0.5}
    d = {k: v.to(dev) for k, v in c.items()}
    announce("vocab confident targets", dt)
    loss, lse = f2.fairy2i_vocab_loss(d["h"], d["W"], d["t"])
    z, _, wl, bl, wo, bo, _, at = reference(c)
    f = 1 - (z[torch.arange(N), at] - wl).exp()
    assert (f < 2.0 ** -18).any() and (f > 0.9).any() and ((f > 2.0 ** -15) & (f < 2.0 ** -8)).any()
    close(lse, wl, bl, "lse")
    close(loss, wo, bo, "loss")
    dh, dW = f2.fairy2i_vocab_loss_backward(d["h"], d["W"], d["t"], lse, d["g"])
    wh, bh, wW, bW = grad_reference(c)
    close(dh, wh, bh, "dh")
    close(dW, wW, bW, "dW")
