"""A packed model beside the model it came from, in the run its operators are made for: an original layer and
vocabulary head, the layer packed in two bits (and once kept at four), the head kept at four; the twin drafts,
the original verifies; the twin's output is distilled from the original's top logits, through adapters, and
the gradients are clipped.  Against 64 bits on the values that enter each call, against differences of the
whole run's loss, and captured in a graph."""
import pytest
import torch

from gpu_util import announce, device
from test_gpu_verify import reference as verified

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
S, D, K2, M2, V, R, TOP, TEMP = 6, 3, 384, 256, 900, 8, 12, 1.5      # sequences, drafts, 2m, 2n, vocabulary, rank


class Twin:
    def __init__(self, dt, dev, seed=1):
        g = torch.Generator(device=dev).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
        self.g, self.dt, self.dev = g, dt, dev
        self.R = rnd(M2, K2) * K2 ** -0.5                                # the original layer and head
        self.W = (rnd(V, M2) * 3 * M2 ** -0.5).to(dt)
        self.two = f2.fairy2i_quantize(self.R, 2)
        self.four = self.at_four_bits(self.R, 64)
        self.head = self.at_four_bits(self.W.float(), 32)
        self.x = rnd(S * (D + 1), K2).to(dt)                              # what the layer reads at every position
        self.A, self.B = (rnd(1, R, K2) * K2 ** -0.5).to(dt), (rnd(1, M2, R) * 0.1).to(dt)
        self.alpha = torch.ones(1, device=dev)
        self.seg = (torch.tensor([0, S * (D + 1)], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev))
        self.u, self.r = torch.rand(S, D, generator=g, device=dev), torch.rand(S, generator=g, device=dev)
        self.pick = torch.rand(S, D, 1, generator=g, device=dev, dtype=torch.float64)
        self.weights = torch.full((S * (D + 1),), TEMP * TEMP / (S * (D + 1)), device=dev)
        # the original's outputs
        y = self.x.float() @ self.R.t()
        self.logits = y @ self.W.float().t()
        self.p = torch.softmax(self.logits, 1).view(S, D + 1, V).contiguous()
        best = self.logits.topk(TOP, 1)
        self.top_index, self.top_logit = best.indices, best.values
        self.top_index[::5, TOP // 2:] = -1                              # shorter lists

    def at_four_bits(self, W, group):
        """The nearest of sixteen steps between each group's ends."""
        rows, cols = W.shape
        w = W.view(rows, cols // group, group)
        low, high = w.amin(2), w.amax(2)
        scale = ((high - low) / 15).bfloat16()
        zero = (-low / scale.float()).round().clamp(0, 15)
        codes = ((w / scale.float()[:, :, None]).round() + zero[:, :, None]).clamp(0, 15)
        self.real = ((codes - zero[:, :, None]) * scale.float()[:, :, None]).view(rows, cols)
        return f2.fairy2i_pack_w4(codes.to(torch.uint8).view(rows, cols).contiguous(), scale, group, zero.to(torch.uint8))

    def draft(self):
        """The twin's probabilities at the drafted positions, in products of at most 16 tokens."""
        rows = self.x.view(S, D + 1, K2)[:, :D].reshape(S * D, K2)
        out = []
        for a in range(0, S * D, 16):
            y = f2.fairy2i_gemv(self.two["packed"], self.two["scales"], rows[a:a + 16].bfloat16().contiguous())
            out.append(f2.fairy2i_gemv_w4(self.head, y.to(self.dt)))
        q = torch.softmax(torch.cat(out), 1).view(S, D, V)
        sums = q.double().cumsum(2)
        return q, (sums <= self.pick * sums[:, :, -1:]).sum(2).clamp(max=V - 1)

    def forward(self, A=None, B=None):
        y = f2.fairy2i_gemm(self.two["packed"], self.two["scales"], self.x, y_dtype=self.dt)
        f2.fairy2i_lora(self.x, self.A if A is None else A, self.B if B is None else B, self.alpha, *self.seg, y)
        return y, *f2.fairy2i_distill(y, self.W, self.top_index, self.top_logit, TEMP)

    def step(self):
        y, loss, lse = self.forward()
        dy, dW = f2.fairy2i_distill_backward(y, self.W, self.top_index, self.top_logit, lse, self.weights, TEMP)
        _, dA, dB = f2.fairy2i_lora_backward(dy, self.x, self.A, self.B, self.alpha, *self.seg)
        clipped = [torch.empty_like(dA), torch.empty_like(dB)]
        norm = f2.fairy2i_clip_grads([dA, dB], 0.05, out=clipped)
        return {"y": y, "loss": loss, "lse": lse, "dy": dy, "dW": dW, "dA": dA, "dB": dB, "norm": norm, "cA": clipped[0]}


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_draft_and_verify(dt):
    dev = device()
    t = Twin(dt, dev)
    announce("twin draft", dt)
    q, x = t.draft()
    tokens, accepted = f2.fairy2i_verify_draft(t.p, q.contiguous(), x, t.u, t.r)
    c = {"p": t.p.cpu(), "q": q.cpu(), "draft": x.cpu(), "u": t.u.cpu(), "r": t.r.cpu(), "draft_len": None}
    want, kept = verified(c)
    assert torch.equal(tokens.cpu(), want) and torch.equal(accepted.cpu(), kept)
    assert (tokens.gather(1, accepted.long()[:, None]) >= 0).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_four_bits_are_nearer_than_two(dt):
    """What the layer is kept at four bits for: its output is the product with the rounded weights, and
    nearer the original's than the two-bit layer's."""
    dev = device()
    t = Twin(dt, dev)
    x = t.x[:16].contiguous()
    layer = t.at_four_bits(t.R, 64)
    announce("twin layers", dt)
    y4 = f2.fairy2i_gemv_w4(layer, x)
    want = x.double() @ t.real.double().t()
    size = x.double().abs() @ (t.real.double().abs() + 40 * t.real.double().abs().amax()).t()
    assert ((y4.double() - want).abs() <= (4 * 64 + 6 + 40) * E24 * size).all()
    y2 = f2.fairy2i_gemv(t.two["packed"], t.two["scales"], x.bfloat16())
    true = x.float() @ t.R.t()
    assert (y4 - true).norm() < 0.5 * (y2 - true).norm()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_distillation_step_against_64_bits(dt):
    dev = device()
    t = Twin(dt, dev)
    announce("twin step", dt)
    o = t.step()
    d = lambda v: v.double()
    u = torch.finfo(dt).eps / 2
    l = d(o["y"]) @ d(t.W).t() / TEMP
    lse = torch.logsumexp(l, 1)
    used = t.top_index >= 0
    z = torch.where(used, d(t.top_logit) / TEMP, torch.full((), float("-inf"), dtype=torch.float64, device=dev))
    teacher = torch.softmax(z, 1)
    at = t.top_index.clamp(min=0)
    la = l.gather(1, at)
    loss = torch.where(teacher > 0, teacher * (teacher.clamp(min=1e-300).log() - la + lse[:, None]), torch.zeros_like(la)).sum(1)
    spread = (M2 + 32) * E24 * (d(o["y"]).abs() @ d(t.W).abs().t()).max() / TEMP + 2.0 ** -16
    assert (d(o["lse"]) - lse).abs().max() <= spread and (d(o["loss"]) - loss).abs().max() <= 4 * spread
    p = torch.softmax(l, 1).scatter_add_(1, at, -teacher) * d(t.weights)[:, None] / TEMP
    size = (torch.softmax(l, 1).scatter_add_(1, at, teacher) * d(t.weights)[:, None] / TEMP) @ d(t.W).abs()
    dy = p @ d(t.W)
    assert ((d(o["dy"]) - dy).abs() <= u * dy.abs() + (2 * u + 4 * spread + V * E24) * size).all()
    y, x = d(o["dy"]), d(t.x)
    n = x.shape[0]
    wA, wB = (y @ d(t.B[0])).t() @ x, y.t() @ (x @ d(t.A[0]).t())
    bA = ((M2 + n + 64) * E24 + 2.0 ** -24) * (y.abs() @ d(t.B[0]).abs()).t() @ x.abs()
    bB = ((K2 + n + 64) * E24 + 2.0 ** -24) * y.abs().t() @ (x.abs() @ d(t.A[0]).abs().t())
    assert ((d(o["dA"][0]) - wA).abs() <= bA).all() and ((d(o["dB"][0]) - wB).abs() <= bB).all()


def test_gradients_against_differences():
    """Whole-run differences of the weighted loss along random directions of A and B, fp32 throughout.  A logit
    moves by at most `move` per unit of t; the truncation is under t^2 / 6 times 4 move^3 and the losses'
    rounding under 2^-16 each (weights sum to TEMP^2)."""
    dev = device()
    t = Twin(torch.float32, dev)
    o = t.step()
    y0 = t.forward()[0]
    for name, grad in (("A", o["dA"]), ("B", o["dB"])):
        base = getattr(t, name)
        v = torch.randn(base.shape, generator=torch.Generator().manual_seed(2)).to(dev) * (0.05 if name == "A" else 0.3)
        h, vals = 2.0 ** -6, []
        for sign in (1, -1):
            announce("twin difference", name, sign)
            y, loss, _ = t.forward(**{name: base + sign * h * v})
            vals.append((loss.double() * t.weights.double()).sum().item())
        move = ((y - y0) @ t.W.t()).abs().max().item() / h / TEMP
        want, got = (vals[0] - vals[1]) / (2 * h), (grad.double() * v.double()).sum().item()
        assert abs(got - want) <= TEMP ** 2 * (h * h * 4 * move ** 3 / 6 + 2 * 2.0 ** -16 / (2 * h)), (name, got, want)


def test_run_in_a_graph():
    """Four-bit products, verification and a distillation step captured together: replays with eager runs
    between equal the eager run."""
    dev = device()
    t = Twin(torch.bfloat16, dev)
    q, x = t.draft()
    q, xs = q.contiguous(), t.x[:16].contiguous()
    run = lambda: {**t.step(), "tokens": f2.fairy2i_verify_draft(t.p, q, x, t.u, t.r)[0], "y4": f2.fairy2i_gemv_w4(t.four, xs)}
    want = {k: v.clone() for k, v in run().items()}
    announce("twin graph")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for k in range(4):
        for v in got.values():
            v.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), (k, name)
        again = run()
        assert torch.equal(again["cA"], want["cA"]) and torch.equal(again["tokens"], want["tokens"])
