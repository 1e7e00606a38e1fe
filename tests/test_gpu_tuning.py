"""The operators beside the packed layers in the run they are made for: a frozen packed layer with
low-rank adapters of two tenants, the vocabulary loss on its output, the gradients of the adapters, and
their global norm and clipping -- against 64 bits on the values that enter each call, against
differences of the whole run's loss, and captured in a graph."""
import math

import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24

N, M2, K2, V, R, L = 48, 256, 384, 700, 8, 3            # tokens, 2n, 2m, vocabulary, rank, adapters


class Step:
    """One tuning step on fixed buffers."""

    def __init__(self, dt, dev, seed=1):
        g = torch.Generator(device=dev).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
        self.layer = f2.fairy2i_quantize(rnd(M2, K2) * 0.05, 2)
        self.x = rnd(N, K2).to(dt)
        self.A, self.B = (rnd(L, R, K2) * K2 ** -0.5).to(dt), (rnd(L, M2, R) * 0.3).to(dt)
        self.alpha = torch.tensor([2.0, 0.5, 1.0], device=dev)
        self.seg_start = torch.tensor([0, 20, 21, 40], dtype=torch.int32, device=dev)    # the last rows: none
        self.seg_adapter = torch.tensor([0, 2, 0], dtype=torch.int32, device=dev)         # adapter 0 twice, 1 never
        self.W = (rnd(V, M2) * M2 ** -0.5).to(dt)
        self.target = torch.randint(0, V, (N,), generator=g, device=dev)
        self.target[::7] = -100
        self.g = (self.target >= 0).float() / (self.target >= 0).sum()
        self.R = f2.fairy2i_dequantize(self.layer["packed"], self.layer["scales"], K2 // 2)
        self.max_norm = 0.05

    def forward(self, A=None, B=None):
        y = f2.fairy2i_gemm(self.layer["packed"], self.layer["scales"], self.x, y_dtype=self.x.dtype)
        f2.fairy2i_lora(self.x, self.A if A is None else A, self.B if B is None else B, self.alpha, self.seg_start,
                        self.seg_adapter, y)
        return y, *f2.fairy2i_vocab_loss(y, self.W, self.target)

    def run(self):
        y, loss, lse = self.forward()
        dy, _ = f2.fairy2i_vocab_loss_backward(y, self.W, self.target, lse, self.g, want_dW=False)
        dx_base = dy.float() @ self.R                          # through the frozen layer's real form
        dx, dA, dB = f2.fairy2i_lora_backward(dy, self.x, self.A, self.B, self.alpha, self.seg_start, self.seg_adapter,
                                              dx_base=dx_base, dx=dx_base.clone())
        clipped = [torch.empty_like(dA), torch.empty_like(dB)]
        norm = f2.fairy2i_clip_grads([dA, dB], self.max_norm, out=clipped)
        return {"y": y, "loss": loss, "lse": lse, "dy": dy, "dx": dx, "dA": dA, "dB": dB, "norm": norm, "cA": clipped[0],
                "cB": clipped[1]}


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_step_against_64_bits(dt):
    dev = device()
    st = Step(dt, dev)
    announce("tuning step", dt)
    o = st.run()
    u = torch.finfo(dt).eps / 2
    d = lambda t: t.double()
    z = d(o["y"]) @ d(st.W).t()
    ok = st.target >= 0
    at, row = st.target.clamp(min=0), torch.arange(N, device=dev)
    lse = torch.logsumexp(z, 1)
    loss = torch.where(ok, lse - z[row, at], torch.zeros_like(lse))
    spread = (M2 + 16) * E24 * (d(o["y"]).abs() @ d(st.W).abs().t()).max() + 2.0 ** -17
    assert (d(o["lse"]) - lse).abs().max() <= spread and (d(o["loss"]) - loss).abs().max() <= 2 * spread
    p = torch.softmax(z, 1)
    p[row, at] -= 1
    p = p * d(st.g)[:, None] * ok[:, None]
    dy = p @ d(st.W)
    assert ((d(o["dy"]) - dy).abs() <= u * dy.abs() + (2 * u + 4 * spread + V * E24) * (p.abs() @ d(st.W).abs())).all()
    # the adapters' gradients, from the dy that entered the call
    wA, wB, bA, bB = (torch.zeros(s, dtype=torch.float64, device=dev) for s in ((L, R, K2), (L, M2, R), (L, R, K2), (L, M2, R)))
    split = 2.0 ** -24
    for a, i, j in ((0, 0, 20), (2, 20, 21), (0, 21, 40)):
        x, y, al = d(st.x[i:j]), d(o["dy"][i:j]), d(st.alpha[a])
        wA[a] += al * (y @ d(st.B[a])).t() @ x
        wB[a] += al * y.t() @ (x @ d(st.A[a]).t())
        bA[a] += ((M2 + N + 64) * E24 + split) * al * (y.abs() @ d(st.B[a]).abs()).t() @ x.abs()
        bB[a] += ((K2 + N + 64) * E24 + split) * al * y.abs().t() @ (x.abs() @ d(st.A[a]).abs().t())
    assert ((d(o["dA"]) - wA).abs() <= bA).all() and ((d(o["dB"]) - wB).abs() <= bB).all()
    assert not o["dA"][1].any() and not o["dB"][1].any()
    norm = math.sqrt(float((d(o["dA"]) ** 2).sum() + (d(o["dB"]) ** 2).sum()))
    assert abs(o["norm"].item() - norm) <= 2.0 ** -23 * norm
    c = min(1.0, st.max_norm / (norm + 1e-6))
    for got, g in ((o["cA"], o["dA"]), (o["cB"], o["dB"])):
        assert ((d(got) - c * d(g)).abs() <= 2.0 ** -22 * d(g).abs()).all()


def test_gradients_against_differences():
    """Whole-run differences of the mean loss along random directions of A and B (the packed layer's own
    output does not depend on them), fp32 throughout.  A logit moves by at most `move` per unit of t;
    the truncation is under t^2 / 6 times 4 move^3 and the losses' rounding under 2^-17 each."""
    dev = device()
    st = Step(torch.float32, dev)
    o = st.run()
    y0 = st.forward()[0]
    for name, grad in (("A", o["dA"]), ("B", o["dB"])):
        base = getattr(st, name)
        v = torch.randn(base.shape, generator=torch.Generator().manual_seed(2)).to(dev) * (0.05 if name == "A" else 0.3)
        t, vals = 2.0 ** -6, []
        for sign in (1, -1):
            announce("tuning difference", name, sign)
            y, loss, _ = st.forward(**{name: base + sign * t * v})
            vals.append((loss.double() * st.g.double()).sum().item())
        move = ((y - y0) @ st.W.t()).abs().max().item() / t
        want, got = (vals[0] - vals[1]) / (2 * t), (grad.double() * v.double()).sum().item()
        assert abs(got - want) <= t * t * 4 * move ** 3 / 6 + 2 * 2.0 ** -17 / (2 * t), (name, got, want)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_step_in_a_graph(dt):
    """The library's calls of a step captured (dx's own product stays outside): replays with eager
    steps between equal the eager step."""
    dev = device()
    st = Step(dt, dev)
    want = {k: v.clone() for k, v in st.run().items()}
    dx_base = want["dy"].float() @ st.R
    dx_out = torch.empty_like(dx_base)       # rows that no call writes: memory of its own, outside the graph's pool
    announce("tuning graph", dt)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        y, loss, lse = st.forward()
        dy, _ = f2.fairy2i_vocab_loss_backward(y, st.W, st.target, lse, st.g, want_dW=False)
        dx, dA, dB = f2.fairy2i_lora_backward(dy, st.x, st.A, st.B, st.alpha, st.seg_start, st.seg_adapter, dx_base=dx_base,
                                              dx=dx_out)
        norm = f2.fairy2i_clip_grads([dA, dB], st.max_norm)      # in place
    for k in range(4):
        for t in (y, loss, lse, dy, dx, dA, dB, norm):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want["y"]) and torch.equal(loss, want["loss"]) and torch.equal(dy, want["dy"]), k
        assert torch.equal(dA, want["cA"]) and torch.equal(dB, want["cB"]) and torch.equal(norm, want["norm"]), k
        assert torch.equal(dx[:40], want["dx"][:40]) and (dx[40:] == 7.0).all(), k
        eager = st.run()
        assert torch.equal(eager["cA"], want["cA"])
