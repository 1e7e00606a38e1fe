"""Verification of drafted tokens (fairy2i_verify_draft) against the definition, sequence by sequence in 64
bits on the host.  Tokens have to be equal: products and differences are exact there and here, and sums of up
to 2^17 fp64 terms are off by under 2^-36 of themselves in any order, so that with r a multiple of 2^-24 a
token could differ only where a border of the summed weights lies that near r (under 2^-17 a row of 2^17
entries whose borders are spread evenly; the inputs are fixed)."""
import math

import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(S, D, V, dt, greedy, seed, spread=2.0, noise=0.7):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(S, D + 1, V, generator=g) * spread
    p = torch.softmax(z, 2).to(dt)
    q = torch.softmax(z[:, :D] + noise * torch.randn(S, D, V, generator=g), 2).to(dt)
    draft = q.float().argmax(2) if greedy else torch.multinomial(q.float().view(S * D, V), 1, generator=g).view(S, D)
    c = {"p": p, "q": None if greedy else q, "draft": draft, "u": torch.rand(S, D, generator=g), "r": torch.rand(S, generator=g),
         "draft_len": torch.randint(0, D + 1, (S,), generator=g, dtype=torch.int32)}
    c["draft_len"][::3] = D
    return c


def reference(c):
    S, D = c["draft"].shape
    V = c["p"].shape[2]
    tokens, accepted = torch.full((S, D + 1), -1), torch.zeros(S, dtype=torch.int32)
    positive = lambda w: torch.where((w > 0) & (w < math.inf), w, torch.zeros_like(w))
    for s in range(S):
        length = D if c["draft_len"] is None else min(max(int(c["draft_len"][s]), 0), D)
        a = 0
        while a < length:
            x = int(c["draft"][s, a])
            if not 0 <= x < V:
                break
            q = 1.0 if c["q"] is None else c["q"][s, a, x].item()
            if not c["u"][s, a].item() * q < c["p"][s, a, x].item():
                break
            a += 1
        w = positive(c["p"][s, a].double())
        if a < length:
            if c["q"] is None:
                rest = c["p"][s, a].double().clone()
                if 0 <= int(c["draft"][s, a]) < V:
                    rest[int(c["draft"][s, a])] = 0.0
            else:
                rest = c["p"][s, a].double() - c["q"][s, a].double()
            rest = positive(rest)
            if rest.sum() > 0:
                w = rest
        sums = w.cumsum(0)
        over = torch.nonzero((sums > c["r"][s].double() * sums[-1]) & (w > 0))[:, 0]
        some = torch.nonzero(w > 0)[:, 0]
        tokens[s, :a] = c["draft"][s, :a]
        tokens[s, a] = over[0] if len(over) else some[-1] if len(some) else -1
        accepted[s] = a
    return tokens, accepted


def call(c, dev, **kw):
    d = {k: None if v is None else v.to(dev) for k, v in c.items()}
    return f2.fairy2i_verify_draft(d["p"], d["q"], d["draft"], d["u"], d["r"], draft_len=d["draft_len"], **kw)


def check(c, dev, label):
    announce("verify", label)
    tokens, accepted = call(c, dev)
    want, kept = reference(c)
    assert torch.equal(accepted.cpu(), kept), label
    assert torch.equal(tokens.cpu(), want), label
    return want, kept


SIZES = [(1, 1, 1), (1, 1, 2), (2, 63, 3), (5, 4, 63), (3, 2, 4095), (4, 3, 4096), (7, 5, 4097), (33, 8, 5003), (2, 3, 32000),
         (1, 4, 131072), (40, 1, 8193), (3, 2, 40960), (2, 4, 40961), (600, 1, 700), (3, 2, 262147)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("greedy", [False, True], ids=["sampled", "greedy"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "S%d-D%d-V%d" % s)
def test_against_the_definition(size, greedy, dt):
    dev = device()
    for seed in range(3):
        c = make(*size, dt, greedy, seed)
        check(c, dev, (size, greedy, dt, seed))
    c["draft_len"] = None
    check(c, dev, (size, greedy, dt, "all drafts"))


def test_every_position_is_reached():
    """Drafts kept to the end, refused at the first and at places between, short drafts."""
    dev = device()
    c = make(400, 6, 50, F32, False, 9)
    _, kept = check(c, dev, "positions")
    full = c["draft_len"]
    assert set(kept.tolist()) == set(range(7))
    assert ((kept == full) & (full < 6)).any() and ((kept < full) & (kept > 0)).any()


def test_same_distributions_keep_every_draft():
    dev = device()
    c = make(50, 5, 300, F32, False, 10, noise=0.0)
    c["draft_len"] = None
    _, kept = check(c, dev, "p = q")
    assert (kept == 5).all()


@pytest.mark.parametrize("V", [5000, 50000])
def test_rows_without_weight(V):
    """p nowhere above q though the draft is refused (p itself is drawn from); a row of zeros; NaN, infinity and
    negative values among the entries; a draft outside the vocabulary; lengths outside 0..D; u and r NaN."""
    dev = device()
    S, D = 12, 2
    c = make(S, D, V, F32, False, 11)
    c["draft_len"][:] = D
    c["u"][:, 0] = 0.9999
    c["p"][0, 0], c["q"][0, 0] = 0.1 / V, 1.0 / V                  # refused, and p < q everywhere
    c["p"][1, 0] = 0.0                                            # nothing at all
    c["p"][2, 0, ::7], c["p"][2, 0, 1::7] = float("nan"), float("inf")
    c["p"][3, 0] = -c["p"][3, 0]
    c["q"][4, 0, ::2] = float("nan")
    c["draft"][5, 0], c["draft"][6, 0], c["draft"][6, 1] = V, 3, -1
    c["p"][6, 0, 3] = 1.0
    c["draft_len"][7], c["draft_len"][8] = -5, 100
    c["u"][9, 0] = float("nan")
    c["r"][10] = float("nan")
    c["p"][11, 0] = 0.0
    c["p"][11, 0, V - 1] = 1e-38
    c["draft"][1, 0], c["draft"][11, 0] = 0, 5
    want, kept = check(c, dev, "rows without weight")
    assert want[1, 0] == -1 and kept[7] == 0 and want[11, 0] == V - 1 and kept[5] == 0 and kept[6] == 1 and kept[9] == 0


def test_unused_drafts_hold_anything():
    """Behind a sequence's last draft nothing of draft, u or q is used."""
    dev = device()
    c = make(30, 6, 700, F32, False, 12)
    want, kept = reference(c)
    behind = torch.arange(6)[None, :] >= c["draft_len"][:, None]
    c["draft"] = torch.where(behind, torch.full_like(c["draft"], 1 << 50), c["draft"])
    c["u"] = torch.where(behind, torch.full_like(c["u"], float("nan")), c["u"])
    c["q"] = torch.where(behind[:, :, None], torch.full_like(c["q"], float("nan")), c["q"])
    announce("verify unused drafts")
    tokens, accepted = call(c, dev)
    assert torch.equal(accepted.cpu(), kept) and torch.equal(tokens.cpu(), want)


@pytest.mark.parametrize("V", [9000, 60000])
@pytest.mark.parametrize("dt", [F32, BF])
def test_borders(dt, V):
    """Weights that are powers of two, r at the borders themselves: a border belongs to the entry behind it, and
    entries without weight are never drawn."""
    dev = device()
    w = torch.zeros(V)
    at = torch.tensor([0, 1, 15, 16, 255, 256, 4095, 4096, 4097, 8191, 8192, V - 1])
    w[at] = 0.0625
    rs = torch.arange(0, 12).float() / 12
    rs = torch.cat([torch.arange(0, 13).float() * 0.0625 / 0.75, torch.tensor([0.0, 1.0, 1.0 - 2.0 ** -24, 0.5])])
    S = len(rs)
    c = {"p": w.repeat(S, 2, 1).to(dt), "q": None, "draft": torch.full((S, 1), 3), "u": torch.zeros(S, 1), "r": rs, "draft_len": None}
    want, _ = check(c, dev, ("borders", dt))
    assert set(want[:, 0].tolist()) <= set(at.tolist())
    # twelve equal weights, twelve whole multiples of their share that fp32 holds exactly
    quarter = torch.zeros(V)
    quarter[at[::3]] = 0.25
    rs = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.25 - 2.0 ** -26])
    c = {"p": quarter.repeat(5, 2, 1).to(dt), "q": None, "draft": torch.full((5, 1), 3), "u": torch.zeros(5, 1), "r": rs,
         "draft_len": None}
    want, _ = check(c, dev, ("quarters", dt))
    assert want[:, 0].tolist() == [0, 16, 4095, 8191, 0]


def test_tokens_are_distributed_as_the_target():
    """The point of it: whatever the draft's distribution, the first token of every sequence is distributed as
    p.  S independent draws of one of V tokens: each count is within 6 standard deviations of S p_v."""
    dev = device()
    S, V = 200000, 7
    g = torch.Generator().manual_seed(13)
    p1, q1 = torch.softmax(torch.randn(V, generator=g), 0), torch.softmax(torch.randn(V, generator=g), 0)
    c = {"p": p1.repeat(S, 2, 1), "q": q1.repeat(S, 1, 1), "draft": torch.multinomial(q1, S, True, generator=g).view(S, 1),
         "u": torch.rand(S, 1, generator=g), "r": torch.rand(S, generator=g), "draft_len": None}
    announce("verify distribution")
    tokens, accepted = call(c, dev)
    count = torch.bincount(tokens[:, 0].cpu(), minlength=V).double()
    want = S * p1.double()
    assert ((count - want).abs() <= 6 * (want * (1 - p1.double())).sqrt()).all()
    rate = torch.minimum(p1, q1).double().sum().item()
    assert abs(accepted.double().mean().item() - rate) <= 6 * math.sqrt(rate * (1 - rate) / S)
    assert (tokens[accepted == 0, 1] == -1).all() and (tokens[accepted == 1, 1] >= 0).all()


def test_any_alignment_and_borders_of_outputs():
    """p and q at odd offsets; the elements before and behind the outputs stay as they were."""
    dev = device()
    for dt, V in ((F32, 4999), (BF, 4999), (F32, 49999), (BF, 49999)):
        c = make(5, 3, V, dt, False, 14)
        want, kept = reference(c)
        flat = lambda t, off: torch.cat([torch.zeros(off, dtype=t.dtype), t.flatten()]).to(dev)[off:].view(t.shape)
        tokens = torch.full((5 * 4 + 4,), 99, device=dev)
        accepted = torch.full((5 + 2,), 99, dtype=torch.int32, device=dev)
        announce("verify alignment", dt)
        f2.fairy2i_verify_draft(flat(c["p"], 1), flat(c["q"], 3), c["draft"].to(dev), c["u"].to(dev), c["r"].to(dev),
                                draft_len=c["draft_len"].to(dev), tokens=tokens[2:22].view(5, 4), accepted=accepted[1:6])
        assert torch.equal(tokens[2:22].view(5, 4).cpu(), want) and torch.equal(accepted[1:6].cpu(), kept)
        assert (tokens[:2] == 99).all() and (tokens[22:] == 99).all() and accepted[0] == 99 and accepted[6] == 99


def test_streams_graphs_and_shared_workspace():
    dev = device()
    cs = [make(9, 4, 50001, F32, False, 20), make(9, 4, 50001, F32, False, 21)]
    want = [reference(c) for c in cs]
    d = {k: v.to(dev) for k, v in cs[0].items()}
    run = lambda **kw: f2.fairy2i_verify_draft(d["p"], d["q"], d["draft"], d["u"], d["r"], draft_len=d["draft_len"], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    announce("verify on a side stream")
    tokens, accepted = run(stream=side)
    side.synchronize()
    assert torch.equal(tokens.cpu(), want[0][0]) and torch.equal(accepted.cpu(), want[0][1])
    ws = torch.empty(f2.fairy2i_verify_draft_workspace_bytes(9, 4, 50001), dtype=torch.uint8, device=dev)
    announce("verify graphs")
    graphs = []
    for _ in range(2):                                  # two graphs over one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            out = run(workspace=ws)
        graphs.append((g, out))
    for k in range(4):
        for name, t in cs[k % 2].items():
            d[name].copy_(t)
        for g, out in graphs:
            ws.fill_(255)
            out[0].fill_(7)
            out[1].fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0].cpu(), want[k % 2][0]) and torch.equal(out[1].cpu(), want[k % 2][1]), k
            assert torch.equal(run()[0].cpu(), want[k % 2][0])


@pytest.mark.parametrize("dt", [F32, BF])
def test_offsets_past_32_bits(dt):
    """The last of 64 (bf16: two sequences of 64) rows of 2^24 entries begins past 2^32 bytes."""
    dev = device()
    S, D, V = (1 if dt == F32 else 2), 63, 1 << 24
    announce("verify offsets", dt)
    p = torch.zeros((S, D + 1, V), dtype=dt, device=dev)
    draft = torch.arange(D, device=dev).repeat(S, 1) + V - D
    p.view(S, D + 1, V)[:, torch.arange(D, device=dev), draft[0]] = 1.0
    p[S - 1, D, V - 2], p[S - 1, D, V - 1] = 0.25, 0.5
    p[0, D, 5] = 1.0 if S > 1 else 0.0
    u = torch.full((S, D), 0.5, device=dev)
    r = torch.full((S,), 0.4, device=dev)
    tokens, accepted = f2.fairy2i_verify_draft(p, None, draft, u, r)
    assert (accepted == D).all() and torch.equal(tokens[:, :D], draft)
    assert tokens[S - 1, D] == V - 1 and (S == 1 or tokens[0, D] == 5)
