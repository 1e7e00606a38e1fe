"""Low-rank adapters of many requests beside a shared projection (fairy2i_lora, _grouped, _backward)
against the formulas in 64 bits on the CPU.

Tolerances come from the arithmetic.  With u the outputs' unit roundoff (finfo.eps / 2) and all
sums in fp32 (2^-24 per addition of at most K + r + 64 terms, in any order), an output is off by at
most  (K + r + 64) 2^-24 * (sum of the absolute terms) + split * alpha |B| |h| + u |y|,  where split
is what is left of h after its bf16 parts: 2^-16 for two parts (bf16 y), 2^-24 for three (fp32 y), 0
for fp32 inputs.  In the gradient dh is contracted over 2n and split the same way for dx; dA and dB
add at most N more fp32 terms."""
import numpy as np
import pytest
import torch

from gpu_util import announce, device

import widely_linear_gemv_amd as f2

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24


def unit(dt):
    return torch.finfo(dt).eps / 2


def make(N, K, M, r, L, spans, ids, dt, ydt, seed, dev):
    """Inputs on the GPU; spans: the segments' row offsets, ids their adapters."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    c = {"x": rnd(N, K).to(dt), "A": (rnd(L, r, K) * K ** -0.5).to(dt), "B": (rnd(L, M, r) * r ** -0.5).to(dt),
         "alpha": torch.rand(L, generator=g) + 0.5, "base": rnd(N, M).to(ydt), "dy": rnd(N, M).to(dt),
         "dx_base": rnd(N, K).to(ydt), "seg_start": torch.tensor(spans, dtype=torch.int32),
         "seg_adapter": torch.tensor(ids, dtype=torch.int32)}
    return c, {k: v.to(dev) for k, v in c.items()}


def spans_of(c):
    st, ad, L, N = c["seg_start"].tolist(), c["seg_adapter"].tolist(), c["A"].shape[0], c["x"].shape[0]
    return [(a, max(st[s], 0), min(st[s + 1], N)) for s, a in enumerate(ad) if 0 <= a < L and st[s + 1] > st[s]]


def reference(c, y0):
    """(y, bound): rows without an adapter are y0's, bound 0."""
    x, A, B, al = (c[k].double() for k in ("x", "A", "B", "alpha"))
    y, bound = y0.double().clone(), torch.zeros(y0.shape, dtype=torch.float64)
    K, r = x.shape[1], A.shape[1]
    bf = c["x"].dtype == torch.bfloat16
    split = 0.0 if not bf else (2.0 ** -16 if c["base"].dtype == torch.bfloat16 else E24)
    for a, i, j in spans_of(c):
        h = x[i:j] @ A[a].t()
        y[i:j] = c["base"][i:j].double() + al[a] * (h @ B[a].t())
        terms = al[a] * ((x[i:j].abs() @ A[a].abs().t()) @ B[a].abs().t()) + c["base"][i:j].double().abs()
        bound[i:j] = (K + r + 64) * E24 * terms + split * al[a] * (h.abs() @ B[a].abs().t()) \
            + unit(c["base"].dtype) * y[i:j].abs()
    return y, bound


def close(got, want, bound, label):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), label
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, (label, over)


CASES = [  # N, K, M, r, L, spans, ids
    (1, 128, 2, 1, 1, [0, 1], [0]),
    (1, 4096, 4096, 16, 4, [0, 1], [2]),
    (5, 128, 66, 3, 3, [0, 1, 1, 4], [2, 0, 1]),                       # an empty segment, a trailing row
    (16, 256, 258, 8, 20, list(range(17)), [3, -1, 19, 0, 1, 1, 3, 7, 20, 5, 6, 8, 9, 10, 11, 12]),   # one row each
    (33, 384, 1006, 23, 5, [0, 7, 20, 33], [4, 4, 0]),                  # odd rank, the same adapter twice
    (70, 640, 514, 24, 4, [3, 20, 21, 50, 64], [1, 3, -1, 2]),          # rows before the first segment
    (130, 1408, 130, 40, 2, [0, 65, 130], [1, 0]),
    (257, 256, 320, 128, 3, [0, 100, 101, 257], [2, 1, 0]),
    (200, 11008, 192, 64, 2, [0, 200], [1]),
    (300, 384, 514, 16, 3, [0, 100, 101, 290], [2, 0, 1]),             # long segments and small ranks
    (513, 256, 1006, 24, 4, [0, 37, 260, 261, 513], [1, 3, -1, 0]),
    (1100, 128, 15104, 8, 2, [0, 600, 1100], [1, 0]),                   # two row tiles a workgroup
    (700, 1280, 256, 48, 2, [5, 333, 700], [0, 1]),
]


@pytest.mark.parametrize("dt,ydt", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                    (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "N%d-K%d-M%d-r%d" % c[:4])
def test_forward(case, dt, ydt):
    dev = device()
    N, K, M, r, L, spans, ids = case
    announce("lora", case, dt, ydt)
    c, d = make(N, K, M, r, L, spans, ids, dt, ydt, 11, dev)
    y = torch.full((N, M), 7.0, dtype=ydt, device=dev)
    got = f2.fairy2i_lora(d["x"], d["A"], d["B"], d["alpha"], d["seg_start"], d["seg_adapter"], d["base"], y=y)
    assert got is y
    want, bound = reference(c, torch.full((N, M), 7.0, dtype=ydt))
    close(got, want, bound, case)
    # in place: the same values, other rows keep base
    inplace = f2.fairy2i_lora(d["x"], d["A"], d["B"], d["alpha"], d["seg_start"], d["seg_adapter"], d["base"])
    assert inplace is d["base"]
    own = torch.zeros(N, dtype=torch.bool)
    for _, i, j in spans_of(c):
        own[i:j] = True
    assert torch.equal(inplace.cpu()[own], got.cpu()[own]) and torch.equal(inplace.cpu()[~own], c["base"][~own])


@pytest.mark.parametrize("count", [1, 3, 9])
def test_grouped_equals_single(count):
    """Projections of different widths in one call (nine: two launches) against a call each."""
    dev = device()
    N, K, r, L = 19, 512, 16, 3
    spans, ids = [0, 4, 5, 19], [2, 0, 1]
    items, want = [], []
    for k in range(count):
        M = 64 * (k + 1) + 2 * (k % 2)
        _, d = make(N, K, M, r, L, spans, ids, torch.bfloat16, torch.float32, 20 + k, dev)
        if k == 0:
            x, ss, sa = d["x"], d["seg_start"], d["seg_adapter"]
        announce("lora grouped", k, M)
        want.append(f2.fairy2i_lora(x, d["A"], d["B"], d["alpha"], ss, sa, d["base"], y=torch.zeros_like(d["base"])))
        items.append((d["A"], d["B"], d["alpha"], d["base"], torch.zeros_like(d["base"])))
    got = f2.fairy2i_lora_grouped(x, items, ss, sa)
    for k, (a, b) in enumerate(zip(got, want)):
        # the contraction may be cut into other chunks when launches are shared: same fp32 bound
        assert torch.allclose(a, b, rtol=0, atol=(K + r + 64) * E24 * 64), k


def test_many_segments():
    """More segments than a wave compares at once, most of one row."""
    dev = device()
    N, K, M, r, L = 300, 128, 128, 8, 7
    spans = list(range(0, 290)) + [290, 300]
    ids = [(5 * s) % 8 - 1 for s in range(len(spans) - 1)]
    c, d = make(N, K, M, r, L, spans, ids, torch.bfloat16, torch.float32, 31, dev)
    announce("lora many segments")
    y = f2.fairy2i_lora(d["x"], d["A"], d["B"], d["alpha"], d["seg_start"], d["seg_adapter"], d["base"])
    want, bound = reference(c, c["base"])
    close(y, want, bound, "many")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_requests_do_not_mix(dt):
    """NaN and infinity in one request's row, adapter or base stay in its own rows."""
    dev = device()
    N, K, M, r, L = 20, 256, 128, 16, 4
    spans, ids = [0, 1, 6, 7, 20], [0, 1, 2, 3]
    c, d = make(N, K, M, r, L, spans, ids, dt, torch.float32, 41, dev)
    clean = f2.fairy2i_lora(d["x"], d["A"], d["B"], d["alpha"], d["seg_start"], d["seg_adapter"], d["base"],
                            y=torch.zeros_like(d["base"]))
    for what in ("x", "A", "B", "base", "alpha"):
        bad = {k: v.clone() for k, v in d.items()}
        if what in ("x", "base"):
            bad[what][0] = float("nan")
            bad[what][6] = float("inf")
        else:
            bad[what][0] = float("nan")
            bad[what][2] = float("inf")
        announce("lora isolation", what, dt)
        y = f2.fairy2i_lora(bad["x"], bad["A"], bad["B"], bad["alpha"], bad["seg_start"], bad["seg_adapter"], bad["base"],
                            y=torch.zeros_like(bad["base"]))
        assert not torch.isfinite(y[0]).any() and not torch.isfinite(y[6]).all(), what
        rest = [i for i in range(N) if i not in (0, 6)]
        assert torch.equal(y[rest], clean[rest]), what


def backward_reference(c):
    x, A, B, al, dy = (c[k].double() for k in ("x", "A", "B", "alpha", "dy"))
    N, K = x.shape
    M, r = B.shape[1], A.shape[1]
    bf = c["x"].dtype == torch.bfloat16
    split = 0.0 if not bf else (2.0 ** -16 if c["dx_base"].dtype == torch.bfloat16 else E24)
    dx, bx = c["dx_base"].double().clone(), torch.zeros(N, K, dtype=torch.float64)
    dA, bA, dB, bB = (torch.zeros_like(t) for t in (A, A, B, B))
    for a, i, j in spans_of(c):
        dh, h = al[a] * (dy[i:j] @ B[a]), al[a] * (x[i:j] @ A[a].t())
        dh_abs, h_abs = al[a] * (dy[i:j].abs() @ B[a].abs()), al[a] * (x[i:j].abs() @ A[a].abs().t())
        dx[i:j] += dh @ A[a]
        bx[i:j] = (M + r + 64) * E24 * (dh_abs @ A[a].abs() + c["dx_base"][i:j].double().abs()) \
            + split * (dh.abs() @ A[a].abs()) + unit(c["dx_base"].dtype) * dx[i:j].abs()
        dA[a] += dh.t() @ x[i:j]
        bA[a] += (M + N + 64) * E24 * (dh_abs.t() @ x[i:j].abs()) + 2 * split * (dh_abs.t() @ x[i:j].abs())
        dB[a] += dy[i:j].t() @ h
        bB[a] += (K + N + 64) * E24 * (dy[i:j].abs().t() @ h_abs) + 2 * split * (dy[i:j].abs().t() @ h_abs)
    return dx, bx, dA, bA, dB, bB


@pytest.mark.parametrize("dt,ydt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                    (torch.float32, torch.float32)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "N%d-K%d-M%d-r%d" % c[:4])
def test_backward(case, dt, ydt):
    dev = device()
    N, K, M, r, L, spans, ids = case
    announce("lora backward", case, dt, ydt)
    c, d = make(N, K, M, r, L, spans, ids, dt, ydt, 51, dev)
    args = [d[k] for k in ("dy", "x", "A", "B", "alpha", "seg_start", "seg_adapter")]
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=torch.float32, device=dev)
    dx, dA, dB = f2.fairy2i_lora_backward(*args, dx_base=d["dx_base"], dx=d["dx_base"].clone(), dA=nan(d["A"]), dB=nan(d["B"]))
    wx, bx, wA, bA, wB, bB = backward_reference(c)
    close(dx, wx, bx, "dx")
    close(dA, wA, bA, "dA")
    close(dB, wB, bB, "dB")
    for a in set(range(L)) - {s[0] for s in spans_of(c)}:          # no row uses it: exactly zero
        assert not dA[a].any() and not dB[a].any()
    none, dA2, dB2 = f2.fairy2i_lora_backward(*args)                # no dx; the same sums again, bit for bit
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    again = f2.fairy2i_lora_backward(*args, dx_base=d["dx_base"])[0]
    assert again is d["dx_base"] and torch.equal(again, dx)


@pytest.mark.parametrize("N", [2, 100])
@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
def test_h_past_the_largest_bf16(N, ydt):
    """h = (2^128 - 2^120) + 1.5 2^119 fits fp32 but not bf16: y = 2^-100 h is finite.  Off by at most 2^-16 h
    (its parts), the rounding of the fp32 sum and of y, which are under 2^-23 and u of y."""
    dev = device()
    K, M = 128, 64
    x = torch.zeros((N, K), dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = 2.0 ** 127 * (2 - 2.0 ** -7), 1.5 * 2.0 ** 119
    A, B = torch.zeros((1, 1, K), dtype=torch.bfloat16), torch.full((1, M, 1), 2.0 ** -100, dtype=torch.bfloat16)
    A[0, 0, :2] = 1.0
    announce("lora h past bf16", N, ydt)
    y = f2.fairy2i_lora(x.to(dev), A.to(dev), B.to(dev), torch.ones(1, device=dev),
                        torch.tensor([0, N], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev),
                        base=torch.zeros((N, M), dtype=ydt, device=dev))
    want = torch.full((N, M), (2.0 ** 127 * (2 - 2.0 ** -7) + 1.5 * 2.0 ** 119) * 2.0 ** -100, dtype=torch.float64)
    close(y, want, want * (2.0 ** -16 + 2.0 ** -23 + unit(ydt)), "y")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [40, 300])
def test_gradients_of_requests_do_not_mix(dt, N):
    """NaN and infinity in the rows of one adapter, and in rows without any, reach no other gradient."""
    dev = device()
    K, M, r, L = 256, 130, 16, 3
    spans, ids = [0, N // 3, N // 2, N - 5], [0, 1, 2]              # the last five rows: none
    c, d = make(N, K, M, r, L, spans, ids, dt, torch.float32, 91, dev)
    args = lambda e: [e[k] for k in ("dy", "x", "A", "B", "alpha", "seg_start", "seg_adapter")]
    announce("lora gradient isolation", dt, N)
    dx, dA, dB = f2.fairy2i_lora_backward(*args(d), dx_base=d["dx_base"], dx=d["dx_base"].clone())
    bad = {k: v.clone() for k, v in d.items()}
    for name in ("x", "dy"):
        bad[name][N // 3] = float("nan")                             # adapter 1's first row
        bad[name][N // 2 - 1] = float("inf")                         # and its last
        bad[name][N - 3] = float("nan")
    dx2, dA2, dB2 = f2.fairy2i_lora_backward(*args(bad), dx_base=d["dx_base"], dx=d["dx_base"].clone())
    for a in (0, 2):
        assert torch.equal(dA2[a], dA[a]) and torch.equal(dB2[a], dB[a]), a
    assert not torch.isfinite(dA2[1]).any() and not torch.isfinite(dB2[1]).any()
    rows = [i for i in range(N) if i not in (N // 3, N // 2 - 1)]
    assert torch.equal(dx2[rows], dx[rows])


def test_backward_against_differences():
    """d/dt of sum(y * dy) along a random direction of (x, A, B), by central differences of the
    forward call.  Truncation is exactly zero for the cubic's odd part up to t^2 |dA dB dx| terms:
    with directions of size 1 and t = 2^-6 the forward's fp32 rounding dominates."""
    dev = device()
    N, K, M, r, L = 24, 128, 64, 4, 2
    c, d = make(N, K, M, r, L, [0, 9, 24], [1, 0], torch.float32, torch.float32, 61, dev)
    zero = torch.zeros(N, M, device=dev)
    dx, dA, dB = f2.fairy2i_lora_backward(d["dy"], d["x"], d["A"], d["B"], d["alpha"], d["seg_start"], d["seg_adapter"],
                                          dx_base=torch.zeros(N, K, device=dev))
    for name, grad in (("x", dx), ("A", dA), ("B", dB)):
        v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(7)).to(dev)
        t = 2.0 ** -6
        vals = []
        for sign in (1, -1):
            e = dict(d)
            e[name] = d[name] + sign * t * v
            announce("difference", name, sign)
            y = f2.fairy2i_lora(e["x"], e["A"], e["B"], e["alpha"], e["seg_start"], e["seg_adapter"], zero,
                                y=torch.zeros_like(zero))
            vals.append((y.double() * d["dy"].double()).sum().item())
        want = (vals[0] - vals[1]) / (2 * t)
        got = (grad.double() * v.double()).sum().item()
        # the map is linear in each of x, A and B, so the difference is exact but for the forward's
        # rounding: (K + r + 64) 2^-24 of the absolute terms, of both calls, over 2 t
        h = d["x"].abs().double() @ d["A"].abs().double().sum(0).t()
        terms = 1.5 * (h @ d["B"].abs().double().sum(0).t() * d["dy"].abs().double()).sum().item()
        assert abs(got - want) <= 2 * (K + r + 64) * E24 * terms / (2 * t), name


def test_other_stream_and_graph():
    """On a stream of its own, and captured with its output's producer: every replay, with eager work
    between, equals the eager result."""
    dev = device()
    N, K, M, r, L = 16, 512, 512, 16, 8
    c, d = make(N, K, M, r, L, list(range(17)), [s % 9 - 1 for s in range(16)], torch.bfloat16, torch.float32, 71, dev)
    args = [d[k] for k in ("x", "A", "B", "alpha", "seg_start", "seg_adapter")]
    want = f2.fairy2i_lora(*args, d["base"], y=d["base"].clone()).clone()
    gargs = [d["dy"], *args]
    grads = [t.clone() for t in f2.fairy2i_lora_backward(*gargs, dx_base=d["dx_base"], dx=d["dx_base"].clone())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    announce("lora on a side stream")
    y = f2.fairy2i_lora(*args, d["base"], y=d["base"].clone(), stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    announce("lora graphs")
    outs, graphs = [], []
    for _ in range(2):                                   # two graphs alive at once
        buf, dxo = d["base"].clone(), d["dx_base"].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            buf.copy_(d["base"])
            f2.fairy2i_lora(*args, buf)
            gr = f2.fairy2i_lora_backward(*gargs, dx_base=d["dx_base"], dx=dxo)
        graphs.append(g)
        outs.append((buf, gr))
    for k in range(4):
        for g, (buf, gr) in zip(graphs, outs):
            buf.zero_()
            gr[1].fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(buf, want), k
            for a, b in zip(gr, grads):
                assert torch.equal(a, b), k
        assert torch.equal(f2.fairy2i_lora(*args, d["base"], y=d["base"].clone()), want)


def test_largest_pool_offsets():
    """An adapter past 2^31 elements of its pool, and one past 2^32 bytes."""
    dev = device()
    N, K, M, r, L = 3, 11008, 64, 128, 1600                          # 2.25e9 elements of A
    announce("lora large pool")
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn((N, K), generator=g, device=dev).bfloat16()
    A = torch.zeros((L, r, K), dtype=torch.bfloat16, device=dev)
    B = torch.zeros((L, M, r), dtype=torch.bfloat16, device=dev)
    for a in (0, 800, L - 1):
        A[a] = torch.randn((r, K), generator=g, device=dev) * K ** -0.5
        B[a] = torch.randn((M, r), generator=g, device=dev) * r ** -0.5
    al = torch.ones(L, device=dev)
    ss, sa = torch.arange(4, dtype=torch.int32, device=dev), torch.tensor([L - 1, 0, 800], dtype=torch.int32, device=dev)
    y = f2.fairy2i_lora(x, A, B, al, ss, sa, torch.zeros((N, M), device=dev))
    for i, a in enumerate((L - 1, 0, 800)):
        xd, Ad, Bd = x[i].double().cpu(), A[a].double().cpu(), B[a].double().cpu()
        want = Bd @ (Ad @ xd)
        bound = (K + r + 64) * E24 * (Bd.abs() @ (Ad.abs() @ xd.abs())) + 2 * E24 * want.abs()
        close(y[i], want, bound, a)


def test_decode_step_with_adapters():
    """stack.DecodeStep with adapters on some projections: each output is the plain step's plus its
    rows' adapters, eager and captured."""
    from widely_linear_gemv_amd import stack
    dev = device()
    B, r, L = 4, 8, 3
    layers, xs, adapters = [], [], []
    g = torch.Generator(device=dev).manual_seed(81)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
    pools = {}
    layer, pool = [], []
    for name, rows, cols, _ in stack.PROJECTIONS:
        q = f2.fairy2i_quantize(rnd(rows, cols) * 0.02, 2)
        layer.append((q["packed"], q["scales"]))
        pool.append(None if name in ("k", "o") else
                    ((rnd(L, r, cols) * cols ** -0.5).bfloat16(), rnd(L, rows, r).bfloat16(), torch.rand(L, device=dev)))
    widths = {grp: cols for _, _, cols, grp in stack.PROJECTIONS}
    layers, adapters = [layer], [pool]
    xs = [[rnd(B, widths[grp]).bfloat16() for grp in range(stack.GROUPS)]]
    segments = (torch.tensor([0, 1, 3, 4], dtype=torch.int32, device=dev), torch.tensor([2, -1, 0], dtype=torch.int32, device=dev))
    announce("decode step with adapters")
    plain = [[y.clone() for y in ys] for ys in stack.DecodeStep(layers, xs).run()]
    step = stack.DecodeStep(layers, xs, adapters=adapters, segments=segments)
    got = [[y.clone() for y in ys] for ys in step.run()]
    graph = step.capture()
    for p, (name, rows, cols, grp) in enumerate(stack.PROJECTIONS):
        want = plain[0][p].clone()
        if pool[p] is not None:
            f2.fairy2i_lora(xs[0][grp], *pool[p], *segments, want)
        scale = (cols + r + 64) * E24 * 40 * want.abs().max().item()
        assert torch.allclose(got[0][p], want, rtol=0, atol=scale), name
        assert torch.equal(got[0][p][1:3], plain[0][p][1:3]), name
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(step.ys[0], got[0]):
            assert torch.equal(a, b)
