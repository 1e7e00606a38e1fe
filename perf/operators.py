"""Cases that time the operators put beside the packed layers: low-rank adapters of many requests
(forward and gradient), the vocabulary cross entropy (loss and gradient) and gradient clipping.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once)
or, where `own` is true, through the library.  Shapes follow the LLaMA-2 7B projections that the
library's workloads use (4096 x 4096, 11008 x 4096, a vocabulary of 32000) and odd sizes around them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
IGNORED = -100


# ---------------------------------------------------------------------------------- cases ----

def listed():
    return [
        # one request decoding one token with its own adapter, beside the o projection
        {"name": "lora decode 1", "op": "lora", "N": 1, "cols": 4096, "rows": 4096, "items": 1, "r": 16, "L": 8,
         "S": 1, "x": "bf16", "y": "f32", "bare": 0.0},
        # a decode batch, every request with its own adapter, beside q, k and v
        {"name": "lora decode 16 qkv", "op": "lora", "N": 16, "cols": 4096, "rows": 4096, "items": 3, "r": 16, "L": 32,
         "S": 16, "x": "bf16", "y": "f32", "bare": 0.1},
        # prompts of several tenants of ragged lengths, beside gate and up
        {"name": "lora prompts gate/up", "op": "lora", "N": 2048, "cols": 4096, "rows": 11008, "items": 2, "r": 32, "L": 8,
         "S": 7, "x": "bf16", "y": "bf16", "bare": 0.1},
        # full-precision activations, odd rank, row count and output count
        {"name": "lora prompts f32 odd", "op": "lora", "N": 517, "cols": 1408, "rows": 1006, "items": 1, "r": 23, "L": 5,
         "S": 9, "x": "f32", "y": "f32", "bare": 0.2},
        # tuning one adapter on a batch of sequences, beside an attention projection
        {"name": "lora grad 2048", "op": "lora_grad", "N": 2048, "cols": 4096, "rows": 4096, "r": 16, "L": 1, "S": 4,
         "x": "bf16", "y": "bf16", "bare": 0.0},
        # tuning several adapters at once in full precision, odd sizes
        {"name": "lora grad f32 odd", "op": "lora_grad", "N": 389, "cols": 1408, "rows": 1006, "r": 12, "L": 6, "S": 11,
         "x": "f32", "y": "f32", "bare": 0.2},
        # scoring the draft of a few tokens
        {"name": "loss score 24", "op": "loss", "N": 24, "K": 4096, "V": 32000, "x": "bf16", "ignored": 0.0},
        # perplexity of a 2048-token window
        {"name": "loss score 2048", "op": "loss", "N": 2048, "K": 4096, "V": 32000, "x": "bf16", "ignored": 0.0},
        # a tuning step's loss and gradients over a 2048-token batch with padding
        {"name": "loss step 2048", "op": "loss_grad", "N": 2048, "K": 4096, "V": 32000, "x": "bf16", "ignored": 0.1},
        # the same in full precision, odd sizes
        {"name": "loss step f32 odd", "op": "loss_grad", "N": 263, "K": 1088, "V": 5003, "x": "f32", "ignored": 0.2},
        # the adapters' gradients of the 32-layer stack (two tensors a projection)
        {"name": "clip stack", "op": "clip", "tensors": 448, "numel": 88064, "x": "f32", "max_norm": 1.0},
        # a handful of small odd tensors, nothing to clip
        {"name": "clip few", "op": "clip", "tensors": 6, "numel": 4099, "x": "bf16", "max_norm": 1e6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["lora", "lora", "lora_grad", "loss", "loss_grad", "clip"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "lora":
        N = _log(rng, 1, 2048)
        return {"op": op, "N": N, "cols": 128 * _log(rng, 2, 86), "rows": 2 * _log(rng, 64, 5504),
                "items": rng.randint(1, 3), "r": _log(rng, 4, 128), "L": _log(rng, 1, 32),
                "S": min(N, _log(rng, 1, 24)), "x": x, "y": "f32" if x == "f32" else rng.choice(["bf16", "f32"]),
                "bare": rng.choice([0.0, 0.1, 0.3])}
    if op == "lora_grad":
        N = _log(rng, 32, 2048)
        return {"op": op, "N": N, "cols": 128 * _log(rng, 2, 86), "rows": 2 * _log(rng, 64, 5504),
                "r": _log(rng, 4, 64), "L": _log(rng, 1, 8), "S": min(N, _log(rng, 1, 12)), "x": x, "y": x,
                "bare": rng.choice([0.0, 0.2])}
    if op in ("loss", "loss_grad"):
        return {"op": op, "N": _log(rng, 1 if op == "loss" else 16, 2048), "K": 64 * _log(rng, 4, 64),
                "V": _log(rng, 1000, 32003), "x": x, "ignored": rng.choice([0.0, 0.1, 0.4])}
    return {"op": op, "tensors": _log(rng, 2, 400), "numel": _log(rng, 1000, 90000), "x": x,
            "max_norm": rng.choice([1.0, 0.1, 1e6])}


# --------------------------------------------------------------------------------- inputs ----

def _segments(case, rnd):
    """Ragged segments: S + 1 nondecreasing row offsets and an adapter (or -1) for each.  With 3 or
    more segments and more rows than segments, one is empty and the last rows belong to none."""
    N, S, L = case["N"], case["S"], case["L"]
    spare = N > S and S >= 3
    end = N - (1 + N // 64) if spare else N
    cuts = sorted(rnd.sample(range(1, end), S - 1)) if S > 1 and end > S else list(range(1, S))
    start = [0] + cuts + [end]
    if spare:
        start[2] = start[1]
    ids = [-1 if rnd.random() < case["bare"] else rnd.randrange(L) for _ in range(S)]
    if all(a < 0 for a in ids):
        ids[0] = 0
        if S == 1 or start[1] == start[0]:
            ids[-1] = 0
    return start, ids


def _normal(shape, std, gen, dtype):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _DT[case["x"]]
    st = dict(case)
    if case["op"] in ("lora", "lora_grad"):
        N, K, M, r, L = case["N"], case["cols"], case["rows"], case["r"], case["L"]
        start, ids = _segments(case, random.Random(seed))
        st["seg_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        st["seg_adapter"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
        st["xs"] = _normal((N, K), 1.0, gen, dt)
        st["alpha"] = torch.rand((L,), generator=gen, device=DEV) + 1.0
        layers = []
        for _ in range(case.get("items", 1)):
            A = _normal((L, r, K), K ** -0.5, gen, dt)
            B = _normal((L, M, r), r ** -0.5, gen, dt)
            layers.append((A, B))
        st["layers"] = layers
        if case["op"] == "lora":
            st["base"] = [_normal((N, M), 1.0, gen, _DT[case["y"]]) for _ in layers]
            st["out"] = [b.clone() for b in st["base"]]
        else:
            st["dy"] = _normal((N, M), 1.0, gen, dt)
            st["dx_base"] = _normal((N, K), 1.0, gen, _DT[case["y"]])
            st["dx"] = st["dx_base"].clone()
    elif case["op"] in ("loss", "loss_grad"):
        N, K, V = case["N"], case["K"], case["V"]
        st["h"] = _normal((N, K), 1.0, gen, dt)
        st["W"] = _normal((V, K), 1.4 * K ** -0.5, gen, dt)
        u = torch.rand((N,), generator=gen, device=DEV)
        t = (float(V) ** u.double()).long().clamp_(1, V) - 1          # frequent tokens have low numbers
        skip = torch.rand((N,), generator=gen, device=DEV) < case["ignored"]
        skip[0] = False
        st["target"] = torch.where(skip, torch.full_like(t, IGNORED), t)
        st["g"] = (~skip).float() / (~skip).sum()
    else:
        cut = random.Random(case["numel"])                            # every third tensor is shorter
        sizes = [case["numel"] - (cut.randrange(case["numel"] // 2) if k % 3 == 2 else 0)
                 for k in range(case["tensors"])]
        pad = [-(-s // 8) * 8 for s in sizes]
        flat = _normal((sum(pad),), 0.02, gen, dt)
        out = torch.zeros_like(flat)
        at = [sum(pad[:k]) for k in range(len(pad))]
        st["grads"] = [flat[a:a + s] for a, s in zip(at, sizes)]
        st["outs"] = [out[a:a + s] for a, s in zip(at, sizes)]
        st["out"] = out
        st["sizes"] = sizes
    return st


# ---------------------------------------------------------------------------------- plain ----

def _row_adapter(st):
    """Adapter of each row, -1 for none."""
    rows = torch.arange(st["N"], device=DEV)
    seg = (rows[:, None] >= st["seg_start"][None, :].long()).sum(1) - 1
    inside = (seg >= 0) & (seg < st["S"])
    ids = st["seg_adapter"].long()[seg.clamp(0, st["S"] - 1)]
    return torch.where(inside & (ids >= 0) & (ids < st["L"]), ids, torch.full_like(ids, -1))


def _spread(v, ids, L):
    """[N][r] -> [N][L r]: each row's r values in its adapter's place, zeros elsewhere."""
    mine = (ids[:, None] == torch.arange(L, device=DEV)[None, :]).to(v.dtype)
    return (mine[:, :, None] * v[:, None, :]).reshape(v.shape[0], -1)


def _pick(v, ids, L):
    """[N][L r] -> [N][r]: the values in each row's adapter's place."""
    v = v.reshape(v.shape[0], L, -1)
    return v[torch.arange(v.shape[0], device=DEV), ids.clamp(min=0)]


def _plain_lora(st, layer, base, out):
    A, B = layer
    L, r = A.shape[0], A.shape[1]
    ids = _row_adapter(st)
    h = _pick(st["xs"].float() @ A.float().reshape(L * r, -1).t(), ids, L)
    h = h * st["alpha"][ids.clamp(min=0)][:, None]
    d = _spread(h, ids, L) @ B.float().permute(0, 2, 1).reshape(L * r, -1)
    out.copy_(torch.where((ids >= 0)[:, None], (base.float() + d).to(base.dtype), out))
    return out


def _plain_lora_grad(st):
    A, B = (t.float() for t in st["layers"][0])
    L, r = A.shape[0], A.shape[1]
    ids = _row_adapter(st)
    x, dy = st["xs"].float(), st["dy"].float()
    al = torch.where(ids >= 0, st["alpha"][ids.clamp(min=0)], torch.zeros((), device=DEV))[:, None]
    h = _spread(_pick(x @ A.reshape(L * r, -1).t(), ids, L) * al, ids, L)
    Bt = B.permute(0, 2, 1).reshape(L * r, -1)
    dh = _spread(_pick(dy @ Bt.t(), ids, L) * al, ids, L)
    dx = (st["dx_base"].float() + dh @ A.reshape(L * r, -1)).to(st["dx_base"].dtype)
    st["dx"].copy_(torch.where((ids >= 0)[:, None], dx, st["dx"]))
    dA = (dh.t() @ x).reshape(A.shape)
    dB = (h.t() @ dy).reshape(L, r, -1).permute(0, 2, 1).contiguous()
    return {"dx": st["dx"], "dA": dA, "dB": dB}


def _plain_loss(st):
    V = st["W"].shape[0]
    logits = st["h"].float() @ st["W"].float().t()
    top = logits.max(1, keepdim=True).values
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    t = st["target"]
    valid = (t >= 0) & (t < V)
    at = logits[torch.arange(t.shape[0], device=DEV), t.clamp(0, V - 1)]
    return logits, lse, torch.where(valid, lse - at, torch.zeros_like(lse)), valid


def _plain_loss_grad(st):
    logits, lse, loss, valid = _plain_loss(st)
    t = st["target"].clamp(0, logits.shape[1] - 1)
    p = (logits - lse[:, None]).exp()
    p[torch.arange(t.shape[0], device=DEV), t] -= 1.0
    p = p * torch.where(valid, st["g"], torch.zeros_like(st["g"]))[:, None]
    dh = (p @ st["W"].float()).to(st["h"].dtype)
    dW = (p.t() @ st["h"].float()).to(st["W"].dtype)
    return {"loss": loss, "lse": lse, "dh": dh, "dW": dW}


def _plain_clip(st):
    flat = torch.cat([g.reshape(-1) for g in st["grads"]])
    norm = flat.double().square().sum().sqrt()
    c = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0).float()
    parts = torch.split((flat.float() * c).to(flat.dtype), st["sizes"])
    [o.copy_(p) for o, p in zip(st["outs"], parts)]
    return {"norm": norm.float().reshape(1), "out": st["out"]}


# ------------------------------------------------------------------------------------ run ----

def run(st):
    op = st["op"]
    if own:
        import widely_linear_gemv_amd as f2
        if op == "lora":
            if len(st["layers"]) == 1:
                A, B = st["layers"][0]
                return [f2.fairy2i_lora(st["xs"], A, B, st["alpha"], st["seg_start"], st["seg_adapter"], st["base"][0],
                                        y=st["out"][0])]
            return f2.fairy2i_lora_grouped(st["xs"], [(A, B, st["alpha"], b, y) for (A, B), b, y in
                                                      zip(st["layers"], st["base"], st["out"])],
                                           st["seg_start"], st["seg_adapter"])
        if op == "lora_grad":
            A, B = st["layers"][0]
            dx, dA, dB = f2.fairy2i_lora_backward(st["dy"], st["xs"], A, B, st["alpha"], st["seg_start"],
                                                  st["seg_adapter"], dx_base=st["dx_base"], dx=st["dx"])
            return {"dx": dx, "dA": dA, "dB": dB}
        if op == "loss":
            loss, lse = f2.fairy2i_vocab_loss(st["h"], st["W"], st["target"])
            return {"loss": loss, "lse": lse}
        if op == "loss_grad":
            loss, lse = f2.fairy2i_vocab_loss(st["h"], st["W"], st["target"])
            dh, dW = f2.fairy2i_vocab_loss_backward(st["h"], st["W"], st["target"], lse, st["g"])
            return {"loss": loss, "lse": lse, "dh": dh, "dW": dW}
        norm = f2.fairy2i_clip_grads(st["grads"], st["max_norm"], out=st["outs"])
        return {"norm": norm, "out": st["out"]}
    if op == "lora":
        return [_plain_lora(st, layer, b, y) for layer, b, y in zip(st["layers"], st["base"], st["out"])]
    if op == "lora_grad":
        return _plain_lora_grad(st)
    if op == "loss":
        _, lse, loss, _ = _plain_loss(st)
        return {"loss": loss, "lse": lse}
    if op == "loss_grad":
        return _plain_loss_grad(st)
    return _plain_clip(st)


# ------------------------------------------------------------------------------- accounting ----

def _used(case):
    """Rows that have an adapter and distinct adapters among them, on average over inputs."""
    rows = case["N"] * (1.0 - case["bare"])
    return rows, min(case["L"], max(1.0, case["S"] * (1.0 - case["bare"])))


def work(case):
    e = 2 if case["x"] == "bf16" else 4
    op = case["op"]
    if op in ("lora", "lora_grad"):
        ye = 2 if case["y"] == "bf16" else 4
        K, M, r = case["cols"], case["rows"], case["r"]
        rows, used = _used(case)
        if op == "lora":
            it = case["items"]
            return {"bytes": rows * K * e + it * (used * r * (K + M) * e + 2 * rows * M * ye),
                    "flops": 2.0 * it * rows * r * (K + M)}
        return {"bytes": rows * (K + M) * e + used * r * (K + M) * e + 2 * rows * K * ye + case["L"] * r * (K + M) * 4,
                "flops": 2.0 * rows * r * (3 * K + 2 * M)}
    if op in ("loss", "loss_grad"):
        N, K, V = case["N"], case["K"], case["V"]
        once = (N * K + V * K) * e + N * 16
        if op == "loss":
            return {"bytes": once, "flops": 2.0 * N * K * V}
        return {"bytes": 2 * once, "flops": 6.0 * N * K * V}
    total = case["tensors"] * case["numel"] * (1 - 0.25 / 3)
    return {"bytes": 2.0 * total * e, "flops": 3.0 * total}


# ------------------------------------------------------------------------------------ exact ----

def exact(case, seed):
    """The outputs in 64 bits, segment by segment and row by row of the definition."""
    st = prepare(case, seed)
    op = case["op"]
    if op in ("lora", "lora_grad"):
        start, ids = st["seg_start"].tolist(), st["seg_adapter"].tolist()
        x = st["xs"].double()
        spans = [(a, start[s], start[s + 1]) for s, a in enumerate(ids) if 0 <= a < case["L"]]
        if op == "lora":
            outs = []
            for (A, B), base, y in zip(st["layers"], st["base"], st["out"]):
                o = y.double()
                for a, i, j in spans:
                    o[i:j] = base[i:j].double() + st["alpha"][a].double() * (
                        x[i:j] @ A[a].double().t() @ B[a].double().t())
                outs.append(o)
            return outs
        A, B = (t.double() for t in st["layers"][0])
        dy, dx = st["dy"].double(), st["dx"].double()
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
        for a, i, j in spans:
            al = st["alpha"][a].double()
            dh = al * (dy[i:j] @ B[a])
            dx[i:j] = st["dx_base"][i:j].double() + dh @ A[a]
            dA[a] += dh.t() @ x[i:j]
            dB[a] += al * (dy[i:j].t() @ (x[i:j] @ A[a].t()))
        return {"dx": dx, "dA": dA, "dB": dB}
    if op in ("loss", "loss_grad"):
        h, W, t = st["h"].double(), st["W"].double(), st["target"]
        keep = torch.nonzero(t >= 0)[:, 0]
        z = h @ W.t()
        lse = torch.logsumexp(z, 1)
        loss = torch.zeros_like(lse)
        loss[keep] = lse[keep] - z[keep, t[keep]]
        if op == "loss":
            return {"loss": loss, "lse": lse}
        p = torch.zeros_like(z)
        p[keep] = torch.softmax(z[keep], 1) * st["g"].double()[keep, None]
        p[keep, t[keep]] -= st["g"].double()[keep]
        return {"loss": loss, "lse": lse, "dh": p @ W, "dW": p.t() @ h}
    parts = [g.double() for g in st["grads"]]
    norm = math.sqrt(sum(float((g * g).sum()) for g in parts))
    c = min(1.0, case["max_norm"] / (norm + 1e-6))
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for g in parts:
        out[at:at + g.numel()] = g * c
        at += -(-g.numel() // 8) * 8
    return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV), "out": out}
