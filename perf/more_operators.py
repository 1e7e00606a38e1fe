"""Cases that time the operators for a packed model beside the model it came from: products with layers
kept at four bits, distillation from the original's top logits (loss and gradient), and verification of
tokens that the packed model drafted for the original.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, in 64 where a
sampled token depends on it, rounded once) or, where `own` is true, through the library.  Shapes follow
the LLaMA-2 7B projections that the library's workloads use (4096 x 4096, 4096 x 11008, a vocabulary of
32000) and odd sizes around them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------- cases ----

def listed():
    return [
        # one token through an attention projection kept at four bits
        {"name": "w4 decode 1", "op": "w4", "rows": 4096, "cols": 4096, "group": 128, "B": 1, "x": "bf16", "y": "bf16",
         "scales": "bf16", "zeros": True},
        # one token through a vocabulary head kept at four bits
        {"name": "w4 head 1", "op": "w4", "rows": 32000, "cols": 4096, "group": 128, "B": 1, "x": "bf16", "y": "f32",
         "scales": "bf16", "zeros": False},
        # a decode batch through the down projection, fine groups with full-precision scales
        {"name": "w4 down 16", "op": "w4", "rows": 4096, "cols": 11008, "group": 64, "B": 16, "x": "bf16", "y": "bf16",
         "scales": "f32", "zeros": True},
        # full-precision activations of a few requests, odd sizes, a short last group
        {"name": "w4 f32 odd", "op": "w4", "rows": 1003, "cols": 1405, "group": 32, "B": 5, "x": "f32", "y": "f32",
         "scales": "f32", "zeros": True},
        # scoring a short answer against the teacher's list
        {"name": "distill score 24", "op": "distill", "N": 24, "K": 4096, "V": 32000, "top": 8, "x": "bf16", "t": "f32",
         "temperature": 1.0, "ignored": 0.0},
        # validation loss of a 2048-token window
        {"name": "distill score 2048", "op": "distill", "N": 2048, "K": 4096, "V": 32000, "top": 64, "x": "bf16",
         "t": "bf16", "temperature": 2.0, "ignored": 0.1},
        # a training step's loss and gradients over a 2048-token batch with padding
        {"name": "distill step 2048", "op": "distill_grad", "N": 2048, "K": 4096, "V": 32000, "top": 32, "x": "bf16",
         "t": "bf16", "temperature": 2.0, "ignored": 0.1},
        # the same in full precision, odd sizes
        {"name": "distill step f32 odd", "op": "distill_grad", "N": 263, "K": 1088, "V": 5003, "top": 17, "x": "f32",
         "t": "f32", "temperature": 1.5, "ignored": 0.2},
        # one request with four drafted tokens
        {"name": "verify 1", "op": "verify", "S": 1, "D": 4, "V": 32000, "x": "f32", "greedy": False},
        # a serving batch, drafts of up to five tokens, a large vocabulary
        {"name": "verify 64", "op": "verify", "S": 64, "D": 5, "V": 131072, "x": "f32", "greedy": False},
        # many requests with greedy drafts, probabilities in bf16
        {"name": "verify 256 greedy", "op": "verify", "S": 256, "D": 3, "V": 32000, "x": "bf16", "greedy": True},
        # a small vocabulary of odd size, long drafts
        {"name": "verify odd", "op": "verify", "S": 23, "D": 8, "V": 5003, "x": "bf16", "greedy": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["w4", "w4", "distill", "distill_grad", "verify", "verify"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "w4":
        return {"op": op, "rows": _log(rng, 100, 32000), "cols": _log(rng, 64, 11008), "group": rng.choice([32, 64, 128]),
                "B": rng.choice([1, 1, 2, 3, 4, 5, 8, 11, 16]), "x": x, "y": "f32" if x == "f32" else rng.choice(["bf16", "f32"]),
                "scales": rng.choice(["bf16", "f32"]), "zeros": rng.choice([True, False])}
    if op in ("distill", "distill_grad"):
        return {"op": op, "N": _log(rng, 1 if op == "distill" else 16, 2048), "K": 64 * _log(rng, 4, 64),
                "V": _log(rng, 1000, 32000), "top": _log(rng, 1, 128), "x": x, "t": rng.choice(["bf16", "f32"]),
                "temperature": rng.choice([1.0, 1.5, 2.0, 4.0]), "ignored": rng.choice([0.0, 0.1, 0.4])}
    return {"op": op, "S": _log(rng, 1, 256), "D": rng.randint(1, 8), "V": _log(rng, 1000, 131072),
            "x": rng.choice(["bf16", "f32"]), "greedy": rng.choice([False, False, True])}


# --------------------------------------------------------------------------------- inputs ----

def _normal(shape, std, gen, dtype):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * std).to(dtype)


def _uniform(shape, gen):
    return torch.rand(shape, generator=gen, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    dt = _DT[case["x"]]
    if case["op"] == "w4":
        rows, cols, G = case["rows"], case["cols"], case["group"]
        groups = -(-cols // G)
        # codes of a normal weight rounded to a group's sixteen steps
        st["codes"] = torch.randn((rows, cols), generator=gen, device=DEV).mul_(3.0).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        st["scale"] = ((_uniform((rows, groups), gen) + 0.5) * (cols ** -0.5 / 3.0)).to(_DT[case["scales"]])
        st["zero"] = (torch.randint(5, 11, (rows, groups), generator=gen, device=DEV, dtype=torch.uint8)
                      if case["zeros"] else None)
        st["xs"] = _normal((case["B"], cols), 1.0, gen, dt)
        if own:
            import widely_linear_gemv_amd as f2
            st["layer"] = f2.fairy2i_pack_w4(st["codes"], st["scale"], G, st["zero"])
    elif case["op"] in ("distill", "distill_grad"):
        N, K, V, top = case["N"], case["K"], case["V"], min(case["top"], case["V"])
        st["h"] = _normal((N, K), 1.0, gen, dt)
        st["W"] = _normal((V, K), 2.0 * K ** -0.5, gen, dt)
        # the teacher is near the student: the same logits and some of its own
        logits = st["h"].float() @ st["W"].float().t()
        logits = logits + torch.randn(logits.shape, generator=gen, device=DEV)
        best = logits.topk(top, 1)
        st["top_logit"] = best.values.to(_DT[case["t"]])
        index = best.indices
        # some lists are shorter (their last slots unused), padding tokens have none
        short = _uniform((N,), gen) < 0.25
        length = torch.where(short, torch.randint(1, top + 1, (N,), generator=gen, device=DEV),
                             torch.full((N,), top, device=DEV))
        skip = _uniform((N,), gen) < case["ignored"]
        skip[0] = False
        length = torch.where(skip, torch.zeros_like(length), length)
        used = torch.arange(top, device=DEV)[None, :] < length[:, None]
        st["top_index"] = torch.where(used, index, torch.full_like(index, -1))
        st["g"] = (~skip).float() / (~skip).sum()
    else:
        S, D, V = case["S"], case["D"], case["V"]
        z = _normal((S, D + 1, V), 2.5, gen, torch.float32)
        st["p"] = torch.softmax(z, 2).to(dt)
        draft = torch.softmax(z[:, :D] + _normal((S, D, V), 0.7, gen, torch.float32), 2).to(dt)
        if case["greedy"]:
            st["q"], st["draft"] = None, draft.float().argmax(2)
        else:
            sums = draft.double().cumsum(2)
            at = _uniform((S, D, 1), gen).double() * sums[:, :, -1:]
            st["q"], st["draft"] = draft, (sums <= at).sum(2).clamp(max=V - 1)
        length = torch.randint(0, D + 1, (S,), generator=gen, device=DEV)
        full = _uniform((S,), gen) < 0.75
        st["draft_len"] = torch.where(full, torch.full_like(length, D), length).to(torch.int32)
        st["u"] = _uniform((S, D), gen)
        st["r"] = _uniform((S,), gen)
    return st


# ---------------------------------------------------------------------------------- plain ----

def _plain_w4(st):
    G, cols = st["group"], st["cols"]
    zero = 8.0 if st["zero"] is None else st["zero"].float().repeat_interleave(G, 1)[:, :cols]
    W = (st["codes"].float() - zero) * st["scale"].float().repeat_interleave(G, 1)[:, :cols]
    return (st["xs"].float() @ W.t()).to(_DT[st["y"]])


def _plain_distill(st):
    tau, V = st["temperature"], st["W"].shape[0]
    index = st["top_index"]
    used = (index >= 0) & (index < V)
    counts = used.any(1)
    z = torch.where(used, st["top_logit"].float() / tau, torch.full((), -math.inf, device=DEV))
    high = torch.where(counts, z.max(1).values, torch.zeros((), device=DEV))
    e = (z - high[:, None]).exp()
    total = torch.where(counts, e.sum(1), torch.ones((), device=DEV))
    t = e / total[:, None]
    log_t = torch.where(used, z - high[:, None] - total.log()[:, None], torch.zeros((), device=DEV))
    l = (st["h"].float() @ st["W"].float().t()) / tau
    best = l.max(1, keepdim=True).values
    lse = (l - best).exp().sum(1).log() + best[:, 0]
    at = l.gather(1, index.clamp(0, V - 1))
    loss = (t * (log_t - at + lse[:, None])).sum(1)
    return l, lse, torch.where(counts, loss, torch.zeros_like(loss)), t, counts


def _plain_distill_grad(st):
    l, lse, loss, t, counts = _plain_distill(st)
    p = (l - lse[:, None]).exp()
    p.scatter_add_(1, st["top_index"].clamp(0, l.shape[1] - 1), -t)        # unused slots add 0
    p = p * torch.where(counts, st["g"] / st["temperature"], torch.zeros_like(st["g"]))[:, None]
    dh = (p @ st["W"].float()).to(st["h"].dtype)
    dW = (p.t() @ st["h"].float()).to(st["W"].dtype)
    return {"loss": loss, "lse": lse, "dh": dh, "dW": dW}


def _plain_verify(st):
    p, q, x = st["p"], st["q"], st["draft"]
    S, D, V = x.shape[0], x.shape[1], p.shape[2]
    row, pos = torch.arange(S, device=DEV), torch.arange(D, device=DEV)[None, :]
    length = st["draft_len"].long()
    px = p[:, :D].gather(2, x[:, :, None])[:, :, 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, x[:, :, None])[:, :, 0].double()
    good = (st["u"].double() * qx < px) & (pos < length[:, None])
    accepted = good.long().cumprod(1).sum(1)
    refused = accepted < length
    target = p[row, accepted].double()
    at = accepted.clamp(max=D - 1)
    if q is None:
        other = torch.zeros_like(target)
        other[row, x[row, at]] = math.inf
    else:
        other = q[row, at].double()
    rest = (target - other).clamp(min=0)
    keep = refused & (rest.sum(1) > 0)
    w = torch.where(keep[:, None], rest, target)
    sums = w.cumsum(1)
    index = (sums <= st["r"].double()[:, None] * sums[:, -1:]).sum(1)
    last = (torch.arange(V, device=DEV)[None, :] * (w > 0)).max(1).values
    index = torch.minimum(index, last)
    index = torch.where(sums[:, -1] > 0, index, torch.full_like(index, -1))
    place = torch.arange(D + 1, device=DEV)[None, :]
    drafts = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(place < accepted[:, None], drafts, torch.full_like(drafts, -1))
    tokens[row, accepted] = index
    return {"tokens": tokens, "accepted": accepted.to(torch.int32)}


# ------------------------------------------------------------------------------------ run ----

def run(st):
    op = st["op"]
    if own:
        import widely_linear_gemv_amd as f2
        if op == "w4":
            return f2.fairy2i_gemv_w4(st["layer"], st["xs"], y_dtype=_DT[st["y"]])
        if op == "distill":
            loss, lse = f2.fairy2i_distill(st["h"], st["W"], st["top_index"], st["top_logit"], st["temperature"])
            return {"loss": loss, "lse": lse}
        if op == "distill_grad":
            loss, lse = f2.fairy2i_distill(st["h"], st["W"], st["top_index"], st["top_logit"], st["temperature"])
            dh, dW = f2.fairy2i_distill_backward(st["h"], st["W"], st["top_index"], st["top_logit"], lse, st["g"],
                                                 st["temperature"])
            return {"loss": loss, "lse": lse, "dh": dh, "dW": dW}
        tokens, accepted = f2.fairy2i_verify_draft(st["p"], st["q"], st["draft"], st["u"], st["r"],
                                                   draft_len=st["draft_len"])
        return {"tokens": tokens, "accepted": accepted}
    if op == "w4":
        return _plain_w4(st)
    if op == "distill":
        _, lse, loss, _, _ = _plain_distill(st)
        return {"loss": loss, "lse": lse}
    if op == "distill_grad":
        return _plain_distill_grad(st)
    return _plain_verify(st)


# ------------------------------------------------------------------------------- accounting ----

def work(case):
    e = 2 if case["x"] == "bf16" else 4
    op = case["op"]
    if op == "w4":
        rows, cols, B = case["rows"], case["cols"], case["B"]
        groups = -(-cols // case["group"])
        each = (2 if case["scales"] == "bf16" else 4) + (0.5 if case["zeros"] else 0)
        return {"bytes": rows * cols / 2 + rows * groups * each + B * cols * e + B * rows * (2 if case["y"] == "bf16" else 4),
                "flops": 2.0 * B * rows * cols}
    if op in ("distill", "distill_grad"):
        N, K, V, top = case["N"], case["K"], case["V"], min(case["top"], case["V"])
        once = (N * K + V * K) * e + N * top * (8 + (2 if case["t"] == "bf16" else 4)) + N * 8
        if op == "distill":
            return {"bytes": once, "flops": 2.0 * N * K * V}
        return {"bytes": 2 * once, "flops": 6.0 * N * K * V}
    S, D, V = case["S"], case["D"], case["V"]
    rows = 1 if case["greedy"] else 2
    return {"bytes": S * (rows * V * e + D * (12 + rows * e) + (D + 1) * 8 + 12), "flops": 3.0 * S * V}


# ------------------------------------------------------------------------------------ exact ----

def exact(case, seed):
    """The outputs in 64 bits: group by group, through dense teacher distributions, sequence by sequence."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "w4":
        G, cols = case["group"], case["cols"]
        y = torch.zeros((case["B"], case["rows"]), dtype=torch.float64, device=DEV)
        for k, j in enumerate(range(0, cols, G)):
            c = st["codes"][:, j:j + G].double()
            c -= 8.0 if st["zero"] is None else st["zero"][:, k:k + 1].double()
            y += (st["xs"][:, j:j + G].double() @ c.t()) * st["scale"][:, k].double()
        return y
    if op in ("distill", "distill_grad"):
        h, W, tau = st["h"].double(), st["W"].double(), case["temperature"]
        V = W.shape[0]
        ls = torch.log_softmax(h @ W.t() / tau, 1)
        lse = torch.logsumexp(h @ W.t() / tau, 1)
        # teacher: its logits at the listed entries, nothing elsewhere
        dense = torch.full_like(ls, -math.inf)
        n, k = torch.nonzero((st["top_index"] >= 0) & (st["top_index"] < V), as_tuple=True)
        dense[n, st["top_index"][n, k]] = st["top_logit"][n, k].double() / tau
        live = torch.zeros(h.shape[0], dtype=torch.bool, device=DEV)
        live[n] = True
        t = torch.zeros_like(ls)
        t[live] = torch.softmax(dense[live], 1)
        loss = (torch.xlogy(t, t) - t * ls).sum(1)
        if op == "distill":
            return {"loss": loss, "lse": lse}
        p = (ls.exp() - t) * (st["g"].double() * live / tau)[:, None]
        return {"loss": loss, "lse": lse, "dh": p @ W, "dW": p.t() @ h}
    p, q = st["p"].double().cpu(), None if st["q"] is None else st["q"].double().cpu()
    x, u, r = st["draft"].tolist(), st["u"].double().tolist(), st["r"].double().tolist()
    D = case["D"]
    tokens, accepted = [], []
    for s, length in enumerate(st["draft_len"].tolist()):
        a = 0
        while a < length and u[s][a] * (1.0 if q is None else q[s, a, x[s][a]].item()) < p[s, a, x[s][a]].item():
            a += 1
        w = p[s, a]
        if a < length:
            rest = w.clone()
            if q is None:
                rest[x[s][a]] = 0.0
            else:
                rest = (w - q[s, a]).clamp(min=0)
            if rest.sum().item() > 0:
                w = rest
        sums = w.cumsum(0)
        over = torch.nonzero(sums > r[s] * sums[-1])
        some = torch.nonzero(w > 0)
        v = over[0].item() if len(over) else some[-1].item() if len(some) else -1
        tokens.append(x[s][:a] + [v] + [-1] * (D - a))
        accepted.append(a)
    return {"tokens": torch.tensor(tokens, dtype=torch.int64, device=DEV),
            "accepted": torch.tensor(accepted, dtype=torch.int32, device=DEV)}
