"""Operators around the learner's products, as cases that can be timed and checked.

* ``rows``   rows sorted by expert and back in BF16 or FP32: the stable sort with
  the copies (``permute``), its gradient (``permute_grad``), the weighted sum of
  a token's expert outputs (``combine``) and its gradient with respect to rows
  and weights (``combine_grad``);
* ``norm``   the global gradient norm over many tensors with the clipping factor
  that AdamW takes (``factor``), and gradients clipped by it (``clip``);
* ``verify`` drafted tokens verified against the target's probabilities from
  given random numbers: how many stand, the token that follows, log probabilities.

With ``own`` false, ``run`` computes them with elementary torch operations in
FP32, rounded once at the end; with ``own`` true it calls this package.
"""
import math

import torch

own = False


def _minite():
    from nvfp4_w4a4_moe_permute_gb300 import minite
    return minite


# --------------------------------------------------------------------------- the cases


def listed():
    return [
        # one token of a sampled sequence on its way to 8 of 128 experts: latency is all
        dict(name="permute_one_token", op="rows", kind="permute", tokens=1, topk=8, experts=128,
             hidden=2048, dtype="bfloat16", skew=0.0, dropped=0.0),
        # one 4096-token micro-batch into expert order
        dict(name="permute_micro_batch", op="rows", kind="permute", tokens=4096, topk=8, experts=128,
             hidden=2048, dtype="bfloat16", skew=0.0, dropped=0.0),
        # the gradient of that copy: every token sums its experts' activation gradients
        dict(name="permute_grad_micro_batch", op="rows", kind="permute_grad", tokens=4096, topk=8,
             experts=128, hidden=2048, dtype="bfloat16", skew=0.0, dropped=0.0),
        # one rank's part of a batch in FP32: most slots belong to experts elsewhere, odd sizes
        dict(name="permute_odd_fp32", op="rows", kind="permute", tokens=3001, topk=4, experts=9,
             hidden=1001, dtype="float32", skew=0.5, dropped=0.6),
        # a long packed batch, outputs weighted on the way back to token order
        dict(name="combine_long", op="rows", kind="combine", tokens=32768, topk=8, experts=128,
             hidden=2048, dtype="bfloat16", skew=1.2, dropped=0.0),
        # its gradient for one micro-batch, with respect to the rows and to the router's weights
        dict(name="combine_grad_micro_batch", op="rows", kind="combine_grad", tokens=4096, topk=8,
             experts=128, hidden=2048, dtype="bfloat16", skew=0.0, dropped=0.0),
        # norms and a router alone (what is trained when the experts are frozen): latency counts
        dict(name="norm_router", op="norm", kind="factor", tensors=6, elements=300001,
             dtype="bfloat16", order=2.0),
        # the FP32 gradient sums of a 128-expert layer, the factor handed to the optimizer
        dict(name="norm_layer", op="norm", kind="factor", tensors=9, elements=604_241_920,
             dtype="float32", order=2.0),
        # FP32 sums of a whole small model, clipped into the BF16 buffers that are sent or kept
        dict(name="clip_model", op="norm", kind="clip", tensors=291, elements=400_000_003,
             dtype="float32", order=2.0),
        # four drafts of one sequence, logits in FP32 as a sampler has them
        dict(name="verify_one_sequence", op="verify", sequences=1, drafts=4, vocab=131072,
             dtype="float32", by_model=True, ragged=False),
        # a batch of sequences with up to four drafts each, an odd vocabulary
        dict(name="verify_batch", op="verify", sequences=64, drafts=4, vocab=100003,
             dtype="bfloat16", by_model=True, ragged=True),
        # drafts that were looked up (no draft distribution), a large batch
        dict(name="verify_lookup", op="verify", sequences=256, drafts=7, vocab=32768,
             dtype="bfloat16", by_model=False, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "rows", "norm", "verify"])
    if op == "rows":
        e = _log(rng, 1, 256)
        return dict(op=op, kind=rng.choice(["permute", "permute_grad", "combine", "combine_grad"]),
                    tokens=_log(rng, 1, 12000), topk=min(e, rng.choice([1, 2, 4, 6, 8])), experts=e,
                    hidden=rng.choice([1, 8, 8]) * _log(rng, 5, 256),
                    dtype=rng.choice(["bfloat16", "float32"]), skew=rng.choice([0.0, 0.0, 1.2]),
                    dropped=rng.choice([0.0, 0.0, 0.5]))
    if op == "norm":
        tensors = _log(rng, 1, 400)
        return dict(op=op, kind=rng.choice(["factor", "clip"]), tensors=tensors,
                    elements=_log(rng, 1000, 250_000_000) + tensors,
                    dtype=rng.choice(["bfloat16", "float32", "mixed"]),
                    order=rng.choice([2.0, 2.0, math.inf]))
    return dict(op=op, sequences=_log(rng, 1, 128), drafts=rng.choice([0, 1, 2, 3, 4, 5, 7]),
                vocab=_log(rng, 500, 131072), dtype=rng.choice(["bfloat16", "float32"]),
                by_model=rng.random() < 0.6, ragged=rng.random() < 0.5)


# --------------------------------------------------------------------------- their inputs


def _sizes(case):
    """Sizes of the tensors: a few large ones, a long tail of small ones, odd ones among them."""
    n, total = case["tensors"], case["elements"]
    w = [1.0 / (i + 1) ** 1.5 for i in range(n)]
    s = sum(w)
    sizes = [max(1, int((total - n) * x / s)) for x in w]
    sizes[0] += total - sum(sizes)
    return sizes


def _types(case):
    """The gradients' types."""
    if case["dtype"] == "mixed":
        return [torch.bfloat16 if i % 3 else torch.float32 for i in range(case["tensors"])]
    return [getattr(torch, case["dtype"])] * case["tensors"]


def _starts(sizes):
    """Each tensor's place in a flat buffer: multiples of 256 elements, and the buffer's size."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // 256) * 256
    return starts, at


def _route(case, seed):
    """topk experts of each token without repetition, -1 where a slot is not used."""
    g = torch.Generator().manual_seed(seed)
    t, k, e = case["tokens"], case["topk"], case["experts"]
    p = torch.arange(1, e + 1, dtype=torch.float64) ** -case["skew"]
    p = p[torch.randperm(e, generator=g)]
    ids = torch.multinomial(p.expand(t, e), k, generator=g).to(torch.int32)
    ids[torch.rand(t, k, generator=g) < case["dropped"]] = -1
    w = torch.softmax(torch.randn(t, k, generator=g), 1)
    return ids, w


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    state = dict(case=case)
    if case["op"] == "rows":
        t, k, h, dtype = case["tokens"], case["topk"], case["hidden"], getattr(torch, case["dtype"])
        ids, w = _route(case, seed)
        state |= dict(ids=ids.to(dev), weights=w.to(dev))
        kind = case["kind"]
        if kind in ("permute", "combine_grad"):
            x = randn(t, h, dtype=dtype)
            x[:, :: 100] *= 20  # outlier channels
            state["x"] = x
        if kind != "permute":
            state["dest"] = _sort(state["ids"], case["experts"])[2].to(torch.int32)
            state["rows"] = randn(t * k, h, dtype=dtype)
        # buffers that a training program keeps from step to step
        if kind == "permute":
            state["kept"] = dict(rows=torch.zeros(t * k, h, device=dev, dtype=dtype),
                                 offsets=torch.zeros(case["experts"] + 1, device=dev, dtype=torch.int32),
                                 perm_src=torch.zeros(t * k, device=dev, dtype=torch.int32),
                                 dest_row=torch.zeros(t, k, device=dev, dtype=torch.int32))
        elif kind == "combine_grad":
            state["drows"] = torch.zeros(t * k, h, device=dev, dtype=dtype)
        return state
    if case["op"] == "norm":
        sizes = _sizes(case)
        state["grads"] = [randn(n, std=3e-4, dtype=d) for n, d in zip(sizes, _types(case))]
        state["max_norm"] = 0.1 if case["order"] == 2.0 else 1e-4
        if case["kind"] == "clip":
            starts, total = _starts(sizes)   # the flat buffer that is sent, or that the optimizer reads
            state["flat"] = torch.zeros(total, device=dev, dtype=torch.bfloat16)
            state["out"] = [state["flat"][a: a + n] for a, n in zip(starts, sizes)]
        return state
    b, s, v, dtype = case["sequences"], case["drafts"], case["vocab"], getattr(torch, case["dtype"])
    base = randn(b, s + 1, v, std=2.5)
    target = base.to(dtype)
    q = (base[:, :s] + randn(b, s, v, std=0.5)).to(dtype)   # what the draft model thinks
    del base
    pick = torch.softmax(q.float().view(b * s, v) / 0.8, 1) if s else None
    tokens = torch.multinomial(pick, 1, generator=g).view(b, s).to(torch.int32) if s else \
        torch.zeros(b, 0, device=dev, dtype=torch.int32)
    if case["ragged"] and s:   # some sequences got fewer drafts
        some = torch.randint(0, s + 1, (b, 1), generator=g, device=dev)
        some = torch.where(torch.rand(b, 1, generator=g, device=dev) < 0.5, s, some)
        tokens[torch.arange(s, device=dev)[None] >= some] = -1
    noise = torch.empty(b, v, device=dev).exponential_(generator=g).clamp_(min=1e-30)
    state |= dict(target=target, draft=q if case["by_model"] and s else None, tokens=tokens,
                  uniforms=torch.rand(b, s, generator=g, device=dev), noise=noise, temperature=0.8)
    return state


# --------------------------------------------------------------------------- the plain forms


def _sort(ids, experts):
    """(order of the pairs, offsets, row of every pair or -1): by expert, token, slot."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(experts, device=ids.device)).sum(0) if experts <= 16 else \
        torch.zeros(experts + 1, device=ids.device, dtype=torch.long).scatter_add_(
            0, key, torch.ones_like(key))[:experts]
    offsets = torch.zeros(experts + 1, device=ids.device, dtype=torch.long)
    offsets[1:] = counts.cumsum(0)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    dest = torch.where(key < experts, row, -1).view(ids.shape)
    return order, offsets, dest


def _rows(state):
    case = state["case"]
    k, dtype = case["topk"], getattr(torch, case["dtype"])
    if case["kind"] == "permute":
        order, offsets, dest = _sort(state["ids"], case["experts"])
        live = torch.arange(order.numel(), device=order.device) < offsets[-1]
        src = torch.where(live, order // k, -1)
        rows = torch.where(live[:, None], state["x"][order // k], torch.zeros((), device=order.device, dtype=dtype))
        return dict(rows=rows, offsets=offsets.to(torch.int32), perm_src=src.to(torch.int32),
                    dest_row=dest.to(torch.int32))
    dest = state["dest"].long()
    live = dest >= 0
    at = dest.clamp(min=0)
    if case["kind"] == "combine_grad":
        dy, w = state["x"].float(), state["weights"]
        dw = torch.empty_like(w)
        drows = state["drows"]
        for j in range(k):   # slot by slot, so that FP32 copies of all rows are never alive at once
            r = state["rows"][at[:, j]].float()
            dw[:, j] = torch.where(live[:, j], (r * dy).sum(1), 0.0)
            to = at[:, j]
            new = (dy * w[:, j, None]).to(dtype)
            if case["dropped"]:
                new, to = new[live[:, j]], to[live[:, j]]
            drows[to] = new
        return dict(drows=drows, dweights=dw)
    y = torch.zeros(case["tokens"], case["hidden"], device=dest.device)
    for j in range(k):
        r = torch.where(live[:, j, None], state["rows"][at[:, j]].float(), 0.0)
        y += r if case["kind"] == "permute_grad" else r * state["weights"][:, j, None]
    return y.to(dtype)


def _norm(state):
    case, grads = state["case"], state["grads"]
    if case["order"] == 2.0:
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()
    else:
        norm = torch.stack([g.float().abs().max() for g in grads]).max().double()
    scale = (state["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    res = dict(norm=norm.float().view(1), scale=scale.view(1))
    if case["kind"] == "clip":
        for o, g in zip(state["out"], grads):
            o.copy_(g.float() * scale)
        res["out"] = state["flat"]
    return res


def _verify(state):
    x, q, tokens, t = state["target"], state["draft"], state["tokens"].long(), state["temperature"]
    b, s = tokens.shape
    v = x.shape[-1]
    dev = x.device
    y = x.float() / t
    top = y.amax(2, keepdim=True)
    logp = y - top - (y - top).exp().sum(2, keepdim=True).log()
    lq = None
    if q is not None:
        z = q.float() / t
        top = z.amax(2, keepdim=True)
        lq = z - top - (z - top).exp().sum(2, keepdim=True).log()
    at = tokens.clamp(min=0)[..., None]
    lp_x = logp[:, :s].gather(2, at)[..., 0]
    p_x = lp_x.double().exp()
    q_x = 1.0 if lq is None else lq.gather(2, at)[..., 0].double().exp()
    drafted = (tokens >= 0).long().cumprod(1)
    stands = (drafted * (state["uniforms"].double() * q_x < p_x).long()).cumprod(1)
    n, given = stands.sum(1), drafted.sum(1)
    rows = torch.arange(b, device=dev)
    last = logp[rows, n]
    p = last.double().exp()
    falls = n < given   # the next draft was refused: what is left of p without q
    if s:
        i = n.clamp(max=s - 1)
        if lq is None:
            q_row = torch.zeros(b, v, device=dev, dtype=torch.float64)
            q_row.scatter_(1, at[rows, i], 1.0)
        else:
            q_row = lq[rows, i].double().exp()
        r = (p - q_row).clamp(min=0)
        r = torch.where((falls & (r.amax(1) > 0))[:, None], r, p)
    else:
        r = p
    race = r / state["noise"].double()
    new = (race == race.amax(1, keepdim=True)).to(torch.int8).argmax(1)   # ties: the lowest index
    out = torch.full((b, s + 1), -1, device=dev, dtype=torch.int32)
    lps = torch.zeros(b, s + 1, device=dev)
    out[:, :s] = torch.where(stands > 0, tokens, -1)
    lps[:, :s] = torch.where(stands > 0, lp_x, 0.0)
    out[rows, n] = new.to(torch.int32)
    lps[rows, n] = last.gather(1, new[:, None])[:, 0]
    return dict(tokens=out, accepted=n.to(torch.int32), logprobs=lps)


def run(state):
    case = state["case"]
    if not own:
        return dict(rows=_rows, norm=_norm, verify=_verify)[case["op"]](state)
    M = _minite()
    if case["op"] == "rows":
        if case["kind"] == "permute":
            return M.permute_rows(state["x"], state["ids"], case["experts"], into=state["kept"])
        if case["kind"] == "permute_grad":
            return M.permute_rows_backward(state["rows"], state["dest"])
        if case["kind"] == "combine":
            return M.combine_rows(state["rows"], state["dest"], state["weights"])
        drows, dweights = M.combine_rows_backward(state["x"], state["rows"], state["dest"],
                                                  state["weights"], out=state["drows"])
        return dict(drows=drows, dweights=dweights)
    if case["op"] == "norm":
        if case["kind"] == "factor":
            return M.grad_norm(state["grads"], max_norm=state["max_norm"], order=case["order"])
        r = M.clip_grads(state["grads"], state["max_norm"], order=case["order"], out=state["out"])
        return dict(r, out=state["flat"])
    return M.verify_drafts(state["target"], state["tokens"], state["uniforms"], state["noise"],
                           draft_logits=state["draft"], temperature=state["temperature"])


# --------------------------------------------------------------------------- what a pass needs


def work(case):
    if case["op"] == "rows":
        size = 4 if case["dtype"] == "float32" else 2
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        live = t * k * (1 - case["dropped"])
        row, tok, pairs = live * h * size, t * h * size, 4 * t * k
        if case["kind"] == "permute":
            return dict(bytes=tok + row + 3 * pairs, flops=0)
        if case["kind"] == "permute_grad":
            return dict(bytes=tok + row + pairs, flops=live * h)
        if case["kind"] == "combine":
            return dict(bytes=tok + row + 2 * pairs, flops=2 * live * h)
        return dict(bytes=tok + 2 * row + 3 * pairs, flops=3 * live * h)
    if case["op"] == "norm":
        read = sum(n * d.itemsize for n, d in zip(_sizes(case), _types(case)))
        if case["kind"] == "factor":
            return dict(bytes=read + 8, flops=2 * case["elements"])
        return dict(bytes=read + 2 * case["elements"] + 8, flops=3 * case["elements"])
    size = 4 if case["dtype"] == "float32" else 2
    b, s, v = case["sequences"], case["drafts"], case["vocab"]
    rows = b * (s + 1) + (b * s if case["by_model"] else 0)
    return dict(bytes=rows * v * size + 4 * b * v + 16 * b * (s + 1), flops=4 * rows * v + 4 * b * v)


# --------------------------------------------------------------------------- in 64 bits


def _exact_rows(s, case):
    k, e = case["topk"], case["experts"]
    t, h, dev = case["tokens"], case["hidden"], s["ids"].device
    pairs = [[] for _ in range(e)]
    for i, x in enumerate(s["ids"].reshape(-1).tolist()):
        if 0 <= x < e:
            pairs[x].append(i)
    order = torch.tensor([i for p in pairs for i in p], dtype=torch.long)
    dest = torch.full((t * k,), -1, dtype=torch.long)
    dest[order] = torch.arange(order.numel())
    order, dest = order.to(dev), dest.view(t, k).to(dev)
    if case["kind"] == "permute":
        src = torch.full((t * k,), -1, dtype=torch.int32, device=dev)
        src[: order.numel()] = (order // k).to(torch.int32)
        rows = torch.zeros(t * k, h, dtype=s["x"].dtype, device=dev)
        rows[: order.numel()] = s["x"].index_select(0, order // k)
        off = torch.tensor([0] + [len(p) for p in pairs]).cumsum(0).to(torch.int32).to(dev)
        return dict(rows=rows, offsets=off, perm_src=src, dest_row=dest.to(torch.int32))
    w = s["weights"].double().reshape(-1)
    if case["kind"] == "permute_grad":
        w = torch.ones_like(w)
    step = max(1, (1 << 25) // h)
    if case["kind"] in ("combine", "permute_grad"):
        y = torch.zeros(t, h, dtype=torch.float64, device=dev)
        for a in range(0, order.numel(), step):
            o = order[a: a + step]
            y.index_add_(0, o // k, s["rows"][a: a + o.numel()].double() * w[o][:, None])
        return y
    drows = torch.zeros(t * k, h, dtype=torch.float64, device=dev)
    dw = torch.zeros(t * k, dtype=torch.float64, device=dev)
    for a in range(0, order.numel(), step):
        o = order[a: a + step]
        d = s["x"][o // k].double()
        drows[a: a + o.numel()] = d * w[o][:, None]
        dw[o] = torch.einsum("ij,ij->i", d, s["rows"][a: a + o.numel()].double())
    return dict(drows=drows, dweights=dw.view(t, k))


def _exact_norm(s, case):
    total, piece = 0.0, 1 << 26
    for g in s["grads"]:
        for a in range(0, g.numel(), piece):
            d = g[a: a + piece].double()
            part = float(torch.dot(d, d)) if case["order"] == 2.0 else float(d.abs().max())
            total = total + part if case["order"] == 2.0 else max(total, part)
    norm = math.sqrt(total) if case["order"] == 2.0 else total
    scale = min(1.0, s["max_norm"] / (norm + 1e-6))
    dev = s["grads"][0].device
    res = dict(norm=torch.tensor([norm], dtype=torch.float64, device=dev),
               scale=torch.tensor([scale], dtype=torch.float64, device=dev))
    if case["kind"] == "clip":
        starts, total = _starts(_sizes(case))
        res["out"] = torch.zeros(total, dtype=torch.float32, device=dev)
        for a, g in zip(starts, s["grads"]):
            res["out"][a: a + g.numel()] = (g.double() * scale).float()
    return res


def _exact_verify(s, case):
    b, d, v, t = case["sequences"], case["drafts"], case["vocab"], s["temperature"]
    dev = s["target"].device
    tokens = torch.full((b, d + 1), -1, dtype=torch.int32)
    lps = torch.zeros(b, d + 1, dtype=torch.float64)
    accepted = torch.zeros(b, dtype=torch.int32)
    drafts, uniforms = s["tokens"].tolist(), s["uniforms"].tolist()
    for i in range(b):
        logp = torch.log_softmax(s["target"][i].double() / t, 1)
        p = logp.exp()
        q = torch.softmax(s["draft"][i].double() / t, 1) if s["draft"] is not None else None
        n, left = 0, None
        while n < d and drafts[i][n] >= 0:
            x = drafts[i][n]
            if uniforms[i][n] * (1.0 if q is None else float(q[n, x])) < float(p[n, x]):
                tokens[i, n], lps[i, n] = x, float(logp[n, x])
                n += 1
                continue
            other = q[n] if q is not None else torch.zeros(v, dtype=torch.float64, device=dev).index_fill_(
                0, torch.tensor([x], device=dev), 1.0)
            left = torch.relu(p[n] - other)
            break
        if left is None or float(left.max()) <= 0:
            left = p[n]
        new = int(torch.argmax(left / s["noise"][i].double()))
        tokens[i, n], lps[i, n], accepted[i] = new, float(logp[n, new]), n
    return dict(tokens=tokens.to(dev), accepted=accepted.to(dev), logprobs=lps.to(dev))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(rows=_exact_rows, norm=_exact_norm, verify=_exact_verify)[case["op"]](s, case)
