"""The learner's BF16 operators, as cases that can be timed and checked.

Three operators that one policy-update step of the learner runs next to the
NVFP4 expert MLP:

* ``experts``  matrix products grouped by expert over ragged row ranges, in
  BF16 with FP32 sums: forward (``out = a w^T``), activation gradient
  (``out = a w``, the weight read as stored) and weight gradient
  (``dw[e] += dy_e^T x_e``);
* ``logprobs`` the log probability of a given token of each row of logits,
  with the row's entropy and top alternatives, and their gradient;
* ``adamw``    one AdamW step over many tensors at once, with FP32 states or
  with 8-bit ones (E4M3 codes, one FP32 scale for each block of 256).

With ``own`` false, ``run`` computes them with elementary torch operations in
FP32, rounded once at the end; with ``own`` true it calls this package.
"""
import math

import torch

own = False

BLOCK = 256                                    # elements that share one scale of an 8-bit state
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
E4M3_MAX, TINY = 448.0, 2.0 ** -126


def _minite():
    from nvfp4_w4a4_moe_permute_gb300 import minite
    return minite


# --------------------------------------------------------------------------- the cases


def listed():
    return [
        # one token of a sampled sequence: 8 of 128 experts, one row each; the weights' bytes are all
        dict(name="experts_one_token", op="experts", kind="forward", tokens=1, topk=8, experts=128,
             n=1536, k=2048, skew=0.0),
        # a small layer with sizes that fill no tile: 602 rows over 9 experts, latency counts
        dict(name="experts_small_wgrad", op="experts", kind="wgrad", tokens=301, topk=2, experts=9,
             n=200, k=136, skew=0.0, out="bfloat16", accumulate=False),
        # the gate_up product of one 4096-token micro-batch
        dict(name="experts_gate_up", op="experts", kind="forward", tokens=4096, topk=8, experts=128,
             n=1536, k=2048, skew=0.0),
        # the gradient that flows back through gate_up when a few experts get most of the tokens
        dict(name="experts_skewed_dgrad", op="experts", kind="dgrad", tokens=8192, topk=8,
             experts=128, n=2048, k=1536, skew=1.2),
        # the gate_up weight gradient of one micro-batch, added to the FP32 sum over micro-batches
        dict(name="experts_wgrad", op="experts", kind="wgrad", tokens=4096, topk=8, experts=128,
             n=1536, k=2048, skew=0.0, out="float32", accumulate=True),
        # one decoded token, logits in FP32 as a sampler has them, 20 alternatives reported
        dict(name="logprobs_one_token", op="logprobs", kind="serve", rows=1, vocab=131072,
             dtype="float32", alternatives=20, masked=0.0, banned=0.5),
        # a batch of sequences at one decode step, an odd vocabulary
        dict(name="logprobs_sampler_batch", op="logprobs", kind="serve", rows=64, vocab=100003,
             dtype="bfloat16", alternatives=20, masked=0.0, banned=0.0),
        # one micro-batch of the learner, a quarter of it prompt tokens that have no loss
        dict(name="logprobs_learner", op="logprobs", kind="train", rows=4096, vocab=131072,
             dtype="bfloat16", alternatives=0, masked=0.25, banned=0.0),
        # a long packed batch
        dict(name="logprobs_learner_long", op="logprobs", kind="train", rows=8192, vocab=131072,
             dtype="bfloat16", alternatives=0, masked=0.0, banned=0.0),
        # norms and a router alone (what is trained when the experts are frozen): latency counts
        dict(name="adamw_router", op="adamw", tensors=6, elements=300001, bits=32, param="float32",
             copies=False),
        # every tensor of one 128-expert layer: FP32 master weights with their BF16 copies
        dict(name="adamw_layer", op="adamw", tensors=9, elements=604_241_920, bits=32,
             param="float32", copies=True),
        # a whole small model held in BF16 with 8-bit states
        dict(name="adamw_8bit_model", op="adamw", tensors=291, elements=400_000_003, bits=8,
             param="bfloat16", copies=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "logprobs", "adamw"])
    if op == "experts":
        kind = rng.choice(["forward", "dgrad", "wgrad"])
        e = _log(rng, 1, 128)
        topk = min(e, rng.choice([1, 2, 4, 8]))
        c = dict(op=op, kind=kind, tokens=_log(rng, 1, 4096), topk=topk, experts=e,
                 n=8 * _log(rng, 8, 192), k=8 * _log(rng, 8, 256),
                 skew=rng.choice([0.0, 0.0, 1.2]))
        if kind == "wgrad":
            c["out"] = rng.choice(["float32", "bfloat16"])
            c["accumulate"] = c["out"] == "float32" and rng.random() < 0.5
        return c
    if op == "logprobs":
        kind = rng.choice(["serve", "train"])
        serve = kind == "serve"
        return dict(op=op, kind=kind, rows=_log(rng, 1, 512 if serve else 6000),
                    vocab=_log(rng, 500, 160000) if serve else _log(rng, 500, 131072),
                    dtype=rng.choice(["float32", "bfloat16"]) if serve else "bfloat16",
                    alternatives=rng.choice([1, 5, 20, 32]) if serve else 0,
                    masked=0.0 if serve else rng.choice([0.0, 0.3]),
                    banned=rng.choice([0.0, 0.5]))
    tensors = _log(rng, 1, 400)
    param = rng.choice(["float32", "bfloat16"])
    return dict(op=op, tensors=tensors, elements=_log(rng, 1000, 300_000_000) + tensors,
                bits=rng.choice([8, 32]), param=param,
                copies=param == "float32" and rng.random() < 0.5)


# --------------------------------------------------------------------------- their inputs


def _routing(case, seed):
    """Rows of each expert: every token takes topk experts without repetition."""
    e = case["experts"]
    g = torch.Generator().manual_seed(seed)
    p = torch.arange(1, e + 1, dtype=torch.float64) ** -case["skew"]
    p = p[torch.randperm(e, generator=g)]
    ids = torch.multinomial(p.expand(case["tokens"], e), case["topk"], generator=g)
    counts = torch.bincount(ids.reshape(-1), minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return offsets, int(counts.max())


def _sizes(case):
    """Sizes of the tensors: a few large ones, a long tail of small ones, odd ones among them."""
    n, total = case["tensors"], case["elements"]
    w = [1.0 / (i + 1) ** 1.5 for i in range(n)]
    s = sum(w)
    sizes = [max(1, int((total - n) * x / s)) for x in w]
    sizes[0] += total - sum(sizes)
    return sizes


def _starts(sizes):
    """Each tensor's place in a flat buffer: whole blocks, so that no block spans two tensors."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    state = dict(case=case)
    if case["op"] == "experts":
        offsets, most = _routing(case, seed)
        m, n, k, e = case["tokens"] * case["topk"], case["n"], case["k"], case["experts"]
        state |= dict(offsets=offsets.to(dev), most=most)
        x = randn(m, k)
        x[:, :: 100] *= 20  # outlier channels
        state["x"] = x
        if case["kind"] == "wgrad":
            state["dy"] = randn(m, n, std=1e-3)
            state["out"] = randn(e, n, k, std=1e-2, dtype=torch.float32) if case["accumulate"] else None
        elif case["kind"] == "forward":
            state["w"] = randn(e, n, k, std=0.02)
        else:
            state["w"] = randn(e, k, n, std=0.02)
        return state
    if case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        logits = randn(rows, vocab, std=2.0, dtype=getattr(torch, case["dtype"]))
        targets = torch.randint(0, vocab, (rows,), generator=g, device=dev, dtype=torch.int32)
        # the model has learned something: the tokens it sampled stand out
        logits.scatter_add_(1, targets.long()[:, None],
                            randn(rows, 1, std=3.0, dtype=logits.dtype) + 8.0)
        if case["banned"]:  # a grammar's mask, the given token always allowed
            ban = torch.rand(vocab, generator=g, device=dev) < case["banned"]
            keep = logits.gather(1, targets.long()[:, None])
            logits[:, ban] = float("-inf")
            logits.scatter_(1, targets.long()[:, None], keep)
        off = torch.randperm(rows, generator=g, device=dev)[: int(rows * case["masked"])]
        targets[off] = -1
        state |= dict(logits=logits, targets=targets, temperature=0.8)
        if case["kind"] == "train":
            state |= dict(grad_logprob=randn(rows, std=1e-3, dtype=torch.float32),
                          grad_entropy=randn(rows, std=1e-4, dtype=torch.float32))
        return state
    sizes = _sizes(case)
    starts, total = _starts(sizes)
    live = torch.zeros(total, device=dev, dtype=torch.bool)
    for s, n in zip(starts, sizes):
        live[s: s + n] = True
    p = randn(total, std=0.02, dtype=torch.float32).mul_(live)
    m = randn(total, std=1e-4, dtype=torch.float32).mul_(live)
    v = randn(total, std=2e-4, dtype=torch.float32).square_().add_(1e-9).mul_(live)
    if case["bits"] == 8:
        state["exp_avg"], state["exp_avg_scale"] = _encode(m)
        state["exp_avg_sq"], state["exp_avg_sq_scale"] = _encode_sq(v)
    else:
        state["exp_avg"], state["exp_avg_sq"] = m, v
    p = p.to(getattr(torch, case["param"]))
    grads = [randn(n, std=3e-4) for n in sizes]
    state |= dict(flat=p, params=[p[s: s + n] for s, n in zip(starts, sizes)], grads=grads,
                  starts=starts, sizes=sizes, total=total, step=100,
                  grad_scale=torch.full((1,), 0.7, device=dev))
    if case["copies"]:
        state["flat_copy"] = p.to(torch.bfloat16)
        state["copies"] = [state["flat_copy"][s: s + n] for s, n in zip(starts, sizes)]
    if own:  # the optimizer that a training program builds once over its tensors and states
        kept = {k: state[k] for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
                if k in state}
        state["opt"] = _minite().AdamW(
            state["params"], copies=state.get("copies"), state_bits=case["bits"], lr=LR,
            betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state=dict(kept, step=state["step"]))
    return state


# --------------------------------------------------------------------------- the plain forms


def _padded(x, offsets, most):
    """[rows, c] in expert order -> FP32 [experts, most, c], zero where an expert has no row."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device)
    live = at < offsets[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)].float().mul_(live[..., None])


def _experts(state):
    case, offsets, most = state["case"], state["offsets"].long(), state["most"]
    x = _padded(state["x"], offsets, most)
    if case["kind"] == "wgrad":
        dy = _padded(state["dy"], offsets, most)
        dw = torch.bmm(dy.transpose(1, 2), x)
        if case["accumulate"]:
            return state["out"].add_(dw)
        return dw.to(getattr(torch, case["out"]))
    w = state["w"].float()
    y = torch.bmm(x, w.transpose(1, 2) if case["kind"] == "forward" else w)
    row = torch.arange(state["x"].shape[0], device=x.device)
    e = torch.searchsorted(offsets[1:], row, right=True)
    return y[e, row - offsets[e]].to(torch.bfloat16)


def _logprobs(state):
    case, targets = state["case"], state["targets"].long()
    live = targets >= 0
    x = state["logits"].float() / state["temperature"]
    x = x - x.amax(1, keepdim=True)
    logp = x - x.exp().sum(1, keepdim=True).log()
    p = logp.exp()
    ent = -torch.where(p > 0, p * logp, 0.0).sum(1)
    picked = logp.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    res = dict(logprob=torch.where(live, picked, 0.0), entropy=torch.where(live, ent, 0.0))
    if case["alternatives"]:
        ids = torch.sort(state["logits"], dim=1, descending=True, stable=True).indices
        ids = ids[:, : case["alternatives"]]  # ties: the lowest index first
        res["alt_ids"] = ids.to(torch.int32)
        res["alt_logprobs"] = logp.gather(1, ids)
    if case["kind"] == "train":
        gl = torch.where(live, state["grad_logprob"], 0.0)
        ge = torch.where(live, state["grad_entropy"], 0.0)
        d = -p * (gl[:, None] + ge[:, None] * (logp.clamp(min=-1e30) + ent[:, None]))
        d.scatter_add_(1, targets.clamp(min=0)[:, None], gl[:, None])
        res["dlogits"] = (d / state["temperature"]).to(state["logits"].dtype)
    return res


def _scale(amax):
    return (amax / E4M3_MAX).clamp(min=TINY)


def _encode(m):
    """E4M3 codes of blocks of 256 and their scales."""
    b = m.view(-1, BLOCK)
    s = _scale(b.abs().amax(1))
    return (b * (1.0 / s)[:, None]).to(torch.float8_e4m3fn).view(-1), s


def _encode_sq(v):
    """The same of sqrt(v); one above zero never becomes zero."""
    r = v.sqrt().view(-1, BLOCK)
    s = _scale(r.amax(1))
    c = (r * (1.0 / s)[:, None]).clamp(min=2.0 ** -9).mul_(r > 0)
    return c.to(torch.float8_e4m3fn).view(-1), s


def _adamw(state):
    case = state["case"]
    eight = case["bits"] == 8
    state["step"] += 1
    bc1, bc2 = 1 - BETA1 ** state["step"], 1 - BETA2 ** state["step"]
    g = torch.zeros(state["total"], device=state["flat"].device)
    torch._foreach_copy_([g[s: s + n] for s, n in zip(state["starts"], state["sizes"])], state["grads"])
    g.mul_(state["grad_scale"])
    m, v = state["exp_avg"], state["exp_avg_sq"]
    if eight:
        m = (m.float().view(-1, BLOCK) * state["exp_avg_scale"][:, None]).view(-1)
        v = (v.float().view(-1, BLOCK) * state["exp_avg_sq_scale"][:, None]).square().view(-1)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    u = m / (v.sqrt() * (1 / math.sqrt(bc2)) + EPS)
    p = state["flat"].float() * (1 - LR * DECAY) - u * (LR / bc1)
    state["flat"].copy_(p)
    res = dict(params=state["flat"])
    if case["copies"]:
        res["copies"] = state["flat_copy"].copy_(p)
    if eight:
        for name, (codes, scale) in (("exp_avg", _encode(m)), ("exp_avg_sq", _encode_sq(v))):
            res[name] = state[name].copy_(codes)
            res[name + "_scale"] = state[name + "_scale"].copy_(scale)
    else:
        res["exp_avg"] = state["exp_avg"].copy_(m)
        res["exp_avg_sq"] = state["exp_avg_sq"].copy_(v)
    return res


def run(state):
    case = state["case"]
    if not own:
        return dict(experts=_experts, logprobs=_logprobs, adamw=_adamw)[case["op"]](state)
    M = _minite()
    if case["op"] == "experts":
        if case["kind"] == "wgrad":
            return M.grouped_wgrad_bf16(state["dy"], state["x"], state["offsets"], out=state["out"],
                                        out_dtype=getattr(torch, case["out"]),
                                        accumulate=case["accumulate"])
        return M.grouped_gemm_bf16(state["x"], state["w"], state["offsets"],
                                   w_as_stored=case["kind"] == "dgrad")
    if case["op"] == "logprobs":
        r = M.token_logprobs(state["logits"], state["targets"], temperature=state["temperature"],
                             alternatives=case["alternatives"])
        res = dict(logprob=r["logprob"], entropy=r["entropy"])
        if case["alternatives"]:
            res |= dict(alt_ids=r["alt_ids"], alt_logprobs=r["alt_logprobs"])
        if case["kind"] == "train":
            res["dlogits"] = M.token_logprobs_backward(
                state["logits"], state["targets"], r, state["grad_logprob"], state["grad_entropy"],
                temperature=state["temperature"])
        return res
    opt = state["opt"]
    opt.step(state["grads"], grad_scale=state["grad_scale"])
    res = dict(params=state["flat"], exp_avg=opt.exp_avg, exp_avg_sq=opt.exp_avg_sq)
    if case["copies"]:
        res["copies"] = state["flat_copy"]
    if case["bits"] == 8:
        res |= dict(exp_avg_scale=opt.exp_avg_scale, exp_avg_sq_scale=opt.exp_avg_sq_scale)
    return res


# --------------------------------------------------------------------------- what a pass needs


def work(case):
    if case["op"] == "experts":
        m, n, k, e = case["tokens"] * case["topk"], case["n"], case["k"], case["experts"]
        p = [(i + 1) ** -case["skew"] for i in range(e)]
        s = sum(p)
        # experts that get a row, with the draws taken as independent
        hit = sum(1 - (1 - x / s) ** m for x in p)
        if case["tokens"] == 1:
            hit = case["topk"]
        if case["kind"] == "wgrad":
            size = 4 if case["out"] == "float32" else 2
            w = e * n * k * size + (hit * n * k * size if case["accumulate"] else 0)
            if case["accumulate"]:  # an expert without rows keeps its sum untouched
                w -= (e - hit) * n * k * size
        else:
            w = hit * n * k * 2
        return dict(bytes=2 * m * (n + k) + w, flops=2 * m * n * k)
    if case["op"] == "logprobs":
        size = 4 if case["dtype"] == "float32" else 2
        live = case["rows"] - int(case["rows"] * case["masked"])
        read = live * case["vocab"] * size
        if case["kind"] == "serve":
            return dict(bytes=read + case["rows"] * (12 + 8 * case["alternatives"]),
                        flops=5 * live * case["vocab"])
        write = case["rows"] * case["vocab"] * size
        return dict(bytes=read + write + 20 * case["rows"], flops=12 * live * case["vocab"])
    p = 8 if case["param"] == "float32" else 4
    per = p + 2 + (2 if case["copies"] else 0) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
    return dict(bytes=per * case["elements"], flops=16 * case["elements"])


# --------------------------------------------------------------------------- in 64 bits


def _exact_experts(s, case):
    off = s["offsets"].tolist()
    m, n, k, e = s["x"].shape[0], case["n"], case["k"], case["experts"]
    if case["kind"] == "wgrad":
        out = torch.zeros(e, n, k, device="cuda", dtype=torch.float32 if e * n * k > 1 << 27 else torch.float64)
        for i in range(e):
            a, b = off[i], off[i + 1]
            dw = s["dy"][a:b].double().t() @ s["x"][a:b].double()
            out[i] = dw + s["out"][i].double() if case["accumulate"] else dw
        return out
    out = torch.empty(m, n, device="cuda", dtype=torch.float64)
    for i in range(e):
        a, b = off[i], off[i + 1]
        w = s["w"][i].double()
        out[a:b] = s["x"][a:b].double() @ (w.t() if case["kind"] == "forward" else w)
    return out


def _exact_logprobs(s, case):
    rows, vocab, t = case["rows"], case["vocab"], s["temperature"]
    res = dict(logprob=torch.zeros(rows, device="cuda", dtype=torch.float64),
               entropy=torch.zeros(rows, device="cuda", dtype=torch.float64))
    alt = case["alternatives"]
    if alt:
        res["alt_ids"] = None
        res["alt_logprobs"] = torch.zeros(rows, alt, device="cuda", dtype=torch.float64)
    if case["kind"] == "train":
        res["dlogits"] = torch.zeros(rows, vocab, device="cuda", dtype=torch.float32)
    for r0 in range(0, rows, 256):
        cut = slice(r0, min(rows, r0 + 256))
        x = s["logits"][cut].double().div_(t)
        y = s["targets"][cut].long()
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - top)
        z = e.sum(1, keepdim=True)
        p = e / z
        lse = top + z.log()
        plogp = torch.special.entr(p)
        h = plogp.sum(1)
        on = (y >= 0).double()
        res["logprob"][cut] = on * (x.gather(1, y.clamp(min=0)[:, None]) - lse)[:, 0]
        res["entropy"][cut] = on * h
        if alt:
            res["alt_logprobs"][cut] = x.topk(alt, dim=1).values - lse
        if case["kind"] == "train":
            gl, ge = (on * s[k][cut].double() for k in ("grad_logprob", "grad_entropy"))
            d = (plogp - p * h[:, None]) * ge[:, None] - p * gl[:, None]
            d[torch.arange(d.shape[0], device="cuda"), y.clamp(min=0)] += gl
            res["dlogits"][cut] = (d / t).float()
    return res


def _exact_adamw(s, case):
    out = {k: torch.empty_like(s["flat"], dtype=torch.float32) for k in ("params",)}
    eight, step, total = case["bits"] == 8, s["step"] + 1, s["total"]
    state_type = torch.float8_e4m3fn if eight else torch.float32
    out["exp_avg"] = torch.empty(total, device="cuda", dtype=state_type)
    out["exp_avg_sq"] = torch.empty(total, device="cuda", dtype=state_type)
    if eight:
        out["exp_avg_scale"] = torch.empty(total // BLOCK, device="cuda", dtype=torch.float64)
        out["exp_avg_sq_scale"] = torch.empty(total // BLOCK, device="cuda", dtype=torch.float64)
    grad = torch.zeros(total, device="cuda", dtype=torch.bfloat16)
    for at, n, g in zip(s["starts"], s["sizes"], s["grads"]):
        grad[at: at + n] = g
    clip = s["grad_scale"].double()
    piece = 1 << 25
    for a in range(0, total, piece):
        c = slice(a, min(total, a + piece))
        b = slice(c.start // BLOCK, c.stop // BLOCK)
        g = grad[c].double() * clip
        m, v = s["exp_avg"][c].double(), s["exp_avg_sq"][c].double()
        if eight:
            m = m * s["exp_avg_scale"][b].double().repeat_interleave(BLOCK)
            v = (v * s["exp_avg_sq_scale"][b].double().repeat_interleave(BLOCK)) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        step_size = LR / (1 - BETA1 ** step)
        den = torch.sqrt(v / (1 - BETA2 ** step)) + EPS
        p = s["flat"][c].double()
        out["params"][c] = (p - LR * DECAY * p - step_size * m / den).float()
        if not eight:
            out["exp_avg"][c], out["exp_avg_sq"][c] = m.float(), v.float()
            continue
        for name, x in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
            x = x.view(-1, BLOCK)
            scale = (x.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
            code = x / scale[:, None]
            if name == "exp_avg_sq":
                code = torch.where(x > 0, code.clamp(min=2.0 ** -9), code)
            out[name][c] = code.float().to(torch.float8_e4m3fn).view(-1)
            out[name + "_scale"][b] = scale
    if case["copies"]:
        out["copies"] = out["params"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(experts=_exact_experts, logprobs=_exact_logprobs, adamw=_exact_adamw)[case["op"]](s, case)
