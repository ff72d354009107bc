"""Cases that measure the training-step operators: expert products, global gradient clipping, the clipped policy loss.

With ``own`` false ``run`` computes a case in elementary torch operations, in 32 bits whatever the inputs' type and
rounded once at the end; with ``own`` true it makes the calls of ``conv2d_backward_implicit_bwd_gb300.train``.

The operators, on row-major tensors:

experts   Rows of x [rows, k] sorted by expert; expert e owns rows offsets[e] .. offsets[e+1]-1 and the filter
          w[e] [n, k].  forward: y = x w[e]^T.  data: dx = dy w[e].  weight: dw[e] (+)= dy_e^T x_e.  Rows of no expert
          (past offsets[-1]) give zero rows.
clip      norm = sqrt(sum of squares over all tensors), coef = min(1, max_norm / (norm + 1e-6)), every tensor times coef.
policy    logp_t = s z_t[a_t] - logsumexp(s z_t); r = exp(logp - old); d = ref - logp;
          loss = sum_t w_t (-min(r A, clip(r, 1-lo, 1+hi) A) + kl (exp(d) - d - 1));
          dlogits_t = g c_t s (onehot(a_t) - softmax(s z_t)) with c_t = dloss/dlogp_t.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LO, HI, KL, SCALE = 0.2, 0.28, 0.04, 0.8
MAX_NORM = 1.0


def listed():
    experts = dict(op="experts", dtype="bf16", spare=0, accumulate=False)
    return [
        # serving, one token that the router sends to 8 of 64 experts: latency, and 8 filters to read
        dict(experts, name="experts fwd one token", dir="forward", experts=64, rows=8, k=1024, n=2048),
        # serving, a decode batch: few rows for each expert, every filter is read
        dict(experts, name="experts fwd decode", dir="forward", experts=64, rows=256, k=2048, n=1024),
        # a prompt of odd length over an odd number of experts, widths that end inside tiles, a padded row buffer
        dict(experts, name="experts fwd odd", dir="forward", experts=13, rows=3111, k=520, n=1000, spare=41),
        # training, up-projection of a batch
        dict(experts, name="experts fwd train", dir="forward", experts=16, rows=16384, k=1024, n=2048),
        # training, gradient of the rows; the largest product
        dict(experts, name="experts data train", dir="data", experts=32, rows=32768, k=2048, n=2048),
        # training, gradient of the filters, added to 32-bit gradients over micro-batches
        dict(experts, name="experts weight add f32", dir="weight", experts=16, rows=16384, k=1024, n=2048, accumulate=True),
        # 32-bit tensors of odd widths: a small router-sized layer kept in full precision
        dict(experts, name="experts weight f32 odd", dir="weight", dtype="f32", experts=7, rows=777, k=100, n=131),
        # the norm and clipping of a small model's gradients, in place: latency
        dict(op="clip", name="clip small f32", dtype="f32", count=48, elements=200_003, inplace=True),
        # a large model's gradients, 16-bit matrices and 32-bit vectors, clipped into the optimiser's buffers
        dict(op="clip", name="clip large mixed", dtype="mixed", count=310, elements=700_000_000, inplace=False),
        # loss and its gradient in one call, the training step's form
        dict(op="policy", name="policy loss and grad", dir="both", dtype="bf16", tokens=8192, vocab=32768),
        # log-probabilities and loss alone, an odd vocabulary in 32 bits
        dict(op="policy", name="policy forward odd f32", dir="forward", dtype="f32", tokens=1021, vocab=50257),
        # the gradient from saved statistics, a short sequence of a wide vocabulary
        dict(op="policy", name="policy backward", dir="backward", dtype="bf16", tokens=300, vocab=128000),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("experts", "experts", "experts", "clip", "policy"))
    if op == "experts":
        way = rng.choice(("forward", "data", "weight"))
        if rng.random() < 0.2:
            return dict(op=op, dir=way, dtype="f32", experts=log(1, 16), rows=log(1, 1500), k=log(8, 300), n=log(8, 300), spare=rng.choice((0, 5)), accumulate=way == "weight" and rng.random() < 0.5)
        return dict(op=op, dir=way, dtype="bf16", experts=log(1, 64), rows=log(1, 20000), k=8 * log(8, 256), n=8 * log(8, 256), spare=rng.choice((0, 0, 17)),
                    accumulate=way == "weight" and rng.random() < 0.5)
    if op == "clip":
        return dict(op=op, dtype=rng.choice(("f32", "bf16", "mixed")), count=log(1, 300), elements=log(3000, 300_000_000), inplace=rng.random() < 0.5)
    vocab = log(2, 131072)
    return dict(op=op, dir=rng.choice(("forward", "backward", "both")), dtype=rng.choice(("f32", "bf16")), tokens=log(1, max(2, min(8192, (1 << 27) // vocab))), vocab=vocab)


# ---- sizes that follow from the case alone ---------------------------------
def expert_rows(case):
    """Rows of each expert, unevenly shared; at most one in four experts is left without any."""
    r = random.Random("%d/%d" % (case["experts"], case["rows"]))
    share = [0.0 if case["experts"] > 3 and r.random() < 0.06 else r.uniform(0.4, 1.6) for _ in range(case["experts"])]
    if not any(share):
        share[0] = 1.0
    picks = r.choices(range(case["experts"]), share, k=case["rows"]) if case["rows"] >= 2 * case["experts"] else [r.randrange(case["experts"]) for _ in range(case["rows"])]
    rows = [0] * case["experts"]
    for e in picks:
        rows[e] += 1
    return rows


def tensor_sizes(case):
    """Elements of each tensor: every second one a vector of up to 4096, the matrices share the rest unevenly."""
    r = random.Random("%d/%d" % (case["count"], case["elements"]))
    vectors = [0 if i % 2 == 0 else min(r.randrange(1, 4097), case["elements"] // (2 * case["count"])) for i in range(case["count"])]
    share = [r.uniform(0.2, 1.8) if i % 2 == 0 else 0.0 for i in range(case["count"])]
    left = case["elements"] - sum(vectors)
    return [v if i % 2 else max(1, int(left * share[i] / sum(share))) for i, v in enumerate(vectors)]


# ---- inputs ----------------------------------------------------------------
def normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare_experts(case, gen, seed):
    dt = DTYPES[case["dtype"]]
    rows = expert_rows(case)
    random.Random(seed).shuffle(rows)
    offsets = [sum(rows[:e]) for e in range(len(rows) + 1)]
    total, k, n, e = case["rows"] + case["spare"], case["k"], case["n"], case["experts"]
    s = dict(offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), longest=max(rows))
    if case["dir"] != "data":
        s["x"] = normal(gen, (total, k), dt)
    if case["dir"] != "forward":
        s["dy"] = normal(gen, (total, n), dt, 0.01)
    if case["dir"] != "weight":
        s["w"] = normal(gen, (e, n, k), dt, 1.0 / math.sqrt(k))
    elif case["accumulate"]:
        s["dw"] = normal(gen, (e, n, k), torch.float32, 0.01)
    return s


def prepare_clip(case, gen, seed):
    kinds = {"f32": ("f32",), "bf16": ("bf16",), "mixed": ("bf16", "f32")}[case["dtype"]]
    sizes = tensor_sizes(case)
    flat, outs, grads, into = {}, {}, [None] * len(sizes), [None] * len(sizes)
    for j, kind in enumerate(kinds):
        mine = [i for i in range(len(sizes)) if i % len(kinds) == j]
        at, total = [], 0
        for i in mine:  # a bucket of each type, its tensors on 64-element boundaries
            at.append(total)
            total += -(-sizes[i] // 64) * 64
        scale = 10.0 * MAX_NORM / math.sqrt(case["elements"])
        flat[kind] = normal(gen, (total,), DTYPES[kind], scale)
        if not case["inplace"]:
            outs[kind] = torch.zeros_like(flat[kind])
        for i, a in zip(mine, at):
            grads[i] = flat[kind][a:a + sizes[i]]
            into[i] = outs[kind][a:a + sizes[i]] if not case["inplace"] else None
            flat[kind][a + sizes[i]:a + -(-sizes[i] // 64) * 64] = 0
    return dict(grads=grads, into=None if case["inplace"] else into, flat=flat if case["inplace"] else outs)


def prepare_policy(case, gen, seed):
    t, v, dt = case["tokens"], case["vocab"], DTYPES[case["dtype"]]
    logits = torch.empty((t, v), dtype=dt, device="cuda")
    step = max(1, (1 << 27) // v)
    logp, lse = [], []
    tokens = torch.randint(0, v, (t,), generator=gen, device="cuda", dtype=torch.int32)
    for i in range(0, t, step):
        logits[i:i + step] = normal(gen, logits[i:i + step].shape, dt, 2.0)
        z = logits[i:i + step].float() * SCALE
        lse.append(torch.logsumexp(z, 1))
        logp.append(z.gather(1, tokens[i:i + step, None].long())[:, 0] - lse[-1])
    logp, lse = torch.cat(logp), torch.cat(lse)
    kept = (torch.rand((t,), generator=gen, device="cuda") < 0.9).float()
    kept[0] = 1.0
    s = dict(logits=logits, tokens=tokens)
    advantage, weight = normal(gen, (t,), torch.float32) + 0.3, kept / kept.sum()
    old, ref = logp + normal(gen, (t,), torch.float32, 0.15), logp + normal(gen, (t,), torch.float32, 0.2)
    if case["dir"] == "backward":
        s.update(lse=lse, coef=-weight * advantage * torch.exp(logp - old), grad=torch.full((1,), 2.0, device="cuda"))
    else:
        s.update(advantage=advantage, weight=weight, old=old, ref=ref)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return dict({"experts": prepare_experts, "clip": prepare_clip, "policy": prepare_policy}[case["op"]](case, gen, seed), case=case)


# ---- the framework's calls -------------------------------------------------
@functools.lru_cache(maxsize=None)
def expert_plan(experts, k, n, dtype):
    from conv2d_backward_implicit_bwd_gb300 import train
    return train.Experts(experts, k, n, dtype)


@functools.lru_cache(maxsize=None)
def clip_plan(sizes, dtypes):
    from conv2d_backward_implicit_bwd_gb300 import train
    return train.GradClip(sizes, dtypes)


@functools.lru_cache(maxsize=None)
def policy_plan(vocab, dtype):
    from conv2d_backward_implicit_bwd_gb300 import train
    return train.PolicyLoss(vocab, dtype, clip_low=LO, clip_high=HI, kl=KL, scale=SCALE)


def run_own(state, case):
    if case["op"] == "experts":
        plan = expert_plan(case["experts"], case["k"], case["n"], case["dtype"])
        if case["dir"] == "forward":
            return plan.forward(state["x"], state["w"], state["offsets"])
        if case["dir"] == "data":
            return plan.backward_data(state["dy"], state["w"], state["offsets"])
        return plan.backward_weight(state["dy"], state["x"], state["offsets"], out=state.get("dw"), accumulate=case["accumulate"])
    if case["op"] == "clip":
        if "plan" not in state:
            state["plan"] = clip_plan(tuple(g.numel() for g in state["grads"]), tuple("f32" if g.dtype == torch.float32 else "bf16" for g in state["grads"]))
        norm, coef = state["plan"].clip(state["grads"], MAX_NORM, out=state["into"])
        return dict(state["flat"], norm=norm, coef=coef)
    plan = policy_plan(case["vocab"], case["dtype"])
    if case["dir"] == "backward":
        return plan.backward(state["logits"], state["tokens"], state["lse"], state["coef"], grad=state["grad"])
    args = (state["logits"], state["tokens"], state["advantage"], state["weight"])
    if case["dir"] == "both":
        loss, logp, dlogits = plan.forward_backward(*args, old_logp=state["old"], ref_logp=state["ref"])
        return dict(loss=loss, logp=logp, dlogits=dlogits)
    loss, logp, lse, coef = plan.forward(*args, old_logp=state["old"], ref_logp=state["ref"])
    return dict(loss=loss, logp=logp, lse=lse, coef=coef)


# ---- the plain forms -------------------------------------------------------
def by_expert(t, offsets, longest):
    """Rows of t as [experts, longest, width] in 32 bits, zero past each expert's rows."""
    j = torch.arange(longest, device="cuda")
    at = offsets[:-1, None].long() + j
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], t[at.clamp(max=t.shape[0] - 1)].float(), 0.0)


def to_rows(p, offsets, total, dtype):
    """[experts, longest, width] back to rows; rows of no expert are zero."""
    row = torch.arange(total, device="cuda", dtype=torch.int32)
    e = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    inside = e < offsets.numel() - 1
    e = e.clamp(max=offsets.numel() - 2)
    return torch.where(inside[:, None], p[e, (row - offsets[e]).clamp(0, p.shape[1] - 1).long()], 0.0).to(dtype)


def run_plain(state, case):
    if case["op"] == "experts":
        off, longest = state["offsets"], state["longest"]
        if case["dir"] == "forward":
            x = state["x"]
            return to_rows(torch.bmm(by_expert(x, off, longest), state["w"].float().transpose(1, 2)), off, x.shape[0], x.dtype)
        dy = state["dy"]
        if case["dir"] == "data":
            return to_rows(torch.bmm(by_expert(dy, off, longest), state["w"].float()), off, dy.shape[0], dy.dtype)
        dw = torch.bmm(by_expert(dy, off, longest).transpose(1, 2), by_expert(state["x"], off, longest))
        if case["accumulate"]:
            return state["dw"].add_(dw)
        return dw
    if case["op"] == "clip":
        squares = [g.float().square().sum() for g in state["grads"]]
        norm = torch.stack(squares).sum().sqrt().reshape(1)
        coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        into = state["into"] if state["into"] is not None else state["grads"]
        torch._foreach_copy_(into, [(g.float() * coef).to(g.dtype) for g in state["grads"]])
        return dict(state["flat"], norm=norm, coef=coef)
    logits, at = state["logits"], state["tokens"].long()[:, None]
    z = logits.float() * SCALE
    if case["dir"] == "backward":
        p = torch.exp(z - state["lse"][:, None])
        c = state["coef"] * state["grad"] * SCALE
        return (p.scatter_add(1, at, torch.full_like(p[:, :1], -1.0)) * -c[:, None]).to(logits.dtype)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    logp = z.gather(1, at)[:, 0] - lse
    w, a = state["weight"], state["advantage"]
    r, d = torch.exp(logp - state["old"]), state["ref"] - logp
    loss = (w * (-torch.minimum(r * a, r.clamp(1 - LO, 1 + HI) * a) + KL * (torch.exp(d) - d - 1))).sum().reshape(1)
    coef = w * (torch.where(r * a <= r.clamp(1 - LO, 1 + HI) * a, -r * a, 0.0) + KL * (1 - torch.exp(d)))
    kept = w != 0
    logp, lse = torch.where(kept, logp, 0.0), torch.where(kept, lse, 0.0)
    if case["dir"] == "forward":
        return dict(loss=loss, logp=logp, lse=lse, coef=coef)
    p = e / total
    return dict(loss=loss, logp=logp, dlogits=(p.scatter_add(1, at, torch.full_like(p[:, :1], -1.0)) * (-coef * SCALE)[:, None]).to(logits.dtype))


def run(state):
    return run_own(state, state["case"]) if own else run_plain(state, state["case"])


# ---- what a pass cannot do without -----------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2, "mixed": 3}[case["dtype"]]
    if case["op"] == "experts":
        rows = expert_rows(case)
        m, k, n, total = case["rows"], case["k"], case["n"], case["rows"] + case["spare"]
        flops = 2.0 * m * k * n
        used = sum(r > 0 for r in rows)
        if case["dir"] == "forward":
            return dict(bytes=size * (m * k + used * n * k + total * n), flops=flops)
        if case["dir"] == "data":
            return dict(bytes=size * (m * n + used * n * k + total * k), flops=flops)
        return dict(bytes=size * m * (k + n) + 4 * k * n * (2 * used if case["accumulate"] else case["experts"]), flops=flops)
    if case["op"] == "clip":
        sizes = tensor_sizes(case)
        total = sum(n * ({"f32": 4, "bf16": 2}[case["dtype"]] if case["dtype"] != "mixed" else (2, 4)[i % 2]) for i, n in enumerate(sizes))
        return dict(bytes=2 * total + 8, flops=3 * sum(sizes))
    t, v = case["tokens"], case["vocab"]
    return dict(bytes=size * t * v * (1 if case["dir"] == "forward" else 2) + 28 * t, flops=t * v * {"forward": 4, "backward": 4, "both": 8}[case["dir"]])


# ---- the definition in 64 bits ---------------------------------------------
def exact_experts(case, s):
    off = s["offsets"].tolist()
    total = case["rows"] + case["spare"]
    if case["dir"] == "weight":
        out = s["dw"].double() if case["accumulate"] else torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros((total, case["n"] if case["dir"] == "forward" else case["k"]), dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        if case["dir"] == "forward":
            out[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
        elif case["dir"] == "data":
            out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
        else:
            out[e] += s["dy"][a:b].double().T @ s["x"][a:b].double()
    return out


def exact_clip(case, s):
    square = 0.0
    for g in s["grads"]:
        for part in g.split(1 << 26):
            square += float(torch.dot(part.double(), part.double()))
    norm = math.sqrt(square)
    coef = min(1.0, MAX_NORM / (norm + 1e-6))
    for g, o in zip(s["grads"], s["into"] or s["grads"]):
        o.copy_(g)
    flat = {kind: f.double() * coef for kind, f in s["flat"].items()}
    one = torch.ones(1, dtype=torch.float64, device="cuda")
    return dict(flat, norm=one * norm, coef=one * coef)


def exact_policy(case, s):
    parts, step = [], max(1, (1 << 26) // case["vocab"])
    for i in range(0, case["tokens"], step):
        rows = slice(i, i + step)
        z = SCALE * s["logits"][rows].double()
        at = s["tokens"][rows].long()
        pick = torch.zeros_like(z)
        pick[torch.arange(len(at), device="cuda"), at] = 1.0
        if case["dir"] == "backward":
            soft = torch.exp(z - s["lse"][rows].double()[:, None])
            parts.append(dict(dlogits=float(s["grad"]) * SCALE * s["coef"][rows].double()[:, None] * (pick - soft)))
            continue
        lse = torch.logsumexp(z, 1)
        logp = (z * pick).sum(1) - lse
        w, a = s["weight"][rows].double(), s["advantage"][rows].double()
        r = torch.exp(logp - s["old"][rows].double())
        d = s["ref"][rows].double() - logp
        held = r.clamp(1.0 - LO, 1.0 + HI)
        free = r * a <= held * a
        loss = w * (KL * (torch.expm1(d) - d) - torch.where(free, r * a, held * a))
        coef = w * (-KL * torch.expm1(d) - torch.where(free, r * a, torch.zeros_like(a)))
        kept = (w != 0).double()
        part = dict(loss=loss, logp=logp * kept, lse=lse * kept, coef=coef)
        if case["dir"] == "both":
            part["dlogits"] = SCALE * coef[:, None] * (pick - torch.exp(z - lse[:, None]))
        parts.append(part)
    whole = {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
    if case["dir"] == "backward":
        return whole["dlogits"]
    whole["loss"] = whole["loss"].sum().reshape(1)
    return {key: whole[key] for key in (("loss", "logp", "dlogits") if case["dir"] == "both" else ("loss", "logp", "lse", "coef"))}


def exact(case, seed):
    s = prepare(case, seed)
    return {"experts": exact_experts, "clip": exact_clip, "policy": exact_policy}[case["op"]](case, s)
