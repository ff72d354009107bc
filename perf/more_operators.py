"""Cases that measure two more training-step operators: token log-probabilities and orthogonalised updates.

With ``own`` false ``run`` computes a case in elementary torch operations, in 32 bits whatever the inputs' type and
rounded once at the end; with ``own`` true it makes the calls of ``conv2d_backward_implicit_bwd_gb300.train``.

The operators, on row-major tensors:

logp      lse_t = log sum_v exp(s z_tv); logp_t = s z_t[a_t] - lse_t; H_t = -sum_v p_tv (s z_tv - lse_t) with
          p_tv = exp(s z_tv - lse_t); the `top` largest logits of a row in falling order (ties: the lowest index), as
          log-probabilities and indices.  Rows with a negative token are masked: zeros, and -1 for their indices.
          Backward, from gradients gl of logp and ge of H: dz_tv = s (gl_t ([v = a_t] - p_tv) - ge_t p_tv (s z_tv - lse_t + H_t)).
orth      X = u / |u| (Frobenius norm, each matrix of a batch), then `steps` times X <- a X + b (X X^T) X + c (X X^T)^2 X.
          apply: u is the given matrix.  update: m <- beta m + g, u = g + beta m, w <- (1 - lr decay) w - lr sqrt(max(1, rows / cols)) X,
          and a 16-bit copy of w.
"""
import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SCALE = 0.8
STEPS, COEF = 5, (3.4445, -4.7750, 2.0315)
LR, BETA, DECAY = 0.02, 0.95, 0.1


def listed():
    logp = dict(op="logp", dtype="bf16", top=0, banned=0.0)
    orth = dict(op="orth", dtype="bf16")
    return [
        # serving, one token: what a sampler reports with it, twenty alternatives over a wide vocabulary; latency
        dict(logp, name="logp one token top 20", dir="forward", rows=1, vocab=128000, top=20),
        # serving, a decode batch with a few alternatives each, part of the vocabulary ruled out by a grammar
        dict(logp, name="logp decode top 5", dir="forward", rows=64, vocab=128000, top=5, banned=0.3),
        # training, old or reference log-probabilities of sampled sequences, and their entropy
        dict(logp, name="logp sequences", dir="forward", rows=8192, vocab=32768),
        # scoring a text of odd length with alternatives, an odd vocabulary in 32 bits
        dict(logp, name="logp odd f32 top 8", dir="forward", dtype="f32", rows=1021, vocab=50257, top=8),
        # training, gradients of log-probability and entropy
        dict(logp, name="logp grad", dir="backward", rows=8192, vocab=32768),
        # the same of a small vocabulary of odd width in 32 bits: a router's or a small policy's actions
        dict(logp, name="logp grad narrow f32", dir="backward", dtype="f32", rows=5000, vocab=1009),
        # the update of a small layer of odd widths: latency
        dict(orth, name="orth update small odd", dir="update", dtype="f32", batch=1, rows=100, cols=131),
        # a single square matrix
        dict(orth, name="orth apply square", dir="apply", batch=1, rows=1000, cols=1000),
        # two wide matrices with 32-bit gradients: down-projections of dense layers
        dict(orth, name="orth update wide f32", dir="update", dtype="f32", batch=2, rows=1024, cols=4096),
        # the experts' up-projections, high matrices, as an update of 32-bit masters from 16-bit gradients
        dict(orth, name="orth update experts", dir="update", batch=16, rows=2048, cols=1024),
        # the experts' down-projections, the matrices alone
        dict(orth, name="orth apply experts", dir="apply", batch=32, rows=1024, cols=2048),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.5:
        vocab = log(2, 131072)
        way, dtype = rng.choice(("forward", "forward", "backward")), rng.choice(("f32", "bf16"))
        top = min(vocab, rng.choice((0, 1, 5, 20, 32))) if way == "forward" else 0
        return dict(op="logp", dir=way, dtype=dtype, rows=log(1, max(2, min(8192, (1 << 27) // vocab))), vocab=vocab, top=top, banned=rng.choice((0.0, 0.0, 0.3)))
    rows, cols = log(8, 2048), log(8, 4096)
    lo, hi = min(rows, cols), max(rows, cols)
    batch = log(1, max(1, min(64, (1 << 35) // (lo * lo * hi))))
    return dict(op="orth", dir=rng.choice(("apply", "update")), dtype="bf16", batch=batch, rows=rows, cols=cols) if rng.random() < 0.6 else \
        dict(op="orth", dir="update", dtype="f32", batch=batch, rows=rows, cols=cols)


# ---- inputs ----------------------------------------------------------------
def normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare_logp(case, gen):
    t, v, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    logits = torch.empty((t, v), dtype=dt, device="cuda")
    tokens = torch.randint(0, v, (t,), generator=gen, device="cuda", dtype=torch.int32)
    for at in range(0, t, max(1, (1 << 27) // v)):
        part = logits[at:at + max(1, (1 << 27) // v)]
        part.copy_(normal(gen, part.shape, dt, 2.5))
        if case["banned"]:
            part.masked_fill_(torch.rand(part.shape, generator=gen, device="cuda") < case["banned"], -math.inf)
    logits.scatter_(1, tokens[:, None].long(), normal(gen, (t, 1), dt, 2.5) + 4.0)  # a sampled token is a likely one
    tokens[5::16] = -1  # padding of the sequences
    s = dict(logits=logits, tokens=tokens)
    if case["dir"] == "backward":
        lse, entropy = [], []
        for z in logits.split(max(1, (1 << 26) // v)):
            z = z.float() * SCALE
            lse.append(torch.logsumexp(z, 1))
            z -= lse[-1][:, None]
            entropy.append(-torch.where(z > -math.inf, torch.exp(z) * z, 0.0).sum(1))
        kept = tokens >= 0
        s.update(lse=torch.cat(lse) * kept, entropy=torch.cat(entropy) * kept,
                 gl=normal(gen, (t,), torch.float32, 1.0 / t), ge=normal(gen, (t,), torch.float32, 0.1 / t))
    return s


def gradient(case, gen):
    """Matrices as gradients are: a few directions of falling weight over noise."""
    b, m, n = case["batch"], case["rows"], case["cols"]
    r = min(32, m, n)
    fall = torch.exp(-0.15 * torch.arange(r, device="cuda"))
    g = torch.bmm(normal(gen, (b, m, r), torch.float32) * fall, normal(gen, (b, r, n), torch.float32))
    return g.add_(normal(gen, (b, m, n), torch.float32), alpha=0.2).mul_(1e-3)


def prepare_orth(case, gen):
    s = dict(grad=gradient(case, gen).to(DTYPES[case["dtype"]]))
    if case["dir"] == "update":
        s["momentum"] = gradient(case, gen) * 5.0
        s["weight"] = normal(gen, s["momentum"].shape, torch.float32, 1.0 / math.sqrt(case["cols"]))
        s["copy"] = s["weight"].bfloat16()
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return dict({"logp": prepare_logp, "orth": prepare_orth}[case["op"]](case, gen), case=case)


# ---- the framework's calls -------------------------------------------------
@functools.lru_cache(maxsize=None)
def logp_plan(vocab, dtype, top):
    from conv2d_backward_implicit_bwd_gb300 import train
    return train.TokenLogp(vocab, dtype, top=top, scale=SCALE)


@functools.lru_cache(maxsize=2)
def orth_plan(batch, rows, cols, dtype):
    from conv2d_backward_implicit_bwd_gb300 import train
    return train.Orthogonal(batch, rows, cols, dtype, steps=STEPS, coefficients=COEF)


def run_own(state, case):
    if case["op"] == "logp":
        plan = logp_plan(case["vocab"], case["dtype"], case["top"])
        if case["dir"] == "backward":
            return plan.backward(state["logits"], state["tokens"], state["lse"], state["entropy"], grad_logp=state["gl"], grad_entropy=state["ge"])
        logp, entropy, lse, top_logp, top_tokens = plan.forward(state["logits"], state["tokens"])
        return dict(logp=logp, entropy=entropy, lse=lse, top_logp=top_logp, top_tokens=top_tokens)
    plan = orth_plan(case["batch"], case["rows"], case["cols"], case["dtype"])
    if case["dir"] == "apply":
        return plan.apply(state["grad"])
    plan.update(state["weight"], state["grad"], state["momentum"], LR, beta=BETA, decay=DECAY, copy=state["copy"])
    return dict(weight=state["weight"], momentum=state["momentum"], copy=state["copy"])


# ---- the plain forms -------------------------------------------------------
def largest(z, count):
    """Indices of each row's largest values, ties by the lowest index: a key of the value's order and the index."""
    bits = (z.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits - 1, bits)  # rises with the value
    index = torch.arange(z.shape[1], device="cuda")
    return (order * (1 << 32) + (0xffffffff - index)).topk(count, dim=1).indices


def plain_logp(state, case):
    logits, tokens = state["logits"], state["tokens"]
    kept = tokens >= 0
    at = tokens.clamp(min=0).long()[:, None]
    z = logits.float() * SCALE
    if case["dir"] == "backward":
        u = z - state["lse"][:, None]
        p = torch.exp(u)
        gl, ge = state["gl"] * kept, state["ge"] * kept
        d = -p * (gl[:, None] + ge[:, None] * (u.clamp(min=-1e4) + state["entropy"][:, None]))
        d.scatter_add_(1, at, gl[:, None])
        return torch.where(kept[:, None], d * SCALE, 0.0).to(logits.dtype)
    top = z.amax(1, keepdim=True)
    u = z - top
    e = torch.exp(u)
    total = e.sum(1, keepdim=True)
    logs = torch.log(total)
    entropy = logs[:, 0] - (e * u.clamp(min=-1e4)).sum(1) / total[:, 0]
    lse = (top + logs)[:, 0]
    logp = u.gather(1, at)[:, 0] - logs[:, 0]
    out = dict(logp=torch.where(kept, logp, 0.0), entropy=torch.where(kept, entropy, 0.0), lse=torch.where(kept, lse, 0.0), top_logp=None, top_tokens=None)
    if case["top"]:
        best = largest(logits, case["top"])
        out["top_logp"] = torch.where(kept[:, None], u.gather(1, best) - logs, 0.0)
        out["top_tokens"] = torch.where(kept[:, None], best, -1).int()
    return out


def newton_schulz(u):
    a, b, c = COEF
    x = u / u.square().sum((1, 2), keepdim=True).sqrt()
    high = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if high else x
    for _ in range(STEPS):
        s = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return x.transpose(1, 2) if high else x


def plain_orth(state, case):
    g = state["grad"].float()
    if case["dir"] == "apply":
        return newton_schulz(g).to(state["grad"].dtype).contiguous()
    m, w = state["momentum"], state["weight"]
    m.mul_(BETA).add_(g)
    o = newton_schulz(g + BETA * m)
    w.mul_(1 - LR * DECAY).sub_(o, alpha=LR * math.sqrt(max(1.0, case["rows"] / case["cols"])))
    state["copy"].copy_(w)
    return dict(weight=w, momentum=m, copy=state["copy"])


def run(state):
    case = state["case"]
    if own:
        return run_own(state, case)
    return plain_logp(state, case) if case["op"] == "logp" else plain_orth(state, case)


# ---- what a pass cannot do without -----------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2}[case["dtype"]]
    if case["op"] == "logp":
        t, v = case["rows"], case["vocab"]
        kept = t - len(range(5, t, 16))
        if case["dir"] == "forward":
            return dict(bytes=size * kept * v + 4 * t + (12 + 8 * case["top"]) * t, flops=6 * kept * v)
        return dict(bytes=size * (kept + t) * v + 20 * t, flops=9 * kept * v)
    b, lo, hi = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # both symmetric products count once for each pair of elements
    flops = float(STEPS * b * (lo * (lo + 1) * hi + lo * (lo + 1) * lo + 2 * lo * lo * hi))
    return dict(bytes=b * lo * hi * (2 * size if case["dir"] == "apply" else size + 18), flops=flops)


# ---- the definition in 64 bits ---------------------------------------------
def exact_logp(case, s):
    parts = []
    for rows in torch.arange(case["rows"]).split(max(1, (1 << 25) // case["vocab"])):
        z = s["logits"][rows[0]:rows[-1] + 1].double()
        token = s["tokens"][rows[0]:rows[-1] + 1].long()
        live = (token >= 0).double()
        pick = torch.zeros_like(z)
        pick[torch.arange(len(token), device="cuda"), token.clamp(min=0)] = 1.0
        if case["dir"] == "backward":
            lse, ent = (s[k][rows[0]:rows[-1] + 1].double()[:, None] for k in ("lse", "entropy"))
            gl, ge = ((s[k][rows[0]:rows[-1] + 1].double() * live)[:, None] for k in ("gl", "ge"))
            p = torch.exp(SCALE * z - lse) * live[:, None]
            plogp = torch.special.xlogy(p, p)  # p log p, 0 where p is 0
            parts.append(dict(d=SCALE * (gl * (pick - p) - ge * (plogp + p * ent))))
            continue
        lp = torch.log_softmax(SCALE * z, 1)
        p = lp.exp()
        part = dict(logp=torch.nan_to_num(lp, neginf=0.0).mul(pick).sum(1) * live, entropy=-torch.special.xlogy(p, p).sum(1) * live,
                    lse=torch.logsumexp(SCALE * z, 1) * live)
        if case["top"]:
            order = z.sort(dim=1, descending=True, stable=True).indices[:, :case["top"]]
            part["top_logp"] = torch.where(live[:, None] > 0, lp.gather(1, order), 0.0)
        parts.append(part)
    whole = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["dir"] == "backward":
        return whole["d"]
    return dict(whole, top_logp=whole.get("top_logp"), top_tokens=None)


def exact_orth(case, s):
    a, b, c = COEF
    g = s["grad"].double()
    momentum = None
    if case["dir"] == "update":
        momentum = BETA * s["momentum"].double() + g
        g = g + BETA * momentum
    found = []
    for x in g:  # polynomial of the smaller side's Gram matrix
        x = x / torch.linalg.matrix_norm(x)
        eye = torch.eye(min(x.shape), dtype=torch.float64, device="cuda")
        for _ in range(STEPS):
            if x.shape[0] > x.shape[1]:
                q = x.T @ x
                x = x @ (a * eye + q @ (b * eye + c * q))
            else:
                q = x @ x.T
                x = (a * eye + q @ (b * eye + c * q)) @ x
        found.append(x)
    x = torch.stack(found)
    if momentum is None:
        return x
    w = s["weight"].double() * (1.0 - LR * DECAY) - LR * math.sqrt(max(1.0, case["rows"] / case["cols"])) * x
    return dict(weight=w, momentum=momentum, copy=w)


def exact(case, seed):
    s = prepare(case, seed)
    return exact_logp(case, s) if case["op"] == "logp" else exact_orth(case, s)
