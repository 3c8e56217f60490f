"""Cases, inputs, plain forms and 64-bit values of the operators on a row's log-probabilities.

Two operators stand next to the cross-entropy pass and read the same logits:

  logprobs / logprobs_grad   log-probabilities of given tokens, the entropy, and the most likely
                             tokens with theirs; the gradient through the log-probabilities and
                             the entropy (what a policy is trained by)
  distill / distill_eval / distill_grad
                             the divergence from a teacher that is known by its top logits: loss
                             and gradient in one pass, the loss alone, the gradient from saved
                             statistics

``own`` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and
the package's operators.  A case's ``op`` names the operator and its direction.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100
NEG = float("-inf")


def listed():
    return [
        # one decoding step of 4 sequences, 5 alternatives shown beside each token: latency
        {"name": "logprobs_decode", "op": "logprobs", "N": 4, "V": 32000, "dtype": "f32", "given": 1, "top": 5,
         "entropy": False, "masked": False, "pad": 0, "ignored": 0.0},
        # one decoding step of a large batch, three rows of four under a grammar, the last with nothing allowed
        {"name": "logprobs_batch", "op": "logprobs", "N": 256, "V": 128000, "dtype": "bf16", "given": 1, "top": 20,
         "entropy": True, "masked": True, "pad": 0, "ignored": 0.0},
        # a prompt scored: every position's own token and the likeliest; an odd vocabulary in padded rows
        {"name": "logprobs_prompt", "op": "logprobs", "N": 4096, "V": 50257, "dtype": "bf16", "given": 1, "top": 1,
         "entropy": False, "masked": False, "pad": 64, "ignored": 0.0},
        # a teacher's top logits stored for a batch of a student
        {"name": "logprobs_teacher", "op": "logprobs", "N": 4096, "V": 128000, "dtype": "bf16", "given": 0, "top": 64,
         "entropy": False, "masked": False, "pad": 0, "ignored": 0.0},
        # a policy's sampled tokens and its entropy, a tenth of the positions padding
        {"name": "logprobs_policy", "op": "logprobs", "N": 16384, "V": 32000, "dtype": "bf16", "given": 1, "top": 0,
         "entropy": True, "masked": False, "pad": 0, "ignored": 0.1},
        # the policy's gradient, entropy bonus included
        {"name": "logprobs_grad", "op": "logprobs_grad", "N": 4096, "V": 128000, "dtype": "bf16", "given": 1,
         "entropy": True, "masked": False, "pad": 0, "ignored": 0.1},
        # few rows of an odd vocabulary, eight labels scored in each
        {"name": "logprobs_grad_odd", "op": "logprobs_grad", "N": 513, "V": 50257, "dtype": "f16", "given": 8,
         "entropy": False, "masked": False, "pad": 0, "ignored": 0.0},
        # a student's training step against 64 stored logits a position, a tenth of them padding
        {"name": "distill_step", "op": "distill", "N": 4096, "V": 128000, "dtype": "bf16", "K": 64, "tau": 2.0,
         "normalize": True, "reduce": True, "pad": 0, "ignored": 0.1},
        # a handful of positions in float32: latency
        {"name": "distill_small", "op": "distill", "N": 16, "V": 32000, "dtype": "f32", "K": 20, "tau": 1.0,
         "normalize": True, "reduce": True, "pad": 0, "ignored": 0.0},
        # an odd number of rows of an odd vocabulary, the teacher's log-probabilities taken as they are
        {"name": "distill_odd", "op": "distill", "N": 1023, "V": 50257, "dtype": "f16", "K": 100, "tau": 1.0,
         "normalize": False, "reduce": False, "pad": 0, "ignored": 0.1},
        # the loss alone on held-out text
        {"name": "distill_eval", "op": "distill_eval", "N": 2048, "V": 100277, "dtype": "bf16", "K": 256, "tau": 1.0,
         "normalize": True, "reduce": False, "pad": 0, "ignored": 0.0},
        # the gradient alone, for a loss that is weighted after it is known
        {"name": "distill_grad", "op": "distill_grad", "N": 2048, "V": 65536, "dtype": "bf16", "K": 128, "tau": 2.0,
         "normalize": True, "reduce": False, "pad": 0, "ignored": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs", "logprobs_grad", "distill", "distill", "distill_eval",
                     "distill_grad"])
    V = rng.choice([4096, 8192, 32000, 50257, 65536, 100277, 128000, 151937, 256000, _log(rng, 300, 200000)])
    case = {"op": op, "N": _log(rng, 1, min(8192, 2 ** 27 // V)), "V": V,
            "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "pad": rng.choice([0, 0, 64]),
            "ignored": rng.choice([0.0, 0.1])}
    if op.startswith("logprobs"):
        case["given"] = rng.choice([1, 1, 1, _log(rng, 2, 32)])
        case["masked"] = rng.random() < 0.3
        case["entropy"] = rng.random() < 0.5
        if op == "logprobs":
            case["top"] = rng.choice([0, 1, 5, 20, _log(rng, 2, 256)])
            if rng.random() < 0.2:
                case["given"] = 0
                case["top"] = case["top"] or 20
        return case
    case["K"] = rng.choice([20, 64, 100, _log(rng, 1, min(1024, V))])
    case["normalize"] = rng.random() < 0.7
    case["tau"] = rng.choice([1.0, 2.0, round(rng.uniform(0.5, 5.0), 2)]) if case["normalize"] else 1.0
    case["reduce"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------------------ inputs
def _rows(t, step):
    for k in range(0, t.shape[0], step):
        yield slice(k, k + step)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N, V, op = case["N"], case["V"], case["op"]
    wide = -(-V // case["pad"]) * case["pad"] if case["pad"] else V
    s = {"case": case}

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    # a broad floor of logits and some likely tokens above it: a model is sure of a few
    x = torch.empty(N, wide, dtype=dt, device="cuda").normal_(0.0, 2.5, generator=gen)[:, :V]
    P = max(case.get("K", 0), case.get("given", 0), 16)  # distinct places in each row
    places = (torch.randint(0, V, (N, 1), generator=gen, device="cuda") + torch.arange(P, device="cuda") * (V // P)) % V
    likely = places[:, :16]
    lift = 6 + 8 * rand(N, 1) - 0.7 * torch.arange(16, device="cuda") + rand(N, 16)
    x.scatter_add_(1, likely, lift.to(dt))
    s["logits"] = x
    dropped = rand(N) < case["ignored"]
    if N > 1:
        dropped[0] = False  # a batch has a row that counts
    else:
        dropped[:] = False
    if op.startswith("logprobs"):
        if case["masked"]:
            # a grammar allows one token of 64 and the likeliest; nothing in the last row of more than two
            under = torch.arange(N, device="cuda") % 4 != 0
            for r in _rows(x, 1024):
                n = x[r].shape[0]
                blocked = (torch.rand(n, V, generator=gen, device="cuda") > 1 / 64) & under[r][:, None]
                blocked.scatter_(1, likely[r, :4], False)
                x[r].masked_fill_(blocked, NEG)
            if N > 2:
                x[N - 1] = NEG
        G = case["given"]
        s["tokens"] = None
        if G:
            tokens = places[:, :G].clone()
            far = rand(N, G) < 0.3
            tokens[far] = torch.randint(0, V, (N, G), generator=gen, device="cuda")[far]
            tokens[dropped] = IGNORE
            s["tokens"] = tokens[:, 0].contiguous() if G == 1 else tokens
        if op == "logprobs_grad":
            s["grad_logprobs"] = torch.empty(s["tokens"].shape, device="cuda").normal_(generator=gen)
            s["grad_entropy"] = 0.01 * (1 + rand(N)) if case["entropy"] else None
            s["stats"] = _stats(x, 1.0)  # what the forward pass has left
        return s
    K = case["K"]
    z = 14 - 9 * torch.log1p(torch.arange(K, device="cuda")) / math.log(K + 1) + 1.5 * rand(N, K)
    z = z.sort(dim=1, descending=True).values
    if not case["normalize"]:
        z = z - torch.log(torch.exp(z).sum(1, keepdim=True) * (1.05 + 0.3 * rand(N, 1)))  # some of it on other tokens
    tokens = places[:, :K].clone()
    short = torch.arange(N, device="cuda") % 8 == 5  # rows with half as many
    tokens[:, (K + 1) // 2:].masked_fill_(short[:, None], IGNORE)
    tokens[dropped] = IGNORE
    s["tokens"], s["teacher"] = tokens, z.contiguous()
    s["dloss"] = rand(N) + 0.5 if not case["reduce"] else None
    s["count"] = (tokens[:, 0] != IGNORE).sum().reshape(1)
    if op == "distill":
        s["grad"] = torch.empty_like(x)
    if op == "distill_grad":
        m, logd, _, _ = _stats(x, 1 / case["tau"]).unbind(1)
        zz = z.masked_fill(tokens == IGNORE, NEG)
        top = zz.amax(1)
        logq = torch.log(torch.exp((zz - top[:, None]) / case["tau"]).sum(1))
        empty = tokens[:, 0] == IGNORE
        s["stats"] = torch.stack([m, logd, top.masked_fill(empty, NEG), logq.masked_fill(empty, 0.0)], 1)
    return s


def _stats(x, scale):
    """(max, log of the summed exp(scale (x - max)), entropy, 0) of each row in float32; -inf first where a row has
    nothing."""
    out = torch.zeros(x.shape[0], 4, device="cuda")
    for r in _rows(x, max(1, 2 ** 26 // x.shape[1])):
        d = x[r].double()
        m = d.amax(1, keepdim=True)
        y = scale * (d - m)
        e = torch.exp(y)
        total = e.sum(1)
        out[r, 0], out[r, 1] = m[:, 0].float(), torch.log(total).float()
        out[r, 2] = (torch.log(total) - (e * y.clamp(min=-1e4)).sum(1) / total).float()
    out[out[:, 0] == NEG, 1:] = 0.0
    return out


# -------------------------------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import vocabulary_cross_entropy_pass_gb300 as ce
    case = s["case"]
    op = case["op"]
    if op == "logprobs":
        lp, ent, top, top_lp, _ = ce.ce_logprobs_fwd(s["logits"], s["tokens"], top_k=case["top"],
                                                     entropy=case["entropy"])
        return {"logprobs": lp, "entropy": ent, "top": top, "top_logprobs": top_lp}
    if op == "logprobs_grad":
        return ce.ce_logprobs_bwd(s["logits"], s["stats"], s["tokens"], grad_logprobs=s["grad_logprobs"],
                                  grad_entropy=s["grad_entropy"])
    how = {"temperature": case["tau"], "normalize": case["normalize"]}
    if op == "distill":
        loss, grad = ce.ce_distill_fwd_bwd(s["logits"], s["tokens"], s["teacher"], reduce_loss=case["reduce"],
                                           dloss=s["dloss"], grad=s["grad"], **how)
        return {"loss": loss, "grad": grad}
    if op == "distill_eval":
        return ce.ce_distill_fwd(s["logits"], s["tokens"], s["teacher"], reduce_loss=case["reduce"], **how)[0]
    return ce.ce_distill_bwd(s["logits"], s["tokens"], s["teacher"], s["stats"], reduce_loss=case["reduce"],
                             dloss=s["dloss"], n_non_ignore=s["count"], **how)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op.startswith("logprobs"):
        x = s["logits"].float()
        N, V = x.shape
        t = None if s["tokens"] is None else s["tokens"].view(N, -1)
        skip = torch.zeros(N, dtype=torch.bool, device="cuda") if t is None else (t == IGNORE).all(1)
        if op == "logprobs_grad":
            lp = x - s["stats"][:, :1] - s["stats"][:, 1:2]
            p = torch.exp(lp)
            gl = s["grad_logprobs"].view(N, -1).masked_fill(t == IGNORE, 0.0)
            g = -p * gl.sum(1, keepdim=True)
            if s["grad_entropy"] is not None:
                g = g - s["grad_entropy"][:, None] * p * (lp.clamp(min=-1e4) + s["stats"][:, 2:3])
            g.masked_fill_((skip | (s["stats"][:, 0] == NEG))[:, None], 0.0)
            rows = torch.arange(N, device="cuda")[:, None].expand_as(t)
            gl = gl.masked_fill((skip | (s["stats"][:, 0] == NEG))[:, None], 0.0)
            g.index_put_((rows, t.clamp(min=0)), gl, accumulate=True)
            return g.to(dt)
        m = x.amax(1, keepdim=True)
        none = m == NEG  # nothing is allowed: every log-probability is -inf
        y = x - m.masked_fill(none, 0.0)
        e = torch.exp(y)
        d = e.sum(1, keepdim=True)
        logd = torch.log(d).masked_fill(none, 0.0)
        out = {"logprobs": None, "entropy": None, "top": None, "top_logprobs": None}
        if t is not None:
            lp = torch.gather(y, 1, t.clamp(min=0)) - logd
            out["logprobs"] = lp.masked_fill(t == IGNORE, 0.0).view(s["tokens"].shape)
        if case["entropy"]:
            ent = logd - (e * y.clamp(min=-1e4)).sum(1, keepdim=True) / d
            out["entropy"] = ent.masked_fill(none, 0.0).masked_fill(skip[:, None], 0.0)[:, 0]
        if case["top"]:
            val, idx = torch.sort(x, dim=1, descending=True, stable=True)
            val, idx = val[:, :case["top"]], idx[:, :case["top"]]
            lp = val - m.masked_fill(none, 0.0) - logd
            out["top"] = idx.masked_fill(skip[:, None], IGNORE)
            out["top_logprobs"] = lp.masked_fill(skip[:, None], 0.0)
        return out
    tau, t = case["tau"], s["tokens"]
    N = t.shape[0]
    keep = t != IGNORE
    z = (s["teacher"] / tau).masked_fill(~keep, NEG)
    logq = z
    if case["normalize"]:
        zm = z.amax(1, keepdim=True).clamp(min=-1e30)
        logq = z - zm - torch.log(torch.exp(z - zm).sum(1, keepdim=True))
    q = torch.exp(logq).masked_fill(~keep, 0.0)
    x = s["logits"].float() / tau
    m = x.amax(1, keepdim=True)
    y = x - m
    logd = torch.log(torch.exp(y).sum(1, keepdim=True))
    row = keep[:, :1]
    n = row.sum()
    out = {}
    if op != "distill_grad":
        lp = torch.gather(y, 1, t.clamp(min=0)) - logd
        terms = torch.where(keep, q * (logq - lp), 0.0)
        loss = tau * tau * terms.sum(1)
        out["loss"] = (loss.double().sum() / n).float().view(1) if case["reduce"] else loss
        if op == "distill_eval":
            return out["loss"]
    g = s["dloss"][:, None] if s["dloss"] is not None else (1.0 / n).float()
    grad = torch.exp(y - logd) * q.sum(1, keepdim=True)
    grad.masked_fill_(~row, 0.0)
    rows = torch.arange(N, device="cuda")[:, None].expand_as(t)
    grad.index_put_((rows, t.clamp(min=0)), -q, accumulate=True)
    out["grad"] = (grad * (tau * g)).to(dt)
    return out["grad"] if op == "distill_grad" else out


# ----------------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    """The definition in float64 from the inputs' own values, a few rows at a time: log_softmax in place of the
    statistics, the likeliest tokens by one integer key of value and place."""
    s = prepare(case, seed)
    x, op = s["logits"], case["op"]
    N, V = x.shape
    parts = [_exact_rows(case, s, x, r, op) for r in _rows(x, max(1, 2 ** 27 // V))]
    if isinstance(parts[0], dict):
        out = {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
    else:
        out = torch.cat(parts)
    if op.startswith("distill") and case["reduce"] and op != "distill_grad":
        n = int((s["tokens"][:, 0] != IGNORE).sum())
        if op == "distill_eval":
            return (out.sum() / n).view(1)
        out["loss"] = (out["loss"].sum() / n).view(1)
    return out


def _exact_rows(case, s, x, r, op):
    x = x[r].double()
    n, V = x.shape
    at = torch.arange(n, device="cuda")[:, None]
    if op.startswith("logprobs"):
        t = s["tokens"]
        t = None if t is None else t[r].view(n, -1)
        skip = None if t is None else (t == IGNORE).sum(1) == t.shape[1]
        none = torch.isneginf(x).sum(1) == V
        lp = torch.log_softmax(x, 1)
        lp[none] = NEG
        p = torch.exp(lp)
        surprise = torch.where(p > 0, -lp, torch.zeros_like(lp))
        ent = torch.einsum("nv,nv->n", p, surprise)
        if op == "logprobs_grad":
            gl = s["grad_logprobs"][r].view(n, -1).double()
            gl = torch.where((t == IGNORE) | none[:, None] | skip[:, None], 0.0, gl)
            g = -p * gl.sum(1)[:, None]
            if s["grad_entropy"] is not None:
                ge = torch.where(skip, 0.0, s["grad_entropy"][r].double())
                g += ge[:, None] * p * (surprise - ent[:, None])
            for k in range(t.shape[1]):
                g[at[:, 0], t[:, k].clamp(min=0)] += gl[:, k]
            return g
        out = {"logprobs": None, "entropy": None, "top": None, "top_logprobs": None}
        if t is not None:
            got = torch.where(t == IGNORE, 0.0, lp[at, t.clamp(min=0)])
            out["logprobs"] = got.view((n,) + s["tokens"].shape[1:])
        if case["entropy"]:
            out["entropy"] = ent if skip is None else torch.where(skip, 0.0, ent)
        if case["top"]:
            bits = (s["logits"][r].float() + 0.0).view(torch.int32).long()
            order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)  # grows with the value
            key = order * V + (V - 1 - torch.arange(V, device="cuda"))
            idx = V - 1 - torch.topk(key, case["top"], dim=1, sorted=True).values % V
            out["top"] = idx if skip is None else torch.where(skip[:, None], IGNORE, idx)
            got = lp[at, idx]
            out["top_logprobs"] = got if skip is None else torch.where(skip[:, None], 0.0, got)
        return out
    tau, t = case["tau"], s["tokens"][r]
    z = s["teacher"][r].double() / tau
    keep = t != IGNORE
    logq = z - torch.logsumexp(torch.where(keep, z, NEG), 1, keepdim=True) if case["normalize"] else z
    q = torch.where(keep, torch.exp(logq), 0.0)
    lp = torch.log_softmax(x / tau, 1)
    loss = tau ** 2 * torch.where(keep, q * (logq - lp[at, t.clamp(min=0)]), 0.0).sum(1)
    if op == "distill_eval":
        return loss
    if s["dloss"] is not None:
        g = s["dloss"][r].double()
    else:
        g = torch.full((n,), 1.0, dtype=torch.float64, device="cuda") / int((s["tokens"][:, 0] != IGNORE).sum())
    grad = torch.exp(lp) * q.sum(1, keepdim=True)
    hit = torch.zeros_like(grad).scatter_add_(1, t.clamp(min=0), q)
    grad = (grad - hit) * (g * tau)[:, None]
    return grad if op == "distill_grad" else {"loss": loss, "grad": grad}


# -------------------------------------------------------------------------------------------- work
def work(case):
    op, N, V, e = case["op"], case["N"], case["V"], BYTES[case["dtype"]]
    read = N * (1 - case["ignored"]) * V * e  # a padded row's logits need not be read
    if op.startswith("logprobs"):
        G = case["given"]
        if op == "logprobs":
            return {"bytes": read + N * (12 * G + 12 * case["top"] + 4 * case["entropy"]), "flops": 6 * N * V}
        return {"bytes": read + N * V * e + N * (12 * G + 16 + 4 * case["entropy"]), "flops": 6 * N * V}
    lists = N * case["K"] * 12
    if op == "distill_eval":
        return {"bytes": read + lists + 4 * N, "flops": 4 * N * V}
    return {"bytes": read + N * V * e + lists + 4 * N, "flops": 6 * N * V}
