"""Cases, inputs, plain forms and 64-bit values of the operators at the two ends of the vocabulary.

Three operators sit around the cross-entropy pass and are measured here:

  embed / embed_grad    rows of the (V, H) vocabulary matrix by token, times a scale; the gradient
                        summed over equal tokens, written whole or added to the float32 gradient
                        that the lm_head step of a tied matrix has already filled
  norm / norm_grad      the residual's addition and the root-mean-square norm in front of the
                        lm_head, in the input's type or in 8 bits with scales; its gradients
  logits / logits_grad  repetition, frequency and presence penalties, sparse biases, a grammar's
                        bit mask and the temperature on the logits; the gradient through them

``own`` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and
the package's operators.  A case's ``op`` names the operator and its direction.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
EPS = 1e-6
TINY = 2.0 ** -126  # the least scale of 8-bit values
NEG = float("-inf")


def listed():
    return [
        # one decoding step of a batch of 16 sequences: latency
        {"name": "embed_decode", "op": "embed", "N": 16, "V": 32000, "H": 4096, "dtype": "bf16", "scale": 1.0},
        # a training batch of 8 sequences of 4096 tokens, rows scaled by sqrt(H)
        {"name": "embed_batch", "op": "embed", "N": 32768, "V": 128000, "H": 4096, "dtype": "bf16", "scale": 64.0},
        # a short fine-tuning step with an odd width, whole float32 gradient
        {"name": "embed_grad_odd", "op": "embed_grad", "N": 1023, "V": 8192, "H": 1001, "dtype": "f32", "scale": 1.0,
         "tied": False},
        # the gradient of a training batch added to a tied matrix's float32 gradient
        {"name": "embed_grad_tied", "op": "embed_grad", "N": 16384, "V": 128000, "H": 4096, "dtype": "bf16",
         "scale": 64.0, "tied": True},
        # the last norm of one decoding step of 8 sequences: latency
        {"name": "norm_decode", "op": "norm", "N": 8, "H": 4096, "dtype": "bf16", "residual": True},
        # the last norm of a training batch of 4 sequences of 4096 tokens
        {"name": "norm_batch", "op": "norm", "N": 16384, "H": 4096, "dtype": "bf16", "residual": True},
        # a prompt's norm in front of a product in 8 bits, one scale for 128 columns
        {"name": "norm_fp8", "op": "norm", "N": 8192, "H": 8192, "dtype": "bf16", "residual": True, "fp8": "e4m3",
         "group": 128},
        # the norm's gradients of the training batch
        {"name": "norm_grad", "op": "norm_grad", "N": 16384, "H": 4096, "dtype": "bf16", "residual": True},
        # the same for an odd number of rows of an odd width, no residual stream
        {"name": "norm_grad_odd", "op": "norm_grad", "N": 2049, "H": 5001, "dtype": "f16", "residual": False},
        # one decoding step of 4 sequences of about a thousand tokens: latency
        {"name": "logits_decode", "op": "logits", "N": 4, "V": 32000, "dtype": "f32", "hist": 1000, "bias": 16,
         "mask": False, "pad": 0},
        # one decoding step of a large batch, three rows of four under a grammar
        {"name": "logits_batch", "op": "logits", "N": 512, "V": 128000, "dtype": "bf16", "hist": 4096, "bias": 64,
         "mask": True, "pad": 0},
        # the gradient of 4096 sampled positions through the penalties and the mask they were sampled
        # under; an odd vocabulary in rows padded to 64 columns
        {"name": "logits_grad", "op": "logits_grad", "N": 4096, "V": 50257, "dtype": "bf16", "hist": 256, "bias": 0,
         "mask": True, "pad": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm", "norm_grad", "logits", "logits_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("embed"):
        V = rng.choice([4096, 8192, 32000, 50257, 65536, 100277, 128000])
        H = rng.choice([512, 1024, 2048, 4096, 5120, 8192, _log(rng, 65, 5000)])
        N = _log(rng, 1, min(32768, 2 ** 27 // (H * BYTES[dtype])))
        case = {"op": op, "N": N, "V": V, "H": H, "dtype": dtype, "scale": rng.choice([1.0, math.sqrt(H)])}
        if op == "embed_grad":
            case["tied"] = V * H > 2 ** 26 or rng.random() < 0.3  # a whole gradient of at most 256 MB
        return case
    if op.startswith("norm"):
        H = rng.choice([1024, 2048, 4096, 5120, 8192, 16384, 8 * _log(rng, 16, 1500), _log(rng, 65, 9000)])
        N = _log(rng, 1, min(32768, 2 ** 27 // (H * BYTES[dtype])))
        case = {"op": op, "N": N, "H": H, "dtype": dtype, "residual": rng.random() < 0.7}
        if op == "norm" and rng.random() < 0.4:
            case["fp8"] = rng.choice(["e4m3", "e4m3", "e5m2"])
            case["group"] = rng.choice([0, 32, 64, 128])
        return case
    V = rng.choice([4096, 8192, 32000, 50257, 65536, 100277, 128000, 256000])
    N = _log(rng, 1, min(4096, 2 ** 26 // V))
    return {"op": op, "N": N, "V": V, "dtype": dtype, "hist": rng.choice([0, _log(rng, 16, 8192)]),
            "bias": rng.choice([0, 32, 300]), "mask": rng.random() < 0.6, "pad": rng.choice([0, 64])}


# ------------------------------------------------------------------------------------------ inputs
def _zipf(gen, shape, V):
    """Tokens whose k-th has a probability of about 1/k, as words have; the ids shuffled over the vocabulary."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    k = torch.exp(u * math.log(V + 1)).to(torch.int64).clamp_(1, V) - 1
    return (k * 7919 + 11) % V  # a prime that divides no V here: every id is met


def _normal(gen, shape, dtype, sigma=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, sigma, generator=gen)


def _fraction(gen, n, lo, hi):
    return torch.rand(n, generator=gen, device="cuda") * (hi - lo) + lo


def _mask(gen, N, V):
    """Bits of allowed tokens: row 0, 4, 8, ... free; the others one token of 64; the last row (of more than two) none."""
    W = (V + 31) // 32
    bits = torch.full((N, W), -1, dtype=torch.int32, device="cuda")
    full = torch.randint(-2 ** 31, 2 ** 31, (6, N, W), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    few = full[0] & full[1] & full[2] & full[3] & full[4] & full[5]
    under = torch.arange(N, device="cuda") % 4 != 0
    bits[under] = few[under]
    if N > 2:
        bits[N - 1] = 0
    return bits


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N = case["N"]
    s = {"case": case}
    if case["op"].startswith("embed"):
        V, H = case["V"], case["H"]
        s["tokens"] = _zipf(gen, (N,), V)
        if case["op"] == "embed":
            s["weight"] = _normal(gen, (V, H), dt, 0.02)
        else:
            s["grad_out"] = _normal(gen, (N, H), dt, 1e-2)
            if case["tied"]:
                s["grad"] = _normal(gen, (V, H), torch.float32, 1e-2)
        return s
    if case["op"].startswith("norm"):
        H = case["H"]
        s["weight"] = 1 + _normal(gen, (H,), torch.float32, 0.1)
        s["weight"] = s["weight"].to(dt)
        if case["op"] == "norm":
            s["x"] = _normal(gen, (N, H), dt)
            s["residual"] = _normal(gen, (N, H), dt, 3.0) if case["residual"] else None
        else:
            s["h"] = _normal(gen, (N, H), dt, 3.0)
            s["grad_out"] = _normal(gen, (N, H), dt)
            s["grad_h"] = _normal(gen, (N, H), dt) if case["residual"] else None
        return s
    V = case["V"]
    wide = -(-V // case["pad"]) * case["pad"] if case["pad"] else V
    s["logits"] = _normal(gen, (N, wide), dt, 3.0)[:, :V]
    if case["op"] == "logits_grad":
        s["grad_out"] = _normal(gen, (N, wide), dt, 1e-2)[:, :V]
    L = case["hist"]
    if L:
        s["history"] = _zipf(gen, (N, L), V)
        s["history_lengths"] = torch.randint(L // 2, L + 1, (N,), generator=gen, device="cuda")
        s["prompt_lengths"] = torch.randint(0, L // 2 + 1, (N,), generator=gen, device="cuda")
        s["repetition_penalty"] = _fraction(gen, N, 1.0, 1.3)
        s["frequency_penalty"] = _fraction(gen, N, 0.0, 0.5)
        s["presence_penalty"] = _fraction(gen, N, 0.0, 0.5)
    K = case["bias"]
    if K:
        first = torch.randint(0, V, (N, 1), generator=gen, device="cuda")
        s["bias_tokens"] = (first + torch.arange(K, device="cuda") * (V // K)) % V
        s["bias_values"] = _normal(gen, (N, K), torch.float32, 5.0)
    if case["mask"]:
        s["mask"] = _mask(gen, N, V)
    s["temperature"] = _fraction(gen, N, 0.5, 1.5)
    return s


_LOGITS_ARGS = ("history", "history_lengths", "prompt_lengths", "repetition_penalty", "frequency_penalty",
                "presence_penalty", "bias_tokens", "bias_values", "mask", "temperature")


# -------------------------------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import vocabulary_cross_entropy_pass_gb300 as ce
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return ce.ce_embed_fwd(s["tokens"], s["weight"], scale=case["scale"])
    if op == "embed_grad":
        if case["tied"]:
            return ce.ce_embed_bwd(s["grad_out"], s["tokens"], case["V"], scale=case["scale"],
                                   grad_weight=s["grad"], accumulate=True)
        return ce.ce_embed_bwd(s["grad_out"], s["tokens"], case["V"], scale=case["scale"])
    if op == "norm":
        quant = FP8[case["fp8"]][0] if "fp8" in case else None
        y, h, scales = ce.ce_rmsnorm_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=quant,
                                         group_size=case.get("group", 0))
        return {"y": y, "h": h if s["residual"] is not None else None, "scales": scales}
    if op == "norm_grad":
        gx, gw = ce.ce_rmsnorm_bwd(s["grad_out"], s["h"], s["weight"], eps=EPS, grad_h=s["grad_h"])
        return {"x": gx, "weight": gw}
    args = {k: s[k] for k in _LOGITS_ARGS if k in s}
    if op == "logits":
        return ce.ce_logits_process(s["logits"], **args)
    for k in ("prompt_lengths", "frequency_penalty", "presence_penalty", "bias_tokens", "bias_values"):
        args.pop(k, None)  # terms that the gradient does not see
    return ce.ce_logits_process_bwd(s["grad_out"], s["logits"], **args)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op == "embed":
        return (s["weight"][s["tokens"]].float() * case["scale"]).to(dt)
    if op == "embed_grad":
        rows = s["grad_out"].float() * case["scale"]
        grad = s["grad"] if case["tied"] else torch.zeros(case["V"], case["H"], device="cuda")
        return grad.index_add_(0, s["tokens"], rows)
    if op == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        y = h * rstd * s["weight"].float()
        out = {"y": None, "h": h.to(dt) if s["residual"] is not None else None, "scales": None}
        if "fp8" not in case:
            out["y"] = y.to(dt)
            return out
        kind, top = FP8[case["fp8"]]
        group = case["group"] or case["H"]
        G = -(-case["H"] // group)
        wide = torch.nn.functional.pad(y, (0, G * group - case["H"])).view(case["N"], G, group)
        scales = (wide.abs().amax(-1) / top).clamp(min=TINY)
        q = (wide / scales[:, :, None]).clamp(-top, top).view(case["N"], -1)[:, :case["H"]]
        out["y"], out["scales"] = q.to(kind), scales
        return out
    if op == "norm_grad":
        h, g, w = s["h"].float(), s["grad_out"].float(), s["weight"].float()
        rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        n = h * rstd
        gw = g * w
        gx = rstd * (gw - n * (gw * n).mean(-1, keepdim=True))
        if s["grad_h"] is not None:
            gx = gx + s["grad_h"].float()
        return {"x": gx.to(dt), "weight": (g * n).sum(0)}
    x = s["logits"].float()
    N, V = x.shape
    y = x if op == "logits" else s["grad_out"].float()
    if "history" in s:
        at = torch.arange(s["history"].shape[1], device="cuda")[None]
        inside = at < s["history_lengths"][:, None]
        seen = torch.zeros(N, V, device="cuda").scatter_add_(1, s["history"], inside.float()) > 0
        r = s["repetition_penalty"][:, None]
        if op == "logits":
            new = inside & (at >= s["prompt_lengths"][:, None])
            count = torch.zeros(N, V, device="cuda").scatter_add_(1, s["history"], new.float())
            y = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
            y = y - s["frequency_penalty"][:, None] * count - s["presence_penalty"][:, None] * (count > 0)
        else:
            y = torch.where(seen, torch.where(x > 0, y / r, y * r), y)
    if op == "logits" and "bias_tokens" in s:
        y = y.scatter_add(1, s["bias_tokens"], s["bias_values"])
    y = y / s["temperature"][:, None]
    if "mask" in s:
        at = torch.arange(V, device="cuda")
        allowed = (s["mask"][:, at // 32] >> (at % 32)) & 1
        y = torch.where(allowed != 0, y, NEG if op == "logits" else 0.0)
    return y.to(dt)


# ----------------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    """The definition in float64, from the inputs' own values: sums by counting and by sorted runs,
    where the plain form scatters."""
    s = prepare(case, seed)
    op = case["op"]
    N = case["N"]
    if op == "embed":
        return torch.index_select(s["weight"], 0, s["tokens"]).double().mul_(case["scale"])
    if op == "embed_grad":
        # running sums over the tokens in sorted order, a run's sum the difference at its ends
        order = torch.argsort(s["tokens"], stable=True)
        ids, n = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        ends = torch.cumsum(n, 0) - 1
        run_sum = torch.cumsum(s["grad_out"].double()[order], 0)[ends]
        run_sum[1:] = run_sum[1:] - run_sum[:-1].clone()
        out = s["grad"].double() if case["tied"] else torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
        out[ids] += run_sum * case["scale"]
        return out
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h += s["residual"].double()
        y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True).square() / case["H"] + EPS)
        y = y * s["weight"].double()
        out = {"y": y, "h": h if s["residual"] is not None else None, "scales": None}
        if "fp8" in case:
            top = FP8[case["fp8"]][1]
            cols = torch.arange(case["H"], device="cuda") // (case["group"] or case["H"])
            G = int(cols[-1]) + 1
            m = torch.zeros(N, G, dtype=torch.float64, device="cuda")
            m.scatter_reduce_(1, cols[None].expand(N, -1), y.abs(), "amax")
            out["scales"] = torch.clamp(m / top, min=TINY)
            out["y"] = y / out["scales"][:, cols]
        return out
    if op == "norm_grad":
        h, w, g = s["h"].double(), s["weight"].double(), s["grad_out"].double()
        inv = 1 / torch.sqrt(h.square().sum(1) / case["H"] + EPS)
        dot = torch.einsum("nh,h,nh->n", g, w, h)
        gx = g * w * inv[:, None] - h * (inv ** 3 * dot / case["H"])[:, None]
        if s["grad_h"] is not None:
            gx += s["grad_h"].double()
        return {"x": gx, "weight": torch.einsum("nh,nh,n->h", g, h, inv)}
    V = case["V"]
    x = s["logits"].double()
    row = torch.arange(N, device="cuda")[:, None]
    y = x.clone() if op == "logits" else s["grad_out"].double()
    if "history" in s:
        L = case["hist"]
        at = torch.arange(L, device="cuda")[None].expand(N, L)
        cell = row * V + s["history"]
        every = at < s["history_lengths"][:, None]
        seen = torch.bincount(cell[every], minlength=N * V).view(N, V)
        factor = torch.where(x > 0, 1 / s["repetition_penalty"].double()[:, None], s["repetition_penalty"].double()[:, None])
        y *= torch.where(seen > 0, factor, 1.0)
        if op == "logits":
            late = torch.bincount(cell[every & (at >= s["prompt_lengths"][:, None])], minlength=N * V).view(N, V)
            y -= late.double() * s["frequency_penalty"].double()[:, None]
            y -= late.sign().double() * s["presence_penalty"].double()[:, None]
    if op == "logits" and "bias_tokens" in s:
        y[row, s["bias_tokens"]] += s["bias_values"].double()  # a row's biased tokens differ
    y /= s["temperature"].double()[:, None]
    if "mask" in s:
        word = s["mask"].repeat_interleave(32, dim=1)[:, :V]
        bit = torch.ones(1, dtype=torch.int32, device="cuda") << (torch.arange(V, device="cuda", dtype=torch.int32) % 32)
        y[(word & bit[None]) == 0] = NEG if op == "logits" else 0.0
    return y


# -------------------------------------------------------------------------------------------- work
def _distinct(N, V):
    """Expected number of different tokens among N of the distribution above."""
    edge = np.log(np.arange(1, V + 2)) / math.log(V + 1)
    return float(np.sum(-np.expm1(N * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12)))))


def work(case):
    op, N, e = case["op"], case["N"], BYTES[case["dtype"]]
    if op == "embed":
        H = case["H"]
        return {"bytes": N * 8 + _distinct(N, case["V"]) * H * e + N * H * e, "flops": N * H}
    if op == "embed_grad":
        V, H = case["V"], case["H"]
        rows = 2 * _distinct(N, V) if case["tied"] else V
        return {"bytes": N * 8 + N * H * e + rows * H * 4, "flops": 2 * N * H}
    if op == "norm":
        H = case["H"]
        streams = 3 if case["residual"] else 1  # x, the residual in and out
        G = -(-H // (case["group"] or H)) if "fp8" in case else 0
        out = H + 4 * G if "fp8" in case else H * e
        return {"bytes": N * (streams * H * e + out) + H * e, "flops": 6 * N * H}
    if op == "norm_grad":
        H = case["H"]
        streams = 4 if case["residual"] else 3  # h, the gradients in and out
        return {"bytes": N * streams * H * e + H * (e + 4), "flops": 12 * N * H}
    V = case["V"]
    free = (N + 3) // 4
    read = free * V + (N - free) * V / 64 if case["mask"] else N * V  # a forbidden logit need not be read
    bits = N * -(-V // 32) * 4 if case["mask"] else 0
    lists = N * (case["hist"] * 8 * 0.75 + (case["bias"] * 12 if op == "logits" else 0) + 40)
    return {"bytes": read * e + N * V * e + bits + lists, "flops": 2 * N * V}
