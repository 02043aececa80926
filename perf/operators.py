"""The cases on which the training-loss operators and the gradient clipping are measured.

What stands before an optimizer step: log-probabilities of given tokens (from logits, or from
hidden states and the vocabulary matrix), a preference loss or a clipped policy loss with its
gradient on the logits, and the global norm and clipping of the parameters' gradients. The
vocabulary of 50257 and the widths 768, 2048 and 3200 are this repository's own workloads';
other vocabularies are generic.

`run` computes a case with plain torch operations in 32 bits, or, where `own` is set, with the
framework's operators. `exact` computes it in 64 bits, written apart.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
NEG = float("-inf")


# ---- the cases --------------------------------------------------------------------------
def _logp(name, T, V, dtype, grad, entropy, masked=0, pad=0, temperature=1.0):
    return {"name": name, "op": "logp", "T": T, "V": V, "dtype": dtype, "grad": grad, "entropy": entropy,
            "masked": masked, "pad": pad, "temperature": temperature}


def _pref(name, T, V, dtype, pairs, kind, smoothing=0.0, average=False, pad=0):
    return {"name": name, "op": "preference", "T": T, "V": V, "dtype": dtype, "pairs": pairs, "kind": kind,
            "smoothing": smoothing, "average": average, "pad": pad, "beta": 0.1}


def _policy(name, T, V, dtype, seqs, reduce, adv, kl="k3", kl_coef=0.05, entropy_coef=0.0, dual=0.0, pad=0,
            temperature=1.0):
    return {"name": name, "op": "policy", "T": T, "V": V, "dtype": dtype, "seqs": seqs, "reduce": reduce, "adv": adv,
            "kl": kl, "kl_coef": kl_coef, "entropy_coef": entropy_coef, "dual": dual, "pad": pad,
            "temperature": temperature}


def _linear(name, T, V, D, dtype, entropy, masked=0):
    return {"name": name, "op": "linear", "T": T, "V": V, "D": D, "dtype": dtype, "entropy": entropy, "masked": masked}


def _clip(name, model, d, layers, src, count=0):
    return {"name": name, "op": "clip", "model": model, "d": d, "layers": layers, "src": src, "count": count}


def listed():
    return [
        # one sampled token's log-probability and entropy after a decoding step: latency
        _logp("logp 1 token", 1, 50257, "bf16", False, True),
        # scoring a batch of responses under a frozen model
        _logp("logp 4096 tokens fp16", 4096, 50257, "fp16", False, True, masked=1),
        # a loss of the user's own between the two directions, logits in 32 bits, a ragged batch
        _logp("logp + gradient fp32", 2039, 50257, "fp32", True, True, masked=1, temperature=0.7),
        # a small preference batch: three pairs of short answers
        _pref("preference 3 pairs", 349, 50257, "bf16", 3, "sigmoid", smoothing=0.1),
        # a full preference batch: sixteen pairs, prompts masked
        _pref("preference 16 pairs", 8192, 50257, "bf16", 16, "sigmoid"),
        # the smallest policy micro-batch: four short answers
        _policy("policy 61 tokens", 61, 50257, "bf16", 4, "sequence", "sequence"),
        # a full policy micro-batch, with the entropy bonus and the second clip
        _policy("policy 8192 tokens", 8192, 50257, "bf16", 24, "token", "sequence", entropy_coef=0.01, dual=3.0),
        # a few tokens scored against the small vocabulary matrix: bound by reading the matrix
        _linear("linear logp 16 tokens", 16, 50257, 768, "bf16", True),
        # reference log-probabilities of a batch: bound by the product
        _linear("linear logp 8192 tokens", 8192, 50257, 2048, "bf16", True, masked=1),
        # the norm vectors and biases of a small model: latency
        _clip("clip 26 vectors", "vectors", 768, 26, "fp32"),
        # all gradients of the small model as 32-bit tensors of their own, into the flat bf16 gradient
        _clip("clip 124M fp32", "ln", 768, 12, "fp32"),
        # all gradients of the 1.3B model in bf16
        _clip("clip 1.3B bf16", "plain", 2048, 24, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp", "preference", "policy", "linear", "clip"])
    if op == "clip":
        model = rng.choice(["vectors", "ln", "plain", "ragged", "ragged"])
        src = rng.choice(["fp32", "bf16", "fp16", "mixed"])
        if model == "vectors":
            c = _clip("", model, _log(rng, 1, 5000), rng.randint(1, 60), src)
        elif model == "ragged":
            c = _clip("", model, _log(rng, 100, 1 << 21), 0, src, count=_log(rng, 2, 600))
        else:
            c = _clip("", model, rng.choice([256, 768, 1024, 1600]), rng.randint(1, 16), src)
    elif op == "linear":
        D = 8 * _log(rng, 8, 400)
        V = _log(rng, 1000, 130000)
        T = min(_log(rng, 1, 8192), max(1, int(8192 * 50257 * 2048 / (V * D))))
        c = _linear("", T, V, D, rng.choice(["bf16", "fp16"]), rng.random() < 0.5, masked=rng.randint(0, 1))
    else:
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        V = rng.choice([50257, 50304, _log(rng, 1000, 160000), 2 * _log(rng, 500, 80000) + 1])
        cap = 8192 * 50257 * 2 // (V * SIZE[dtype])
        T = min(_log(rng, 1 if op == "logp" else 8, 8192), cap)
        pad = rng.choice([0, 0, 0, V // 50])
        if op == "logp":
            c = _logp("", T, V, dtype, rng.random() < 0.5, rng.random() < 0.5, masked=rng.randint(0, 1), pad=pad,
                      temperature=rng.choice([1.0, 1.0, 0.6, 1.3]))
        elif op == "preference":
            c = _pref("", T, V, dtype, max(1, min(T // 4, _log(rng, 1, 48))), rng.choice(["sigmoid", "hinge", "ipo"]),
                      smoothing=rng.choice([0.0, 0.1]), average=rng.random() < 0.3, pad=pad)
        else:
            c = _policy("", T, V, dtype, max(1, min(T // 2, _log(rng, 1, 64))), rng.choice(["token", "sequence", "sum"]),
                        rng.choice(["token", "sequence"]), kl=rng.choice(["k1", "k2", "k3"]),
                        kl_coef=rng.choice([0.0, 0.05]), entropy_coef=rng.choice([0.0, 0.01]),
                        dual=rng.choice([0.0, 3.0]), pad=pad, temperature=rng.choice([1.0, 0.8]))
    del c["name"]
    return c


def _lengths(T, seqs):
    """Ragged sequence lengths that add up to T; every fifth sequence is empty where there are ten or more."""
    r = random.Random(1000003 * T + seqs)
    w = [0.0 if seqs >= 10 and i % 5 == 3 else r.uniform(0.4, 1.6) for i in range(seqs)]
    total, out = sum(w), []
    for x in w:
        out.append(int(T * x / total))
    out[0] += T - sum(out)
    return out


def _prompt(n):
    return n // 4


def _live_rows(case):
    """Which rows carry a loss: a quarter of each sequence is prompt."""
    if case["op"] in ("logp", "linear"):
        return case["T"] - (case["T"] // 4 if case["masked"] else 0)
    lens = _lengths(case["T"], 2 * case["pairs"] if case["op"] == "preference" else case["seqs"])
    return sum(n - _prompt(n) for n in lens)


def _numels(case):
    d, layers = case["d"], case["layers"]
    if case["model"] == "vectors":
        return [d] * layers
    if case["model"] == "ragged":
        r = random.Random(7 * case["count"] + d)
        return [max(0, int(d * math.exp(r.uniform(-3.0, 0.5))) | (i & 1)) if i % 17 else i % 3 for i in range(case["count"])]
    sizes = [50257 * d]
    for _ in range(layers):
        if case["model"] == "ln":
            sizes += [d, d]
        sizes += [d * 3 * d, d * d]
        if case["model"] == "ln":
            sizes += [d, d]
        sizes += [d * 4 * d, 4 * d * d]
    if case["model"] == "ln":
        sizes += [d, d]
    return sizes


def _source(case, i):
    return case["src"] if case["src"] != "mixed" else ("fp32", "bf16", "fp16")[i % 3]


def work(case):
    if case["op"] == "clip":
        n = _numels(case)
        return {"bytes": sum(k * (SIZE[_source(case, i)] + 2) for i, k in enumerate(n)), "flops": 3 * sum(n)}
    T, V, live = case["T"], case["V"], _live_rows(case)
    if case["op"] == "linear":
        return {"bytes": SIZE[case["dtype"]] * case["D"] * (live + V) + 20 * T, "flops": 2.0 * live * V * case["D"]}
    e = SIZE[case["dtype"]]
    if case["op"] == "logp":
        n = live * V * e + (T * V * e if case["grad"] else 0)
        return {"bytes": n + 20 * T, "flops": live * V * (12 if case["grad"] else 6)}
    return {"bytes": live * V * e + T * V * e + 24 * T, "flops": 12 * live * V}


# ---- the inputs -------------------------------------------------------------------------
def _logits(case, gen):
    """Logits as a language model gives them: a broad spread, the token that follows lifted by
    some amount, and, where the vocabulary is padded, the padding at minus infinity."""
    T, V = case["T"], case["V"]
    x = torch.empty((T, V), dtype=TYPES[case["dtype"]], device=DEV).normal_(0.0, 2.0, generator=gen)
    n = V - case["pad"]
    y = torch.randint(0, n, (T,), device=DEV, generator=gen)
    lift = torch.rand(T, device=DEV, generator=gen) * 14.0
    x.scatter_add_(1, y[:, None], lift[:, None].to(x.dtype))
    if case["pad"]:
        x[:, n:] = NEG
    return x, y


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int64, device=DEV)


def _mask_prompts(y, lens):
    keep = torch.cat([torch.arange(n) >= _prompt(n) for n in lens]).to(DEV)
    return torch.where(keep, y, torch.full_like(y, -1))


def _true_logp(x, y, temperature):
    """The policy's own log-probabilities, 256 rows at a time."""
    out = []
    for i in range(0, x.shape[0], 256):
        z = x[i:i + 256].float() / temperature
        out.append(z.gather(1, y[i:i + 256, None])[:, 0] - z.logsumexp(1))
    return torch.cat(out)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": dict(case)}
    T = case.get("T")
    if case["op"] == "clip":
        s["grads"] = [torch.randn(n, device=DEV, generator=gen).mul_(1e-3 * (1 + i % 5)).to(TYPES[_source(case, i)])
                      for i, n in enumerate(_numels(case))]
        total = sum(_numels(case))
        s["flat"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
        # about half of the norm that such gradients have: every pass clips
        s["max_norm"] = 0.5 * 3.3e-3 * math.sqrt(max(1, total))
        if own:
            import zero_gradient_reduce_scatter_gb300 as zg
            s["plan"] = zg.GradClip(s["grads"], list(s["flat"].split(_numels(case))))
        return s
    if case["op"] == "linear":
        D = case["D"]
        s["weight"] = (torch.randn((case["V"], D), device=DEV, generator=gen) * (2.0 / math.sqrt(D))).to(TYPES[case["dtype"]])
        s["targets"] = torch.randint(0, case["V"], (T,), device=DEV, generator=gen)
        h = torch.randn((T, D), device=DEV, generator=gen)
        lift = torch.rand((T, 1), device=DEV, generator=gen) * 3.0
        s["hidden"] = (h + lift * s["weight"].float()[s["targets"]]).to(TYPES[case["dtype"]])
        if case["masked"]:
            s["targets"][: T // 4] = -1
        return s
    s["logits"], y = _logits(case, gen)
    if case["op"] == "logp":
        s["targets"] = y
        if case["masked"]:
            s["targets"] = torch.where(torch.arange(T, device=DEV) < T // 4, torch.full_like(y, -1), y)
        if case["grad"]:
            s["dlogp"] = torch.randn(T, device=DEV, generator=gen) / T
            s["dentropy"] = torch.randn(T, device=DEV, generator=gen) / (10 * T)
        return s
    seqs = 2 * case["pairs"] if case["op"] == "preference" else case["seqs"]
    lens = _lengths(T, seqs)
    s["offsets"] = _offsets(lens)
    s["targets"] = _mask_prompts(y, lens)
    temperature = case.get("temperature", 1.0)
    logp = _true_logp(s["logits"], y, temperature)
    s["ref_logp"] = logp - 0.05 - 0.2 * torch.randn(T, device=DEV, generator=gen)
    if case["op"] == "policy":
        # steps of 0.02 keep the ratio off the clip's edges, where rounding alone would choose the side
        step = torch.round(torch.randn(T, device=DEV, generator=gen) * 8.0) + 0.5
        s["old_logp"] = logp - 0.02 * step
        n = T if case["adv"] == "token" else seqs
        s["advantages"] = 0.4 + torch.randn(n, device=DEV, generator=gen)
    return s


# ---- the plain forms --------------------------------------------------------------------
def _softmax(logits, targets, temperature):
    x = logits.float() / temperature
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    live = targets >= 0
    zy = x.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    logp = torch.where(live, zy - lse, torch.zeros_like(lse))
    return x, e / total, torch.where(live, lse, torch.zeros_like(lse)), logp, live


def _entropy(x, p, lse, live):
    px = torch.where(p > 0, p * x, torch.zeros_like(p)).sum(1)
    return torch.where(live, lse - px, torch.zeros_like(lse))


def _dlogits(x, p, lse, entropy, live, targets, g, h, temperature, dtype):
    """dx = (g (onehot - p) - h p (log p + H)) / temperature, rows without a target zero."""
    g = torch.where(live, g, torch.zeros_like(g))
    d = p * -g[:, None]
    if h is not None:
        h = torch.where(live, h, torch.zeros_like(h))
        d -= torch.where(p > 0, h[:, None] * p * (x - lse[:, None] + entropy[:, None]), torch.zeros_like(p))
    d.scatter_add_(1, targets.clamp(min=0)[:, None], g[:, None])
    d = d / temperature
    return torch.where(live[:, None], d, torch.zeros_like(d)).to(dtype)


def _by_sequence(offsets, T):
    """The sequence of every token, and how many there are."""
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(T, device=offsets.device), right=True), offsets.numel() - 1


def _run_logp(s, c):
    x, p, lse, logp, live = _softmax(s["logits"], s["targets"], c["temperature"])
    out = {"logp": logp, "lse": lse}
    entropy = _entropy(x, p, lse, live) if c["entropy"] or c["grad"] else None
    if c["entropy"]:
        out["entropy"] = entropy
    if c["grad"]:
        out["dlogits"] = _dlogits(x, p, lse, entropy, live, s["targets"], s["dlogp"], s["dentropy"] if c["entropy"] else None,
                                  c["temperature"], s["logits"].dtype)
    return out


def _run_linear(s, c):
    x = s["hidden"].float() @ s["weight"].float().T
    x, p, lse, logp, live = _softmax(x, s["targets"], 1.0)
    out = {"logp": logp, "lse": lse}
    if c["entropy"]:
        out["entropy"] = _entropy(x, p, lse, live)
    return out


def _run_preference(s, c):
    x, p, lse, logp, live = _softmax(s["logits"], s["targets"], 1.0)
    seq, n = _by_sequence(s["offsets"], c["T"])
    delta = torch.where(live, logp - s["ref_logp"], torch.zeros_like(logp))
    total = torch.zeros(n, device=DEV).index_add_(0, seq, delta)
    count = torch.zeros(n, device=DEV).index_add_(0, seq, live.float()).clamp(min=1.0)
    per = count if c["average"] else torch.ones_like(count)
    chosen, rejected = (total / per)[0::2], (total / per)[1::2]
    margin, b, eps = chosen - rejected, c["beta"], c["smoothing"]
    if c["kind"] == "sigmoid":
        t = b * margin
        soft = lambda v: torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))  # noqa: E731
        loss = (1 - eps) * soft(-t) + eps * soft(t)
        dm = b * (1 / (1 + torch.exp(-t)) - (1 - eps))
    elif c["kind"] == "hinge":
        loss = torch.clamp(1 - b * margin, min=0)
        dm = torch.where(b * margin < 1, -b * torch.ones_like(margin), torch.zeros_like(margin))
    else:
        loss = (margin - 1 / (2 * b)) ** 2
        dm = 2 * (margin - 1 / (2 * b))
    g = torch.stack([dm, -dm], 1).reshape(-1) / per / c["pairs"]
    return {"loss": loss.mean(), "pair_loss": loss, "chosen_reward": b * chosen, "rejected_reward": b * rejected,
            "dlogits": _dlogits(x, p, lse, None, live, s["targets"], g[seq], None, 1.0, s["logits"].dtype)}


def _run_policy(s, c):
    x, p, lse, logp, live = _softmax(s["logits"], s["targets"], c["temperature"])
    entropy = _entropy(x, p, lse, live) if c["entropy_coef"] else torch.zeros_like(lse)
    seq, n = _by_sequence(s["offsets"], c["T"])
    zero = torch.zeros_like(logp)
    adv = s["advantages"] if c["adv"] == "token" else s["advantages"][seq]
    r = torch.exp(logp - s["old_logp"])
    plain, clipped = -r * adv, -r.clamp(0.8, 1.28) * adv
    loss = torch.maximum(plain, clipped)
    off = ((adv > 0) & (r > 1.28)) | ((adv < 0) & (r < 0.8))
    if c["dual"]:
        off = off | ((adv < 0) & (r > c["dual"]))
        loss = torch.where(adv < 0, torch.minimum(loss, -c["dual"] * adv), loss)
    g = torch.where(off, zero, plain)
    d = s["ref_logp"] - logp
    kl = {"k1": -d, "k2": 0.5 * d * d, "k3": torch.exp(d) - d - 1}[c["kl"]]
    dkl = {"k1": torch.ones_like(d), "k2": -d, "k3": 1 - torch.exp(d)}[c["kl"]]
    loss = loss + c["kl_coef"] * kl - c["entropy_coef"] * entropy
    g = g + c["kl_coef"] * dkl
    count = torch.zeros(n, device=DEV).index_add_(0, seq, live.float())
    tokens = live.float().sum().clamp(min=1.0)
    if c["reduce"] == "token":
        w = torch.ones_like(logp) / tokens
    elif c["reduce"] == "sequence":
        w = (1 / count.clamp(min=1.0) / (count > 0).float().sum().clamp(min=1.0))[seq]
    else:
        w = torch.ones_like(logp)
    w = torch.where(live, w, zero)
    mean = lambda v: torch.where(live, v, zero).sum() / tokens  # noqa: E731
    return {"loss": torch.where(live, loss * w, zero).sum(), "logp": logp, "entropy": entropy if c["entropy_coef"] else None,
            "clip_fraction": mean(off.float()), "kl": mean(kl),
            "dlogits": _dlogits(x, p, lse, entropy, live, s["targets"], g * w, -c["entropy_coef"] * w if c["entropy_coef"] else None,
                                c["temperature"], s["logits"].dtype)}


def _run_clip(s, c):
    norms = torch.stack([t.float().square().sum() for t in s["grads"]]).sqrt()
    norm = norms.square().sum().sqrt()
    scale = torch.clamp(s["max_norm"] / norm, max=1.0)
    torch.cat([(t.float() * scale).to(torch.bfloat16) for t in s["grads"]], out=s["flat"])
    return {"norm": norm, "scale": scale, "norms": norms, "flat": s["flat"]}


def _own(s, c):
    import zero_gradient_reduce_scatter_gb300 as zg
    if c["op"] == "logp":
        f = zg.token_logp(s["logits"], s["targets"], temperature=c["temperature"], entropy=c["entropy"])
        out = {"logp": f.logp, "lse": f.lse}
        if c["entropy"]:
            out["entropy"] = f.entropy
        if c["grad"]:
            out["dlogits"] = zg.token_logp_backward(s["logits"], s["targets"], f, s["dlogp"],
                                                    s["dentropy"] if c["entropy"] else None, temperature=c["temperature"])
        return out
    if c["op"] == "linear":
        f = zg.linear_logp(s["hidden"], s["weight"], s["targets"], entropy=c["entropy"])
        out = {"logp": f.logp, "lse": f.lse}
        if c["entropy"]:
            out["entropy"] = f.entropy
        return out
    if c["op"] == "preference":
        r = zg.preference_loss(s["logits"], s["targets"], s["offsets"], s["ref_logp"], beta=c["beta"], kind=c["kind"],
                               label_smoothing=c["smoothing"], average=c["average"])
        return {"loss": r.loss, "pair_loss": r.pair_loss, "chosen_reward": r.chosen_reward,
                "rejected_reward": r.rejected_reward, "dlogits": r.dlogits}
    if c["op"] == "policy":
        r = zg.policy_loss(s["logits"], s["targets"], s["advantages"], s["old_logp"], s["ref_logp"], offsets=s["offsets"],
                           clip_low=0.2, clip_high=0.28, dual_clip=c["dual"], kl=c["kl"], kl_coef=c["kl_coef"],
                           entropy_coef=c["entropy_coef"], reduce=c["reduce"], temperature=c["temperature"])
        return {"loss": r.loss, "logp": r.logp, "entropy": r.entropy if c["entropy_coef"] else None,
                "clip_fraction": r.clip_fraction, "kl": r.kl, "dlogits": r.dlogits}
    r = s["plan"].clip(s["max_norm"])
    return {"norm": r.norm, "scale": r.scale, "norms": r.norms, "flat": s["flat"]}


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"logp": _run_logp, "linear": _run_linear, "preference": _run_preference, "policy": _run_policy,
            "clip": _run_clip}[c["op"]](state, c)


# ---- the definition in 64 bits ----------------------------------------------------------
def _exact_rows(x, y, temperature):
    """One block of rows in 64 bits: log p of the whole vocabulary, lse, the target's log p."""
    z = x.double() / temperature
    lse = torch.logsumexp(z, 1)
    logq = z - lse[:, None]
    return logq, lse, logq.gather(1, y.clamp(min=0)[:, None])[:, 0]


def _exact_tokens(s, c, rows):
    """logp, lse and entropy of every token, a block of rows at a time."""
    T = c["T"]
    y = s["targets"]
    logp, lse, ent = (torch.zeros(T, dtype=torch.float64, device=DEV) for _ in range(3))
    for i in range(0, T, rows):
        k = slice(i, min(T, i + rows))
        x = s["logits"][k] if "logits" in s else s["hidden"][k].double() @ s["weight64"].T
        logq, le, lp = _exact_rows(x, y[k], c.get("temperature", 1.0))
        q = logq.exp()
        on = y[k] >= 0
        logp[k] = torch.where(on, lp, torch.zeros_like(lp))
        lse[k] = torch.where(on, le, torch.zeros_like(le))
        ent[k] = torch.where(on, -(q * logq.masked_fill(q == 0, 0.0)).sum(1), torch.zeros_like(le))
    return logp, lse, ent


def _exact_grad(s, c, g, h, ent, rows):
    """The gradient on the logits, a block of rows at a time."""
    temperature = c.get("temperature", 1.0)
    out = torch.zeros((c["T"], c["V"]), dtype=torch.float64, device=DEV)
    y = s["targets"]
    for i in range(0, c["T"], rows):
        k = slice(i, min(c["T"], i + rows))
        logq, _, _ = _exact_rows(s["logits"][k], y[k], temperature)
        q = logq.exp()
        hot = torch.zeros_like(q).scatter_(1, y[k].clamp(min=0)[:, None], 1.0)
        d = g[k, None] * (hot - q)
        if h is not None:
            d = d - h[k, None] * q * (logq.masked_fill(q == 0, 0.0) + ent[k, None])
        out[k] = d / temperature * (y[k] >= 0)[:, None]
    return out


def exact(case, seed):
    s, c, rows = prepare(case, seed), dict(case), 256
    if c["op"] == "clip":
        norms = torch.stack([t.double().pow(2).sum().sqrt() for t in s["grads"]])
        norm = norms.pow(2).sum().sqrt()
        scale = min(1.0, s["max_norm"] / float(norm)) if float(norm) > 0 else 1.0
        flat = torch.cat([t.double().mul_(scale) for t in s["grads"]])
        return {"norm": norm, "scale": torch.tensor(scale, dtype=torch.float64), "norms": norms, "flat": flat}
    if c["op"] == "linear":
        s["weight64"] = s["weight"].double()
        logp, lse, ent = _exact_tokens(s, c, rows)
        return {"logp": logp, "lse": lse, **({"entropy": ent} if c["entropy"] else {})}
    logp, lse, ent = _exact_tokens(s, c, rows)
    live = s["targets"] >= 0
    if c["op"] == "logp":
        out = {"logp": logp, "lse": lse}
        if c["entropy"]:
            out["entropy"] = ent
        if c["grad"]:
            out["dlogits"] = _exact_grad(s, c, s["dlogp"].double(), s["dentropy"].double() if c["entropy"] else None, ent, rows)
        return out
    bounds = s["offsets"].tolist()
    spans = [slice(a, b) for a, b in zip(bounds, bounds[1:])]
    if c["op"] == "preference":
        g, losses, rewards = torch.zeros_like(logp), [], []
        ratio = (logp - s["ref_logp"].double()) * live
        n = [max(1, int(live[k].sum())) if c["average"] else 1 for k in spans]
        for i in range(c["pairs"]):
            up, down = float(ratio[spans[2 * i]].sum()) / n[2 * i], float(ratio[spans[2 * i + 1]].sum()) / n[2 * i + 1]
            m, b, eps = up - down, c["beta"], c["smoothing"]
            if c["kind"] == "sigmoid":
                loss = (1 - eps) * math.log1p(math.exp(-b * m)) + eps * math.log1p(math.exp(b * m))
                dm = b * (eps / (1 + math.exp(-b * m)) - (1 - eps) / (1 + math.exp(b * m)))
            elif c["kind"] == "hinge":
                loss, dm = max(0.0, 1 - b * m), (-b if b * m < 1 else 0.0)
            else:
                loss, dm = (m - 0.5 / b) ** 2, 2 * m - 1 / b
            losses.append(loss)
            rewards.append((b * up, b * down))
            g[spans[2 * i]] = dm / c["pairs"] / n[2 * i]
            g[spans[2 * i + 1]] = -dm / c["pairs"] / n[2 * i + 1]
        f = lambda v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
        return {"loss": f(sum(losses) / len(losses)), "pair_loss": f(losses), "chosen_reward": f([r[0] for r in rewards]),
                "rejected_reward": f([r[1] for r in rewards]), "dlogits": _exact_grad(s, c, g, None, ent, rows)}
    adv, w = torch.zeros_like(logp), torch.zeros_like(logp)
    counts = [int(live[k].sum()) for k in spans]
    for i, k in enumerate(spans):
        adv[k] = s["advantages"][k].double() if c["adv"] == "token" else s["advantages"][i].double()
        w[k] = {"token": 1.0 / max(1, sum(counts)), "sum": 1.0,
                "sequence": 1.0 / max(1, counts[i]) / max(1, sum(x > 0 for x in counts))}[c["reduce"]]
    w = w * live
    ratio = (logp - s["old_logp"].double()).exp()
    keep = torch.where(adv >= 0, ratio <= 1.28, ratio >= 0.8)
    surrogate = torch.where(keep, ratio, torch.where(adv >= 0, 1.28, 0.8).double()) * adv
    if c["dual"]:
        low = (adv < 0) & (ratio > c["dual"])
        surrogate, keep = torch.where(low, c["dual"] * adv, surrogate), keep & ~low
    gap = logp - s["ref_logp"].double()
    kl, dkl = {"k1": (gap, torch.ones_like(gap)), "k2": (gap.pow(2) / 2, gap),
               "k3": (torch.expm1(-gap) + gap, -torch.expm1(-gap))}[c["kl"]]
    loss = -surrogate + c["kl_coef"] * kl - c["entropy_coef"] * ent
    g = (-(ratio * adv) * keep + c["kl_coef"] * dkl) * w
    tokens = max(1, sum(counts))
    return {"loss": (loss * w).sum(), "logp": logp, "entropy": ent if c["entropy_coef"] else None,
            "clip_fraction": ((~keep) & live).double().sum() / tokens, "kl": (kl * live).sum() / tokens,
            "dlogits": _exact_grad(s, c, g, -c["entropy_coef"] * w if c["entropy_coef"] else None, ent, rows)}
