"""The cases on which distillation and the embedding of tokens are measured.

Distillation before an optimizer step: a teacher's most likely tokens with their log-probabilities
(`top_logits`), and the divergence of a student's logits from them with its gradient (`distill_loss`).
The other end of the vocabulary matrix: the rows of a batch of tokens, and their gradient, sorted by
token, into a gradient of the whole matrix (`embedding`, `embedding_backward`). The vocabulary of
50257 and the widths 768, 2048 and 3200 are this repository's own workloads'; others are generic.

`run` computes a case with plain torch operations in 32 bits (64 for the few numbers of a token's
list), or, where `own` is set, with the framework's operators. `exact` computes it in 64 bits,
written apart.
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
def _top(name, T, V, k, dtype, masked=0, pad=0, temperature=1.0):
    return {"name": name, "op": "top", "T": T, "V": V, "k": k, "dtype": dtype, "masked": masked, "pad": pad,
            "temperature": temperature}


def _distill(name, T, V, k, dtype, seqs, kind="forward", tail="rest", known_rest=True, ragged=0, ce_coef=0.0, reduce="token",
             pad=0, temperature=1.0):
    return {"name": name, "op": "distill", "T": T, "V": V, "k": k, "dtype": dtype, "seqs": seqs, "kind": kind, "tail": tail,
            "known_rest": bool(known_rest), "ragged": ragged, "ce_coef": ce_coef, "reduce": reduce, "pad": pad,
            "temperature": temperature}


def _embed(name, T, V, D, dtype, scale=1.0, masked=0):
    return {"name": name, "op": "embed", "T": T, "V": V, "D": D, "dtype": dtype, "scale": scale, "masked": masked}


def _embed_grad(name, T, V, D, dtype, scale=1.0, masked=0, into="new"):
    return {"name": name, "op": "embed_grad", "T": T, "V": V, "D": D, "dtype": dtype, "scale": scale, "masked": masked,
            "into": into}


def listed():
    return [
        # the alternatives to one sampled token, beside a decoding step: latency
        _top("top 20 of 1 token", 1, 50257, 20, "bf16"),
        # a teacher's lists for a batch whose prompts are masked
        _top("top 64 of 8192 tokens", 8192, 50257, 64, "bf16", masked=1),
        # a teacher of a wider vocabulary, logits in 32 bits, long lists
        _top("top 256 of 1021 wide fp32", 1021, 151936, 256, "fp32", temperature=2.0),
        # the smallest distillation micro-batch: four short answers, lists cut where the teacher is sure
        _distill("distill 61 tokens", 61, 50257, 32, "bf16", 4, ragged=1, reduce="sequence"),
        # a full micro-batch of lists of 64
        _distill("distill 8192 tokens", 8192, 50257, 64, "bf16", 24),
        # on the student's own samples: reverse divergence, a label term, a wider vocabulary
        _distill("distill 2039 wide reverse", 2039, 151936, 128, "bf16", 16, kind="reverse", ce_coef=0.1),
        # the token of a decoding step
        _embed("embedding 1 token", 1, 50257, 768, "bf16"),
        # a training batch's tokens, scaled by the root of the width
        _embed("embedding 16384 tokens", 16384, 50257, 2048, "bf16", scale=45.25, masked=1),
        # a small micro-batch: most of the work is the rows that no token has
        _embed_grad("embedding gradient 512", 512, 50257, 768, "bf16"),
        # a training batch's gradient in 32 bits
        _embed_grad("embedding gradient 16384 fp32", 16384, 50257, 2048, "fp32", scale=45.25, masked=1),
        # a tied matrix: added to the gradient that the output product has left
        _embed_grad("embedding gradient tied", 65536, 50257, 2048, "bf16", into="sum"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "top", "distill", "distill", "embed", "embed_grad", "embed_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("embed", "embed_grad"):
        D = rng.choice([768, 2048, 3200, 8 * _log(rng, 4, 400), _log(rng, 24, 1000) | 1])
        V = rng.choice([50257, _log(rng, 500, 200000)])
        V = max(500, min(V, 50257 * 2048 * 4 // (D * SIZE[dtype])))
        T = min(_log(rng, 1, 65536), 65536 * 2048 * 2 // (D * SIZE[dtype]))
        scale = rng.choice([1.0, 1.0, math.sqrt(D)])
        if op == "embed":
            c = _embed("", T, V, D, dtype, scale, masked=rng.randint(0, 1))
        else:
            c = _embed_grad("", T, V, D, dtype, scale, masked=rng.randint(0, 1), into=rng.choice(["new", "given", "sum"]))
    else:
        V = rng.choice([50257, 50304, 151936, _log(rng, 1000, 160000), 2 * _log(rng, 500, 80000) + 1])
        cap = 8192 * 50257 * 2 // (V * SIZE[dtype])
        T = max(1, min(_log(rng, 1 if op == "top" else 8, 8192), cap))
        pad = rng.choice([0, 0, 0, V // 50])
        temperature = rng.choice([1.0, 1.0, 0.7, 1.5])
        if op == "top":
            c = _top("", T, V, _log(rng, 1, 512), dtype, masked=rng.randint(0, 1), pad=pad, temperature=temperature)
        else:
            kind = rng.choice(["forward", "forward", "reverse", "js"])
            tail = rng.choice(["rest", "rest", "drop", "renormalise"]) if kind == "forward" else "rest"
            c = _distill("", T, V, _log(rng, 4, 256), dtype, max(1, min(T // 2, _log(rng, 1, 64))), kind, tail,
                         known_rest=rng.random() < 0.7, ragged=rng.randint(0, 1), ce_coef=rng.choice([0.0, 0.0, 0.5]),
                         reduce=rng.choice(["token", "sequence", "sum"]), pad=pad, temperature=temperature)
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


def _live(case):
    """Tokens that are not masked: a quarter of the batch, or of each sequence, is prompt."""
    if case["op"] == "distill":
        return sum(n - n // 4 for n in _lengths(case["T"], case["seqs"]))
    return case["T"] - (case["T"] // 4 if case["masked"] else 0)


def _distinct(case):
    """Expected number of different tokens among those that are not masked (see _tokens)."""
    V, n = case["V"], _live(case)
    r = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log1p(1.0 / r) / math.log(V + 1.0)
    return float((1.0 - (1.0 - p).pow(n)).sum())


def work(case):
    T, V, e, live = case["T"], case["V"], SIZE[case["dtype"]], _live(case)
    if case["op"] == "top":
        return {"bytes": live * V * e + 8 * T + (12 * case["k"] + 8) * T, "flops": 6 * live * V}
    if case["op"] == "distill":
        return {"bytes": (live + T) * V * e + 12 * case["k"] * live + 20 * T, "flops": 12 * live * V}
    row = case["D"] * e
    if case["op"] == "embed":
        return {"bytes": _distinct(case) * row + T * row + 8 * T, "flops": T * case["D"]}
    rows = 2 * _distinct(case) if case["into"] == "sum" else V
    return {"bytes": live * row + rows * row + 8 * T, "flops": live * case["D"]}


# ---- the inputs -------------------------------------------------------------------------
def _teacher(case, gen):
    """A teacher's logits in 32 bits: a broad spread, the token that follows lifted by some amount,
    and, where the vocabulary is padded, the padding at minus infinity."""
    T, V = case["T"], case["V"]
    x = torch.empty((T, V), device=DEV).normal_(0.0, 2.0, generator=gen)
    n = V - case["pad"]
    y = torch.randint(0, n, (T,), device=DEV, generator=gen)
    x.scatter_add_(1, y[:, None], torch.rand((T, 1), device=DEV, generator=gen) * 14.0)
    if case["pad"]:
        x[:, n:] = NEG
    return x, y


def _tokens(case, gen):
    """Token ids as text has them: the probability of rank r falls as 1 / r, ranks in no order of ids."""
    T, V = case["T"], case["V"]
    u = torch.rand(T, device=DEV, generator=gen, dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp(0, V - 1)
    t = (rank * _coprime(V) + 17) % V
    if case["masked"]:
        t[: T // 4] = -1
    return t


def _coprime(V):
    m = int(0.6180339887 * V) | 1
    while math.gcd(m, V) != 1:
        m += 2
    return m


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": dict(case)}
    T, V, dtype = case["T"], case["V"], TYPES[case["dtype"]]
    if case["op"] == "top":
        x, y = _teacher(case, gen)
        s["logits"] = x.to(dtype)
        s["targets"] = torch.where(torch.arange(T, device=DEV) < T // 4, torch.full_like(y, -1), y) if case["masked"] else None
        return s
    if case["op"] == "distill":
        x, y = _teacher(case, gen)
        k = min(case["k"], V)
        z = x / case["temperature"]
        lse = torch.logsumexp(z, 1)
        top = torch.topk(z, k, dim=1)
        s["index"], s["teacher_logp"] = top.indices, top.values - lse[:, None]
        rest = torch.zeros((T, V), dtype=torch.bool, device=DEV).scatter_(1, top.indices, True)
        if case["ragged"]:  # as a teacher's lists that end where a share of its mass is reached
            ends = torch.randint(1, k + 1, (T, 1), device=DEV, generator=gen)
            gone = torch.arange(k, device=DEV)[None, :] >= ends
            rest.scatter_(1, top.indices, ~gone)
            s["index"] = s["index"].masked_fill(gone, -1)
            s["teacher_logp"] = s["teacher_logp"].masked_fill(gone, NEG)
        s["teacher_rest"] = torch.logsumexp(z.masked_fill_(rest, NEG), 1) - lse if case["known_rest"] else None
        del z, rest, top
        # the student's logits are the teacher's, off by what is still to be learnt
        x += torch.empty_like(x).normal_(0.0, 1.0, generator=gen)
        s["logits"] = x.to(dtype)
        lens = _lengths(T, case["seqs"])
        off = [0]
        for n in lens:
            off.append(off[-1] + n)
        s["offsets"] = torch.tensor(off, dtype=torch.int64, device=DEV)
        keep = torch.cat([torch.arange(n) >= n // 4 for n in lens]).to(DEV)
        s["targets"] = torch.where(keep, y, torch.full_like(y, -1))
        return s
    D = case["D"]
    s["tokens"] = _tokens(case, gen)
    if case["op"] == "embed":
        s["weight"] = (torch.randn((V, D), device=DEV, generator=gen) * 0.02).to(dtype)
        return s
    s["dhidden"] = (torch.randn((T, D), device=DEV, generator=gen) * 1e-3).to(dtype)
    if case["into"] != "new":
        s["grad"] = (torch.randn((V, D), device=DEV, generator=gen) * 1e-3).to(dtype)
    return s


# ---- the plain forms --------------------------------------------------------------------
def _run_top(s, c):
    x = s["logits"].float()
    T, V = x.shape
    # whole numbers in the order of the values, the lower place first among equal ones
    bits = (x + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32) + (0xFFFFFFFF - torch.arange(V, device=DEV))
    index = 0xFFFFFFFF - (torch.topk(order, c["k"], dim=1).values & 0xFFFFFFFF)
    z = x / c["temperature"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True).double()
    lse = m.double() + torch.log(total)
    logp = (z.gather(1, index) - m).double() - torch.log(total)
    rest = torch.log(e.scatter(1, index, 0.0).sum(1, keepdim=True).double()) - torch.log(total)
    if s["targets"] is not None:
        on = (s["targets"] >= 0)[:, None]
        index = torch.where(on, index, torch.full_like(index, -1))
        logp, lse, rest = (torch.where(on, v, torch.zeros_like(v)) for v in (logp, lse, rest))
    return {"index": index, "logp": logp.float(), "lse": lse[:, 0].float(), "rest": rest[:, 0].float()}


def _run_distill(s, c):
    T, V = s["logits"].shape
    live = s["targets"] >= 0
    there = (s["index"] >= 0) & (s["teacher_logp"] > NEG)
    place = torch.where(there, s["index"], torch.full_like(s["index"], V))
    listed_ = torch.zeros((T, V + 1), dtype=torch.bool, device=DEV).scatter_(1, place, True)[:, :V]
    z = s["logits"].float() / c["temperature"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    zr = torch.where(listed_, torch.zeros_like(e), e).sum(1, keepdim=True)
    log_total = torch.log(total.double())
    # a token's list, and the rest of the vocabulary behind it as one more entry
    none = torch.full_like(log_total, NEG)
    lq = (z.gather(1, s["index"].clamp(min=0)) - m).double() - log_total
    lp = s["teacher_logp"].double()
    lp = torch.where(there, lp, torch.full_like(lp, NEG))
    if c["tail"] == "renormalise":
        lp = lp - torch.log(torch.exp(lp).sum(1, keepdim=True))
    if c["tail"] == "rest":
        if s["teacher_rest"] is not None:
            rest = s["teacher_rest"].double()[:, None]
        else:
            rest = torch.log((1.0 - torch.exp(lp).sum(1, keepdim=True)).clamp(min=2.0 ** -24))
    else:
        rest = none
    lq = torch.cat([lq, torch.log(zr.double()) - log_total], 1)
    lp = torch.cat([lp, rest], 1)
    there = torch.cat([there, torch.full_like(live[:, None], c["tail"] == "rest")], 1)
    p, q = torch.exp(lp), torch.exp(lq)
    zero = torch.zeros_like(lq)
    if c["kind"] == "forward":
        div = torch.where(there & (p > 0), p * (lp - lq), zero)
        g = torch.where(there, -p, zero)
    elif c["kind"] == "reverse":
        div = torch.where(there, q * (lq - lp), zero)
        g = div
    else:
        lm = torch.log(0.5 * p + 0.5 * q)
        div = torch.where(there, 0.5 * torch.where(p > 0, p * (lp - lm), zero) + 0.5 * q * (lq - lm), zero)
        g = torch.where(there, 0.5 * q * (lq - lm), zero)
    kl = div.sum(1)
    shift = g.sum(1, keepdim=True)  # of the gradient on the entries' log q, taken from every logit by its share
    y = s["targets"].clamp(min=0)[:, None]
    logp = ((z.gather(1, y) - m).double() - log_total)[:, 0]
    offsets = s["offsets"]
    seq = torch.searchsorted(offsets[1:].contiguous(), torch.arange(T, device=DEV), right=True)
    count = torch.zeros(offsets.numel() - 1, dtype=torch.float64, device=DEV).index_add_(0, seq, live.double())
    tokens = live.double().sum().clamp(min=1.0)
    if c["reduce"] == "token":
        w = torch.ones_like(kl) / tokens
    elif c["reduce"] == "sequence":
        w = (1.0 / count.clamp(min=1.0) / (count > 0).double().sum().clamp(min=1.0))[seq]
    else:
        w = torch.ones_like(kl)
    w = torch.where(live, w, torch.zeros_like(w))
    off = torch.zeros_like(kl)
    loss = torch.where(live, (kl - c["ce_coef"] * logp) * w, off).sum()
    # an unlisted logit's share: its part of the rest's gradient, less its part of the sum of all
    per = torch.where(zr[:, 0] > 0, g[:, -1] / zr[:, 0].double(), off) - (shift[:, 0] - c["ce_coef"]) / total[:, 0].double()
    d = e * per[:, None].float()
    entry = g[:, :-1] - q[:, :-1] * (shift - c["ce_coef"])
    d = torch.cat([d, torch.zeros_like(d[:, :1])], 1).scatter_(1, place, entry.float())
    d.scatter_add_(1, y, torch.full_like(y, -c["ce_coef"], dtype=torch.float32))
    d = d[:, :V] * (w / c["temperature"]).float()[:, None]
    d = torch.where(live[:, None], d, torch.zeros_like(d)).to(s["logits"].dtype)
    kl, logp = torch.where(live, kl, off), torch.where(live, logp, off)
    return {"loss": loss.float(), "kl": (kl.sum() / tokens).float(), "token_kl": kl.float(), "logp": logp.float(), "dlogits": d}


def _run_embed(s, c):
    t = s["tokens"]
    rows = s["weight"][t.clamp(min=0)].float() * c["scale"]
    return torch.where((t >= 0)[:, None], rows, torch.zeros_like(rows)).to(s["weight"].dtype)


def _run_embed_grad(s, c):
    t, x = s["tokens"], s["dhidden"]
    live = t >= 0
    # a row behind the last takes what carries no gradient
    d = torch.zeros((c["V"] + 1, c["D"]), device=DEV).index_add_(0, torch.where(live, t, torch.full_like(t, c["V"])), x.float())
    d = d[:-1] * c["scale"]
    if c["into"] == "sum":
        d = d + s["grad"].float()
    if c["into"] == "new":
        return d.to(x.dtype)
    return s["grad"].copy_(d)


def _own(s, c):
    import zero_gradient_reduce_scatter_gb300 as zg
    if c["op"] == "top":
        r = zg.top_logits(s["logits"], c["k"], s["targets"], temperature=c["temperature"])
        return {"index": r.index, "logp": r.logp, "lse": r.lse, "rest": r.rest}
    if c["op"] == "distill":
        r = zg.distill_loss(s["logits"], s["targets"], s["index"], s["teacher_logp"], s["teacher_rest"], offsets=s["offsets"],
                            kind=c["kind"], tail=c["tail"], ce_coef=c["ce_coef"], reduce=c["reduce"], temperature=c["temperature"])
        return {"loss": r.loss, "kl": r.kl, "token_kl": r.token_kl, "logp": r.logp, "dlogits": r.dlogits}
    if c["op"] == "embed":
        return zg.embedding(s["weight"], s["tokens"], scale=c["scale"])
    return zg.embedding_backward(s["tokens"], s["dhidden"], c["V"], scale=c["scale"], out=s.get("grad"), accumulate=c["into"] == "sum")


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"top": _run_top, "distill": _run_distill, "embed": _run_embed, "embed_grad": _run_embed_grad}[c["op"]](state, c)


# ---- the definition in 64 bits ----------------------------------------------------------
def _exact_top(s, c):
    x, k = s["logits"], c["k"]
    T = x.shape[0]
    index = torch.full((T, k), -1, dtype=torch.int64, device=DEV)
    logp = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    lse, rest = torch.zeros(T, dtype=torch.float64, device=DEV), torch.zeros(T, dtype=torch.float64, device=DEV)
    for i in range(0, T, 256):
        rows = slice(i, min(T, i + 256))
        on = torch.ones(rows.stop - i, dtype=torch.bool, device=DEV) if s["targets"] is None else s["targets"][rows] >= 0
        z = x[rows].double() / c["temperature"]
        v, at = torch.sort(z, dim=1, descending=True, stable=True)
        le = torch.logsumexp(v, 1)
        index[rows] = torch.where(on[:, None], at[:, :k], index[rows])
        logp[rows] = (v[:, :k] - le[:, None]) * on[:, None]
        lse[rows] = le * on
        rest[rows] = torch.where(on, torch.logsumexp(v[:, k:], 1) - le, rest[rows])
    return {"index": index, "logp": logp, "lse": lse, "rest": rest}


def _exact_distill(s, c):
    T, V = s["logits"].shape
    k = s["index"].shape[1]
    f64 = dict(dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist()
    on = s["targets"] >= 0
    counts = [int(on[a:b].sum()) for a, b in zip(bounds, bounds[1:])]
    w = torch.zeros(T, **f64)
    for n, a, b in zip(counts, bounds, bounds[1:]):
        w[a:b] = {"token": 1.0 / max(1, sum(counts)), "sum": 1.0,
                  "sequence": 1.0 / max(1, n) / max(1, sum(v > 0 for v in counts))}[c["reduce"]]
    w = w * on
    kl, logp, grad = torch.zeros(T, **f64), torch.zeros(T, **f64), torch.zeros((T, V), **f64)
    for i in range(0, T, 128):
        rows = slice(i, min(T, i + 128))
        n = rows.stop - i
        logq = torch.log_softmax(s["logits"][rows].double() / c["temperature"], 1)
        idx, lp = s["index"][rows], s["teacher_logp"][rows].double()
        used = (idx >= 0) & (lp > NEG)
        # which entry a place of the vocabulary belongs to: its own, or k, the rest
        entry = torch.full((n, V), k, dtype=torch.int64, device=DEV)
        r, j = used.nonzero(as_tuple=True)
        entry[r, idx[r, j]] = j
        lqe = torch.full((n, k + 1), NEG, **f64)
        lqe[r, j] = logq[r, idx[r, j]]
        lqe[:, k] = torch.logsumexp(logq.masked_fill(entry < k, NEG), 1)
        lpe = torch.full((n, k + 1), NEG, **f64)
        lpe[r, j] = lp[r, j]
        if c["tail"] == "rest":
            lpe[:, k] = s["teacher_rest"][rows].double() if s["teacher_rest"] is not None else \
                torch.log((1.0 - lpe.exp().sum(1)).clamp(min=2.0 ** -24))
        elif c["tail"] == "renormalise":
            lpe = lpe - torch.logsumexp(lpe, 1, keepdim=True)
        if c["tail"] != "rest":
            lqe[:, k] = NEG
        p, q = lpe.exp(), lqe.exp()
        fp, fq = lpe.clamp(min=-1e4), lqe.clamp(min=-1e4)  # finite where they are multiplied by 0
        # dq: the derivative by an entry's probability
        if c["kind"] == "forward":
            value, dq = p * (fp - fq), torch.where(q > 0, -p / q, torch.zeros_like(q))
        elif c["kind"] == "reverse":
            value, dq = q * (fq - fp), torch.where(q > 0, fq - fp + 1.0, torch.zeros_like(q))
        else:
            lm = torch.log((p + q) / 2).clamp(min=-1e4)
            value, dq = (p * (fp - lm) + q * (fq - lm)) / 2, torch.where(q > 0, (fq - lm) / 2, torch.zeros_like(q))
        kl[rows] = value.sum(1) * on[rows]
        y = s["targets"][rows].clamp(min=0)[:, None]
        logp[rows] = logq.gather(1, y)[:, 0] * on[rows]
        # by a place's probability, then through the softmax
        u = dq.gather(1, entry)
        prob = logq.exp()
        g = prob * (u - (prob * u).sum(1, keepdim=True)) + c["ce_coef"] * prob
        g.scatter_add_(1, y, torch.full(y.shape, -c["ce_coef"], **f64))
        grad[rows] = g * (w[rows] / c["temperature"])[:, None]
    return {"loss": ((kl - c["ce_coef"] * logp) * w).sum(), "kl": kl.sum() / max(1, sum(counts)), "token_kl": kl, "logp": logp,
            "dlogits": grad}


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    if c["op"] == "top":
        return _exact_top(s, c)
    if c["op"] == "distill":
        return _exact_distill(s, c)
    t = s["tokens"]
    if c["op"] == "embed":
        return torch.nn.functional.one_hot((t < 0).long(), 2)[:, :1].double() * s["weight"].double()[t.clamp(min=0)] * c["scale"]
    d = torch.zeros((c["V"], c["D"]), dtype=torch.float64, device=DEV)
    at = (t >= 0).nonzero()[:, 0]
    d.index_put_((t[at],), s["dhidden"][at].double() * c["scale"], accumulate=True)
    return d + s["grad"].double() if c["into"] == "sum" else d
