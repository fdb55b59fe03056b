"""Timed cases of the scoring operators and of the teacher cache in few bits.

Three things a distillation run does next to its loss: it scores given tokens (their
log-probability, the entropy of the distribution they were taken from and the most likely
alternatives) from logits that a server or a trunk has at hand, or straight from hidden
states and the LM head, without logits in memory, when it trains on drawn text; and it keeps
the teacher's top-K cache in 8 or 4 bits a logit, written once and read in every epoch.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) while
``own`` is false, and through this package's public calls while it is true.
"""
import math

import torch

own = False

TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = 32       # slots of a cached row that share a scale
SPAN = 4096.0    # a cached logit further below its row's largest has no probability


# ---------------------------------------------------------------- cases
def _score(name, B, V, x, top, mixed=False, pad=0):
    return {"name": name, "op": "score", "B": B, "V": V, "x": x, "top": top, "mixed": mixed, "pad": pad}


def _train(name, B, V, x, temperature):
    return {"name": name, "op": "train", "B": B, "V": V, "x": x, "temperature": temperature}


def _fused(name, T, d, V, tau, grad):
    return {"name": name, "op": "fused", "T": T, "d": d, "V": V, "tau": tau, "grad": grad}


def _cache(name, T, K, V, bits):
    return {"name": name, "op": "cache", "T": T, "K": K, "V": V, "bits": bits}


def listed():
    return [
        # one generated token with its alternatives, as a server returns them: latency
        _score("score_1x201088_top20", 1, 201088, "fp32", 20),
        # a generation batch with alternatives
        _score("score_64x201088_top20", 64, 201088, "fp32", 20),
        # a server's batch, a temperature per row, 16-bit logits
        _score("score_512x151936_mixed", 512, 151936, "bf16", 5, mixed=True),
        # an odd vocabulary inside padded rows, many alternatives (a top-K record from logits)
        _score("score_203x50261_top100", 203, 50261, "fp16", 100, pad=43),
        # policy gradient with an entropy bonus on logits in memory: both directions
        _train("train_2048x128256", 2048, 128256, "bf16", 1.0),
        # the same for a short, ragged batch in 32 bits
        _train("train_187x50261", 187, 50261, "fp32", 0.8),
        # hidden states and head, no logits in memory, both directions: a small step
        _fused("fused_256x256x4096", 256, 256, 4096, 1.0, True),
        # the same for a step of a 20-billion-parameter student's length
        _fused("fused_4096x2880x201088", 4096, 2880, 201088, 1.0, True),
        # scoring a batch of drawn text under a frozen model: forward alone, ragged
        _fused("fused_score_3001x4096x151936", 3001, 4096, 151936, 0.9, False),
        # a micro-batch's rows of the teacher cache, written and read back
        _cache("cache_500x64_8bit", 500, 64, 50261, 8),
        # one step's teacher cache
        _cache("cache_32768x100_8bit", 32768, 100, 201088, 8),
        # a long-context step's cache in 4 bits
        _cache("cache_262144x100_4bit", 262144, 100, 201088, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["score", "train", "fused", "cache"])
    if kind == "score":
        V = _log(rng, 1000, 201088)
        c = _score("", _log(rng, 1, 512), V, rng.choice(["fp32", "bf16", "fp16"]), rng.choice([0, 1, 5, 20, 64, 100, 128]),
                   mixed=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 8, 64]))
    elif kind == "train":
        B, V = _log(rng, 1, 4096), _log(rng, 1000, 201088)
        while B * V > 2048 * 128256:
            B = max(1, B // 2)
        c = _train("", B, V, rng.choice(["fp32", "bf16", "fp16"]), round(rng.uniform(0.5, 1.5), 2))
    elif kind == "fused":
        T, V, d = _log(rng, 1, 8192), _log(rng, 1000, 201088), 8 * _log(rng, 16, 512)
        while T * V * d > 4096 * 201088 * 2880:
            T = max(1, T // 2)
        c = _fused("", T, d, V, round(rng.uniform(0.5, 2.0), 2), rng.random() < 0.6)
    else:
        K = _log(rng, 1, 1024)
        T = _log(rng, 1, 262144)
        while T * K > 262144 * 100:
            T = max(1, T // 2)
        c = _cache("", T, K, _log(rng, 2048, 201088), rng.choice([8, 8, 4]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def ids(high, *shape):
        return torch.randint(0, high, shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] in ("score", "train"):
        B, V, pad = case["B"], case["V"], case.get("pad", 0)
        # logits of a language model: a wide bulk, some tens of likely tokens, some rows sharp and
        # some flat, the last ids of the vocabulary never produced
        x = normal(B, V + pad) * 1.8
        hot = ids(V - V // 200, B, 40)
        x.scatter_add_(1, hot, 6.0 + 6.0 * uniform(B, 40))
        x.mul_(0.5 + uniform(B, 1))
        x[:, V - V // 200:] = -math.inf
        s["logits"] = x.to(TYPE[case["x"]])[:, :V]
        # the given tokens: mostly likely ones
        s["tokens"] = torch.where(uniform(B) < 0.8, hot[:, 0], ids(V - V // 200, B))
    if case["op"] == "score":
        s["temperature"] = 1.0
        if case["mixed"]:
            s["temperature"] = 0.5 + uniform(case["B"])
    elif case["op"] == "train":
        B = case["B"]
        s["mask"] = uniform(B) >= 0.1  # a prompt's positions are not trained on
        s["grad_logprob"] = normal(B) / B  # advantages
        s["grad_entropy"] = torch.full((B,), -0.01 / B, device="cuda")
    elif case["op"] == "fused":
        T, d, V = case["T"], case["d"], case["V"]
        W = normal(V, d) / math.sqrt(d)
        s["tokens"] = ids(V, T)
        # hidden states after the final norm, leaning towards the token that follows
        lean = (8.0 * uniform(T, 1)) * (uniform(T, 1) < 0.7)
        s["H"] = (1.5 * normal(T, d) + lean * W[s["tokens"]]).to(torch.bfloat16)
        s["W"] = W.to(torch.bfloat16)
        s["mask"] = uniform(T) >= 0.1
        s["grad_logprob"] = normal(T) / T
        s["grad_entropy"] = torch.full((T,), -0.01 / T, device="cuda")
    elif case["op"] == "cache":
        T, K, V = case["T"], case["K"], case["V"]
        # a teacher's largest logits, in order, a few slots without a logit
        z = normal(T, K) * (1.0 + uniform(T, 1)) + 8.0
        z = torch.sort(z, dim=1, descending=True).values
        if K > 1:
            z[:, 1:].masked_fill_(uniform(T, K - 1) < 0.001, -math.inf)
        s["logits"] = z
        s["ids"] = ids(V, T, K).to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms
def _row_terms(x, temperature):
    """log q, q (0 where a logit is -inf), and q log q of rows of logits."""
    x = x / temperature
    m = x.amax(dim=1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logq = z - torch.log(total)
    q = e / total
    return logq, q, torch.where(q > 0, q * logq, torch.zeros_like(q))


def _plain_score(s):
    c = s["case"]
    x = s["logits"].float()
    t = s["temperature"]
    t = t[:, None] if isinstance(t, torch.Tensor) else t
    logq, q, qlogq = _row_terms(x, t)
    out = {"logprob": logq.gather(1, s["tokens"][:, None])[:, 0], "entropy": -qlogq.sum(1)}
    if c["top"]:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_ids"] = order.to(torch.int32)
        out["top_logprobs"] = logq.gather(1, order)
    return out


def _plain_train(s):
    c = s["case"]
    x = s["logits"].float()
    logq, q, qlogq = _row_terms(x, c["temperature"])
    keep = s["mask"].float()
    logprob = logq.gather(1, s["tokens"][:, None])[:, 0]
    entropy = -qlogq.sum(1)
    a = (s["grad_logprob"] * keep)[:, None]
    b = (s["grad_entropy"] * keep)[:, None]
    dx = -a * q - b * (qlogq + q * entropy[:, None])
    dx.scatter_add_(1, s["tokens"][:, None], a)
    return {"logprob": torch.where(s["mask"], logprob, torch.zeros_like(logprob)),
            "entropy": torch.where(s["mask"], entropy, torch.zeros_like(entropy)),
            "grad": (dx / c["temperature"]).to(TYPE[c["x"]])}


def _plain_fused(s):
    c = s["case"]
    H, W = s["H"].float(), s["W"].float()
    x = torch.matmul(H, W.t())
    logq, q, qlogq = _row_terms(x, c["tau"])
    del x
    logprob = logq.gather(1, s["tokens"][:, None])[:, 0]
    del logq
    entropy = -qlogq.sum(1)
    keep = s["mask"]
    out = {"logprob": torch.where(keep, logprob, torch.zeros_like(logprob)),
           "entropy": torch.where(keep, entropy, torch.zeros_like(entropy))}
    if c["grad"]:
        a = (s["grad_logprob"] * keep)[:, None]
        b = (s["grad_entropy"] * keep)[:, None]
        ds = qlogq.addcmul_(q, entropy[:, None]).mul_(-b)
        ds.sub_(q.mul_(a))
        ds.scatter_add_(1, s["tokens"][:, None], a)
        ds.div_(c["tau"])
        out["dH"] = torch.matmul(ds, W).to(torch.bfloat16)
        out["dW"] = torch.matmul(ds.t(), H).to(torch.bfloat16)
    return out


def _plain_cache(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    levels = float(2 ** c["bits"] - 2)  # the last code stands for -inf
    z = s["logits"]
    z = torch.where(z < z.amax(dim=1, keepdim=True) - SPAN, torch.full_like(z, -math.inf), z)
    pad = -K % GROUP
    if pad:
        z = torch.cat([z, torch.full((T, pad), -math.inf, device=z.device)], 1)
    z = z.reshape(T, -1, GROUP)
    has = z > -math.inf
    top = z.amax(dim=2, keepdim=True)
    low = torch.where(has, z, torch.full_like(z, math.inf)).amin(dim=2, keepdim=True)
    some = top > -math.inf
    top = torch.where(some, top, torch.zeros_like(top))
    span = torch.where(some, top - low, torch.zeros_like(top))
    step = span / levels
    # the nearest level, also where a logit lies next to the middle of two: in 64 bits
    wide = torch.where(some, top.double() - low.double(), torch.zeros_like(top, dtype=torch.float64))
    code = torch.where((span > 0) & has, torch.round((top.double() - z.double()) * levels / wide), torch.zeros_like(z, dtype=torch.float64))
    code = code.float()
    value = torch.where(has, top - code * step, torch.full_like(z, -math.inf))
    return {"ids": s["ids"].clone(), "logits": value.reshape(T, -1)[:, :K].contiguous()}


def run(s):
    c = s["case"]
    if not own:
        return {"score": _plain_score, "train": _plain_train, "fused": _plain_fused, "cache": _plain_cache}[c["op"]](s)
    import lm_head_top_tcgen05_gb300 as fkl

    if c["op"] == "score":
        r = fkl.token_logprobs(s["logits"], s["tokens"], temperature=s["temperature"], top_n=c["top"])
        out = {"logprob": r.logprob, "entropy": r.entropy}
        if c["top"]:
            out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
        return out
    if c["op"] == "train":
        x = s["logits"].detach().requires_grad_()
        r = fkl.token_logprobs(x, s["tokens"], temperature=c["temperature"], mask=s["mask"])
        grad, = torch.autograd.grad((r.logprob, r.entropy), (x,), (s["grad_logprob"], s["grad_entropy"]))
        return {"logprob": r.logprob.detach(), "entropy": r.entropy.detach(), "grad": grad}
    if c["op"] == "fused":
        if not c["grad"]:
            logprob, entropy = fkl.fused_logprobs(s["H"], s["W"], s["tokens"], s["mask"], tau=c["tau"])
            return {"logprob": logprob, "entropy": entropy}
        H, W = s["H"].detach().requires_grad_(), s["W"].detach().requires_grad_()
        logprob, entropy = fkl.fused_logprobs(H, W, s["tokens"], s["mask"], tau=c["tau"])
        dH, dW = torch.autograd.grad((logprob, entropy), (H, W), (s["grad_logprob"], s["grad_entropy"]))
        return {"logprob": logprob.detach(), "entropy": entropy.detach(), "dH": dH, "dW": dW}
    cache = fkl.quantize_cache(s["ids"], s["logits"], c["V"], bits=c["bits"])
    ids, logits = fkl.dequantize_cache(cache)
    return {"ids": ids, "logits": logits}


# ---------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "score":
        B, V = case["B"], case["V"]
        # one read of the logits; a subtraction, an exponential and two sums for each
        return {"bytes": B * V * SIZE[case["x"]] + B * (8 + 8 + 8 * case["top"] + (4 if case["mixed"] else 0)),
                "flops": 5 * B * V}
    if case["op"] == "train":
        B, V = case["B"], case["V"]
        # the softmax's sums first, then its gradient: the logits are read in each direction
        return {"bytes": 3 * B * V * SIZE[case["x"]] + B * 33, "flops": 11 * B * V}
    if case["op"] == "fused":
        T, d, V = case["T"], case["d"], case["V"]
        # the projection; for the gradients the projection again (no logits in memory) and two products
        way = 4 if case["grad"] else 1
        return {"bytes": (2 if case["grad"] else 1) * 2 * (T * d + V * d) + T * 25, "flops": way * 2 * T * V * d}
    T, K = case["T"], case["K"]
    bits = max(1, case["V"].bit_length())
    words = 2 * -(-K // GROUP) + -(-K * case["bits"] // 32) + -(-K * bits // 32)
    # ids and logits read, the record written; the record read, ids and logits written
    return {"bytes": 2 * T * (8 * K + 4 * words), "flops": 8 * T * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "cache":
        # what the record stands for: the levels between each 32 slots' largest and smallest logit
        out = torch.empty(case["T"], case["K"], dtype=torch.float64, device="cuda")
        last = 2 ** case["bits"] - 2
        z = s["logits"].double()
        z = z.masked_fill(z < z.max(dim=1).values.unsqueeze(1) - SPAN, -math.inf)
        for at in range(0, case["K"], GROUP):
            part = z[:, at:at + GROUP]
            high = part.max(dim=1).values.unsqueeze(1)
            deep = part.masked_fill(torch.isneginf(part), math.inf).min(dim=1).values.unsqueeze(1)
            n = ((high - part) * last / (high - deep)).nan_to_num(nan=0.0, posinf=0.0).round()
            out[:, at:at + GROUP] = (high - n * (high - deep) / last).masked_fill(torch.isneginf(part), -math.inf)
        return {"ids": s["ids"], "logits": out}
    if op == "fused":
        T, d, V = case["T"], case["d"], case["V"]
        if 2.0 * T * V * d * (3 if case["grad"] else 1) > 3e12 or T * V > 2e9:
            return None
        x = s["H"].double() @ s["W"].double().t()
        scale, on = case["tau"], s["mask"]
    else:
        if case["B"] * case["V"] > 3e8:
            return None
        x = s["logits"].double()
        scale, on = (s["temperature"] if op == "score" else case["temperature"]), s.get("mask")
    scale = scale.double().unsqueeze(1) if isinstance(scale, torch.Tensor) else scale
    lse = torch.logsumexp(x / scale, dim=1)
    rows = torch.arange(x.shape[0], device=x.device)
    logprob = x[rows, s["tokens"]] / (scale.squeeze(1) if isinstance(scale, torch.Tensor) else scale) - lse
    p = torch.softmax(x / scale, dim=1)
    entropy = torch.special.entr(p).sum(dim=1)
    if on is not None:
        out = {"logprob": logprob * on, "entropy": entropy * on}
    else:
        out = {"logprob": logprob, "entropy": entropy}
    if op == "score" and case["top"]:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
        out["top_ids"] = order.to(torch.int32)
        out["top_logprobs"] = torch.gather(x / scale, 1, order) - lse.unsqueeze(1)
    if op == "train" or (op == "fused" and case["grad"]):
        gl = s["grad_logprob"].double() * on
        ge = s["grad_entropy"].double() * on
        # d entropy / d logit = p (entr(p)/p - entropy), entr(p) = -p log p
        ds = (torch.special.entr(p) - p * entropy.unsqueeze(1)) * ge.unsqueeze(1) - p * gl.unsqueeze(1)
        ds[rows, s["tokens"]] += gl
        ds /= scale
        if op == "train":
            out["grad"] = ds
        else:
            out["dH"], out["dW"] = ds @ s["W"].double(), ds.t() @ s["H"].double()
    return out
