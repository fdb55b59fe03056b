"""Timed cases of the generation operators: the 8-bit LM head and the sampler.

Distillation on a student's own text draws that text first: every step multiplies a few
hidden states by the LM head, held in 8-bit integers for generation, and draws one token
per row from the logits; the scoring of a prompt multiplies many rows at once.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) while
``own`` is false, and through this package's public calls while it is true.
"""
import math

import torch

own = False

OUT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ONE = 2.0 ** 40  # weight of the row's largest logit in the sampler's fixed-point sums


# ---------------------------------------------------------------- cases
def _linear(name, M, N, K, x, out):
    return {"name": name, "op": "int8_linear", "M": M, "N": N, "K": K, "x": x, "out": out}


def _sample(name, B, V, x, temperature, top_k, top_p, min_p, mixed=False, pad=0):
    return {"name": name, "op": "sample", "B": B, "V": V, "x": x, "temperature": temperature, "top_k": top_k,
            "top_p": top_p, "min_p": min_p, "mixed": mixed, "pad": pad}


def listed():
    return [
        # one sequence, one projection of the model's width: the smallest call, where latency counts
        _linear("linear_1x4096x2880", 1, 4096, 2880, "bf16", "bf16"),
        # one sequence at the LM head: bound by reading the 8-bit weights
        _linear("linear_1x201088x2880", 1, 201088, 2880, "bf16", "fp32"),
        # a small generation batch at the LM head
        _linear("linear_8x201088x2880", 8, 201088, 2880, "bf16", "fp32"),
        # a generation batch at the LM head of a wider model, fp16 hidden states
        _linear("linear_64x151936x4096", 64, 151936, 4096, "fp16", "fp32"),
        # a ragged batch, an odd vocabulary (rows of the output unaligned), an uneven depth
        _linear("linear_203x50261x1456", 203, 50261, 1456, "fp32", "fp32"),
        # scoring a prompt at the LM head: bound by the tensor cores
        _linear("linear_4096x201088x2880", 4096, 201088, 2880, "bf16", "bf16"),
        # a projection over a long prompt
        _linear("linear_8192x4096x4096", 8192, 4096, 4096, "bf16", "bf16"),
        # one sequence with the usual filters: latency
        _sample("sample_1x201088_k50_p95", 1, 201088, "fp32", 0.7, 50, 0.95, 0.0),
        # a generation batch that keeps a nucleus of the whole vocabulary
        _sample("sample_64x201088_p90", 64, 201088, "fp32", 1.0, 0, 0.9, 0.0),
        # the on-policy setting: the model's own distribution, nothing cut off
        _sample("sample_256x128256_full", 256, 128256, "fp32", 1.0, 0, 1.0, 0.0),
        # a server's batch, each row with its own settings, 16-bit logits
        _sample("sample_512x201088_mixed", 512, 201088, "bf16", 0.9, 40, 0.9, 0.02, mixed=True),
        # an odd vocabulary inside padded rows, min-p
        _sample("sample_37x50261_minp", 37, 50261, "fp16", 1.3, 0, 1.0, 0.05, pad=43),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        M, N = _log(rng, 1, 8192), _log(rng, 1024, 201088)
        K = 16 * rng.randint(32, 256)
        while M * N * K > 4096 * 201088 * 2880:
            M = max(1, M // 2)
        c = _linear("", M, N, K, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["bf16", "fp16", "fp32"]))
    else:
        c = _sample("", _log(rng, 1, 512), _log(rng, 1000, 201088), rng.choice(["fp32", "bf16", "fp16"]),
                    round(rng.uniform(0.3, 1.5), 2), rng.choice([0, 0, 1, 20, 64, 300, 2000]),
                    rng.choice([1.0, 0.5, 0.8, 0.9, 0.95, 0.99]), rng.choice([0.0, 0.0, 0.02, 0.1]),
                    mixed=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 8, 64]))
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

    if case["op"] == "int8_linear":
        M, N, K = case["M"], case["N"], case["K"]
        # hidden states after the final norm: unit variance, a few channels several times larger
        channel = 1.0 + 7.0 * (uniform(K) < 0.01)
        x = (normal(M, K) * channel).to(OUT[case["x"]])
        # the head in 8 bits, one scale per output channel, as its owner laid it out once
        w = normal(N, K) * 0.02
        scale = w.abs().amax(dim=1) / 127.0
        w.div_(scale[:, None]).round_()
        return {"case": case, "x": x, "wq": w.to(torch.int8), "w_scale": scale}
    B, V, pad = case["B"], case["V"], case["pad"]
    # logits of a language model: a wide bulk, some tens of likely tokens, some rows sharp and
    # some flat, the last ids of the vocabulary never produced
    x = normal(B, V + pad) * 1.8
    hot = torch.randint(0, V, (B, 40), generator=g, device="cuda")
    x.scatter_add_(1, hot, 6.0 + 6.0 * uniform(B, 40))
    x.mul_(0.5 + uniform(B, 1))
    x[:, V - V // 200:] = -math.inf
    logits = x.to(OUT[case["x"]])[:, :V]
    s = {"case": case, "logits": logits, "u": uniform(B), "temperature": case["temperature"],
         "top_k": case["top_k"], "top_p": case["top_p"], "min_p": case["min_p"]}
    if case["mixed"]:  # a server's rows: greedy ones, ones without each filter, others around the case's values
        t = case["temperature"] * (0.5 + uniform(B))
        s["temperature"] = torch.where(uniform(B) < 0.1, torch.zeros_like(t), t)
        k = (max(case["top_k"], 8) * (0.5 + uniform(B))).to(torch.int32)
        s["top_k"] = torch.where(uniform(B) < 0.4, torch.zeros_like(k), k)
        p = 0.5 * (case["top_p"] + uniform(B))
        s["top_p"] = torch.where(uniform(B) < 0.3, torch.ones_like(p), p)
        q = case["min_p"] * uniform(B)
        s["min_p"] = torch.where(uniform(B) < 0.5, torch.zeros_like(q), q)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_linear(s):
    x = s["x"].float()
    scale = x.abs().amax(dim=1, keepdim=True) / 127.0
    q = torch.where(scale > 0, torch.round(x / scale), torch.zeros_like(x)).clamp(-127.0, 127.0)
    y = torch.matmul(q, s["wq"].float().t())
    return (y * scale * s["w_scale"]).to(OUT[s["case"]["out"]])


def _column(v, B, dtype, device):
    if isinstance(v, torch.Tensor):
        return v.to(dtype)[:, None]
    return torch.full((B, 1), v, dtype=dtype, device=device)


def _plain_sample(s):
    x = s["logits"].float()
    B, V = x.shape
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    t = _column(s["temperature"], B, torch.float32, x.device)
    k = _column(s["top_k"], B, torch.int64, x.device)
    p = _column(s["top_p"], B, torch.float32, x.device)
    mp = _column(s["min_p"], B, torch.float32, x.device)
    greedy = ~(t > 0)
    t = torch.where(greedy, torch.ones_like(t), t)
    k = torch.where(greedy, torch.ones_like(k), torch.where((k <= 0) | (k > V), torch.full_like(k, V), k))
    m = x.amax(dim=1, keepdim=True)
    top = x == m
    z = torch.where(top, torch.zeros_like(x), (x - m) * (1.0 / t))
    e = torch.where(x > -math.inf, torch.exp(z), torch.zeros_like(x))
    # weights as whole multiples of 2^-40 of the largest one: their sums do not depend on the order
    w = (e * ONE).to(torch.int64)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    at = torch.arange(V, device=x.device)[None, :]
    ws = torch.where(at < k, ws, torch.zeros_like(ws))
    before = ws.cumsum(1) - ws
    total = ws.sum(1, keepdim=True)
    limit = torch.ceil(p.double() * total.double()).to(torch.int64)
    keep = (at < k) & ((p >= 1) | (at == 0) | (before < limit))
    kept = torch.zeros_like(keep).scatter_(1, order, keep) & ((e >= mp) | top)
    w = torch.where(kept, w, torch.zeros_like(w))
    total = w.sum(1, keepdim=True)
    r = (s["u"][:, None].double() * total.double()).to(torch.int64)
    r = torch.minimum(torch.clamp(r, min=0), total - 1)
    token = (w.cumsum(1) <= r).sum(1, keepdim=True)
    none = ~(m > -math.inf)
    token = torch.where(none, torch.zeros_like(token), token).clamp(max=V - 1)
    logprob = z.gather(1, token) - torch.log(total.float() / ONE)
    token = torch.where(none, torch.full_like(token, -1), token)
    logprob = torch.where(none, torch.full_like(logprob, math.nan), logprob)
    return token[:, 0].to(torch.int32), logprob[:, 0]


def run(s):
    if own:
        import lm_head_top_tcgen05_gb300 as fkl

        if s["case"]["op"] == "int8_linear":
            return fkl.int8_linear(s["x"], s["wq"], s["w_scale"], out_dtype=OUT[s["case"]["out"]])
        return fkl.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"])
    return _plain_linear(s) if s["case"]["op"] == "int8_linear" else _plain_sample(s)


# ---------------------------------------------------------------- work and exact values
def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "int8_linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size[case["x"]] + N * K + 4 * N + M * N * size[case["out"]],
                "flops": 2 * M * N * K}
    B, V = case["B"], case["V"]
    # one read of the logits; a subtraction, a product, an exponential and a sum for each
    return {"bytes": B * V * size[case["x"]] + 12 * B + (16 * B if case["mixed"] else 0), "flops": 4 * B * V}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int8_linear":
        if 2 * case["M"] * case["N"] * case["K"] > 2e12:
            return None
        x = s["x"].double()
        unit = x.abs().max(dim=1).values.div(127.0).unsqueeze(1)
        q = torch.nan_to_num(x / unit).round()
        rows = []
        for at in range(0, case["N"], 32768):
            w = s["wq"][at:at + 32768].double() * s["w_scale"][at:at + 32768].double().unsqueeze(1)
            rows.append(((q * unit) @ w.t()).cpu())
        return torch.cat(rows, 1)
    if case["B"] * case["V"] > 512 * 65536:
        return None
    x = s["logits"].cpu().double()
    u = s["u"].cpu().double()

    def of(name, b):
        v = s[name]
        return float(v[b]) if isinstance(v, torch.Tensor) else float(v)

    tokens, logs = [], []
    for b in range(case["B"]):
        row = x[b]
        ids = torch.arange(row.numel())[row > -math.inf]
        val, at = torch.sort(row[ids], descending=True, stable=True)
        ids = ids[at]
        T = of("temperature", b)
        k = 1 if not T > 0 else int(of("top_k", b))
        if k > 0:
            val, ids = val[:k], ids[:k]
        score = (val - val[0]) / (T if T > 0 else 1.0)
        prob = torch.softmax(score, 0)
        if of("top_p", b) < 1:
            count = 1 + int((prob.cumsum(0)[:-1] < of("top_p", b)).sum())
            score, ids = score[:count], ids[:count]
        alive = torch.exp(score) >= min(of("min_p", b), 1.0)
        ids, back = torch.sort(ids[alive])
        prob = torch.softmax(score[alive], 0)[back]
        pick = int((prob.cumsum(0) <= u[b]).sum().clamp(max=prob.numel() - 1))
        tokens.append(int(ids[pick]))
        logs.append(float(prob[pick].log()))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64)
