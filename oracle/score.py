"""Float64 CPU oracle of the scoring operators and of the teacher cache in few bits.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (same rules as ``oracle/dense_kl.py``).

    score   z = x / T, logprob = z_tok - logsumexp(z), entropy = -sum q log q, gradients, alternatives
    cache   ids of id_bits, codes of the nearest of 2^bits - 1 levels between 32 slots' largest and smallest
"""
from __future__ import annotations

import numpy as np

SPAN = 4096.0
GROUP = 32


def score(x, tokens, temperature=1.0, mask=None):
    """(logprob, entropy, logq [B, V], q [B, V]) in float64.  NaN logits count as -inf, +inf ids share all."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    B, V = x.shape
    T = np.broadcast_to(np.asarray(temperature, dtype=np.float64), (B,))
    logprob, entropy = np.empty(B), np.empty(B)
    logq, q = np.full((B, V), np.nan), np.full((B, V), np.nan)
    for b in range(B):
        if mask is not None and not mask[b]:
            logprob[b] = entropy[b] = 0.0
            continue
        m = x[b].max()
        if m == -np.inf or not (np.isfinite(T[b]) and T[b] > 0):
            logprob[b] = entropy[b] = np.nan
            continue
        if m == np.inf:
            z = np.where(x[b] == np.inf, 0.0, -np.inf)
        else:
            z = (x[b] - m) / T[b]
        s = z - np.log(np.exp(z).sum())
        p = np.exp(s)
        logq[b], q[b] = s, p
        entropy[b] = -(p[p > 0] * s[p > 0]).sum()
        logprob[b] = s[tokens[b]] if 0 <= tokens[b] < V else np.nan
    return logprob, entropy, logq, q


def score_gradient(logq, q, entropy, tokens, grad_logprob, grad_entropy, temperature=1.0, mask=None):
    """d sum_b (a_b logprob_b + b_b entropy_b) / d x, float64 [B, V]; NaN rows as documented."""
    B, V = q.shape
    T = np.broadcast_to(np.asarray(temperature, dtype=np.float64), (B,))
    dx = np.zeros((B, V))
    for b in range(B):
        if mask is not None and not mask[b]:
            continue
        if not 0 <= tokens[b] < V or np.isnan(entropy[b]):
            dx[b] = np.nan
            continue
        safe = np.where(q[b] > 0, logq[b], 0.0)
        dx[b] = -grad_logprob[b] * q[b] - grad_entropy[b] * q[b] * (safe + entropy[b])
        dx[b, tokens[b]] += grad_logprob[b]
        dx[b] /= T[b]
    return dx


def alternatives(row, n):
    """Ids of the row's n largest logits above -inf, largest first, ties by the lower id; -1 beyond them."""
    row = np.asarray(row, dtype=np.float64)
    ids = np.flatnonzero(row > -np.inf)  # NaN compares false
    ids = ids[np.lexsort((ids, -row[ids]))][:n]
    return np.concatenate([ids, np.full(n - ids.size, -1, dtype=ids.dtype)])


# ---------------------------------------------------------------- the cache's format, bit by bit
def id_bits(V):
    return max(1, int(V).bit_length())


def cache_words(K, V, bits):
    return 2 * -(-K // GROUP) + -(-K * bits // 32) + -(-K * id_bits(V) // 32)


def _bits(values, width):
    """Values of `width` bits one after the other, as 32-bit words."""
    stream = sum(int(v) << (k * width) for k, v in enumerate(values))
    return [(stream >> (32 * i)) & 0xFFFFFFFF for i in range(-(-len(values) * width // 32))]


def cache_pack(ids, logits, V, bits):
    """uint32 [T, words]."""
    ids, logits = np.asarray(ids), np.asarray(logits, dtype=np.float32)
    T, K = ids.shape
    levels, none, no_id = 2 ** bits - 2, 2 ** bits - 1, 2 ** id_bits(V) - 1
    out = np.zeros((T, cache_words(K, V, bits)), dtype=np.uint32)
    for t in range(T):
        z = logits[t]
        bad = np.isnan(z).any() or (z == np.inf).any()
        least = np.float32(-np.inf) if bad or not (z > -np.inf).any() else z.max() - np.float32(SPAN)
        scales, codes = [], []
        for k in range(0, K, GROUP):
            part = z[k:k + GROUP]
            has = np.zeros(part.shape, bool) if bad else (part > -np.inf) & (part >= least)
            top = part[has].max() if has.any() else np.float32(0)
            low = part[has].min() if has.any() else np.float32(0)
            step = np.float32(top - low) / np.float32(levels)
            scales += [np.float32(np.nan) if bad else top, step]
            for v, ok in zip(part, has):
                wide = float(top) - float(low)
                codes.append(none if not ok else 0 if wide == 0 else int(np.rint((float(top) - float(v)) * levels / wide)))
        stored = [int(i) if 0 <= i < V else no_id for i in ids[t]]
        out[t] = np.concatenate([np.array(scales, dtype=np.float32).view(np.uint32),
                                 np.array(_bits(codes, bits) + _bits(stored, id_bits(V)), dtype=np.uint32)])
    return out


def cache_unpack(records, K, V, bits):
    """(ids int32 [T, K], logits float32 [T, K])."""
    records = np.asarray(records, dtype=np.uint32)
    T, G = records.shape[0], -(-K // GROUP)
    cw, ib = -(-K * bits // 32), id_bits(V)

    def take(words, width):
        stream = sum(int(w) << (32 * i) for i, w in enumerate(words))
        return [(stream >> (k * width)) & (2 ** width - 1) for k in range(K)]

    ids, logits = np.empty((T, K), dtype=np.int32), np.empty((T, K), dtype=np.float32)
    for t in range(T):
        scales = records[t, :2 * G].view(np.float32)
        for k, (c, i) in enumerate(zip(take(records[t, 2 * G:2 * G + cw], bits), take(records[t, 2 * G + cw:], ib))):
            top, step = scales[2 * (k // GROUP)], scales[2 * (k // GROUP) + 1]
            none = c == 2 ** bits - 1 and not np.isnan(top)
            logits[t, k] = np.float32(-np.inf) if none else np.float32(top - np.float32(np.float32(c) * step))
            ids[t, k] = i if i < V else -1
    return ids, logits
