"""Plain fp64 reference of the serving operators on a dense cache.

TEST INFRASTRUCTURE ONLY.  Only the test-suite imports this module; the library
never calls it and it imports nothing from the library.

  * attend: one query's softmax attention over a set of tokens, from the
    textbook formula; no tokens give a zero output.
  * window_attention: query i of row b stands at p = len_b - n_q + i and sees the
    tokens t <= p with t < sinks or t > p - window.
  * decode_weights: the attention weight every token of a KV head receives from
    the head's query group.
  * evict: the kept positions of every row and KV head.
  * error_bound: how far an evaluation with exact products of the bf16 inputs,
    fp32 accumulation and fp32 softmax may be from these values.
"""

from __future__ import annotations

import numpy as np


def attend(q, k, v, scale):
    """(output [d], weights [t], sum_t p_t |v_t| [d]) of one query."""
    if len(k) == 0:
        z = np.zeros(v.shape[-1])
        return z, np.zeros(0), z
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p, p @ np.abs(v)


def visible(pos, window, sinks):
    """Positions that the query at `pos` sees, ascending."""
    t = np.arange(max(0, pos + 1))
    return t[(t < sinks) | (pos - t < window)]


def score_size(q, k, scale):
    """The largest sum of |products| of a score: what its rounding errors scale with."""
    return 0.0 if len(k) == 0 else scale * (np.abs(k) @ np.abs(q)).max()


def error_bound(size, absv, ref, d, bf16, p_bits=24):
    """Elementwise bound.  A score is d exact products accumulated in d / 16
    tensor-core steps, each off by at most 2^-22 of the running sum of
    magnitudes (truncated alignment), `size` in all; an error e of the scores
    changes every weight by a factor within 1 +- 2 e (numerator and sum).  exp2,
    the normalisation and the fp32 sums add at most 2^-19, weights rounded to
    p_bits bits 2^-p_bits; all of it relative to sum p |v|.  A bf16 output adds
    half a step of its own."""
    rel = 2 * (d / 16) * 2.0**-22 * size + 2.0**-19 + (2.0**-p_bits if p_bits < 24 else 0.0)
    return rel * absv * (1 + 2.0**-8) + (2.0**-8 if bf16 else 2.0**-24) * np.abs(ref)


def window_attention(q, k, v, lens, window, sinks, scale, bf16=False, p_bits=24):
    """q [B, Hq, n_q, d], k, v [B, Hkv, T, d] -> (out, bound)."""
    B, Hq, n_q, d = q.shape
    G = Hq // k.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        for i in range(n_q):
            t = visible(int(lens[b]) - n_q + i, window, sinks)
            for h in range(Hq):
                kk, vv = k[b, h // G][t], v[b, h // G][t]
                o, _, absv = attend(q[b, h, i], kk, vv, scale)
                out[b, h, i] = o
                tol[b, h, i] = error_bound(score_size(q[b, h, i], kk, scale), absv, o, d, bf16, p_bits)
    return out, tol


def decode_weights(q, k, v, lens, scale):
    """q [B, Hq, d] -> (weights [B, Hkv, T], their bound)."""
    B, Hq, d = q.shape
    Hkv, T = k.shape[1:3]
    w, tol = np.zeros((B, Hkv, T)), np.zeros((B, Hkv, T))
    for b in range(B):
        n = int(lens[b])
        for h in range(Hq):
            kv = h * Hkv // Hq
            _, p, _ = attend(q[b, h], k[b, kv, :n], v[b, kv, :n], scale)
            rel = 2 * (d / 16) * 2.0**-22 * score_size(q[b, h], k[b, kv, :n], scale) + 2.0**-19
            w[b, kv, :n] += p
            tol[b, kv, :n] += rel * p
    return w, tol


def prefix_attention(q, kp, vp, k, v, lens, scale, bf16=False, p_bits=24):
    """q [B, Hq, d], kp, vp [Hkv, P, d], k, v [B, Hkv, T, d] -> (out, bound)."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        for h in range(Hq):
            kv, n = h * Hkv // Hq, int(lens[b])
            kk, vv = np.concatenate([kp[kv], k[b, kv, :n]]), np.concatenate([vp[kv], v[b, kv, :n]])
            o, _, absv = attend(q[b, h], kk, vv, scale)
            out[b, h] = o
            tol[b, h] = error_bound(score_size(q[b, h], kk, scale), absv, o, d, bf16, p_bits)
    return out, tol


def evict(weights, lens, keep, sinks, recent):
    """Kept positions per (row, KV head): a list of lists, ascending."""
    out = []
    for b in range(weights.shape[0]):
        n = int(lens[b])
        for h in range(weights.shape[1]):
            if n <= keep:
                out.append(list(range(n)))
                continue
            w = np.nan_to_num(weights[b, h, :n], nan=0.0, posinf=np.inf)
            w = np.maximum(w, 0.0)
            always = [t for t in range(n) if t < sinks or t >= n - recent]
            rest = [t for t in range(n) if not (t < sinks or t >= n - recent)]
            rest.sort(key=lambda t: (-w[t], t))
            out.append(sorted(always + rest[:keep - len(always)]))
    return out
