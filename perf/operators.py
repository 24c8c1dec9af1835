"""Cases of the serving operators on a dense bf16 cache, beside their plain forms.

Four operators, each reached through rank_bit_kv_b200.kvc:

- ``window_attn``: attention of the last n_q tokens of every row with a causal
  sliding window and a few first tokens (sinks) that stay visible;
- ``decode_accum``: single-token decode attention that also adds each cached
  token's attention weight to a running sum per KV head;
- ``evict``: keeps, per KV head, the tokens with the largest running sums (and
  the first and the most recent ones) and compacts the cache to them;
- ``prefix_decode``: single-token decode of a batch whose rows share one long
  prefix, stored once, followed by each row's own tokens.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the library.  ``exact`` computes it in
64 bits from the definition.
"""

import math

import torch

own = False


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # one sequence, one new token: the latency of a single-stream chat
        dict(name="window_token_b1", op="window", B=1, Hq=32, Hkv=8, d=128, T=4096, n_q=1,
             window=1024, sinks=4, ragged=False, bf16=False),
        # a served batch deep into a long context, rows of unequal length
        dict(name="window_token_b16_64k", op="window", B=16, Hq=32, Hkv=8, d=128, T=65536, n_q=1,
             window=8192, sinks=16, ragged=True, bf16=True),
        # a chunk of a chunked prefill, odd sizes, 7 query heads per KV head of width 64
        dict(name="window_chunk_odd_d64", op="window", B=3, Hq=14, Hkv=2, d=64, T=2777, n_q=201,
             window=301, sinks=7, ragged=True, bf16=True),
        # the prefill of a whole prompt
        dict(name="window_prefill_8k", op="window", B=1, Hq=32, Hkv=8, d=128, T=8192, n_q=8192,
             window=2048, sinks=4, ragged=False, bf16=True),
        # one sequence whose cache is to be trimmed later
        dict(name="accum_b1_2k", op="accum", B=1, Hq=32, Hkv=8, d=128, T=2048, ragged=False,
             bf16=False),
        # no grouping, width 64, odd and unequal lengths
        dict(name="accum_b5_odd_d64", op="accum", B=5, Hq=12, Hkv=12, d=64, T=9001, ragged=True,
             bf16=False),
        # a served batch at 32K tokens
        dict(name="accum_b8_32k", op="accum", B=8, Hq=32, Hkv=8, d=128, T=32768, ragged=False,
             bf16=True),
        # trimming one sequence to a quarter
        dict(name="evict_b1_4k", op="evict", B=1, Hkv=8, d=128, T=4096, keep=1024, sinks=4,
             recent=256, ragged=False),
        # trimming a served batch, rows of unequal length
        dict(name="evict_b8_32k", op="evict", B=8, Hkv=8, d=128, T=32768, keep=8192, sinks=16,
             recent=2048, ragged=True),
        # a few requests behind a short system prompt
        dict(name="prefix_b4_1k", op="prefix", B=4, Hq=32, Hkv=8, d=128, P=1000, T=65,
             ragged=True, bf16=False),
        # a batch behind a document
        dict(name="prefix_b32_8k", op="prefix", B=32, Hq=32, Hkv=8, d=128, P=8192, T=1024,
             ragged=True, bf16=True),
        # a large batch of short answers behind a long document
        dict(name="prefix_b128_32k", op="prefix", B=128, Hq=32, Hkv=8, d=128, P=32768, T=512,
             ragged=True, bf16=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["window", "window", "accum", "evict", "prefix"])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "prefix":
        G = rng.choice([1, 2, 4, 7, 8])
    d = rng.choice([64, 128, 128])
    c = dict(op=op, Hkv=Hkv, d=d, ragged=rng.random() < 0.6)
    if op != "evict":
        c.update(Hq=G * Hkv, bf16=rng.random() < 0.6)
    budget = 1 << 22                       # tokens x KV heads of a cache, at most
    if op == "window":
        c["T"] = _log(rng, 64, 65536)
        c["B"] = min(_log(rng, 1, 32), max(1, budget // (c["T"] * Hkv)))
        c["n_q"] = 1
        if rng.random() < 0.6:             # a chunk or a whole prompt
            c["bf16"] = rng.random() < 0.85
            most = (1 << 31) // (c["B"] * c["Hq"] * c["T"])     # scores of the plain form
            c["n_q"] = min(_log(rng, 2, 8192), c["T"], max(1, most))
        c["window"] = _log(rng, 16, max(17, min(c["T"], 16384)))
        c["sinks"] = rng.choice([0, 1, 4, 16, 33, 64])
        pairs = 240 * 10**9 // (4 * c["Hq"] * d * c["B"])       # query-token pairs, at most
        c["n_q"] = max(1, min(c["n_q"], pairs // min(c["T"], c["window"] + c["sinks"])))
    elif op == "accum":
        c["T"] = _log(rng, 16, 65536)
        c["B"] = min(_log(rng, 1, 32), max(1, budget // (2 * c["T"] * Hkv)))
    elif op == "evict":
        c["T"] = _log(rng, 128, 65536)
        c["B"] = min(_log(rng, 1, 32), max(1, budget // (2 * c["T"] * Hkv)))
        c["sinks"] = rng.choice([0, 4, 16])
        c["keep"] = max(32, int(c["T"] * rng.uniform(0.05, 0.5)))
        c["recent"] = int((c["keep"] - c["sinks"]) * rng.uniform(0.0, 0.6))
    else:
        c["P"] = _log(rng, 64, 32768)
        c["T"] = _log(rng, 1, 2048)
        c["B"] = min(_log(rng, 2, 128), max(1, budget // (2 * c["T"] * Hkv)))
    return c


def _lens(case):
    """Length of every row: T, or (ragged) between T / 2 and T."""
    T, B = case["T"], case["B"]
    return [T - (b * T) // (2 * B) if case["ragged"] else T for b in range(B)]


def work(case):
    lens, Hkv, d = _lens(case), case["Hkv"], case["d"]
    row = 2 * 2 * d                        # bytes of one token's key and value of one KV head
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        read = sum(lens) * Hkv * 4                              # running sums
        # the kept rows and their sums, read and written, and their positions
        return dict(bytes=read + kept * Hkv * (2 * row + 4 + 4), flops=0)
    B, Hq = case["B"], case["Hq"]
    out = 2 if case["bf16"] else 4
    if case["op"] == "window":
        W, S, n_q = case["window"], case["sinks"], case["n_q"]
        span, pairs = 0, 0
        for n in lens:
            first = max(0, n - n_q)                             # position of the first query
            lo = max(0, first - W + 1)
            span += n - lo + min(S, lo)
            # queries whose window reaches back to the start see p + 1 tokens,
            # the others the window and the sinks before it
            x = max(first, min(n, W + S))
            pairs += (x * (x + 1) - first * (first + 1)) // 2 + (n - x) * (W + S)
        return dict(bytes=span * Hkv * row + B * Hq * n_q * d * (2 + out), flops=4 * Hq * d * pairs)
    if case["op"] == "accum":
        tokens = sum(lens)
        return dict(bytes=tokens * Hkv * (row + 8) + B * Hq * d * (2 + out), flops=4 * Hq * d * tokens)
    tokens = sum(lens)
    return dict(bytes=(tokens + case["P"]) * Hkv * row + B * Hq * d * (2 + out),
                flops=4 * Hq * d * (tokens + B * case["P"]))


# --------------------------------------------------------------------------- inputs


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _inputs(case, seed):
    """Keys, values, queries and running sums.  Keys and queries are N(0, 1)
    (scores of about unit spread after the 1/sqrt(d) scale); the first tokens'
    keys lean towards a direction that the queries share, as attention sinks
    do.  Running sums fall off as attention weights do: most of them small."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, d, T = case["B"], case["Hkv"], case["d"], case["T"]
    s = {}
    s["k"] = _normal(gen, B, Hkv, T, d).bfloat16()
    s["v"] = _normal(gen, B, Hkv, T, d).bfloat16()
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    if case["op"] in ("accum", "evict"):
        s["weights"] = 0.05 * torch.exp(1.5 * _normal(gen, B, Hkv, T))
        s["weights"] *= torch.arange(T, device="cuda") < s["lens"][:, None, None]
    if case["op"] == "evict":
        # the destination: room for a quarter more tokens than are kept
        cap = case["keep"] + case["keep"] // 4
        s["k2"] = torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, device="cuda")
        s["v2"] = torch.zeros_like(s["k2"])
        s["weights2"] = torch.zeros(B, Hkv, cap, device="cuda")
        return s
    lean = _normal(gen, Hkv, 1, d)
    lead = s["k"]
    if case["op"] == "prefix":
        s["kp"] = _normal(gen, Hkv, case["P"], d).bfloat16()
        s["vp"] = _normal(gen, Hkv, case["P"], d).bfloat16()
        lead = s["kp"]
    lead[..., :4, :] += lean.bfloat16()
    Hq, n_q = case["Hq"], case.get("n_q", 1)
    q = _normal(gen, B, Hkv, Hq // Hkv * n_q, d) + 0.3 * lean
    shape = (B, Hq, n_q, d) if case["op"] == "window" else (B, Hq, d)
    s["q"] = q.bfloat16().reshape(shape)
    s["out"] = torch.empty(shape, dtype=torch.bfloat16 if case["bf16"] else torch.float32, device="cuda")
    return s


def _cache(kvc, layout, k, v, n_tokens, lens=None):
    cache = kvc.Cache(layout)
    cache.bufs["k_dense"] = k.view(torch.uint8).reshape(-1)
    cache.bufs["v_dense"] = v.view(torch.uint8).reshape(-1)
    cache.n_tokens = n_tokens
    cache.seq_lens = lens
    return cache


def _dense(kvc, case, batch, tokens):
    return kvc.Layout(kvc.make_desc("dense", batch=batch, n_q_heads=case.get("Hq", case["Hkv"]),
                                    n_kv_heads=case["Hkv"], head_dim=case["d"], max_tokens=tokens,
                                    out_bf16=int(case.get("bf16", False))))


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # the layout, the cache over the tensors above and the workspace that a
        # serving program keeps
        from rank_bit_kv_b200 import kvc

        s["kvc"] = kvc
        s["layout"] = _dense(kvc, case, case["B"], case["T"])
        s["cache"] = _cache(kvc, s["layout"], s["k"], s["v"], case["T"],
                            s["lens"] if case["ragged"] else None)
        if case["op"] == "window":
            ws = s["layout"].window_workspace_bytes(case["T"], case["n_q"])
        elif case["op"] == "accum":
            ws = s["layout"].accum_workspace_bytes(case["T"])
        elif case["op"] == "prefix":
            s["prefix_layout"] = _dense(kvc, case, 1, case["P"])
            s["prefix"] = _cache(kvc, s["prefix_layout"], s["kp"], s["vp"], case["P"])
            ws = s["layout"].prefix_workspace_bytes(case["T"], case["P"])
        else:
            cap = s["k2"].shape[2]
            s["layout2"] = _dense(kvc, case, case["B"], cap)
            s["cache2"] = _cache(kvc, s["layout2"], s["k2"], s["v2"], 0)
            ws = 0
        s["ws"] = torch.empty(ws, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    if not own:
        return {"window": _window, "accum": _accum, "evict": _evict, "prefix": _prefix}[case["op"]](s, case)
    kvc = s["kvc"]
    if case["op"] == "window":
        kvc.window_attn(s["layout"], s["cache"], s["q"], s["out"], s["ws"], case["window"], case["sinks"])
        return s["out"]
    if case["op"] == "accum":
        kvc.decode_accum(s["layout"], s["cache"], s["q"], s["weights"], s["out"], s["ws"])
        return s["out"], s["weights"]
    if case["op"] == "evict":
        kept, lens = kvc.evict(s["layout"], s["cache"], s["layout2"], s["cache2"], s["weights"], s["weights2"],
                               case["keep"], case["sinks"], case["recent"])
        return kept, lens, s["k2"], s["v2"], s["weights2"]
    kvc.prefix_decode(s["prefix_layout"], s["prefix"], s["layout"], s["cache"], s["q"], s["out"], s["ws"])
    return s["out"]


def _softmax(x, seen):
    """Softmax over the last axis of the scores that are seen; all zero where none is."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _attend(q, k, v, seen):
    """Weights and outputs of queries [.., r, d] over keys and values [.., t, d]."""
    p = _softmax(q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1]), seen)
    return p, p @ v


def _window(s, case):
    B, Hkv, d, T, W, n_q = (case[x] for x in ("B", "Hkv", "d", "T", "window", "n_q"))
    G = case["Hq"] // Hkv
    # the tokens of a row that any of its queries sees: the span of the windows
    # and the sinks before it
    n = s["lens"].long()[:, None]
    span = min(T, W + n_q - 1)
    start = (n - span).clamp_min(0)
    at = torch.cat([torch.arange(min(case["sinks"], T), device="cuda").expand(B, -1),
                    start + torch.arange(span, device="cuda")], 1)
    once = torch.arange(at.shape[1], device="cuda") >= min(case["sinks"], T)
    once = (once | (at < start)) & (at < n)
    rows = at[:, None, :, None].expand(B, Hkv, -1, d)
    k = s["k"].gather(2, rows).float()
    v = s["v"].gather(2, rows).float() * once[:, None, :, None]
    pos = (n - n_q + torch.arange(n_q, device="cuda"))[:, :, None]
    seen = (at[:, None] <= pos) & ((at[:, None] < case["sinks"]) | (at[:, None] > pos - W)) & once[:, None]
    seen = seen[:, None, None].expand(B, 1, G, n_q, -1).reshape(B, 1, G * n_q, -1)
    _, o = _attend(s["q"].float().reshape(B, Hkv, G * n_q, d), k, v, seen)
    s["out"].copy_(o.reshape(B, case["Hq"], n_q, d))
    return s["out"]


def _accum(s, case):
    B, Hkv, d, T = (case[x] for x in ("B", "Hkv", "d", "T"))
    seen = (torch.arange(T, device="cuda") < s["lens"][:, None])[:, None, None]
    p, o = _attend(s["q"].float().reshape(B, Hkv, -1, d), s["k"].float(), s["v"].float(), seen)
    s["weights"] += p.sum(2)
    s["out"].copy_(o.reshape(B, case["Hq"], d))
    return s["out"], s["weights"]


def _evict(s, case):
    T, keep = case["T"], case["keep"]
    t = torch.arange(T, device="cuda")
    n = s["lens"].long()[:, None, None]
    w = s["weights"].masked_fill((t < case["sinks"]) | (t >= n - case["recent"]), math.inf)
    w = w.masked_fill(t >= n, -math.inf)
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :min(keep, T)]
    first = torch.sort(first.masked_fill(first >= n, T), dim=-1).values
    held = first < T
    kept = torch.full((*first.shape[:2], keep), -1, dtype=torch.int32, device="cuda")
    kept[..., :first.shape[2]] = first.masked_fill(~held, -1)
    rows = first.clamp_max(T - 1)
    for dst, src in (("k2", "k"), ("v2", "v")):
        got = s[src].gather(2, rows[..., None].expand(-1, -1, -1, case["d"]))
        s[dst][:, :, :rows.shape[2]] = torch.where(held[..., None], got, s[dst][:, :, :rows.shape[2]])
    s["weights2"].zero_()
    s["weights2"][..., :rows.shape[2]] = s["weights"].gather(2, rows) * held
    return kept, s["lens"].clamp_max(keep), s["k2"], s["v2"], s["weights2"]


def _prefix(s, case):
    B, Hkv, d, T, P = (case[x] for x in ("B", "Hkv", "d", "T", "P"))
    q = s["q"].float().reshape(B, Hkv, -1, d)
    G = q.shape[2]
    # scores against the prefix for all rows at once, then each row's own tokens
    x = (q.transpose(0, 1).reshape(Hkv, B * G, d) @ s["kp"].float().transpose(-1, -2)) / math.sqrt(d)
    x = x.reshape(Hkv, B, G, P).transpose(0, 1)
    y = q @ s["k"].float().transpose(-1, -2) / math.sqrt(d)
    seen = (torch.arange(P + T, device="cuda") - P < s["lens"][:, None])[:, None, None]
    p = _softmax(torch.cat([x, y], -1), seen)
    o = (p[..., :P].transpose(0, 1).reshape(Hkv, B * G, P) @ s["vp"].float()).reshape(Hkv, B, G, d).transpose(0, 1)
    o = o + p[..., P:] @ s["v"].float()
    s["out"].copy_(o.reshape(B, case["Hq"], d))
    return s["out"]


# --------------------------------------------------------------------------- 64 bits


def _attend64(q, k, v, allowed):
    """One head in 64 bits: weights [r, t] and outputs [r, d]."""
    e = torch.einsum("rd,td->rt", q.double(), k.double()) * q.shape[-1] ** -0.5
    e = torch.where(allowed, e, torch.full_like(e, -math.inf))
    w = torch.nan_to_num(torch.softmax(e, dim=1), nan=0.0)
    return w, torch.einsum("rt,td->rd", w, v.double())


def exact(case, seed):
    s = _inputs(case, seed)
    lens, Hkv = _lens(case), case["Hkv"]
    if case["op"] == "evict":
        return _exact_evict(case, s, lens)
    G = case["Hq"] // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if case["op"] == "accum" else None
    for b, n in enumerate(lens):
        for h in range(Hkv):
            k, v = s["k"][b, h, :n], s["v"][b, h, :n]
            heads = slice(h * G, (h + 1) * G)
            if case["op"] == "window":
                t = torch.arange(n, device="cuda")
                p = torch.arange(n - case["n_q"], n, device="cuda")[:, None]
                allowed = (t <= p) & ((t < case["sinks"]) | (p - t < case["window"]))
                for g in range(h * G, (h + 1) * G):
                    out[b, g] = _attend64(s["q"][b, g], k, v, allowed)[1]
                continue
            if case["op"] == "prefix":
                k, v = torch.cat([s["kp"][h], k]), torch.cat([s["vp"][h], v])
            allowed = torch.ones(1, len(k), dtype=torch.bool, device="cuda")
            w, out[b, heads] = _attend64(s["q"][b, heads], k, v, allowed)
            if weights is not None:
                weights[b, h, :n] += w.sum(0)
    return out if weights is None else (out, weights)


def _exact_evict(case, s, lens):
    keep = case["keep"]
    kept = torch.full((case["B"], case["Hkv"], keep), -1, dtype=torch.int32)
    order = torch.argsort(-s["weights"].double(), dim=-1, stable=True).tolist()
    for b, n in enumerate(lens):
        always = set(range(min(case["sinks"], n))) | set(range(max(0, n - case["recent"]), n))
        for h in range(case["Hkv"]):
            left = (t for t in order[b][h] if t < n and t not in always)
            chosen = sorted([*always, *(t for t, _ in zip(left, range(min(keep, n) - len(always))))])
            kept[b, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            for dst, src in (("k2", "k"), ("v2", "v"), ("weights2", "weights")):
                s[dst][b, h, :len(chosen)] = s[src][b, h, chosen]
    new = torch.tensor([min(n, keep) for n in lens], dtype=torch.int32)
    return kept, new, s["k2"].double(), s["v2"].double(), s["weights2"].double()
