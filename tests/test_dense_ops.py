"""Serving operators on the dense cache: window attention with sinks, decode
with accumulated weights, eviction, shared-prefix decode.

The fp64 reference (oracle/dense_ops.py) is pinned on the CPU; the kernels are
compared with it elementwise within its bound, which is derived from the
arithmetic (exact products, fp32 accumulation and softmax, the output's
rounding)."""

import ctypes as C

import numpy as np
import pytest

from oracle import dense_ops as D
from rank_bit_kv_b200 import kvc, synth

F = 0x10000                                   # 16-byte aligned, never dereferenced


def dense(B=2, Hq=8, Hkv=2, d=128, T=64, L=1, bf16=0, scale=0.0):
    return kvc.Layout(kvc.make_desc("dense", batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d,
                                    max_tokens=T, n_layers=L, out_bf16=bf16, softmax_scale=scale))


# ----------------------------------------------------------------- reference pins (CPU)


def test_reference_window_matches_masked_sdpa():
    import torch

    rng = np.random.default_rng(0)
    B, Hq, Hkv, T, n_q, d, W, S = 2, 4, 2, 37, 11, 16, 6, 3
    q, k, v = (rng.standard_normal(s) for s in ((B, Hq, n_q, d), (B, Hkv, T, d), (B, Hkv, T, d)))
    lens = [37, 20]
    out, _ = D.window_attention(q, k, v, lens, W, S, d**-0.5)
    for b, n in enumerate(lens):
        p = np.arange(n - n_q, n)[:, None]
        t = np.arange(n)[None]
        mask = torch.from_numpy((t <= p) & ((t < S) | (t > p - W)))
        kk, vv = (torch.from_numpy(x[b, :, :n]).repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b]), kk, vv, attn_mask=mask)
        np.testing.assert_allclose(out[b], ref.numpy(), rtol=1e-10, atol=1e-12)


def test_reference_window_limits():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal(s) for s in ((1, 2, 5, 8), (1, 1, 9, 8), (1, 1, 9, 8)))
    one, _ = D.window_attention(q, k, v, [9], 1, 0, 1.0)         # only the token itself
    np.testing.assert_allclose(one[0, 0], v[0, 0, 4:9])
    full, _ = D.window_attention(q, k, v, [9], 100, 0, 1.0)
    same, _ = D.window_attention(q, k, v, [9], 2, 9, 1.0)        # everything is a sink
    np.testing.assert_allclose(full, same)
    short, _ = D.window_attention(q, k, v, [2], 100, 0, 1.0)     # queries before the first token
    assert (short[0, :, :3] == 0).all() and np.allclose(short[0, 0, 3], v[0, 0, 0])


def test_reference_weights_sum_to_the_group():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((2, 6, 8), (2, 2, 30, 8), (2, 2, 30, 8)))
    w, _ = D.decode_weights(q, k, v, [30, 7], 0.3)
    np.testing.assert_allclose(w.sum(-1), 3.0)
    assert (w[1, :, 7:] == 0).all()


def test_reference_evict_brute_force():
    rng = np.random.default_rng(3)
    w = rng.random((2, 2, 40))
    w[0, 0, 5:25] = 0.5
    for (b, h), got in zip(((0, 0), (0, 1), (1, 0), (1, 1)), D.evict(w, [40, 9], 12, 2, 3)):
        n = (40, 9)[b]
        if n <= 12:
            assert got == list(range(n))
            continue
        assert len(got) == 12 and got == sorted(got) and {0, 1, 37, 38, 39} <= set(got)
        left = set(range(2, 37)) - set(got)
        for t in set(got) & set(range(2, 37)):
            assert all((w[b, h, t], -t) > (w[b, h, x], -x) for x in left)


def test_reference_prefix_is_one_attention_over_both_parts():
    rng = np.random.default_rng(4)
    q, kp, vp = (rng.standard_normal(s) for s in ((2, 4, 8), (2, 5, 8), (2, 5, 8)))
    k, v = rng.standard_normal((2, 2, 2, 6, 8))
    out, _ = D.prefix_attention(q, kp, vp, k, v, [6, 0], 0.4)
    whole_k = np.concatenate([np.broadcast_to(kp, (2, *kp.shape)), k], 2)
    whole_v = np.concatenate([np.broadcast_to(vp, (2, *vp.shape)), v], 2)
    ref, _ = D.window_attention(q[:, :, None], whole_k, whole_v, [11, 5], 100, 0, 0.4)
    np.testing.assert_allclose(out, ref[:, :, 0])


# ----------------------------------------------------------------- refusals (CPU)


def _cs(n, **kw):
    c = kvc.CacheDesc()
    c.k_dense = c.v_dense = F
    c.n_tokens = n
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _status(st):
    return kvc.STATUS[st]


BIG = 1 << 40


def test_window_refusals():
    L, lay = kvc.lib(), dense()
    f = C.c_void_p(F)

    def call(c=None, q=f, n_q=1, window=8, sinks=0, out=f, ws=f, n=BIG, lay=lay):
        return _status(L.kvc_window_attn(lay.h if lay else None, C.byref(c if c is not None else _cs(64)), q, n_q,
                                         window, sinks, out, ws, n, None))

    assert call(lay=None) == "KVC_EINVAL"
    assert call(q=None) == "KVC_EINVAL" and call(out=None) == "KVC_EINVAL"
    assert call(n_q=0) == "KVC_EINVAL" and call(window=0) == "KVC_EINVAL" and call(sinks=-1) == "KVC_EINVAL"
    assert call(n_q=65) == "KVC_ECAPACITY" and call(c=_cs(65)) == "KVC_ECAPACITY"
    assert call(c=_cs(-1)) == "KVC_EINVAL"
    assert call(c=_cs(64, k_dense=None)) == "KVC_EINVAL"
    assert call(c=_cs(64, v_dense=F + 8)) == "KVC_EALIGN" and call(c=_cs(64, seq_lens=F + 4)) == "KVC_EALIGN"
    assert call(q=C.c_void_p(F + 2)) == "KVC_EALIGN" and call(out=C.c_void_p(F + 8)) == "KVC_EALIGN"
    assert call(c=_cs(64, layer=2)) == "KVC_EINVAL"
    assert call(ws=None) == "KVC_EWORKSPACE" and call(n=100) == "KVC_EWORKSPACE"
    assert call(ws=C.c_void_p(F + 8)) == "KVC_EALIGN"
    c1 = synth.config("c1")
    assert call(lay=kvc.Layout(kvc.desc_from_config(c1)), c=_cs(64)) == "KVC_EUNSUPPORTED"
    wide = dense(B=256, Hq=64, Hkv=64, T=1 << 20, L=8)
    assert call(lay=wide, n_q=1 << 20) == "KVC_EUNSUPPORTED"
    assert L.kvc_window_workspace_bytes(wide.h, 64, 1 << 20) == 0
    assert L.kvc_window_workspace_bytes(None, 64, 1) == 0


def test_accum_refusals():
    L, lay = kvc.lib(), dense()
    f = C.c_void_p(F)

    def call(lay=lay, c=None, w=f, n=BIG, q=f):
        return _status(L.kvc_decode_accum(lay.h, C.byref(c or _cs(64)), q, w, f, f, n, None))

    assert call(w=None) == "KVC_EINVAL" and call(w=C.c_void_p(F + 4)) == "KVC_EALIGN"
    assert call(q=None) == "KVC_EINVAL"
    assert call(n=L.kvc_window_workspace_bytes(lay.h, 64, 1)) == "KVC_EWORKSPACE"
    assert call(c=_cs(65)) == "KVC_ECAPACITY"
    assert call(lay=dense(Hq=8192, Hkv=1)) == "KVC_EUNSUPPORTED"


def test_evict_refusals():
    L = kvc.lib()
    a, b = dense(T=64), dense(T=32)
    MB = 1 << 20
    p = {n: C.c_void_p(F + i * MB) for i, n in enumerate(("w", "w2", "kept", "lens"))}
    src = _cs(64, k_dense=F + 8 * MB, v_dense=F + 9 * MB)
    dst = _cs(0, k_dense=F + 10 * MB, v_dense=F + 11 * MB)

    def call(A=a, src=src, Bl=b, dst=dst, keep=16, sinks=2, recent=4, **kw):
        x = {**p, **kw}
        return _status(L.kvc_evict(A.h, C.byref(src), Bl.h, C.byref(dst), x["w"], x["w2"], keep, sinks, recent,
                                   x["kept"], x["lens"], None))

    assert call(w=None) == "KVC_EINVAL" and call(kept=None) == "KVC_EINVAL" and call(lens=None) == "KVC_EINVAL"
    assert call(keep=0) == "KVC_EINVAL" and call(sinks=-1) == "KVC_EINVAL" and call(recent=-1) == "KVC_EINVAL"
    assert call(sinks=10, recent=7) == "KVC_EINVAL"
    assert call(keep=16, sinks=2**31 - 1, recent=2**31 - 1) == "KVC_EINVAL"
    assert call(keep=33) == "KVC_ECAPACITY"
    assert call(Bl=dense(B=3, T=32)) == "KVC_EINVAL" and call(Bl=dense(d=64, T=32)) == "KVC_EINVAL"
    assert call(Bl=dense(T=32, L=2)) == "KVC_EINVAL"
    assert call(w2=C.c_void_p(F + MB + 4)) == "KVC_EALIGN"
    # overlaps: another capacity over the same buffers, K in place but not V, sums over keys, lens over seq_lens
    over = _cs(0, k_dense=src.k_dense, v_dense=src.v_dense)
    assert call(dst=over) == "KVC_EINVAL"
    assert call(Bl=a, dst=_cs(0, k_dense=src.k_dense, v_dense=F + 11 * MB)) == "KVC_EINVAL"
    assert call(w2=C.c_void_p(src.k_dense)) == "KVC_EINVAL"
    assert call(kept=p["w"]) == "KVC_EINVAL"
    held = _cs(64, k_dense=src.k_dense, v_dense=src.v_dense, seq_lens=F + 5 * MB)
    assert call(src=held, lens=C.c_void_p(F + 5 * MB)) == "KVC_EINVAL"
    assert call(dst=_cs(0, k_dense=F + 10 * MB, v_dense=F + 10 * MB)) == "KVC_EINVAL"


def test_prefix_refusals():
    L = kvc.lib()
    lay, pre = dense(B=3), dense(B=1, T=32)
    f = C.c_void_p(F)

    def call(pre=pre, pc=None, lay=lay, c=None, n=BIG, q=f):
        return _status(L.kvc_prefix_decode(pre.h, C.byref(pc or _cs(32)), lay.h, C.byref(c or _cs(64)), q, f, f, n,
                                           None))

    assert call(q=None) == "KVC_EINVAL"
    assert call(pre=dense(B=2, T=32)) == "KVC_EINVAL"
    assert call(pre=dense(B=1, T=32, d=64)) == "KVC_EINVAL" and call(pre=dense(B=1, T=32, Hkv=4)) == "KVC_EINVAL"
    assert call(pre=dense(B=1, T=32, L=2)) == "KVC_EINVAL"
    assert call(pre=dense(B=1, T=32, scale=0.5)) == "KVC_EINVAL"
    assert call(pc=_cs(33)) == "KVC_ECAPACITY" and call(c=_cs(65)) == "KVC_ECAPACITY"
    assert call(n=L.kvc_window_workspace_bytes(lay.h, 64, 1)) == "KVC_EWORKSPACE"
    assert call(pre=kvc.Layout(kvc.desc_from_config(synth.config("c1", B=1)))) == "KVC_EUNSUPPORTED"


def test_workspace_grows_with_the_call():
    lay = dense(B=4, Hq=32, Hkv=8, T=4096, L=2)
    for f in (lambda n: lay.window_workspace_bytes(n), lambda n: lay.window_workspace_bytes(4096, n),
              lambda n: lay.accum_workspace_bytes(n), lambda n: lay.prefix_workspace_bytes(n, 4096),
              lambda n: lay.prefix_workspace_bytes(4096, n)):
        sizes = [f(n) for n in (1, 7, 128, 129, 1000, 4096)]
        assert sizes == sorted(sizes) and sizes[0] >= 256


def test_plans_stay_within_the_workspace():
    """What a call's plan uses ends inside the bytes that the size query asks for."""
    L = kvc.lib()
    fn = L.kvc_test_dense_plan_bytes
    fn.restype, fn.argtypes = C.c_int64, [C.c_void_p] + [C.c_int32] * 6
    rng = np.random.default_rng(5)
    for _ in range(3000):
        B, Hkv, G, T = (int(2 ** rng.uniform(0, x)) for x in (8, 4, 6.5, 17))
        lay = dense(B, G * Hkv, Hkv, int(rng.choice([64, 128])), T, int(rng.integers(1, 4)), int(rng.integers(0, 2)))
        n, n_q = int(rng.integers(0, T + 1)), int(min(T, 2 ** rng.uniform(0, 12)))
        W, S, layer = int(2 ** rng.uniform(0, 17)), int(rng.integers(0, 70)), int(rng.integers(0, 2))
        need = (lay.window_workspace_bytes(n, n_q), lay.accum_workspace_bytes(n), lay.prefix_workspace_bytes(n, n_q))
        for op, have in enumerate(need):
            used = fn(lay.h, op, n, n_q, W, S, layer)
            assert have == 0 or 0 <= used <= have, (B, Hkv, G, T, n, n_q, W, S, layer, op, used, have)
        # a workspace sized for longer contexts and more query tokens serves shorter ones
        assert need[0] == 0 or lay.window_workspace_bytes(n // 2, max(1, n_q // 3)) <= need[0]


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch

    lay = dense()
    cache = kvc.Cache(lay, device="cpu")
    cache.n_tokens = 64
    q = torch.zeros(2, 8, 1, 128, dtype=torch.bfloat16)
    out, ws = torch.zeros(2, 8, 1, 128), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        kvc.window_attn(lay, cache, q, out, ws, 8)
    for bad in (dict(q=q[:1]), dict(q=q.float()), dict(q=q[..., :64]), dict(out=out.bfloat16()),
                dict(q=q.transpose(0, 1)), dict(q=q[:, :, 0])):
        a = {"q": q, "out": out, **bad}
        with pytest.raises(ValueError):
            kvc.window_attn(lay, cache, a["q"], a["out"], ws, 8)
    with pytest.raises(ValueError, match="weights"):
        kvc.decode_accum(lay, cache, q[:, :, 0].contiguous(), torch.zeros(2, 2, 63), out[:, :, 0].contiguous(), ws)
    with pytest.raises(ValueError, match="dense"):
        c1 = kvc.Layout(kvc.desc_from_config(synth.config("c1")))
        kvc.window_attn(c1, kvc.Cache(c1, device="cpu"), q, out, ws, 8)


# ----------------------------------------------------------------- GPU


def _f64(t):
    return t.double().cpu().numpy()


class Problem:
    """A dense cache of random tokens; what lies past the lengths is NaN."""

    def __init__(self, B, Hq, Hkv, d, T, lens=None, cap=None, bf16=0, seed=0, L=1, stale=float("nan"), scale=0.0):
        import torch

        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims = (B, Hq, Hkv, d, T)
        cap = cap or T
        lead = (L,) if L > 1 else ()
        self.lead, self.lens = lead, [T] * B if lens is None else lens
        self.layout = dense(B, Hq, Hkv, d, cap, L, bf16, scale)
        self.scale = scale or d**-0.5
        self.cache = kvc.Cache(self.layout)
        mk = lambda: torch.randn(*lead, B, Hkv, cap, d, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.k, self.v = mk(), mk()
        for b, n in enumerate(self.lens):
            self.k[..., b, :, n:, :] = stale
            self.v[..., b, :, n:, :] = stale
        self.cache.bufs["k_dense"] = self.k.view(torch.uint8).reshape(-1)
        self.cache.bufs["v_dense"] = self.v.view(torch.uint8).reshape(-1)
        self.cache.n_tokens = T
        if lens is not None:
            self.cache.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.gen, self.bf16 = g, bf16

    def queries(self, *mid, gain=1.0):
        import torch

        B, Hq, _, d, _ = self.dims
        q = (gain * torch.randn(*self.lead, B, Hq, *mid, d, generator=self.gen, device="cuda")).bfloat16()
        out = torch.full(q.shape, float("nan"), device="cuda",
                         dtype=torch.bfloat16 if self.bf16 else torch.float32)
        return q, out

    def ws(self, n):
        import torch

        return torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")

    def window(self, q, out, window, sinks, ws=None):
        w = self.ws(self.layout.window_workspace_bytes(self.cache.n_tokens, q.shape[-2])) if ws is None else ws
        kvc.window_attn(self.layout, self.cache, q, out, w, window, sinks)
        return w


def within(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - ref) - tol
    assert (off <= 0).all(), f"{what}: {int((off > 0).sum())} of {off.size} beyond the bound, worst by {off.max():.3e} " \
                             f"(error {np.abs(got - ref).max():.3e})"


def _p_bits(bf16):
    return 8 if bf16 else 24


WINDOW = [
    # B, Hq, Hkv, d, T, lens, n_q, window, sinks, bf16
    (1, 4, 1, 128, 1, None, 1, 1, 0, 0),                      # one token
    (2, 8, 2, 128, 300, None, 1, 64, 4, 0),
    (2, 8, 2, 128, 300, [300, 1], 1, 64, 4, 1),
    (3, 8, 8, 64, 129, [129, 0, 17], 1, 1, 0, 0),             # a row without tokens; window of one
    (2, 14, 2, 64, 211, [211, 100], 1, 37, 37, 1),            # seven heads per KV head
    (1, 33, 1, 128, 70, None, 1, 1000, 0, 0),                 # 33 heads on one KV head, window past the length
    (2, 16, 1, 64, 95, [95, 94], 1, 16, 200, 0),              # sinks past the length
    (2, 8, 2, 128, 333, [333, 129], 2, 33, 5, 0),
    (2, 8, 2, 128, 333, [333, 2], 5, 33, 5, 1),               # more queries than tokens
    (1, 8, 2, 64, 90, [50], 8, 3, 2, 0),
    (2, 6, 2, 128, 200, [200, 141], 67, 50, 3, 1),
    (1, 4, 4, 128, 150, None, 150, 150, 0, 1),                # whole prompt, full causal
    (1, 8, 1, 64, 257, None, 257, 31, 9, 1),
    (2, 4, 2, 128, 140, [0, 140], 33, 20, 1, 0),
    (1, 5, 1, 128, 400, None, 129, 128, 16, 1),
    (1, 2, 1, 128, 520, [513], 300, 140, 130, 1),             # sinks of more than a tile
    (2, 12, 4, 64, 300, [300, 7], 100, 1, 0, 1),
    (1, 40, 1, 128, 160, None, 20, 24, 2, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_window_parity(case):
    B, Hq, Hkv, d, T, lens, n_q, W, S, bf16 = case
    p = Problem(B, Hq, Hkv, d, T, lens, cap=T + 5, bf16=bf16, seed=T + n_q)
    q, out = p.queries(n_q, gain=1.5)
    ws = p.window(q, out, W, S)
    ref, tol = D.window_attention(_f64(q), _f64(p.k), _f64(p.v), p.lens, W, S, p.scale, bool(bf16), _p_bits(bf16))
    within(_f64(out), ref, tol)
    assert int(ws[:4].view(dtype=__import__("torch").int32)) in (0, -1414812757)     # no wait gave up


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,bf16", [(1, 0), (1, 1), (7, 0), (200, 1), (200, 0)])
def test_window_long_context(n_q, bf16):
    """Long contexts split over blocks: against the definition in 64 bits on the GPU."""
    import torch

    p = Problem(2, 8, 2, 128, 9001, [9001, 4097], cap=9100, bf16=bf16, seed=5)
    q, out = p.queries(n_q, gain=2.0)
    for W, S in ((5000, 20), (9001, 0), (17, 3)):
        out.fill_(float("nan"))
        p.window(q, out, W, S)
        for b, n in enumerate(p.lens):
            pos = torch.arange(n - n_q, n, device="cuda")[:, None]
            t = torch.arange(n, device="cuda")
            seen = (t <= pos) & ((t < S) | (t > pos - W))
            for h in range(8):
                k, v = p.k[b, h // 4, :n].double(), p.v[b, h // 4, :n].double()
                s = (q[b, h].double() @ k.T * p.scale).masked_fill(~seen, -float("inf"))
                pr = torch.softmax(s, -1)
                ref, absv = pr @ v, pr @ v.abs()
                size = float((q[b, h].double().abs() @ k.abs().T).max() * p.scale)
                tol = D.error_bound(size, _f64(absv), _f64(ref), 128, bool(bf16), _p_bits(bf16))
                within(_f64(out[b, h]), _f64(ref), tol, f"W {W} row {b} head {h}")


@pytest.mark.gpu
def test_window_large_scores_and_one_dominant_token():
    p = Problem(1, 8, 2, 128, 700, bf16=0, seed=9)
    q, out = p.queries(3, gain=1.0)
    p.k[0, 0, 450] = 12 * q[0, 1, 1]                         # a score of about 130
    q *= 8
    p.window(q, out, 400, 8)
    ref, tol = D.window_attention(_f64(q), _f64(p.k), _f64(p.v), p.lens, 400, 8, p.scale)
    within(_f64(out), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,bf16,bad", [(6, 0, float("nan")), (6, 1, float("inf")), (150, 1, float("nan")),
                                          (150, 1, float("inf")), (150, 0, -float("inf"))])
def test_window_non_finite_value_reaches_only_the_queries_that_see_it(n_q, bf16, bad):
    p = Problem(1, 4, 2, 128, 320, bf16=bf16, seed=3)
    at = 320 - n_q // 2                                     # seen by the later queries
    p.v[0, 1, at, 5] = bad
    q, out = p.queries(n_q)
    W = n_q // 3 + 1
    p.window(q, out, W, 2)
    v = _f64(p.v)
    v[0, 1, at, 5] = 0.0
    ref, tol = D.window_attention(_f64(q), _f64(p.k), v, p.lens, W, 2, p.scale, bool(bf16), _p_bits(bf16))
    got = _f64(out)
    pos = np.arange(320 - n_q, 320)
    sees = (pos >= at) & (pos - at < W)
    assert sees.any() and not sees.all()
    assert not np.isfinite(got[0, 2:, sees, 5]).any()
    clean = np.ones(got.shape, bool)
    clean[0, 2:, sees] = False
    within(got[clean], ref[clean], tol[clean])


@pytest.mark.gpu
def test_window_non_finite_key_reaches_only_the_queries_that_see_it():
    p = Problem(1, 2, 1, 64, 200, bf16=1, seed=4)
    p.k[0, 0, 120, 3] = float("nan")
    q, out = p.queries(150)
    p.window(q, out, 10, 0)
    got, pos = _f64(out), np.arange(50, 200)
    sees = (pos >= 120) & (pos < 130)
    assert np.isnan(got[0, :, sees]).all() and np.isfinite(got[0, :, ~sees]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n_q", [1, 40])
def test_window_layers(n_q):
    p = Problem(2, 4, 2, 64, 130, [130, 61], L=3, bf16=1, seed=6)
    q, out = p.queries(n_q)
    p.window(q, out, 40, 4)
    for l in range(3):
        ref, tol = D.window_attention(_f64(q[l]), _f64(p.k[l]), _f64(p.v[l]), p.lens, 40, 4, p.scale, True, 8)
        within(_f64(out[l]), ref, tol, f"layer {l}")
    p.cache.layer = 2
    one = out[1].clone().fill_(0)
    p.window(q[1].contiguous(), one, 40, 4)
    ref, tol = D.window_attention(_f64(q[1]), _f64(p.k[1]), _f64(p.v[1]), p.lens, 40, 4, p.scale, True, 8)
    within(_f64(one), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,bf16", [(1, 0), (1, 1), (300, 1)])
def test_window_calls_repeat_bitwise_and_leave_the_rest_alone(n_q, bf16):
    import torch

    p = Problem(2, 8, 2, 128, 2000, [2000, 1501], bf16=bf16, seed=8)
    q, _ = p.queries(n_q)
    room = torch.full((q.numel() + 512,), 7.0, device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    out = room[256:-256].view(q.shape)
    k, v = p.k.clone(), p.v.clone()
    p.window(q, out, 900, 4)
    first = out.clone()
    p.window(q, out, 900, 4)
    assert torch.equal(first, out)
    assert (room[:256] == 7).all() and (room[-256:] == 7).all()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(k, p.k) and same(v, p.v)


ACCUM = [
    # B, Hq, Hkv, d, T, lens, bf16
    (1, 4, 1, 128, 1, None, 0),
    (2, 8, 2, 128, 300, [300, 0], 0),
    (2, 14, 2, 64, 517, [517, 16], 1),
    (1, 33, 1, 128, 257, None, 0),
    (3, 4, 4, 64, 1025, [1024, 1025, 3], 0),
    (1, 20, 2, 128, 2300, None, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ACCUM, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_accum_parity(case):
    import torch

    B, Hq, Hkv, d, T, lens, bf16 = case
    p = Problem(B, Hq, Hkv, d, T, lens, cap=T + 3, bf16=bf16, seed=T)
    w = torch.rand(B, Hkv, T + 3, generator=p.gen, device="cuda")
    w0 = _f64(w)
    ws = p.ws(p.layout.accum_workspace_bytes(T))
    want, tol = w0.copy(), np.zeros(w0.shape)
    for step in range(2):
        q, out = p.queries(gain=1.5)
        kvc.decode_accum(p.layout, p.cache, q, w, out, ws)
        ref, bound = D.window_attention(_f64(q)[:, :, None], _f64(p.k), _f64(p.v), p.lens, T, 0, p.scale, bool(bf16), _p_bits(bf16))
        within(_f64(out), ref[:, :, 0], bound[:, :, 0], f"step {step}")
        dw, dt = D.decode_weights(_f64(q), _f64(p.k), _f64(p.v), p.lens, p.scale)
        want += dw
        tol += dt + 2.0**-24 * want                          # the addition's own rounding
        within(_f64(w), want, tol, f"weights after step {step}")
    for b, n in enumerate(p.lens):
        assert np.array_equal(_f64(w)[b, :, n:], w0[b, :, n:])


@pytest.mark.gpu
def test_accum_long_context_sums_to_the_group():
    import torch

    p = Problem(2, 8, 2, 128, 40000, [40000, 33333], bf16=1, seed=11)
    q, out = p.queries(gain=2.0)
    w = torch.zeros(2, 2, 40000, device="cuda")
    kvc.decode_accum(p.layout, p.cache, q, w, out, p.ws(p.layout.accum_workspace_bytes(40000)))
    plain = torch.empty_like(out)
    p.window(q[:, :, None].contiguous(), plain[:, :, None], 40000, 0)
    # the same sums in another order, then rounded: at most one step of bf16 apart
    assert ((out.double() - plain.double()).abs() <= 2.0**-7 * plain.double().abs() + 1e-5).all()
    np.testing.assert_allclose(_f64(w).sum(-1), 4.0, rtol=1e-5)
    for b, n in enumerate(p.lens):
        for h in range(2):
            s = q[b, 4 * h:4 * h + 4].double() @ p.k[b, h, :n].double().T * p.scale
            ref = torch.softmax(s, -1).sum(0)
            assert ((w[b, h, :n].double() - ref).abs() <= 2e-5 * ref).all()
        assert (w[b, :, n:] == 0).all()


EVICT = [
    # B, Hkv, d, T, lens, keep, sinks, recent, spread
    (1, 1, 128, 1, None, 1, 0, 0, "random"),
    (2, 2, 128, 300, None, 64, 4, 16, "random"),
    (2, 2, 64, 300, [300, 64], 64, 4, 16, "random"),          # one row already fits
    (3, 2, 64, 257, [257, 0, 100], 50, 0, 0, "ties"),
    (2, 3, 128, 999, [999, 500], 333, 1, 332, "random"),      # nothing but protected tokens
    (1, 2, 128, 5000, None, 1, 0, 0, "random"),
    (1, 2, 128, 5000, None, 4999, 0, 0, "same"),
    (2, 1, 64, 2048, [2048, 2047], 2046, 7, 100, "odd"),
    (1, 1, 64, 60001, None, 20000, 4, 1000, "random"),        # sums beyond shared memory
]


def _sums(kind, shape, gen):
    import torch

    if kind == "ties":
        return torch.randint(0, 4, shape, generator=gen, device="cuda").float() / 4
    if kind == "same":
        return torch.full(shape, 0.25, device="cuda")
    w = torch.rand(shape, generator=gen, device="cuda") ** 4
    if kind == "odd":                                        # NaN, negative, infinite, tiny, -0
        for i, x in enumerate((float("nan"), -1.0, float("inf"), 1e-42, -0.0, 0.0)):
            w[..., 10 + i::97] = x
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_evict_exact(case, in_place):
    import torch

    B, Hkv, d, T, lens, keep, sinks, recent, kind = case
    p = Problem(B, Hkv, Hkv, d, T, lens, cap=T + 2, seed=T)
    w = _sums(kind, (B, Hkv, T + 2), p.gen)
    k0, v0, w0 = p.k.clone(), p.v.clone(), w.clone()
    if in_place:
        lay2, cache2, k2, v2, w2 = p.layout, p.cache, p.k, p.v, w
    else:
        o = Problem(B, Hkv, Hkv, d, keep + 9, seed=1)
        lay2, cache2, k2, v2 = o.layout, o.cache, o.k, o.v
        w2 = torch.full((B, Hkv, keep + 9), 5.0, device="cuda")
    k1, v1 = k2.clone(), v2.clone()
    kept, new = kvc.evict(p.layout, p.cache, lay2, cache2, w, w2, keep, sinks, recent)
    assert new.tolist() == [min(n, keep) for n in p.lens]
    bits = lambda x: x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)  # noqa: E731
    for (b, h), want in zip(((b, h) for b in range(B) for h in range(Hkv)),
                            D.evict(w0.cpu().numpy(), p.lens, keep, sinks, recent)):
        n = len(want)
        assert kept[b, h].tolist() == want + [-1] * (keep - n)
        at = torch.tensor(want, dtype=torch.long, device="cuda")
        for got, src in ((k2, k0), (v2, v0), (w2, w0)):
            assert torch.equal(bits(got[b, h, :n]), bits(src[b, h][at]))
        assert (w2[b, h, n:] == 0).all()
        for got, before in ((k2, k1), (v2, v1)):
            assert torch.equal(bits(got[b, h, n:]), bits(before[b, h, n:]))
    if not in_place:
        assert torch.equal(bits(k0), bits(p.k)) and torch.equal(bits(w0), bits(w))


@pytest.mark.gpu
def test_evict_layers():
    import torch

    p = Problem(2, 2, 2, 64, 120, [120, 70], L=3, seed=2)
    w = torch.rand(3, 2, 2, 120, generator=p.gen, device="cuda")
    o = Problem(2, 2, 2, 64, 40, L=3, seed=3)
    w2 = torch.empty(3, 2, 2, 40, device="cuda")
    kept, new = kvc.evict(p.layout, p.cache, o.layout, o.cache, w, w2, 32, 2, 5)
    assert new.tolist() == [32, 32]
    for l in range(3):
        for i, want in enumerate(D.evict(w[l].cpu().numpy(), p.lens, 32, 2, 5)):
            b, h = divmod(i, 2)
            assert kept[l, b, h].tolist() == want
            assert torch.equal(o.k[l, b, h, :32], p.k[l, b, h][torch.tensor(want, device="cuda")])
    p.cache.layer = o.cache.layer = 3
    kept1, _ = kvc.evict(p.layout, p.cache, o.layout, o.cache, w[2].contiguous(), w2[2].contiguous(), 32, 2, 5)
    assert torch.equal(kept1, kept[2])


PREFIX = [
    # B, Hq, Hkv, d, P, T, lens, bf16
    (1, 4, 1, 128, 1, 1, None, 0),
    (2, 8, 2, 128, 100, 40, [40, 0], 0),
    (3, 14, 2, 64, 333, 17, [17, 1, 9], 1),
    (5, 8, 8, 128, 257, 60, [60, 3, 59, 0, 17], 0),
    (9, 8, 2, 128, 700, 33, None, 1),                         # 36 rows per KV head
    (33, 8, 2, 64, 500, 20, None, 1),                         # 132 rows per KV head
    (2, 33, 1, 128, 150, 30, None, 0),
    (70, 8, 2, 128, 300, 5, [1, 2, 3, 4, 5, 0, 5] * 10, 1),   # 280 rows per KV head
    (40, 8, 2, 128, 400, 9, None, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c[:6] + c[7:])))
def test_prefix_parity(case):
    B, Hq, Hkv, d, P, T, lens, bf16 = case
    p = Problem(B, Hq, Hkv, d, T, lens, cap=T + 4, bf16=bf16, seed=P)
    pre = Problem(1, Hq, Hkv, d, P, cap=P + 30, seed=P + 1)
    q, out = p.queries(gain=1.5)
    ws = p.ws(p.layout.prefix_workspace_bytes(T, P))
    kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q, out, ws)
    ref, tol = D.prefix_attention(_f64(q), _f64(pre.k)[0, :, :P], _f64(pre.v)[0, :, :P], _f64(p.k), _f64(p.v), p.lens,
                                  p.scale, bool(bf16), _p_bits(bf16))
    within(_f64(out), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [2, 64])
def test_prefix_empty_parts(B):
    import torch

    p = Problem(B, 8, 2, 128, 20, cap=24, bf16=1, seed=1)
    pre = Problem(1, 8, 2, 128, 50, [50], cap=64, seed=2)
    q, out = p.queries()
    ws = p.ws(p.layout.prefix_workspace_bytes(20, 50))
    for n_pre, n_own in ((0, 20), (50, 0), (0, 0), (13, 20)):
        pre.cache.seq_lens.fill_(n_pre)
        p.cache.n_tokens = n_own
        kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q, out, ws)
        ref, tol = D.prefix_attention(_f64(q), _f64(pre.k)[0, :, :n_pre], _f64(pre.v)[0, :, :n_pre], _f64(p.k), _f64(p.v),
                                      [n_own] * B, p.scale, True, 8)
        within(_f64(out), ref, tol, f"{n_pre} + {n_own}")
    pre.cache.n_tokens = 0
    pre.cache.seq_lens = None
    p.cache.n_tokens = 20
    kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q, out, ws)
    alone = torch.empty_like(out)
    p.window(q[:, :, None].contiguous(), alone[:, :, None], 100, 0)
    # the same sums merged in another order: at most one step of bf16 apart
    assert ((out.double() - alone.double()).abs() <= 2.0**-7 * alone.double().abs() + 1e-5).all()


@pytest.mark.gpu
def test_prefix_layers():
    p = Problem(34, 4, 2, 64, 9, L=2, bf16=1, seed=5)
    pre = Problem(1, 4, 2, 64, 200, L=2, seed=6)
    q, out = p.queries()
    ws = p.ws(p.layout.prefix_workspace_bytes(9, 200))
    kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q, out, ws)
    for l in range(2):
        ref, tol = D.prefix_attention(_f64(q[l]), _f64(pre.k[l])[0], _f64(pre.v[l])[0], _f64(p.k[l]), _f64(p.v[l]),
                                      p.lens, p.scale, True, 8)
        within(_f64(out[l]), ref, tol, f"layer {l}")


@pytest.mark.gpu
def test_serving_run_prefill_decode_evict_decode():
    """The operators as a serving program uses them: prefill with the window,
    append and decode with accumulated weights, evict in place, go on."""
    import torch

    B, Hq, Hkv, d, cap, n0 = 2, 8, 2, 128, 96, 70
    lay = dense(B, Hq, Hkv, d, cap)
    cache = kvc.Cache(lay)
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ks, vs = rnd(B, Hkv, n0, d), rnd(B, Hkv, n0, d)
    kvc.append(lay, cache, ks, vs, [0] * B, n0)
    cache.n_tokens = n0
    ws = torch.empty(max(lay.window_workspace_bytes(cap, n0), lay.accum_workspace_bytes(cap)), dtype=torch.uint8,
                     device="cuda")
    q = rnd(B, Hq, n0, d)
    out = torch.empty(q.shape, device="cuda")
    kvc.window_attn(lay, cache, q, out, ws, 32, 4)
    k, v = _f64(ks), _f64(vs)
    ref, tol = D.window_attention(_f64(q), k, v, [n0] * B, 32, 4, d**-0.5)
    within(_f64(out), ref, tol, "prefill")
    w = torch.zeros(B, Hkv, cap, device="cuda")
    ref_w = np.zeros((B, Hkv, n0))
    n = n0
    for step in range(30):
        kn, vn, qn = rnd(B, Hkv, 1, d), rnd(B, Hkv, 1, d), rnd(B, Hq, d)
        kvc.append(lay, cache, kn, vn, [n] * B, 1)
        n += 1
        cache.n_tokens = n
        k, v = np.concatenate([k, _f64(kn)], 2), np.concatenate([v, _f64(vn)], 2)
        o = torch.empty(qn.shape, device="cuda")
        kvc.decode_accum(lay, cache, qn, w, o, ws)
        ref, tol = D.window_attention(_f64(qn)[:, :, None], k, v, [n] * B, n, 0, d**-0.5)
        within(_f64(o), ref[:, :, 0], tol[:, :, 0], f"step {step}")
        dw, _ = D.decode_weights(_f64(qn), k, v, [n] * B, d**-0.5)
        ref_w = np.concatenate([ref_w, np.zeros((B, Hkv, 1))], 2) + dw
        np.testing.assert_allclose(_f64(w)[:, :, :n], ref_w, rtol=1e-4)
        if step % 10 == 9:
            kept, lens = kvc.evict(lay, cache, lay, cache, w, w, 60, 4, 16)
            assert lens.tolist() == [60] * B
            at = kept.long().cpu().numpy()
            k, v = (np.take_along_axis(x, at[..., None], 2) for x in (k, v))
            ref_w = np.take_along_axis(ref_w, at, 2)
            n = 60
            cache.n_tokens = n


@pytest.mark.gpu
def test_captured_graphs_sharing_a_workspace_and_other_streams():
    import torch

    p = Problem(2, 8, 2, 128, 1500, [1500, 900], bf16=1, seed=21)
    pre = Problem(1, 8, 2, 128, 600, seed=22)
    w = torch.zeros(2, 2, 1500, device="cuda")
    q1, o1 = p.queries(1)
    q2, o2 = p.queries(130)
    q3, o3 = p.queries()
    o4 = o3.clone()
    n = max(p.layout.window_workspace_bytes(1500, 130), p.layout.accum_workspace_bytes(1500),
            p.layout.prefix_workspace_bytes(1500, 600))
    ws = p.ws(n)

    def calls_a():
        p.window(q1, o1, 700, 4, ws)
        p.window(q2, o2, 300, 4, ws)

    def calls_b():
        kvc.decode_accum(p.layout, p.cache, q3, w, o3, ws)
        kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q3, o4, ws)

    calls_a()
    calls_b()
    want = [x.clone() for x in (o1, o2, o3, o4, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for f in (calls_a, calls_b):
            f()                                              # on a stream of its own, before the capture
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                f()
            graphs.append(g)
    torch.cuda.synchronize()
    w.zero_()
    for x in (o1, o2, o3, o4):
        x.zero_()
    for g in (graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for got, ref in zip((o1, o2, o3, o4, w), want):
        assert torch.equal(got, ref)


@pytest.mark.gpu
def test_evict_captured_in_place():
    import torch

    p = Problem(1, 2, 2, 128, 400, seed=30)
    w = torch.rand(1, 2, 400, generator=p.gen, device="cuda")
    k0, w0 = p.k.clone(), w.clone()
    kept, _ = kvc.evict(p.layout, p.cache, p.layout, p.cache, w, w, 100, 4, 10)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept2, _ = kvc.evict(p.layout, p.cache, p.layout, p.cache, w, w, 100, 4, 10)
    p.k.copy_(k0)
    w.copy_(w0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, kept2)
    for h in range(2):
        assert torch.equal(p.k[0, h, :100], k0[0, h][kept[0, h].long()])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache whose element offsets pass 2^32: one late unit against a small cache of the same tokens."""
    import torch

    B, Hkv, T, d = 2, 9, 1 << 21, 128                        # 18 units of 2^28 elements
    big = dense(B, Hkv, Hkv, d, T)
    cache = kvc.Cache(big)                                   # zeros
    small = Problem(1, 1, 1, d, 3000, seed=40)
    for name, x in (("k_dense", small.k), ("v_dense", small.v)):
        cache.bufs[name].view(torch.bfloat16).view(B, Hkv, T, d)[1, 8, :3000] = x[0, 0]
    cache.seq_lens = torch.tensor([1, 3000], dtype=torch.int32, device="cuda")
    cache.n_tokens = 3000
    for n_q in (1, 200):
        q1, o1 = small.queries(n_q)
        small.window(q1, o1, 1000, 4)
        q = torch.zeros(B, Hkv, n_q, d, dtype=torch.bfloat16, device="cuda")
        q[1, 8] = q1[0, 0]
        out = torch.empty(q.shape, device="cuda")
        ws = torch.empty(big.window_workspace_bytes(3000, n_q), dtype=torch.uint8, device="cuda")
        kvc.window_attn(big, cache, q, out, ws, 1000, 4)
        assert (out[1, 8] - o1[0, 0]).abs().max() < 1e-5


def _on_gpu(q, k, v, seen, scale, bf16):
    """(out, bound) of one head in 64 bits: q [r, d], k, v [t, d], seen [r, t]."""
    import torch

    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T * scale).masked_fill(~seen, -float("inf"))
    p = torch.nan_to_num(torch.softmax(s, -1))
    out, absv = p @ v, p @ v.abs()
    size = float((q.abs() @ k.abs().T).max() * scale) if len(k) else 0.0
    return _f64(out), D.error_bound(size, _f64(absv), _f64(out), q.shape[-1], bool(bf16), _p_bits(bf16)), p.sum(0)


FLAT_LENS = [[4000, 1, 0, 3999, 2500, 16, 0, 3000], None, [0] * 7 + [4000], [4000] + [0] * 7]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", FLAT_LENS, ids=["ragged", "full", "last", "first"])
@pytest.mark.parametrize("n_q,bf16,d,W,S", [(1, 0, 128, 4000, 0), (1, 1, 64, 3900, 70), (5, 0, 64, 3500, 3),
                                            (3, 1, 128, 4000, 0)])
def test_window_large_calls(lens, n_q, bf16, d, W, S):
    """Enough tokens for every warp of the GPU: tiles dealt out across rows and heads."""
    import torch

    p = Problem(8, 12, 4, d, 4000, lens, cap=4011, bf16=bf16, seed=50)
    q, out = p.queries(n_q, gain=1.5)
    p.window(q, out, W, S)
    for b, n in enumerate(p.lens):
        pos = torch.arange(n - n_q, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")
        for h in range(12):
            ref, tol, _ = _on_gpu(q[b, h], p.k[b, h // 3, :n], p.v[b, h // 3, :n],
                                  (t <= pos) & ((t < S) | (t > pos - W)), p.scale, bf16)
            within(_f64(out[b, h]), ref, tol, f"row {b} head {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("lens", FLAT_LENS[:2], ids=["ragged", "full"])
@pytest.mark.parametrize("Hq,bf16,d", [(12, 0, 128), (16, 1, 128), (4, 0, 64), (132, 0, 64)])
def test_accum_large_calls(lens, Hq, bf16, d):
    import torch

    p = Problem(8, Hq, 4, d, 4000, lens, cap=4011, bf16=bf16, seed=51)
    q, out = p.queries(gain=1.5)
    w = torch.rand(8, 4, 4011, generator=p.gen, device="cuda")
    w0 = w.double()
    kvc.decode_accum(p.layout, p.cache, q, w, out, p.ws(p.layout.accum_workspace_bytes(4000)))
    G = Hq // 4
    for b, n in enumerate(p.lens):
        every = torch.ones(G, n, dtype=torch.bool, device="cuda")
        for h in range(4):
            k = p.k[b, h, :n]
            ref, tol, dw = _on_gpu(q[b, h * G:(h + 1) * G], k, p.v[b, h, :n], every, p.scale, bf16)
            within(_f64(out[b, h * G:(h + 1) * G]), ref, tol, f"row {b} head {h}")
            size = float((q[b, h * G:(h + 1) * G].double().abs() @ k.double().abs().T).max() * p.scale) if n else 0.0
            want = w0[b, h, :n] + dw
            rel = 2 * (d / 16) * 2.0**-22 * size + 2.0**-19
            assert ((w[b, h, :n].double() - want).abs() <= rel * dw + 2.0**-24 * want).all()
        assert torch.equal(w[b, :, n:].double(), w0[b, :, n:])


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [0, 1])
@pytest.mark.parametrize("B,T,P", [(64, 600, 4000), (64, 0, 4000), (64, 600, 0), (3, 9, 40000)])
def test_prefix_large_calls(bf16, B, T, P):
    import torch

    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, T + 1, B)]
    p = Problem(B, 16, 4, 128, max(T, 1), lens, cap=T + 7, bf16=bf16, seed=52)
    p.cache.n_tokens = T
    pre = Problem(1, 16, 4, 128, max(P, 1), cap=P + 3, seed=53)
    pre.cache.n_tokens = P
    q, out = p.queries(gain=1.5)
    kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q, out, p.ws(p.layout.prefix_workspace_bytes(T, P)))
    for b in range(0, B, 5):
        for h in range(4):
            k = torch.cat([pre.k[0, h, :P], p.k[b, h, :lens[b]]])
            v = torch.cat([pre.v[0, h, :P], p.v[b, h, :lens[b]]])
            ref, tol, _ = _on_gpu(q[b, 4 * h:4 * h + 4], k, v,
                                  torch.ones(4, len(k), dtype=torch.bool, device="cuda"), p.scale, bf16)
            within(_f64(out[b, 4 * h:4 * h + 4]), ref, tol, f"row {b} head {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", [(1, 1, 64, 400001, None, 150000, 4, 1000, "random"),     # beyond a cluster's shared memory
                                  (3, 2, 64, 20000, [20000, 8191, 0], 5000, 0, 0, "ties"),   # two blocks and more per head
                                  (2, 4, 128, 33000, [33000, 4097], 4096, 4096, 0, "random"),
                                  (40, 8, 64, 4100, None, 100, 3, 50, "same")],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_evict_long_rows(case, in_place):
    test_evict_exact(case, in_place)


def test_calls_refuse_more_rows_than_an_index_holds():
    L = kvc.lib()
    f = C.c_void_p(F)
    wide = dense(B=256, Hq=4096 * 64, Hkv=64, T=64, L=64)
    assert L.kvc_accum_workspace_bytes(wide.h, 64) == 0 and L.kvc_prefix_workspace_bytes(wide.h, 64, 64) == 0
    assert _status(L.kvc_decode_accum(wide.h, C.byref(_cs(64)), f, f, f, f, BIG, None)) == "KVC_EUNSUPPORTED"
    pre = dense(B=1, Hq=4096 * 64, Hkv=64, T=64, L=64)
    assert _status(L.kvc_prefix_decode(pre.h, C.byref(_cs(64)), wide.h, C.byref(_cs(64)), f, f, f, BIG,
                                       None)) == "KVC_EUNSUPPORTED"


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [0, 1])
def test_empty_cache_gives_zeros(bf16):
    import torch

    p = Problem(2, 8, 2, 128, 64, bf16=bf16, seed=60)
    p.k.fill_(float("nan"))
    p.v.fill_(float("nan"))
    p.cache.n_tokens = 0
    for n_q in (1, 3, 60):
        q, out = p.queries(n_q)
        p.window(q, out, 8, 2)
        assert (out == 0).all()
    q, out = p.queries()
    w = torch.full((2, 2, 64), 3.0, device="cuda")
    kvc.decode_accum(p.layout, p.cache, q, w, out, p.ws(p.layout.accum_workspace_bytes(0)))
    assert (out == 0).all() and (w == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 40])
def test_prefix_non_finite_own_token_stays_in_its_row(rows):
    """A NaN value of one row's own token, an infinite query of another: nobody else's output notices."""
    p = Problem(rows, 8, 2, 128, 20, cap=24, bf16=1, seed=61)
    pre = Problem(1, 8, 2, 128, 300, seed=62)
    q, out = p.queries()
    p.v[0, 1, 7, 3] = float("nan")
    q[1, 0, 5] = float("inf")
    kvc.prefix_decode(pre.layout, pre.cache, p.layout, p.cache, q, out, p.ws(p.layout.prefix_workspace_bytes(20, 300)))
    got = _f64(out)
    assert np.isnan(got[0, 4:, 3]).all() and not np.isfinite(got[1, 0]).any()
    v, qq = _f64(p.v), _f64(q)
    v[0, 1, 7, 3], qq[1, 0, 5] = 0.0, 0.0
    ref, tol = D.prefix_attention(qq, _f64(pre.k)[0], _f64(pre.v)[0], _f64(p.k), v, p.lens, p.scale, True, 8)
    clean = np.ones(got.shape, bool)
    clean[0, 4:, 3] = clean[1, 0] = False
    within(got[clean], ref[clean], tol[clean])


@pytest.mark.gpu
def test_window_scores_that_outgrow_the_reference():
    """Scores that keep rising along the tokens, by far more than 2^24 a tile, and fall again."""
    p = Problem(1, 4, 1, 64, 900, bf16=1, seed=63)
    q, out = p.queries(300)
    import torch

    t = np.concatenate([np.linspace(0, 60, 600), np.linspace(60, -60, 300)])
    q += 2.0

    p.k[0, 0] = (p.k[0, 0].float() * 0.1 + torch.tensor(t, device="cuda").float()[:, None] / 4).bfloat16()
    for W in (900, 250):
        p.window(q, out, W, 3)
        ref, tol = D.window_attention(_f64(q), _f64(p.k), _f64(p.v), p.lens, W, 3, p.scale, True, 8)
        within(_f64(out), ref, tol, f"window {W}")


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    import torch

    ps = [Problem(2, 16, 2, 128, 1200, [1200, 700], bf16=1, seed=70 + i) for i in range(2)]
    io = [p.queries(96) for p in ps]
    want = []
    for p, (q, o) in zip(ps, io):
        p.window(q, o, 300, 4)
        want.append(o.clone())
        o.zero_()
    ws = [p.ws(p.layout.window_workspace_bytes(1200, 96)) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, (q, o), w, s in zip(ps, io, ws, streams):
            with torch.cuda.stream(s):
                p.window(q, o, 300, 4, w)
    torch.cuda.synchronize()
    for (_, o), ref in zip(io, want):
        assert torch.equal(o, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,Hq", [(150, 8), (20, 8), (600, 32)])
def test_bounded_waits_give_up_report_and_leave_the_context_usable(n_q, Hq):
    import torch

    p = Problem(1, Hq, 2, 128, 700, bf16=1, seed=80)
    q, out = p.queries(n_q)
    lib = kvc.lib()
    lib.kvc_test_skip_tile_copies(1)
    try:
        ws = p.window(q, out, 400, 4)                       # the waits run out (0.5 s) and the blocks end
        torch.cuda.synchronize()
    finally:
        lib.kvc_test_skip_tile_copies(0)
    assert int(ws[:4].view(torch.int32)) & kvc.DEV_WAIT_TIMEOUT
    p.window(q, out, 400, 4, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    ref, tol = D.window_attention(_f64(q)[:, :1], _f64(p.k)[:, :1], _f64(p.v)[:, :1], p.lens, 400, 4, p.scale, True, 8)
    within(_f64(out)[:, :1], ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("d,T,n_q,W,S,G,bad", [(128, 200, 70, 33, 5, 4, False), (64, 200, 70, 200, 0, 4, True),
                                               (128, 700, 65, 130, 40, 4, False), (128, 90, 90, 90, 0, 3, True),
                                               (64, 1500, 130, 500, 64, 2, False)])
def test_window_many_blocks_of_few_tiles(d, T, n_q, W, S, G, bad):
    """Enough row blocks to fill the SMs twice, with few tokens each."""
    import torch

    B, Hkv = 19, 8
    lens = [T, 0, 1, T - 1, n_q, n_q - 1, T // 2] + [T - 3 * i for i in range(B - 7)]
    p = Problem(B, Hkv * G, Hkv, d, T, lens, cap=T + 3, bf16=1, seed=90)
    if bad:
        p.v[0, 2, T - 20, 1] = float("nan")                  # seen by some queries of its row only
    q, out = p.queries(n_q, gain=1.5)
    p.window(q, out, W, S)
    v = p.v.clone()
    if bad:
        v[0, 2, T - 20, 1] = 0
    for b, n in enumerate(lens):
        pos = torch.arange(n - n_q, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")
        seen = (t <= pos) & ((t < S) | (t > pos - W))
        for h in range(0, Hkv * G, 3 if b else 1):
            ref, tol, _ = _on_gpu(q[b, h], p.k[b, h // G, :n], v[b, h // G, :n], seen, p.scale, True)
            got = _f64(out[b, h])
            if bad and b == 0 and h // G == 2:
                hit = seen[:, T - 20].cpu().numpy()
                assert hit.any() and not hit.all() and np.isnan(got[hit, 1]).all()
                got, ref, tol = got[~hit], ref[~hit], tol[~hit]
            within(got, ref, tol, f"row {b} head {h}")


@pytest.mark.gpu
def test_offsets_past_32_bits_in_the_other_kernels():
    """The tcgen05 kernel, the weighted decode, the shared prefix and the eviction on a late unit of a
    cache whose element offsets pass 2^32, against a small cache of the same tokens."""
    import torch

    B, Hkv, T, d, n = 2, 9, 1 << 21, 128, 3000               # 18 units of 2^28 elements
    big = dense(B, Hkv, Hkv, d, T, bf16=1)
    cache = kvc.Cache(big)                                   # zeros
    small = Problem(1, 1, 1, d, n, bf16=1, seed=41)
    kv = {name: cache.bufs[name].view(torch.bfloat16).view(B, Hkv, T, d) for name in ("k_dense", "v_dense")}
    kv["k_dense"][1, 8, :n], kv["v_dense"][1, 8, :n] = small.k[0, 0], small.v[0, 0]
    cache.seq_lens = torch.tensor([1, n], dtype=torch.int32, device="cuda")
    cache.n_tokens = n
    close = lambda a, b: ((a.double() - b.double()).abs() <= 2.0**-7 * b.double().abs() + 1e-4).all()  # noqa: E731
    # prefill rows on tcgen05: the same scores in another split, one step of bf16 apart at most
    q1, o1 = small.queries(200)
    small.window(q1, o1, 1000, 4)
    q = torch.zeros(B, Hkv, 200, d, dtype=torch.bfloat16, device="cuda")
    q[1, 8] = q1[0, 0]
    out = torch.empty_like(q)
    ws = torch.empty(max(big.window_workspace_bytes(n, 200), big.accum_workspace_bytes(n),
                         big.prefix_workspace_bytes(n, 100)), dtype=torch.uint8, device="cuda")
    kvc.window_attn(big, cache, q, out, ws, 1000, 4)
    assert close(out[1, 8], o1[0, 0])
    # one token with weights, and behind a prefix
    qa, oa = small.queries()
    w1 = torch.zeros(1, 1, n, device="cuda")
    kvc.decode_accum(small.layout, small.cache, qa, w1, oa, small.ws(small.layout.accum_workspace_bytes(n)))
    q = torch.zeros(B, Hkv, d, dtype=torch.bfloat16, device="cuda")
    q[1, 8] = qa[0, 0]
    out = torch.empty_like(q)
    w = torch.zeros(B, Hkv, T, device="cuda")
    kvc.decode_accum(big, cache, q, w, out, ws)
    assert close(out[1, 8], oa[0, 0])
    assert ((w[1, 8, :n] - w1[0, 0]).abs() <= 1e-5 * w1[0, 0]).all() and (w[1, 8, n:] == 0).all()
    pre = Problem(1, Hkv, Hkv, d, 100, seed=42)
    kvc.prefix_decode(pre.layout, pre.cache, big, cache, q, out, ws)
    ref, tol = D.prefix_attention(_f64(q)[1:, 8:], _f64(pre.k)[0, 8:], _f64(pre.v)[0, 8:], _f64(small.k), _f64(small.v),
                                  [n], d**-0.5, True, 8)
    within(_f64(out)[1:, 8:], ref, tol)
    # eviction in place
    w[1, 8, :n] = torch.rand(n, generator=small.gen, device="cuda")
    w0 = w[1, 8, :n].clone()
    kept, lens = kvc.evict(big, cache, big, cache, w, w, 700, 4, 50)
    assert lens.tolist() == [1, 700]
    want = D.evict(w0[None, None].cpu().numpy(), [n], 700, 4, 50)[0]
    assert kept[1, 8].tolist() == want
    at = torch.tensor(want, device="cuda")
    for name, src in (("k_dense", small.k), ("v_dense", small.v)):
        assert torch.equal(kv[name][1, 8, :700], src[0, 0][at])
    assert torch.equal(w[1, 8, :700], w0[at]) and (w[1, 8, 700:] == 0).all()


@pytest.mark.gpu
def test_evict_of_an_empty_cache():
    import torch

    p = Problem(2, 2, 2, 64, 50, cap=60, seed=43)
    p.cache.n_tokens = 0
    w, w2 = torch.ones(2, 2, 60, device="cuda"), torch.ones(2, 2, 40, device="cuda")
    o = Problem(2, 2, 2, 64, 40, seed=44)
    k1 = o.k.clone()
    kept, lens = kvc.evict(p.layout, p.cache, o.layout, o.cache, w, w2, 32, 4, 8)
    assert (kept == -1).all() and lens.tolist() == [0, 0] and (w2 == 0).all() and torch.equal(o.k, k1)
