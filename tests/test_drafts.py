"""Speculative decoding without a GPU: the float64 definitions against closed
forms and brute force, the rotary frequencies, and the entry points' argument
checks (no call here launches a kernel)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import drafts as OD
from paged_kv_cache_store_gb300 import build as pabuild


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.load_library()


# ---------------------------------------------------------------- definitions

def test_rope_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 128))
    y, _ = OD.rope(x, [0, 0, 0], 128, 1e4)
    assert np.allclose(x, y)
    # Scores depend on the distance alone.
    q, k = rng.standard_normal((2, 1, 1, 128))
    for inter in (False, True):
        dots = [float((OD.rope(q, [p], 96, 1e4, interleaved=inter)[0] *
                       OD.rope(k, [p - 7], 96, 1e4, interleaved=inter)[0]).sum()) for p in (7, 100, 5000)]
        assert np.allclose(dots, dots[0])
    # The two layouts are one rotation, up to the order of the values.
    order = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2), np.arange(64, 128)])
    a, _ = OD.rope(x, [5, 6, 7], 64, 1e4, interleaved=True)
    b, _ = OD.rope(x[..., order], [5, 6, 7], 64, 1e4)
    assert np.allclose(a[..., order], b)
    assert np.array_equal(a[..., 64:], x[..., 64:])
    # A normed head has the weight's mean square.
    z, _ = OD.rope(x, [1, 2, 3], 128, 1e4, weight=np.ones(128), eps=0.0)
    assert np.allclose((z * z).mean(-1), 1.0)


SCALINGS = [None, ("linear", 4.0), ("ntk", 8.0), ("yarn", 4.0, 32768.0), ("yarn", 16.0, 4096.0, 16.0, 2.0)]


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("rotary", [16, 32, 64, 96, 128])
def test_rope_frequencies(L, rotary, scaling):
    for theta in (1e4, 1e6):
        r = pa.rope_frequencies(rotary, theta, scaling, interleaved=True, device="cpu")
        f, gain = OD.frequencies(rotary, theta, scaling)
        turns = np.array([int(x) % (1 << 64) for x in r.freqs.tolist()], np.float64) / 2.0 ** 64
        # A few roundings to 64 bits (pow, the division by 2 pi) and 2^-64 absolute.
        assert np.all(np.abs(turns - f / (2 * math.pi)) <= 2.0 ** -47 * f + 2.0 ** -63)
        assert r.gain == np.float32(gain) and r.interleaved


def test_yarn_keeps_short_waves_and_divides_long_ones():
    plain, _ = OD.frequencies(128, 1e6)
    f, gain = OD.frequencies(128, 1e6, ("yarn", 4.0, 32768.0))
    assert f[0] == plain[0] and np.isclose(f[-1], plain[-1] / 4) and np.all(np.diff(f) < 0)
    assert np.isclose(gain, 0.1 * math.log(4) + 1)


def test_rope_frequencies_refusals(L):
    for kw in (dict(rotary_dim=8), dict(rotary_dim=40), dict(rotary_dim=144), dict(theta=1.0), dict(theta=float("nan")),
               dict(theta=float("inf")), dict(scaling=("linear", 0.5)), dict(scaling=("ntk", float("inf"))),
               dict(scaling=("yarn", 4.0, 0.0)), dict(scaling=("yarn", 4.0, 4096.0, 1.0, 2.0))):
        with pytest.raises(pa.PagedAttentionError):
            pa.rope_frequencies(**{**dict(rotary_dim=128, device="cpu"), **kw})
    for scaling in (("other", 1.0), "linear", ("linear",), ("linear", 1.0, 2.0), ("yarn", 4.0), ("yarn", 4.0, 1.0, 2.0)):
        with pytest.raises(ValueError):
            pa.rope_frequencies(scaling=scaling, device="cpu")
    f, g = (C.c_uint64 * 64)(), C.c_float()
    assert L.pa_rope_frequencies(None, C.byref(g), 128, 1e4, 0, 1, 0, 32, 1) == pa.PA_ERR_INVALID_ARG
    assert L.pa_rope_frequencies(f, C.byref(g), 128, 1e4, 4, 1, 0, 32, 1) == pa.PA_ERR_INVALID_ARG


def test_trees():
    sees, depth = OD.ancestors(np.array([-1, 0, 0, 1, 3, 2]))
    assert depth.tolist() == [0, 1, 1, 2, 3, 2]
    assert OD.as_bits(sees).tolist() == [1, 3, 5, 11, 27, 37]
    chain, _ = OD.ancestors(np.arange(64) - 1)
    assert OD.as_bits(chain)[-1] == -1 and OD.as_bits(chain)[3] == 15


def test_tree_attention_of_a_path_is_causal_attention():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 20, 128))
    q = rng.standard_normal((6, 2, 128))
    sees, _ = OD.ancestors(np.array([-1, 0, 0, 1, 3, 2]))
    out, _ = OD.attend(q, k, v, sees, 0.1)
    path = [0, 1, 3, 4]                      # the ancestors of node 4, as a chain of their own
    rows = list(range(14)) + [14 + i for i in path]
    chain, _ = OD.attend(q[path], k[rows], v[rows], np.tril(np.ones((4, 4), bool)), 0.1)
    assert np.allclose(out[path], chain)
    for i, w in enumerate(path):
        x = q[w] @ k[rows[:15 + i]].T * 0.1
        p = np.exp(x) / np.exp(x).sum(-1, keepdims=True)
        assert np.allclose(out[w], p @ v[rows[:15 + i]])


def brute_first_token(p, q, n):
    """Distribution of a step's first token with n children drawn from q, by
    summing over all children and the ends of the unit interval of each u."""
    V = len(p)

    def rec(w, left, k):
        if k == n:
            return (w / w.sum()) if w.sum() > 0 else p
        out = np.zeros(V)
        for x in range(V):
            keep = min(1.0, w[x] / (q[x] * left)) if q[x] * left > 0 else 0.0
            e = np.zeros(V)
            e[x] = 1
            nw = np.maximum(w - left * q, 0)
            out += q[x] * (keep * e + ((1 - keep) * rec(nw, nw.sum(), k + 1) if keep < 1 else 0))
        return out

    return rec(p, 1.0, 0)


@pytest.mark.parametrize("n", [1, 2, 3])
def test_verification_keeps_the_targets_distribution(n):
    """In closed form: whatever the drafts' distribution, the token that comes
    first is distributed as the target's."""
    rng = np.random.default_rng(n)
    for _ in range(5):
        p, q = rng.dirichlet(np.ones(5), 2)
        assert np.allclose(brute_first_token(p, q, n), p)


def test_verify_samples_the_targets_distribution():
    """The definition itself, drawn often: with drawn children and with chosen ones."""
    rng = np.random.default_rng(3)
    V, N = 6, 20000
    z, zq = rng.standard_normal((2, V))
    p, q = np.exp(z) / np.exp(z).sum(), np.exp(zq) / np.exp(zq).sum()
    parents = np.array([[-1, 0, 0]] * N)
    logits = np.broadcast_to(z, (N, 3, V))
    noise, u = rng.exponential(size=(N, V)), rng.random((N, 3))
    drawn = np.concatenate([np.zeros((N, 1), int), rng.choice(V, size=(N, 2), p=q)], 1)
    chosen = np.broadcast_to([0, 2, 4], (N, 3))
    for tokens, probs in ((drawn, np.broadcast_to(q, (N, 2, V))), (chosen, None)):
        t, nodes, counts, _ = OD.verify(logits, tokens, parents, u, noise, np.ones(N), probs)
        got = np.bincount(t[:, 0], minlength=V) / N
        assert np.all(np.abs(got - p) < 5 * np.sqrt(p * (1 - p) / N))  # five standard errors
        assert np.all((counts == 1) | (counts == 2)) and np.all(nodes[:, 0] == 0)


def test_compaction():
    cache = np.arange(6 * 4, dtype=np.int64).reshape(6, 4, 1)
    table = np.array([[5, 0, 3, -1]])
    got = OD.compact(cache, table, [10], np.array([[0, 2, 3, -1, -1]]), [3])
    want = cache.copy()
    want[0, 2], want[0, 3] = cache[0, 3], cache[3, 0]  # positions 7, 8 -> 6, 7
    assert np.array_equal(got, want)


# ---------------------------------------------------------------- argument checks

P = C.c_void_p(256)
ODD = C.c_void_p(264)



def test_rope_argument_checks(L):
    def call(**kw):
        a = dict(oq=P, oqs=2048, ok=P, oks=1024, q=P, qs=2048, k=P, ks=1024, pos=P, f=P, r=128, inter=0, gain=1.0,
                 wq=None, wk=None, eps=1e-6, n=4, hq=16, hkv=8, d=128, st=None)
        a.update(kw)
        return L.pa_rope(*a.values())

    def store(**kw):
        a = dict(oq=P, oqs=2048, q=P, qs=2048, k=P, ks=1024, v=P, vs=1024, pos=P, f=P, r=128, inter=0, gain=1.0,
                 wq=None, wk=None, eps=1e-6, kc=P, vc=P, slots=P, n=4, hq=16, hkv=8, d=128, ns=1024, st=None)
        a.update(kw)
        return L.pa_rope_store_kvcache(*a.values())

    bad = pa.PA_ERR_INVALID_ARG
    for fn, null in ((call, ("oq", "ok", "q", "k", "pos", "f")), (store, ("oq", "q", "k", "v", "pos", "f", "kc", "vc", "slots"))):
        assert fn(n=0) == pa.PA_OK
        assert fn(n=-1) == bad
        for name in null:
            assert fn(**{name: None}) == bad, name
        assert fn(d=64) == pa.PA_ERR_UNSUPPORTED
        assert fn(hq=0) == bad and fn(hkv=0) == bad
        for r in (0, 8, 24, 136):
            assert fn(r=r) == pa.PA_ERR_UNSUPPORTED
        assert fn(inter=2) == bad
        assert fn(eps=-1.0) == bad and fn(eps=float("nan")) == bad
        assert fn(qs=2040) == bad and fn(qs=2052) == bad and fn(oqs=1024) == bad and fn(ks=1020) == bad
        assert fn(q=ODD) == bad and fn(k=ODD) == bad and fn(wq=ODD) == bad and fn(f=C.c_void_p(260)) == bad
        assert fn(n=0x7fffffff) == bad
    assert store(vs=1000) == bad and store(ns=0) == bad and store(kc=ODD) == bad
    assert call(oks=512) == bad


def test_tree_metadata_argument_checks(L):
    def call(**kw):
        a = dict(m=P, p=P, s=P, par=None, ctx=P, lens=None, bt=P, mb=4, batch=2, n=8, B=16, st=None)
        a.update(kw)
        return L.pa_tree_metadata(*a.values())

    assert call(batch=0) == pa.PA_OK
    assert call(n=65) == pa.PA_ERR_UNSUPPORTED
    for kw in (dict(batch=-1), dict(n=0), dict(m=None), dict(p=None), dict(s=None), dict(ctx=None), dict(bt=None),
               dict(mb=0), dict(B=0), dict(m=C.c_void_p(260))):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw


def test_decode_tree_argument_checks(L):
    def call(**kw):
        a = dict(out=P, q=P, qs=2048, k=P, v=P, bt=P, mb=16, ctx=P, lens=None, mask=None, batch=4, t=8, hq=16, hkv=8,
                 d=128, B=256, nb=64, scale=0.088, ws=P, wsb=1 << 30, st=None)
        a.update(kw)
        return L.pa_decode_tree(*a.values())

    assert call(batch=0) == pa.PA_OK
    for kw in (dict(batch=-1), dict(t=0), dict(out=None), dict(q=None), dict(k=None), dict(v=None), dict(bt=None),
               dict(ctx=None), dict(hq=12), dict(hkv=0), dict(qs=2040), dict(qs=2052), dict(scale=0.0),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(mb=0), dict(B=0), dict(nb=0), dict(q=ODD),
               dict(k=ODD), dict(out=ODD), dict(ws=ODD), dict(ws=C.c_void_p(272)), dict(mask=C.c_void_p(260))):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(hq=24), dict(hq=128), dict(d=64), dict(B=24), dict(t=65), dict(batch=2049), dict(nb=1 << 24),
               dict(batch=2048, mb=1 << 20, nb=1024, B=1024)):
        assert call(**kw) == pa.PA_ERR_UNSUPPORTED, kw
    assert call(ws=None) == pa.PA_ERR_WORKSPACE and call(wsb=1000) == pa.PA_ERR_WORKSPACE
    need = L.pa_decode_tree_workspace_size(16, 8, 128, 8)
    assert call(wsb=need - 1) == pa.PA_ERR_WORKSPACE
    assert L.pa_decode_tree_workspace_size(16, 8, 128, 64) >= need > 0
    for shape in ((16, 8, 64, 8), (24, 8, 128, 8), (12, 8, 128, 8), (16, 8, 128, 65), (16, 8, 128, 0), (0, 8, 128, 8)):
        assert L.pa_decode_tree_workspace_size(*shape) == 0


def test_verify_argument_checks(L):
    def call(**kw):
        a = dict(ot=P, on=P, oc=P, lg=P, ls=1024, f32=0, tok=P, par=None, u=P, e=P, es=1000, temp=P, q=P, qs=1000, qr=7,
                 lens=None, batch=3, n=8, vocab=1000, st=None)
        a.update(kw)
        return L.pa_verify_drafts(*a.values())

    assert call(batch=0) == pa.PA_OK
    for kw in (dict(batch=-1), dict(n=0), dict(vocab=0), dict(vocab=-1), dict(ot=None), dict(on=None), dict(oc=None),
               dict(lg=None), dict(tok=None), dict(u=None), dict(e=None), dict(temp=None), dict(f32=2), dict(ls=999),
               dict(ls=1004), dict(ls=1002, f32=1), dict(es=998), dict(es=1002), dict(qs=996), dict(qs=1001),
               dict(qr=6), dict(lg=ODD), dict(e=ODD), dict(q=ODD)):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(n=65), dict(batch=65536), dict(vocab=(1 << 30) + 8, ls=1 << 31, es=1 << 31, qs=1 << 31)):
        assert call(**kw) == pa.PA_ERR_UNSUPPORTED, kw


def test_compact_argument_checks(L):
    def call(**kw):
        a = dict(k=P, kl=1 << 20, v=P, vl=1 << 20, bt=P, mb=4, ctx=P, lens=None, nodes=P, counts=P, batch=2, n=8, layers=2,
                 hkv=8, d=128, B=16, nb=64, st=None)
        a.update(kw)
        return L.pa_compact_kvcache(*a.values())

    assert call(batch=0) == pa.PA_OK and call(layers=0) == pa.PA_OK
    for kw in (dict(batch=-1), dict(layers=-1), dict(n=0), dict(k=None), dict(v=None), dict(bt=None), dict(ctx=None),
               dict(nodes=None), dict(counts=None), dict(hkv=0), dict(mb=0), dict(B=0), dict(nb=0), dict(kl=4),
               dict(vl=0), dict(k=ODD)):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    for kw in (dict(n=65), dict(d=64)):
        assert call(**kw) == pa.PA_ERR_UNSUPPORTED, kw


def test_binding_refuses_cpu_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    r = pa.rope_frequencies(device="cpu")
    with pytest.raises(TypeError):
        pa.rope(bf(2, 4, 128), bf(2, 2, 128), i32(2), r)
    with pytest.raises(TypeError):
        pa.decode_tree(bf(2, 3, 4, 128), bf(4, 16, 2, 128), bf(4, 16, 2, 128), i32(2, 2), i32(2))
    with pytest.raises(TypeError):
        pa.tree_metadata(i32(2, 3), i32(2), i32(2, 2), 16)
    with pytest.raises(TypeError):
        pa.verify_drafts(torch.zeros(2, 3, 50), i32(2, 3), None, torch.zeros(2, 3), torch.zeros(2, 50), torch.ones(2))
    with pytest.raises(TypeError):
        pa.compact_kvcache(bf(4, 16, 2, 128), bf(4, 16, 2, 128), i32(2, 2), i32(2), i32(2, 3), i32(2))
