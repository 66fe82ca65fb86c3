"""A step of speculative decoding as an engine runs it -- metadata, rotation and
store, attention, verification, compaction -- on streams, in CUDA graphs, and over
pools beyond 32-bit offsets; each part against oracle/drafts.py."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import drafts as OD
from paged_kv_cache_store_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits
from gpu_util import dev_bf16, dev_i32, host_bits, host_f64

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, T, VOCAB = 16, 8, 2, 128, 9, 613
SCALE = 1 / math.sqrt(D)


def bits(rng, *shape):
    return f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def f64(b):
    return bf16_bits_to_f32(b).astype(np.float64)


class Step:
    """Sequences with a rotated context in the pool and a drafted tree each."""

    def __init__(self, seed, before, lens):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, batch = np.array(lens, np.int32), len(before)
        self.ctx = (np.array(before) + self.lens).astype(np.int32)
        need = -(-self.ctx // B)
        self.bt = np.full((batch, 8), -1, np.int32)
        ids, at = rng.permutation(int(need.sum()) + 2), 0
        for b in range(batch):
            self.bt[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.kc, self.vc = bits(rng, len(ids), B, HKV, D), bits(rng, len(ids), B, HKV, D)
        self.parents = np.stack([OD.random_parents(rng, T) for _ in before])
        self.qkv = bits(rng, batch * T, HQ + 2 * HKV, D)
        self.tokens = rng.integers(0, VOCAB, (batch, T)).astype(np.int32)
        self.logits = (rng.standard_normal((batch, T, VOCAB)) * 0.5).astype(np.float32)
        for b in range(batch):  # most drafts are what the target says
            for c in range(1, T):
                if rng.random() < 0.7:
                    self.logits[b, self.parents[b, c], self.tokens[b, c]] += 14.0
        self.u = rng.random((batch, T)).astype(np.float32)
        self.noise = rng.exponential(size=(batch, VOCAB)).astype(np.float32)
        self.temps = np.ones(batch, np.float32)
        self.batch = batch

    def device(self):
        d = dict(kc=dev_bf16(self.kc), vc=dev_bf16(self.vc), bt=dev_i32(self.bt), ctx=dev_i32(self.ctx),
                 lens=dev_i32(self.lens), parents=dev_i32(self.parents), qkv=dev_bf16(self.qkv),
                 tokens=dev_i32(self.tokens), u=torch.from_numpy(self.u).cuda(), temps=torch.from_numpy(self.temps).cuda())
        wide = -(-VOCAB // 8) * 8
        d["logits"] = torch.zeros(self.batch, T, wide, device="cuda")[..., :VOCAB]
        d["noise"] = torch.ones(self.batch, wide, device="cuda")[:, :VOCAB]
        d["logits"].copy_(torch.from_numpy(self.logits))
        d["noise"].copy_(torch.from_numpy(self.noise))
        return d


ROPE = {}


def run(d, ws, stream=None):
    """One step; everything it makes."""
    r = ROPE.setdefault("r", None) or ROPE.update(r=pa.rope_frequencies(D, 1e6)) or ROPE["r"]
    m = pa.tree_metadata(d["parents"], d["ctx"], d["bt"], B, d["lens"], stream=stream)
    q, k, v = d["qkv"][:, :HQ], d["qkv"][:, HQ:HQ + HKV], d["qkv"][:, HQ + HKV:]
    q = pa.rope_store_kvcache(q, k, v, m.positions, r, d["kc"], d["vc"], m.slot_mapping, stream=stream)
    out = pa.decode_tree(q.view(-1, T, HQ, D), d["kc"], d["vc"], d["bt"], d["ctx"], m.tree_mask, SCALE, d["lens"], ws,
                         stream=stream)
    kept = pa.verify_drafts(d["logits"], d["tokens"], d["parents"], d["u"], d["noise"], d["temps"], draft_lens=d["lens"],
                            stream=stream)
    pa.compact_kvcache(d["kc"], d["vc"], d["bt"], d["ctx"], kept.nodes, kept.counts, d["lens"], stream=stream)
    return out, kept


def check(s, d, out, kept):
    """A step against the definitions, and its cache against one in which the kept
    tokens alone were stored, one after the other."""
    assert pa.get_device_error() == (0, 0)
    kc, vc = s.kc.copy(), s.vc.copy()
    sees = [OD.ancestors(p) for p in s.parents]
    r = ROPE["r"]
    pos = np.zeros(s.batch * T, np.int32)
    for b in range(s.batch):
        n = s.lens[b]
        pos[b * T:b * T + n] = s.ctx[b] - n + sees[b][1][:n]
    q, k = pa.rope(dev_bf16(s.qkv[:, :HQ]), dev_bf16(s.qkv[:, HQ:HQ + HKV]), dev_i32(pos), r)  # (tested elsewhere)
    q, k, v = host_f64(q).reshape(-1, T, HQ, D), host_bits(k), s.qkv[:, HQ + HKV:]
    for b in range(s.batch):
        for i in range(s.lens[b]):
            p = s.ctx[b] - s.lens[b] + i
            kc[s.bt[b, p // B], p % B], vc[s.bt[b, p // B], p % B] = k[b * T + i], v[b * T + i]
    want, tol = OD.decode_tree(q, f64(kc), f64(vc), s.bt, s.ctx, [x[0] for x in sees], SCALE, s.lens)
    assert np.all(np.abs(host_f64(out) - want) <= tol)
    t, nodes, counts, margin = OD.verify(s.logits, s.tokens, s.parents, s.u, s.noise, s.temps, None, s.lens)
    assert np.all(margin[s.lens > 0] > 2.0 ** -14)
    assert np.array_equal(kept.tokens.cpu().numpy(), t) and np.array_equal(kept.nodes.cpu().numpy(), nodes)
    assert np.array_equal(kept.counts.cpu().numpy(), counts)
    kc, vc = (OD.compact(c, s.bt, s.ctx, nodes, counts, s.lens) for c in (kc, vc))
    assert np.array_equal(host_bits(d["kc"]), kc) and np.array_equal(host_bits(d["vc"]), vc)
    line, after = s.kc.copy(), s.ctx - s.lens + counts
    for b in range(s.batch):
        for j in range(counts[b]):
            p = s.ctx[b] - s.lens[b] + j
            line[s.bt[b, p // B], p % B] = k[b * T + nodes[b, j]]
    for b in range(s.batch):
        assert np.array_equal(OD.rows_of(kc, s.bt[b], after[b]), OD.rows_of(line, s.bt[b], after[b]))
    return counts


LENS = [9, 9, 0, 1, 5, 9, 9, 3]
BEFORE = [0, 17, 0, 100, 31, 64, 90, 7]


def test_a_step():
    s = Step(1, BEFORE, LENS)
    d = s.device()
    counts = check(s, d, *run(d, pa.decode_tree_workspace(HQ, HKV, D, T)))
    assert counts.max() > 2
    # The next step's decode reads the kept path: the same as over a cache that never saw the others.
    ctx = dev_i32(s.ctx - s.lens + counts)
    q = dev_bf16(bits(s.rng, s.batch, HQ, D))
    a = pa.decode(q, d["kc"], d["vc"], d["bt"], ctx, SCALE)
    b = pa.decode_tree(q[:, None], d["kc"], d["vc"], d["bt"], ctx, None, SCALE)[:, 0]
    assert torch.all((a.float() - b.float()).abs() <= 2e-2) and pa.get_device_error() == (0, 0)


def test_steps_on_streams_of_their_own():
    """Two steps at once, each with its workspace, inputs made on the stream that uses them."""
    steps = [Step(i, BEFORE, LENS) for i in (2, 3)]
    streams = [torch.cuda.Stream() for _ in steps]
    results = []
    for s, st in zip(steps, streams):
        with torch.cuda.stream(st):
            results.append((s.device(), pa.decode_tree_workspace(HQ, HKV, D, T)))
    outs = [None, None]
    for _ in range(5):
        for i, ((d, ws), st, s) in enumerate(zip(results, streams, steps)):
            with torch.cuda.stream(st):
                d["kc"].copy_(dev_bf16(s.kc))
                d["vc"].copy_(dev_bf16(s.vc))
                outs[i] = run(d, ws)
    torch.cuda.synchronize()
    for s, (d, _), o in zip(steps, results, outs):
        check(s, d, *o)


def test_the_stream_argument():
    s = Step(4, BEFORE, LENS)
    d, ws = s.device(), pa.decode_tree_workspace(HQ, HKV, D, T)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o = run(d, ws, stream=st)
    st.synchronize()
    check(s, d, *o)


def test_steps_captured_into_graphs_that_share_a_workspace():
    """Two graphs over one workspace, replayed in turn on changed inputs."""
    steps = [Step(i, BEFORE, LENS) for i in (5, 6, 7, 8)]
    ws = pa.decode_tree_workspace(HQ, HKV, D, T)
    side = torch.cuda.Stream()
    made = []
    with torch.cuda.stream(side):
        for s in steps[:2]:
            d = s.device()
            run(d, ws)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                o = run(d, ws)
            made.append((d, g, o))
        for turn in range(2):
            for (d, g, o), s in zip(made, steps[2 * turn:2 * turn + 2]):
                for name, x in s.device().items():
                    if name in ("kc", "vc") and x.shape[0] != d[name].shape[0]:
                        n = min(len(x), len(d[name]))
                        d[name][:n].copy_(x[:n])
                    else:
                        d[name].copy_(x)
                g.replay()
                torch.cuda.synchronize()
                pool = len(d["kc"])
                s.kc, s.vc = (np.concatenate([c, c[:max(0, pool - len(c))]])[:pool] for c in (s.kc, s.vc))
                check(s, d, *o)


def test_the_same_call_gives_the_same_bits():
    s = Step(9, [60] * 8, [9] * 8)
    d, ws = s.device(), pa.decode_tree_workspace(16, 2, D, 40)
    rng = np.random.default_rng(0)
    kc, vc = dev_bf16(bits(rng, 400, B, 2, D)), dev_bf16(bits(rng, 400, B, 2, D))
    bt = torch.randperm(400, device="cuda").to(torch.int32).view(2, 200)
    for t, hq in ((5, 2), (40, 16)):
        q = dev_bf16(bits(rng, 2, t, hq, D))
        args = (q, kc, vc, bt, dev_i32([3200, 1999]))
        want = pa.decode_tree(*args, workspace=ws)
        for _ in range(20):
            assert torch.equal(pa.decode_tree(*args, workspace=ws), want)
    kept = run(d, None)[1]
    assert all(torch.equal(x, y) for x, y in zip(kept, run(s.device(), None)[1]))


def test_offsets_beyond_32_bits():
    """Pools of more than 2^31 elements, and rows of logits and draft probabilities
    more than 2^31 elements from the first."""
    rng = np.random.default_rng(10)
    nb = (1 << 31) // (256 * HKV * D) + 40
    kc, vc = (torch.zeros(nb, 256, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 7
    q, k, v = bits(rng, n, HQ, D), bits(rng, n, HKV, D), bits(rng, n, HKV, D)
    base = (nb - 2) * 256 + 250
    slots = dev_i32(np.arange(n) + base)
    r = pa.rope_frequencies(D, 1e4)
    pos = dev_i32(np.arange(n) + 250)
    rq, rk = pa.rope(dev_bf16(q), dev_bf16(k), pos, r)
    oq = pa.rope_store_kvcache(dev_bf16(q), dev_bf16(k), dev_bf16(v), pos, r, kc, vc, slots)
    assert torch.equal(oq, rq) and torch.equal(kc.view(-1, HKV, D)[base:base + n], rk)
    assert torch.equal(vc.view(-1, HKV, D)[base:base + n], dev_bf16(v))
    bt = dev_i32([[nb - 2, nb - 1]])
    out = pa.decode_tree(oq[None], kc, vc, bt, dev_i32([257]), None, SCALE)
    hk, hv = (host_f64(c[nb - 2:]).reshape(512, HKV, D)[:257] for c in (kc, vc))
    want, tol = OD.decode_tree(host_f64(oq)[None], hk[None], hv[None], np.zeros((1, 2), np.int32), [257],
                               [np.tril(np.ones((n, n), bool))], SCALE)
    assert np.all(np.abs(host_f64(out) - want) <= tol)
    pa.compact_kvcache(kc, vc, bt, dev_i32([257]), dev_i32([[0, 2, 5, 6, -1, -1, -1]]), dev_i32([4]))
    assert torch.equal(kc.view(-1, HKV, D)[base:base + 4], rk[[0, 2, 5, 6]])
    assert pa.get_device_error() == (0, 0)
    del kc, vc
    vocab, nodes, batch = 200003, 64, 170  # 170 * 64 rows: 2.2e9 logits
    wide = -(-vocab // 8) * 8
    logits = torch.zeros(batch, nodes, wide, dtype=torch.bfloat16, device="cuda")[..., :vocab]
    probs = torch.zeros(batch, nodes, wide, device="cuda")[..., :vocab]
    tokens = rng.integers(0, vocab, (batch, nodes)).astype(np.int32)
    logits[-1, torch.arange(63), torch.from_numpy(tokens[-1, 1:].astype(np.int64)).cuda()] = 60.0
    logits[-1, 63, 77777] = 60.0
    probs[-1, torch.arange(63), torch.from_numpy(tokens[-1, 1:].astype(np.int64)).cuda()] = 1.0
    kept = pa.verify_drafts(logits, dev_i32(tokens), None, torch.full((batch, nodes), 0.5, device="cuda"),
                            torch.ones(batch, wide, device="cuda")[:, :vocab], torch.ones(batch, device="cuda"),
                            draft_probs=probs)
    assert int(kept.counts[-1]) == nodes and kept.tokens[-1].tolist() == tokens[-1, 1:].tolist() + [77777]
    assert pa.get_device_error() == (0, 0)


def test_infinite_temperatures_and_numbers_at_their_ends():
    rng = np.random.default_rng(11)
    logits = torch.zeros(3, 2, 40, device="cuda")
    logits.copy_(torch.from_numpy(rng.standard_normal((3, 2, 40)).astype(np.float32)) * 1e30)
    logits[:, :, 0] = float("-inf")
    noise = np.ones((3, 40), np.float32)
    noise[:, 17] = 0.5
    r = pa.verify_drafts(logits, dev_i32([[0, 0], [0, 3], [0, 3]]), None,
                         torch.tensor([[0.0, 0.0], [0.0, 0.0], [0.0, 0.5]], device="cuda"),
                         torch.from_numpy(noise).cuda(), torch.full((3,), float("inf"), device="cuda"))
    # Equal probabilities to all but the -inf: token 0 is never kept, 3 is at u = 0.
    assert r.tokens.tolist() == [[17, -1], [3, 17], [17, -1]] and r.counts.tolist() == [1, 2, 1]


@pytest.mark.parametrize("batch,n,vocab", [(2, 12, 40000), (3, 5, 40000), (12, 6, 20000)])
def test_verification_captured_and_on_two_streams_at_once(batch, n, vocab):
    """Wide clusters too: replays follow what the buffers hold, and calls on two
    streams at once do not meet."""
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits = torch.randn(batch, n, vocab, device="cuda", generator=g) * 3
        q = torch.softmax(logits[:, :n - 1] + torch.randn(batch, n - 1, vocab, device="cuda", generator=g) * 0.3, -1)
        tok = torch.zeros(batch, n, dtype=torch.int32, device="cuda")
        for c in range(1, n):
            tok[:, c] = torch.multinomial(q[:, c - 1], 1, generator=g)[:, 0].int()
        return [logits, tok, torch.rand(batch, n, device="cuda", generator=g),
                torch.empty(batch, vocab, device="cuda").exponential_(generator=g),
                torch.ones(batch, device="cuda"), q]

    def run(x, out=None):
        return pa.verify_drafts(x[0], x[1], None, x[2], x[3], x[4], draft_probs=x[5], out=out)

    sets = [inputs(s) for s in (1, 2, 3)]
    want = [run(x) for x in sets]
    assert any(int(w.counts.max()) > 2 for w in want)
    held = [t.clone() for t in sets[0]]
    out = pa.Verified(*(torch.empty_like(t) for t in want[0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(held, out)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run(held, out)
    torch.cuda.current_stream().wait_stream(side)
    for x, w in zip(sets, want):
        for t, s in zip(held, x):
            t.copy_(s)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(8):
        for i, (s, x) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(run(x))
    torch.cuda.synchronize()
    for gs, w in zip(got, want):
        assert all(torch.equal(a, b) for r in gs for a, b in zip(r, w))
    assert pa.get_device_error() == (0, 0)
