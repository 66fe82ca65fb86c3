"""GPU parity of the speculative-decoding entry points with their float64
definitions (oracle/drafts.py), within the bounds that the oracle derives; copies
and whole numbers exactly."""
import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import drafts as OD
from paged_kv_cache_store_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits
from gpu_util import dev_bf16, dev_i32, host_bits, host_f64

pytestmark = pytest.mark.gpu


def bits(rng, *shape, std=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


def f64(b):
    return bf16_bits_to_f32(b).astype(np.float64)


def near(got, want, tol, what=""):
    ok = (np.abs(got - want) <= tol) | (np.isnan(want) & np.isnan(got)) | (got == want)
    assert np.all(ok), (what, int((~ok).sum()), float(np.nanmax(np.abs(got - want) - tol)))


# ---------------------------------------------------------------- rope

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [16, 32, 64, 80, 96, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 3), (16, 8), (64, 8)])
def test_rope_and_store(hq, hkv, rotary, interleaved):
    rng = np.random.default_rng(hq * 1000 + rotary)
    for n in (1, 5, 77):
        q, k, v = bits(rng, n, hq, 128), bits(rng, n, hkv, 128, std=3), bits(rng, n, hkv, 128)
        pos = rng.integers(0, 1 << 20, n).astype(np.int32)
        scaling = [None, ("linear", 2.0), ("ntk", 4.0), ("yarn", 4.0, 4096.0)][n % 4]
        norm = n != 5
        w = [bits(rng, 128) for _ in range(2)] if norm else [None, None]
        W = [None if x is None else dev_bf16(x) for x in w]
        r = pa.rope_frequencies(rotary, 1e4, scaling, interleaved)
        P = dev_i32(pos)
        want = [OD.rope(f64(x), pos, rotary, 1e4, scaling, interleaved, None if y is None else f64(y))
                for x, y in ((q, w[0]), (k, w[1]))]
        oq, ok = pa.rope(dev_bf16(q), dev_bf16(k), P, r, *W)
        near(host_f64(oq), *want[0], "q")
        near(host_f64(ok), *want[1], "k")
        # The store: what rope and store_kvcache leave, in a pool that keeps its other rows.
        pool = bits(rng, 9, 16, hkv, 128)
        slots = rng.permutation(9 * 16)[:n].astype(np.int32)
        slots[::3] = -1
        kc, vc, kc2, vc2 = (dev_bf16(pool) for _ in range(4))
        S = dev_i32(slots)
        oq2 = pa.rope_store_kvcache(dev_bf16(q), dev_bf16(k), dev_bf16(v), P, r, kc, vc, S, *W)
        pa.store_kvcache(ok, dev_bf16(v), kc2, vc2, S)
        assert torch.equal(oq2, oq) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert pa.get_device_error() == (0, 0)


def test_rope_inside_a_fused_projection_and_in_place():
    rng = np.random.default_rng(5)
    qkv_h = bits(rng, 33, 24, 128)
    pos = rng.integers(0, 4000, 33).astype(np.int32)
    r, P = pa.rope_frequencies(128, 1e6), dev_i32(pos)
    qkv = dev_bf16(qkv_h)
    q, k = qkv[:, :16], qkv[:, 16:20]
    wq, wk = OD.rope(f64(qkv_h[:, :16]), pos, 128, 1e6), OD.rope(f64(qkv_h[:, 16:20]), pos, 128, 1e6)
    a, b = pa.rope(q, k, P, r)
    near(host_f64(a), *wq)
    near(host_f64(b), *wk)
    c, d = pa.rope(q, k, P, r, out_q=q, out_k=k)
    assert c is q and torch.equal(q, a) and torch.equal(k, b)
    assert np.array_equal(host_bits(qkv[:, 20:]), qkv_h[:, 20:])   # the values beside them
    one, _ = pa.rope(qkv[:1, :16], qkv[:1, 16:20], P[:1], r)       # a lone row's stride does not matter
    assert one.shape == (1, 16, 128)


def test_rope_far_and_negative_positions():
    rng = np.random.default_rng(6)
    pos = np.array([0, 1, 131071, 1 << 24, (1 << 24) + 1, (1 << 31) - 1, -1, -(1 << 31), 1 << 30], np.int32)
    q, k = bits(rng, 9, 2, 128), bits(rng, 9, 1, 128)
    r = pa.rope_frequencies(128, 1e4)
    # The oracle's angles: exact products of the table, which is f_i to 2^-64 turns.
    turns = np.array([[int(p) * int(f) % (1 << 64) for f in r.freqs.tolist()] for p in pos], np.float64) / 2.0 ** 64
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    x = f64(q)
    want = np.concatenate([x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s], -1)
    _, tol = OD.rope(x, np.zeros(9), 128, 1e4)
    size = np.abs(x[..., :64]) + np.abs(x[..., 64:])
    tol = np.concatenate([size, size], -1) * 2.0 ** -19
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    near(host_f64(pa.rope(dev_bf16(q), dev_bf16(k), dev_i32(pos), r)[0]), want, tol)


def test_rope_norm_of_large_and_small_heads():
    rng = np.random.default_rng(7)
    q = bits(rng, 6, 2, 128)
    scale = np.array([1e-30, 1e-4, 1.0, 1e4, 1e15, 0.0], np.float32)
    q = f32_to_bf16_bits(bf16_bits_to_f32(q) * scale[:, None, None])
    w = bits(rng, 128)
    r = pa.rope_frequencies(64, 1e4)
    pos = np.arange(6, dtype=np.int32)
    want = OD.rope(f64(q), pos, 64, 1e4, weight=f64(w))
    got = pa.rope(dev_bf16(q), dev_bf16(q), dev_i32(pos), r, dev_bf16(w), None)[0]
    near(host_f64(got), *want)


def test_rope_bad_slot_is_recorded():
    rng = np.random.default_rng(8)
    q, k = dev_bf16(bits(rng, 3, 4, 128)), dev_bf16(bits(rng, 3, 2, 128))
    pool = bits(rng, 2, 16, 2, 128)
    kc, vc = dev_bf16(pool), dev_bf16(pool)
    r = pa.rope_frequencies()
    pa.rope_store_kvcache(q, k, k, dev_i32([0, 1, 2]), r, kc, vc, dev_i32([-5, 32, -1]))
    assert pa.get_device_error() == (pa.PA_DEV_BAD_SLOT, 1)
    assert np.array_equal(host_bits(kc), pool) and np.array_equal(host_bits(vc), pool)


# ---------------------------------------------------------------- trees and their attention

class Tree:
    """A batch with scattered tables, its drafts' rows in the pool."""

    def __init__(self, seed, before, T, hq, hkv, B, lens=None, parents=None, spare=3):
        rng = self.rng = np.random.default_rng(seed)
        batch = len(before)
        self.lens = None if lens is None else np.array(lens, np.int32)
        n = np.full(batch, T) if lens is None else self.lens
        self.ctx = (np.array(before) + n).astype(np.int32)
        need = -(-self.ctx // B)
        nb = int(need.sum()) + spare
        ids = rng.permutation(nb)
        self.bt = np.full((batch, int(need.max()) + 1), -1, np.int32)
        at = 0
        for b in range(batch):
            self.bt[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.parents = np.stack([OD.random_parents(rng, T) for _ in range(batch)]) if parents is None else parents
        self.sees = [OD.ancestors(p)[0] for p in self.parents]
        self.kc, self.vc = bits(rng, nb, B, hkv, 128), bits(rng, nb, B, hkv, 128)
        self.q = bits(rng, batch, T, hq, 128)
        self.scale, self.B, self.T = 1 / np.sqrt(128), B, T

    def masks(self):
        return torch.from_numpy(np.stack([OD.as_bits(s) for s in self.sees])).cuda()

    def run(self, **kw):
        a = dict(q=dev_bf16(self.q), k_cache=dev_bf16(self.kc), v_cache=dev_bf16(self.vc), block_tables=dev_i32(self.bt),
                 context_lens=dev_i32(self.ctx), tree_mask=self.masks(), softmax_scale=self.scale,
                 draft_lens=None if self.lens is None else dev_i32(self.lens))
        a.update(kw)
        return pa.decode_tree(**a)

    def check(self, **kw):
        out = self.run(**kw)
        assert pa.get_device_error() == (0, 0)
        want, tol = OD.decode_tree(f64(self.q), f64(self.kc), f64(self.vc), self.bt, self.ctx, self.sees, self.scale,
                                   self.lens)
        near(host_f64(out), want, tol, (self.ctx.tolist()[:8], self.T))
        return out


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 16, 17, 31, 32, 33, 63, 64])
def test_tree_sizes_and_groups(T, hq, hkv):
    Tree(T * 10 + hq, [0, 1, 62, 63, 64, 65, 127, 200, 450], T, hq, hkv, 64).check()


@pytest.mark.parametrize("B", [16, 32, 48, 64, 80, 128, 256, 512])
def test_block_sizes(B):
    Tree(B, [0, B - 1, B, B + 1, 2 * B + 7, 700], 7, 4, 2, B).check()
    Tree(B + 1, [3, 300], 64, 8, 1, B).check()


@pytest.mark.parametrize("hq,hkv,before", [(8, 2, [9000, 3, 4097, 700]), (8, 1, [20000]), (32, 8, [5000, 5001]),
                                           (1, 1, [30000, 17])])
def test_items_cut_between_many_ctas(hq, hkv, before):
    for T in (1, 5, 40):
        Tree(T + hq, before, T, hq, hkv, 256).check()


@pytest.mark.parametrize("T,hq,hkv,tiles", [(5, 8, 2, 6), (5, 8, 2, 7), (40, 8, 2, 10), (40, 8, 2, 11), (3, 4, 4, 17)])
def test_short_items_whole_and_cut(T, hq, hkv, tiles):
    """Block tables too short for a cut, so that one kernel does it all, and just long enough."""
    rng = np.random.default_rng(tiles)
    for batch in (1, 3, 19, 40, 77):
        before = rng.integers(0, 64 * tiles - T + 1, batch)
        before[0] = 64 * tiles - T
        t = Tree(tiles + batch, before, T, hq, hkv, 64)
        t.bt = np.ascontiguousarray(t.bt[:, :tiles])
        t.check()


def test_the_workspace_may_hold_anything():
    for T, hq, hkv, before in ((5, 8, 2, [9000, 40, 700]), (40, 8, 2, [5000, 3]), (64, 8, 1, [300, 9000])):
        t = Tree(T, before, T, hq, hkv, 64)
        ws = pa.decode_tree_workspace(hq, hkv, 128, T)
        want = t.check(workspace=ws.fill_(0))
        assert torch.equal(t.run(workspace=ws), want)
        assert torch.equal(t.run(workspace=ws.fill_(255)), want)
        assert torch.equal(t.run(workspace=ws.random_()), want)


def test_ragged_batches_and_padding():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 17, 40)
    lens[:3] = 0, 16, 1
    before = rng.integers(0, 500, 40) * (lens > 0)
    t = Tree(11, before, 16, 16, 8, 256, lens=lens)
    out = t.check(out=torch.full((40, 16, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda"))
    for b in range(40):
        assert not out[b, lens[b]:].any()


def test_ragged_row_blocks():
    """Rows of a sequence over several row blocks and half blocks, some of them empty."""
    Tree(12, [100, 5, 300, 64], 64, 8, 1, 64, lens=[64, 1, 17, 33]).check()
    Tree(13, [100, 5, 300], 64, 16, 2, 64, lens=[16, 48, 32]).check()


def test_chain_without_a_mask():
    for T in (1, 6, 64):
        chain = np.broadcast_to(np.arange(T) - 1, (3, T))
        t = Tree(T, [0, 77, 600], T, 8, 4, 128, parents=chain)
        a, b = t.check(), t.check(tree_mask=None)
        assert torch.equal(a, b)


def test_one_draft_is_a_decode_step():
    t = Tree(20, [0, 5, 255, 256, 3000], 1, 16, 8, 256)
    out = t.check()
    ref = pa.decode(dev_bf16(t.q[:, 0]), dev_bf16(t.kc), dev_bf16(t.vc), dev_i32(t.bt), dev_i32(t.ctx), t.scale)
    want, tol = OD.decode_tree(f64(t.q), f64(t.kc), f64(t.vc), t.bt, t.ctx, t.sees, t.scale)
    near(host_f64(ref), want[:, 0], 2 * tol[:, 0])  # two kernels, each within its bound
    near(host_f64(out)[:, 0], host_f64(ref), 2 * tol[:, 0])


def test_any_pattern_and_rows_that_see_nothing():
    rng = np.random.default_rng(21)
    t = Tree(21, [0, 0, 64, 130, 0], 24, 8, 4, 64)
    t.sees = [rng.random((24, 24)) < 0.2 for _ in range(5)]
    t.sees[0][:] = False          # no context, nothing seen
    t.sees[1][5:] = False
    t.sees[4][::2] = False
    out = t.check()
    assert not out[0].any()


def test_mask_bits_past_the_drafts_do_not_count():
    t = Tree(22, [10, 70], 8, 4, 4, 16, lens=[3, 8])
    m = t.masks()
    noisy = m | (torch.tensor([-1 << 3, -1 << 8], device="cuda")[:, None] & ~0)
    assert torch.equal(t.run(tree_mask=noisy), t.run(tree_mask=m))


@pytest.mark.parametrize("T,hq,hkv", [(9, 8, 2), (64, 8, 1), (64, 8, 2)])
def test_hidden_values_do_not_matter(T, hq, hkv):
    """NaN and infinities in keys and values of drafts that a row does not see, and in
    slots past the last key; rows that see them follow the formula."""
    t = Tree(T, [5, 64, 1000], T, hq, hkv, 64)
    clean = host_f64(t.run())
    bad = T // 2
    for b in range(3):
        p = t.ctx[b] - T + bad
        blk, off = t.bt[b, p // 64], p % 64
        t.kc[blk, off, :, 3] = 0x7FC0              # NaN
        t.vc[blk, off, 0, 7] = 0x7FC0
        t.vc[blk, off, -1, 9] = 0x7F80             # +inf
        t.vc[blk, off, -1, 11] = 0xFF80            # -inf
        last, lo = t.bt[b, t.ctx[b] // 64 if t.ctx[b] % 64 else 0], t.ctx[b] % 64
        if lo:
            t.kc[last, lo:] = 0x7FC0
            t.vc[last, lo:] = 0x7F80
    got = host_f64(t.run())
    for b in range(3):
        for i in range(T):
            if t.sees[b][i, bad]:
                assert np.all(np.isnan(got[b, i]))  # its score is NaN
            else:
                assert np.array_equal(got[b, i], clean[b, i])
    # Values alone: seen rows get the infinity and the NaN in those dimensions only.
    t.kc = np.where(t.kc == 0x7FC0, 0x3F80, t.kc).astype(np.uint16)
    t.check_v = host_f64(t.run())
    want, tol = OD.decode_tree(f64(t.q), f64(t.kc), np.where(np.isfinite(f64(t.vc)), f64(t.vc), 0), t.bt, t.ctx, t.sees,
                               t.scale)
    G = hq // hkv
    for b in range(3):
        for i in range(T):
            seen = t.sees[b][i, bad]
            w = want[b, i].copy()
            if seen:
                w[:G, 7] = np.nan
                w[-G:, 9], w[-G:, 11] = np.inf, -np.inf
            near(t.check_v[b, i], w, tol[b, i], (b, i))


def test_scores_of_every_size():
    for std in (1e-3, 3.0, 30.0):
        t = Tree(int(std), [0, 300, 1500], 6, 8, 4, 64)
        t.q = bits(t.rng, 3, 6, 8, 128, std=std)
        t.check()


def test_many_sequences():
    rng = np.random.default_rng(30)
    Tree(30, rng.integers(0, 40, 2048), 3, 2, 1, 16).check()


def test_strided_queries_and_given_outputs():
    t = Tree(31, [7, 300], 5, 8, 4, 64)
    want = t.check()
    wide = torch.full((2, 5, 20, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 4:12] = dev_bf16(t.q)
    ws = pa.decode_tree_workspace(8, 4, 128, 64)
    out = torch.empty_like(want)
    assert t.run(q=wide[:, :, 4:12], workspace=ws, out=out) is out and torch.equal(out, want)
    assert torch.equal(t.run(workspace=ws), want)
    ws2 = pa.decode_tree_workspace(8, 4, 128, 5)
    Tree(311, [30000], 5, 8, 1, 64).check(workspace=pa.decode_tree_workspace(8, 1, 128, 5))
    t2 = Tree(312, [30000, 5], 5, 8, 4, 64)
    assert torch.equal(t2.check(workspace=ws2), t2.run(workspace=ws2))   # used before
    with pytest.raises(ValueError):
        t.run(q=wide[:, :3, 4:12])
    with pytest.raises(ValueError):
        t.run(tree_mask=t.masks()[:, :4])
    with pytest.raises(TypeError):
        t.run(tree_mask=t.masks().int())


def test_one_workspace_for_calls_of_many_shapes():
    ws = pa.decode_tree_workspace(8, 1, 128, 64)
    for T, hq, hkv, before in ((64, 8, 1, [4000, 100]), (1, 8, 8, [9000]), (5, 4, 1, [7000, 2, 3]), (64, 8, 1, [4000, 100])):
        t = Tree(T, before, T, hq, hkv, 64)
        assert torch.equal(t.check(workspace=ws), t.run())


def test_lengths_that_do_not_fit_are_recorded():
    t = Tree(33, [100, 200, 300], 4, 4, 2, 64)
    want, tol = OD.decode_tree(f64(t.q), f64(t.kc), f64(t.vc), t.bt, t.ctx, t.sees, t.scale)
    for ctx in (3, -1, t.bt.shape[1] * 64 + 1):
        c = t.ctx.copy()
        c[1] = ctx
        out = t.run(context_lens=dev_i32(c))
        assert pa.get_device_error() == (pa.PA_DEV_BAD_CONTEXT, 1)
        assert not out[1].any()
        # The others' keys are cut elsewhere without it: within the bound, not bit by bit.
        near(host_f64(out)[::2], want[::2], tol[::2])
    out = t.run(draft_lens=dev_i32([4, 5, 4]))
    assert pa.get_device_error() == (pa.PA_DEV_BAD_CONTEXT, 1) and not out[1].any()


def test_bad_block_ids_read_as_zeros_and_are_recorded_when_checked():
    t = Tree(34, [300], 4, 4, 2, 64)
    bt = t.bt.copy()
    bt[0, 1] = 1 << 20
    pa.set_checked(True)
    try:
        out = t.run(block_tables=dev_i32(bt))
        assert pa.get_device_error() == (pa.PA_DEV_BAD_BLOCK, 1)
    finally:
        pa.set_checked(False)
    t.kc[t.bt[0, 1]], t.vc[t.bt[0, 1]] = 0, 0
    assert torch.equal(out, t.run())


def test_metadata():
    rng = np.random.default_rng(40)
    for T in (1, 7, 64):
        lens = rng.integers(0, T + 1, 50)
        before = rng.integers(0, 300, 50) * (lens > 0)
        t = Tree(T, before, T, 1, 1, 48, lens=lens)
        m = pa.tree_metadata(dev_i32(t.parents), dev_i32(t.ctx), dev_i32(t.bt), 48, dev_i32(t.lens))
        assert pa.get_device_error() == (0, 0)
        mask, pos, slots = (x.cpu().numpy().reshape(50, T) for x in m)
        for b in range(50):
            n, first = lens[b], t.ctx[b] - lens[b]
            sees, depth = OD.ancestors(t.parents[b])
            p = first + np.arange(n)
            assert np.array_equal(mask[b, :n], OD.as_bits(sees)[:n]) and np.array_equal(pos[b, :n], first + depth[:n])
            assert np.array_equal(slots[b, :n], t.bt[b, p // 48] * 48 + p % 48)
            assert np.all(mask[b, n:] == 0) and np.all(pos[b, n:] == 0) and np.all(slots[b, n:] == -1)
        if T > 1:
            chain = pa.tree_metadata(None, dev_i32(t.ctx), dev_i32(t.bt), 48, dev_i32(t.lens), num_drafts=T)
            same = pa.tree_metadata(dev_i32(np.broadcast_to(np.arange(T) - 1, (50, T))), dev_i32(t.ctx), dev_i32(t.bt),
                                    48, dev_i32(t.lens))
            assert all(torch.equal(x, y) for x, y in zip(chain, same))


def test_metadata_records_bad_trees_and_lengths():
    t = Tree(41, [100, 200], 5, 1, 1, 16)
    par = t.parents.copy()
    par[1, 3] = 3
    pa.tree_metadata(dev_i32(par), dev_i32(t.ctx), dev_i32(t.bt), 16)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TREE, 8)
    m = pa.tree_metadata(dev_i32(t.parents), dev_i32([105, 3]), dev_i32(t.bt), 16)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_CONTEXT, 1)
    assert not m.tree_mask[1].any() and torch.all(m.slot_mapping[5:] == -1)


# ---------------------------------------------------------------- verification

def place(x, dtype, pad=0):
    x = np.asarray(x)
    t = torch.full((*x.shape[:-1], -(-x.shape[-1] // 8) * 8 + pad), float("nan"), dtype=dtype,
                   device="cuda")[..., :x.shape[-1]]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return t


def verify_case(seed, batch, T, vocab, dtype, drawn, chain=False, lens=None, temps=None, close=0.5, peak=3.0):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((batch, T, vocab)) * peak
    parents = np.stack([np.arange(T) - 1 if chain else OD.random_parents(rng, T) for _ in range(batch)]).astype(np.int32)
    temps = np.ones(batch, np.float32) if temps is None else np.asarray(temps, np.float32)
    x = (logits + close * rng.standard_normal(logits.shape)) / temps[:, None, None]
    e = np.exp(x - x.max(-1, keepdims=True))
    probs = (e / e.sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.zeros((batch, T), np.int32)
    for b in range(batch):
        order = {}
        for c in range(1, T):
            v = int(parents[b, c])
            k = order[v] = order.get(v, -1) + 1
            if drawn:
                tokens[b, c] = np.argmax(x[b, v] + rng.gumbel(size=vocab))
            else:
                tokens[b, c] = np.argsort(-x[b, v])[min(k, vocab - 1)]
    return dict(logits=place(logits.astype(np.float32), dtype), tokens=tokens, parents=parents,
                u=rng.random((batch, T)).astype(np.float32), noise=rng.exponential(size=(batch, vocab)).astype(np.float32),
                temps=temps, probs=probs if drawn else None, lens=lens)


def run_verify(s, **kw):
    a = dict(logits=s["logits"], tokens=dev_i32(s["tokens"]), parents=dev_i32(s["parents"]),
             uniforms=torch.from_numpy(s["u"]).cuda(), exp_noise=place(s["noise"], torch.float32),
             temperatures=torch.from_numpy(s["temps"]).cuda(),
             draft_probs=None if s["probs"] is None else place(s["probs"], torch.float32),
             draft_lens=None if s["lens"] is None else dev_i32(s["lens"]))
    a.update(kw)
    return pa.verify_drafts(**a)


def check_verify(s, **kw):
    """Every sequence whose decisions are further from the other way than fp32 sums
    and exponentials can be off (2^-14; a probability of a row this wide is off by
    under 2^-17, a difference of two by that of the larger)."""
    r = run_verify(s, **kw)
    assert pa.get_device_error() == (0, 0)
    t, nodes, counts, margin = OD.verify(s["logits"].double().cpu().numpy(), s["tokens"], s["parents"], s["u"], s["noise"],
                                         s["temps"], s["probs"], s["lens"])
    sure = margin > 2.0 ** -14
    assert sure.mean() > 0.9
    for got, want in zip(r, (t, nodes, counts)):
        assert np.array_equal(got.cpu().numpy()[sure], want[sure])
    return counts


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 500, 2049, 4096, 5003])
def test_verify_vocabularies(vocab, dtype, drawn):
    check_verify(verify_case(vocab, 24, 6, vocab, dtype, drawn))


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 17, 32, 33, 64])
def test_verify_tree_sizes(T, drawn):
    counts = check_verify(verify_case(T, 20, T, 700, torch.bfloat16, drawn, close=0.3))
    counts2 = check_verify(verify_case(T + 100, 20, T, 700, torch.float32, drawn, chain=True, close=0.05))
    if T >= 5:
        assert counts2.max() > 3 or counts.max() > 1


@pytest.mark.parametrize("batch", [1, 2, 37, 150, 310, 700])
def test_verify_batches(batch):
    """Every cluster size, and more sequences than run at once."""
    check_verify(verify_case(batch, batch, 4, 20011, torch.bfloat16, batch % 2 == 0))


@pytest.mark.parametrize("batch,T,vocab,chain,drawn,dtype", [
    (1, 8, 151936, True, True, torch.bfloat16),      # a short drawn chain: its rows at once
    (3, 9, 151936, True, True, torch.bfloat16),      # one node more: one after the other
    (5, 8, 151936, True, False, torch.bfloat16), (2, 8, 151936, False, True, torch.float32),
    (40, 6, 50021, True, True, torch.float32), (5, 33, 40000, False, False, torch.bfloat16),
    (4, 64, 32768, False, True, torch.bfloat16), (20, 64, 1100, False, True, torch.float32),
    (20, 64, 1027, False, False, torch.bfloat16)])
def test_verify_rows_at_once_and_one_after_the_other(batch, T, vocab, chain, drawn, dtype):
    check_verify(verify_case(batch + T, batch, T, vocab, dtype, drawn, chain=chain, close=0.1 if chain else 0.3))


def test_verify_a_sequence_has_the_same_result_in_either_way():
    """Trees and chains, long and short ones, in one batch; and a bad node, which leaves no chain."""
    s = verify_case(61, 6, 12, 40000, torch.bfloat16, True, chain=True, close=0.1,
                    lens=np.array([8, 9, 12, 1, 0, 8], np.int32))
    s["parents"][2, 6:] = 3
    counts = check_verify(s)
    assert counts[:2].max() > 2
    s["parents"][5, 7] = 9                    # past the node itself: out of the tree
    r = run_verify(s)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TREE, 5 * 12 + 7)
    t = dict(s, lens=np.array([8, 9, 12, 1, 0, 7], np.int32))
    want = run_verify(t)
    assert all(torch.equal(x, y) for x, y in zip(r, want))


def test_verify_masked_logits_of_many_rows():
    """The same masks where rows are read one after the other."""
    low = float(torch.finfo(torch.bfloat16).min)
    for mask in (-np.inf, low):
        for dtype in (torch.bfloat16, torch.float32):
            s = verify_case(62, 6, 64, 1203, dtype, False)
            s["logits"][:, :, ::3] = mask
            s["logits"][0] = mask
            s["logits"][1, :, 1:] = mask
            s["logits"][2, :, 5] = float("nan")
            s["logits"][3, :, 7] = float("inf")
            check_verify(s)


def test_verify_many_siblings():
    """Residuals of many rejected children, drawn and chosen: all under the root."""
    for drawn in (True, False):
        s = verify_case(50, 64, 33, 40, torch.float32, drawn, close=3.0)
        s["parents"] = np.broadcast_to(np.array([-1] + [0] * 32, np.int32), (64, 33)).copy()
        rng = np.random.default_rng(51)
        if drawn:
            p = s["probs"][:, 0].astype(np.float64)
            s["tokens"] = np.stack([rng.choice(40, 33, p=x / x.sum()) for x in p]).astype(np.int32)
        else:
            s["tokens"] = np.stack([rng.permutation(40)[:33] for _ in range(64)]).astype(np.int32)
            s["tokens"][:, 20] = s["tokens"][:, 3]  # a candidate given twice
        check_verify(s)


def test_verify_ragged_temperatures_and_padding():
    rng = np.random.default_rng(52)
    lens = rng.integers(0, 9, 60).astype(np.int32)
    lens[:2] = 0, 8
    s = verify_case(52, 60, 8, 3000, torch.bfloat16, True, lens=lens, temps=rng.uniform(0.2, 3.0, 60))
    check_verify(s)
    r = run_verify(s)
    assert int(r.counts[0]) == 0 and torch.all(r.tokens[0] == -1) and torch.all(r.nodes[0] == -1)


def test_verify_greedy():
    s = verify_case(53, 30, 6, 1000, torch.float32, False, close=0.01, temps=np.full(30, 1e-6))
    r = run_verify(s)
    lg = s["logits"].double().cpu().numpy()
    for b in range(30):
        v, kept = 0, []
        while True:
            best = int(lg[b, v].argmax())
            kept.append(best)
            nxt = [c for c in range(v + 1, 6) if s["parents"][b, c] == v and s["tokens"][b, c] == best]
            if not nxt:
                break
            v = nxt[0]
        assert r.tokens[b, :len(kept)].tolist() == kept and int(r.counts[b]) == len(kept)


def test_verify_equal_distributions_keep_everything():
    """q = p, as the kernel's own target would be: every draft is kept, whatever u."""
    s = verify_case(54, 16, 6, 4000, torch.float32, True, chain=True, close=0.0)
    s["u"][:] = 0.999
    assert np.all(check_verify(s) == 6)


def test_verify_masked_logits():
    low = float(torch.finfo(torch.bfloat16).min)
    for mask in (-np.inf, low):
        s = verify_case(55, 12, 5, 900, torch.bfloat16, False)
        s["logits"][:, :, ::3] = mask
        s["logits"][0] = mask                    # nothing, or everything alike
        s["logits"][1, :, 1:] = mask
        s["logits"][2, :, 5] = float("nan")
        s["logits"][3, :, 7] = float("inf")
        check_verify(s)
        d = verify_case(56, 12, 5, 900, torch.float32, True)
        d["logits"][:, :, ::2] = mask
        check_verify(d)


def test_verify_probabilities_of_zero():
    s = verify_case(57, 20, 4, 300, torch.float32, True)
    s["probs"][:, :, ::2] = 0.0
    s["u"][:5] = 0.0
    check_verify(s)
    s["probs"][:] = 0.0
    s["probs"][..., 3] = 1.0
    check_verify(s)


def test_verify_extreme_noise_and_lowest_index():
    s = verify_case(58, 4, 2, 100, torch.float32, False)
    s["logits"][:] = 0.0
    s["noise"][:] = 1.0
    s["tokens"][:] = 99
    s["u"][:] = 0.5
    r = run_verify(s)
    assert r.tokens[:, 0].tolist() == [0] * 4 and r.counts.tolist() == [1] * 4
    s["noise"][:, 41] = 0.0
    assert run_verify(s).tokens[:, 0].tolist() == [41] * 4
    s["noise"][:, 40] = 1e-12                     # the same after the clamp: the lower index
    assert run_verify(s).tokens[:, 0].tolist() == [40] * 4


def test_verify_chains_without_parents_and_strided_rows():
    s = verify_case(59, 10, 5, 777, torch.float32, True, chain=True)
    a = run_verify(s)
    b = run_verify(s, parents=None, logits=place(s["logits"].cpu().numpy(), torch.float32, pad=16),
                   draft_probs=place(s["probs"][:, :4], torch.float32, pad=8),
                   exp_noise=place(s["noise"], torch.float32, pad=8))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(ValueError):
        run_verify(s, draft_probs=place(s["probs"][:, :3], torch.float32))
    with pytest.raises(ValueError):
        run_verify(s, uniforms=torch.zeros(10, 4, device="cuda"))
    out = pa.Verified(*(torch.empty_like(x) for x in a))
    assert run_verify(s, out=out) is out and all(torch.equal(x, y) for x, y in zip(a, out))


def test_verify_records_bad_inputs():
    def same_but(r, want, b):
        keep = [i for i in range(6) if i != b]
        return all(torch.equal(x[keep], y[keep]) for x, y in zip(r, want))

    s = verify_case(60, 6, 5, 300, torch.float32, False)
    want = run_verify(s)
    t = dict(s, temps=s["temps"].copy())
    t["temps"][2] = 0.0
    r = run_verify(t)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TEMPERATURE, 2)
    assert int(r.counts[2]) == 0 and torch.all(r.tokens[2] == -1) and same_but(r, want, 2)
    t = dict(s, tokens=s["tokens"].copy())
    t["tokens"][1, 3] = 300
    r = run_verify(t)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TOKEN, 8) and 3 not in r.nodes[1].tolist() and same_but(r, want, 1)
    t = dict(s, parents=s["parents"].copy())
    t["parents"][4, 2] = 2
    r = run_verify(t)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TREE, 22) and 2 not in r.nodes[4].tolist() and same_but(r, want, 4)
    r = run_verify(s, draft_lens=dev_i32([5, 5, 5, 6, 5, 5]))
    assert pa.get_device_error() == (pa.PA_DEV_BAD_CONTEXT, 3) and int(r.counts[3]) == 0 and same_but(r, want, 3)


# ---------------------------------------------------------------- compaction

def random_paths(rng, parents, lens=None):
    batch, T = parents.shape
    nodes, counts = np.full((batch, T), -1, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        n = T if lens is None else lens[b]
        if n == 0:
            continue
        path = [0]
        for c in range(1, n):
            if parents[b, c] == path[-1] and rng.random() < 0.8:
                path.append(c)
        nodes[b, :len(path)], counts[b] = path, len(path)
    return nodes, counts


@pytest.mark.parametrize("T,hkv,B", [(1, 1, 16), (2, 3, 16), (9, 8, 48), (33, 2, 64), (64, 1, 16), (64, 8, 256)])
def test_compact(T, hkv, B):
    rng = np.random.default_rng(T)
    lens = rng.integers(0, T + 1, 30)
    t = Tree(T, rng.integers(0, 100, 30) * (lens > 0), T, hkv, hkv, B, lens=lens)
    for ragged in (True, False):
        n = lens if ragged else None
        keep = slice(None) if ragged else np.nonzero(t.ctx >= T)[0]
        ctx, bt, par = t.ctx[keep], t.bt[keep], t.parents[keep]
        nodes, counts = random_paths(rng, par, n)
        kc, vc = dev_bf16(t.kc), dev_bf16(t.vc)
        pa.compact_kvcache(kc, vc, dev_i32(bt), dev_i32(ctx), dev_i32(nodes), dev_i32(counts),
                           None if n is None else dev_i32(n))
        assert pa.get_device_error() == (0, 0)
        assert np.array_equal(host_bits(kc), OD.compact(t.kc, bt, ctx, nodes, counts, n))
        assert np.array_equal(host_bits(vc), OD.compact(t.vc, bt, ctx, nodes, counts, n))


def test_compact_all_layers():
    rng = np.random.default_rng(70)
    t = Tree(70, [5, 60, 0], 12, 2, 2, 16)
    nodes, counts = random_paths(rng, t.parents)
    pools = [[bits(rng, *t.kc.shape) for _ in range(5)] for _ in range(2)]
    whole = torch.stack([torch.stack([dev_bf16(x) for x in p]) for p in pools])  # [2, layers, ...]
    pa.compact_kvcache(whole[0], whole[1], dev_i32(t.bt), dev_i32(t.ctx), dev_i32(nodes), dev_i32(counts))
    for i in range(2):
        for x, layer in zip(pools[i], whole[i]):
            assert np.array_equal(host_bits(layer), OD.compact(x, t.bt, t.ctx, nodes, counts))
    # Layers further apart, and K and V interleaved by layer.
    mixed = torch.stack([torch.stack([dev_bf16(p[l]) for p in pools]) for l in range(5)])  # [layers, 2, ...]
    pa.compact_kvcache(mixed[:, 0], mixed[:, 1], dev_i32(t.bt), dev_i32(t.ctx), dev_i32(nodes), dev_i32(counts))
    assert torch.equal(mixed[:, 0], whole[0]) and torch.equal(mixed[:, 1], whole[1])
    assert pa.get_device_error() == (0, 0)
    args = [dev_i32(x) for x in (t.bt, t.ctx, nodes, counts)]
    pa.compact_kvcache(whole[0][:0], whole[1][:0], *args)
    with pytest.raises(ValueError):
        pa.compact_kvcache(whole[0][:1].expand(2, -1, -1, -1, -1), whole[1][:2], *args)
    with pytest.raises(ValueError):
        pa.compact_kvcache(whole[0].transpose(1, 2), whole[1].transpose(1, 2), *args)
    with pytest.raises(TypeError):
        pa.compact_kvcache(whole[0].float(), whole[1].float(), *args)


def test_compact_records_bad_paths_blocks_and_lengths():
    t = Tree(71, [20, 20], 6, 1, 1, 16)
    par = np.array([[0, 2, 4, 3, 5, -1], [0, 1, 3, 4, -1, -1]], np.int32)
    counts = np.array([5, 4], np.int32)

    def run(nodes, bt=t.bt, ctx=t.ctx):
        kc, vc = dev_bf16(t.kc), dev_bf16(t.vc)
        pa.compact_kvcache(kc, vc, dev_i32(bt), dev_i32(ctx), dev_i32(nodes), dev_i32(counts))
        return host_bits(kc), pa.get_device_error()

    got, err = run(par)
    assert err == (pa.PA_DEV_BAD_TREE, 3)
    assert np.array_equal(got, OD.compact(t.kc, t.bt, t.ctx, par, np.array([3, 4])))
    good = np.array([[0, 2, 4, -1, -1, -1], [0, 1, 3, 4, -1, -1]], np.int32)
    counts[0] = 3
    got, err = run(np.where(good == 4, 6, good))
    assert err[0] == pa.PA_DEV_BAD_TREE
    bt = t.bt.copy()
    bt[1, 1] = -1
    got, err = run(good, bt=bt)
    assert err == (pa.PA_DEV_BAD_BLOCK, bt.shape[1] + 1)
    assert np.array_equal(got, OD.compact(t.kc, t.bt, t.ctx, good, np.array([3, 0])))
    got, err = run(good, ctx=np.array([26, 5], np.int32))
    assert err == (pa.PA_DEV_BAD_CONTEXT, 1)
    assert np.array_equal(got, OD.compact(t.kc, t.bt, t.ctx, good, np.array([3, 0])))
