"""Speculative decoding where it can go wrong: calls that the documentation allows
and that the tests of each entry point's ordinary range do not reach."""
import ctypes as C
import glob
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import drafts as OD
from paged_kv_cache_store_gb300 import build as pabuild
from gpu_util import dev_i32, host_f64
from test_gpu_drafts import Tree, check_verify, f64, near, place, run_verify, verify_case

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- trees

@pytest.mark.parametrize("T,hq,lens", [(17, 8, (17, 16)), (17, 8, (17, 16, 16, 3)), (33, 8, (33, 1, 17)), (5, 8, (5, 4))])
def test_infinite_values_of_drafts_in_runs_of_short_sequences(T, hq, lens):
    """Many one-tile sequences a CTA, most second row tiles empty or with a few rows, so
    that warps without rows run ahead of those with some; each sequence has a draft with
    an infinite value, which the rows that see it get and the others do not."""
    batch = 1800
    rng = np.random.default_rng(T + len(lens))
    n = np.array([lens[b % len(lens)] for b in range(batch)], np.int32)
    t = Tree(T * 7 + len(lens), rng.integers(0, 65 - T, batch), T, hq, 1, 64, lens=n)
    bad = np.where(np.arange(batch) % 2 == 0, 0, rng.integers(0, n))
    for b in range(batch):
        p = t.ctx[b] - n[b] + bad[b]
        t.vc[t.bt[b, p // 64], p % 64, 0, 7] = 0x7F80
    want, tol = OD.decode_tree(f64(t.q), f64(t.kc), np.where(np.isfinite(f64(t.vc)), f64(t.vc), 0), t.bt, t.ctx, t.sees,
                               t.scale, t.lens)
    for b in range(batch):
        want[b, np.nonzero(t.sees[b][:n[b], bad[b]])[0], :, 7] = np.inf
    for _ in range(5):
        out = t.run()
        assert pa.get_device_error() == (0, 0)
        near(host_f64(out), want, tol)


@pytest.mark.parametrize("T,hq,hkv,tiles", [(5, 8, 2, 8), (5, 8, 2, 9), (5, 8, 2, 12), (5, 8, 2, 13), (40, 8, 2, 12),
                                            (40, 8, 2, 13), (64, 8, 1, 12), (64, 8, 1, 13), (40, 8, 2, 20),
                                            (40, 8, 2, 21)])
def test_block_tables_around_the_width_that_one_launch_serves(T, hq, hkv, tiles):
    """Every item with a CTA of its own, and more items than CTAs; one sequence of the
    table's width, others shorter."""
    rng = np.random.default_rng(tiles)
    for batch in (1, 2, 5, 80):
        before = rng.integers(0, 64 * tiles - T + 1, batch)
        before[0] = 64 * tiles - T
        t = Tree(tiles + batch, before, T, hq, hkv, 64)
        t.bt = np.ascontiguousarray(t.bt[:, :tiles])
        t.check()


def test_metadata_of_block_ids_whose_slots_do_not_fit():
    """No slot, rather than one that wraps into another sequence's rows."""
    for bad, B in ((1 << 28, 16), (1 << 27, 16), ((1 << 31) - 1, 256), ((1 << 28) + 3, 48)):
        bt = np.array([[5, 7], [4, bad]], np.int32)
        ctx = np.array([B + 2, B + 2], np.int32)
        m = pa.tree_metadata(None, dev_i32(ctx), dev_i32(bt), B, num_drafts=4)
        assert pa.get_device_error() == (pa.PA_DEV_BAD_BLOCK, 3)
        slots = m.slot_mapping.view(2, 4).tolist()
        assert slots[0] == [5 * B + B - 2, 5 * B + B - 1, 7 * B, 7 * B + 1]
        assert slots[1] == [4 * B + B - 2, 4 * B + B - 1, -1, -1]
        assert m.positions.view(2, 4)[1].tolist() == [B - 2, B - 1, B, B + 1]
    # The last slot that fits.
    last = dev_i32([[(1 << 27) - 1]])
    m = pa.tree_metadata(None, dev_i32([16]), last, 16, num_drafts=2)
    assert m.slot_mapping.tolist() == [(1 << 31) - 2, (1 << 31) - 1]
    assert pa.get_device_error() == (0, 0)


# ---------------------------------------------------------------- verification

@pytest.mark.parametrize("batch,n,vocab,dtype", [(1, 12, 151936, torch.bfloat16), (48, 12, 151936, torch.bfloat16),
                                                 (48, 9, 40000, torch.float32), (200, 64, 2000, torch.float32)])
def test_verify_lowest_index_of_equal_weights(batch, n, vocab, dtype):
    """The only child is rejected, and some 200 entries all over the row share the largest
    weight over noise: the first of them is the token, whichever thread met it."""
    for seed in range(4 if batch > 1 else 40):
        rng = np.random.default_rng(seed)
        logits = torch.from_numpy(rng.standard_normal((batch, 1, vocab)).astype(np.float32)).to(dtype).cuda()
        noise = torch.full((batch, vocab), 1e6, device="cuda")
        probs = torch.zeros(batch, 1, vocab, device="cuda")
        first = []
        for b in range(batch):
            at = rng.choice(np.arange(1, vocab), 200, replace=False)
            logits[b, 0, at], noise[b, at] = 3.0, 1.0
            first.append(int(at.min()))
        probs[:, :, 0] = 1.0
        tokens = torch.zeros(batch, n, dtype=torch.int32, device="cuda")
        r = pa.verify_drafts(logits.repeat(1, n, 1), tokens, None, torch.full((batch, n), 0.99, device="cuda"), noise,
                             torch.ones(batch, device="cuda"), draft_probs=probs.repeat(1, n, 1))
        assert r.counts.tolist() == [1] * batch and r.tokens[:, 0].tolist() == first
    assert pa.get_device_error() == (0, 0)


@pytest.mark.parametrize("batch,n,vocab,drawn", [(4, 12, 151936, True), (48, 12, 40000, True), (48, 12, 40000, False),
                                                 (1, 64, 40000, False), (8, 7, 40000, True)])
def test_verify_decisions_next_to_the_border(batch, n, vocab, drawn):
    """u q within a few units in the last place of w at every node: either way is right,
    but all CTAs of a sequence have to go the same (they would wait for each other else)."""
    rng = np.random.default_rng(batch + n)
    logits = torch.from_numpy(rng.standard_normal((batch, n, vocab)).astype(np.float32)).cuda()
    p = torch.softmax(logits.double(), -1)
    tokens = torch.from_numpy(rng.integers(0, vocab, (batch, n)).astype(np.int32)).cuda()
    at = tokens[:, 1:].long().unsqueeze(-1)
    px = p[:, :-1].gather(2, at)[..., 0]           # of each node's child, in a chain
    nudge = torch.from_numpy(1 + rng.integers(-4, 5, (batch, n - 1)) * 2.0 ** -24).cuda()
    u, probs = torch.zeros(batch, n, device="cuda"), None
    if drawn:
        u[:, 1:] = 0.5
        probs = torch.zeros(batch, n - 1, vocab, device="cuda").scatter_(2, at, (2 * px * nudge).float().unsqueeze(-1))
    else:
        u[:, 1:] = (px * nudge).float()
    for seed in range(5):
        noise = torch.from_numpy(rng.exponential(size=(batch, vocab)).astype(np.float32)).cuda()
        r = pa.verify_drafts(logits, tokens, None, u, noise, torch.ones(batch, device="cuda"), draft_probs=probs)
        assert pa.get_device_error() == (0, 0)
        for b in range(batch):
            c = int(r.counts[b])
            assert 1 <= c <= n and r.nodes[b].tolist() == list(range(c)) + [-1] * (n - c)
            assert r.tokens[b, :c - 1].tolist() == tokens[b, 1:c].tolist() and 0 <= int(r.tokens[b, c - 1]) < vocab


@pytest.mark.parametrize("vocab,n,dtype", [(500, 5, torch.float32), (20011, 5, torch.float32), (5003, 40, torch.float32),
                                           (151936, 9, torch.float32), (1203, 7, torch.bfloat16)])
def test_verify_candidates_behind_one_that_held_nearly_everything(vocab, n, dtype):
    """The first candidate, rejected, has probability 1 - 2^-8 .. 1 - 2^-20; the others'
    decisions are about what is left, of which u w are 4 % from the border.

    What is left is a sum of its own, not the difference from 1: the kernel's probabilities
    are off by under 2^-17, and 2^-14 is asked of a margin elsewhere."""
    batch = 40
    rng = np.random.default_rng(vocab + n)
    logits = rng.standard_normal((batch, n, vocab)) * 2
    tokens = np.stack([rng.permutation(vocab)[:n] for _ in range(batch)]).astype(np.int32)
    parents = np.zeros((batch, n), np.int32)
    parents[:, 0] = -1
    u = np.full((batch, n), 1 - 2.0 ** -24, np.float32)
    for b in range(batch):
        left = 2.0 ** -rng.uniform(8, 20)
        logits[b, 0, tokens[b, 2:]] = 6 + rng.standard_normal(n - 2)
        others = np.delete(np.arange(vocab), tokens[b, 1])
        logits[b, 0, tokens[b, 1]] = np.log(np.exp(logits[b, 0, others]).sum() * (1 - left) / left)
    lg = place(logits.astype(np.float32), dtype)
    z = lg[:, 0].double().cpu().numpy()
    for b in range(batch):
        w = np.exp(z[b] - z[b].max())
        for c in range(2, n):
            w[tokens[b, c - 1]] = 0
            ratio = w[tokens[b, c]] / w.sum()
            if c == n - 1 or rng.random() < 0.5 / n:
                u[b, c] = ratio * 0.96              # kept
                break
            u[b, c] = min(ratio * 1.04, 1 - 2.0 ** -24)
    noise = rng.exponential(size=(batch, vocab)).astype(np.float32)
    # The oracle without that candidate: the same residual, and margins of the others alone.
    z = lg.double().cpu().numpy()
    z[np.arange(batch), 0, tokens[:, 1]] = -np.inf
    want = OD.verify(z, tokens, parents, u, noise, np.ones(batch))
    r = pa.verify_drafts(lg, torch.from_numpy(tokens).cuda(), torch.from_numpy(parents).cuda(),
                         torch.from_numpy(u).cuda(), place(noise, torch.float32), torch.ones(batch, device="cuda"))
    assert pa.get_device_error() == (0, 0)
    sure = want[3] > 2.0 ** -14
    assert sure.mean() > 0.9 and np.all(want[2] <= 2) and want[2].sum() > batch
    for got, w in zip(r, want):
        assert np.array_equal(got.cpu().numpy()[sure], w[sure])


@pytest.mark.parametrize("batch,n,vocab,dtype", [(30, 8, 32000, torch.bfloat16), (70, 8, 32000, torch.bfloat16),
                                                 (130, 7, 32000, torch.float32), (310, 6, 40000, torch.bfloat16)])
def test_verify_drawn_chains_of_few_and_many_sequences(batch, n, vocab, dtype):
    """Chains whose rows are read at once while each sequence has several CTAs, and one
    after the other above that; drafts that are mostly kept, and mostly rejected."""
    for close in (0.1, 3.0):
        check_verify(verify_case(batch + n, batch, n, vocab, dtype, True, chain=True, close=close))


def test_verify_padded_rows_may_hold_anything():
    """No error of a row that takes part in nothing, whatever its buffers hold."""
    for drawn, T, vocab in ((True, 6, 5003), (False, 12, 50000)):
        lens = np.array([T, 0, 3, 0, 0, 0], np.int32)
        s = verify_case(T, 6, T, vocab, torch.float32, drawn, lens=lens)
        check_verify(s)
        want = run_verify(s)
        pad = lens == 0
        s["temps"][pad] = [0.0, float("nan"), -1.0, float("inf")]
        s["tokens"][pad], s["parents"][pad] = 1 << 30, 77
        s["u"][pad] = s["noise"][pad] = np.nan
        s["logits"][torch.from_numpy(pad).cuda()] = float("nan")
        r = run_verify(s)
        assert pa.get_device_error() == (0, 0)
        assert all(torch.equal(x, y) for x, y in zip(r, want))
        assert r.counts[torch.from_numpy(pad).cuda()].tolist() == [0] * 4


NO_WIDE_CLUSTERS = """
#include <cuda_runtime.h>
template <typename K>
cudaError_t fake_max_clusters(int *n, K *, const cudaLaunchConfig_t *cfg) {
    *n = 1;
    for (unsigned i = 0; i < cfg->numAttrs; ++i)
        if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension && cfg->attrs[i].val.clusterDim.x > 8) *n = 0;
    return cudaSuccess;
}
template <typename... E, typename... A>
cudaError_t fake_launch(const cudaLaunchConfig_t *cfg, void (*kernel)(E...), A &&...args) {
    int n = 0;
    fake_max_clusters(&n, kernel, cfg);
    return n ? cudaLaunchKernelEx(cfg, kernel, static_cast<A &&>(args)...) : cudaErrorInvalidClusterSize;
}
#define cudaOccupancyMaxActiveClusters fake_max_clusters
#define cudaLaunchKernelEx fake_launch
"""


def test_verify_on_a_device_without_clusters_of_16(tmp_path):
    """The calls that ask for such clusters are faked, to say that the device has none: up to
    four sequences of a large vocabulary are then served by clusters of eight."""
    pabuild.build()
    fake, obj, lib = tmp_path / "fake.h", tmp_path / "pa_draft.o", tmp_path / "libpa_fake.so"
    fake.write_text(NO_WIDE_CLUSTERS)
    nvcc = [pabuild.nvcc()] + pabuild.ARCH
    subprocess.run(nvcc + pabuild.NVCC_FLAGS + ["-include", str(fake), "-c", os.path.join(pabuild.CSRC, "pa_draft.cu"),
                                                "-o", str(obj)], check=True, capture_output=True)
    others = [o for o in glob.glob(os.path.join(pabuild.BUILD, "*.o")) if os.path.basename(o) != "pa_draft.o"]
    subprocess.run(nvcc + ["-shared", "-o", str(lib), str(obj)] + others, check=True, capture_output=True)
    call = C.CDLL(str(lib)).pa_verify_drafts
    call.restype, call.argtypes = pa.SIGNATURES["pa_verify_drafts"]
    for batch, n, drawn in ((1, 6, True), (4, 20, False), (3, 12, True)):
        s = verify_case(batch * n, batch, n, 50000, torch.bfloat16, drawn, close=0.2)
        want = check_verify(s)
        lg, noise = s["logits"], place(s["noise"], torch.float32)
        tok, par = dev_i32(s["tokens"]), dev_i32(s["parents"])
        u, temps = torch.from_numpy(s["u"]).cuda(), torch.from_numpy(s["temps"]).cuda()
        q = place(s["probs"], torch.float32) if drawn else None
        out = [torch.empty_like(tok), torch.empty_like(tok), torch.empty(batch, dtype=torch.int32, device="cuda")]
        for _ in range(2):  # asked, and known
            rc = call(*(x.data_ptr() for x in out), lg.data_ptr(), lg.stride(1), 0, tok.data_ptr(), par.data_ptr(),
                      u.data_ptr(), noise.data_ptr(), noise.stride(0), temps.data_ptr(), q.data_ptr() if drawn else None,
                      q.stride(1) if drawn else 0, n if drawn else 0, None, batch, n, 50000,
                      torch.cuda.current_stream().cuda_stream)
            assert rc == pa.PA_OK
            r = pa.verify_drafts(lg, tok, par, u, noise, temps, draft_probs=q)
            assert all(torch.equal(x, y) for x, y in zip(out, r)) and out[2].tolist() == want.tolist()
