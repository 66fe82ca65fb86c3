"""GPU parity of pa_logprobs with its float64 definition (oracle/logprobs.py),
through the C ABI; the ids and their order exactly, the rest within the bound
that the oracle derives for an fp32 evaluation of each row."""
import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle.logprobs import logprobs as define
from paged_kv_cache_store_gb300.workloads import QWEN3_VOCAB, make_sampler, bf16_bits_to_f32
from gpu_util import dev_i32

pytestmark = pytest.mark.gpu
F32 = np.float32


def place(x, dtype, pad=0):
    """x [rows, vocab] on the GPU, rows `pad` further logits apart (and 16-byte aligned)."""
    rows, vocab = x.shape
    t = torch.full((rows, -(-vocab // 8) * 8 + pad), float("nan"), dtype=dtype, device="cuda")[:, :vocab]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)).cuda())
    return t


def compare(r, x, tokens, top, temps=None):
    """Results r for rows of logits x (float64)."""
    want = define(x, tokens, top, temps)
    for got, name, tol in ((r.logprobs, "logprobs", "tol_logprobs"), (r.entropy, "entropy", "tol_entropy"),
                           (r.top_logprobs, "top_logprobs", "tol_top")):
        if got is None:
            assert top == 0
            continue
        g, w = got.double().cpu().numpy(), want[name]
        fin = np.isfinite(w)
        assert np.array_equal(g[~fin], w[~fin], equal_nan=True), (name, g[~fin], w[~fin])
        off = np.abs(g[fin] - w[fin]) - want[tol][fin]
        assert not np.any(off > 0), (name, float(off.max()))
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), want["top_ids"])


def check(x, tokens, top, temps=None, dtype=torch.bfloat16, pad=0):
    lg = place(x, dtype, pad)
    r = pa.logprobs(lg, dev_i32(tokens), top, None if temps is None else torch.from_numpy(temps).cuda())
    assert pa.get_device_error() == (0, 0)
    compare(r, lg.double().cpu().numpy(), tokens, top, temps)


def normal(seed, rows, vocab, std=2.0):
    return (np.random.default_rng(seed).standard_normal((rows, vocab)) * std).astype(F32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [0, 1, 5, 8, 9, 16, 17, 20, 32])
def test_top_sizes(top, dtype):
    rng = np.random.default_rng(top)
    check(normal(top, 3, 32003), rng.integers(0, 32003, 3), top, dtype=dtype, pad=16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 32, 33, 255, 256, 257, 1000, 2047, 2049, 4095, 4097, 16391, 50257])
def test_vocabulary_sizes(vocab, dtype):
    rng = np.random.default_rng(vocab)
    check(normal(vocab, 4, vocab), rng.integers(0, vocab, 4), min(vocab, 20), dtype=dtype,
          temps=rng.uniform(0.3, 2.0, 4).astype(F32))


@pytest.mark.parametrize("vocab", [20011, 3001])
@pytest.mark.parametrize("rows", [1, 2, 40, 75, 151, 320, 700])
def test_row_counts(rows, vocab):
    """Every cluster size and both CTA sizes, and more rows than CTAs that run at once."""
    rng = np.random.default_rng(rows)
    for dtype in (torch.bfloat16, torch.float32):
        check(normal(rows, rows, vocab), rng.integers(0, vocab, rows), 20, dtype=dtype)


def test_qwen3_vocabulary_at_the_sampling_temperatures():
    s = make_sampler("logprobs", 77, 16, QWEN3_VOCAB)
    rng = np.random.default_rng(0)
    check(bf16_bits_to_f32(s.logits), rng.integers(0, QWEN3_VOCAB, 16), 20, s.temperatures)


def test_peaked_and_flat_rows():
    x = normal(5, 6, 5000, 0.01)
    x[0, 4321] = 60.0          # one entry holds the row: a log probability near 0
    x[1] = 0.0                 # uniform: all tied, ids 0, 1, 2, ...
    x[2] = 1e30                # uniform and large
    x[3, ::2] = 20.0
    x[4] *= 1e4                # wide
    x[5] -= 500.0
    check(x, [4321, 17, 4999, 1, 0, 3], 32, dtype=torch.float32)
    check(x, [0, 0, 0, 0, 0, 0], 32)


def test_ties_take_the_lowest_indices():
    rng = np.random.default_rng(8)
    for vocab in (600, 9000, 70001):
        check(rng.integers(-2, 3, (4, vocab)).astype(F32), rng.integers(0, vocab, 4), 32)
    x = np.zeros((2, 3000), F32)
    x[0, 1::2] = -0.0          # equal to +0
    check(x, [1, 2], 16, dtype=torch.float32)


def test_masked_rows():
    """-inf and the type's lowest value where a grammar or padding masks; rows
    where the mask leaves a few entries, one, or nothing."""
    vocab = 40000
    low = float(torch.finfo(torch.bfloat16).min)
    for mask in (-np.inf, low):
        x = np.full((5, vocab), mask, F32)
        x[0, [5, 39999, 777]] = [1.0, 1.0, 2.0]
        x[1, 12345] = -3.0
        x[3, 20000:] = normal(1, 1, 20000)[0]
        x[4, :100] = normal(2, 1, 100)[0]
        for top in (5, 32):
            check(x, [5, 12345, 9, 100, 100], top)
            check(x, [777, 0, 0, 30000, 3], top, dtype=torch.float32,
                  temps=np.array([0.5, 1.0, 0.01, 2.0, 1e-6], F32))


def test_nan_and_infinite_logits():
    x = normal(3, 6, 9001)
    x[0, 77] = np.nan
    x[1, [3, 9000]] = np.inf
    x[2] = np.nan
    x[3] = np.nan
    x[3, [1, 8000]] = [2.0, 5.0]          # fewer entries than alternatives
    x[4, :] = np.nan
    x[4, ::3] = -np.inf
    for dtype in (torch.float32, torch.bfloat16):
        for top in (0, 5, 32):
            check(x, [77, 1, 2, 3, 4, 5], top, dtype=dtype)


def test_large_entries_packed_together():
    """Orders and layouts in which one thread, warp or CTA owns every large entry."""
    for vocab in (60000, 30000):
        up = np.linspace(-30, 30, vocab, dtype=F32)
        block = up.copy()
        block[1000:1400] = 50 + np.arange(400, dtype=F32)
        x = [up, up[::-1], block]
        for step in (1024, 2048):  # a vector for each of 128 or 256 threads
            stride, every = up.copy(), normal(1, 1, vocab)[0]
            stride[0::step] = 100 + np.arange(len(stride[0::step]), dtype=F32)   # one thread's first logits
            for k in range(8):  # one thread's every logit
                every[k::step] = 40 + 0.01 * np.arange(len(every[k::step]), dtype=F32)
            x += [stride, every]
        x = np.stack(x)
        for rows in (x, np.repeat(x, 90, axis=0)):
            for top in (5, 32):
                check(rows, np.arange(len(rows)) % vocab, top, dtype=torch.float32)


def test_overflowing_collection():
    """More entries at the threshold than the kernel collects."""
    vocab = 400000
    x = np.full((700, vocab), -5.0, F32)
    own = np.concatenate([np.arange(8 * t + j, vocab, 2048) for t in range(31) for j in range(8)])
    x[:, own] = 1.0 + np.random.default_rng(0).random(len(own), dtype=F32)
    # 31 lanes of a warp hold only large logits, the threshold comes from the 32nd: all of them pass.
    t = torch.from_numpy(x[:1]).cuda().expand(700, -1).contiguous()
    r = pa.logprobs(t, dev_i32(np.zeros(700, np.int32)), 32)
    want = define(x[:1].astype(np.float64), [0], 32)
    assert (r.top_ids.cpu().numpy() == want["top_ids"]).all()
    assert np.abs(r.entropy.double().cpu().numpy() - want["entropy"]).max() <= want["tol_entropy"][0]


def test_tokens_outside_and_bad_temperatures():
    x = normal(4, 5, 3001)
    lg = place(x, torch.float32)
    temps = torch.tensor([1.0, 1.0, 1.0, 0.0, float("nan")], device="cuda")
    pa.get_device_error()
    r = pa.logprobs(lg, dev_i32([-1, 3001, 2, 3, 4]), 5)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TOKEN, 1)
    assert torch.isneginf(r.logprobs[:2]).all() and torch.isfinite(r.logprobs[2:]).all()
    r = pa.logprobs(lg[3:4], dev_i32([3]), 5, temps[3:4])
    assert pa.get_device_error() == (pa.PA_DEV_BAD_TEMPERATURE, 0)
    assert torch.isnan(r.logprobs).all() and torch.isnan(r.top_logprobs).all() and (r.top_ids == -1).all()
    r = pa.logprobs(lg, dev_i32([0, 1, 2, 3, 4]), 5, temps)
    assert pa.get_device_error()[0] == pa.PA_DEV_BAD_TEMPERATURE
    assert torch.isfinite(r.entropy[:3]).all() and torch.isnan(r.entropy[3:]).all() and (r.top_ids[3:] == -1).all()


def test_after_the_sampler_in_a_captured_step():
    """Sampler, then the log probabilities of what it picked, captured and
    replayed; the same outputs as eager calls, on another stream too."""
    s = make_sampler("graph", 6, 4, 9001)
    logits = torch.zeros(4, 9008, dtype=torch.bfloat16, device="cuda")[:, :9001]
    noise = torch.ones(4, 9008, device="cuda")[:, :9001]
    logits.copy_(torch.from_numpy(bf16_bits_to_f32(s.logits)))
    noise.copy_(torch.from_numpy(s.exp_noise))
    temps, tok = torch.from_numpy(s.temperatures).cuda(), torch.zeros(4, dtype=torch.int32, device="cuda")

    def step(out=None):
        pa.sample_gumbel(logits, temps, noise, out=tok)
        return pa.logprobs(logits, tok, 7, temps, out=out)

    out = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out)
    for i in range(3):
        logits.copy_(torch.from_numpy(normal(i, 4, 9001)).cuda())
        g.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pa.logprobs(logits, tok, 7, temps, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, other))
    assert pa.get_device_error() == (0, 0)


def test_offsets_beyond_32_bits():
    """The last rows of more than 2^31 logits."""
    rows, vocab = 16000, 151936
    big = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    big[-2:].copy_(torch.from_numpy(normal(2, 2, vocab)).cuda())
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    r = pa.logprobs(big, tok, 3)
    compare(pa.Logprobs(*(t[-2:] for t in r)), big[-2:].double().cpu().numpy(), [0, 0], 3)


def test_refusals_of_the_binding():
    lg, tok = torch.zeros(2, 64, device="cuda"), dev_i32([0, 1])
    for call, err in ((lambda: pa.logprobs(lg.half(), tok), TypeError),
                      (lambda: pa.logprobs(lg, tok.long()), TypeError),
                      (lambda: pa.logprobs(lg, tok[:1]), ValueError),
                      (lambda: pa.logprobs(lg.t(), dev_i32([0] * 64)), ValueError),
                      (lambda: pa.logprobs(lg, tok, temperatures=torch.ones(3, device="cuda")), ValueError),
                      (lambda: pa.logprobs(lg, tok, 65), pa.PagedAttentionError),
                      (lambda: pa.logprobs(lg, tok, 33), pa.PagedAttentionError),
                      (lambda: pa.logprobs(lg, tok, -1), pa.PagedAttentionError),
                      (lambda: pa.logprobs(torch.zeros(2, 65, device="cuda"), tok), pa.PagedAttentionError),
                      (lambda: pa.logprobs(lg, tok, 2, out=pa.logprobs(lg, tok, 3)), ValueError)):
        with pytest.raises(err):
            call()
