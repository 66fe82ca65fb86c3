"""GPU tests of pa_logprobs at its edges: ties in the ragged end of a row,
infinite temperatures, sizes beyond 32 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from gpu_util import dev_i32
from test_gpu_logprobs import check, normal, place

pytestmark = pytest.mark.gpu


def device_us(call, reps=20):
    """The fastest of `reps` calls, by events."""
    best = float("inf")
    for _ in range(reps + 2):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 151943), (3, 40007), (700, 9007)])
def test_ties_in_the_ragged_end(rows, vocab, dtype):
    """The last vocab % 8 logits are a row's largest and equal."""
    x = normal(vocab, min(rows, 3), vocab)
    x[:, -7:] = 50.0
    x = np.resize(x, (rows, vocab))
    for top in (1, 2, 3, 5, 7, 8, 32):
        check(x, [vocab - 1] * rows, top, dtype=dtype)


def test_ties_in_the_ragged_end_take_no_longer():
    """Equal logits in the ragged end are selected in one collection, as distinct
    ones are (passes over the row, one per alternative, take several times as
    long as the whole call)."""
    rows, vocab = 640, 151943
    x = torch.from_numpy(normal(1, 1, vocab)).cuda().expand(rows, -1)
    tied = torch.empty(rows, vocab + 1, device="cuda")[:, :vocab]
    apart = torch.empty(rows, vocab + 1, device="cuda")[:, :vocab]
    for t in (tied, apart):
        t.copy_(x)
        t[:, -7:] = 50.0
    apart[:, -7:] += torch.arange(7, device="cuda")
    tok = dev_i32(np.zeros(rows, np.int32))
    for top in (2, 5, 6):
        out = pa.logprobs(tied, tok, top)
        want = torch.arange(vocab - 7, vocab - 7 + top, dtype=torch.int32, device="cuda")
        assert (out.top_ids == want).all()
        t = device_us(lambda: pa.logprobs(tied, tok, top, out=out))
        assert t <= 2 * device_us(lambda: pa.logprobs(apart, tok, top, out=out)), (top, t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [3, 8, 1001, 40000, 40007])
def test_infinite_and_huge_temperatures(vocab, dtype):
    """T = inf: uniform over what is not -inf, in whole and in ragged rows."""
    x = normal(vocab, 5, vocab)
    x[1, 1:] = -np.inf
    x[2, ::2] = -np.inf
    x[3, ::2] = float(torch.finfo(torch.bfloat16).min)
    x[4, 0] = -np.inf
    for t in (np.inf, 3e38, 1e20):
        check(x, [0, 1, 2, 0, vocab - 1], min(5, vocab), np.full(5, t, np.float32), dtype=dtype)


def test_sizes_beyond_32_bits_are_refused():
    tok = dev_i32([0])
    lg = torch.zeros(1, (1 << 32) + 8, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: pa.logprobs(lg, tok), lambda: pa.logprobs(lg[:, :64], tok, 1 << 32),
                 lambda: pa.logprobs(lg[:, :64], tok, -(1 << 32))):
        with pytest.raises((ValueError, pa.PagedAttentionError)):
            call()
    many = torch.zeros((1 << 32) + 1, dtype=torch.int32, device="cuda")
    wide = lg.view(-1)[:8].expand((1 << 32) + 1, 8)
    with pytest.raises(ValueError):
        pa.logprobs(wide, many)
