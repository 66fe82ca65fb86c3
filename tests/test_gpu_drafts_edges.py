"""Speculative decoding where it can go wrong: calls that the documentation allows
and that the tests of each entry point's ordinary range do not reach."""
import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import drafts as OD
from gpu_util import host_f64
from test_gpu_drafts import Tree, f64, near

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
