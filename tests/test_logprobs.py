"""pa_logprobs without a GPU: its float64 definition against closed forms and
torch, and the entry point's argument checks (no call here launches a kernel)."""
import ctypes as C

import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle.logprobs import logprobs as define
from paged_kv_cache_store_gb300 import build as pabuild


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.load_library()


def test_closed_forms():
    x = np.log(np.array([[1.0, 2.0, 3.0, 2.0]]))
    r = define(x, [1], 4)
    assert np.allclose(r["logprobs"], np.log(0.25)) and r["top_ids"].tolist() == [[2, 1, 3, 0]]
    p = np.array([1, 2, 3, 2]) / 8
    assert np.allclose(r["entropy"], -(p * np.log(p)).sum())
    r = define(np.zeros((1, 1000)), [-1], 3)
    assert np.allclose(r["entropy"], np.log(1000)) and r["logprobs"][0] == -np.inf
    assert r["top_ids"].tolist() == [[0, 1, 2]]
    r = define(np.array([[-np.inf, 0.0, np.nan], [-np.inf] * 3, [1.0, -np.inf, -np.inf]]), [1, 1, 0], 3)
    assert np.isnan(r["entropy"][0]) and r["top_ids"].tolist() == [[1, 0, 2], [0, 1, 2], [0, 1, 2]]
    assert r["entropy"][1] == 0 and r["logprobs"][1] == -np.inf and r["logprobs"][2] == 0 and r["entropy"][2] == 0


def test_against_torch():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 777, generator=g, dtype=torch.float64) * 3
    t = torch.rand(5, generator=g, dtype=torch.float64) + 0.3
    r = define(x.numpy(), [0, 5, 776, 9, 1], 9, t.numpy())
    d = torch.distributions.Categorical(logits=x / t[:, None])
    assert np.allclose(r["logprobs"], d.log_prob(torch.tensor([0, 5, 776, 9, 1])).numpy())
    assert np.allclose(r["entropy"], d.entropy().numpy())
    assert np.array_equal(r["top_ids"], x.topk(9).indices.numpy())


def test_argument_checks(L):
    p = C.c_void_p(256)

    def call(**kw):
        a = dict(lp=p, h=p, ids=p, tl=p, lg=p, ls=1024, fp32=0, t=None, tok=p, rows=4, vocab=1000, k=5, stream=None)
        a.update(kw)
        return L.pa_logprobs(*a.values())

    assert call(rows=0) == pa.PA_OK
    assert call(rows=-1) == pa.PA_ERR_INVALID_ARG
    assert call(vocab=0) == pa.PA_ERR_INVALID_ARG
    for null in ("lp", "h", "ids", "tl", "lg", "tok"):
        assert call(**{null: None}) == pa.PA_ERR_INVALID_ARG
    assert call(k=-1) == pa.PA_ERR_INVALID_ARG
    assert call(k=33) == pa.PA_ERR_UNSUPPORTED
    assert call(vocab=4, k=5) == pa.PA_ERR_INVALID_ARG
    assert call(vocab=(1 << 30) + 8, ls=1 << 31) == pa.PA_ERR_UNSUPPORTED
    assert call(fp32=2) == pa.PA_ERR_INVALID_ARG
    assert call(ls=999) == pa.PA_ERR_INVALID_ARG
    assert call(ls=1004) == pa.PA_ERR_INVALID_ARG          # bf16 rows stay 16-byte aligned
    assert call(ls=1002, fp32=1) == pa.PA_ERR_INVALID_ARG
    assert call(lg=C.c_void_p(264)) == pa.PA_ERR_INVALID_ARG
