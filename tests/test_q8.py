"""The 8-bit pool without a GPU: its float64 definition against worked values,
closed forms and torch's own conversion, and the argument checks of the entry
points (no call here launches a kernel)."""
import ctypes as C

import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import q8
from paged_kv_cache_store_gb300 import build as pabuild
from paged_kv_cache_store_gb300.workloads import bf16_bits_to_f32, normal_bf16


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.load_library()


def test_e4m3_values():
    v = q8.e4m3_values()
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and np.isnan(v[0x7F])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(v, nan=1e9), np.nan_to_num(t, nan=1e9))


def test_worked_rows():
    x = np.zeros((4, 128))
    x[0, :3] = [448.0, -1.0, 0.1]       # the largest code at scale 1
    x[1, :3] = [449.0, 18.0, 19.0]      # just above: scale 2; 9 and 9.5 (a tie, to even)
    x[2, :3] = [127.0, 0.5, 1.5]        # int8: 0.5 -> 0, 1.5 -> 2
    c, s = q8.quantise(x, "e4m3")
    assert s.tolist() == [127, 128, 126, 1]  # 127 <= 448 * 2^-1; a row of zeros has 2^-126
    got = q8.values(c, s, "e4m3")
    assert got[0, :3].tolist() == [448.0, -1.0, 0.1015625]
    assert got[1, :3].tolist() == [448.0, 18.0, 20.0]
    c, s = q8.quantise(x, "int8")
    assert s.tolist() == [129, 129, 127, 1]
    assert q8.values(c, s, "int8")[2, :3].tolist() == [127.0, 0.0, 2.0]
    x[3, 9] = np.nan
    c, s = q8.quantise(x, "int8")
    assert s[3] == 255 and not c[3].any() and np.isnan(q8.values(c, s, "int8")[3]).all()


@pytest.mark.parametrize("fmt,rel", [("e4m3", 2.0 ** -4), ("int8", 0.0)])
def test_definition_against_torch_and_its_bounds(fmt, rel):
    """The scale is the smallest power of two that fits; the codes are torch's
    conversion of the scaled values; the error bounds that pa.h gives hold."""
    x = bf16_bits_to_f32(normal_bf16(3, 1, (500, 128))).astype(np.float64)
    x *= np.exp2(np.random.default_rng(0).integers(-100, 100, (500, 1)))
    c, s = q8.quantise(x, fmt)
    a = np.abs(x).max(-1)
    scale = np.exp2(s.astype(np.float64) - 127)
    assert np.all(a <= q8.LIMIT[fmt] * scale) and np.all(a > q8.LIMIT[fmt] * scale / 2)
    y = torch.from_numpy(x / scale[:, None])
    t = y.float().to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else y.round().to(torch.int8).view(torch.uint8)
    assert np.array_equal(t.numpy(), c)
    err = np.abs(q8.values(c, s, fmt) - x)
    if fmt == "e4m3":
        big = np.abs(x) > 2.0 ** -15 * a[:, None]
        assert np.all(err[big] <= rel * np.abs(x)[big]) and np.all(err <= 2.0 ** -10 * scale[:, None] + rel * np.abs(x))
    else:
        assert np.all(err <= a[:, None] / 126)


def test_decode_definition_is_softmax_attention():
    rng = np.random.default_rng(1)
    kc, vc = (rng.integers(0, 0x70, (3, 2, 16, 128), dtype=np.uint8) for _ in range(2))
    ks, vs = (rng.integers(118, 123, (3, 2, 16), dtype=np.uint8) for _ in range(2))
    q = rng.standard_normal((2, 4, 128))
    out, tol = q8.decode(q, kc, ks, vc, vs, "e4m3", [[2, 0], [1, -1]], [20, 0], 0.05)
    K = torch.from_numpy(q8.values(kc, ks, "e4m3")[[2, 0]]).transpose(1, 2).reshape(32, 2, 128)[:20]
    V = torch.from_numpy(q8.values(vc, vs, "e4m3")[[2, 0]]).transpose(1, 2).reshape(32, 2, 128)[:20]
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[0])[:, None], K.transpose(0, 1).repeat_interleave(2, 0),
        V.transpose(0, 1).repeat_interleave(2, 0), scale=0.05)[:, 0]
    assert np.abs(out[0] - want.numpy()).max() < 1e-10 and not out[1].any()
    assert np.all(tol[0] > 0)


P = C.c_void_p(256)


def _rows(fn, **kw):
    a = dict(k=P, ks=1024, v=P, vs=1024, kc=P, vc=P, sk=P, sv=P, slots=P, n=4, hkv=8, d=128, B=256, nb=64, fmt=0,
             stream=None)
    a.update(kw)
    return fn(*a.values())


@pytest.mark.parametrize("name", ["pa_store_kvcache_q8", "pa_load_kvcache_q8"])
def test_rows_argument_checks(L, name):
    fn = getattr(L, name)
    assert _rows(fn, n=0) == pa.PA_OK
    assert _rows(fn, n=-1) == pa.PA_ERR_INVALID_ARG
    for null in ("k", "v", "kc", "vc", "sk", "sv", "slots"):
        assert _rows(fn, **{null: None}) == pa.PA_ERR_INVALID_ARG
    for unaligned in ("k", "v", "kc", "vc", "sk", "sv"):
        assert _rows(fn, **{unaligned: C.c_void_p(264)}) == pa.PA_ERR_INVALID_ARG
    assert _rows(fn, ks=1016) == pa.PA_ERR_INVALID_ARG         # shorter than a row
    assert _rows(fn, vs=1028) == pa.PA_ERR_INVALID_ARG         # not a multiple of 8
    assert _rows(fn, d=64) == pa.PA_ERR_UNSUPPORTED
    assert _rows(fn, B=24) == pa.PA_ERR_UNSUPPORTED
    assert _rows(fn, hkv=0) == pa.PA_ERR_INVALID_ARG
    assert _rows(fn, nb=0) == pa.PA_ERR_INVALID_ARG
    assert _rows(fn, fmt=2) == pa.PA_ERR_INVALID_ARG
    assert _rows(fn, nb=1 << 20) == pa.PA_ERR_UNSUPPORTED      # 2^31 rows: one too many for int32
    assert b"row indices" in L.pa_last_error_message()


def _decode(L, **kw):
    a = dict(out=P, q=P, qs=2048, kc=P, vc=P, sk=P, sv=P, bt=P, mb=16, ctx=P, batch=4, hq=16, hkv=8, d=128, B=256,
             nb=64, fmt=1, scale=0.088, ws=P, wsb=1 << 30, stream=None)
    a.update(kw)
    return L.pa_decode_q8(*a.values())


def test_decode_argument_checks(L):
    assert _decode(L, batch=0) == pa.PA_OK
    assert _decode(L, batch=-1) == pa.PA_ERR_INVALID_ARG
    for null in ("out", "q", "kc", "vc", "sk", "sv", "bt", "ctx"):
        assert _decode(L, **{null: None}) == pa.PA_ERR_INVALID_ARG
    for unaligned in ("out", "q", "kc", "vc", "sk", "sv", "ws"):
        assert _decode(L, **{unaligned: C.c_void_p(264)}) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, hq=12) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, hq=24) == pa.PA_ERR_UNSUPPORTED          # a group of 3
    assert _decode(L, d=64) == pa.PA_ERR_UNSUPPORTED
    assert _decode(L, B=24) == pa.PA_ERR_UNSUPPORTED
    assert _decode(L, mb=0) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, mb=1 << 23) == pa.PA_ERR_UNSUPPORTED     # positions overflow int32
    assert _decode(L, batch=2048, mb=1 << 20, B=1024) == pa.PA_ERR_UNSUPPORTED  # tile prefix overflows
    assert _decode(L, fmt=-1) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, qs=2040) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, qs=2052) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, scale=0.0) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, scale=float("inf")) == pa.PA_ERR_INVALID_ARG
    assert _decode(L, batch=2049) == pa.PA_ERR_UNSUPPORTED
    n = L.pa_decode_q8_workspace_size(16, 8, 128)
    assert _decode(L, wsb=n - 1) == pa.PA_ERR_WORKSPACE
    assert _decode(L, ws=None) == pa.PA_ERR_WORKSPACE
    assert L.pa_decode_q8_workspace_size(24, 8, 128) == 0 and L.pa_decode_q8_workspace_size(16, 8, 64) == 0
    assert L.pa_decode_q8_workspace_size(64, 8, 128) <= 32 << 20


def test_decode_store_argument_checks(L):
    def call(**kw):
        a = dict(out=P, q=P, qs=2048, nk=P, nks=1024, nv=P, nvs=1024, kc=P, vc=P, sk=P, sv=P, bt=P, mb=16, ctx=P,
                 batch=4, hq=16, hkv=8, d=128, B=256, nb=64, fmt=1, scale=0.088, ws=P, wsb=1 << 30, stream=None)
        a.update(kw)
        return L.pa_decode_store_q8(*a.values())

    assert call(batch=0) == pa.PA_OK
    assert call(nk=None) == pa.PA_ERR_INVALID_ARG
    assert call(nv=None) == pa.PA_ERR_INVALID_ARG
    assert call(nk=C.c_void_p(264)) == pa.PA_ERR_INVALID_ARG
    assert call(nks=1016) == pa.PA_ERR_INVALID_ARG
    assert call(nvs=1028) == pa.PA_ERR_INVALID_ARG
    assert call(hq=24) == pa.PA_ERR_UNSUPPORTED                # pa_decode_q8's own checks follow
    assert call(ws=None) == pa.PA_ERR_WORKSPACE


def test_binding_refuses_host_tensors():
    pool = [torch.zeros(2, 2, 16, 128, dtype=torch.int8) for _ in range(2)] + \
           [torch.zeros(2, 2, 16, dtype=torch.uint8) for _ in range(2)]
    with pytest.raises(TypeError):
        pa.load_kvcache_q8(*pool, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        pa.store_kvcache_q8(*(torch.zeros(1, 2, 128, dtype=torch.bfloat16) for _ in range(2)), *pool,
                            torch.zeros(1, dtype=torch.int32))
