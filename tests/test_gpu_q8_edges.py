"""GPU tests of the 8-bit pool at its edges: workspaces that serve several
shapes, rows at both ends of bf16's range, scores whose factors leave fp32's
range, sizes beyond 32 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_store_gb300 as pa
from oracle import q8
from paged_kv_cache_store_gb300.workloads import f32_to_bf16_bits, make_decode, normal_bf16
from gpu_util import dev_bf16, dev_i32, host_f64
from test_gpu_q8 import FMTS, check_decode, check_store, dev_pool, f64, make_pool, rows, same_bytes

pytestmark = pytest.mark.gpu


def bits(x):
    with np.errstate(over="ignore"):
        return f32_to_bf16_bits(np.asarray(x).astype(np.float32))


@pytest.mark.parametrize("fused", [False, True])
def test_one_workspace_serves_every_gqa_group(fused):
    """A workspace sized for the largest group, used by calls of every group in
    turn: what one call leaves in it is nothing to the next."""
    ws = pa.decode_q8_workspace(64, 8)
    for hq, ctx in [(64, [4000, 77, 1300]), (16, [5000, 5000]), (8, [3000, 1, 900, 6000]), (32, [7000, 255]),
                    (64, [2500, 9]), (16, [1, 4000, 17])]:
        inp = make_decode(f"ws {hq}", 20 + hq, len(ctx), hq, 8, ctx)
        kc, vc, ks, vs = make_pool(inp, "int8")
        pool = dev_pool(kc, vc, ks, vs, "int8")
        kw = {}
        if fused:
            nk, nv = rows(hq, 1, len(ctx), 8), rows(hq, 2, len(ctx), 8)
            kw = dict(new_k=dev_bf16(nk), new_v=dev_bf16(nv))
            at = [int(inp.block_tables[b][(c - 1) // 256]) * 256 + (c - 1) % 256 for b, c in enumerate(ctx)]
            q8.store(f64(nk), kc, ks, at, "int8")
            q8.store(f64(nv), vc, vs, at, "int8")
        out = torch.full((len(ctx), hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        pa.decode_q8(dev_bf16(inp.q), *pool, dev_i32(inp.block_tables), dev_i32(inp.context_lens), inp.scale,
                     workspace=ws, out=out, **kw)
        assert pa.get_device_error() == (0, 0)
        want, tol = q8.decode(f64(inp.q), kc, ks, vc, vs, "int8", inp.block_tables, inp.context_lens, inp.scale)
        assert np.all(np.abs(host_f64(out) - want) <= tol), (hq, ctx)


def top_rows():
    """Rows whose largest magnitudes are bf16's last values (0x7f7f is the
    largest), at and around what a code would round up to 2^128."""
    x = f64(normal_bf16(21, 1, (48, 2, 128))) * 2.0 ** 122
    key = bits(x)
    for i in range(40):
        key[i, :, 7 + i] = 0x7F7F - i
        key[i, :, 99 - i] = 0xFF7F - i // 2
    key[40] = 0x7F7F
    key[41] = 0xFF7E
    key[42, :, ::2] = 0x7F60
    return key


@pytest.mark.parametrize("fmt", FMTS)
def test_finite_rows_read_back_finite(fmt):
    """The largest bf16 numbers too: codes as the definition has them, values
    finite and within the documented error."""
    key = top_rows()
    n, hkv = key.shape[:2]
    slots = np.arange(n, dtype=np.int32)
    check_store(key, key[::-1].copy(), slots, 3, 16, fmt)
    pool = pa.kvcache_q8(3, 16, hkv, dtype=FMTS[fmt])
    pa.store_kvcache_q8(dev_bf16(key), dev_bf16(key), *pool, dev_i32(slots))
    x = f64(key)
    for t in pa.load_kvcache_q8(*pool, dev_i32(slots)):
        got = host_f64(t)
        assert np.isfinite(got).all()
        a = np.abs(x).max(-1, keepdims=True)
        if fmt == "e4m3":
            big = np.abs(x) >= 2.0 ** -13 * a
            assert np.all(np.abs(got - x)[big] <= 2.0 ** -4 * np.abs(x)[big])
        else:
            assert np.all(np.abs(got - x) <= a / 85)


@pytest.mark.parametrize("fmt", FMTS)
def test_fused_store_of_rows_at_the_top(fmt):
    key = top_rows()
    n, hkv = key.shape[:2]
    inp = make_decode("top", 22, n, 4, hkv, [1 + i % 5 for i in range(n)], block_size=16)
    host = make_pool(inp, fmt)
    apart, fused = dev_pool(*host, fmt), dev_pool(*host, fmt)
    bt, c, new = dev_i32(inp.block_tables), dev_i32(inp.context_lens), dev_bf16(key)
    pa.store_kvcache_q8(new, new, *apart, pa.slot_mapping_decode(bt, c, 16))
    pa.decode_q8(dev_bf16(inp.q), *fused, bt, c, inp.scale, new_k=new, new_v=new)
    assert same_bytes(fused, apart)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("power", [-122, -119, -115, -110, -70, 70, 110, 122])
def test_decode_of_small_and_large_values(power, fmt):
    """Value rows near both ends of bf16's range: the outputs are of their size."""
    ctx = [1, 3, 40, 700, 5000]
    inp = make_decode("values", 23, len(ctx), 8, 2, ctx)
    inp.v_cache[:] = bits(f64(inp.v_cache) * 2.0 ** power)
    out = check_decode(inp, fmt)
    assert (out.abs().amax(-1) > 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_of_every_scale_byte(fmt):
    """Value rows under the smallest and the largest scale bytes, 0 and 254 too
    (which the store does not write), with codes that keep the values in range."""
    inp = make_decode("bytes", 24, 4, 8, 2, [17, 64, 300, 1])
    kc, vc, ks, vs = make_pool(inp, fmt)
    one = np.random.default_rng(3).choice(np.array([0x38, 0xB8, 0x30, 0] if fmt == "e4m3" else [1, 255, 0, 1],
                                                   np.uint8), size=vc.shape)
    for byte in (0, 1, 2, 7, 252, 253, 254):
        check_decode(inp, fmt, (kc, one if byte > 200 else vc, ks, np.full_like(vs, byte)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k_power,q_power,scale_power", [(124, -110, -18), (125, -120, -9), (-115, 120, -9), (-122, 118, 0)])
def test_decode_scores_of_huge_and_tiny_factors(k_power, q_power, scale_power, fmt):
    """Ordinary scores that are products of a huge and a tiny factor."""
    inp = make_decode("factors", 25, 4, 8, 2, [33, 700, 2, 128])
    inp.k_cache[:] = bits(f64(inp.k_cache) * 2.0 ** k_power)
    q = bits(f64(inp.q) * 2.0 ** q_power)
    check_decode(inp, fmt, q=q, scale=2.0 ** scale_power)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_of_huge_keys_that_are_orthogonal_to_huge_queries(fmt):
    inp = make_decode("orthogonal", 26, 3, 8, 2, [33, 700, 2])
    k, q = f64(inp.k_cache) * 2.0 ** 122, f64(inp.q) * 2.0 ** 120
    k[..., 64:] = 0.0
    q[..., :64] = 0.0
    inp.k_cache[:] = bits(k)
    out = check_decode(inp, fmt, q=bits(q), scale=1.0)
    assert torch.isfinite(out).all()


def test_a_table_wider_than_32_bits_is_refused():
    pool = pa.kvcache_q8(2, 16, 1)
    q, ctx = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda"), dev_i32([3])
    bt = torch.zeros(1, (1 << 32) + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pa.decode_q8(q, *pool, bt, ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("spread", [12, 16, 18, 20, 24])
def test_decode_q_spread_within_a_head(spread, fmt):
    """A head whose largest element meets only zeros, so that its scores are
    those of elements 2^spread smaller."""
    inp = make_decode("spread", 27, 4, 8, 2, [33, 700, 2, 128])
    k, q = f64(inp.k_cache), f64(inp.q) * 2.0 ** -spread
    k[..., 5] = 0.0
    q[..., 5] = 1.5
    inp.k_cache[:] = bits(k)
    check_decode(inp, fmt, q=bits(q), scale=2.0 ** (spread - 4))


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_q_at_both_ends_of_the_range(fmt):
    """Heads whose largest element is bf16's largest, near its smallest, or 0."""
    inp = make_decode("ends", 29, 4, 8, 2, [33, 700, 2, 128])
    base = f64(inp.q)
    for power, scale in ((125, 2.0 ** -125), (-93, 2.0 ** 93), (-96, 2.0 ** 96), (-112, 2.0 ** 112),
                         (-124, 2.0 ** 124)):
        q = base * 2.0 ** power * 0.25
        q[1, 3] = 0.0
        if power > 0:
            q[0, 0, 9] = 3.3895313892515355e38
            q[2, 5, 7] = -3.3895313892515355e38
        check_decode(inp, fmt, q=bits(q), scale=scale / 8)


@pytest.mark.parametrize("fmt", FMTS)
def test_several_tokens_of_one_sequence_in_a_batch(fmt):
    """Draft tokens of one sequence scored as rows of a batch, over one table at
    lengths n, n + 1, n + 2: stored by a call of their own (the fused store's
    slots may not lie in another row's context)."""
    for n in (30, 31, 254, 1500):
        inp = make_decode("draft", 28, 3, 8, 2, [n + 3] * 3)
        bt = np.repeat(inp.block_tables[:1], 3, axis=0)
        ctx = np.array([n + 1, n + 2, n + 3], np.int32)
        one = make_decode("draft", 28, 3, 8, 2, [n + 3] * 3)
        one.block_tables, one.context_lens = bt, ctx
        kc, vc, ks, vs = make_pool(one, fmt)
        pool = dev_pool(kc, vc, ks, vs, fmt)
        nk, nv = rows(n, 1, 3, 2), rows(n, 2, 3, 2)
        slots = pa.slot_mapping_decode(dev_i32(bt), dev_i32(ctx), 256)
        pa.store_kvcache_q8(dev_bf16(nk), dev_bf16(nv), *pool, slots)
        at = slots.cpu().numpy()
        q8.store(f64(nk), kc, ks, at, fmt)
        q8.store(f64(nv), vc, vs, at, fmt)
        out = pa.decode_q8(dev_bf16(inp.q), *pool, dev_i32(bt), dev_i32(ctx), inp.scale)
        want, tol = q8.decode(f64(inp.q), kc, ks, vc, vs, fmt, bt, ctx, inp.scale)
        assert np.all(np.abs(host_f64(out) - want) <= tol)
