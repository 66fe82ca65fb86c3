"""GPU parity of the 8-bit pool (pa_store_kvcache_q8, pa_load_kvcache_q8,
pa_decode_q8) with its float64 definition (oracle/q8.py), through the C ABI.

Store and load are compared bit by bit: a scale is a power of two, so a code is
one rounding of the bf16 value and reading it back is exact.

Decode is held to the bound that oracle/q8.py derives for each output."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import paged_kv_cache_store_gb300 as pa
from oracle import q8
from paged_kv_cache_store_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits, make_decode, normal_bf16
from gpu_util import dev_bf16, dev_i32, host_bits, host_f64

pytestmark = pytest.mark.gpu
FMTS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def dev_u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_pool(kc, vc, ks, vs, fmt):
    return dev_u8(kc).view(FMTS[fmt]), dev_u8(vc).view(FMTS[fmt]), dev_u8(ks), dev_u8(vs)


def host_u8(t):
    return t.view(torch.uint8).cpu().numpy()


def stale_pool(seed, nb, hkv, B):
    """Pool contents that were never written: any byte."""
    rng = np.random.default_rng(seed)
    return [rng.integers(0, 256, (nb, hkv, B, 128), dtype=np.uint8) for _ in range(2)] + \
           [rng.integers(0, 256, (nb, hkv, B), dtype=np.uint8) for _ in range(2)]


def rows(seed, tag, n, hkv, spread=0):
    """bf16 bits of n rows, each (token, head) with its own power of two in [-spread, spread]."""
    x = f64(normal_bf16(seed, tag, (n, hkv, 128)))
    if spread:
        x *= np.exp2(np.random.default_rng(seed + tag).integers(-spread, spread + 1, (n, hkv, 1)))
    return f32_to_bf16_bits(x.astype(np.float32))


def check_store(key, val, slots, nb, B, fmt, dkey=None, dval=None):
    hkv = key.shape[1]
    kc, vc, ks, vs = stale_pool(3, nb, hkv, B)
    pool = dev_pool(kc, vc, ks, vs, fmt)
    pa.store_kvcache_q8(dev_bf16(key) if dkey is None else dkey, dev_bf16(val) if dval is None else dval, *pool,
                        dev_i32(slots))
    q8.store(f64(key), kc, ks, slots, fmt)
    q8.store(f64(val), vc, vs, slots, fmt)
    for got, want, name in zip(pool, (kc, vc, ks, vs), ("k codes", "v codes", "k scales", "v scales")):
        assert np.array_equal(host_u8(got), want), name
    assert pa.get_device_error() == (0, 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv,n,nb,B", [(8, 64, 4, 256), (8, 1, 2, 256), (1, 1, 1, 16), (2, 333, 30, 16),
                                        (3, 77, 6, 48), (4, 2000, 70, 32)])
def test_store_bit_exact(hkv, n, nb, B, fmt):
    rng = np.random.default_rng(n)
    slots = rng.permutation(nb * B)[:n].astype(np.int32)
    if n > 1:
        slots[rng.random(n) < 0.15] = -1
    check_store(rows(n, 1, n, hkv), rows(n, 2, n, hkv, 20), slots, nb, B, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_store_range_edges(fmt):
    """Rows of zeros, of the smallest and the largest magnitudes, at the limits
    of a code's range, on ties, with infinities and NaNs."""
    n = 40
    x = f64(normal_bf16(9, 1, (n, 2, 128)))
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 2.0 ** -133                     # smallest bf16 subnormal
    x[3] *= 2.0 ** -128
    x[4] = 3.3895313892515355e38           # largest bf16
    x[5] = np.where(np.arange(128) % 2 == 0, 1.0, 2.0 ** -133)
    x[6, :, 3] = np.inf
    x[7, 0, 5] = -np.inf
    x[8, 1, 127] = np.nan
    x[9] = np.nan
    x[10] = np.arange(128) - 64.0          # ties of both formats
    x[11] = (np.arange(128) + 0.5) * 0.5
    for i, m in enumerate((1.75, 1.7578125, 1.984375, 1.9921875, 1.0, 1.5)):  # 448, just above, 127, just above
        x[12 + i] = 0.3 * x[12 + i] / np.abs(x[12 + i]).max()
        x[12 + i, :, 64] = -m * 2.0 ** (3 * i - 5)
    with np.errstate(over="ignore"):
        key = f32_to_bf16_bits(x.astype(np.float32))
    key[9] = 0x7FC1                        # bf16 NaNs with payloads
    key[8, 1, 127] = 0xFF81
    check_store(key, key[::-1].copy(), np.arange(n, dtype=np.int32), 3, 16, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_store_strided_fused_qkv_rows(fmt):
    n, hq, hkv, d = 50, 16, 8, 128
    qkv = normal_bf16(5, 1, (n, (hq + 2 * hkv), d))
    t = dev_bf16(qkv)
    slots = np.random.default_rng(5).permutation(8 * 64)[:n].astype(np.int32)
    check_store(qkv[:, hq:hq + hkv].copy(), qkv[:, hq + hkv:].copy(), slots, 8, 64, fmt,
                t[:, hq:hq + hkv], t[:, hq + hkv:])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv,nb,B", [(8, 6, 256), (1, 3, 16), (3, 7, 48)])
def test_load_bit_exact(hkv, nb, B, fmt):
    """Every code and scale byte, repeated slots, padding; outputs strided."""
    kc, vc, ks, vs = stale_pool(11, nb, hkv, B)
    ks[0, 0, :4] = [0, 1, 254, 255]
    rng = np.random.default_rng(1)
    slots = np.concatenate([rng.integers(0, nb * B, 200), [-1, -7, 0, 0, 1, 2, 3]]).astype(np.int32)
    pool = dev_pool(kc, vc, ks, vs, fmt)
    n = len(slots)
    wide = torch.full((n, hkv + 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = pa.load_kvcache_q8(*pool, dev_i32(slots), out_k=wide[:, :hkv])
    assert pa.get_device_error() == (0, 0)
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        c, s = c.transpose(0, 2, 1, 3).reshape(nb * B, hkv, 128), s.transpose(0, 2, 1).reshape(nb * B, hkv)
        want = np.where((slots < 0)[:, None, None], 0.0, q8.values(c[slots], s[slots], fmt))
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want).float().to(torch.bfloat16)  # exact in bf16's normal range
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=1234.0), torch.nan_to_num(want, nan=1234.0))
    assert torch.all(wide[:, hkv] == 7.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv", [1, 2, 3, 4, 5, 7, 8])
def test_long_calls_of_every_head_count(hkv, fmt):
    """Calls long enough for every number of rows that a unit may take, and
    head counts that such a number does not divide."""
    n, nb, B = 6000, 130, 48
    rng = np.random.default_rng(hkv)
    slots = rng.permutation(nb * B)[:n].astype(np.int32)
    slots[rng.random(n) < 0.1] = -1
    key, value = rows(hkv, 1, n, hkv), rows(hkv, 2, n, hkv, 20)
    check_store(key, value, slots, nb, B, fmt)
    kc, vc, ks, vs = stale_pool(3, nb, hkv, B)
    q8.store(f64(key), kc, ks, slots, fmt)
    q8.store(f64(value), vc, vs, slots, fmt)
    got = pa.load_kvcache_q8(*dev_pool(kc, vc, ks, vs, fmt), dev_i32(slots))
    for t, x in zip(got, (key, value)):
        want = np.where((slots < 0)[:, None, None], 0.0, q8.values(*q8.quantise(f64(x), fmt), fmt))
        assert np.array_equal(f64(t.view(torch.int16).cpu().numpy().view(np.uint16)), want)


def test_out_of_range_slots_are_recorded():
    kc, vc, ks, vs = stale_pool(2, 2, 2, 16)
    pool = dev_pool(kc, vc, ks, vs, "int8")
    slots = dev_i32([3, 2 * 16, -1, 31])
    key = dev_bf16(rows(1, 1, 4, 2))
    pa.get_device_error()
    pa.store_kvcache_q8(key, key, *pool, slots)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_SLOT, 1)
    k, v = pa.load_kvcache_q8(*pool, slots)
    assert pa.get_device_error() == (pa.PA_DEV_BAD_SLOT, 1)
    assert torch.all(k[1] == 0) and torch.all(v[1] == 0)
    q8.store(f64(rows(1, 1, 4, 2)), kc, ks, [3, -1, -1, 31], "int8")
    assert np.array_equal(host_u8(pool[0]), kc) and np.array_equal(host_u8(pool[2]), ks)


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------

def make_pool(inp, fmt, spread=0):
    """The generator's pool, quantised; slots that no context holds keep stale bytes."""
    nb, B, hkv = inp.num_blocks, inp.block_size, inp.num_kv_heads
    kc, vc, ks, vs = stale_pool(inp.batch, nb, hkv, B)
    held = np.zeros((nb, B), bool)
    for b in range(inp.batch):
        pos = np.arange(int(inp.context_lens[b]))
        held[inp.block_tables[b][pos // B], pos % B] = True
    rng = np.random.default_rng(4)
    for x, c, s in ((inp.k_cache, kc, ks), (inp.v_cache, vc, vs)):
        x = f64(x)
        if spread:
            x = x * np.exp2(rng.integers(-spread, spread + 1, (nb, B, hkv, 1)))
        cc, ss = q8.quantise(x, fmt)
        blk, off = np.nonzero(held)
        c[blk, :, off], s[blk, :, off] = cc[blk, off], ss[blk, off]
    return kc, vc, ks, vs


def check_decode(inp, fmt, pool=None, q=None, dq=None, scale=None, spread=0):
    kc, vc, ks, vs = make_pool(inp, fmt, spread) if pool is None else pool
    q = inp.q if q is None else q
    scale = inp.scale if scale is None else scale
    out = pa.decode_q8(dev_bf16(q) if dq is None else dq, *dev_pool(kc, vc, ks, vs, fmt), dev_i32(inp.block_tables),
                       dev_i32(inp.context_lens), scale)
    assert pa.get_device_error() == (0, 0)
    want, tol = q8.decode(f64(q), kc, ks, vc, vs, fmt, inp.block_tables, inp.context_lens, scale)
    got = host_f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    err = np.abs(got - want) - tol
    assert not np.any(err > 0), (float(np.nanmax(err)), np.unravel_index(np.nanargmax(err), err.shape))
    return out


EDGE_CTX = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 256, 257, 513, 1000]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,hkv", [(8, 8), (16, 8), (32, 8), (64, 8), (3, 3), (8, 1)])
def test_decode_edge_lengths(hq, hkv, fmt):
    check_decode(make_decode("edge", 100 + hq, len(EDGE_CTX), hq, hkv, EDGE_CTX), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B", [16, 32, 48, 64, 128, 256, 512])
def test_decode_block_sizes(B, fmt):
    ctx = [1, B - 1, B, B + 1, 3 * B + 7, 700]
    check_decode(make_decode("B", 200 + B, len(ctx), 8, 2, ctx, block_size=B, extra_table_cols=2), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch,hq,hkv,ctx", [(1, 1, 1, 1), (1, 8, 1, 9000), (2, 8, 2, 20000), (1, 4, 2, 33)])
def test_decode_few_long(batch, hq, hkv, ctx, fmt):
    check_decode(make_decode("long", 300, batch, hq, hkv, [ctx] * batch), fmt)


def test_decode_wide_scales():
    """Rows that differ by 2^20 in magnitude: the weight that counts belongs to
    a small value row, or to a large one."""
    for fmt in FMTS:
        check_decode(make_decode("wide", 17, 5, 8, 2, [40, 333, 64, 1000, 7]), fmt, spread=10, scale=1e-3)


def test_decode_many_short_sequences():
    ctx = np.random.default_rng(3).integers(0, 90, size=300)
    inp = make_decode("short", 31, 300, 8, 2, np.maximum(ctx, 1))
    inp.context_lens[:] = ctx
    out = check_decode(inp, "int8")
    assert torch.all(out[torch.from_numpy(ctx == 0).cuda()] == 0)


@pytest.mark.parametrize("hq,hkv", [(8, 1), (1, 1)])
def test_decode_largest_batch(hq, hkv):
    ctx = np.random.default_rng(5).integers(1, 40, size=2048)
    ctx[::7] = 1
    check_decode(make_decode("2048", 33, 2048, hq, hkv, ctx, block_size=16), "e4m3")


def test_decode_no_context_at_all():
    inp = make_decode("zero", 34, 5, 8, 2, [1] * 5)
    inp.context_lens[:] = 0
    inp.block_tables[:] = -1
    assert not check_decode(inp, "int8").any()


def test_decode_q_of_extreme_sizes():
    inp = make_decode("q", 41, 3, 8, 2, [50, 300, 17])
    q = f64(inp.q)
    q[0] *= 2.0 ** 100
    q[1, 3] = 0.0
    q[1, 4] *= 2.0 ** -130
    q[2, :, 7] *= 2.0 ** 12
    inp.k_cache[:] = f32_to_bf16_bits((f64(inp.k_cache) * 2.0 ** -4).astype(np.float32))
    bits = f32_to_bf16_bits(q.astype(np.float32))
    inp.q[:] = bits
    # Sequence 0 alone has |x| far above 64; a scale of 2^-100 brings it back.
    one = make_decode("q", 41, 3, 8, 2, [50, 300, 17])
    one.q[:] = bits
    one.context_lens[:] = [50, 0, 0]
    check_decode(one, "e4m3", scale=2.0 ** -103)
    inp.context_lens[:] = [0, 300, 17]
    check_decode(inp, "e4m3", scale=2.0 ** -12)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_nan_rows_stay_in_their_head(fmt):
    inp = make_decode("nan", 51, 4, 8, 2, [100, 40, 700, 64])
    kc, vc, ks, vs = make_pool(inp, fmt)
    bt = inp.block_tables
    ks[bt[1][0], 0, 7] = 255                  # a key of sequence 1, kv head 0
    vs[bt[2][600 // 256], 1, 600 % 256] = 255  # a value row of sequence 2, kv head 1
    for s in (ks, vs):
        s[bt[3][0], :, 64:] = 255             # past sequence 3's context: never read
    kc[bt[3][0], :, 64:] = vc[bt[3][0], :, 64:] = 0x7F
    out = check_decode(inp, fmt, (kc, vc, ks, vs))
    got = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(got)
    want[1, :4] = want[2, 4:] = True
    assert np.array_equal(got, want)


def test_decode_q_with_infinities_and_nans():
    """A head's q with a NaN or an infinity makes that head's output NaN, no other's."""
    inp = make_decode("q nan", 55, 3, 8, 2, [40, 333, 64])
    pool = make_pool(inp, "e4m3")
    bits = inp.q.copy()
    bits[0, 1, 3], bits[1, 6, 127], bits[2, 0, 0] = 0x7F80, 0x7FC0, 0xFF80
    out = pa.decode_q8(dev_bf16(bits), *dev_pool(*pool, "e4m3"), dev_i32(inp.block_tables), dev_i32(inp.context_lens),
                       inp.scale)
    clean = check_decode(inp, "e4m3", pool)
    hit = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 6] = hit[2, 0] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


def test_pool_beyond_32_bit_offsets():
    """Blocks in the last part of pools of more than 2^32 bytes."""
    nb, B, hkv = 17000, 256, 8
    pool = [torch.empty(nb, hkv, B, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)] + \
           [torch.empty(nb, hkv, B, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert pool[0].numel() > 1 << 32
    bt = np.array([[nb - 1, 3], [nb - 700, -1]], np.int32)
    ctx, n = np.array([300, 200], np.int32), 500
    k, v, q = rows(1, 1, n, hkv), rows(1, 2, n, hkv), normal_bf16(1, 3, (2, 16, 128))
    cu = dev_i32([0, 300, 500])
    slots = pa.slot_mapping_prefill(dev_i32(bt), cu, cu, B, total_q=n)
    pa.store_kvcache_q8(dev_bf16(k), dev_bf16(v), *pool, slots)
    small = [np.zeros((4, hkv, B, 128), np.uint8) for _ in range(2)] + [np.zeros((4, hkv, B), np.uint8) for _ in range(2)]
    where = np.concatenate([np.arange(300), 2 * B + np.arange(200)])  # the same rows in a small pool
    q8.store(f64(k), small[0], small[2], where, "e4m3")
    q8.store(f64(v), small[1], small[3], where, "e4m3")
    lk, lv = pa.load_kvcache_q8(*pool, slots)
    sk, sv = pa.load_kvcache_q8(*dev_pool(*small, "e4m3"), dev_i32(where))
    assert torch.equal(lk, sk) and torch.equal(lv, sv)
    args = dev_bf16(q), dev_i32(ctx)
    out = pa.decode_q8(args[0], *pool, dev_i32(bt), args[1])
    want = pa.decode_q8(args[0], *dev_pool(*small, "e4m3"), dev_i32([[0, 1], [2, -1]]), args[1])
    assert torch.equal(out, want) and torch.isfinite(out).all()
    assert pa.get_device_error() == (0, 0)


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace."""
    a = make_decode("a", 92, 6, 16, 8, [3000, 40, 700, 1, 2048, 999])
    b = make_decode("b", 93, 3, 16, 8, [5000, 6000, 31])
    jobs = []
    for inp, fmt in ((a, "e4m3"), (b, "int8")):
        args = [dev_bf16(inp.q), *dev_pool(*make_pool(inp, fmt), fmt), dev_i32(inp.block_tables),
                dev_i32(inp.context_lens), inp.scale]
        jobs.append((args, pa.decode_q8(*args), pa.decode_q8_workspace(16, 8), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for j, (args, _, ws, s) in enumerate(jobs):
            got[j].append(pa.decode_q8(*args, workspace=ws, stream=s))
    torch.cuda.synchronize()
    for j, (_, want, _, _) in enumerate(jobs):
        assert all(torch.equal(g, want) for g in got[j])


def test_decode_strided_q_is_the_same():
    inp = make_decode("strided", 61, 4, 8, 2, [100, 40, 700, 64])
    pool = make_pool(inp, "int8")
    wide = torch.zeros(4, 12, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = dev_bf16(inp.q)
    assert torch.equal(check_decode(inp, "int8", pool), check_decode(inp, "int8", pool, dq=wide[:, 2:10]))


def test_decode_bad_context_and_bad_blocks():
    inp = make_decode("bad", 71, 4, 8, 2, [100, 600, 700, 64])
    kc, vc, ks, vs = make_pool(inp, "e4m3")
    dev = dev_pool(kc, vc, ks, vs, "e4m3")
    ctx = dev_i32([100, 600, 5000, -3])
    pa.get_device_error()
    out = pa.decode_q8(dev_bf16(inp.q), *dev, dev_i32(inp.block_tables), ctx, inp.scale)
    code, where = pa.get_device_error()
    assert code == pa.PA_DEV_BAD_CONTEXT and where in (2, 3)
    assert torch.all(out[3] == 0)             # a negative length is taken as 0
    bt = inp.block_tables.copy()
    bt[1, 0] = inp.num_blocks                  # reads as zeros
    pa.set_checked(True)
    try:
        out = pa.decode_q8(dev_bf16(inp.q), *dev, dev_i32(bt), dev_i32(inp.context_lens), inp.scale)
        code, where = pa.get_device_error()
    finally:
        pa.set_checked(False)
    assert (code, where) == (pa.PA_DEV_BAD_BLOCK, bt.shape[1])
    zk = [np.concatenate([a, np.zeros_like(a[:1])]) for a in (kc, vc, ks, vs)]
    want, tol = q8.decode(f64(inp.q), zk[0], zk[2], zk[1], zk[3], "e4m3", bt, inp.context_lens, inp.scale)
    assert np.all(np.abs(host_f64(out) - want) <= tol)


def test_decode_shared_blocks_and_repeats():
    """Tables that share blocks; the same call again (and after another shape
    on the same workspace) gives the same bits."""
    inp = make_decode("shared", 8, 6, 16, 4, [1025, 1300, 2048, 2000, 1100, 600], shared_prefix_seqs=4,
                      shared_prefix_blocks=4)
    kc, vc, ks, vs = make_pool(inp, "e4m3")
    dev = dev_pool(kc, vc, ks, vs, "e4m3")
    ws = pa.decode_q8_workspace(16, 4)
    q, bt, ctx = dev_bf16(inp.q), dev_i32(inp.block_tables), dev_i32(inp.context_lens)
    a = pa.decode_q8(q, *dev, bt, ctx, inp.scale, workspace=ws)
    pa.decode_q8(q[:2], *dev, bt[:2], ctx[:2], inp.scale, workspace=ws)
    for _ in range(5):
        assert torch.equal(a, pa.decode_q8(q, *dev, bt, ctx, inp.scale, workspace=ws))
    want, tol = q8.decode(f64(inp.q), kc, ks, vc, vs, "e4m3", inp.block_tables, inp.context_lens, inp.scale)
    assert np.all(np.abs(host_f64(a) - want) <= tol)


# ---------------------------------------------------------------------------
# The store fused into the decode
# ---------------------------------------------------------------------------

def same_bytes(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,hkv,B,ctx", [(16, 8, 256, EDGE_CTX), (64, 8, 16, EDGE_CTX), (3, 3, 48, EDGE_CTX),
                                          (8, 2, 32, [0, 1, 0, 32, 33, 5000, 64, 0]), (8, 1, 512, [9000])])
def test_decode_store_is_store_then_decode(hq, hkv, B, ctx, fmt):
    """Outputs, codes and scales bit by bit, rows inside a wider tensor; slots
    that hold stale bytes (NaN codes and scales among them) before the call."""
    inp = make_decode("fused", 7, len(ctx), hq, hkv, [max(c, 1) for c in ctx], block_size=B)
    inp.context_lens[:] = ctx
    host = make_pool(inp, fmt)
    nk, nv = rows(3, 1, len(ctx), hkv, 5), rows(3, 2, len(ctx), hkv, 5)
    nk[0, 0, 3] = 0x7F80 if ctx[0] > 1 else nk[0, 0, 3]
    wide = dev_bf16(np.concatenate([nk, nv], axis=1))
    dk, dv = wide[:, :hkv], wide[:, hkv:]
    bt, c, q = dev_i32(inp.block_tables), dev_i32(inp.context_lens), dev_bf16(inp.q)
    apart, fused = dev_pool(*host, fmt), dev_pool(*host, fmt)
    pa.store_kvcache_q8(dk, dv, *apart, pa.slot_mapping_decode(bt, c, B))
    want = pa.decode_q8(q, *apart, bt, c, inp.scale)
    ws = pa.decode_q8_workspace(hq, hkv)
    for _ in range(2):  # the second call stores the same rows again
        got = pa.decode_q8(q, *fused, bt, c, inp.scale, workspace=ws, new_k=dk, new_v=dv)
        assert torch.equal(torch.nan_to_num(got, nan=77.0), torch.nan_to_num(want, nan=77.0))
        assert same_bytes(fused, apart)
    assert pa.get_device_error() == (0, 0)


def test_decode_store_with_an_invalid_block():
    inp = make_decode("bad slot", 9, 2, 8, 2, [100, 300])
    pool = dev_pool(*make_pool(inp, "e4m3"), "e4m3")
    before = [t.clone() for t in pool]
    bt = inp.block_tables.copy()
    bt[0, 0], bt[1, 1] = -1, inp.num_blocks
    new = dev_bf16(rows(1, 1, 2, 2))
    out = pa.decode_q8(dev_bf16(inp.q), *pool, dev_i32(bt), dev_i32(inp.context_lens), inp.scale, new_k=new, new_v=new)
    assert same_bytes(pool, before) and torch.isfinite(out).all() and not out[0].any()
    pa.get_device_error()
    pa.decode_q8(dev_bf16(inp.q), *pool, dev_i32(inp.block_tables), dev_i32([5000, -1]), inp.scale, new_k=new, new_v=new)
    assert pa.get_device_error()[0] == pa.PA_DEV_BAD_CONTEXT and same_bytes(pool, before)
    with pytest.raises(ValueError):
        pa.decode_q8(dev_bf16(inp.q), *pool, dev_i32(bt), dev_i32(inp.context_lens), new_k=new)
    with pytest.raises(ValueError):
        pa.decode_q8(dev_bf16(inp.q), *pool, dev_i32(bt), dev_i32(inp.context_lens), new_k=new, new_v=new[:1])


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

def test_prefill_then_decode_steps():
    """An engine's steps over the 8-bit pool: store two prompts' rows, read
    them back for the prefill of a chunk, then decode steps that store one
    token each.  Block tables from the block manager's layout (any order)."""
    B, hq, hkv, fmt = 32, 8, 2, "int8"
    scale = 1.0 / math.sqrt(128)
    lens, bt = [70, 33], np.array([[5, 2, 7, 1], [4, 0, 3, -1]], np.int32)
    pool = pa.kvcache_q8(8, B, hkv, dtype=FMTS[fmt])
    kc, vc = (np.zeros((8, hkv, B, 128), np.uint8) for _ in range(2))
    ks, vs = (np.zeros((8, hkv, B), np.uint8) for _ in range(2))
    cu = np.cumsum([0] + lens).astype(np.int32)
    total = int(cu[-1])
    k, v, q = rows(1, 1, total, hkv), rows(1, 2, total, hkv), normal_bf16(1, 3, (total, hq, 128))
    slots = pa.slot_mapping_prefill(dev_i32(bt), dev_i32(cu), dev_i32(cu), B, total_q=total)
    pa.store_kvcache_q8(dev_bf16(k), dev_bf16(v), *pool, slots)
    h = slots.cpu().numpy()
    q8.store(f64(k), kc, ks, h, fmt)
    q8.store(f64(v), vc, vs, h, fmt)
    lk, lv = pa.load_kvcache_q8(*pool, slots)
    out = pa.prefill_varlen(dev_bf16(q), lk, lv, dev_i32(cu), dev_i32(cu), max(lens), max(lens), scale)
    want = O.prefill(q, host_bits(lk), host_bits(lv), cu, cu, scale)
    assert np.abs(host_f64(out).reshape(want.shape) - want).max() <= 2e-2
    ws = pa.decode_q8_workspace(hq, hkv)
    ctx = np.array(lens, np.int32)
    for step in range(3):
        ctx += 1
        nk, nv, nq = rows(step, 4, 2, hkv), rows(step, 5, 2, hkv), normal_bf16(step, 6, (2, hq, 128))
        s = pa.slot_mapping_decode(dev_i32(bt), dev_i32(ctx), B)
        pa.store_kvcache_q8(dev_bf16(nk), dev_bf16(nv), *pool, s)
        out = pa.decode_q8(dev_bf16(nq), *pool, dev_i32(bt), dev_i32(ctx), scale, workspace=ws)
        h = s.cpu().numpy()
        q8.store(f64(nk), kc, ks, h, fmt)
        q8.store(f64(nv), vc, vs, h, fmt)
        want, tol = q8.decode(f64(nq), kc, ks, vc, vs, fmt, bt, ctx, scale)
        assert np.all(np.abs(host_f64(out) - want) <= tol)
    assert np.array_equal(host_u8(pool[0]), kc) and np.array_equal(host_u8(pool[3]), vs)
    assert pa.get_device_error() == (0, 0)


def test_captured_step_replays_with_new_inputs():
    inp = make_decode("graph", 81, 5, 8, 2, [100, 40, 700, 64, 1])
    pool = dev_pool(*make_pool(inp, "e4m3"), "e4m3")
    eager = [t.clone() for t in pool]
    q, bt, ctx = dev_bf16(inp.q), dev_i32(inp.block_tables), dev_i32(inp.context_lens)
    nk, nv = dev_bf16(rows(1, 1, 5, 2)), dev_bf16(rows(1, 2, 5, 2))
    ws, slots, out = pa.decode_q8_workspace(8, 2), torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty_like(q)

    def step(p, w, o):
        pa.slot_mapping_decode(bt, ctx, inp.block_size, out=slots)
        pa.store_kvcache_q8(nk, nv, *p, slots)
        return pa.decode_q8(q, *p, bt, ctx, inp.scale, workspace=w, out=o)

    # Warm-up before capture, on a pool of its own (a captured step does not run).
    step([t.clone() for t in pool], pa.decode_q8_workspace(8, 2), torch.empty_like(q))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(pool, ws, out)
    for i in range(3):
        q.copy_(dev_bf16(normal_bf16(i, 7, (5, 8, 128))))
        nk.copy_(dev_bf16(rows(i, 8, 5, 2)))
        ctx.copy_(dev_i32([100 + i, 40 + i, 650, 64 - i, i]))
        g.replay()
        torch.cuda.synchronize()
        want = step(eager, pa.decode_q8_workspace(8, 2), torch.empty_like(q))
        assert torch.equal(out, want)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pool, eager))
    assert pa.get_device_error() == (0, 0)


def test_other_stream():
    inp = make_decode("stream", 91, 3, 8, 2, [100, 40, 700])
    pool = make_pool(inp, "int8")
    want = check_decode(inp, "int8", pool)
    s = torch.cuda.Stream()
    args = [dev_bf16(inp.q), *dev_pool(*pool, "int8"), dev_i32(inp.block_tables), dev_i32(inp.context_lens)]
    s.wait_stream(torch.cuda.current_stream())
    got = pa.decode_q8(*args, inp.scale, stream=s)
    k, _ = pa.load_kvcache_q8(*args[1:5], dev_i32([0, 5]), stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.isfinite(k).any()


def test_refusals_of_the_binding():
    pool = pa.kvcache_q8(2, 16, 2)
    key = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = dev_i32([0, 1, 2])
    with pytest.raises(TypeError):
        pa.store_kvcache_q8(key.float(), key, *pool, slots)
    with pytest.raises(ValueError):
        pa.store_kvcache_q8(key, key[:2], *pool, slots)
    with pytest.raises(ValueError):
        pa.store_kvcache_q8(key, key, *pool, slots[:2])
    with pytest.raises(ValueError):
        pa.store_kvcache_q8(key, key, pool[0], pool[1], pool[2][:1], pool[3][:1], slots)
    with pytest.raises(TypeError):
        pa.store_kvcache_q8(key, key, pool[0], pool[1].view(torch.int8), pool[2], pool[3], slots)
    with pytest.raises(TypeError):
        pa.load_kvcache_q8(*pool, slots.long())
    with pytest.raises(pa.PagedAttentionError):
        pa.load_kvcache_q8(*pool, slots, out_k=torch.zeros(3, 258, 128, dtype=torch.bfloat16, device="cuda")
                           .view(-1)[4:4 + 3 * 256].view(3, 2, 128))
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    bt, ctx = dev_i32([[0, 1]]), dev_i32([5])
    with pytest.raises(ValueError):
        pa.decode_q8(q, *pool, bt[:, :1].expand(2, 1), ctx)
    with pytest.raises(pa.PagedAttentionError):
        pa.decode_q8(q, *pool, bt, ctx, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        pa.decode_q8(q, *pool, bt, ctx, out=torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        pa.kvcache_q8(2, 16, 2, dtype=torch.bfloat16)
