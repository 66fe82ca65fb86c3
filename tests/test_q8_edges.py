"""The 8-bit pool's documented errors and its ends of the range, in the
definition (no GPU)."""
import numpy as np
import pytest

from oracle import q8
from paged_kv_cache_store_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits

LARGEST = bf16_bits_to_f32(np.array([0x7F7F], np.uint16)).astype(np.float64)[0]


def bf16(x):
    return bf16_bits_to_f32(f32_to_bf16_bits(np.asarray(x, np.float32))).astype(np.float64)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_finite_row_has_finite_values(fmt):
    """Each of bf16's last 200 numbers as a row's largest, the others below it:
    every value read back is a finite bf16 number, and the nearest such."""
    held = q8.e4m3_values()[:127] if fmt == "e4m3" else np.arange(128.0)
    for b in range(0x7F7F - 199, 0x7F80):
        row = np.resize(np.arange(b - 300, b + 1), 128)
        row[0] = b
        x = bf16_bits_to_f32(row.astype(np.uint16)).astype(np.float64) * np.where(np.arange(128) % 3 == 1, -1, 1)
        c, s = q8.quantise(x[None], fmt)
        got = q8.values(c, s, fmt)[0]
        assert np.all(np.abs(got) <= LARGEST)
        grid = held * 2.0 ** (float(s[0]) - 127)
        grid = grid[grid <= LARGEST]
        assert np.array_equal(np.abs(got - x), np.abs(np.abs(x)[:, None] - grid).min(-1))
