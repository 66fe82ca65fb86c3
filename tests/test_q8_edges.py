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


SWEEP = np.concatenate([np.exp2(np.linspace(-17, 0, 120)), [0.0, 1.0, -1.0, 0.5, -0.5, 2.0 ** -13, 2.0 ** -16, 0.25]])


@pytest.mark.parametrize("top", [224.5, 225.0, 300.0, 447.0, 448.0, 1.0, 2.0 ** -60 * 230, 2.0 ** 119 * 225, LARGEST])
def test_e4m3_error_bound(top):
    """The larger of 2^-4 of a value and 2^-10 * 2^e; the former from 2^-13 of the
    row's largest magnitude on."""
    a = bf16(top)
    x = bf16(a * SWEEP)
    c, s = q8.quantise(x[None], "e4m3")
    err = np.abs(q8.values(c, s, "e4m3")[0] - x)
    big = np.abs(x) >= 2.0 ** -13 * a
    assert np.all(err[big] <= 2.0 ** -4 * np.abs(x)[big])
    assert np.all(err <= np.maximum(2.0 ** -10 * np.exp2(float(s[0]) - 127), 2.0 ** -4 * np.abs(x)))


def test_e4m3_relative_bound_ends_above_2_to_minus_15():
    x = np.zeros(128)
    x[:2] = 225.0, 0.0069580078125          # above 2^-15 of the row's largest
    c, s = q8.quantise(x[None], "e4m3")
    assert abs(q8.values(c, s, "e4m3")[0, 1] - x[1]) > 2.0 ** -4 * x[1]


@pytest.mark.parametrize("top", [63.75, 64.0, 100.0, 126.5, 127.0, 1.0, 2.0 ** -100 * 65, 2.0 ** 121 * 127])
def test_int8_error_bound(top):
    """1/126 of the row's largest magnitude."""
    a = bf16(top)
    x = bf16(a * SWEEP)
    c, s = q8.quantise(x[None], "int8")
    assert np.all(np.abs(q8.values(c, s, "int8")[0] - x) <= a / 126)


def test_int8_error_at_the_ends_of_the_range():
    """1/85 where the largest magnitude is the largest bf16 number; half of
    2^-126 for rows under the smallest scale."""
    x = bf16(LARGEST * SWEEP)
    c, s = q8.quantise(x[None], "int8")
    assert s[0] == 249 and np.all(np.abs(q8.values(c, s, "int8")[0] - x) <= LARGEST / 85)
    for top in (2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -121, 2.0 ** -120.1):
        x = bf16(top * SWEEP)
        c, s = q8.quantise(x[None], "int8")
        assert s[0] == 1 and np.all(np.abs(q8.values(c, s, "int8")[0] - x) <= 2.0 ** -127)


def test_e4m3_rows_under_the_smallest_scale():
    """2^-4 of a value from 2^-132 on, whatever the row's largest magnitude."""
    for top in (2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -119):
        x = bf16(top * SWEEP)
        c, s = q8.quantise(x[None], "e4m3")
        err = np.abs(q8.values(c, s, "e4m3")[0] - x)
        assert s[0] == 1 and np.all(err <= 2.0 ** -4 * np.abs(x))
