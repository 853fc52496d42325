"""Cosines and sines that ts_kv_append_chunk_rope turns rows by, each against its own size.

A float32 row of pairs (1, 0) comes out as (cos a, sin a). The angle is a whole number of
2^-64 turns a position, off by two of them at most (its two parts are cut off), times the
position: 2 pi position 2^-63 in all. It is rounded to float32 once (2^-24 of itself), sine
and cosine are off by two units in the last place at most (4 * 2^-24) and their product
with the row's value is rounded once: 6 * 2^-24 of the result beside the first term. The
expected angles are fractions, reduced with 50 digits of pi."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_46_gb300 as ts
from long_context_cases import DEV, i32

pytestmark = pytest.mark.gpu

TURN = 2 * Fraction("3.14159265358979323846264338327950288419716939937511")
POSITIONS = [0, 1, 2, 3, 7, 100, 4097, 131_071, 16_777_217, 2 ** 31 - 2]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _angle(pos, freq):
    a = pos * Fraction(float(freq))
    return float(a - round(a / TURN) * TURN)


def _check(freq, D, interleaved):
    half, B = D // 2, len(POSITIONS)
    freq = np.asarray(freq, dtype=np.float32)
    assert freq.shape == (half,)
    row = torch.zeros(D)
    one = np.arange(half) * 2 if interleaved else np.arange(half)
    two = one + 1 if interleaved else one + half
    row[one] = 1.0
    rows = row.expand(B, 1, D).contiguous().to(DEV)
    pools = [torch.zeros(1, 16, 1, D, device=DEV) for _ in "kv"]
    got = ts.ts_kv_append_chunk_rope(rows, rows, rows, *pools, i32(np.full((B, 1), -1)), i32(np.array(POSITIONS) + 1),
                                     i32(np.arange(B + 1)), torch.from_numpy(freq).to(DEV), interleaved=interleaved)
    got = got[:, 0].double().cpu().numpy()
    a = np.array([[_angle(p, f) for f in freq] for p in POSITIONS])
    cut = 2 * math.pi * 2.0 ** -63 * np.array(POSITIONS, dtype=np.float64)[:, None]
    for name, x, want in (("cos", got[:, one], np.cos(a)), ("sin", got[:, two], np.sin(a))):
        err, bound = np.abs(x - want), 6 * 2.0 ** -24 * np.abs(want) + cut
        worst = np.unravel_index(np.argmax(err - bound), err.shape)
        assert np.all(err <= bound), (name, POSITIONS[worst[0]], freq[worst[1]], x[worst], want[worst])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_angles_of_usual_frequencies(D, interleaved):
    for base in (10_000.0, 500_000.0, 1e8):
        _check(base ** (-np.arange(D // 2) / (D // 2)), D, interleaved)


@pytest.mark.parametrize("D", [64, 128])
def test_angles_of_slow_frequencies(D):
    _check(2.0 ** -np.linspace(4, 36, D // 2), D, False)
    none = np.zeros(D // 2)
    none[::3] = 1e-7
    _check(none, D, True)


@pytest.mark.parametrize("D", [64, 128])
def test_angles_of_negative_and_of_fast_frequencies(D):
    sign = np.where(np.arange(D // 2) % 3 == 0, 1.0, -1.0)
    _check(-(2.0 ** -np.linspace(4, 36, D // 2)), D, False)
    _check(sign * 500_000.0 ** (-np.arange(D // 2) / (D // 2)), D, True)
    _check(sign * 2.0 ** np.linspace(-3, 40, D // 2), D, False)
