"""Pins for oracle.layer: E4M3 rounding against torch's cast and the 256 codes,
norm and attention against pure-Python loops, the rotation against complex
products, row scales against their definition."""

import cmath
import math

import numpy as np
import pytest
import torch

from oracle import formats, layer


def test_e4m3_round_matches_the_codes_and_torch():
    codes = formats.e4m3_value(np.arange(256))
    codes = codes[np.isfinite(codes)]
    assert np.array_equal(layer.e4m3_round(codes), codes)
    r = np.random.default_rng(1)
    x = (r.standard_normal(20000) * np.exp2(r.uniform(-12, 9, 20000))).astype(np.float32)
    x = np.concatenate([x, [0.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6, 447.9, 448.0, 17.0, 19.0]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(layer.e4m3_round(x), want)
    assert layer.e4m3_round(1e9) == 448 and layer.e4m3_round(-1e9) == -448


def test_quantise_rows():
    y = np.array([[1.0, -2.0, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0], [np.nan, 3.0, -1.0, 0.0]], dtype=np.float32)
    v, s = layer.quantise(y)
    assert s[0] == np.float32(2.0) / np.float32(448) and s[1] == np.float32(2.0 ** -100)
    assert v[0, 1] == -448 and v[0, 0] == 224 and np.all(v[1] == 0)
    assert s[2] == np.float32(3.0) / np.float32(448) and np.isnan(v[2, 0]) and v[2, 1] == 448


def test_rms_norm_against_loops():
    r = np.random.default_rng(2)
    x, w = r.standard_normal((3, 5)), r.standard_normal(5)
    y = layer.rms_norm(x, w, 1e-3)
    for t in range(3):
        d = math.sqrt(sum(v * v for v in x[t]) / 5 + 1e-3)
        for i in range(5):
            assert y[t, i] == pytest.approx(x[t, i] / d * w[i], rel=1e-14)
    assert np.all(layer.rms_norm(np.zeros((1, 5)), w, 1e-6) == 0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_by_the_axis_position(interleaved):
    r = np.random.default_rng(3)
    T, D, rot, sections = 4, 12, 8, [1, 2, 1]
    x = r.standard_normal((T, 2, D)).astype(np.float32)
    angle = np.arange(30)[:, None] * np.array([1.0, 0.5, 0.25, 0.125])[None, :]
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = r.integers(0, 30, (3, T))
    y = layer.rope(x, pos, table, sections, interleaved)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    for t in range(T):
        for f, a in enumerate([0, 1, 1, 2]):
            i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + 4)
            for h in range(2):
                z = complex(x[t, h, i], x[t, h, j]) * cmath.exp(1j * angle[pos[a, t], f])
                assert abs(complex(y[t, h, i], y[t, h, j]) - z) <= 1e-6 * (1 + abs(z))
    same = layer.rope(x, np.full((1, T), 99), table, None, interleaved)
    assert np.array_equal(same, x)                       # outside the table


def test_attend_against_loops_and_edges():
    r = np.random.default_rng(4)
    q, k, v = r.standard_normal((4, 8)), r.standard_normal((5, 2, 8)), r.standard_normal((5, 2, 8))
    out, lse, mag = layer.attend(q, k, v, 0.3)
    for h in range(4):
        w = [math.exp(0.3 * sum(q[h, d] * k[t, h // 2, d] for d in range(8))) for t in range(5)]
        assert lse[h] == pytest.approx(math.log(sum(w)), rel=1e-13)
        for d in range(8):
            assert out[h, d] == pytest.approx(sum(w[t] * v[t, h // 2, d] for t in range(5)) / sum(w), rel=1e-12)
    assert np.all(mag >= np.abs(out) - 1e-15)
    out, lse, _ = layer.attend(q, k[:1], v[:1], 0.3)
    assert np.allclose(out, np.repeat(v[0], 2, 0))       # one token: its value
    out, lse, _ = layer.attend(q, k[:0], v[:0], 0.3)
    assert np.all(out == 0) and np.all(lse == -np.inf)
