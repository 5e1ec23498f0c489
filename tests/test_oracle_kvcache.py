"""Pins of the 64-bit reference of the rotation and the 8-bit page rows (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import kvcache as ref


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    # a quarter turn a position: (a, b) -> (-b, a) -> (-a, -b) -> (b, -a) -> (a, b)
    x = rng(0).standard_normal((5, 1, 4))
    w = np.array([math.pi / 2, math.pi / 2])
    y = ref.rotate(x, np.arange(5), w, interleaved)
    a, b = (np.s_[..., 0::2], np.s_[..., 1::2]) if interleaved else (np.s_[..., :2], np.s_[..., 2:])
    want = x.copy()
    for p, (sa, sb) in enumerate([((1, 0), (0, 1)), ((0, -1), (1, 0)), ((-1, 0), (0, -1)), ((0, 1), (-1, 0)),
                                  ((1, 0), (0, 1))]):
        want[p][a] = sa[0] * x[p][a] + sa[1] * x[p][b]
        want[p][b] = sb[0] * x[p][a] + sb[1] * x[p][b]
    np.testing.assert_allclose(y, want, atol=1e-12)
    # position 0 is the identity, the dimensions past the rotated ones pass through
    np.testing.assert_array_equal(ref.rotate(x, np.zeros(5), w[:1], interleaved), x)
    np.testing.assert_array_equal(ref.rotate(x, np.arange(5), w[:1], interleaved)[..., 2:], x[..., 2:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_gives_relative_positions(interleaved):
    """<R(i) q, R(j) k> depends on i - j alone."""
    q, k = rng(1).standard_normal((2, 1, 1, 16))
    w = 10000.0 ** (-np.arange(0, 16, 2) / 16)
    dot = lambda i, j: float(np.sum(ref.rotate(q, [i], w, interleaved) * ref.rotate(k, [j], w, interleaved)))
    assert abs(dot(7, 3) - dot(1004, 1000)) < 1e-9
    assert abs(dot(7, 3) - dot(8, 3)) > 1e-3


@pytest.mark.parametrize("interleaved", [False, True])
def test_transposed_map_is_the_gradient(interleaved):
    g = rng(2)
    x, dy = g.standard_normal((2, 3, 2, 16))
    pos, w = np.array([0, 5, 123]), g.uniform(0.01, 1, 4)
    loss = lambda z: float(np.sum(dy * ref.rotate(z, pos, w, interleaved, 1.3)))
    dx = ref.rotate(dy, pos, w, interleaved, 1.3, transposed=True)
    for at in [(0, 0, 0), (1, 1, 3), (2, 0, 7), (2, 1, 15)]:
        e = np.zeros_like(x)
        e[at] = 1e-5
        assert abs((loss(x + e) - loss(x - e)) / 2e-5 - dx[at]) < 1e-8


def test_e4m3_codes_against_the_type():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(ref.e4m3_value(codes.numpy()),
                                  codes.view(torch.float8_e4m3fn).double().numpy())
    # nearest, ties to even: every value, every midpoint, and values beside them
    v = ref._VALUES
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng(3).uniform(0, 448, 1000)])
    x = np.concatenate([x, -x]).astype(np.float32)   # the type converts from fp32
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_code(x), want)
    assert list(ref.e4m3_code([500.0, -1e30, np.inf, np.nan])) == [0x7e, 0xfe, 0x7e, 0x7f]


def test_row_exponent_is_the_smallest():
    g = rng(4)
    x = g.standard_normal((500, 8)) * np.exp(g.uniform(-60, 60, (500, 1)))
    x[0] = 0
    x[1] = [448.0] + [0] * 7
    x[2] = [np.nextafter(448.0, 1e9)] + [0] * 7
    x[3] = [np.nan, 3.0] + [0] * 6
    e = ref.row_exponent(x)
    top = np.nanmax(np.abs(x), axis=-1)
    assert np.all(top <= np.ldexp(448.0, e))
    some = e > -126
    assert np.all(top[some] > np.ldexp(448.0, e[some] - 1))
    assert e[0] == -126 and e[1] == 0 and e[2] == 1 and e[3] == -7
    codes, exps = ref.quantise(x)
    got = ref.page_values(codes[:, None, None], exps[:, None, None])[:, 0, 0]
    # half a step of a normal value, or of a subnormal one
    err = np.abs(got - x)
    assert np.all((err <= 2.0 ** -4 * np.abs(x) + np.ldexp(2.0 ** -10, e)[:, None]) | np.isnan(x))


def test_decode_equals_the_oracles():
    """On plain values, against the oracle's decode (itself pinned)."""
    import oracle
    g = rng(5)
    B, L, Hq, Hkv, d, W, S = 3, 40, 6, 3, 8, 7, 5
    q, k, v = g.standard_normal((B, Hq, d)), g.standard_normal((B, L, Hkv, d)), g.standard_normal((B, L, Hkv, d))
    lens, gate = np.array([40, 9, 1], np.int32), np.array([0, 0, 1], np.uint8)
    exps = np.full((B, L, Hkv), 127, np.uint8)
    o, lse, *_ = ref.decode(q, k, v, exps, lens, gate, W, S, 0.3)
    want, want_lse = oracle.decode_anchored(q, k, v, lens, gate, W, S, 0.3, want_lse=True)
    np.testing.assert_allclose(o, want, atol=1e-12)
    np.testing.assert_allclose(lse, want_lse, atol=1e-12)
    assert np.all(ref.decode(q, k, v, exps, [0, 0, 0], gate, W, S, 0.3)[0] == 0)
