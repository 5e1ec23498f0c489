"""Frequencies that are not finite, and ones far above 1: NaN in their pair alone, as position times
frequency is, and the angle modulo a turn as exactly as for small ones."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import swiattn_inputs as inp
from oracle import kvcache as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_router_gb300 as m
    return m


def freqs(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


BAD = {3: math.nan, 10: math.inf, 17: -math.inf}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", ["rope", "rope_backward"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_frequency_that_is_not_finite_spoils_its_pair_alone(swa, name, dtype, interleaved):
    x = inp.randn((2, 5, 3, 64), dtype, inp._gen(31)).cuda()
    w, good = freqs(48), freqs(48)
    pairs = []
    for f, value in BAD.items():
        w[f] = value
        pairs += [2 * f, 2 * f + 1] if interleaved else [f, f + 24]
    got, _ = getattr(swa, name)(x, None, w.cuda(), interleaved=interleaved)
    want, _ = getattr(swa, name)(x, None, good.cuda(), interleaved=interleaved)
    want[..., pairs] = math.nan
    torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)


def test_append_with_such_a_frequency(swa):
    g = inp._gen(32)
    q, k, v = (inp.randn((6, h, 64), torch.bfloat16, g).cuda() for h in (4, 2, 2))
    w = freqs(64)
    w[5] = math.inf
    table, lens = torch.arange(6, dtype=torch.int32).view(6, 1).cuda(), torch.arange(1, 7, dtype=torch.int32).cuda()
    pages = [torch.zeros((6, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    out = swa.append_paged(q, k, v, *pages, table, lens, w.cuda())
    rows = torch.arange(6).cuda(), torch.arange(6).cuda()
    for t in (out, pages[0][rows]):
        bad = torch.isnan(t)
        assert bool(bad[..., [5, 37]].all()) and int(bad.sum()) == bad[..., 0].numel() * 2
    assert torch.equal(pages[1][rows], v)
    e4m3 = [p.to(torch.float8_e4m3fn) for p in pages]
    exps = [torch.zeros((6, 2, 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    swa.append_paged(q, k, v, *e4m3, table, lens, w.cuda(), k_exp=exps[0], v_exp=exps[1])
    codes = e4m3[0].view(torch.uint8)[rows]
    assert bool((codes[..., [5, 37]] & 0x7f == 0x7f).all()) and int((codes & 0x7f == 0x7f).sum()) == 24
    assert swa.get_device_error() == 0


def test_frequencies_above_one(swa):
    """w up to 2^40 at positions up to 2^20, against rational arithmetic.  The fraction of a turn is
    right to 2^-63 of the turns made (2^-66 or so of them here after the product's own truncation,
    2^-64 of a turn a position), the rest as for small frequencies."""
    w = torch.tensor([1.5, 3.0, 100.25, 4096.125, 5000.0, 2.0 ** 20 + 0.5, 2.0 ** 40, 1e9 / 3], dtype=torch.float64)
    positions = [0, 1, 7, 1000, 65537, 1 << 20]
    x = inp.randn((1, len(positions), 2, 64), torch.float32, inp._gen(33))
    got, _ = swa.rope(x.cuda(), None, w.cuda(), positions=torch.tensor([positions], dtype=torch.int32).cuda())
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    theta, off = np.zeros((len(positions), 8)), np.zeros((len(positions), 8))
    for i, p in enumerate(positions):
        for f in range(8):
            a = Fraction(float(w[f])) * p / two_pi
            theta[i, f] = float((a - math.floor(a)) * two_pi)
            off[i, f] = 2 * math.pi * (float(a) * 2.0 ** -63 + p * 2.0 ** -64)
    c, s = np.cos(theta)[None, :, None], np.sin(theta)[None, :, None]
    y = x.double().numpy()
    a, b = y[..., :8], y[..., 8:16]
    want = y.copy()
    want[..., :8], want[..., 8:16] = a * c - b * s, b * c + a * s
    tol = 6 * 2.0 ** -24 * ref.pair_sums(y, w.numpy())
    tol[..., :8] += off[None, :, None] * (np.abs(a) + np.abs(b))
    tol[..., 8:16] += off[None, :, None] * (np.abs(a) + np.abs(b))
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
