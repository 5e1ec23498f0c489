"""Decode over 8-bit pages at large scores, held to a bound that a wrong power of two cannot meet.

The keys are 1 in one dimension and 0 .. -4 in another, the query two powers of two, the softmax
scale ln 2 times a power of two: every score (base 2) is a whole number that fp32 holds, the same
for the kernel and the reference, and the softmax weights are powers of two.  The value rows are
positive and carry exponents of their own, so that the sums do not cancel.

Tolerance.  What is left to round: the weights' exponentials (2^-22 each), fp32 sums of at most 700
terms (2^-14.5 of the sum in the worst order; the 2^-24 steps of one warp's few dozen terms and of
the join make 2^-17), the weights in fp16, exact powers of two down to 2^-24 of their reference,
which is at most 2^8 below the largest weight, and a bf16 half step:
  |o - o64| <= 2^-8 |o64| + 2^-16 sum_j p_j |v_j| + n 16 2^-25 max_j p_j 2^(e_j)
(values are under 16).  lse: 2^-22 of itself, and 2^-16.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kvcache as ref
from test_gpu_decode_e4m3 import Cache, f64, swa  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def scored(lens, Hq, Hkv, d, page, p, sign, q_up=0, k_up=0, code=1.0, seed=21):
    """Scores sign * 2^p - j * step, j in 0 .. 4 by row, step 8 or what fp32 holds beside 2^p; the
    factors 2^q_up and 2^k_up more in the query and the keys, the latter held as `code` (e4m3)."""
    unit = min(code, 64.0)   # so that 4 of it are an e4m3 value
    c = Cache(lens, [1] * len(lens), Hq, Hkv, d, 64, 0, page, seed)
    r = np.random.default_rng(seed)
    seen = [np.swapaxes(e, 1, 2) != 255 for e in c.exps]   # [page, slot, head]
    k = np.zeros(c.codes[0].shape)
    k[..., 7] = sign * code
    k[..., 8] = -unit * r.integers(0, 5, k.shape[:-1])
    v = r.integers(0x30, 0x50, k.shape)
    kb, vb = np.full(seen[0].shape, 127 + k_up - int(math.log2(code))), 127 + r.integers(-12, 13, seen[0].shape)
    for i, (codes, byte) in enumerate(((ref.e4m3_code(k), kb), (v, vb))):
        c.codes[i] = np.where(seen[i][..., None], codes, 0x7f).astype(np.uint8)
        c.exps[i] = np.ascontiguousarray(np.swapaxes(np.where(seen[i], byte, 255), 1, 2).astype(np.uint8))
    c.q.zero_()
    c.q[..., 7] = 2.0 ** (p + q_up)
    c.q[..., 8] = 2.0 ** (max(3, p - 20) + q_up) * (code / unit)
    return c


def check(c, scale, o, lse):
    with np.errstate(invalid="ignore", over="ignore"):
        k, v = (ref.contiguous(ref.page_values(x, e), c.table) for x, e in zip(c.codes, c.exps))
    ve = ref.contiguous(np.swapaxes(c.exps[1], 1, 2)[..., None], c.table)[..., 0]
    want, want_lse, absum, peak, _ = ref.decode(f64(c.q), k, v, ve, c.lens, c.gate, c.W, c.S, scale)
    n = c.lens[:, None, None]
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * absum + n * 16 * 2.0 ** -25 * peak[..., None]
    assert np.all(tol < 0.01 * want)   # neither zeros nor a factor of two pass
    err = np.abs(f64(o) - want)
    assert np.all(err <= tol), (np.max(err / want), np.max(err / tol))
    assert np.all(np.abs(f64(lse) - want_lse) <= 2.0 ** -22 * np.abs(want_lse) + 2.0 ** -16)


def run(swa, c, scale):
    o, lse = swa.decode_paged_e4m3(*c.args(), scale=scale, want_lse=True)
    assert swa.get_device_error() == 0
    return o, lse


LN2 = float(np.float32(math.log(2.0)))
SHAPES = [([1, 40, 700], 2, 1, 128, 16), ([33, 500], 12, 1, 128, 32), ([5, 300], 4, 2, 64, 4), ([129], 13, 1, 64, 2)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("p", [3, 20, 24, 26, 27, 60, 127])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", SHAPES)
def test_value_exponents_at_large_scores(swa, lens, Hq, Hkv, d, page, p, sign):  # noqa: F811
    """Value rows keep their powers of two whatever the size of the scores (in base 2, 2^24 and up:
    the steps of fp32 are as large as the exponents)."""
    c = scored(lens, Hq, Hkv, d, page, min(p, 126), sign)
    scale = LN2 * (2.0 if p == 127 else 1.0)
    check(c, scale, *run(swa, c, scale))


@pytest.mark.parametrize("p,q_up,k_up,scale_up,code", [
    (119, 8, -8, 0, 256),       # q to 2^127, keys as append writes them: codes of 256, a small power of two
    (20, 100, -100, 0, 256),
    (10, -120, 120, 0, 1),      # the reverse
    (3, -129, 127, 2, 1),       # both at the ends of their types
    (24, -60, -60, 120, 256),   # the scale makes up for both
    (24, -130, 10, 120, 1),
    (60, 60, 60, -120, 256),    # products past fp32, scores inside
    (24, 90, 35, -125, 256),
    (70, 57, -133, 76, 2.0 ** -9),
])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", SHAPES)
def test_scores_inside_fp32_whatever_their_factors(swa, lens, Hq, Hkv, d, page, p, q_up, k_up, scale_up, code):  # noqa: F811
    """Only the score has to be in the range of fp32, not the query, the key row's power of two and
    the softmax scale multiplied in some order."""
    scale = LN2 * 2.0 ** scale_up
    c = scored(lens, Hq, Hkv, d, page, p, 1, q_up, k_up, code)
    bits = c.q[0, 0, 7:9].float().log2().numpy()
    assert np.all(bits == np.rint(bits)) and bits.min() >= -126   # powers of two, none rounded away
    check(c, scale, *run(swa, c, scale))


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("below", [10, 20, 25, 28, 31])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [([320], 4, 1, 128, 16), ([600], 12, 1, 64, 4)])
def test_small_weights_beside_a_large_one(swa, lens, Hq, Hkv, d, page, below, first):  # noqa: F811
    """One key of score 0 whose value row is zero in the even dimensions; all others at -below with
    positive values there.  The even dimensions come from weights of 2^-below of the largest alone,
    powers of two, which 16 bits hold to 2^-31: they are right to a bf16 half step and the sums."""
    c = scored(lens, Hq, Hkv, d, page, 3, 1)
    top = 0 if first else lens[0] - 1
    for b in range(len(lens)):
        for t in range(lens[b]):
            at = c.table[b, t // page], t % page
            c.codes[0][at] = 0
            c.codes[0][at][..., 8] = ref.e4m3_code(np.array(0.0 if t == top else -1.0))
            c.codes[1][at] = 0x40 + t % 3 if t != top else np.tile([0, 0x40], d // 2)
            c.exps[0][at[0], :, at[1]] = c.exps[1][at[0], :, at[1]] = 127
    c.q[..., 7] = 0
    c.q[..., 8] = below
    o, lse = run(swa, c, LN2)
    k, v = (ref.contiguous(np.nan_to_num(ref.page_values(x, e), nan=0.0, posinf=0.0), c.table) for x, e in zip(c.codes, c.exps))
    ve = ref.contiguous(np.swapaxes(c.exps[1], 1, 2)[..., None], c.table)[..., 0]
    want, want_lse, absum, _, _ = ref.decode(f64(c.q), k, v, ve, c.lens, c.gate, c.W, c.S, LN2)
    err = np.abs(f64(o) - want)
    assert np.all(want > 0) and np.all(err <= 2.0 ** -8 * want + 2.0 ** -16 * absum), np.max(err / want)
    assert np.all(np.abs(f64(lse) - want_lse) <= 2.0 ** -16)


@pytest.mark.parametrize("lens,Hq,Hkv,d,page", SHAPES)
def test_weights_as_exact_as_fp32(swa, lens, Hq, Hkv, d, page):  # noqa: F811
    """Scores that are multiples of 5/8 in base 2, exact, so that the weights fill their mantissas; values
    of both signs, so that results far below the sum of absolute terms show the weights' own error.
    Left are the exponentials (2^-22 each, of weights and sum), the weights' two halves (2^-22) and fp32
    sums of a part's few dozen terms (2^-19): 2^-17 of the sum of absolute terms, and a bf16 half step."""
    c = scored(lens, Hq, Hkv, d, page, 3, 1)
    r = np.random.default_rng(22)
    c.codes[1] = np.where(c.codes[1] == 0x7f, 0x7f, c.codes[1] | (r.integers(0, 2, c.codes[1].shape) << 7)).astype(np.uint8)
    c.q[..., 7] = 0.0
    c.q[..., 8] = 0.625
    o, lse = run(swa, c, LN2)
    with np.errstate(invalid="ignore", over="ignore"):
        k, v = (ref.contiguous(ref.page_values(x, e), c.table) for x, e in zip(c.codes, c.exps))
    ve = ref.contiguous(np.swapaxes(c.exps[1], 1, 2)[..., None], c.table)[..., 0]
    want, want_lse, absum, _, _ = ref.decode(f64(c.q), k, v, ve, c.lens, c.gate, c.W, c.S, LN2)
    err = np.abs(f64(o) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * absum), np.max(err / absum)
    assert np.all(np.abs(f64(lse) - want_lse) <= 2.0 ** -17)
