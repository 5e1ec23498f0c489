"""64-bit reference of the position rotation, the paged append and the 8-bit page rows.

TEST INFRASTRUCTURE ONLY, as the rest of this package: plain numpy, written from the definitions,
sharing nothing with the CUDA path.  Decode over 8-bit pages is the oracle's own decode on the
values the pages stand for (``page_values``, ``contiguous``).
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def rotate(x, positions, inv_freq, interleaved=False, factor=1.0, transposed=False):
    """x [..., H, d] at positions [...]: each pair of dimensions turned by position * inv_freq."""
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(inv_freq, dtype=np.float64)
    theta = np.asarray(positions, dtype=np.float64)[..., None, None] * w
    c, s = factor * np.cos(theta), factor * np.sin(theta)
    if transposed:
        s = -s
    r = 2 * len(w)
    y = x.copy()
    first, second = (np.s_[..., 0:r:2], np.s_[..., 1:r:2]) if interleaved else (np.s_[..., :r // 2], np.s_[..., r // 2:r])
    a, b = x[first], x[second]
    y[first] = a * c - b * s
    y[second] = b * c + a * s
    return y


def pair_sums(x, inv_freq, interleaved=False):
    """|a| + |b| of each dimension's pair (0 where the rotation does not reach): the scale of the
    rotation's rounding errors."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    r = 2 * len(inv_freq)
    y = np.zeros_like(x)
    if interleaved:
        y[..., 0:r:2] = y[..., 1:r:2] = x[..., 0:r:2] + x[..., 1:r:2]
    else:
        y[..., :r // 2] = y[..., r // 2:r] = x[..., :r // 2] + x[..., r // 2:r]
    return y


def e4m3_value(code):
    """The value of e4m3 codes (uint8): sign, four exponent bits (bias 7), three mantissa bits;
    exponent 0 is subnormal, 0x7f and 0xff are NaN, there is no infinity."""
    code = np.asarray(code, dtype=np.int64)
    sign = np.where(code & 0x80, -1.0, 1.0)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((code & 0x7f) == 0x7f, np.nan, sign * v)


_VALUES = np.array([e4m3_value(c) for c in range(0x7f)])   # the non-negative codes, ascending


def e4m3_code(x):
    """Nearest e4m3 code, ties to the even code, the largest finite value beyond it, NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), E4M3_MAX)
    hi = np.searchsorted(_VALUES, a)              # _VALUES[hi - 1] < a <= _VALUES[hi]
    lo = np.maximum(hi - 1, 0)
    below, above = a - _VALUES[lo], _VALUES[hi] - a
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == _VALUES[hi], hi, code)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7f, code).astype(np.uint8)


def row_exponent(x):
    """e of each row (last dimension): the smallest integer in [-126, 127] with the row's largest
    finite or infinite |x| at most 448 * 2^e (NaN passed over)."""
    amax = np.max(np.where(np.isnan(x), 0.0, np.abs(x)), axis=-1)
    m, e = np.frexp(np.where(np.isinf(amax), 2.0 ** 128, amax))   # m in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875)
    return np.clip(np.where(amax == 0, -126, e), -126, 127).astype(np.int64)


def quantise(x):
    """(codes uint8 [..., d], exponent bytes uint8 [...]) of rows along the last dimension."""
    x = np.asarray(x, dtype=np.float64)
    e = row_exponent(x)
    return e4m3_code(np.ldexp(x, -e[..., None])), (e + 127).astype(np.uint8)


def page_values(codes, exps):
    """The values that pages [P, page, Hkv, d] of codes with exponent bytes [P, Hkv, page] stand for."""
    scale = np.ldexp(1.0, np.asarray(exps, dtype=np.int64) - 127)
    return e4m3_value(codes) * np.swapaxes(scale, 1, 2)[..., None]


def places(starts, seq_lens, block_table, page_size, num_pages, tokens):
    """Position and pool row of every token, row -1 where it is passed over; and whether any token
    was bad input."""
    pos, row, bad = np.zeros(tokens, np.int64), np.full(tokens, -1, np.int64), False
    for b, length in enumerate(np.asarray(seq_lens, dtype=np.int64)):
        first, last = (b, b + 1) if starts is None else (int(starts[b]), int(starts[b + 1]))
        for t in range(first, last):
            if length == 0:
                continue
            p = length - (last - t)
            if p < 0 or p // page_size >= block_table.shape[1]:
                bad = True
                continue
            page = int(block_table[b, p // page_size])
            if page < 0 or page >= num_pages:
                bad = True
                continue
            pos[t], row[t] = p, page * page_size + p % page_size
    return pos, row, bad


def contiguous(pages, block_table):
    """[B, max_pages * page_size, Hkv, d] out of a pool [P, page_size, Hkv, d]."""
    B, max_pages = block_table.shape
    return pages[np.asarray(block_table)].reshape(B, max_pages * pages.shape[1], *pages.shape[2:])


def visited(length, gate, W, S):
    """The cache entries that the query at the end of `length` tokens reads."""
    lo = 0 if gate else max(0, length - W)
    return np.concatenate([np.arange(min(S, lo)), np.arange(lo, length)]).astype(np.int64)


def decode(q, k, v, v_exps, seq_lens, gate, W, S, scale):
    """Decode over values k, v [B, L, Hkv, d] (v_exps [B, L, Hkv]: the exponent bytes of v's rows).
    Returns o, lse and, for tolerances: sum_j p_j |v_j| [B, Hq, d]; the largest weight of a row of
    8-bit values, max_j p_j 2^(byte - 127) [B, Hq]; and max_j scale sum_c |q_c k_jc| [B, Hq]."""
    B, Hq, d = q.shape
    Hkv = k.shape[2]
    o, absum = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    lse, peak, size = np.full((B, Hq), -np.inf), np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        at = visited(int(seq_lens[b]), gate[b], W, S)
        if len(at) == 0:
            continue
        for h in range(Hq):
            kk, vv = k[b, at, h // (Hq // Hkv)], v[b, at, h // (Hq // Hkv)]
            s = scale * (kk @ q[b, h])
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            lse[b, h] = m + np.log(e.sum())
            o[b, h], absum[b, h] = p @ vv, p @ np.abs(vv)
            peak[b, h] = np.max(p * np.ldexp(1.0, v_exps[b, at, h // (Hq // Hkv)].astype(np.int64) - 127))
            size[b, h] = scale * np.max(np.abs(kk) @ np.abs(q[b, h]))
    return o, lse, absum, peak, size
