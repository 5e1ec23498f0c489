"""What the tree attention makes of NaN and infinity in the entries that its tokens read first, beside
neighbours that do not read them.  Tolerances are those of test_gpu_tree."""
import numpy as np
import pytest
import torch

from oracle import kvcache as ref
from test_gpu_append import f64, raw, swa  # noqa: F401  (swa: the fixture)
from test_gpu_tree import KINDS, Case

pytestmark = pytest.mark.gpu


def put(c, which, b, j, x):
    """x in the third dimension of entry j of sequence b, all key heads (e4m3: NaN, whatever x)."""
    page = c.pages[which].shape[1]
    p, s = c.table[b, j // page], j % page
    if c.kind == "e4m3":
        c.pages[which].view(torch.uint8)[p, s, :, 3] = 0x7f
    else:
        c.pages[which][p, s, :, 3] = x


def values(c):
    c.values = [ref.page_values(raw(p), raw(e)) if c.kind == "e4m3" else f64(p) for p, e in zip(c.pages, c.exps)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base,W,S,keys", [
    (700, 100, 0, [0]),                # the first key of routed rows
    (700, 100, 5, [0]),                # of all rows, by their anchors
    (700, 100, 0, [0, 1, 2, 3]),       # a run of leading keys
    (700, 100, 0, [601]),              # the first key of the shallowest tokens' windows
    (300, 1, 0, [300]),                # a token's own, alone in its window
    (0, 50, 0, [0]),                   # no cache: the first drafted token
    (3, 5000, 0, [0, 40]),
])
def test_a_nan_in_the_first_keys_that_a_token_reads_reaches_it(swa, base, W, S, keys, d, kind):
    c = Case([40, 9], [base, 200], 4, 2, d, 16, kind, W, S, routed=0.25, seed=41)
    for j in keys:
        put(c, 0, 0, j, np.nan)
    values(c)
    got = c.run(swa)
    seen = ref.tree_visible(c.parents[:40], c.gate[:40], base, W, S)[:, keys].any(1)
    reads = np.concatenate([seen, np.zeros(9, bool)])
    assert reads.any() and swa.get_device_error() == 0
    o, lse = f64(got[0]), f64(got[1])
    assert np.isnan(o[reads]).all() and np.isnan(lse[reads]).all()
    want = c.reference()
    assert np.array_equal(np.isnan(want[1]).all(1), reads)
    c.check(got, want)   # the others


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("leading", [1, 3])
def test_leading_scores_of_minus_infinity_weigh_nothing(swa, leading, kind):
    """Rows that are computed again, because of a value that only their neighbours read, and whose first
    keys have a score of -infinity."""
    base, W = 700, 100
    c = Case([40], [base], 2, 2, 64, 16, kind, W, routed=0.25, seed=42)
    c.q[..., 3] = c.q[..., 3].abs() + 1
    put(c, 1, 0, 50, np.nan)   # a value of routed rows alone
    firsts = range(base - W + 1, base - W + 1 + leading)   # of the shallowest tokens' windows
    for j in firsts:
        put(c, 0, 0, j, 0.0)
    values(c)
    with np.errstate(invalid="ignore"):
        size = c.reference()[3]
    for j in firsts:
        put(c, 0, 0, j, -np.inf)
    values(c)
    with np.errstate(invalid="ignore"):
        want = list(c.reference())
    want[3] = size   # of the finite scores
    routed = c.gate[:40] != 0
    want[1][routed] = np.nan   # theirs is finite, but o is not: compared below
    got = c.run(swa)
    assert np.isnan(f64(got[0])[routed][..., 3]).all() and np.isfinite(f64(got[1])).all()
    c.check(got, want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", ["zero rows of 255", "keys of 0", "a key of 255"])
def test_exponent_bytes_mean_the_same_in_rows_that_are_computed_again(swa, case, d):
    """2^(byte - 127) for every byte, with and without a neighbour whose NaN has a row computed again."""
    base, W = 300, 60
    c = Case([30], [base], 4, 2, d, 16, "e4m3", W, routed=0.25, seed=43,
             scale={"zero rows of 255": None, "keys of 0": 2.0 ** 18, "a key of 255": 1.0}[case])
    page_of = lambda j: (c.table[0, j // 16], j % 16)   # noqa: E731
    codes = [p.view(torch.uint8) for p in c.pages]
    if case == "zero rows of 255":   # 0 times 2^128
        for which, j in ((0, 295), (1, 296), (0, 20), (1, 21)):
            p, s = page_of(j)
            codes[which][p, s] = 0
            c.exps[which][p, :, s] = 255
    elif case == "keys of 0":
        c.exps[0][:] = 0
        c.q = torch.ldexp(c.q.double(), torch.tensor(100.0).cuda()).to(c.dtype)
    else:
        p, s = page_of(297)
        codes[0][p, s] = torch.randint(0, 8, codes[0][p, s].shape, dtype=torch.uint8, device="cuda",
                                       generator=torch.Generator("cuda").manual_seed(1))   # up to 7 * 2^-9
        c.exps[0][p, :, s] = 255
        c.q = torch.ldexp(c.q.double(), torch.tensor(-123.0).cuda()).to(c.dtype)
    values(c)
    c.check(c.run(swa))
    put(c, 1, 0, 50, np.nan)   # read by routed rows alone
    values(c)
    with np.errstate(invalid="ignore"):
        want = list(c.reference())
    routed = c.gate[:30] != 0
    assert routed.any() and not routed.all()
    want[1][routed] = np.nan
    got = c.run(swa)
    assert np.isnan(f64(got[0])[routed][..., 3]).all()
    c.check(got, want)


@pytest.mark.parametrize("kind", KINDS)
def test_a_bad_length_of_a_sequence_without_drafts_is_reported(swa, kind):
    c = Case([6, 0, 9], [50, 30, 40], 2, 1, 64, 16, kind, 32, seed=44)
    want = c.reference()
    for length, status in ((-1, 1), (c.table.shape[1] * 16 + 1, 1), (-2 ** 31, 1), (0, 0), (c.table.shape[1] * 16, 0)):
        c.lens[1] = length
        got = c.run(swa)
        assert swa.get_device_error() == status, length
        c.check(got, want)
