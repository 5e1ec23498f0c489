"""GPU parity of decode over 8-bit pages (swiattn_decode_paged_e4m3) against the 64-bit reference on
the values the pages stand for.

Tolerance, from the arithmetic.  Scores are sums of d exact products in fp32, off by at most
d 2^-22 times the sum of their absolute values (A, after the softmax scale); the exponential adds
2^-21.  A weight is therefore off by r = d 2^-22 A + 2^-21 of itself, the sum of weights too, and
the weights of the value product by 2^-11 more (fp16), or by 2^-25 of the largest where they are
subnormal, times at most 448 for each of the n keys.  So
  |o - o64| <= (2 r + 2^-11) sum_j p_j |v_j| + n 448 2^-25 max_j p_j 2^(e_j) + 2^-8 |o64|,
the last half a bf16 step, and lse within r + n 2^-24 (its fp32 sum) + 2^-20.
"""
import math

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


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Cache:
    """A shuffled pool of 8-bit pages with B sequences.  Every row that no query of the given
    lengths, gates, window and anchors visits holds NaN, values and exponents alike."""

    def __init__(self, lens, gate, Hq, Hkv, d, W, S, page, seed, spread=0.5, q_scale=1.0):
        g = inp._gen(seed)
        self.B, self.Hq, self.Hkv, self.d, self.W, self.S, self.page = len(lens), Hq, Hkv, d, W, S, page
        self.lens, self.gate = np.asarray(lens, np.int32), np.asarray(gate, np.uint8)
        self.max_pages = max(1, -(-int(self.lens.max()) // page))
        self.num_pages = self.B * self.max_pages + 2
        self.table = torch.randperm(self.num_pages, generator=g)[:self.B * self.max_pages].to(torch.int32)
        self.table = self.table.view(self.B, -1).numpy()
        self.codes, self.exps = [], []
        seen = np.zeros((self.num_pages, page), bool)
        for b in range(self.B):
            at = ref.visited(int(self.lens[b]), self.gate[b], W, S)
            seen[self.table[b, at // page], at % page] = True
        for _ in "kv":
            x = inp.randn((self.num_pages, page, Hkv, d), torch.float32, g)
            x *= torch.exp(spread * inp.randn((self.num_pages, page, Hkv, 1), torch.float32, g))
            codes, exps = ref.quantise(x.numpy())
            codes[~seen] = 0x7f
            exps[~seen] = 255
            self.codes.append(codes)
            self.exps.append(np.ascontiguousarray(np.swapaxes(exps, 1, 2)))
        self.q = (inp.randn((self.B, Hq, d), torch.float32, g) * q_scale).to(torch.bfloat16)

    def args(self):
        pages = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in self.codes]
        exps = [torch.from_numpy(e).cuda() for e in self.exps]
        return [self.q.cuda(), *pages, *exps, torch.from_numpy(self.table).cuda(),
                torch.from_numpy(self.lens).cuda(), torch.from_numpy(self.gate).cuda(), self.W]

    def reference(self):
        with np.errstate(invalid="ignore", over="ignore"):
            k, v = (ref.contiguous(ref.page_values(c, e), self.table) for c, e in zip(self.codes, self.exps))
        ve = ref.contiguous(np.swapaxes(self.exps[1], 1, 2)[..., None], self.table)[..., 0]
        return ref.decode(f64(self.q), k, v, ve, self.lens, self.gate, self.W, self.S, 1.0 / math.sqrt(self.d))

    def check(self, o, lse):
        want, want_lse, absum, peak, size = self.reference()
        n = np.array([len(ref.visited(int(L), g, self.W, self.S)) for L, g in zip(self.lens, self.gate)])[:, None]
        r = self.d * 2.0 ** -22 * size + 2.0 ** -21
        tol = ((2 * r + 2.0 ** -11)[..., None] * absum + (n * 448 * 2.0 ** -25 * peak)[..., None]
               + 2.0 ** -8 * np.abs(want))
        err = np.abs(f64(o) - want)
        assert np.all(err <= tol), (err.max(), np.max(err - tol))
        got = f64(lse)
        some = n[:, 0] > 0
        assert np.all(np.abs(got[some] - want_lse[some]) <= (r + n * 2.0 ** -24 + 2.0 ** -20)[some])
        assert np.all(np.isneginf(got[~some])) and np.all(f64(o)[~some] == 0)


def run(swa, c, **more):
    o, lse = swa.decode_paged_e4m3(*c.args(), n_anchor=c.S, want_lse=True, **more)
    assert swa.get_device_error() == 0
    return o, lse


@pytest.mark.parametrize("lens,gate,Hq,Hkv,d,W,S,page", [
    ([9000, 4000], [1, 0], 2, 1, 64, 3900, 0, 32),                        # runs of many tiles
    ([20] * 700, [0, 1] * 350, 16, 8, 64, 300, 0, 16),                    # more (sequence, head)s than warps
    ([1], [0], 1, 1, 64, 1, 0, 1),
    ([1], [1], 16, 1, 128, 4, 0, 16),
    ([777], [1], 16, 16, 128, 256, 0, 16),
    ([2, 15, 16, 17, 33], [0, 1, 0, 1, 0], 8, 1, 128, 16, 0, 32),         # around a tile
    ([100, 200, 300], [0, 0, 0], 9, 1, 64, 31, 5, 8),                     # nine heads: two groups
    ([513, 0, 64, 1200], [1, 1, 0, 0], 6, 2, 128, 100, 0, 64),            # an empty slot
    ([1000, 1111, 3, 400], [0, 0, 0, 1], 12, 4, 64, 90, 256, 16),         # anchors
    ([1000, 95, 96, 97, 112], [0, 0, 0, 0, 0], 4, 2, 128, 91, 5, 2),      # anchors and window in one tile
    ([5000, 40], [1, 0], 16, 1, 64, 64, 0, 256),                          # several chunks
    ([3000, 2999], [1, 0], 5, 5, 128, 2000, 17, 1),                       # pages of one token
    ([700], [0], 15, 1, 128, 600, 0, 1024),                               # a page longer than the cache
    ([50] * 70, [0, 1] * 35, 2, 1, 64, 20, 3, 16),                        # many sequences
])
def test_matches_reference(swa, lens, gate, Hq, Hkv, d, W, S, page):
    c = Cache(lens, gate, Hq, Hkv, d, W, S, page, seed=len(lens) * 100 + Hq)
    c.check(*run(swa, c))


@pytest.mark.parametrize("G", range(1, 17))
def test_every_group_size(swa, G):
    c = Cache([90, 17], [0, 1], 2 * G, 2, 128, 40, 8, 16, seed=G)
    c.check(*run(swa, c))


@pytest.mark.parametrize("spread,q_scale", [(12.0, 1.0), (0.5, 30.0), (3.0, 1e-30), (0.0, 1e4)])
def test_rows_and_queries_of_very_different_size(swa, spread, q_scale):
    """Value rows from 2^-50 to 2^50, scores in the hundreds, tiny and large queries."""
    c = Cache([300, 64], [1, 0], 8, 2, 64, 50, 4, 16, seed=3, spread=spread, q_scale=q_scale)
    if spread > 1:   # keys stay of order 1, so that the softmax is not one key alone
        x = np.random.default_rng(4).standard_normal(c.codes[0].shape)
        seen = c.exps[0] != 255
        codes, exps = ref.quantise(x)
        c.codes[0] = np.where(np.swapaxes(seen, 1, 2)[..., None], codes, 0x7f).astype(np.uint8)
        c.exps[0] = np.where(seen, np.swapaxes(exps, 1, 2), 255).astype(np.uint8)
    c.check(*run(swa, c))


def test_visited_entries_exactly(swa):
    """q = 0 gives every visited entry the same weight: lse is ln of their number, and a value row of
    ones at one entry, zeros elsewhere, comes out as 1 / number exactly where that entry is visited."""
    lens, gate, W, S, page = [400, 400, 61, 16], [0, 1, 0, 0], 133, 21, 8
    c = Cache(lens, gate, 3, 1, 64, W, S, page, seed=6)
    c.q.zero_()
    c.codes = [np.full_like(c.codes[0], 0x38), np.zeros_like(c.codes[1])]   # keys 1.0, values 0
    c.exps = [np.full_like(c.exps[0], 127) for _ in "kv"]
    n = np.array([len(ref.visited(L, g, W, S)) for L, g in zip(lens, gate)])
    for j in [0, 1, 15, 16, 20, 21, 22, 60, 61, 266, 267, 268, 300, 398, 399]:
        values = np.zeros_like(c.codes[1])
        for b in range(4):
            if j < c.max_pages * page:
                values[c.table[b, j // page], j % page] = 0x38   # 1.0
        c.codes[1] = values
        o, lse = run(swa, c)
        np.testing.assert_array_equal(np.rint(np.exp(f64(lse))).astype(int), np.repeat(n[:, None], 3, 1))
        hit = np.array([j in ref.visited(L, g, W, S) for L, g in zip(lens, gate)])
        want = np.where(hit, 1.0 / n, 0.0)
        # half a bf16 step, and the sum of the weights
        assert np.all(np.abs(f64(o) - want[:, None, None]) <= 2.0 ** -7 * want[:, None, None]), j


def test_nan_in_a_visited_row_reaches_its_heads_alone(swa):
    for which, at in ((0, 70), (1, 70), (0, 99), (1, 0)):
        c = Cache([100, 100], [1, 1], 4, 2, 64, 10, 0, 16, seed=7)
        c.codes[which][c.table[0, at // 16], at % 16, 1, 5] = 0x7f
        o, _ = run(swa, c)
        bad = torch.isnan(o.cpu())
        want = torch.zeros_like(bad)
        if which == 0:
            want[0, 2:] = True
        else:
            want[0, 2:, 5] = True
        assert torch.equal(bad, want)


def test_result_is_repeatable_and_right_in_any_batch(swa):
    lens, gate = [900, 40, 333, 0, 2000], [1, 0, 0, 1, 0]
    c = Cache(lens, gate, 8, 2, 128, 200, 30, 32, seed=8)
    o, lse = run(swa, c)
    again, _ = run(swa, c)
    assert torch.equal(o, again)
    q, kp, vp, ke, ve, table, sl, gt, W = c.args()
    for b in range(5):
        one, one_lse = swa.decode_paged_e4m3(q[b:b + 1].contiguous(), kp, vp, ke, ve, table[b:b + 1].contiguous(),
                                             sl[b:b + 1].contiguous(), gt[b:b + 1].contiguous(), W, n_anchor=30,
                                             want_lse=True)
        whole = c.lens, c.gate, c.table, c.q, c.B
        c.lens, c.gate, c.table, c.q, c.B = c.lens[b:b + 1], c.gate[b:b + 1], c.table[b:b + 1], c.q[b:b + 1], 1
        c.check(one, one_lse)
        c.lens, c.gate, c.table, c.q, c.B = whole


@pytest.mark.parametrize("page", [16, 4])
@pytest.mark.parametrize("spoil", ["page high", "page low", "long", "negative"])
def test_bad_device_input_is_reported(swa, spoil, page):
    """A bad table entry is read as page 0, a length outside the table is clamped: reported once, and
    the result is that of the corrected input."""
    c = Cache([300, 200], [1, 1], 2, 2, 128, 64, 0, page, seed=9)
    c.codes = [np.where(x == 0x7f, 0, x).astype(np.uint8) for x in c.codes]
    c.exps = [np.where(x == 255, 127, x).astype(np.uint8) for x in c.exps]
    q, kp, vp, ke, ve, table, sl, gt, W = c.args()
    if spoil.startswith("page"):
        table[0, 3] = c.num_pages if spoil == "page high" else -7
        c.table[0, 3] = 0
    else:
        sl[0] = c.max_pages * page + 1 if spoil == "long" else -1
        c.lens[0] = c.max_pages * page if spoil == "long" else 0
    o, lse = swa.decode_paged_e4m3(q, kp, vp, ke, ve, table, sl, gt, W, want_lse=True)
    assert swa.get_device_error() == 1 and swa.get_device_error() == 0
    c.check(o, lse)


def test_workspace_streams_and_graphs(swa):
    c = Cache([600, 100], [1, 0], 4, 2, 128, 64, 0, 16, seed=10)
    a = c.args()
    want = swa.decode_paged_e4m3(*a)
    nbytes = swa.decode_paged_e4m3_workspace(2, c.max_pages, 16, 4, 2, 128, 64)
    room = torch.full((nbytes + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    ws = room[:nbytes]
    assert torch.equal(swa.decode_paged_e4m3(*a, workspace=ws), want)
    assert bool((room[nbytes:] == 0xAB).all())
    with pytest.raises(swa.SwiAttnError):
        swa.decode_paged_e4m3(*a, workspace=ws[:-1])
    with pytest.raises(swa.SwiAttnError):
        swa.decode_paged_e4m3(*a, workspace=room[8:])
    out, out2 = torch.zeros_like(want), torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        swa.decode_paged_e4m3(*a, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    # two graphs that share the workspace, replayed one after the other, with new inputs in between
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        swa.decode_paged_e4m3(*a, out=out, workspace=ws)
    with torch.cuda.graph(g2):
        swa.decode_paged_e4m3(*a, out=out2, workspace=ws)
    a[0].copy_(torch.flip(a[0], [0]))
    a[6].copy_(torch.tensor([333, 80], dtype=torch.int32))
    ws.fill_(0xFF)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    want = swa.decode_paged_e4m3(*a).view(torch.int16)
    # bit by bit: the second sequence's new window reaches rows that hold NaN
    assert torch.equal(out.view(torch.int16), want) and torch.equal(out2.view(torch.int16), want)
    assert bool(torch.isfinite(out[0].float()).all()) and bool(torch.isnan(out[1].float()).all())


def test_serving_run_append_then_decode(swa):
    """Prompts, then three decode steps, as a serving loop makes them: append_paged with the rotation,
    decode_paged_e4m3 on what it wrote, an empty slot in the batch.  Every step's result is held to the
    reference on the pages' own values, and the pages to the rotated keys and the values."""
    Hq, Hkv, d, W, S, page, rot = 6, 2, 64, 40, 8, 16, 64
    B, prompts = 3, [75, 0, 33]
    g = inp._gen(11)
    w = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    max_pages, num_pages = 6, 20
    table = torch.randperm(num_pages, generator=g)[:B * max_pages].to(torch.int32).view(B, max_pages)
    pages = [torch.full((num_pages, page, Hkv, d), 0x7f, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn) for _ in "kv"]
    exps = [torch.full((num_pages, Hkv, page), 255, dtype=torch.uint8).cuda() for _ in "kv"]
    keys, values = [[] for _ in range(B)], [[] for _ in range(B)]
    lens = np.zeros(B, np.int32)
    for step in range(4):
        new = prompts if step == 0 else [1, 0, 1]
        T = sum(new)
        qkv = inp.randn((T, (Hq + 2 * Hkv) * d), torch.bfloat16, g).cuda()
        q, k, v = (p.unflatten(-1, (h, d)) for p, h in zip(qkv.split([Hq * d, Hkv * d, Hkv * d], -1), (Hq, Hkv, Hkv)))
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        lens += np.array(new, np.int32)
        sl = torch.from_numpy(lens.copy()).cuda()
        qr = swa.append_paged(q, k, v, *pages, table.cuda(), sl, w.cuda(), starts=torch.from_numpy(starts).cuda(),
                              k_exp=exps[0], v_exp=exps[1])
        for b in range(B):
            at = slice(starts[b], starts[b + 1])
            pos = np.arange(lens[b] - new[b], lens[b])
            keys[b].append(ref.rotate(f64(k[at]), pos, w.numpy()))
            values[b].append(f64(v[at]))
        last = torch.from_numpy(np.maximum(starts[1:] - 1, 0)).cuda()
        qs = qr[last.long()].contiguous()
        gate = torch.tensor([step % 2, 1, 0], dtype=torch.uint8).cuda()
        o, lse = swa.decode_paged_e4m3(qs, *pages, *exps, table.cuda(), sl, gate, W, n_anchor=S, want_lse=True)
        assert swa.get_device_error() == 0
        c = Cache.__new__(Cache)
        c.B, c.Hq, c.Hkv, c.d, c.W, c.S, c.page = B, Hq, Hkv, d, W, S, page
        c.lens, c.gate, c.table, c.q = lens, gate.cpu().numpy(), table.numpy(), qs.cpu()
        c.codes = [p.view(torch.uint8).cpu().numpy() for p in pages]
        c.exps = [e.cpu().numpy() for e in exps]
        c.check(o, lse)
    for which, rows in enumerate((keys, values)):
        with np.errstate(invalid="ignore", over="ignore"):
            held = ref.contiguous(ref.page_values(c.codes[which], c.exps[which]), table.numpy())
        for b in (0, 2):
            want = np.concatenate(rows[b])
            got = held[b, :lens[b]]
            top = np.abs(want).max(-1, keepdims=True)
            # half an e4m3 step of the value, or of a subnormal one (scale <= 2 top / 448), and
            # the rotation's error
            assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * 2 * top / 448 + 2.0 ** -18 * top)


def test_refusals(swa):
    c = Cache([40], [1], 4, 2, 64, 10, 0, 16, seed=12)
    q, kp, vp, ke, ve, table, sl, gt, W = c.args()
    good = dict(q=q, k_pages=kp, v_pages=vp, k_exp=ke, v_exp=ve, block_table=table, seq_lens=sl, gate=gt, W=W)
    swa.decode_paged_e4m3(**good)
    bad = [
        dict(q=q.cpu()), dict(q=q.float()), dict(q=q[:, :3]), dict(k_pages=kp.view(torch.uint8)), dict(v_pages=vp[:2]),
        dict(k_exp=ke[:1]), dict(v_exp=ve.to(torch.int16)), dict(block_table=table.long()), dict(seq_lens=sl.long()),
        dict(gate=gt.bool()), dict(W=0), dict(n_anchor=-1), dict(scale=0.0), dict(scale=float("inf")),
        dict(block_table=table[:0]), dict(out=torch.zeros_like(q)[:, :2]),
        dict(q=torch.zeros((1, 34, 64), device="cuda", dtype=torch.bfloat16)),
    ]
    for change in bad:
        with pytest.raises((ValueError, swa.SwiAttnError)):
            swa.decode_paged_e4m3(**{**good, **change})
    assert swa.get_device_error() == 0


def test_wait_limit(swa):
    """With a tiny limit a wait for the cache's rows may run out: reported as SWIATTN_ETIMEOUT, the
    context stays usable, and with the default limit the next call is right again."""
    c = Cache([3000, 2500], [1, 1], 4, 2, 128, 64, 0, 16, seed=13)
    a = c.args()
    swa.set_wait_limit_ns(1)
    try:
        swa.decode_paged_e4m3(*a)
        assert swa.get_device_error() in (0, 4)
    finally:
        swa.set_wait_limit_ns(0)
    c.check(*run(swa, c))


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("page", [4, 16])
def test_scores_at_the_ends_of_fp32(swa, page, sign):
    """Scores of +-3.24e38 in base 2 (3.39e38 * 7.5 * 128^-1/2 log2(e)), all alike: weights of one
    each, so o is the value row that all keys share, without any rounding (40 equal terms of 4
    significant bits), and lse is the score in base e to within its fp32 steps (6 roundings)."""
    lens = [1, 40]
    c = Cache(lens, [1, 1], 2, 1, 128, 64, 0, page, 5)
    value = ref.e4m3_value(np.arange(0x30, 0x50, dtype=np.uint8))
    for which in range(2):
        c.codes[which][...] = 0
        c.exps[which][...] = 127
    c.codes[0][..., 7] = ref.e4m3_code(np.array(sign * 7.5))
    c.codes[1][...] = np.tile(np.arange(0x30, 0x50, dtype=np.uint8), 4)
    c.q.zero_()
    c.q[..., 7] = torch.finfo(torch.bfloat16).max
    o, lse = run(swa, c)
    assert np.array_equal(f64(o), np.broadcast_to(np.tile(value, 4), o.shape))
    want = sign * 7.5 * torch.finfo(torch.bfloat16).max / math.sqrt(128)
    assert np.all(np.abs(f64(lse) - want) <= 6 * 2.0 ** -24 * abs(want))
