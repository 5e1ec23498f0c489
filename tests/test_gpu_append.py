"""GPU parity of the paged append (swiattn_append_paged) against the 64-bit reference.

Tolerances as for the rotation (test_gpu_rope): rotated values in fp32 within 6 * 2^-24 (|a| + |b|),
half a bf16 step more where they are stored as bf16.  An e4m3 value is the nearest one to the fp32
value: half a step, 2^-4 of the value (2^-10 of the row's scale where it is subnormal), plus the
rotation's error.  What is not rotated (values, and keys with rot_dim 0) is exact, code by code.
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


def freqs(rot, base=10000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def raw(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


class Setup:
    """New tokens of B sequences (`new` counts, `total` lengths) and a pool with every byte set."""

    def __init__(self, new, total, Hq, Hkv, d, page, kind, seed, starts=True, pad=0, fused=False):
        self.B, self.page, self.Hkv, self.d, self.kind = len(new), page, Hkv, d, kind
        self.dtype = torch.float32 if kind == "f32" else torch.bfloat16
        g = inp._gen(seed)
        self.T = sum(new) + pad
        shape = (self.T, (Hq + 2 * Hkv) * d)
        x = inp.randn(shape, torch.float32, g)
        x *= torch.exp(torch.randn((self.T, 1), generator=g))   # rows of different size
        x = x.to(self.dtype).cuda()
        cut = [Hq * d, Hkv * d, Hkv * d]
        self.q, self.k, self.v = (p.unflatten(-1, (h, d)) for p, h in zip(x.split(cut, -1), (Hq, Hkv, Hkv)))
        if not fused:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.max_pages = max(1, -(-max(total) // page))
        held = self.B * self.max_pages
        self.num_pages = held + 3
        self.table = torch.randperm(self.num_pages, generator=g)[:held].to(torch.int32).view(self.B, -1).cuda()
        self.seq_lens = torch.tensor(total, dtype=torch.int32).cuda()
        self.starts = None
        if starts:
            self.starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        pool = (self.num_pages, page, Hkv, d)
        if kind == "e4m3":
            self.pages = [torch.randint(0, 256, pool, generator=g, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn)
                          for _ in "kv"]
            self.exps = [torch.randint(0, 255, (self.num_pages, Hkv, page), generator=g, dtype=torch.uint8).cuda()
                         for _ in "kv"]
        else:
            self.pages = [inp.randn(pool, self.dtype, g).cuda() for _ in "kv"]
            self.exps = [None, None]
        self.before = [raw(p) for p in self.pages], [None if e is None else raw(e) for e in self.exps]

    def run(self, swa, w, **more):
        args = dict(q=self.q, starts=self.starts)
        args.update(more)
        return swa.append_paged(args.pop("q"), self.k, self.v, *self.pages, self.table, self.seq_lens,
                                None if w is None else w.cuda(), k_exp=self.exps[0], v_exp=self.exps[1], **args)

    def check(self, q_out, w, interleaved=False, factor=1.0, q_before=None):
        starts = None if self.starts is None else self.starts.cpu().numpy()
        pos, row, bad = ref.places(starts, self.seq_lens.cpu().numpy(), self.table.cpu().numpy(), self.page,
                                   self.num_pages, self.T)
        on = row >= 0
        page, slot = row[on] // self.page, row[on] % self.page
        wn = np.zeros(0) if w is None else w.numpy()
        r = 2 * len(wn)

        def turned(x):
            x = f64(x)
            return (ref.rotate(x, pos, wn, interleaved, factor)[on],
                    6 * 2.0 ** -24 * abs(factor) * ref.pair_sums(x, wn, interleaved)[on])

        def half_step(want, tol, eps):   # of the rotated dimensions; the others are copies
            out = tol.copy()
            out[..., :r] += eps * (np.abs(want[..., :r]) + tol[..., :r])
            return out

        eps = 2.0 ** -8 if self.dtype == torch.bfloat16 else 0.0
        if q_out is not None:
            want, tol = turned(self.q)
            assert np.all(np.abs(f64(q_out)[on] - want) <= half_step(want, tol, eps))
            if q_before is not None:   # rows no sequence owns
                np.testing.assert_array_equal(raw(q_out)[~on], raw(q_before)[~on])
        for which, x in enumerate((self.k, self.v)):
            want, tol = turned(x) if which == 0 else (f64(x)[on], np.zeros((int(on.sum()), self.Hkv, self.d)))
            got, untouched = raw(self.pages[which]), np.ones((self.num_pages, self.page), bool)
            untouched[page, slot] = False
            before = self.before[0][which]
            np.testing.assert_array_equal(got[untouched], before[untouched])
            if self.kind != "e4m3":
                value = f64(self.pages[which])[page, slot]
                lim = half_step(want, tol, eps) if which == 0 else tol
                assert np.all(np.abs(value - want) <= lim)
                continue
            exps = raw(self.exps[which])
            un = np.ones(exps.shape, bool)
            un[page, :, slot] = False
            np.testing.assert_array_equal(exps[un], self.before[1][which][un])
            codes, u = got[page, slot], exps[page, :, slot]
            want_codes, want_u = ref.quantise(want)
            if which == 1 or r == 0:
                np.testing.assert_array_equal(codes, want_codes)
                np.testing.assert_array_equal(u, want_u)
                continue
            e = u.astype(np.int64) - 127
            top = np.abs(want).max(-1)
            # the smallest exponent, up to the rotation's error at a border
            assert np.all(top <= np.ldexp(448.0, e) * (1 + 2.0 ** -20))
            assert np.all((e == -126) | (top >= np.ldexp(448.0, e - 1) * (1 - 2.0 ** -20)))
            value = ref.e4m3_value(codes) * np.ldexp(1.0, e)[..., None]
            lim = tol + 2.0 ** -4 * (np.abs(want) + tol) + np.ldexp(2.0 ** -10, e)[..., None]
            assert np.all(np.abs(value - want) <= lim)
            # only a value at a border of two codes may differ from the 64-bit one
            assert np.mean(codes != want_codes) <= 1e-4 + 1.5 / codes.size
        return bad


KINDS = ["bf16", "e4m3", "f32"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,rot,interleaved", [
    ([1], [1], 1, 1, 64, 1, 64, False),
    ([1], [777], 16, 4, 128, 64, 128, False),
    ([5, 1, 0, 33], [5, 100, 7, 97], 3, 1, 64, 16, 16, True),      # chunks that begin and end inside pages
    ([130, 257], [130, 600], 4, 4, 128, 32, 96, False),
    ([1, 2, 3] * 15, [50, 2, 35] * 15, 5, 5, 64, 4, 32, True),     # more sequences than a warp
    ([40], [70000], 2, 2, 128, 256, 128, True),                    # far into a context
    ([21, 9], [70, 9], 24, 8, 128, 16, 80, False),                 # more heads than one block takes
    ([9, 4], [9, 4], 70, 3, 64, 8, 64, True),
])
def test_append_matches_reference(swa, new, total, Hq, Hkv, d, page, rot, interleaved, kind):
    s = Setup(new, total, Hq, Hkv, d, page, kind, seed=sum(new) + rot)
    w = freqs(rot)
    out = s.run(swa, w, interleaved=interleaved, factor=1.1)
    assert swa.get_device_error() == 0
    assert not s.check(out, w, interleaved, 1.1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [1, 16, 33, 1030])
def test_append_step_one_token_each(swa, B, kind):
    """starts None; some empty slots, whose q rows stay as they were."""
    total = [(b * 37) % 300 if b % 5 == 2 else 1 + (b * 61) % 300 for b in range(B)]
    if B > 2:
        total[2] = 0
    s = Setup([1] * B, total, 4, 2, 64, 8, kind, seed=B, starts=False, fused=True)
    before = torch.full((B, 4, 64), 7.0, dtype=s.dtype).cuda()
    out = before.clone()
    assert s.run(swa, freqs(64), out=out) is out
    assert swa.get_device_error() == 0
    assert not s.check(out, freqs(64), q_before=before)


@pytest.mark.parametrize("kind", KINDS)
def test_append_without_rotation_is_exact_and_without_q(swa, kind):
    s = Setup([17, 40], [30, 40], 2, 2, 128, 16, kind, seed=3)
    assert s.run(swa, None, q=None) is None
    assert not s.check(None, None)
    s2 = Setup([17, 40], [30, 40], 2, 2, 128, 16, kind, seed=3)
    q = s2.run(swa, None)
    assert torch.equal(q, s2.q) and torch.equal(s2.pages[0].view(torch.uint8), s.pages[0].view(torch.uint8))


def test_append_padding_rows_are_left_alone(swa):
    """Tokens behind the last sequence, and before the first."""
    s = Setup([3, 4], [3, 10], 2, 1, 64, 4, "e4m3", seed=4, pad=9)
    s.starts += 2   # two rows before the first sequence
    before = torch.full((s.T, 2, 64), 3.0, dtype=s.dtype).cuda()
    out = before.clone()
    s.run(swa, freqs(64), out=out)
    assert swa.get_device_error() == 0
    assert not s.check(out, freqs(64), q_before=before)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_bad_input_is_passed_over_and_reported(swa, kind):
    """A table entry outside the pool, a length shorter than the new tokens, one past the table, a
    negative one: reported, the tokens concerned passed over, the others stored."""
    for spoil in ("page high", "page low", "short", "long", "negative"):
        s = Setup([6, 6, 6], [20, 20, 20], 2, 1, 64, 8, kind, seed=5)
        before = torch.full((18, 2, 64), 3.0, dtype=s.dtype).cuda()
        if spoil == "page high":
            s.table[1, 2] = s.num_pages
        elif spoil == "page low":
            s.table[1, 2] = -1
        else:
            s.seq_lens[1] = {"short": 4, "long": 27, "negative": -5}[spoil]
        out = before.clone()
        s.run(swa, freqs(64), out=out)
        assert swa.get_device_error() == 1 and swa.get_device_error() == 0
        assert s.check(out, freqs(64), q_before=before)


def test_append_starts_out_of_order_stay_inside(swa):
    """starts that the documentation does not allow: whatever is stored stays inside the pool and the
    call's other tensors (rows beside the pool hold their bytes)."""
    s = Setup([4] * 40, [30] * 40, 2, 1, 64, 8, "bf16", seed=6)
    g = inp._gen(7)
    s.starts = torch.randint(-50, 300, (41,), generator=g, dtype=torch.int32).cuda()
    backing = torch.full((s.num_pages + 2, 8, 1, 64), 5.0, dtype=torch.bfloat16).cuda()
    s.pages = [backing[1:-1], s.pages[1]]
    s.run(swa, freqs(64))
    swa.get_device_error()
    assert bool((backing[0] == 5).all()) and bool((backing[-1] == 5).all())


def test_append_special_values(swa):
    """Zero rows, infinities, NaN and tiny rows in e4m3 pages, code by code (no rotation)."""
    s = Setup([6], [6], 1, 1, 64, 8, "e4m3", seed=8)
    for x in (s.k, s.v):
        x[0] = 0
        x[1, 0, 5] = float("inf")
        x[2, 0, 6] = float("-inf")
        x[3, 0, 7] = float("nan")
        x[4] *= 1e-37
        x[5] = 0
        x[5, 0, 9] = -3.3895e38   # the largest bf16
    s.run(swa, None)
    s.check(None, None)
    top = ref.page_values(raw(s.pages[0]), raw(s.exps[0]))[s.table[0, 0].item(), :6, 0]
    with np.errstate(over="ignore"):
        as_f32 = top.astype(np.float32)
    assert np.isposinf(as_f32[1, 5]) and np.isneginf(as_f32[2, 6]) and np.isnan(top[3, 7])


def test_append_on_a_side_stream_and_in_a_graph(swa):
    """Captured once, replayed with other inputs in the same tensors."""
    s = Setup([3, 1], [9, 30], 2, 2, 64, 8, "e4m3", seed=9)
    w = freqs(64).cuda()
    out = torch.zeros_like(s.q)

    def call():
        return swa.append_paged(s.q, s.k, s.v, *s.pages, s.table, s.seq_lens, w, starts=s.starts,
                                k_exp=s.exps[0], v_exp=s.exps[1], out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    s.check(out, freqs(64))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    s2 = Setup([3, 1], [9, 30], 2, 2, 64, 8, "e4m3", seed=10)
    for a, b in zip([s.q, s.k, s.v, s.table, s.seq_lens] + s.pages + s.exps,
                    [s2.q, s2.k, s2.v, s2.table, s2.seq_lens] + s2.pages + s2.exps):
        a.view(torch.uint8).copy_(b.view(torch.uint8)) if a.element_size() == 1 else a.copy_(b)
    s.before = s2.before
    graph.replay()
    torch.cuda.synchronize()
    s.check(out, freqs(64))


def test_append_refusals(swa):
    s = Setup([4], [9], 2, 1, 64, 8, "e4m3", seed=11)
    w = freqs(64).cuda()
    good = dict(q=s.q, k=s.k, v=s.v, k_pages=s.pages[0], v_pages=s.pages[1], block_table=s.table,
                seq_lens=s.seq_lens, inv_freq=w, starts=s.starts, k_exp=s.exps[0], v_exp=s.exps[1])
    swa.append_paged(**good)
    pages = torch.zeros((6, 8, 1, 64), device="cuda", dtype=torch.bfloat16)
    odd = torch.zeros((6, 6, 1, 64), device="cuda", dtype=torch.bfloat16)
    bad = [
        dict(k=s.k.cpu()), dict(k=s.k[:3]), dict(v=s.v.float()), dict(q=s.q[:, :, :32]), dict(k_exp=None),
        dict(v_exp=s.exps[1].transpose(1, 2)), dict(k_exp=s.exps[0].to(torch.int32)), dict(k_pages=pages),
        dict(k_pages=pages.float(), v_pages=pages.float()), dict(block_table=s.table.long()),
        dict(block_table=s.table[0]), dict(seq_lens=s.seq_lens.long()), dict(starts=s.starts[:1]),
        dict(starts=None), dict(inv_freq=freqs(24).cuda()), dict(inv_freq=w.float()), dict(factor=float("inf")),
        dict(out=torch.zeros_like(s.q)[:3]), dict(q=None, out=torch.zeros_like(s.q)),
        dict(k_pages=odd, v_pages=odd), dict(q=s.q.float(), k=s.k.float(), v=s.v.float()),
    ]
    for change in bad:
        with pytest.raises((ValueError, swa.SwiAttnError)):
            swa.append_paged(**{**good, **change})
    assert swa.get_device_error() == 0
    empty = swa.append_paged(s.q[:0], s.k[:0], s.v[:0], *s.pages, s.table, s.seq_lens, w,
                             starts=torch.zeros_like(s.starts), k_exp=s.exps[0], v_exp=s.exps[1])
    assert empty.shape == (0, 2, 64)


def test_append_past_32_bit_offsets(swa):
    """A pool of over 2^32 values: its last pages."""
    Hkv, d, page = 8, 128, 64
    num_pages = (1 << 32) // (page * Hkv * d) + 3
    s = Setup([90], [90], Hkv, Hkv, d, page, "e4m3", seed=12)   # decode wants Hq a multiple of Hkv
    pages = [torch.empty((num_pages, page, Hkv, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in "kv"]
    exps = [torch.empty((num_pages, Hkv, page), dtype=torch.uint8, device="cuda") for _ in "kv"]
    s.run(swa, freqs(128))
    small = s.table.long()[0]
    big = torch.tensor([num_pages - 1, num_pages - 2], device="cuda")
    table = big.to(torch.int32)[None].contiguous()
    q = swa.append_paged(s.q, s.k, s.v, *pages, table, s.seq_lens, freqs(128).cuda(), starts=s.starts, k_exp=exps[0],
                         v_exp=exps[1])
    assert swa.get_device_error() == 0
    for which in (0, 1):
        got = pages[which][big].view(torch.uint8).flatten(0, 1)[:90]
        want = s.pages[which][small].view(torch.uint8).flatten(0, 1)[:90]
        assert torch.equal(got, want)
    gate, W = torch.ones(1, dtype=torch.uint8, device="cuda"), 5
    last = q[-1:].contiguous()
    o = swa.decode_paged_e4m3(last, *pages, *exps, table, s.seq_lens, gate, W)
    want = swa.decode_paged_e4m3(last, *s.pages, *s.exps, s.table, s.seq_lens, gate, W)
    assert swa.get_device_error() == 0 and torch.equal(o, want)
