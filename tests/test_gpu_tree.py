"""GPU parity of the tree attention (swiattn_decode_tree) against the 64-bit reference.

Tolerances.  A score is a sum of d products in fp32, off by at most (d + 4) 2^-24 of
scale sum |q_c k_c| (and 2^-22 of itself in base 2, which that covers 16 times over): ds.  A weight is
off by 2 ds and 2^-16 (the bf16 products take it as two bf16, off by 2^-17; exponential and sums in
fp32 are far nearer), and the sum over n entries by n 2^-23: so o is within
(2 ds + 2^-16 + n 2^-23) sum p |v|, plus half a step of its type, and lse within
ds + (n + 8) 2^-23 and 2^-22 of itself.
"""
import numpy as np
import pytest
import torch

import swiattn_inputs as inp
from oracle import kvcache as ref
from test_gpu_append import f64, raw, swa  # noqa: F401  (swa: the fixture)

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "f32"]


def random_parents(rng, n, deep=0.7):
    """Each token continues the one before it, or any earlier one, or the cache."""
    return [-1 if i == 0 else i - 1 if rng.random() < deep else int(rng.integers(-1, i)) for i in range(n)]


class Case:
    """Sequences of ns drafted tokens after bases cached ones, in scattered pages; every byte of the pool
    that no sequence holds is NaN (in the type's own terms)."""

    def __init__(self, ns, bases, Hq, Hkv, d, page, kind, W, S=0, routed=0.3, seed=0, deep=0.7, pad=0, scale=None):
        rng, g = np.random.default_rng(seed), inp._gen(seed)
        self.kind, self.W, self.S, self.d = kind, W, S, d
        self.scale = scale if scale is not None else d ** -0.5
        self.dtype = torch.float32 if kind == "f32" else torch.bfloat16
        B = len(ns)
        self.lens = np.array([0 if n < 0 else n + b for n, b in zip(ns, bases)])   # n < 0: an empty slot
        ns = [abs(n) for n in ns]
        self.starts = np.concatenate([[0], np.cumsum(ns)])
        self.T = int(self.starts[-1]) + pad
        self.parents = np.array([p for n in ns for p in random_parents(rng, n, deep)] + [-1] * pad)
        self.gate = (rng.random(self.T) < routed).astype(np.uint8)
        max_pages = max(1, -(-int(self.lens.max()) // page)) + 1
        num_pages = B * max_pages + 1
        self.table = rng.permutation(num_pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        shape = (num_pages, page, Hkv, d)
        held = np.zeros((num_pages, page), bool)
        for b in range(B):
            for j in range(int(self.lens[b])):
                held[self.table[b, j // page], j % page] = True
        mask = torch.from_numpy(held)[..., None, None]
        self.pages, self.exps, self.values = [], [None, None], []
        for i in range(2):
            x = inp.randn(shape, torch.float32, g) * torch.exp(0.5 * torch.randn((num_pages, page, Hkv, 1), generator=g))
            if kind == "e4m3":
                codes, e = ref.quantise(x.double().numpy())
                codes[~held] = 0x7f
                self.pages.append(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn))
                self.exps[i] = torch.from_numpy(np.ascontiguousarray(np.swapaxes(e, 1, 2))).cuda()
                self.values.append(ref.page_values(codes, raw(self.exps[i])))
            else:
                x = torch.where(mask, x, torch.nan).to(self.dtype)
                self.pages.append(x.cuda())
                self.values.append(f64(x))
        self.q = inp.randn((self.T, Hq, d), self.dtype, g).cuda()

    def tensors(self):
        return (torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                torch.tensor(self.starts, dtype=torch.int32).cuda(), torch.tensor(self.parents, dtype=torch.int32).cuda(),
                torch.from_numpy(self.gate).cuda())

    def run(self, swa, chains=False, **more):
        table, lens, starts, parents, gate = self.tensors()
        return swa.decode_tree(self.q, *self.pages, table, lens, starts, None if chains else parents, gate, self.W,
                               scale=self.scale, n_anchor=self.S, k_exp=self.exps[0], v_exp=self.exps[1],
                               want_lse=True, **more)

    def reference(self):
        k, v = (ref.contiguous(x, self.table) for x in self.values)
        return ref.decode_tree(f64(self.q), k, v, self.lens, self.starts, self.parents, self.gate, self.W, self.S, self.scale)

    def check(self, got, want=None):
        o, lse = f64(got[0]), f64(got[1])
        want_o, want_lse, absum, size, count = want or self.reference()
        on = ~np.isnan(want_lse[:, 0])
        ds = (self.d + 4) * 2.0 ** -24 * size
        n = count[:, None]
        eps = 2.0 ** -24 if self.kind == "f32" else 2.0 ** -8
        lim = (2 * ds + 2.0 ** -16 + n * 2.0 ** -23)[..., None] * absum
        lim += eps * (np.abs(want_o) + lim)
        err = np.abs(o - want_o)
        assert np.all(err[on] <= lim[on]), np.max((err / lim)[on])
        err, lim = np.abs(lse - want_lse), ds + (n + 8) * 2.0 ** -23 + 2.0 ** -22 * np.abs(want_lse)
        assert np.all(err[on] <= lim[on]), np.max((err / lim)[on])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ns,bases,Hq,Hkv,d,page,W,S", [
    ([1], [0], 1, 1, 64, 1, 1, 0),
    ([1], [0], 1, 1, 128, 16, 5, 0),
    ([8], [769], 4, 2, 128, 16, 256, 0),
    ([3, 17, 1], [127, 128, 129], 2, 2, 64, 32, 64, 0),
    ([5, 0, 33, -4, 2], [11, 7, 300, 9, 0], 6, 2, 64, 8, 100, 37),      # no drafts, an empty slot, no cache
    ([256, 40], [200, 1000], 3, 1, 64, 64, 128, 130),
    ([61], [513], 8, 1, 128, 128, 3, 2),                                  # a window smaller than the tree is deep
    ([9, 30], [400, 260], 16, 1, 128, 2, 4096, 0),
    ([2] * 40, list(range(40)), 2, 1, 64, 4, 8, 3),                       # more sequences than a warp
    ([100], [100], 5, 5, 64, 256, 20, 150),                               # anchors that reach into the tree
    ([64], [640], 128, 1, 64, 16, 200, 0),                                # the most heads to a key head
    ([40, 25], [1500, 900], 4, 2, 128, 64, 300, 500),                     # anchors that meet the window
])
def test_tree_matches_reference(swa, ns, bases, Hq, Hkv, d, page, W, S, kind):
    c = Case(ns, bases, Hq, Hkv, d, page, kind, W, S, seed=sum(ns) + W)
    got = c.run(swa)
    assert swa.get_device_error() == 0
    c.check(got)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("routed", [0.0, 1.0])
def test_tree_gates_all_one_way(swa, routed, kind):
    c = Case([70, 31], [900, 333], 4, 2, 128, 16, kind, 150, 20, routed=routed, seed=3)
    c.check(c.run(swa))


@pytest.mark.parametrize("kind", KINDS)
def test_tree_chains(swa, kind):
    """Without parents each token continues the one before: as with those parents, bit for bit."""
    c = Case([33, 7], [100, 5], 4, 4, 64, 16, kind, 24, seed=4, deep=1.1)
    a, b = c.run(swa), c.run(swa, chains=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(a)


@pytest.mark.parametrize("kind", KINDS)
def test_tree_padding_rows_are_left_alone(swa, kind):
    c = Case([5, 9, -3, 4], [60, 20, 7, 3], 4, 2, 64, 16, kind, 30, seed=5, pad=6)
    c.starts, c.parents = c.starts + 2, np.roll(c.parents, 2)   # two rows before the first sequence
    out = torch.full_like(c.q, 3.0)
    got = c.run(swa, out=out)
    assert got[0] is out and swa.get_device_error() == 0
    c.check(got)
    rows = np.ones(c.T, bool)
    for b in range(4):
        if c.lens[b]:
            rows[c.starts[b]:c.starts[b + 1]] = False
    assert rows.sum() == 9 and bool((out[torch.from_numpy(rows).cuda()] == 3).all())


@pytest.mark.parametrize("kind", KINDS)
def test_tree_masked_nan_and_infinity_stay_out(swa, kind):
    """Values that some tokens of a sequence read and others do not: NaN and infinities reach the ones
    that do, and no other; keys likewise."""
    c = Case([40, 12], [700, 300], 4, 2, 128, 16, kind, 100, routed=0.25, seed=6)
    clean = c.run(swa)
    poison = [(0, 0, 50, np.nan), (1, 0, 120, np.nan), (1, 0, 700 + 11, np.inf), (0, 0, 700 + 20, np.nan), (1, 1, 100, -np.inf)]
    for which, b, j, x in poison:
        p, s = c.table[b, j // 16], j % 16
        if kind == "e4m3":
            c.pages[which].view(torch.uint8)[p, s, 1, 3] = 0x7f
        else:
            c.pages[which][p, s, 1, 3] = x
    got = c.run(swa)
    reads = np.zeros((c.T, 2), bool)   # by key head
    for which, b, j, x in poison:
        first, n = int(c.starts[b]), int(c.starts[b + 1] - c.starts[b])
        seen = ref.tree_visible(c.parents[first:first + n], c.gate[first:first + n], int(c.lens[b]) - n, c.W, c.S)
        reads[first:first + n, 1] |= seen[:, j]
    o = f64(got[0])
    touched = np.repeat(reads, 2, axis=1)
    assert np.array_equal(~np.isfinite(o).all(-1), touched)
    assert 0 < touched.sum() < touched.size / 2
    # the others: the very same parts
    np.testing.assert_allclose(o[~touched], f64(clean[0])[~touched], rtol=2.0 ** -6, atol=2.0 ** -12)
    c.values = [ref.page_values(raw(p), raw(e)) if kind == "e4m3" else f64(p) for p, e in zip(c.pages, c.exps)]
    with np.errstate(invalid="ignore"):
        want = c.reference()
    keep = ~np.repeat(reads, 2, axis=1)
    err = np.abs(o[keep] - want[0][keep])
    lim = ((2 * (c.d + 4) * 2.0 ** -24 * want[3] + 2.0 ** -16 + want[4][:, None] * 2.0 ** -23)[..., None] * want[2])[keep]
    lim += (2.0 ** -24 if kind == "f32" else 2.0 ** -8) * (np.abs(want[0][keep]) + lim)
    assert np.all(err <= lim)


@pytest.mark.parametrize("kind", KINDS)
def test_tree_scores_far_apart(swa, kind):
    """Scores over a range of thousands: one entry takes all of a row's weight, whatever part it is in."""
    c = Case([20], [1000], 2, 1, 64, 16, kind, 400, routed=0.5, seed=7, scale=40.0)
    c.check(c.run(swa))


@pytest.mark.parametrize("kind", KINDS)
def test_tree_large_and_small_values(swa, kind):
    """Value rows from 2^-60 to 2^60 of their size, beside one another."""
    c = Case([16], [300], 2, 1, 128, 16, kind, 100, routed=0.5, seed=8)
    g = inp._gen(8)
    up = torch.randint(-60, 61, c.pages[1].shape[:3], generator=g)
    if kind == "e4m3":
        e = (c.exps[1].cpu().to(torch.int64) + up.transpose(1, 2)).clamp(1, 254).to(torch.uint8)
        c.exps[1] = e.cuda()
        c.values[1] = ref.page_values(raw(c.pages[1]), raw(e))
    else:
        c.pages[1] = torch.ldexp(c.pages[1].double(), up[..., None].cuda().double()).to(c.dtype)
        c.values[1] = f64(c.pages[1])
    c.check(c.run(swa))


def test_tree_agrees_with_decode(swa):
    """One drafted token of each sequence is a decode step."""
    c = Case([1] * 5, [0, 100, 255, 600, 31], 4, 2, 128, 16, "bf16", 64, 16, seed=9)
    o, lse = c.run(swa)
    table, lens, _, _, gate = c.tensors()
    pages = [torch.where(p.isnan(), 0, p) for p in c.pages]   # decode_paged clamps into pages it reads whole
    o2, lse2 = swa.decode_paged(c.q, *pages, table, lens, gate, c.W, n_anchor=c.S, want_lse=True)
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -6 and (lse - lse2).abs().max() < 1e-4


def test_tree_bad_input_is_passed_over_and_reported(swa):
    for spoil in ("short", "long", "negative", "large", "starts", "behind", "before", "parent", "page high", "page low"):
        c = Case([6, 20, 9], [50, 30, 40], 2, 1, 64, 16, "bf16", 32, seed=10)
        if spoil == "large":
            c = Case([6, 257, 9], [50, 30, 40], 2, 1, 64, 16, "bf16", 32, seed=10)
        want = None if spoil == "large" else c.reference()
        bad = [1]
        if spoil in ("short", "long", "negative"):
            c.lens[1] = {"short": 19, "long": c.table.shape[1] * 16 + 1, "negative": -1}[spoil]
        elif spoil in ("starts", "behind", "before"):
            c.starts = np.array({"starts": [0, 26, 20, 35], "behind": [0, 6, 26, 36], "before": [-1, 6, 26, 35]}[spoil])
            bad = [0, 1, 2]
        elif spoil == "parent":
            c.parents[6 + 7] = 7
            want, bad = c.reference(), []
        elif spoil.startswith("page"):
            c.pages[0][0] = 1.0   # page 0 is read in the bad one's place
            c.pages[1][0] = 2.0
            c.table[1, 1] = 0
            for i in range(2):
                c.values[i] = f64(c.pages[i])
            want, bad = c.reference(), []
            c.table[1, 1] = c.pages[0].shape[0] if spoil == "page high" else -1
        out = torch.full_like(c.q, 3.0)
        starts = c.starts
        got = c.run(swa, out=out)
        assert swa.get_device_error() == 1 and swa.get_device_error() == 0, spoil
        if len(bad) == 3:
            assert bool((out == 3).all())
            continue
        if spoil == "large":
            assert bool((out[6:263] == 3).all()) and bool((out[:6] != 3).any()) and bool((out[263:] != 3).any())
            continue
        for b in bad:
            want[1][starts[b]:starts[b + 1]] = np.nan
            assert bool((out[int(starts[b]):int(starts[b + 1])] == 3).all())
        c.check(got, want)


def test_tree_offsets_past_32_bits(swa):
    """A pool of more than 2^32 bytes and elements, the sequence's pages at its end."""
    page, Hkv, d = 64, 16, 128
    num_pages = (1 << 32) // (page * Hkv * d) + 40
    k = torch.empty((num_pages, page, Hkv, d), device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    c = Case([9], [600], 16, 16, d, page, "bf16", 100, seed=11)
    shift = num_pages - c.pages[0].shape[0]
    k[shift:], v[shift:] = c.pages[0], c.pages[1]
    table, lens, starts, parents, gate = c.tensors()
    got = swa.decode_tree(c.q, k, v, table + shift, lens, starts, parents, gate, c.W, want_lse=True)
    want = c.run(swa)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", KINDS)
def test_tree_is_repeatable_in_graphs_and_on_two_streams(swa, kind):
    """Captured once and replayed with other inputs in the same tensors; two calls at once, each with a
    workspace of its own."""
    c = Case([30, 12], [1500, 700], 8, 2, 128, 16, kind, 256, 30, seed=12)
    c2 = Case([12, 30], [1000, 1200], 8, 2, 128, 16, kind, 100, seed=13)
    want, want2 = c.run(swa), c2.run(swa)
    c.check(want)
    again = c.run(swa)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(5):
        for i, x in enumerate((c, c2)):
            with torch.cuda.stream(streams[i]):
                results[i].append(x.run(swa))
    torch.cuda.synchronize()
    for got, w in zip(results, (want, want2)):
        assert all(torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]) for g in got)
    table, lens, starts, parents, gate = c.tensors()
    out = torch.empty_like(c.q)
    ws = torch.empty(swa.decode_tree_workspace(c.T, 2, 8, 2, 128, c.dtype), dtype=torch.uint8, device="cuda")

    def call():
        swa.decode_tree(c.q, *c.pages, table, lens, starts, parents, gate, c.W, scale=c.scale, n_anchor=c.S, k_exp=c.exps[0],
                        v_exp=c.exps[1], out=out, workspace=ws)

    with torch.cuda.stream(streams[0]):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            call()
    c.gate = 1 - c.gate
    c.lens = np.array([1400, 712])
    gate.copy_(torch.from_numpy(c.gate))
    lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = c.run(swa)
    assert torch.equal(got[0], out)
    c.check(got)


def test_speculative_step_end_to_end(swa):
    """Two steps as they would be used: drafted trees appended at their positions (fork of one prompt
    first), verified, the accepted path kept; then the next trees after it.  Against the reference on the
    cache as it should be, for every type of pages."""
    Hq, Hkv, d, page, W = 4, 2, 64, 16, 40
    w = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    for kind in KINDS:
        g, rng = inp._gen(21), np.random.default_rng(21)
        dtype = torch.float32 if kind == "f32" else torch.bfloat16
        prompt, C, max_pages = 75, 3, 12
        num_pages = 5 + C * 8
        pages = [torch.zeros((num_pages, page, Hkv, d), device="cuda",
                             dtype=torch.float8_e4m3fn if kind == "e4m3" else dtype) for _ in "kv"]
        exps = [torch.ones((num_pages, Hkv, page), dtype=torch.uint8, device="cuda") if kind == "e4m3" else None for _ in "kv"]
        e = dict(k_exp=exps[0], v_exp=exps[1])
        # the prompt, then three children of it; the pages that each will need stand in its table
        one = torch.zeros((1, max_pages), dtype=torch.int32)
        one[0, :5] = torch.arange(5)
        k0, v0 = (inp.randn((prompt, Hkv, d), dtype, g).cuda() for _ in "kv")
        lens = torch.tensor([prompt], dtype=torch.int32).cuda()
        swa.append_paged(None, k0, v0, *pages, one.cuda(), lens, w.cuda(),
                         starts=torch.tensor([0, prompt], dtype=torch.int32).cuda(), **e)
        new = torch.arange(5, 5 + C, dtype=torch.int32).cuda()
        table, lens = swa.fork_paged(*pages, one.cuda(), lens, torch.zeros(C, dtype=torch.int32).cuda(), new, **e)
        table[:, 5:] = torch.arange(5 + C, 5 + C + C * 7, dtype=torch.int32).cuda().view(C, 7)
        truth = [[(k0, v0)] for _ in range(C)]   # rows of each child's cache, as given, in order
        for step in range(2):
            ns = [9, 1, 24]
            parents = [random_parents(rng, n, 0.5) for n in ns]
            starts = np.concatenate([[0], np.cumsum(ns)])
            T = int(starts[-1])
            q, k, v = inp.randn((T, Hq, d), dtype, g).cuda(), *(inp.randn((T, Hkv, d), dtype, g).cuda() for _ in "kv")
            gate = torch.randint(0, 2, (T,), generator=g, dtype=torch.uint8)
            base = lens.tolist()
            depth = [len(ref.tree_path(parents[b], t)) - 1 for b in range(C) for t in range(ns[b])]
            pos = np.repeat(base, ns) + np.array(depth)
            lens = lens + torch.tensor(ns, dtype=torch.int32).cuda()
            t_starts, t_parents = (torch.tensor(np.asarray(x), dtype=torch.int32).cuda() for x in (starts, sum(parents, [])))
            qr = swa.append_paged(q, k, v, *pages, table, lens, w.cuda(), starts=t_starts,
                                  positions=torch.tensor(pos, dtype=torch.int32).cuda(), **e)
            o, lse = swa.decode_tree(qr, *pages, table, lens, t_starts, t_parents, gate.cuda(), W, want_lse=True, **e)
            # the reference reads the pages through its own bookkeeping
            values = [ref.page_values(raw(p), raw(x)) if kind == "e4m3" else f64(p) for p, x in zip(pages, exps)]
            c = Case.__new__(Case)
            c.kind, c.W, c.S, c.d, c.scale, c.q = kind, W, 0, d, d ** -0.5, qr
            c.table, c.values, c.lens, c.starts = table.cpu().numpy(), values, lens.cpu().numpy(), starts
            c.parents, c.gate = np.array(sum(parents, [])), gate.numpy()
            c.check((o, lse))
            leaf = [int(rng.integers(-1, n)) for n in ns]
            lens = swa.accept_tree(*pages, table, lens, t_starts, t_parents, torch.tensor(leaf, dtype=torch.int32).cuda(), **e)
            for b in range(C):
                path = ref.tree_path(parents[b], leaf[b]) if leaf[b] >= 0 else []
                truth[b].append((k[starts[b] + np.array(path, int)], v[starts[b] + np.array(path, int)]))
                assert lens[b].item() == base[b] + len(path) == sum(len(x[0]) for x in truth[b])
        assert swa.get_device_error() == 0
        # every cache row is the token that was accepted there, rotated by its place
        for b in range(C):
            kk, vv = (torch.cat([x[i] for x in truth[b]]) for i in range(2))
            # within the rotation's 6 * 2^-24 (|a| + |b|), half a step of the pages' type (e4m3: at least
            # 2^-10 of the row's power of two, which is under 2^-7 of its largest value)
            turned = 6 * 2.0 ** -24 * ref.pair_sums(f64(kk), w.numpy())
            kk = ref.rotate(f64(kk), np.arange(len(kk)), w.numpy())
            for p, x, want, off in zip(pages, exps, (kk, f64(vv)), (turned, 0.0)):
                got = ref.page_values(raw(p), raw(x)) if kind == "e4m3" else f64(p)
                got = ref.contiguous(got, table.cpu().numpy())[b, :len(want)]
                half = {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}[kind] * (np.abs(want) + off)
                if kind == "e4m3":
                    half += 2.0 ** -17 * np.abs(want).max(-1, keepdims=True)
                assert np.all(np.abs(got - want) <= off + half)


def test_tree_binding_refusals(swa):
    c = Case([3], [9], 2, 1, 64, 8, "bf16", 4, seed=14)
    table, lens, starts, parents, gate = c.tensors()
    good = dict(q=c.q, k_pages=c.pages[0], v_pages=c.pages[1], block_table=table, seq_lens=lens, starts=starts,
                parents=parents, gate=gate, W=4)
    for bad in (dict(q=c.q[None]), dict(q=c.q.half()), dict(q=c.q.transpose(0, 1)), dict(k_pages=c.pages[0][None]),
                dict(v_pages=c.pages[1].float()), dict(block_table=table[0]), dict(seq_lens=lens.long()), dict(starts=starts[:1]),
                dict(parents=parents[:2]), dict(gate=gate[:2]), dict(gate=gate.bool()), dict(out=c.q[:2]),
                dict(workspace=c.q), dict(q=c.q.cpu()),
                dict(k_pages=c.pages[0].to(torch.float8_e4m3fn), v_pages=c.pages[1].to(torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            swa.decode_tree(**{**good, **bad})
    for bad in (dict(W=0), dict(n_anchor=-1), dict(scale=0.0), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                dict(q=c.q.float())):
        with pytest.raises(swa.SwiAttnError):
            swa.decode_tree(**{**good, **bad})
    empty = dict(good, q=c.q[:0], parents=parents[:0], gate=gate[:0], starts=torch.zeros_like(starts))
    assert swa.decode_tree(**empty).shape == (0, 2, 64)
