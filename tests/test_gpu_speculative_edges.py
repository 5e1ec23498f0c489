"""The calls of a speculative step at the ends of what they allow: padded batches of fixed shape in one
captured graph, the largest window and anchors, trees with the most rows, batches of many slots or of
none with work.  References and tolerances as in test_gpu_tree and test_gpu_paging."""
import numpy as np
import pytest
import torch

import swiattn_inputs as inp
from test_gpu_append import swa  # noqa: F401  (the fixture)
from test_gpu_paging import accept_setup, flat_parents, ints
from test_gpu_tree import KINDS, Case

pytestmark = pytest.mark.gpu


def test_padded_step_in_a_graph(swa):
    """Append at positions, tree attention and accepted path, captured together over four slots of six
    drafts each, replayed with slots 1 and 3, then 0 and 1, then none in use: what the slots in use get is
    what they get alone, the others' pages and rows stay, and nothing is reported."""
    S, n, Hq, Hkv, d, page, max_pages, W = 4, 6, 4, 2, 64, 8, 6, 11
    g = inp._gen(31)
    num_pages = S * max_pages
    pages0 = [torch.randn((num_pages, page, Hkv, d), generator=g).bfloat16().cuda() for _ in "kv"]
    table = torch.randperm(num_pages, generator=g).view(S, max_pages).int().cuda()
    q, k, v = (inp.randn((S * n, h, d), torch.bfloat16, g).cuda() for h in (Hq, Hkv, Hkv))
    w = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    starts = ints(np.arange(S + 1) * n)
    tree = [-1, 0, 0, 1, 2, 4]
    parents, depth = ints(tree * S), np.array([0, 1, 1, 2, 2, 3])
    gate = torch.randint(0, 2, (S * n,), generator=g, dtype=torch.uint8).cuda()
    lens, positions, leaf = ints([0] * S), ints([0] * (S * n)), ints([5] * S)
    pages = [p.clone() for p in pages0]
    ws = torch.empty(swa.decode_tree_workspace(S * n, S, Hq, Hkv, d, torch.bfloat16), dtype=torch.uint8, device="cuda")
    qr, o, kept = torch.empty_like(q), torch.empty_like(q), torch.empty_like(lens)

    def step():
        swa.append_paged(q, k, v, *pages, table, lens, w, starts=starts, positions=positions, out=qr)
        swa.decode_tree(qr, *pages, table, lens, starts, parents, gate, W, n_anchor=3, out=o, workspace=ws)
        swa.accept_tree(*pages, table, lens, starts, parents, leaf, out=kept)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    side.synchronize()
    for used in ({1: 20, 3: 33}, {0: 6, 1: 41}, {}):
        now = np.array([used.get(b, 0) for b in range(S)])
        lens.copy_(ints(now))
        positions.copy_(ints(np.repeat(now - n, n) + np.tile(depth, S)))
        for p, p0 in zip(pages, pages0):
            p.copy_(p0)
        o.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert swa.get_device_error() == 0
        assert kept.tolist() == [x - n + 4 if x else 0 for x in now]
        alone = [p.clone() for p in pages0]
        for b in range(S):
            rows = slice(b * n, (b + 1) * n)
            if not now[b]:
                assert bool((o[rows] == 5).all())
                continue
            one = (table[b:b + 1].contiguous(), lens[b:b + 1].clone())
            s1, p1 = ints([0, n]), ints(tree)
            a = swa.append_paged(q[rows], k[rows], v[rows], *alone, *one, w, starts=s1, positions=positions[rows].clone())
            want = swa.decode_tree(a, *alone, *one, s1, p1, gate[rows].clone(), W, n_anchor=3)
            swa.accept_tree(*alone, *one, s1, p1, ints([5]))
            # how the keys are split depends on the batch: a part's sums in another order, 2^-16 of the
            # values' size (those of the weights), and a rounding to bf16 on either side
            size = max(float(p.abs().max()) for p in alone)
            err = (o[rows].double() - want.double()).abs()
            assert bool((err <= 2 * (2.0 ** -16 * size + 2.0 ** -8 * want.double().abs())).all())
        assert all(torch.equal(x, y) for x, y in zip(pages, alone))


@pytest.mark.parametrize("kind", KINDS)
def test_largest_window_and_anchors(swa, kind):
    """Either is the whole history, as is a set gate; no sum with them wraps."""
    most = 2 ** 31 - 1
    cases = [Case([12, 3], [500, 0], 4, 2, 64, 16, kind, W, S, routed=r, seed=50)
             for W, S, r in ((most, 0, 0.0), (1, most, 0.0), (most, most, 0.5), (7, 0, 1.0))]
    got = [c.run(swa) for c in cases]
    assert swa.get_device_error() == 0
    for c, x in zip(cases, got):
        c.check(x)


@pytest.mark.parametrize("kind", KINDS)
def test_most_rows_to_a_key_head(swa, kind):
    c = Case([256], [300], 128, 1, 64, 32, kind, 90, 10, routed=0.2, seed=51)
    c.check(c.run(swa))
    assert swa.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_many_slots(swa, kind):
    """More sequences than the plan's block has threads, most of one draft, some empty or without one."""
    rng = np.random.default_rng(52)
    ns = [int(rng.choice([1, 1, 2, 0, -1])) for _ in range(700)]
    c = Case(ns, [int(rng.integers(0, 40)) for _ in ns], 2, 1, 64, 8, kind, 9, 2, seed=52)
    c.check(c.run(swa))
    assert swa.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_no_work_at_all(swa, kind):
    """Rows and sequences, but none that owns any."""
    c = Case([0, 0, -2], [9, 0, 4], 4, 2, 64, 8, kind, 9, seed=53, pad=3)
    out = torch.full_like(c.q, 2.0)
    c.run(swa, out=out)
    assert bool((out == 2).all()) and swa.get_device_error() == 0


def test_accept_of_empty_slots_is_silent(swa):
    rng = np.random.default_rng(54)
    pools, table, _, starts, parents, _ = accept_setup(rng, [4, 4, 4], [9, 9, 9], 2, 8, 2, 64, "e4m3")
    got = swa.accept_tree(*pools.kv, ints(table), ints([0, 0, 0]), ints(starts), flat_parents(parents), ints([3, 99, -7]),
                          **pools.args())
    assert got.tolist() == [0, 0, 0] and swa.get_device_error() == 0
    pools.check()


def test_outputs_over_inputs_are_refused(swa):
    c = Case([3], [9], 2, 1, 64, 8, "bf16", 4, seed=55)
    table, lens, starts, parents, gate = c.tensors()
    with pytest.raises(swa.SwiAttnError):
        swa.decode_tree(c.q, *c.pages, table, lens, starts, parents, gate, 4, out=c.q)
    leaf = ints([2])
    for out in (leaf, lens):
        with pytest.raises(swa.SwiAttnError):
            swa.accept_tree(*c.pages, table, lens, starts, parents, leaf, out=out)
    source, new = ints([0]), ints([1])
    fresh = torch.empty_like(table)
    for pair in ((table, ints([0])), (fresh, lens), (fresh, source), (fresh, new), (fresh, fresh[0, :1])):
        with pytest.raises(swa.SwiAttnError):
            swa.fork_paged(*c.pages, table, lens, source, new, out=pair)
    assert swa.get_device_error() == 0
