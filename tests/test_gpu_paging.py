"""GPU checks of the calls that keep an accepted path and fork sequences (swiattn_accept_tree,
swiattn_fork_paged): bytes, so every comparison is exact, over whole pools."""
import numpy as np
import pytest
import torch

from test_gpu_append import swa  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

KINDS = {"bf16": (torch.bfloat16, 2), "f32": (torch.float32, 4), "e4m3": (torch.float8_e4m3fn, 1)}


class Pools:
    """Pools of random bytes, as tensors and as bytes [layers, pages, page, row] and [layers, pages, Hkv, page]."""

    def __init__(self, rng, layers, num_pages, page, Hkv, d, kind, flat=False):
        dtype, size = KINDS[kind]
        self.bytes, self.exps, self.kv, self.kv_exp = [], [], [], [None, None]
        for i in range(2):
            x = rng.integers(0, 256, (layers, num_pages, page, Hkv * d * size), dtype=np.uint8)
            self.bytes.append(x)
            t = torch.from_numpy(x.copy()).cuda().view(dtype).view(layers, num_pages, page, Hkv, d)
            self.kv.append(t[0] if flat else t)
            if kind == "e4m3":
                e = rng.integers(1, 255, (layers, num_pages, Hkv, page), dtype=np.uint8)
                self.exps.append(e)
                t = torch.from_numpy(e.copy()).cuda()
                self.kv_exp[i] = t[0] if flat else t

    def args(self):
        return dict(k_exp=self.kv_exp[0], v_exp=self.kv_exp[1])

    def move(self, pairs):
        """Rows ((page, slot) from, (page, slot) to), all read before any is written."""
        for x in self.bytes:
            rows = [x[:, p, s].copy() for (p, s), _ in pairs]
            for row, (_, (p, s)) in zip(rows, pairs):
                x[:, p, s] = row
        for x in self.exps:
            rows = [x[:, p, :, s].copy() for (p, s), _ in pairs]
            for row, (_, (p, s)) in zip(rows, pairs):
                x[:, p, :, s] = row

    def check(self):
        for t, x in zip(self.kv + [e for e in self.kv_exp if e is not None], self.bytes + self.exps):
            np.testing.assert_array_equal(t.cpu().contiguous().view(torch.uint8).numpy().reshape(-1), x.reshape(-1))


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def trees(rng, ns, wild=True):
    """Parents of trees of ns tokens: any earlier token, or none."""
    return [[int(rng.integers(-1, i)) if wild else i - 1 for i in range(n)] for n in ns]


def path_of(parents, leaf):
    out = []
    while leaf >= 0:
        out.append(leaf)
        leaf = parents[leaf]
    return out[::-1]


def accept_setup(rng, ns, bases, layers, page, Hkv, d, kind, leaves=None, flat=False):
    B = len(ns)
    lens = [n + b for n, b in zip(ns, bases)]
    max_pages = max(1, -(-max(lens) // page)) + 1
    num_pages = B * max_pages + 2
    table = rng.permutation(num_pages)[:B * max_pages].reshape(B, max_pages)
    parents = trees(rng, ns)
    if leaves is None:
        leaves = [int(rng.integers(-1, n)) if n else 0 for n in ns]
    pools = Pools(rng, layers, num_pages, page, Hkv, d, kind, flat)
    starts = np.concatenate([[0], np.cumsum(ns)])
    return pools, table, lens, starts, parents, leaves


def accept_reference(pools, table, lens, starts, parents, leaves, page):
    out = []
    for b, (n, p) in enumerate(zip(lens, parents)):
        path = path_of(p, leaves[b]) if p else []
        base = n - len(p)
        place = lambda i: (table[b][i // page], i % page)   # noqa: E731
        pools.move([(place(base + t), place(base + i)) for i, t in enumerate(path)])
        out.append(base + len(path))
    return out


def flat_parents(parents):
    return ints([x for p in parents for x in p] or [0])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("ns,bases,layers,page,Hkv,d", [
    ([1], [0], 1, 1, 1, 64),
    ([8], [777], 2, 16, 4, 128),
    ([5, 0, 33, 1, 256], [11, 7, 96, 0, 1023], 3, 32, 3, 64),
    ([17, 40, 3] * 12, [50, 2, 35] * 12, 1, 4, 16, 128),
    ([256, 200], [3, 250], 22, 256, 1, 128),
    ([64], [130], 1, 8, 70, 64),
])
def test_accept_moves_the_path(swa, ns, bases, layers, page, Hkv, d, kind):
    """Trees whose tokens hang on any earlier one, so that paths overlap their own targets."""
    rng = np.random.default_rng(sum(ns) + page)
    pools, table, lens, starts, parents, leaves = accept_setup(rng, ns, bases, layers, page, Hkv, d, kind,
                                                              flat=layers == 1)
    got = swa.accept_tree(*pools.kv, ints(table), ints(lens), ints(starts), flat_parents(parents), ints(leaves),
                          **pools.args())
    assert swa.get_device_error() == 0
    assert got.tolist() == accept_reference(pools, table, lens, starts, parents, leaves, page)
    pools.check()


def test_accept_long_chains_shifted_by_one(swa):
    """Each row of the path moves one slot down, onto the place of the one before: chains of 255 that
    leave out the first token."""
    rng = np.random.default_rng(5)
    pools, table, lens, starts, parents, _ = accept_setup(rng, [256] * 3, [1, 64, 100], 2, 16, 2, 64, "bf16")
    parents = [[-1, -1] + list(range(1, 255)) for _ in range(3)]
    leaves = [255, 200, 1]
    got = swa.accept_tree(*pools.kv, ints(table), ints(lens), ints(starts), flat_parents(parents), ints(leaves))
    assert got.tolist() == [1 + 255, 64 + 200, 100 + 1]
    accept_reference(pools, table, lens, starts, parents, leaves, 16)
    pools.check()


def test_accept_chains_without_parents(swa):
    rng = np.random.default_rng(6)
    pools, table, lens, starts, _, _ = accept_setup(rng, [4, 6, 0], [3, 9, 5], 1, 4, 2, 64, "e4m3")
    out = torch.zeros(3, dtype=torch.int32, device="cuda")
    got = swa.accept_tree(*pools.kv, ints(table), ints(lens), ints(starts), None, ints([1, -1, 7]), out=out,
                          **pools.args())
    assert got is out and out.tolist() == [5, 9, 5]
    pools.check()


def test_accept_bad_input_is_left_alone_and_reported(swa):
    rng = np.random.default_rng(7)
    for spoil in ("leaf", "short", "long", "negative", "starts", "behind", "parent", "page"):
        pools, table, lens, starts, parents, leaves = accept_setup(rng, [6, 6, 6], [14, 14, 14], 2, 8, 2, 64, "e4m3")
        parents = [[-1, -1, 1, 2, 0, 4] for _ in range(3)]
        leaves = [3, 3, 3]
        kept, want_path, skip = list(lens), None, set()
        if spoil == "leaf":
            leaves[1] = 6
        elif spoil in ("short", "long", "negative"):
            lens[1] = kept[1] = {"short": 5, "long": table.shape[1] * 8 + 1, "negative": -3}[spoil]
        elif spoil == "starts":
            starts = np.array([0, 6, 5, 18])   # sequence 1 has -1 tokens, sequence 2 thirteen
        elif spoil == "behind":
            starts = np.array([0, 6, 12, 19])
        elif spoil == "parent":
            parents[1][2] = 2
        else:
            table[1][1], table[1][2] = -1, -1   # slots 8 to 23: nothing of the path moves
        ref_leaves, ref_parents, ref_lens = list(leaves), [list(p) for p in parents], list(lens)
        got = swa.accept_tree(*pools.kv, ints(table), ints(lens), ints(starts), flat_parents(parents), ints(leaves),
                              **pools.args())
        assert swa.get_device_error() == 1 and swa.get_device_error() == 0, spoil
        bad = {"behind": [2], "starts": [1]}.get(spoil, [1])
        if spoil == "parent":
            ref_parents[1] = [-1, -1, -1, 2, 0, 4]   # the path ends there
            bad = []
        if spoil == "starts":
            assert got.tolist()[:2] == [17, lens[1]]
            continue   # sequence 2 is another one than was set up
        want = []
        for b in range(3):
            if spoil == "page" and b == 1:
                want.append(14 + 3)
            elif b in bad:
                want.append(kept[b])
            else:
                want += accept_reference(pools, [table[b]], [ref_lens[b]], None, [ref_parents[b]], [ref_leaves[b]], 8)
        assert got.tolist() == want, spoil
        pools.check()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("lens,C,layers,page,Hkv,d", [
    ([1], 1, 1, 1, 1, 64),
    ([777], 5, 2, 16, 4, 128),
    ([5, 64, 33, 1, 127], 40, 3, 32, 3, 64),
    ([1000, 256, 3], 9, 22, 256, 2, 128),
    ([30, 31], 3, 1, 2, 80, 64),
    ([100], 300, 1, 128, 1, 64),
])
def test_fork_copies_the_last_page(swa, lens, C, layers, page, Hkv, d, kind):
    rng = np.random.default_rng(C + page)
    B = len(lens)
    max_pages = -(-max(lens) // page) + (C % 2)   # with and without room for a next page
    num_pages = B * max_pages + C
    perm = rng.permutation(num_pages)
    table, fresh = perm[:B * max_pages].reshape(B, max_pages), perm[B * max_pages:]
    source, new = rng.integers(0, B, C), fresh.copy()
    if C > 2:
        source[1], new[2] = -1, -1
    pools = Pools(rng, layers, num_pages, page, Hkv, d, kind, flat=layers == 1)
    got, got_lens = swa.fork_paged(*pools.kv, ints(table), ints(lens), ints(source), ints(new), **pools.args())
    assert swa.get_device_error() == 0
    want, pairs = np.zeros((C, max_pages), np.int64), []
    for c in range(C):
        if source[c] < 0:
            continue
        n = lens[source[c]]
        want[c] = table[source[c]]
        if new[c] >= 0 and n // page < max_pages:
            want[c, n // page] = new[c]
            pairs += [((table[source[c]][n // page], s), (new[c], s)) for s in range(n % page)]
    pools.move(pairs)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert got_lens.tolist() == [0 if b < 0 else lens[b] for b in source]
    pools.check()


def test_fork_bad_input_makes_empty_slots(swa):
    rng = np.random.default_rng(3)
    for spoil in ("source", "long", "negative", "new", "page"):
        table, lens = np.arange(12).reshape(3, 4), [13, 21, 30]
        source, new = [0, 1, 2], [12, 13, 14]
        if spoil == "source":
            source[1] = 3
        elif spoil in ("long", "negative"):
            lens[1] = {"long": 33, "negative": -1}[spoil]
        elif spoil == "new":
            new[1] = 15
        else:
            table[1, 2] = 15
        pools = Pools(rng, 2, 15, 8, 1, 64, "e4m3")
        got, got_lens = swa.fork_paged(*pools.kv, ints(table), ints(lens), ints(source), ints(new), **pools.args())
        assert swa.get_device_error() == 1 and swa.get_device_error() == 0, spoil
        assert got_lens.tolist() == [13, 0, 30] and got[1].tolist() == [0] * 4
        assert got[0].tolist() == [0, 12, 2, 3] and got[2].tolist() == [8, 9, 10, 14]
        pools.move([((1, s), (12, s)) for s in range(5)] + [((11, s), (14, s)) for s in range(6)])
        pools.check()


def test_paging_in_a_graph_on_a_side_stream(swa):
    """An accept and a fork captured together, replayed with other lengths and leaves in the same tensors."""
    rng = np.random.default_rng(4)
    pools, table, lens, starts, parents, _ = accept_setup(rng, [9, 9], [20, 3], 2, 8, 2, 64, "bf16")
    parents = [[-1, 0, 1, -1, 3, 4, 0, 6, 7]] * 2
    spare = [p for p in range(pools.kv[0].shape[1]) if p not in table]
    t_table, t_lens, t_starts, t_parents = ints(table), ints(lens), ints(starts), flat_parents(parents)
    leaf, source, new = ints([5, 8]), ints([1]), ints(spare[:1])
    kept = torch.empty_like(t_lens)
    out = (torch.empty((1, table.shape[1]), dtype=torch.int32, device="cuda"), torch.empty_like(source))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [p.clone() for p in pools.kv]

    def call():
        swa.accept_tree(*pools.kv, t_table, t_lens, t_starts, t_parents, leaf, out=kept)
        swa.fork_paged(*pools.kv, t_table, kept, source, new, out=out)

    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    side.synchronize()
    for p, s in zip(pools.kv, state):
        p.copy_(s)
    leaf.copy_(ints([8, 4]))
    graph.replay()
    torch.cuda.synchronize()
    want = accept_reference(pools, table, lens, starts, parents, [8, 4], 8)
    assert kept.tolist() == want and out[1].tolist() == [want[1]]
    at = want[1] // 8
    pools.move([((table[1][at], s), (spare[0], s)) for s in range(want[1] % 8)])
    row = list(table[1])
    row[at] = spare[0]
    assert out[0][0].tolist() == row
    pools.check()


def test_paging_binding_refusals(swa):
    k = torch.zeros((2, 6, 8, 1, 64), device="cuda", dtype=torch.bfloat16)
    table, lens = ints([[0, 1, 2]]), ints([9])
    starts, parents, leaf = ints([0, 3]), ints([-1, 0, 1]), ints([2])
    good = dict(k_pages=k, v_pages=k.clone(), block_table=table, seq_lens=lens, starts=starts, parents=parents, leaf=leaf)
    for bad in (dict(v_pages=k[:1].contiguous()), dict(v_pages=k.float()), dict(k_pages=k.half(), v_pages=k.half()),
                dict(block_table=ints([[0], [1]])), dict(seq_lens=lens.long()), dict(starts=ints([0])),
                dict(parents=parents.long()), dict(parents=parents[None]), dict(leaf=ints([1, 1])), dict(leaf=leaf.cpu()),
                dict(k_pages=k.to(torch.float8_e4m3fn), v_pages=k.to(torch.float8_e4m3fn)), dict(out=ints([1, 2])),
                dict(k_pages=k[0, 0], v_pages=k[0, 0]), dict(k_pages=k.transpose(1, 2))):
        with pytest.raises(ValueError):
            swa.accept_tree(**{**good, **bad})
    with pytest.raises(swa.SwiAttnError):
        swa.accept_tree(**good, out=lens)
    good = dict(k_pages=k, v_pages=k.clone(), block_table=table, seq_lens=lens, source=ints([0, 0]), new_page=ints([3, 4]))
    for bad in (dict(new_page=ints([3])), dict(source=ints([0, 0]).long()), dict(out=(ints([[0, 0, 0]]), ints([0, 0]))),
                dict(block_table=table[0])):
        with pytest.raises(ValueError):
            swa.fork_paged(**{**good, **bad})
    with pytest.raises(swa.SwiAttnError):
        swa.fork_paged(**{**good, "source": ints([0]), "new_page": ints([3])}, out=(table, ints([0])))
