"""The operators of speculative decoding over a paged cache, measured: rotary positions with several
axes (with their gradient), appending tokens at given positions, attention of a tree of drafted
tokens over the cache, keeping the accepted path of a tree, and forking sequences.

Every case has a plain form in elementary torch operations (``own`` false) and the calls a user makes
of the package (``own`` true).  Both take the same prepared state.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LAYERS = 22   # of the 1.5B model that the method's report trains


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One long prompt of text and video: time, height and width in sections of a head's frequencies.
        dict(name="rope_video_32k", op="rope", grad=False, B=1, N=32768, Hq=16, Hkv=16, d=128, rot=128, axes=3,
             spread=False, interleaved=False, fused=False, dtype="bf16"),
        # Training on images, two sequences of 8K with grouped heads: dq and dk of the attention back through the
        # rotation, the axes dealt out to the frequencies in turn, views of one projection's gradient.
        dict(name="rope_grad_2x8k", op="rope", grad=True, B=2, N=8192, Hq=16, Hkv=4, d=128, rot=128, axes=3,
             spread=True, interleaved=False, fused=True, dtype="bf16"),
        # A serving batch takes in prompts with images, of uneven length, into 8-bit pages.
        dict(name="append_images_e4m3", op="append", B=5, new=3001, prior=3000, Hq=16, Hkv=16, d=128, rot=128, axes=3,
             spread=False, interleaved=False, fused=True, page=64, pages="e4m3", dtype="bf16", seed=21),
        # The drafted trees of a batch of sixteen far into their contexts: positions are depths in the tree.
        dict(name="append_trees_bf16", op="append", B=16, new=32, prior=32000, Hq=16, Hkv=16, d=128, rot=128, axes=1,
             spread=False, interleaved=False, fused=True, page=64, pages="bf16", dtype="bf16", seed=22),
        # Verification of the benchmark's decode batch, 16 drafted tokens each, the method's routed fraction.
        dict(name="tree_16x32k", op="tree", B=16, L=32768, ragged=False, empty=0, drafts=16, routed=0.13, Hq=16,
             Hkv=16, d=128, W=1024, anchors=0, page=64, pages="bf16", seed=23),
        # 32 drafted tokens each over 8-bit pages, grouped heads.
        dict(name="tree_8x32k_e4m3", op="tree", B=8, L=32768, ragged=False, empty=0, drafts=32, routed=0.13, Hq=16,
             Hkv=4, d=128, W=1024, anchors=0, page=64, pages="e4m3", seed=24),
        # One short sequence with a few drafts: latency alone counts.
        dict(name="tree_1x777", op="tree", B=1, L=777, ragged=False, empty=0, drafts=8, routed=0.13, Hq=16, Hkv=16,
             d=128, W=256, anchors=0, page=16, pages="bf16", seed=25),
        # A padded batch with large trees of uneven size, anchors, head size 64, groups of three: many rows of
        # queries, of which the routed ones alone need the whole history.
        dict(name="tree_ragged_33", op="tree", B=33, L=8191, ragged=True, empty=2, drafts=201, routed=0.13, Hq=12,
             Hkv=4, d=64, W=512, anchors=256, page=16, pages="bf16", seed=26),
        # The accepted paths of a batch of sixteen, all layers at once.
        dict(name="accept_16", op="accept", layers=LAYERS, B=16, L=32768, drafts=32, Hkv=16, d=128, page=64,
             pages="bf16", seed=27),
        # One sequence on 8-bit pages: latency alone counts.
        dict(name="accept_1_e4m3", op="accept", layers=LAYERS, B=1, L=5003, drafts=16, Hkv=4, d=128, page=16,
             pages="e4m3", seed=28),
        # 64 continuations of four prompts, all layers: the page that each prompt ends in is copied for its children.
        dict(name="fork_4_to_64", op="fork", layers=LAYERS, B=4, C=64, L=5003, Hkv=16, d=128, page=64, pages="bf16",
             seed=29),
        # Beams of one layer's 8-bit cache, small pages: latency alone counts.
        dict(name="fork_8_beams_e4m3", op="fork", layers=1, B=8, C=8, L=3001, Hkv=4, d=128, page=16, pages="e4m3",
             seed=30),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree", "tree", "accept", "fork"])
    d = rng.choice([64, 128])
    seed = rng.randrange(1 << 20)
    if op in ("accept", "fork"):
        Hkv, page, pages = rng.choice([1, 2, 3, 4, 8, 16]), 2 ** rng.randint(0, 8), rng.choice(["bf16", "e4m3", "f32"])
        layers = rng.choice([1, 2, LAYERS])
        L = _log(rng, 1, 65536)
        row = 8 * layers * Hkv * d   # bytes of a token at most
        if op == "accept":
            drafts = _log(rng, 1, 256)
            return dict(op=op, layers=layers, B=_log(rng, 1, max(1, min(64, (1 << 28) // (row * (drafts + 2 * page))))),
                        L=L, drafts=drafts, Hkv=Hkv, d=d, page=page, pages=pages, seed=seed)
        B = _log(rng, 1, 8)
        return dict(op=op, layers=layers, B=B, C=_log(rng, 1, max(1, min(64, (1 << 29) // (row * page) - B))), L=L,
                    Hkv=Hkv, d=d, page=page, pages=pages, seed=seed)
    if op == "tree":
        pages = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
        G, Hkv = rng.choice([1, 1, 2, 3, 4, 5, 8, 16]), _log(rng, 1, 16)
        B, drafts = _log(rng, 1, 64), _log(rng, 1, 256)
        # keys of the cache and products are both bounded
        most = min((1 << 28) // (B * Hkv * d), (1 << (27 if pages == "f32" else 30)) // (B * Hkv * G * drafts))
        L = _log(rng, 1, max(1, min(65536, most)))
        return dict(op=op, B=B, L=L, ragged=rng.random() < 0.6, empty=rng.choice([0, 0, min(1, B - 1)]), drafts=drafts,
                    routed=rng.choice([0.0, 0.02, 0.13, 0.3, 1.0]), Hq=G * Hkv, Hkv=Hkv, d=d, W=_log(rng, 1, 4096),
                    anchors=rng.choice([0, 0, rng.randint(1, 300)]), page=2 ** rng.randint(0, 8), pages=pages,
                    seed=seed)
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4])
    rot = 16 * rng.randint(1, d // 16)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = (3 << 24) // ((Hq + 2 * Hkv) * d)   # tokens
    axes = rng.randint(1, 4)
    common = dict(Hq=Hq, Hkv=Hkv, d=d, rot=rot, axes=axes, spread=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                  fused=rng.random() < 0.5, dtype=dtype)
    if op == "rope":
        T = _log(rng, 1, most)
        B = rng.randint(1, min(4, T))
        return dict(op=op, grad=rng.random() < 0.5, B=B, N=max(1, T // B), **common)
    B = _log(rng, 1, 64)
    return dict(op=op, B=B, new=_log(rng, 1, min(256, most // B) if axes == 1 else max(1, most // B)),
                prior=rng.choice([0, _log(rng, 1, 100000)]), page=2 ** rng.randint(0, 8),
                pages="e4m3" if dtype == "bf16" and rng.random() < 0.6 else dtype, seed=seed, **common)


# ------------------------------------------------------- what a case is about, whatever its values

def _tree(rng, n):
    """Parents of n drafted tokens, -1 the last cached token: the likeliest continuation first, then
    branches off it or off the cache, each laid out after the other and no deeper than the first."""
    chain = max(1, round(n * rng.uniform(0.25, 0.6)))
    parents = list(range(-1, chain - 1))
    while len(parents) < n:
        at = rng.randint(-1, chain - 2)
        for _ in range(min(rng.randint(1, chain - 1 - at), n - len(parents))):
            parents.append(at)
            at = len(parents) - 1
    return parents


def _depths(parents):
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def _sequences(case):
    """For each sequence: its length, the drafted ones among it counted, and the parents of those."""
    rng = random.Random(case["seed"])
    B = case["B"]
    if case["op"] == "append":
        out = []
        for _ in range(B):
            n = case["new"] if B == 1 else max(1, round(case["new"] * rng.uniform(0.3, 1.7)))
            prior = 0 if case["prior"] == 0 else rng.randint(case["prior"] // 2, case["prior"])
            out.append((n + prior, _tree(rng, n) if case["axes"] == 1 else [-1] * n))
        return out
    if case["op"] == "fork":
        return [(rng.randint(max(1, case["L"] // 2), case["L"]), []) for _ in range(B)]
    if case["op"] == "accept":
        out = []
        for _ in range(B):
            n = rng.randint((case["drafts"] + 1) // 2, case["drafts"])
            out.append((n + rng.randint(case["L"] // 2, case["L"]), _tree(rng, n)))
        return out
    out, empty = [], set(rng.sample(range(B), case["empty"]))
    for b in range(B):
        length = rng.randint(1, case["L"]) if case["ragged"] else case["L"]
        n = rng.randint(1, case["drafts"]) if case["ragged"] else case["drafts"]
        out.append((0, []) if b in empty else (max(length, n), _tree(rng, n)))
    return out


def _gates(case):
    """Which drafted tokens of a "tree" case are routed, for each sequence."""
    rng = random.Random(case["seed"] + 1)
    return [[int(rng.random() < case["routed"]) for _ in parents] for _, parents in _sequences(case)]


def _leaves(case):
    """The accepted leaf of each tree of an "accept" case: any token of it, or none."""
    rng = random.Random(case["seed"] + 1)
    return [rng.randint(-1 if rng.random() < 0.1 else 0, len(parents) - 1) for _, parents in _sequences(case)]


def _forks(case):
    """The source of each child of a "fork" case."""
    rng = random.Random(case["seed"] + 1)
    return [rng.randrange(case["B"]) for _ in range(case["C"])]


def _row_bytes(case):
    """Bytes of one key (or value) row of a page."""
    return case["d"] + 1 if case["pages"] == "e4m3" else case["d"] * (2 if case["pages"] == "bf16" else 4)


def work(case):
    Hkv, d, row = case["Hkv"], case["d"], _row_bytes(case) if "pages" in case else 0
    if case["op"] == "accept":
        moved = kept = 0
        for (_, parents), leaf in zip(_sequences(case), _leaves(case)):
            path = []
            while leaf >= 0:
                path.append(leaf)
                leaf = parents[leaf]
            moved += sum(at != i for i, at in enumerate(reversed(path)))
            kept += len(parents)
        return {"bytes": case["layers"] * moved * Hkv * row * 4 + 4 * (kept + 5 * case["B"]), "flops": 0}
    if case["op"] == "fork":
        lens, read, written = _sequences(case), {}, 0
        for b in _forks(case):
            read[b] = lens[b][0] % case["page"]
            written += read[b]
        table = 4 * (max(n for n, _ in lens) // case["page"] + 1)
        return {"bytes": case["layers"] * (sum(read.values()) + written) * Hkv * row * 2 + case["C"] * (table + 16)
                + len(read) * table, "flops": 0}
    size = 4 if case["dtype" if "dtype" in case else "pages"] == "f32" else 2
    Hq = case["Hq"]
    if case["op"] == "tree":
        keys = pairs = tokens = 0
        for (length, parents), gates in zip(_sequences(case), _gates(case)):
            if not parents:
                continue
            n, W = len(parents), case["W"]
            base = length - n
            near = base if any(gates) else min(base, W - 1)   # cached keys that some drafted token reads
            keys += n + near + min(case["anchors"], base - near)
            for depth, gate in zip(_depths(parents), gates):
                lo = 0 if gate else max(0, base + depth - W + 1)
                pairs += base + depth + 1 - lo + min(case["anchors"], lo)
            tokens += n
        return {"bytes": keys * Hkv * 2 * row + tokens * (Hq * (2 * d * size + 4) + 5), "flops": 4 * pairs * Hq * d}
    if case["op"] == "rope":
        T = case["B"] * case["N"]
        return {"bytes": T * (2 * (Hq + Hkv) * d * size + 4 * case["axes"]), "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    T = sum(len(parents) for _, parents in _sequences(case))
    return {"bytes": T * (Hq * d * size * 2 + Hkv * (2 * d * size + 2 * row) + 4 * case["axes"]),
            "flops": 3 * T * (Hq + Hkv) * case["rot"]}


# --------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _heads(rows, case, g, value=True):
    """q, k (and v) of `rows` tokens: tensors of their own, or views of one fused projection."""
    Hq, Hkv, d, dtype = case["Hq"], case["Hkv"], case["d"], DTYPES[case["dtype"]]
    counts = [Hq, Hkv] + ([Hkv] if value else [])
    if not case["fused"]:
        return [_randn((*rows, h, d), dtype, g) for h in counts]
    # the projection holds v too, whether this call uses it or not
    x = _randn((*rows, (Hq + 2 * Hkv) * d), dtype, g)
    parts = x.split([Hq * d, Hkv * d, Hkv * d], dim=-1)
    return [p.unflatten(-1, (h, d)) for p, h in zip(parts, counts)]


def _inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)


def _axis_of(case):
    """The axis that turns each frequency: sections one after another, or dealt out in turn."""
    half, A = case["rot"] // 2, case["axes"]
    return [f % A if case["spread"] else f * A // half for f in range(half)]


def _grid(case, at, g):
    """Positions [axes, ...] of tokens `at` in their sequences: a run of text, along which all axes
    count alike, then frames of patches that count height and width over again."""
    A = case["axes"]
    text = torch.randint(0, 50, (1,), generator=g, device="cuda")
    i = (at - text).clamp_min(0)
    side = 24
    counts = [i // (side * side), i // side % side, i % side, i // (4 * side * side)][-A:] if A > 1 else [i]
    return torch.stack([(torch.minimum(at, text) + c) for c in counts]).to(torch.int32)


def _quantise(x):
    """e4m3 values and power-of-two scales (e8m0) of rows along the last dimension: the smallest
    scale 2^e with max |x| <= 448 * 2^e, and the row divided by it, to the nearest e4m3."""
    amax = x.abs().amax(-1)
    mant, expo = torch.frexp(amax)   # amax = mant * 2^expo, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = (expo - 9 + (mant > 0.875)).clamp(-126, 127)
    e = torch.where(amax == 0, torch.full_like(e, -126), e)
    v = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return v, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _pool(case, lead, g):
    """k and v pages [*lead, page, Hkv, d] (with exponents [*lead, Hkv, page]) full of rows whose size
    differs from token to token, as dict entries."""
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    num = math.prod(lead)
    out = dict(k_exp=None, v_exp=None)
    some = max(1, (1 << 27) // (page * Hkv * d))   # pages at a time
    for name in "kv":
        if case["pages"] == "e4m3":
            pages = torch.empty((num, page, Hkv, d), device="cuda", dtype=torch.float8_e4m3fn)
            exps = torch.empty((num, Hkv, page), device="cuda", dtype=torch.float8_e8m0fnu)
        else:
            pages = torch.empty((num, page, Hkv, d), device="cuda", dtype=DTYPES[case["pages"]])
        for a in range(0, num, some):
            z = min(num, a + some)
            x = torch.randn((z - a, page, Hkv, d), generator=g, device="cuda")
            x *= torch.exp(0.5 * torch.randn((z - a, page, Hkv, 1), generator=g, device="cuda"))
            if case["pages"] == "e4m3":
                value, scale = _quantise(x)
                pages.view(torch.uint8)[a:z] = value.view(torch.uint8)
                exps.view(torch.uint8)[a:z] = scale.view(torch.uint8).transpose(1, 2)
            else:
                pages[a:z] = x.to(pages.dtype)
        out[name + "_pages"] = pages.view(*lead, page, Hkv, d)
        if case["pages"] == "e4m3":
            out[name + "_exp"] = exps.view(*lead, Hkv, page)
    return out


def _table(case, first, last, g, spare):
    """A block table whose entries for pages first[b] .. last[b] are scattered over a pool of just so
    many pages and `spare` more (the last of the pool, in no table); pages that a call does not touch
    are not held."""
    first, last = torch.tensor(first), torch.tensor(last)
    held = last - first + 1
    touched = int(held.sum())
    perm = torch.randperm(touched, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros((len(first), max(1, int(last.max()) + 1)), dtype=torch.int32)
    owner = torch.repeat_interleave(torch.arange(len(first)), held)
    ahead = held.cumsum(0) - held
    table[owner, first[owner] + torch.arange(touched) - ahead[owner]] = perm
    return table.cuda(), touched + spare


def _packed(case):
    """starts, parents and lengths of the sequences' drafted (or new) tokens, on the GPU."""
    seqs = _sequences(case)
    starts = [0]
    for _, parents in seqs:
        starts.append(starts[-1] + len(parents))
    return dict(starts=_ints(starts), seq_lens=_ints([n for n, _ in seqs]),
                parents=_ints([p for _, parents in seqs for p in parents]))


def _prepare_rope(case, g):
    B, N = case["B"], case["N"]
    q, k = _heads((B, N), case, g, value=False)
    at = torch.arange(N, device="cuda").expand(B, N)
    positions = _grid(case, at, g)
    return dict(q=q, k=k, positions=positions, inv_freq=_inv_freq(case["rot"]), axis_of=_axis_of(case))


def _prepare_append(case, g):
    seqs, page, s = _sequences(case), case["page"], _packed(case)
    T = sum(len(p) for _, p in seqs)
    s["q"], s["k"], s["v"] = _heads((T,), case, g)
    if case["axes"] == 1:   # a drafted token sits as far on as it is deep in its tree
        s["positions"] = _ints([n - len(p) + x for n, p in seqs for x in _depths(p)])
        s["axis_of"] = None
    else:
        at = torch.cat([torch.arange(n - len(p), n) for n, p in seqs]).cuda()
        s["positions"], s["axis_of"] = _grid(case, at, g), _axis_of(case)
    s["block_table"], num_pages = _table(case, [(n - len(p)) // page for n, p in seqs],
                                         [(n - 1) // page for n, _ in seqs], g, 8)
    s["inv_freq"] = _inv_freq(case["rot"])
    shape = (num_pages, page, case["Hkv"], case["d"])
    s.update(k_exp=None, v_exp=None)
    for name in "kv":
        if case["pages"] == "e4m3":
            s[name + "_pages"] = torch.zeros(shape, device="cuda", dtype=torch.float8_e4m3fn)
            s[name + "_exp"] = torch.full((num_pages, case["Hkv"], page), 127, device="cuda",
                                          dtype=torch.uint8).view(torch.float8_e8m0fnu)
        else:
            s[name + "_pages"] = torch.zeros(shape, device="cuda", dtype=DTYPES[case["pages"]])
    return s


def _prepare_tree(case, g):
    seqs, page, s = _sequences(case), case["page"], _packed(case)
    s["gate"] = torch.tensor([x for gates in _gates(case) for x in gates], dtype=torch.uint8).cuda()
    s["block_table"], num_pages = _table(case, [0] * len(seqs), [(n + page - 1) // page - 1 for n, _ in seqs], g, 2)
    s.update(_pool(case, (num_pages,), g))
    T = sum(len(p) for _, p in seqs)
    s["q"] = _randn((T, case["Hq"], case["d"]), DTYPES["f32" if case["pages"] == "f32" else "bf16"], g)
    return s


def _prepare_accept(case, g):
    seqs, page, s = _sequences(case), case["page"], _packed(case)
    s["leaf"] = _ints(_leaves(case))
    s["block_table"], num_pages = _table(case, [(n - len(p)) // page for n, p in seqs],
                                         [(n - 1) // page for n, _ in seqs], g, 1)
    s.update(_pool(case, (case["layers"], num_pages), g))
    return s


def _prepare_fork(case, g):
    seqs, page, C = _sequences(case), case["page"], case["C"]
    at = [(n - 1) // page for n, _ in seqs]
    s = dict(seq_lens=_ints([n for n, _ in seqs]), source=_ints(_forks(case)))
    table, num_pages = _table(case, at, at, g, C + 1)
    s["block_table"] = torch.cat([table, torch.zeros_like(table[:, :1])], 1)   # room for the next page
    s["new_page"] = (num_pages - 1 - C + torch.randperm(C, generator=g, device="cuda")).to(torch.int32)
    s.update(_pool(case, (case["layers"], num_pages), g))
    return s


_PREPARE = dict(rope=_prepare_rope, append=_prepare_append, tree=_prepare_tree, accept=_prepare_accept,
                fork=_prepare_fork)


def prepare(case, seed):
    state = _PREPARE[case["op"]](case, _generator(seed))
    state["case"] = case
    return state


# ----------------------------------------------------------------------------------- plain form

def _rotated(x, positions, axis_of, inv_freq, interleaved, sign=1.0):
    """x [..., H, d] in fp32, rotated by positions [axes, ...] (axis_of None: [...]); angles in 64 bits."""
    if axis_of is None:
        turn = positions.double()[..., None]
    else:   # [..., frequencies]: the position on each frequency's own axis
        turn = positions[torch.tensor(axis_of, device=x.device)].double().movedim(0, -1)
    angle = turn * inv_freq
    cos, sin = angle.cos().float()[..., None, :], (sign * angle.sin()).float()[..., None, :]
    rot = 2 * inv_freq.numel()
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s, case):
    sign = -1.0 if case["grad"] else 1.0
    return tuple(_rotated(s[n], s["positions"], s["axis_of"], s["inv_freq"], case["interleaved"], sign).to(s[n].dtype)
                 for n in "qk")


def _plain_append(s, case):
    page, starts, T = case["page"], s["starts"].long(), s["k"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    at = s["seq_lens"].long()[b] - (starts[b + 1] - t)
    row = s["block_table"].long()[b, at // page] * page + at % page

    def turned(x):
        return _rotated(x, s["positions"], s["axis_of"], s["inv_freq"], case["interleaved"])

    out = dict(q=turned(s["q"]).to(s["q"].dtype))
    for name, x in (("k", turned(s["k"])), ("v", s["v"].float())):
        pages = s[name + "_pages"]
        if case["pages"] == "e4m3":
            value, scale = _quantise(x)
            pages.view(torch.uint8).flatten(0, 1)[row] = value.view(torch.uint8)
            exps = s[name + "_exp"]
            exps.view(torch.uint8)[row // page, :, row % page] = scale.view(torch.uint8)
            out[name + "_exp"] = exps
        else:
            pages.flatten(0, 1)[row] = x.to(pages.dtype)
        out[name + "_pages"] = pages
    return out


def _ancestors(s, case):
    """[B, n, n] whether token u of a tree is token t or one of those before it on its path; and which
    of the n tokens there are, n being the most that a tree holds."""
    n = max(len(p) for _, p in _sequences(case))
    starts = s["starts"].long()
    i = torch.arange(n, device="cuda")
    some = i < (starts[1:] - starts[:-1])[:, None]
    at = (starts[:-1, None] + i).clamp_max(s["parents"].numel() - 1)
    parent = torch.where(some, s["parents"].long()[at], torch.full_like(at, -1))
    reach = ((parent[..., None] == i) | (i[:, None] == i)).float()
    for _ in range((n - 1).bit_length()):   # paths of up to 1, 2, 4, ... steps
        reach = (reach @ reach).clamp_max(1.0)
    return reach > 0, some, at


def _plain_tree(s, case):
    B, page, Hq, Hkv, d, W = case["B"], case["page"], case["Hq"], case["Hkv"], case["d"], case["W"]
    table, lens = s["block_table"].long(), s["seq_lens"].long()[:, None, None]
    width = table.shape[1] * page
    reach, some, row = _ancestors(s, case)
    n = reach.shape[1]

    def entries(name):
        pages = s[name + "_pages"]
        if case["pages"] != "e4m3":
            return pages[table].view(B, width, Hkv, d).float()
        value = pages.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        scale = s[name + "_exp"].view(torch.uint8)[table].view(torch.float8_e8m0fnu).float()
        return (value * scale.transpose(2, 3)[..., None]).view(B, width, Hkv, d)

    # Which entries [B, n, width] each token reads.  A drafted entry's own position is its depth on.
    drafted = some.sum(-1)[:, None, None]
    base = lens - drafted
    at = torch.arange(width, device="cuda")
    depth = reach.sum(-1) - 1
    u = (at - base).expand(B, n, width)
    pos = base + depth[..., None]
    inside = (u >= 0) & (u < drafted)
    on_path = torch.gather(reach, 2, u.clamp(0, n - 1)) & inside
    key_pos = torch.where(inside, base + torch.gather(depth[:, None].expand(B, n, n), 2, u.clamp(0, n - 1)), at)
    gate = s["gate"][row] != 0
    near = gate[..., None] | (key_pos > pos - W) | (key_pos < case["anchors"])
    seen = near & ((u < 0) | on_path) & some[..., None]

    q = s["q"].float()[row].view(B, n, Hkv, Hq // Hkv, d)
    score = torch.einsum("bnhgd,blhd->bhgnl", q, entries("k")) / math.sqrt(d)
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    any_seen = seen.any(-1)[:, None, None, :, None]
    top = torch.where(any_seen, score.amax(-1, keepdim=True), torch.zeros((), device="cuda"))
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bhgnd", p, entries("v")) / torch.where(any_seen, total, torch.ones((), device="cuda"))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d).to(s["q"].dtype)
    lse = (top + total.log()).permute(0, 3, 1, 2, 4).reshape(B, n, Hq)
    # back to the packed tokens
    starts, t = s["starts"].long(), torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return dict(o=o[b, t - starts[b]], lse=lse[b, t - starts[b]])


def _plain_accept(s, case):
    page, spare = case["page"], s["k_pages"].shape[1] - 1
    reach, some, _ = _ancestors(s, case)
    B, n = some.shape
    leaf, drafted = s["leaf"].long(), some.sum(-1)
    path = reach[torch.arange(B, device="cuda"), leaf.clamp_min(0)] & (leaf >= 0)[:, None] & some
    count = path.sum(-1)
    base = s["seq_lens"].long() - drafted
    i = torch.arange(n, device="cuda").expand(B, n)
    order = torch.sort((~path).to(torch.uint8), dim=-1, stable=True).indices   # the path first, in order
    last = (drafted - 1)[:, None]
    src = torch.where(i < count[:, None], order, torch.minimum(i, last))   # what is not on it stays
    dst = torch.minimum(i, last)

    def rows(at):   # rows of the pool; trees without tokens touch the spare page alone
        at = base[:, None] + at
        held = torch.gather(s["block_table"].long(), 1, (at // page).clamp_min(0))
        return torch.where(some.any(-1)[:, None], held * page + at % page, torch.full_like(at, spare * page)).flatten()

    src, dst = rows(src), rows(dst)
    out = dict(seq_lens=(base + count).to(torch.int32))
    for name in "kv":
        pages = s[name + "_pages"]
        flat = (pages.view(torch.uint8) if case["pages"] == "e4m3" else pages).flatten(1, 2)
        flat[:, dst] = flat[:, src]
        out[name + "_pages"] = pages
        if case["pages"] == "e4m3":
            exps = s[name + "_exp"].view(torch.uint8)
            exps[:, dst // page, :, dst % page] = exps[:, src // page, :, src % page]
            out[name + "_exp"] = s[name + "_exp"]
    return out


def _plain_fork(s, case):
    page, source = case["page"], s["source"].long()
    lens = s["seq_lens"][source]
    at, rest = (lens // page).long(), lens % page
    table = s["block_table"][source]
    old = torch.gather(table.long(), 1, at[:, None])[:, 0]
    table = table.scatter(1, at[:, None], s["new_page"][:, None])
    new = s["new_page"].long()
    kept = torch.arange(page, device="cuda") < rest[:, None]   # [C, page]
    out = dict(block_table=table, seq_lens=lens)
    for name in "kv":
        pages = s[name + "_pages"]
        flat = pages.view(torch.uint8) if case["pages"] == "e4m3" else pages
        flat[:, new] = torch.where(kept[..., None, None], flat[:, old], flat[:, new])
        out[name + "_pages"] = pages
        if case["pages"] == "e4m3":
            exps = s[name + "_exp"].view(torch.uint8)
            exps[:, new] = torch.where(kept[:, None], exps[:, old], exps[:, new])
            out[name + "_exp"] = s[name + "_exp"]
    return out


_PLAIN = dict(rope=_plain_rope, append=_plain_append, tree=_plain_tree, accept=_plain_accept, fork=_plain_fork)


# ------------------------------------------------------------------------- the package's operators

def _own_rope(s, case):
    import sliding_window_attention_router_gb300 as swa
    call = swa.rope_backward if case["grad"] else swa.rope
    return call(s["q"], s["k"], s["inv_freq"], positions=s["positions"], axes=s["axis_of"],
                interleaved=case["interleaved"])


def _with_exponents(s, out):
    return out if s["k_exp"] is None else dict(out, k_exp=s["k_exp"], v_exp=s["v_exp"])


def _own_append(s, case):
    import sliding_window_attention_router_gb300 as swa
    q = swa.append_paged(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"],
                         s["inv_freq"], starts=s["starts"], positions=s["positions"], axes=s["axis_of"],
                         interleaved=case["interleaved"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    return _with_exponents(s, dict(q=q, k_pages=s["k_pages"], v_pages=s["v_pages"]))


def _own_tree(s, case):
    import sliding_window_attention_router_gb300 as swa
    if "workspace" not in s:   # kept from step to step, as a serving loop does
        nbytes = swa.decode_tree_workspace(s["q"].shape[0], case["B"], case["Hq"], case["Hkv"], case["d"],
                                           s["q"].dtype)
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    o, lse = swa.decode_tree(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], s["starts"],
                             s["parents"], s["gate"], case["W"], n_anchor=case["anchors"], k_exp=s["k_exp"],
                             v_exp=s["v_exp"], want_lse=True, workspace=s["workspace"])
    return dict(o=o, lse=lse)


def _own_accept(s, case):
    import sliding_window_attention_router_gb300 as swa
    lens = swa.accept_tree(s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], s["starts"], s["parents"],
                           s["leaf"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    return _with_exponents(s, dict(seq_lens=lens, k_pages=s["k_pages"], v_pages=s["v_pages"]))


def _own_fork(s, case):
    import sliding_window_attention_router_gb300 as swa
    table, lens = swa.fork_paged(s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], s["source"],
                                 s["new_page"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    return _with_exponents(s, dict(block_table=table, seq_lens=lens, k_pages=s["k_pages"], v_pages=s["v_pages"]))


_OWN = dict(rope=_own_rope, append=_own_append, tree=_own_tree, accept=_own_accept, fork=_own_fork)


def run(state):
    case = state["case"]
    return (_OWN if own else _PLAIN)[case["op"]](state, case)


# ------------------------------------------------------------------------- definition in 64 bits

def _turn(x, positions, axis_of, inv_freq, interleaved, conjugate=False):
    """The rotation as a product of complex numbers: (a + ib) e^(i p w), p on the axis of w."""
    x = x.to(torch.float64)
    r = inv_freq.shape[0]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * r].unflatten(-1, (r, 2)).contiguous())
    else:
        z = torch.complex(x[..., :r].contiguous(), x[..., r:2 * r].contiguous())
    for f in range(r):
        p = positions if axis_of is None else positions[axis_of[f]]
        angle = p.to(torch.float64) * inv_freq[f]
        z[..., f] *= torch.exp((-1j if conjugate else 1j) * angle).unsqueeze(-1)
    y = x.clone()
    if interleaved:
        y[..., :2 * r] = torch.view_as_real(z).flatten(-2)
    else:
        y[..., :r], y[..., r:2 * r] = z.real, z.imag
    return y


def _exact_rope(s, case):
    return tuple(_turn(s[n], s["positions"], s["axis_of"], s["inv_freq"], case["interleaved"], case["grad"])
                 for n in ("q", "k"))


def _nearest_e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, ties to even, kept in 64 bits."""
    _, e = torch.frexp(x)   # |x| in [2^(e-1), 2^e): three mantissa bits make steps of 2^(e-4)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return (x / step).round() * step


def _place(s, case, b, at):
    """Page and slot of entries `at` (a list) of sequence b."""
    at = torch.tensor(at, dtype=torch.int64, device="cuda")
    return s["block_table"].long()[b, at // case["page"]], at % case["page"]


def _exact_append(s, case):
    out = dict(q=_turn(s["q"], s["positions"], s["axis_of"], s["inv_freq"], case["interleaved"]))
    places = [_place(s, case, b, list(range(n - len(p), n))) for b, (n, p) in enumerate(_sequences(case))]
    phys, slot = (torch.cat([p[i] for p in places]) for i in range(2))
    for name, x in (("k", _turn(s["k"], s["positions"], s["axis_of"], s["inv_freq"], case["interleaved"])),
                    ("v", s["v"].double())):
        pages = s[name + "_pages"].double()
        if case["pages"] == "e4m3":
            top = x.abs().amax(-1)
            scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(-126, 127))
            exps = s[name + "_exp"].double()
            exps[phys, :, slot] = scale
            out[name + "_exp"] = exps
            x = _nearest_e4m3(x / scale.unsqueeze(-1))
        pages[phys, slot] = x
        out[name + "_pages"] = pages
    return out


def _path(parents, t):
    out = []
    while t >= 0:
        out.append(t)
        t = parents[t]
    return out[::-1]


def _exact_tree(s, case):
    Hq, Hkv, d, W = case["Hq"], case["Hkv"], case["d"], case["W"]
    T = s["q"].shape[0]
    o = torch.zeros((T, Hq, d), device="cuda", dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, device="cuda", dtype=torch.float64)
    first = 0
    for b, ((length, parents), gates) in enumerate(zip(_sequences(case), _gates(case))):
        n = len(parents)
        if n == 0:
            continue
        base = length - n
        seen = torch.zeros((n, length), dtype=torch.bool)
        depth = _depths(parents)
        for t in range(n):
            lo = 0 if gates[t] else max(0, base + depth[t] - W + 1)
            seen[t, min(lo, base):base] = True
            seen[t, :min(case["anchors"], base)] = True
            for u in _path(parents, t):
                if base + depth[u] >= lo or base + depth[u] < case["anchors"]:
                    seen[t, base + u] = True
        phys, slot = _place(s, case, b, list(range(length)))

        def rows(name):
            x = s[name + "_pages"]
            if case["pages"] != "e4m3":
                return x[phys, slot].double().transpose(0, 1)
            u = s[name + "_exp"].view(torch.uint8)[phys, :, slot].double()
            x = x.view(torch.uint8)[phys, slot].view(torch.float8_e4m3fn).double()
            return (x * torch.exp2(u - 127.0).unsqueeze(-1)).transpose(0, 1)

        q = s["q"][first:first + n].double().transpose(0, 1).reshape(Hkv, Hq // Hkv * n, d)
        score = torch.bmm(q, rows("k").transpose(1, 2)).view(Hq, n, length) * d ** -0.5
        score = score.masked_fill(~seen.cuda(), -math.inf)
        lse[first:first + n] = torch.logsumexp(score, -1).transpose(0, 1)
        p = torch.softmax(score, -1).view(Hkv, -1, length)
        o[first:first + n] = torch.bmm(p, rows("v")).view(Hq, n, d).transpose(0, 1)
        first += n
    return dict(o=o, lse=lse)


def _pools(s, case):
    """The pools as 64-bit values."""
    return {name: s[name].double() for name in ("k_pages", "v_pages", "k_exp", "v_exp") if s[name] is not None}


def _exact_accept(s, case):
    out, lens = _pools(s, case), []
    for b, ((length, parents), leaf) in enumerate(zip(_sequences(case), _leaves(case))):
        base, path = length - len(parents), _path(parents, leaf)
        lens.append(base + len(path))
        from_page, from_slot = _place(s, case, b, [base + t for t in path])
        page, slot = _place(s, case, b, list(range(base, base + len(path))))
        for name, x in out.items():
            if name.endswith("pages"):
                x[:, page, slot] = x[:, from_page, from_slot]
            else:
                x[:, page, :, slot] = x[:, from_page, :, from_slot]
    return dict(out, seq_lens=_ints(lens))


def _exact_fork(s, case):
    out, seqs, page = _pools(s, case), _sequences(case), case["page"]
    table, lens = [], []
    rows, new = s["block_table"].tolist(), s["new_page"].tolist()
    for c, b in enumerate(_forks(case)):
        n = seqs[b][0]
        row = list(rows[b])
        old, row[n // page] = row[n // page], new[c]
        table.append(row)
        lens.append(n)
        for name, x in out.items():
            if name.endswith("pages"):
                x[:, new[c], :n % page] = x[:, old, :n % page]
            else:
                x[:, new[c], :, :n % page] = x[:, old, :, :n % page]
    return dict(out, block_table=_ints(table), seq_lens=_ints(lens))


_EXACT = dict(rope=_exact_rope, append=_exact_append, tree=_exact_tree, accept=_exact_accept, fork=_exact_fork)


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)
