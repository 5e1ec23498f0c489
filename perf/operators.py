"""The key/value cache operators, measured: position rotation (with its gradient), appending to a
paged cache, and decode over 8-bit pages.

Every case has a plain form in elementary torch operations (``own`` false) and the calls a user makes
of the package (``own`` true).  Both take the same prepared state.
"""
from __future__ import annotations

import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One 32K prompt of the routed prefill, q and k rotated before it.
        dict(name="rope_prompt_32k", op="rope", grad=False, B=1, N=32768, Hq=16, Hkv=16, d=128, rot=128,
             interleaved=False, packed=False, fused=False, dtype="bf16"),
        # Training, two sequences of 8K with grouped heads: dq and dk of the attention back through the rotation.
        dict(name="rope_grad_2x8k", op="rope", grad=True, B=2, N=8192, Hq=16, Hkv=4, d=128, rot=128,
             interleaved=False, packed=False, fused=False, dtype="bf16"),
        # fp32 check runs: packed documents of odd length, half of each head rotated, views of one projection.
        dict(name="rope_packed_f32", op="rope", grad=False, B=3, N=1001, Hq=6, Hkv=2, d=64, rot=32,
             interleaved=True, packed=True, fused=True, dtype="f32"),
        # A serving batch takes in several prompts of uneven length, straight from the fused projection.
        dict(name="append_prompts_bf16", op="append", B=5, new=1640, prior=3000, Hq=16, Hkv=4, d=128, rot=128,
             interleaved=False, fused=True, page=64, pages="bf16", dtype="bf16", seed=4),
        # One long prompt into 8-bit pages.
        dict(name="append_prompt_32k_e4m3", op="append", B=1, new=32768, prior=0, Hq=16, Hkv=16, d=128, rot=128,
             interleaved=False, fused=False, page=64, pages="e4m3", dtype="bf16", seed=5),
        # A decode step of a batch of sixteen far into their contexts, one token each.
        dict(name="append_step_16_bf16", op="append", B=16, new=1, prior=32000, Hq=16, Hkv=16, d=128, rot=128,
             interleaved=False, fused=True, page=64, pages="bf16", dtype="bf16", seed=6),
        # The smallest call: the next token of a single sequence; latency alone counts.
        dict(name="append_step_1_e4m3", op="append", B=1, new=1, prior=5000, Hq=16, Hkv=4, d=128, rot=128,
             interleaved=False, fused=True, page=64, pages="e4m3", dtype="bf16", seed=7),
        # The decode workload of the benchmark: 16 x 32K, two sequences routed, on 8-bit pages.
        dict(name="decode_16x32k", op="decode", B=16, L=32768, ragged=False, empty=0, routed=2, Hq=16, Hkv=16,
             d=128, W=1024, anchors=0, page=64, seed=8),
        # Every sequence routed, grouped heads: the longest reads.
        dict(name="decode_8x32k_routed", op="decode", B=8, L=32768, ragged=False, empty=0, routed=8, Hq=16, Hkv=4,
             d=128, W=1024, anchors=0, page=64, seed=9),
        # One short sequence: latency alone counts.
        dict(name="decode_1x777", op="decode", B=1, L=777, ragged=False, empty=0, routed=1, Hq=16, Hkv=16,
             d=128, W=256, anchors=0, page=16, seed=10),
        # A padded serving batch: ragged lengths, empty slots, anchors, groups of three, head size 64.
        dict(name="decode_ragged_33", op="decode", B=33, L=5003, ragged=True, empty=2, routed=5, Hq=12, Hkv=4,
             d=64, W=512, anchors=256, page=16, seed=11),
        # A wide batch in its windows with a few routed sequences, eight query heads to a key head.
        dict(name="decode_64_windows", op="decode", B=64, L=8192, ragged=True, empty=0, routed=3, Hq=16, Hkv=2,
             d=128, W=1024, anchors=0, page=32, seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode"])
    d = rng.choice([64, 128])
    if op == "decode":
        G, Hkv = rng.randint(1, 16), rng.randint(1, 16)
        B = _log(rng, 1, 64)
        L = _log(rng, 1, max(1, min(65536, (1 << 28) // (B * Hkv * d))))
        return dict(op=op, B=B, L=L, ragged=rng.random() < 0.6, empty=rng.choice([0, 0, min(1, B - 1)]),
                    routed=rng.randint(0, B), Hq=G * Hkv, Hkv=Hkv, d=d, W=_log(rng, 1, 4096),
                    anchors=rng.choice([0, 0, rng.randint(1, 300)]), page=2 ** rng.randint(0, 8),
                    seed=rng.randrange(1 << 20))
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4])
    rot = 16 * rng.randint(1, d // 16)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = (3 << 24) // ((Hq + 2 * Hkv) * d)   # tokens
    common = dict(Hq=Hq, Hkv=Hkv, d=d, rot=rot, interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                  dtype=dtype)
    if op == "rope":
        T = _log(rng, 1, most)
        B = rng.randint(1, min(4, T))
        return dict(op=op, grad=rng.random() < 0.5, B=B, N=max(1, T // B), packed=rng.random() < 0.5, **common)
    B = _log(rng, 1, 64)
    new = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, most // B))
    return dict(op=op, B=B, new=new, prior=rng.choice([0, _log(rng, 1, 100000)]), page=2 ** rng.randint(0, 8),
                pages="e4m3" if dtype == "bf16" and rng.random() < 0.6 else dtype, seed=rng.randrange(1 << 20),
                **common)


def _lengths(case):
    """Tokens of each sequence that a case is about, the same for every seed of its values: for
    "append" (new, total) per sequence, for "decode" (length, routed) per sequence."""
    rng = random.Random(case["seed"])
    B = case["B"]
    if case["op"] == "append":
        if case["new"] == 1:
            new = [1] * B
        else:   # uneven, of the given mean
            new = [max(1, round(case["new"] * (1.0 if B == 1 else rng.uniform(0.3, 1.7)))) for _ in range(B)]
        return [(n, n + (0 if case["prior"] == 0 else rng.randint(case["prior"] // 2, case["prior"]))) for n in new]
    lens = [rng.randint(1, case["L"]) if case["ragged"] else case["L"] for _ in range(B)]
    routed = set(rng.sample(range(B), min(B, case["routed"])))
    empty = set(rng.sample(range(B), case["empty"]))
    return [(0 if b in empty else lens[b], int(b in routed)) for b in range(B)]


def _visited(case):
    """Cache entries each sequence's query reads."""
    out = []
    for length, routed in _lengths(case):
        lo = 0 if routed else max(0, length - case["W"])
        out.append(length - lo + min(case["anchors"], lo))
    return out


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "decode":
        keys = sum(_visited(case))
        # e4m3 keys and values, an exponent byte for each row; q, o in bf16 and lse
        return {"bytes": keys * Hkv * (2 * d + 2) + case["B"] * Hq * (4 * d + 4), "flops": 4 * keys * Hq * d}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        T = case["B"] * case["N"]
        return {"bytes": 2 * T * (Hq + Hkv) * d * size, "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    T = sum(n for n, _ in _lengths(case))
    row = d + 1 if case["pages"] == "e4m3" else d * size
    return {"bytes": T * (Hq * d * size * 2 + Hkv * (2 * d * size + 2 * row)),
            "flops": 3 * T * (Hq + Hkv) * case["rot"]}


# --------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _heads(rows, case, dtype, g, value=True):
    """q, k (and v) of `rows` tokens: tensors of their own, or views of one fused projection."""
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    counts = [Hq, Hkv] + ([Hkv] if value else [])
    if not case["fused"]:
        return [_randn((*rows, h, d), dtype, g) for h in counts]
    # the projection holds v too, whether this call uses it or not
    x = _randn((*rows, (Hq + 2 * Hkv) * d), dtype, g)
    parts = x.split([Hq * d, Hkv * d, Hkv * d], dim=-1)
    return [p.unflatten(-1, (h, d)) for p, h in zip(parts, counts)]


def _inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)


def _quantise(x):
    """e4m3 values and power-of-two scales (e8m0) of rows along the last dimension: the smallest
    scale 2^e with max |x| <= 448 * 2^e, and the row divided by it, to the nearest e4m3."""
    amax = x.abs().amax(-1)
    mant, expo = torch.frexp(amax)   # amax = mant * 2^expo, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = (expo - 9 + (mant > 0.875)).clamp(-126, 127)
    e = torch.where(amax == 0, torch.full_like(e, -126), e)
    v = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return v, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _prepare_rope(case, g):
    B, N, dtype = case["B"], case["N"], DTYPES[case["dtype"]]
    q, k = _heads((B, N), case, dtype, g, value=False)
    positions = None
    if case["packed"]:   # documents laid end to end: positions start again at each
        ends = torch.rand((B, N), generator=g, device="cuda") < 3.0 / N
        at = torch.arange(N, device="cuda").expand(B, N)
        first = torch.where(ends, at, torch.zeros_like(at)).cummax(-1).values
        positions = (at - first).to(torch.int32)
    return dict(q=q, k=k, positions=positions, inv_freq=_inv_freq(case["rot"]))


def _prepare_append(case, g):
    B, page, Hkv, d = case["B"], case["page"], case["Hkv"], case["d"]
    lens = _lengths(case)
    T = sum(n for n, _ in lens)
    dtype = DTYPES[case["dtype"]]
    q, k, v = _heads((T,), case, dtype, g)
    new = torch.tensor([n for n, _ in lens])
    total = torch.tensor([t for _, t in lens])
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    max_pages = int((total.max() + page - 1) // page)
    # Physical pages for the pages the new tokens fall on, and spare ones; the pages before them, which
    # this call does not touch, are not held here and their table entries are not used.
    first, last = (total - new) // page, (total - 1) // page
    touched = int((last - first + 1).sum())
    num_pages = touched + 8
    perm = torch.randperm(num_pages, generator=g, device="cuda")[:touched].to(torch.int32).cpu()
    table = torch.zeros((B, max_pages), dtype=torch.int32)
    owner = torch.repeat_interleave(torch.arange(B), last - first + 1)
    ahead = (last - first + 1).cumsum(0) - (last - first + 1)
    table[owner, first[owner] + torch.arange(touched) - ahead[owner]] = perm
    state = dict(q=q, k=k, v=v, inv_freq=_inv_freq(case["rot"]),
                 starts=None if case["new"] == 1 else starts.to(torch.int32).cuda(),
                 seq_lens=total.to(torch.int32).cuda(), block_table=table.cuda(), k_exp=None, v_exp=None)
    if case["pages"] == "e4m3":
        for name in ("k", "v"):
            state[name + "_pages"] = torch.zeros((num_pages, page, Hkv, d), device="cuda", dtype=torch.float8_e4m3fn)
            state[name + "_exp"] = torch.full((num_pages, Hkv, page), 127, device="cuda",
                                              dtype=torch.uint8).view(torch.float8_e8m0fnu)
    else:
        for name in ("k", "v"):
            state[name + "_pages"] = torch.zeros((num_pages, page, Hkv, d), device="cuda", dtype=dtype)
    return state


def _prepare_decode(case, g):
    B, page, Hq, Hkv, d = case["B"], case["page"], case["Hq"], case["Hkv"], case["d"]
    lens = _lengths(case)
    longest = max(n for n, _ in lens)
    max_pages = max(1, -(-longest // page))
    held = [-(-n // page) for n, _ in lens]
    num_pages = sum(held) + 2
    perm = torch.randperm(num_pages, generator=g, device="cuda")[:sum(held)].to(torch.int32).cpu()
    table = torch.zeros((B, max_pages), dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    state = dict(q=_randn((B, Hq, d), torch.bfloat16, g), block_table=table.cuda(),
                 seq_lens=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(),
                 gate=torch.tensor([r for _, r in lens], dtype=torch.uint8).cuda())
    for name in ("k", "v"):
        pages = torch.empty((num_pages, page, Hkv, d), device="cuda", dtype=torch.float8_e4m3fn)
        exps = torch.empty((num_pages, Hkv, page), device="cuda", dtype=torch.float8_e8m0fnu)
        some = max(1, (1 << 28) // (page * Hkv * d))   # pages at a time
        for a in range(0, num_pages, some):
            z = min(num_pages, a + some)
            x = torch.randn((z - a, page, Hkv, d), generator=g, device="cuda")
            # rows of a real cache differ in size from token to token
            x *= torch.exp(0.5 * torch.randn((z - a, page, Hkv, 1), generator=g, device="cuda"))
            value, scale = _quantise(x)
            pages.view(torch.uint8)[a:z] = value.view(torch.uint8)
            exps.view(torch.uint8)[a:z] = scale.view(torch.uint8).transpose(1, 2)
        state[name + "_pages"], state[name + "_exp"] = pages, exps
    return state


def prepare(case, seed):
    g = _generator(seed)
    state = {"rope": _prepare_rope, "append": _prepare_append, "decode": _prepare_decode}[case["op"]](case, g)
    state["case"] = case
    return state


# ----------------------------------------------------------------------------------- plain form

def _rotated(x, positions, inv_freq, interleaved, sign=1.0):
    """x [..., H, d] in fp32, rotated by positions [...]; the angles in 64 bits."""
    angle = positions.double()[..., None] * inv_freq
    cos, sin = angle.cos().float()[..., None, :], (sign * angle.sin()).float()[..., None, :]
    rot = 2 * inv_freq.numel()
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s, case):
    positions = s["positions"]
    if positions is None:
        positions = torch.arange(case["N"], device="cuda").expand(case["B"], case["N"])
    sign = -1.0 if case["grad"] else 1.0
    return tuple(_rotated(s[n], positions, s["inv_freq"], case["interleaved"], sign).to(s[n].dtype) for n in "qk")


def _token_places(s, case):
    """Position of every new token and the row of the pool (page * page_size + slot) it goes to."""
    T, B = s["k"].shape[0], case["B"]
    starts = s["starts"] if s["starts"] is not None else torch.arange(B + 1, device="cuda")
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:].contiguous().long(), t, right=True)
    pos = s["seq_lens"].long()[b] - (starts.long()[b + 1] - t)
    page = case["page"]
    return pos, s["block_table"].long()[b, pos // page] * page + pos % page


def _plain_append(s, case):
    pos, row = _token_places(s, case)
    q = _rotated(s["q"], pos, s["inv_freq"], case["interleaved"]).to(s["q"].dtype)
    out = dict(q=q)
    for name, x in (("k", _rotated(s["k"], pos, s["inv_freq"], case["interleaved"])), ("v", s["v"].float())):
        pages = s[name + "_pages"]
        if case["pages"] == "e4m3":
            value, scale = _quantise(x)
            pages.view(torch.uint8).flatten(0, 1)[row] = value.view(torch.uint8)
            exps, page = s[name + "_exp"], case["page"]
            exps.view(torch.uint8)[row // page, :, row % page] = scale.view(torch.uint8)
            out[name + "_exp"] = exps
        else:
            pages.flatten(0, 1)[row] = x.to(pages.dtype)
        out[name + "_pages"] = pages
    return out


def _visible(s, case, width):
    """[B, width] which cache entries the query of each sequence reads."""
    at = torch.arange(width, device="cuda")[None]
    n = s["seq_lens"].long()[:, None]
    near = (at >= n - case["W"]) | (at < case["anchors"]) | (s["gate"] != 0)[:, None]
    return near & (at < n)


def _plain_decode(s, case):
    B, page, Hq, Hkv, d = case["B"], case["page"], case["Hq"], case["Hkv"], case["d"]
    table = s["block_table"].long()
    width = table.shape[1] * page

    def entries(name):
        value = s[name + "_pages"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        scale = s[name + "_exp"].view(torch.uint8)[table].view(torch.float8_e8m0fnu).float()
        return (value * scale.transpose(2, 3)[..., None]).view(B, width, Hkv, d)

    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    score = torch.einsum("bhgd,blhd->bhgl", q, entries("k")) / math.sqrt(d)
    seen = _visible(s, case, width)
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    some = seen.any(-1)[:, None, None, None]
    top = torch.where(some, score.amax(-1, keepdim=True), torch.zeros((), device="cuda"))
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", p, entries("v")) / torch.where(some, total, torch.ones((), device="cuda"))
    lse = (top + total.log()).view(B, Hq)
    return dict(o=o.view(B, Hq, d).to(s["q"].dtype), lse=lse)


# ------------------------------------------------------------------------- the package's operators

def _own_rope(s, case):
    import sliding_window_attention_router_gb300 as swa
    call = swa.rope_backward if case["grad"] else swa.rope
    return call(s["q"], s["k"], s["inv_freq"], positions=s["positions"], interleaved=case["interleaved"])


def _own_append(s, case):
    import sliding_window_attention_router_gb300 as swa
    q = swa.append_paged(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"],
                         s["inv_freq"], starts=s["starts"], interleaved=case["interleaved"],
                         k_exp=s["k_exp"], v_exp=s["v_exp"])
    out = dict(q=q, k_pages=s["k_pages"], v_pages=s["v_pages"])
    if s["k_exp"] is not None:
        out.update(k_exp=s["k_exp"], v_exp=s["v_exp"])
    return out


def _own_decode(s, case):
    import sliding_window_attention_router_gb300 as swa
    if "workspace" not in s:   # kept from step to step, as a serving loop does
        nbytes = swa.decode_paged_e4m3_workspace(case["B"], s["block_table"].shape[1], case["page"], case["Hq"],
                                                 case["Hkv"], case["d"], case["W"], case["anchors"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    o, lse = swa.decode_paged_e4m3(s["q"], s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"], s["block_table"],
                                   s["seq_lens"], s["gate"], case["W"], n_anchor=case["anchors"], want_lse=True,
                                   workspace=s["workspace"])
    return dict(o=o, lse=lse)


def run(state):
    case = state["case"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "decode": _own_decode}[case["op"]](state, case)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[case["op"]](state, case)


# ------------------------------------------------------------------------- definition in 64 bits

def _turn(x, pos, inv_freq, interleaved, conjugate=False):
    """The rotation as a product of complex numbers: (a + ib) e^(i pos w)."""
    x = x.to(torch.float64)
    r = inv_freq.shape[0]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * r].unflatten(-1, (r, 2)).contiguous())
    else:
        z = torch.complex(x[..., :r].contiguous(), x[..., r:2 * r].contiguous())
    turns = torch.outer(pos.reshape(-1).to(torch.float64), -inv_freq if conjugate else inv_freq)
    z = z * torch.exp(1j * turns).view(*pos.shape, 1, r)
    y = x.clone()
    if interleaved:
        y[..., :2 * r] = torch.view_as_real(z).flatten(-2)
    else:
        y[..., :r], y[..., r:2 * r] = z.real, z.imag
    return y


def _exact_rope(s, case):
    B, N = case["B"], case["N"]
    pos = s["positions"] if case["packed"] else torch.arange(B * N, device="cuda").remainder(N).view(B, N)
    return tuple(_turn(s[n], pos, s["inv_freq"], case["interleaved"], case["grad"]) for n in ("q", "k"))


def _nearest_e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, ties to even, kept in 64 bits."""
    _, e = torch.frexp(x)   # |x| in [2^(e-1), 2^e): three mantissa bits make steps of 2^(e-4)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return (x / step).round() * step


def _exact_append(s, case):
    lens, page = _lengths(case), case["page"]
    pos = torch.cat([torch.arange(t - n, t) for n, t in lens]).cuda()
    owner = torch.repeat_interleave(torch.arange(case["B"]), torch.tensor([n for n, _ in lens])).cuda()
    phys, slot = s["block_table"].long()[owner, pos // page], pos % page
    out = dict(q=_turn(s["q"], pos, s["inv_freq"], case["interleaved"]))
    for name, x in (("k", _turn(s["k"], pos, s["inv_freq"], case["interleaved"])), ("v", s["v"].double())):
        pages = s[name + "_pages"].double()
        if case["pages"] == "e4m3":
            top = x.abs().amax(-1)
            e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(-126, 127)
            scale = torch.exp2(e)
            exps = s[name + "_exp"].double()
            exps[phys, :, slot] = scale
            out[name + "_exp"] = exps
            x = _nearest_e4m3(x / scale.unsqueeze(-1))
        pages[phys, slot] = x
        out[name + "_pages"] = pages
    return out


def _exact_decode(s, case):
    B, page, Hq, Hkv, d = case["B"], case["page"], case["Hq"], case["Hkv"], case["d"]
    o = torch.zeros((B, Hq, d), device="cuda", dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, device="cuda", dtype=torch.float64)
    for b, (n, routed) in enumerate(_lengths(case)):
        if n == 0:
            continue
        lo = 0 if routed else max(0, n - case["W"])
        at = torch.tensor(list(range(min(case["anchors"], lo))) + list(range(lo, n)), device="cuda")
        phys, slot = s["block_table"].long()[b, at // page], at % page

        def rows(name):
            x = s[name + "_pages"].view(torch.uint8)[phys, slot].view(torch.float8_e4m3fn).double()
            u = s[name + "_exp"].view(torch.uint8)[phys, :, slot].double()
            return (x * torch.exp2(u - 127.0).unsqueeze(-1)).transpose(0, 1).repeat_interleave(Hq // Hkv, 0)

        score = torch.bmm(rows("k"), s["q"][b].double().unsqueeze(-1)).squeeze(-1) * d ** -0.5
        lse[b] = torch.logsumexp(score, -1)
        o[b] = torch.bmm(torch.softmax(score, -1).unsqueeze(1), rows("v")).squeeze(1)
    return dict(o=o, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode}[case["op"]](s, case)
