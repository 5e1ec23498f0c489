"""Decode over 8-bit pages where a warp walks 33 tiles and more of one sequence: the look-up of page
numbers 32 tiles at a time, a ring that wraps many times, references raised in the last tile.

So many (sequence, key head)s that the call cuts little or nothing: the length of its blocks is read
back from the workspace and must be at least 33 tiles.  References in 64 bits on the GPU, from the
definition, one sequence at a time.

Exact form: scores are whole numbers in base 2 (0 .. -4, the last key 16), so all weights are powers
of two and exact in fp16; the last key's value row is zero in the even dimensions, which therefore
hold what the rescaling by 2^-16 of the long sum before it leaves.  What is left to round: one fp32
step of 2^-23 for each tile and part (under 100), exponentials (2^-22) and bf16: 2^-15 of the sum of
absolute terms and 2^-8 of the result.  A tile lost or read twice is off by 2^-7 of that sum.
Random form: the bound of test_gpu_decode_e4m3, but what fp16 does not hold fully is counted where it
is: the weights of the values (with their rows' powers of two) under 2^-21 of the largest, each off by
at most 2^-32 of the largest (half the subnormal step 2^-24, the largest being at least 2^7), times
the 8-bit value.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_router_gb300 as m
    return m


class Pool:
    def __init__(self, B, Hq, Hkv, d, page, longest, W, S, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.B, self.Hq, self.Hkv, self.d, self.page, self.W, self.S = g, B, Hq, Hkv, d, page, W, S
        per = -(-longest // page)
        lens = [longest - (7 * b) % 41 for b in range(B)]
        lens[B // 2] = 0
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.gate = (torch.arange(B, device="cuda") % 3 != 0).to(torch.uint8)
        P = B * per + 3
        self.table = torch.randperm(P, generator=g, device="cuda")[:B * per].to(torch.int32).view(B, per)
        self.seen = torch.zeros((P, page), dtype=torch.bool, device="cuda")
        for b in range(B):
            at = self.visited(b)
            self.seen[self.table[b].long()[at // page], at % page] = True
        shape = (P, page, Hkv, d)
        self.k, self.v = (torch.randn(shape, generator=g, device="cuda") for _ in "kv")
        self.ke, self.ve = (torch.randint(125, 130, (P, Hkv, page), generator=g, device="cuda") for _ in "kv")

    def visited(self, b):
        n = int(self.lens[b])
        lo = 0 if int(self.gate[b]) else max(0, n - self.W)
        return torch.cat([torch.arange(min(self.S, lo)), torch.arange(lo, n)]).cuda()

    def rows(self, b, at):
        return self.table[b].long()[at // self.page], at % self.page

    def run(self, swa, q, scale):
        """Values and exponents as they are held, rows that are not visited made NaN; the call; the reference."""
        pages, exps = [], []
        for x, e in ((self.k, self.ke), (self.v, self.ve)):
            codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
            codes[~self.seen] = 0x7f
            e = torch.where(self.seen[:, None, :], e, 255).to(torch.uint8)
            pages.append(codes.view(torch.float8_e4m3fn))
            exps.append(e.contiguous())
        nbytes = swa.decode_paged_e4m3_workspace(self.B, self.table.shape[1], self.page, self.Hq, self.Hkv, self.d,
                                                 self.W, self.S)
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        o, lse = swa.decode_paged_e4m3(q, *pages, *exps, self.table, self.lens, self.gate, self.W, scale=scale,
                                       want_lse=True, n_anchor=self.S, workspace=ws)
        assert swa.get_device_error() == 0
        parts = 2432 + self.B * self.Hkv
        plan = (parts * (self.Hq // self.Hkv) * (self.d + 4) * 4 + 255) // 256 * 256
        assert int(ws[plan + 4 * self.B:plan + 4 * self.B + 4].view(torch.int32)) >= 33
        G = self.Hq // self.Hkv
        for b in range(self.B):
            at = self.visited(b)
            if len(at) == 0:
                assert bool((o[b] == 0).all()) and bool(torch.isneginf(lse[b]).all())
                continue
            phys, slot = self.rows(b, at)
            k, v = (p[phys, slot].double() * torch.exp2(e[phys, :, slot].double() - 127)[..., None]
                    for p, e in zip(pages, exps))
            k, v = (x.transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))   # [Hq, n, d]
            qb = q[b].double()[:, :, None]
            s = scale * (k @ qb)[..., 0]
            p = torch.softmax(s, -1)
            size = scale * (k.abs() @ qb.abs())[..., 0].amax(-1)
            power = torch.exp2(exps[1][phys, :, slot].double() - 127).t().repeat_interleave(G, 0)
            weight = p * power
            top = weight.amax(-1, keepdim=True)
            small = torch.where(weight < 2.0 ** -21 * top, 2.0 ** -32 * top / power, 0.0)
            yield (b, o[b].double(), lse[b].double(), (p[:, None] @ v)[:, 0], torch.logsumexp(s, -1),
                   (p[:, None] @ v.abs())[:, 0], size, (small[:, None] @ v.abs())[:, 0])


SHAPES = [
    (80, 16, 16, 64, 64, 1130, 1050, 20),     # one group of heads, tiles by whole pages
    (82, 15, 15, 128, 4, 600, 560, 33),       # pages under a tile
    (45, 9 * 14, 14, 128, 16, 1100, 1020, 0),  # two groups of heads
    (41, 16 * 15, 15, 64, 8, 570, 545, 5),
]


@pytest.mark.parametrize("B,Hq,Hkv,d,page,longest,W,S", SHAPES)
def test_long_runs_exactly(swa, B, Hq, Hkv, d, page, longest, W, S):
    c = Pool(B, Hq, Hkv, d, page, longest, W, S, seed=41)
    c.k.zero_()
    c.ke.fill_(127)
    c.k[..., 8] = -torch.randint(0, 5, c.k.shape[:-1], generator=c.g, device="cuda").float()
    for b in range(B):
        if int(c.lens[b]):
            row = c.rows(b, c.visited(b)[-1:])
            c.k[row] = 0
            c.k[row[0], row[1], :, 8] = 16
            c.v[row[0], row[1], :, 0::2] = 0
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    q[..., 8] = 1
    for b, o, lse, want, want_lse, absum, _, _ in c.run(swa, q, math.log(2.0)):
        err = (o - want).abs()
        assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * absum).all()), (b, float((err / absum).max()))
        assert bool(((lse - want_lse).abs() <= 2.0 ** -15).all()), b


@pytest.mark.parametrize("B,Hq,Hkv,d,page,longest,W,S", SHAPES)
def test_long_runs_of_random_scores(swa, B, Hq, Hkv, d, page, longest, W, S):
    c = Pool(B, Hq, Hkv, d, page, longest, W, S, seed=42)
    q = (0.5 * torch.randn((B, Hq, d), generator=c.g, device="cuda")).to(torch.bfloat16)
    for b, o, lse, want, want_lse, absum, size, small in c.run(swa, q, 1.0 / math.sqrt(d)):
        r = d * 2.0 ** -22 * size + 2.0 ** -21
        err = (o - want).abs()
        tol = (2 * r + 2.0 ** -11)[:, None] * absum + small + 2.0 ** -8 * want.abs()
        assert bool((tol < 2.0 ** -6 * absum).all())
        assert bool((err <= tol).all()), (b, float((err / tol).max()))
        assert bool(((lse - want_lse).abs() <= r + 2.0 ** -13).all()), b
