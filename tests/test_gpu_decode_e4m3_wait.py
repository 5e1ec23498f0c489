"""Failure detection of decode over 8-bit pages, without a fault: a wait for rows that runs out.

Under a limit of 1 ns a warp only polls for its tiles (it does not suspend, not even at first), a few
times in well under a microsecond, while the rows come from memory that the L2 does not hold: the first
waits give up, the warps wait for their own copies in flight and leave.  The call is then over, the
status is a timeout, and under the default limit the next call in the same context is right."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

SWIATTN_ETIMEOUT = 4


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_router_gb300 as m
    return m


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 128), (24, 2, 64)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(swa, Hq, Hkv, d):
    B, L, page = 4, 20000, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    P = B * -(-L // page)
    table = torch.randperm(P, generator=g, device="cuda").to(torch.int32).view(B, -1)
    pages = [torch.randn((P, page, Hkv, d), generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in "kv"]
    exps = [torch.full((P, Hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in "kv"]
    q = torch.randn((B, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    gate = torch.ones(B, dtype=torch.uint8, device="cuda")

    def call():
        return swa.decode_paged_e4m3(q, *pages, *exps, table, lens, gate, 64, want_lse=True)

    assert swa.get_device_error() == 0
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()   # larger than the L2
    swa.set_wait_limit_ns(1)
    try:
        call()
        torch.cuda.synchronize()
        assert swa.get_device_error() == SWIATTN_ETIMEOUT
    finally:
        swa.set_wait_limit_ns(0)
    o, lse = call()
    assert swa.get_device_error() == 0
    k, v = (p.view(P, page, Hkv, d)[table.long()].view(B, -1, Hkv, d)[:, :L].double().transpose(1, 2) for p in pages)
    G = Hq // Hkv
    for b in range(B):
        kb, vb, qb = k[b].repeat_interleave(G, 0), v[b].repeat_interleave(G, 0), q[b].double()[:, :, None]
        s = (kb @ qb)[..., 0] / math.sqrt(d)
        p = torch.softmax(s, -1)[:, None]
        want, absum = (p @ vb)[:, 0], (p @ vb.abs())[:, 0]
        # the bound of test_gpu_decode_e4m3; all weights are within 2^21 of the largest but a few of e^-15
        # of it, each off by 2^-32 of it, times a value under 8
        r = d * 2.0 ** -22 * (kb.abs() @ qb.abs())[..., 0].amax(-1) / math.sqrt(d) + 2.0 ** -21
        tol = (2 * r + 2.0 ** -11)[:, None] * absum + 2.0 ** -8 * want.abs() + L * 8 * 2.0 ** -32 * p.amax()
        assert bool(((o[b].double() - want).abs() <= tol).all())
        assert bool(((lse[b].double() - torch.logsumexp(s, -1)).abs() <= r + 2.0 ** -13).all())
