"""The training sequence in bf16 on one stream, nothing waited for in between: prefill_backward, then
rope_backward and append_paged on what it wrote.  Both are launched so early that the order of the
grids before them counts.  Every gradient is equal, bit by bit, to that of the same calls with the
stream waited for after each; every round has a gradient of its own in the same buffers, so one read
too early shows."""
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


@pytest.mark.parametrize("B,N,Hq,Hkv,W,rounds", [
    (1, 40, 2, 1, 16, 30),          # one item
    (1, 300, 4, 2, 64, 30),         # a few
    (2, 2048, 8, 1, 256, 20),       # fewer dK/dV items than SMs, each long
    (2, 4096, 16, 4, 1024, 10),     # more than the GPU takes at once
])
def test_gradients_of_the_training_sequence_in_order(swa, B, N, Hq, Hkv, W, rounds):
    d, page = 128, 64
    g = inp._gen(N + Hq)
    q, k, v = (t.cuda() for t in inp.attention_qkv(B, N, Hq, Hkv, d, torch.bfloat16, g))
    gate = inp.bernoulli_gates((B, N), 0.2, g).cuda()
    w = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    d_os = [inp.randn((B, N, Hq, d), torch.bfloat16, g).cuda() for _ in range(3)]
    qr, kr = swa.rope(q, k, w)
    o, lse = swa.prefill(qr, kr, v, gate, W, want_lse=True)
    ws = torch.empty(swa.prefill_backward_workspace(B, N, Hq, Hkv, d, W, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    outs = tuple(torch.empty_like(t) for t in (q, k, v))
    per = -(-N // page)
    table = torch.arange(B * per, dtype=torch.int32).view(B, per).cuda()
    lens = torch.full((B,), N, dtype=torch.int32).cuda()
    starts = (torch.arange(B + 1, dtype=torch.int32) * N).cuda()
    pages = [torch.zeros((B * per, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def step(d_o, wait):
        dq, dk, dv = swa.prefill_backward(qr, kr, v, gate, o, lse, d_o, W, outs=outs, workspace=ws)
        wait()
        back = swa.rope_backward(dq, dk, w)
        wait()
        # the next grid's prerequisite is the rotation now; the backward again, then the append
        swa.prefill_backward(qr, kr, v, gate, o, lse, d_o, W, outs=outs, workspace=ws)
        wait()
        swa.append_paged(None, dk.flatten(0, 1), dv.flatten(0, 1), *pages, table, lens, starts=starts)
        wait()
        return [*back, pages[0].clone(), pages[1].clone()]

    want = [step(d_o, torch.cuda.synchronize) for d_o in d_os]
    # the waited-for run against the definitions: the map of dk as read, the pages a copy of dk and dv
    dk, dv = outs[1], outs[2]
    for got, x in ((want[-1][2], dk), (want[-1][3], dv)):
        assert torch.equal(got.view(B, per * page, Hkv, d)[:, :N], x)
    exact = ref.rotate(dk.double().cpu().numpy(), np.arange(N)[None], w.cpu().numpy(), transposed=True)
    tol = 2.0 ** -8 * np.abs(exact) + 8 * 2.0 ** -24 * ref.pair_sums(dk.double().cpu().numpy(), w.cpu().numpy())
    assert np.all(np.abs(want[-1][1].double().cpu().numpy() - exact) <= tol)
    torch.cuda.synchronize()
    for i in range(rounds):
        got = step(d_os[i % 3], lambda: None)
        for a, b in zip(got, want[i % 3]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), i
    assert swa.get_device_error() == 0
