"""GPU parity of the position rotation (swiattn_rope) and its gradient against the 64-bit
reference, element by element.

Tolerance.  A rotated value is m (a c - b s) in fp32: the cosine and sine carry at most 2 units of
2^-24 from the function and 0.4 from the angle's rounding (2^-28 of a turn), their product with m
one half step (2^-24), the two products and the sum one more each: under 6 * 2^-24 of m (|a| + |b|).
The store to bf16 adds half a step, 2^-8 of the value.  A copied dimension is exact.
"""
import math

import numpy as np
import pytest
import torch

import oracle
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


def check(got, x, pos, w, interleaved, factor, transposed, dtype):
    want = ref.rotate(f64(x), pos, w.numpy(), interleaved, factor, transposed)
    tol = 6 * 2.0 ** -24 * abs(factor) * ref.pair_sums(f64(x), w.numpy(), interleaved)
    if dtype == torch.bfloat16:
        tol[..., :2 * len(w)] += 2.0 ** -8 * (np.abs(want[..., :2 * len(w)]) + tol[..., :2 * len(w)])
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (err.max(), np.max(err - tol))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", [(1, 1, 1, 1, 64, 64), (1, 1, 16, 4, 128, 128), (2, 37, 3, 2, 64, 16),
                                              (3, 129, 5, 1, 128, 48), (1, 300, 33, 7, 128, 112)])
def test_rope_matches_reference(swa, B, N, Hq, Hkv, d, rot, dtype, interleaved, grad):
    g = inp._gen(B * 1000 + N + rot)
    q, k = inp.randn((B, N, Hq, d), dtype, g), inp.randn((B, N, Hkv, d), dtype, g)
    w = freqs(rot)
    call = swa.rope_backward if grad else swa.rope
    qo, ko = call(q.cuda(), k.cuda(), w.cuda(), interleaved=interleaved, factor=1.25)
    pos = np.broadcast_to(np.arange(N), (B, N))
    for got, x in ((qo, q), (ko, k)):
        check(got, x, pos, w, interleaved, 1.25, grad, dtype)


def test_rope_far_and_negative_positions(swa):
    """Positions up to 2^30 and below zero: the angle is exact modulo a turn, so the tolerance does
    not grow with the position.  The reference angle goes through rational arithmetic."""
    from fractions import Fraction
    positions = [0, 1, -1, 65535, 1 << 20, (1 << 20) + 1, 123456789, 1 << 30, -(1 << 30), (1 << 31) - 1]
    w = freqs(64)
    g = inp._gen(5)
    x = inp.randn((1, len(positions), 2, 64), torch.float32, g)
    got, _ = swa.rope(x.cuda(), None, w.cuda(), positions=torch.tensor([positions], dtype=torch.int32).cuda())
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    theta = np.zeros((len(positions), 32))
    for i, p in enumerate(positions):
        for f in range(32):
            a = Fraction(float(w[f])) * p / two_pi
            theta[i, f] = float((a - math.floor(a)) * two_pi)
    c, s = np.cos(theta)[None, :, None], np.sin(theta)[None, :, None]
    a, b = f64(x)[..., :32], f64(x)[..., 32:]
    want = np.concatenate([a * c - b * s, b * c + a * s], -1)
    # a frequency's 64-bit fraction is right to 2^-63 of a turn: 2^-32 at position 2^31
    tol = (6 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -31) * ref.pair_sums(f64(x), w.numpy())
    assert np.all(np.abs(f64(got) - want) <= tol)


def test_rope_views_positions_and_in_place(swa):
    """Views of a fused projection, packed positions, only k, outputs in place: the same bits as
    the contiguous call."""
    B, N, Hq, Hkv, d = 2, 75, 6, 2, 64
    g = inp._gen(6)
    qkv = inp.randn((B, N, (Hq + 2 * Hkv) * d), torch.bfloat16, g).cuda()
    q = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
    k = qkv[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    w = freqs(32).cuda()
    pos = torch.randint(0, 1 << 17, (B, N), generator=g, dtype=torch.int32).cuda()
    qo, ko = swa.rope(q.contiguous(), k.contiguous(), w, positions=pos)
    for got, want in zip(swa.rope(q, k, w, positions=pos), (qo, ko)):
        assert torch.equal(got, want)
    assert swa.rope(q, None, w, positions=pos)[1] is None
    assert torch.equal(swa.rope(None, k, w, positions=pos)[1], ko)
    v_before = qkv[..., (Hq + Hkv) * d:].clone()
    r = swa.rope(q, k, w, positions=pos, out=(q, k))
    assert r[0] is q and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[..., (Hq + Hkv) * d:], v_before)


def test_rope_keeps_nan_and_infinity_in_their_pair(swa):
    x = torch.ones((1, 3, 2, 64))
    x[0, 1, 0, 3] = float("nan")
    x[0, 2, 1, 40] = float("inf")
    for interleaved in (False, True):
        got, _ = swa.rope(x.cuda(), None, freqs(64).cuda(), interleaved=interleaved)
        bad = ~torch.isfinite(got.cpu())
        want = torch.zeros_like(bad)
        want[0, 1, 0, [3, 2] if interleaved else [3, 35]] = True
        want[0, 2, 1, [40, 41] if interleaved else [8, 40]] = True
        assert torch.equal(bad, want)


def test_rope_on_another_stream_and_in_a_graph(swa):
    q = inp.randn((1, 500, 4, 128), torch.bfloat16, inp._gen(7)).cuda()
    w = freqs(128).cuda()
    want, _ = swa.rope(q, None, w)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        swa.rope(q, None, w, out=(out, None))
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.rope(q, None, w, out=(out, None))
    q2 = inp.randn((1, 500, 4, 128), torch.bfloat16, inp._gen(8)).cuda()
    want2, _ = swa.rope(q2, None, w)
    q.copy_(q2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_training_run_rope_prefill_and_back(swa):
    """rope -> prefill -> prefill_backward -> rope_backward against differences of the 64-bit
    forward: the loss is linear in the output, the derivative along a random direction of the
    unrotated q and k is checked.  fp32, so that the differences mean something."""
    B, N, Hq, Hkv, d, W = 1, 48, 4, 2, 64, 9
    g = inp._gen(9)
    q, k, v = inp.attention_qkv(B, N, Hq, Hkv, d, torch.float32, g)
    gate = inp.bernoulli_gates((B, N), 0.3, g)
    do = inp.randn((B, N, Hq, d), torch.float32, g)
    w, scale = freqs(32), 1.0 / math.sqrt(d)
    qr, kr = swa.rope(q.cuda(), k.cuda(), w.cuda())
    o, lse = swa.prefill(qr, kr, v.cuda(), gate.cuda(), W, want_lse=True)
    dqr, dkr, _ = swa.prefill_backward(qr, kr, v.cuda(), gate.cuda(), o, lse, do.cuda(), W)
    dq, dk = swa.rope_backward(dqr, dkr, w.cuda())
    assert swa.get_device_error() == 0
    pos = np.arange(N)[None]

    def loss(q_, k_):
        out = oracle.prefill(ref.rotate(q_, pos, w.numpy()), ref.rotate(k_, pos, w.numpy()), f64(v),
                             gate.numpy(), W, scale)
        return float(np.sum(f64(do) * out))

    r = np.random.default_rng(10)
    for _ in range(3):
        uq, uk = r.standard_normal(q.shape), r.standard_normal(k.shape)
        h = 1e-4   # central differences: error h^2 f''' / 6, about 1e-8 of the derivative here
        want = (loss(f64(q) + h * uq, f64(k) + h * uk) - loss(f64(q) - h * uq, f64(k) - h * uk)) / (2 * h)
        got = float(np.sum(f64(dq) * uq) + np.sum(f64(dk) * uk))
        # the fp32 gradients carry at most 1e-4 an element (the fp32 bound of the backward)
        assert abs(got - want) <= 1e-4 * math.sqrt(dq.numel() + dk.numel()), (got, want)
    # and the rotation's own gradient equals the reference's map of the attention's gradients
    check(dq, dqr.cpu(), pos, w, False, 1.0, True, torch.float32)
    check(dk, dkr.cpu(), pos, w, False, 1.0, True, torch.float32)


def test_rope_refusals(swa):
    q = torch.zeros((1, 4, 2, 128), device="cuda", dtype=torch.bfloat16)
    w = freqs(128).cuda()
    bad = [
        dict(q=q.cpu()), dict(q=q[0]), dict(inv_freq=w.float()), dict(inv_freq=freqs(24).cuda()),
        dict(inv_freq=freqs(256).cuda()), dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
        dict(positions=torch.zeros(4, dtype=torch.int64, device="cuda")), dict(k=q.float()),
        dict(k=torch.zeros((1, 4, 2, 64), device="cuda", dtype=torch.bfloat16)), dict(q=None),
        dict(q=q.transpose(1, 2)), dict(q=q[:, :1].expand(1, 4, 2, 128)), dict(factor=float("nan")),
        dict(out=(q[:, :3], None)), dict(out=(q, q)), dict(q=torch.zeros((1, 4, 2, 96), device="cuda", dtype=torch.bfloat16)),
    ]
    for change in bad:
        args = dict(q=q, k=None, inv_freq=w)
        args.update(change)
        with pytest.raises((ValueError, swa.SwiAttnError)):
            swa.rope(**args)
    assert swa.get_device_error() == 0
    for B, N in ((0, 4), (2, 0)):   # nothing to rotate
        e = torch.zeros((B, N, 2, 128), device="cuda", dtype=torch.bfloat16)
        assert swa.rope(e, e, w)[0].shape == e.shape
