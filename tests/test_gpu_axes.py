"""GPU parity of the rotation with several axes (swiattn_rope_axes), its gradient, and the append at
given positions (swiattn_append_paged_at).

Tolerances as for the rotation (test_gpu_rope): the axis only chooses the position, so a rotated
value is off by at most 6 * 2^-24 m (|a| + |b|), and half a bf16 step, 2^-8 of the value, where it
is stored as bf16.  An e4m3 value is the nearest to that: half a step, 2^-4 of the value or 2^-10 of
the row's scale.
"""
import numpy as np
import pytest
import torch

import swiattn_inputs as inp
from oracle import kvcache as ref
from test_gpu_append import KINDS, Setup, f64, freqs, raw, swa  # noqa: F401  (swa: the fixture)

pytestmark = pytest.mark.gpu


def sections(half, A, spread):
    return [f % A if spread else f * A // half for f in range(half)]


def near(got, x, pos, axes, w, interleaved, factor, transposed, dtype):
    want = ref.rotate_axes(f64(x), pos, axes, w.numpy(), interleaved, factor, transposed)
    r = 2 * len(w)
    tol = 6 * 2.0 ** -24 * abs(factor) * ref.pair_sums(f64(x), w.numpy(), interleaved)
    if dtype == torch.bfloat16:
        tol[..., :r] += 2.0 ** -8 * (np.abs(want[..., :r]) + tol[..., :r])
    assert np.all(np.abs(f64(got) - want) <= tol)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,A,spread", [
    (1, 1, 1, 1, 64, 16, 2, True), (1, 1, 16, 4, 128, 128, 3, False), (2, 37, 3, 2, 64, 48, 3, True),
    (3, 129, 5, 1, 128, 48, 1, False), (1, 300, 33, 7, 128, 112, 4, False), (2, 65, 2, 2, 128, 128, 64, True)])
def test_rope_axes_match_reference(swa, B, N, Hq, Hkv, d, rot, A, spread, dtype, interleaved, grad):
    g = inp._gen(B * 1000 + N + rot + A)
    q, k = inp.randn((B, N, Hq, d), dtype, g), inp.randn((B, N, Hkv, d), dtype, g)
    pos = torch.randint(-3000, 40000, (A, B, N), generator=g, dtype=torch.int32)
    w, axes = freqs(rot), sections(rot // 2, A, spread)
    call = swa.rope_backward if grad else swa.rope
    qo, ko = call(q.cuda(), k.cuda(), w.cuda(), positions=pos.cuda(), axes=axes, interleaved=interleaved, factor=1.25)
    for got, x in ((qo, q), (ko, k)):
        near(got, x, pos.numpy(), axes, w, interleaved, 1.25, grad, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_axes_that_agree_are_one(swa, interleaved):
    """Bit for bit, also with more axes than are used, axes given as a tensor, views, in place."""
    g = inp._gen(11)
    x = inp.randn((2, 70, 8 * 64), torch.bfloat16, g).cuda()
    q, k = x[..., :6 * 64].unflatten(-1, (6, 64)), x[..., 6 * 64:].unflatten(-1, (2, 64))
    pos = torch.randint(0, 1 << 17, (2, 70), generator=g, dtype=torch.int32).cuda()
    w = freqs(64).cuda()
    want = swa.rope(q, k, w, positions=pos, interleaved=interleaved)
    axes = torch.tensor(sections(32, 3, True))
    many = pos[None].repeat(5, 1, 1)
    got = swa.rope(q, k, w, positions=many, axes=axes, interleaved=interleaved, out=(q, k))
    assert got[0] is q and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rope_axes_gradient_is_that_of_differences(swa):
    """The map is linear: <y, R(x + e) - R(x)> = <R' y, e>, up to the 6 * 2^-24 of each element's
    pair on either side (and 2^-23 for the sums in 64 bits, which is nothing)."""
    g = inp._gen(12)
    w, axes = freqs(48).cuda(), sections(24, 3, False)
    pos = torch.randint(0, 9000, (3, 2, 33), generator=g, dtype=torch.int32).cuda()
    x, e, y = (inp.randn((2, 33, 3, 64), torch.float32, g).cuda() for _ in range(3))
    a, b = (swa.rope(t, None, w, positions=pos, axes=axes)[0].double() for t in (x + e, x))
    back = swa.rope_backward(y, None, w, positions=pos, axes=axes)[0].double()
    size = lambda t: torch.from_numpy(ref.pair_sums(f64(t), freqs(48).numpy())).cuda()   # noqa: E731
    lim = 6 * 2.0 ** -24 * (y.double().abs() * (size(x + e) + size(x)) + size(y) * e.double().abs())
    lim += 2.0 ** -24 * y.double().abs() * size(x + e)   # x + e itself is rounded
    assert abs(((a - b) * y.double()).sum() - (back * e.double()).sum()) <= lim.sum()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,rot,A,interleaved", [
    ([1], [1], 1, 1, 64, 1, 64, 1, False),
    ([9], [777], 16, 4, 128, 64, 128, 1, False),
    ([5, 1, 0, 33], [5, 100, 7, 97], 3, 1, 64, 16, 16, 3, True),
    ([130, 57], [130, 600], 4, 4, 128, 32, 96, 4, False),
    ([1, 2, 3] * 15, [50, 2, 35] * 15, 5, 5, 64, 4, 32, 2, True),   # more sequences than a warp
    ([21, 9], [70, 9], 24, 8, 128, 16, 80, 3, False),               # more heads than one block takes
])
def test_append_at_positions(swa, new, total, Hq, Hkv, d, page, rot, A, interleaved, kind):
    s = Setup(new, total, Hq, Hkv, d, page, kind, seed=sum(new) + rot + A, pad=3, fused=True)
    g = inp._gen(99)
    w, axes = freqs(rot), sections(rot // 2, A, True)
    pos = torch.randint(-9, 70000, (A, s.T), generator=g, dtype=torch.int32)
    pos[:, -3:] = torch.tensor([-(1 << 31), (1 << 31) - 1, 5])   # of the padding
    before = torch.full((s.T, Hq, d), 3.0, dtype=s.dtype).cuda()
    out = before.clone()
    at = dict(positions=pos[0].cuda()) if A == 1 else dict(positions=pos.cuda(), axes=axes)
    assert s.run(swa, w, interleaved=interleaved, factor=0.75, out=out, **at) is out
    assert swa.get_device_error() == 0
    place, row, _ = ref.places(s.starts.cpu().numpy(), np.array(total), s.table.cpu().numpy(), page, s.num_pages, s.T)
    on = torch.from_numpy(row >= 0)
    assert bool((out[~on.cuda()] == 3).all())
    # the slots: a copy without rotation goes to the same rows, the rotation beside it
    turned = swa.rope(s.q[None], s.k[None], w.cuda(), positions=pos[:, None].cuda(), axes=axes,
                      interleaved=interleaved, factor=0.75)
    assert torch.equal(out[on.cuda()], turned[0][0][on.cuda()])
    if kind != "e4m3":
        s2 = Setup(new, total, Hq, Hkv, d, page, kind, seed=sum(new) + rot + A, pad=3, fused=True)
        s2.k = turned[1][0]
        s2.run(swa, None)
        assert all(np.array_equal(raw(x), raw(y)) for x, y in zip(s.pages, s2.pages))
        return
    want = ref.rotate_axes(f64(s.k), pos.numpy(), axes, w.numpy(), interleaved, 0.75)[row >= 0]
    tol = 6 * 2.0 ** -24 * 0.75 * ref.pair_sums(f64(s.k), w.numpy(), interleaved)[row >= 0]
    page_at, slot = row[row >= 0] // page, row[row >= 0] % page
    e = raw(s.exps[0])[page_at, :, slot].astype(np.int64) - 127
    value = ref.e4m3_value(raw(s.pages[0])[page_at, slot]) * np.ldexp(1.0, e)[..., None]
    lim = tol + 2.0 ** -4 * (np.abs(want) + tol) + np.ldexp(2.0 ** -10, e)[..., None]
    assert np.all(np.abs(value - want) <= lim)
    codes, u = ref.quantise(f64(s.v)[row >= 0])   # values are not rotated
    np.testing.assert_array_equal(raw(s.pages[1])[page_at, slot], codes)
    np.testing.assert_array_equal(raw(s.exps[1])[page_at, :, slot], u)


def test_append_at_the_slots_positions_is_append(swa):
    for kind in KINDS:
        pools = []
        for at in (False, True):
            s = Setup([6, 11], [6, 40], 4, 2, 128, 8, kind, seed=5)
            pos = torch.cat([torch.arange(6), torch.arange(29, 40)]).to(torch.int32).cuda()
            q = s.run(swa, freqs(128), **(dict(positions=pos) if at else {}))
            pools.append([raw(q)] + [raw(p) for p in s.pages] + [raw(e) for e in s.exps if e is not None])
        assert all(np.array_equal(a, b) for a, b in zip(*pools))


def test_axes_in_a_graph_on_a_side_stream(swa):
    """The axes are read when the call is made: the list may change before the graph is replayed."""
    g = inp._gen(13)
    q = inp.randn((1, 40, 2, 64), torch.bfloat16, g).cuda()
    w, pos = freqs(64).cuda(), torch.randint(0, 500, (3, 1, 40), generator=g, dtype=torch.int32).cuda()
    axes, out = sections(32, 3, False), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        swa.rope(q, None, w, positions=pos, axes=axes, out=(out, None))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            swa.rope(q, None, w, positions=pos, axes=axes, out=(out, None))
    want = sections(32, 3, False)
    axes[:] = [0] * 32
    pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    near(out, q, pos.cpu().numpy(), want, freqs(64), False, 1.0, False, torch.bfloat16)


def test_axes_binding_refusals(swa):
    q = torch.zeros((2, 5, 2, 64), device="cuda", dtype=torch.bfloat16)
    w, pos = freqs(64).cuda(), torch.zeros((3, 2, 5), device="cuda", dtype=torch.int32)
    for bad in (dict(positions=None), dict(positions=pos[0]), dict(positions=pos[:, :1].contiguous()),
                dict(positions=pos.long()), dict(positions=pos.cpu()), dict(axes=[0] * 31), dict(axes=[0] * 31 + [-1]),
                dict(axes=[0] * 31 + [256])):
        args = dict(positions=pos, axes=[0] * 32)
        args.update(bad)
        with pytest.raises(ValueError):
            swa.rope(q, None, w, **args)
    with pytest.raises(swa.SwiAttnError):
        swa.rope(q, None, w, positions=pos, axes=[0] * 31 + [3])
    with pytest.raises(swa.SwiAttnError):
        swa.rope(q, None, w, positions=pos[:0], axes=[0] * 32)
    s = Setup([3], [3], 2, 1, 64, 8, "bf16", seed=1)
    p = torch.zeros((2, 3), device="cuda", dtype=torch.int32)
    for bad in (dict(positions=p), dict(axes=[0] * 32), dict(positions=p[0], axes=[0] * 32), dict(positions=p[0, :2])):
        with pytest.raises(ValueError):
            s.run(swa, freqs(64), **bad)
    with pytest.raises(ValueError):
        s.run(swa, None, positions=p[0])
    with pytest.raises(swa.SwiAttnError):
        s.run(swa, freqs(64), positions=p, axes=[2] * 32)
