"""Host-side refusals of the rotation with axes, the append at given positions, the tree attention and
the calls that keep and fork sequences (no GPU): every argument rule of include/swiattn.h, checked
before anything is launched."""
import numpy as np
import pytest

from oracle import kvcache as ref
from test_abi_cache import BF16, BIG, E4M3, EINVAL, F32, FAKE, ODD, OK, EUNSUPPORTED, lib  # noqa: F401

AXES = bytes([0, 1, 2, 3] * 16)


@pytest.mark.parametrize("name", ["swiattn_rope_axes", "swiattn_rope_axes_backward"])
def test_rope_axes_refusals(lib, name):
    def call(q=FAKE, k=FAKE, pos=FAKE, axes=AXES, n=4, w=FAKE, qo=BIG, ko=BIG, B=2, N=64, Hq=4, Hkv=2, d=128, rot=128,
             inter=0, factor=1.0, qs=512, ks=256, qos=512, kos=256, dt=BF16):
        return getattr(lib, name)(q, k, pos, axes, n, w, qo, ko, B, N, Hq, Hkv, d, rot, inter, factor, qs, ks, qos,
                                  kos, dt, None)
    for bad in (dict(pos=None), dict(axes=None), dict(n=0), dict(n=3), dict(n=-1), dict(n=65), dict(axes=bytes(63) + b"\4"),
                dict(B=0), dict(d=96), dict(rot=24), dict(w=None), dict(q=None), dict(q=ODD), dict(qs=516),
                dict(factor=float("nan")), dict(dt=E4M3)):
        assert call(**bad) == EINVAL, bad


def test_append_at_refusals(lib):
    def call(q=FAKE, k=FAKE, v=FAKE, starts=FAKE, sl=FAKE, bt=FAKE, pos=FAKE, axes=AXES, n=4, w=FAKE, qo=BIG, kp=BIG,
             vps=BIG, ke=BIG, ve=BIG, T=10, B=3, mp=4, ps=16, np_=12, Hq=4, Hkv=2, d=128, rot=128, inter=0, factor=1.0,
             qs=512, ks=256, vs=256, dt=BF16, pdt=BF16):
        return lib.swiattn_append_paged_at(q, k, v, starts, sl, bt, pos, axes, n, w, qo, kp, vps, ke, ve, T, B, mp, ps,
                                           np_, Hq, Hkv, d, rot, inter, factor, qs, ks, vs, dt, pdt, None)
    for bad in (dict(pos=None), dict(axes=None), dict(n=0), dict(n=3), dict(rot=0), dict(w=None), dict(T=-1), dict(ps=12),
                dict(k=ODD), dict(pdt=E4M3, ke=None), dict(dt=F32, pdt=BF16)):
        assert call(**bad) == EINVAL, bad
    assert call(dt=F32, pdt=E4M3) == EUNSUPPORTED
    assert call(T=0) == OK


def test_reference_rotation_with_axes():
    """Axes that agree are one rotation; an axis at position 0 leaves its pairs alone."""
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 2, 64)), 100.0 ** -(np.arange(24) / 24)
    axes, p = np.arange(24) % 3, rng.integers(0, 99, 5)
    for inter in (False, True):
        one = ref.rotate(x, p, w, inter, 1.5)
        np.testing.assert_allclose(ref.rotate_axes(x, [p, p, p], axes, w, inter, 1.5), one, atol=1e-12)
        got = ref.rotate_axes(x, [p, 0 * p, p], axes, w, inter)
        first, second = (np.s_[..., 0:48:2], np.s_[..., 1:48:2]) if inter else (np.s_[..., :24], np.s_[..., 24:48])
        for half in (first, second):
            np.testing.assert_allclose(got[half][..., axes == 1], x[half][..., axes == 1], atol=1e-12)
            np.testing.assert_allclose(got[half][..., axes != 1], (ref.rotate(x, p, w, inter))[half][..., axes != 1],
                                       atol=1e-12)


def test_accept_refusals(lib):
    def call(kp=FAKE, vps=BIG, ke=FAKE, ve=FAKE, bt=FAKE, sl=FAKE, st=FAKE, pa=FAKE, leaf=FAKE, out=BIG, layers=2, T=9,
             B=3, mp=4, ps=16, np_=12, Hkv=2, d=128, pdt=BF16):
        return lib.swiattn_accept_tree(kp, vps, ke, ve, bt, sl, st, pa, leaf, out, layers, T, B, mp, ps, np_, Hkv, d, pdt, None)
    for bad in (dict(kp=None), dict(vps=None), dict(kp=ODD), dict(vps=ODD), dict(bt=None), dict(sl=None), dict(st=None),
                dict(leaf=None), dict(out=None), dict(out=FAKE), dict(layers=0), dict(T=-1), dict(B=0), dict(mp=0), dict(ps=0),
                dict(ps=24), dict(np_=0), dict(ps=1 << 20, mp=1 << 12), dict(Hkv=0), dict(d=96), dict(pdt=3),
                dict(pdt=E4M3, ke=None), dict(pdt=E4M3, ve=None)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(layers=(1 << 14) + 1), dict(B=(1 << 30) + 1)):
        assert call(**bad) == EUNSUPPORTED, bad


def test_fork_refusals(lib):
    def call(kp=FAKE, vps=BIG, ke=FAKE, ve=FAKE, bt=FAKE, sl=FAKE, src=FAKE, new=FAKE, to=BIG, lo=BIG, layers=2, B=3, C=4,
             mp=4, ps=16, np_=12, Hkv=2, d=128, pdt=BF16):
        return lib.swiattn_fork_paged(kp, vps, ke, ve, bt, sl, src, new, to, lo, layers, B, C, mp, ps, np_, Hkv, d, pdt, None)
    for bad in (dict(kp=None), dict(vps=ODD), dict(bt=None), dict(sl=None), dict(src=None), dict(new=None), dict(to=None),
                dict(lo=None), dict(to=FAKE), dict(lo=FAKE), dict(layers=-1), dict(B=0), dict(C=-1), dict(mp=-3), dict(ps=5),
                dict(np_=0), dict(Hkv=-1), dict(d=80), dict(pdt=-1), dict(pdt=E4M3, ke=None)):
        assert call(**bad) == EINVAL, bad
    assert call(C=0) == OK
    assert call(layers=1 << 15) == EUNSUPPORTED


def test_decode_tree_refusals_and_workspace(lib):
    def size(T=20, B=3, Hq=8, Hkv=2, d=128, dt=BF16):
        return lib.swiattn_decode_tree_workspace(T, B, Hq, Hkv, d, dt)
    assert size() > 0 and size() % 256 == 0
    assert size(T=4000) > size() and size(B=200) >= size() and size(dt=F32) > 0
    for bad in (dict(T=-1), dict(B=0), dict(Hq=7), dict(Hkv=0), dict(d=96), dict(dt=E4M3), dict(Hq=258), dict(B=1 << 16),
                dict(T=1 << 24, Hq=16)):
        assert size(**bad) == 0, bad

    def call(q=FAKE, kp=FAKE, vps=FAKE, ke=FAKE, ve=FAKE, bt=FAKE, sl=FAKE, st=FAKE, pa=FAKE, gate=FAKE, o=BIG, T=20, B=3,
             mp=8, ps=16, np_=30, Hq=8, Hkv=2, d=128, W=64, S=0, scale=0.1, dt=BF16, pdt=BF16, ws=FAKE, nbytes=1 << 40):
        return lib.swiattn_decode_tree(q, kp, vps, ke, ve, bt, sl, st, pa, gate, o, None, T, B, mp, ps, np_, Hq, Hkv, d, W, S,
                                       scale, dt, pdt, ws, nbytes, None)
    for bad in (dict(q=None), dict(kp=None), dict(vps=None), dict(bt=None), dict(sl=None), dict(st=None), dict(gate=None),
                dict(o=None), dict(q=ODD), dict(o=ODD), dict(kp=ODD), dict(vps=ODD), dict(T=-1), dict(B=0), dict(mp=0),
                dict(ps=24), dict(np_=0), dict(Hq=9), dict(Hkv=-2), dict(d=32), dict(W=0), dict(S=-1), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(dt=E4M3), dict(dt=F32),
                dict(pdt=F32), dict(pdt=7), dict(pdt=E4M3, ke=None), dict(pdt=E4M3, ve=None), dict(pdt=E4M3, ke=ODD),
                dict(pdt=E4M3, ve=ODD), dict(ws=None), dict(ws=ODD),
                dict(nbytes=size() - 1), dict(ps=1 << 20, mp=1 << 12)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(Hq=258), dict(B=1 << 16), dict(dt=F32, pdt=E4M3), dict(np_=1 << 30)):
        assert call(**bad) == EUNSUPPORTED, bad
    assert call(T=0, q=None, o=None, gate=None, ws=None) == OK


def test_outputs_that_overlap_inputs_are_refused(lib):
    """Several blocks read what one of them writes over; apart by no more than a byte's width is apart."""
    at = 1 << 20

    def accept(bt=0x10000, sl=0x20000, st=0x30000, leaf=0x40000, out=at, B=3, mp=4):
        return lib.swiattn_accept_tree(FAKE, BIG, None, None, bt, sl, st, None, leaf, out, 1, 9, B, mp, 16, 12, 2, 128, BF16, None)
    for bad in (dict(leaf=at), dict(leaf=at + 8), dict(leaf=at - 8), dict(sl=at + 8), dict(sl=at - 8), dict(st=at - 12),
                dict(st=at + 8), dict(bt=at - 44), dict(bt=at + 8)):
        assert accept(**bad) == EINVAL, bad

    def fork(bt=0x10000, sl=0x20000, src=0x30000, new=0x40000, to=at, lo=2 * at, B=3, C=4, mp=4):
        return lib.swiattn_fork_paged(FAKE, BIG, None, None, bt, sl, src, new, to, lo, 1, B, C, mp, 16, 12, 2, 128, BF16, None)
    for out, size in ((at, 64), (2 * at, 16)):
        for bad in (dict(bt=out + size - 4), dict(bt=out - 44), dict(sl=out - 8), dict(sl=out + size - 4), dict(src=out),
                    dict(src=out - 12), dict(new=out + size - 4), dict(new=out - 12)):
            assert fork(**bad) == EINVAL, bad
    assert fork(lo=at + 60) == EINVAL and fork(lo=at - 12) == EINVAL

    def tree(q=at, o=2 * at, scale=0.1, T=2, np_=30):
        return lib.swiattn_decode_tree(q, FAKE, BIG, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, o, None, T, 1, 8, 16, np_, 4, 2,
                                       128, 64, 0, scale, BF16, BF16, FAKE, 1 << 40, None)
    for bad in (dict(o=at), dict(o=at + 2032), dict(o=at - 2032), dict(scale=3e38)):
        assert tree(**bad) == EINVAL, bad
    assert tree(np_=(1 << 27) + 1) == EUNSUPPORTED
