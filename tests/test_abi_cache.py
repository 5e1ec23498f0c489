"""Host-side refusals of the rotation, append and 8-bit decode entry points (no GPU): every
argument rule of include/swiattn.h, checked before anything is launched."""
import ctypes

import pytest

EINVAL, EUNSUPPORTED, OK = 1, 2, 0
F32, BF16, E4M3 = 0, 1, 2
vp = ctypes.c_void_p
FAKE = vp(1 << 20)          # never dereferenced: validation fails first
ODD = vp((1 << 20) + 8)     # not 16-byte aligned
BIG = vp(1 << 21)


@pytest.fixture(scope="module")
def lib():
    from sliding_window_attention_router_gb300 import build
    build.build()
    import sliding_window_attention_router_gb300 as swa
    return swa._load()


@pytest.mark.parametrize("name", ["swiattn_rope", "swiattn_rope_backward"])
def test_rope_refusals(lib, name):
    def call(q=FAKE, k=FAKE, pos=None, w=FAKE, qo=BIG, ko=BIG, B=2, N=64, Hq=4, Hkv=2, d=128, rot=128,
             inter=0, factor=1.0, qs=512, ks=256, qos=512, kos=256, dt=BF16):
        return getattr(lib, name)(q, k, pos, w, qo, ko, B, N, Hq, Hkv, d, rot, inter, factor, qs, ks, qos,
                                  kos, dt, None)
    for bad in (dict(B=0), dict(N=0), dict(B=1 << 16, N=1 << 15), dict(Hq=0), dict(Hkv=-1), dict(d=96),
                dict(rot=0), dict(rot=24), dict(rot=144), dict(d=64, rot=128, qs=512), dict(w=None),
                dict(q=None), dict(qo=None), dict(k=None), dict(q=None, qo=None, k=None, ko=None),
                dict(q=ODD), dict(ko=ODD), dict(qs=504), dict(qs=516), dict(kos=255), dict(qs=-512), dict(qs=0),
                dict(q=BIG, qs=1024), dict(factor=float("nan")), dict(factor=float("inf")), dict(dt=2),
                dict(dt=E4M3), dict(dt=-1)):
        assert call(**bad) == EINVAL, bad


def test_append_refusals(lib):
    def call(q=FAKE, k=FAKE, v=FAKE, starts=FAKE, sl=FAKE, bt=FAKE, w=FAKE, qo=BIG, kp=BIG, vps=BIG, ke=BIG,
             ve=BIG, T=10, B=3, mp=4, ps=16, np_=12, Hq=4, Hkv=2, d=128, rot=128, inter=0, factor=1.0, qs=512,
             ks=256, vs=256, dt=BF16, pdt=BF16):
        return lib.swiattn_append_paged(q, k, v, starts, sl, bt, w, qo, kp, vps, ke, ve, T, B, mp, ps, np_, Hq,
                                        Hkv, d, rot, inter, factor, qs, ks, vs, dt, pdt, None)
    for bad in (dict(T=-1), dict(B=0), dict(mp=0), dict(ps=0), dict(ps=12), dict(np_=0), dict(ps=1 << 20, mp=1 << 12),
                dict(Hq=0), dict(Hkv=0), dict(d=80), dict(rot=8), dict(rot=136), dict(starts=None), dict(k=None),
                dict(v=None), dict(sl=None), dict(bt=None), dict(w=None), dict(q=None), dict(qo=None), dict(kp=None),
                dict(vps=None), dict(pdt=E4M3, ke=None), dict(pdt=E4M3, ve=None), dict(k=ODD), dict(v=ODD),
                dict(q=ODD), dict(qo=ODD), dict(kp=ODD), dict(vps=ODD), dict(qs=511), dict(ks=248), dict(vs=260),
                dict(factor=float("inf")), dict(dt=5), dict(pdt=F32), dict(dt=F32, pdt=BF16), dict(q=BIG, qs=1024)):
        assert call(**bad) == EINVAL, bad
    assert call(dt=F32, pdt=E4M3) == EUNSUPPORTED
    assert call(T=0) == OK
    assert call(T=0, starts=None) == EINVAL   # one token each means T == B


def test_decode_e4m3_refusals_and_workspace(lib):
    def size(B=2, mp=8, ps=16, Hq=8, Hkv=2, d=128, W=64, S=0):
        return lib.swiattn_decode_paged_e4m3_workspace(B, mp, ps, Hq, Hkv, d, W, S)
    assert size() > 0 and size() % 256 == 0
    assert size(B=4) > size() and size(Hq=16) > size()
    for bad in (dict(B=0), dict(mp=0), dict(ps=24), dict(Hq=7), dict(Hkv=0), dict(d=96), dict(W=0), dict(S=-1),
                dict(Hq=34), dict(B=1 << 16), dict(ps=1 << 20, mp=1 << 12)):
        assert size(**bad) == 0, bad

    def call(q=FAKE, kp=FAKE, vps=FAKE, ke=FAKE, ve=FAKE, bt=FAKE, sl=FAKE, gate=FAKE, o=BIG, B=2, mp=8, ps=16, np_=9,
             Hq=8, Hkv=2, d=128, W=64, S=0, scale=0.1, dt=BF16, ws=FAKE, nbytes=1 << 40):
        return lib.swiattn_decode_paged_e4m3(q, kp, vps, ke, ve, bt, sl, gate, o, None, B, mp, ps, np_, Hq, Hkv, d, W,
                                             S, scale, dt, ws, nbytes, None)
    for bad in (dict(q=None), dict(kp=None), dict(vps=None), dict(ke=None), dict(ve=None), dict(bt=None), dict(sl=None),
                dict(gate=None), dict(o=None), dict(q=ODD), dict(kp=ODD), dict(vps=ODD), dict(o=ODD), dict(ke=ODD), dict(ve=ODD), dict(B=0), dict(mp=-1),
                dict(ps=3), dict(np_=0), dict(Hq=9), dict(Hkv=-2), dict(d=32), dict(W=0), dict(S=-2), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(dt=E4M3), dict(dt=7),
                dict(ws=None), dict(ws=ODD), dict(nbytes=size() - 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(Hq=34), dict(B=1 << 16), dict(dt=F32), dict(B=1 << 14, Hq=1 << 17, Hkv=1 << 17)):
        assert call(**bad) == EUNSUPPORTED, bad
