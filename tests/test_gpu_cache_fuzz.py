"""Seeded random shapes of the append and of decode over 8-bit pages against the 64-bit reference, and
the calls at the ends of their ranges.  Tolerances as in test_gpu_append and test_gpu_decode_e4m3, whose
set-ups are used."""
import numpy as np
import pytest
import torch

from test_gpu_append import Setup, freqs
from test_gpu_decode_e4m3 import Cache, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_router_gb300 as m
    return m


@pytest.mark.parametrize("seed", range(16))
def test_append_random_shapes(swa, seed):
    r = np.random.default_rng(1000 + seed)
    B = int(r.integers(1, 50))
    step = r.random() < 0.3
    new = [1] * B if step else [int(n) for n in r.integers(0, 40, B)]
    if sum(new) == 0:
        new[0] = 3
    total = [n + int(r.integers(0, 500)) if n else int(r.integers(0, 50)) for n in new]
    Hkv = int(r.integers(1, 9))
    d = int(r.choice([64, 128]))
    rot = 16 * int(r.integers(1, d // 16 + 1))
    s = Setup(new, total, Hkv * int(r.integers(1, 9)), Hkv, d, 2 ** int(r.integers(0, 8)),
              ["bf16", "e4m3", "f32"][int(r.integers(0, 3))], seed=seed, starts=not step,
              pad=0 if step else int(r.integers(0, 5)), fused=r.random() < 0.5)
    inter = bool(r.random() < 0.5)
    before = torch.full((s.T, s.q.shape[1], d), 3.0, dtype=s.dtype).cuda()
    out = before.clone()
    s.run(swa, freqs(rot), interleaved=inter, factor=0.8, out=out)
    assert swa.get_device_error() == 0
    assert not s.check(out, freqs(rot), inter, 0.8, q_before=before)


@pytest.mark.parametrize("seed", range(16))
def test_decode_random_shapes(swa, seed):
    r = np.random.default_rng(2000 + seed)
    B = int(r.integers(1, 40))
    longest = int(np.exp(r.uniform(0, np.log(3000))))
    lens = [int(n) for n in r.integers(0, longest + 1, B)]
    lens[0] = longest
    Hkv = int(r.integers(1, 6))
    c = Cache(lens, [int(g) for g in r.integers(0, 2, B)], Hkv * int(r.integers(1, 17)), Hkv,
              int(r.choice([64, 128])), int(r.integers(1, 700)), int(r.choice([0, 0, 7, 100])),
              2 ** int(r.integers(0, 10)), seed=seed)
    c.check(*run(swa, c))


def test_decode_of_empty_slots_alone(swa):
    c = Cache([0, 0, 0], [0, 1, 0], 4, 2, 64, 5, 3, 16, seed=1)
    o, lse = run(swa, c)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("page", [16, 2])
def test_decode_at_the_ends_of_window_and_anchors(swa, page):
    """The widest window and the most anchors are the whole history; a window of one key."""
    last = (1 << 31) - 1
    base = Cache([333, 50], [1, 1], 4, 2, 64, 9, 0, page, seed=2)
    want, want_lse = run(swa, base)
    for gate, W, S in ((0, last, 0), (0, 1, last), (0, last, last), (1, last, last)):
        base.gate[:] = gate
        base.W, base.S = W, S
        o, lse = run(swa, base)
        base.check(o, lse)
    one = Cache([333, 50], [0, 0], 4, 2, 64, 1, 0, page, seed=2)
    o, lse = run(swa, one)
    one.check(o, lse)


def test_two_streams_at_once(swa):
    """Two steps of different batches on two streams, each with its own workspace, interleaved call by
    call: the results of the steps alone."""
    setups = [Setup([1] * 40, [200] * 40, 4, 2, 128, 16, "e4m3", seed=20 + i, starts=False) for i in (0, 1)]
    w = freqs(128).cuda()
    gate = torch.tensor([0, 1] * 20, dtype=torch.uint8, device="cuda")

    def step(s, ws=None):
        q = swa.append_paged(s.q, s.k, s.v, *s.pages, s.table, s.seq_lens, w, k_exp=s.exps[0], v_exp=s.exps[1])
        return swa.decode_paged_e4m3(q, *s.pages, *s.exps, s.table, s.seq_lens, gate, 64, workspace=ws)

    for s in setups:   # the pools hold random bytes: make them finite
        for p, e in zip(s.pages, s.exps):
            p.view(torch.uint8).bitwise_and_(0x77)
            e.clamp_(120, 130)
    want = [step(s) for s in setups]
    torch.cuda.synchronize()
    n = swa.decode_paged_e4m3_workspace(40, setups[0].max_pages, 16, 4, 2, 128, 64)
    wss = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in setups]
    streams = [torch.cuda.Stream() for _ in setups]
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(setups):
            with torch.cuda.stream(streams[i]):
                got[i] = step(s, wss[i])
    torch.cuda.synchronize()
    assert swa.get_device_error() == 0
    for g, e in zip(got, want):
        assert bool(torch.isfinite(e.float()).all()) and torch.equal(g, e)
