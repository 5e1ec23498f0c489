"""The binding's calls in Python, as they are made where the compiled module is missing: the tests of
rotation, append, tree attention, accepted paths and forks once more, through them."""
import pytest
import torch

import swiattn_inputs as inp
from test_gpu_append import swa  # noqa: F401  (the fixture)
from test_binding import test_library_errors_and_outputs, test_calls_from_several_threads  # noqa: F401
from test_gpu_binding_refusals import *  # noqa: F401,F403
from test_gpu_rope import test_rope_refusals  # noqa: F401
from test_gpu_speculative_edges import *  # noqa: F401,F403
from test_gpu_tree import (test_speculative_step_end_to_end, test_tree_binding_refusals,  # noqa: F401
                           test_tree_padding_rows_are_left_alone)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def through_python(swa, monkeypatch):  # noqa: F811
    from sliding_window_attention_router_gb300 import _python_calls
    compiled = swa._calls()
    monkeypatch.setattr(swa, "_compiled", _python_calls)
    yield compiled
    assert swa._compiled is _python_calls


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("axes", [False, True])
def test_both_make_the_same_calls(swa, through_python, monkeypatch, kind, axes):  # noqa: F811
    """Rotation and gradient of views of a fused projection, append and tree attention: bit for bit."""
    from sliding_window_attention_router_gb300 import _python_calls
    g = inp._gen(61)
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    T, Hq, Hkv, d, page = 37, 6, 2, 64, 16
    x = inp.randn((T, (Hq + 2 * Hkv) * d), dtype, g).cuda()
    q, k, v = (p.unflatten(-1, (-1, d)) for p in x.split([Hq * d, Hkv * d, Hkv * d], -1))
    w = (100.0 ** -(torch.arange(24, dtype=torch.float64) / 24)).cuda()
    starts = torch.tensor([0, 30, 37], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100, 7], dtype=torch.int32, device="cuda")
    table = torch.arange(14, dtype=torch.int32, device="cuda").view(2, 7)
    at = torch.randint(0, 500, (2, T), generator=g).int().cuda()
    places = dict(positions=at, axes=[0, 1] * 12) if axes else dict(positions=at[0])
    gate = torch.randint(0, 2, (T,), generator=g).to(torch.uint8).cuda()
    parents = torch.cat([torch.arange(-1, 29), torch.arange(-1, 6)]).int().cuda()

    def all_calls():
        pages = [torch.zeros((14, page, Hkv, d), dtype=dtype, device="cuda").to(
            torch.float8_e4m3fn if kind == "e4m3" else dtype) for _ in "kv"]
        e = [torch.ones((14, Hkv, page), dtype=torch.uint8, device="cuda") if kind == "e4m3" else None for _ in "kv"]
        e = dict(k_exp=e[0], v_exp=e[1])
        four = dict(places, positions=places["positions"][:, None] if axes else places["positions"][None])
        out = list(swa.rope(q[None], k[None], w, factor=1.5, **four))
        out += swa.rope_backward(q[None], None, w, interleaved=True, **four)[:1]
        out.append(swa.append_paged(q, k, v, *pages, table, lens, w, starts, **places, **e))
        out += swa.decode_tree(out[-1], *pages, table, lens, starts, parents, gate, 20, 0.2, want_lse=True, n_anchor=3, **e)
        out += [p.view(torch.uint8) for p in pages] + [x for x in e.values() if x is not None]
        return out

    got = all_calls()
    monkeypatch.setattr(swa, "_compiled", through_python)
    want = all_calls()
    monkeypatch.setattr(swa, "_compiled", _python_calls)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want)
    assert swa.get_device_error() == 0
