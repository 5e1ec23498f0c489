"""Which error a refused call raises, and calls with nothing in one of their tensors."""
import pytest
import torch

from test_gpu_append import swa  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("values", [7, 65, 128, 129, 1000])
def test_a_wrong_number_of_frequencies_is_refused_by_the_library(swa, values):  # noqa: F811
    q = torch.zeros((1, 4, 2, 128), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(values, device="cuda", dtype=torch.float64)
    pages, table = torch.zeros((2, 16, 2, 128), device="cuda", dtype=torch.bfloat16), torch.zeros((4, 1), device="cuda", dtype=torch.int32)
    lens = torch.ones(4, device="cuda", dtype=torch.int32)
    p = torch.zeros((1, 4), device="cuda", dtype=torch.int32)
    for call in (lambda: swa.rope(q, None, w), lambda: swa.rope_backward(None, q, w, positions=p),
                 lambda: swa.append_paged(None, q[0], q[0], pages, pages.clone(), table, lens, w),
                 lambda: swa.append_paged(None, q[0], q[0], pages, pages.clone(), table, lens, w, positions=p[0])):
        with pytest.raises(swa.SwiAttnError) as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("axes", [False, True])
def test_q_without_heads_leaves_k_to_be_rotated(swa, axes):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn((2, 5, 3, 64), generator=g, device="cuda", dtype=torch.bfloat16)
    w = 100.0 ** -(torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    more = dict(positions=torch.arange(20, device="cuda", dtype=torch.int32).view(2, 2, 5), axes=[0, 1] * 16) if axes else {}
    for call in (swa.rope, swa.rope_backward):
        want = call(None, k, w, **more)[1]
        for heads in (k[:, :, :0], k.new_empty((2, 5, 0, 64))):
            out = torch.full_like(k, 9.0)   # what the call does not write shows
            got = call(heads, k, w, out=(torch.empty_like(heads), out), **more)
            assert got[1] is out and torch.equal(out, want) and got[0].shape == heads.shape
            assert torch.equal(call(k, heads, w, **more)[0], want)
    assert swa.get_device_error() == 0
