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
