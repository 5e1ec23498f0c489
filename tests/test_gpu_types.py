"""Tensors of a type that the library does not take are refused as other wrong arguments are."""
import pytest
import torch


def test_types_are_named_in_the_refusal():
    import sliding_window_attention_router_gb300 as swa
    assert swa._DT[torch.float32] == swa.F32 and swa._DT[torch.bfloat16] == swa.BF16
    for t in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match=str(t)):
            swa._DT[t]
    assert swa._DT.get(torch.float16, 7) == 7


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.float64])
def test_other_floating_types_are_refused(dtype):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_router_gb300 as swa
    B, N, H, d, page = 2, 3, 2, 64, 16
    x = torch.zeros((B, N, H, d), dtype=dtype, device="cuda")
    w = torch.ones(d // 2, dtype=torch.float64, device="cuda")
    one = x[:, 0].contiguous()
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    gate = torch.ones(B, dtype=torch.uint8, device="cuda")
    same = [torch.zeros((B, page, H, d), dtype=dtype, device="cuda") for _ in "kv"]
    e4m3 = [p.to(torch.float8_e4m3fn) for p in same]
    exps = [torch.zeros((B, H, page), dtype=torch.uint8, device="cuda") for _ in "kv"]
    calls = [
        lambda: swa.rope(x, x, w), lambda: swa.rope_backward(x, None, w), lambda: swa.rope(x[:0], None, w),
        lambda: swa.append_paged(one, one, one, *same, table, lens, w),
        lambda: swa.append_paged(one, one, one, *e4m3, table, lens, w, k_exp=exps[0], v_exp=exps[1]),
        lambda: swa.append_paged(None, one[:0], one[:0], *same, table[:0], lens[:0]),
        lambda: swa.decode_paged_e4m3(one, *e4m3, *exps, table, lens, gate, 4),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, swa.SwiAttnError)):
            call()
            pytest.fail(f"call {i} was not refused")
    assert swa.get_device_error() == 0
