"""The compiled part of the Python binding: it is built, refuses with the binding's own error types
before anything is launched, and keeps what it is given."""
import threading

import pytest
import torch


@pytest.fixture(scope="module")
def swa():
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_router_gb300 as m
    return m


def test_calls_refuse_host_tensors_and_other_objects(swa):
    x, i = torch.zeros((1, 1, 1, 64)), torch.zeros(2, dtype=torch.int32)
    for bad in (x, None, 5, "q", [x]):
        for call in (lambda: swa.rope(bad, None, x), lambda: swa.rope_backward(None, bad, x),
                     lambda: swa.append_paged(None, bad, x, x, x, i, i),
                     lambda: swa.decode_tree(bad, x, x, i, i, i, None, i, 4),
                     lambda: swa.accept_tree(bad, x, i, i, i, None, i),
                     lambda: swa.fork_paged(bad, x, i, i, i, i)):
            with pytest.raises(ValueError, match="must be a CUDA tensor"):
                call()


def test_axes_are_small_whole_numbers(swa):
    x = torch.zeros((1, 1, 1, 64))
    for axes in ([0, 256], [-1], torch.tensor([300])):
        with pytest.raises(ValueError):
            swa.rope(x, None, x, positions=x, axes=axes)
    for axes in (64, [0.5], "0"):   # 64 would be 64 zeros to bytes()
        with pytest.raises(TypeError):
            swa.rope(x, None, x, positions=x, axes=axes)


@pytest.mark.gpu
def test_library_errors_and_outputs(swa):
    k = torch.zeros((3, 16, 2, 64), device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    starts = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(swa.SwiAttnError) as e:   # the lengths cannot be written over while they are read
        swa.accept_tree(k, k.clone(), table, i, starts, None, i, out=i)
    assert e.value.status == 1 and "swiattn_accept_tree" in str(e.value)
    out = torch.empty_like(i)
    assert swa.accept_tree(k, k.clone(), table, i, starts, None, i - 1, out=out) is out
    for pair in ((None, out), (torch.empty_like(table), None)):
        with pytest.raises(ValueError):
            swa.fork_paged(k, k.clone(), table, i, i, i, out=pair)
    with pytest.raises(ValueError, match="float8_e8m0fnu"):
        p = k.to(torch.float8_e4m3fn)
        swa.accept_tree(p, p.clone(), table, i, starts, None, i, k_exp=k, v_exp=k)
    with pytest.raises(TypeError):
        swa.decode_tree(k[0, :1], k, k.clone(), table, i, starts, None, i.to(torch.uint8), "4")
    assert swa.get_device_error() == 0


@pytest.mark.gpu
def test_calls_from_several_threads(swa):
    """The interpreter's lock is given up around a call: each thread's own sequence, on its own
    stream, comes out as alone."""
    def work(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn((20, 4, 64), generator=g, device="cuda", dtype=torch.bfloat16)
        pages = torch.randn((2, 6, 64, 2, 64), generator=g, device="cuda").bfloat16()
        table = torch.randperm(6, generator=g, device="cuda").int()[None]
        lens = torch.tensor([320 + seed], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
        parents = torch.arange(-1, 19, dtype=torch.int32, device="cuda")
        gate = torch.ones(20, dtype=torch.uint8, device="cuda")
        return swa.decode_tree(q, pages[0], pages[1], table, lens, starts, parents, gate, 8)

    alone = [work(s) for s in range(8)]
    torch.cuda.synchronize()
    wrong = []

    def thread(s):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = work(s)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(got, alone[s]):
                    wrong.append(s)

    threads = [threading.Thread(target=thread, args=(s,)) for s in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and swa.get_device_error() == 0
