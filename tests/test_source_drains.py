"""Copies in flight when a CTA gives up, in the source (on a GPU the fault cannot be shown without causing
it).  A warp that copies tiles by TMA may have issued all of its share, fitting the ring, before the warps
that would wait for them give up: so it waits for its last copies however it left its loop, and a call of
its role is followed by those waits unconditionally."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parent.parent / "sliding_window_attention_router_gb300" / "csrc"
ROLES = {"attn_prefill.cu": 1, "attn_dual.cu": 1, "attn_bwd.cu": 2}   # kernels of each


def body(text, at):
    """From the brace before `at` to the one that closes it."""
    depth, i = 0, at
    while depth >= 0:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i]


def kernel_of(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    return text[text.index("__global__"):]


def calls_of(kernel, role):
    """Its calls, not its definition."""
    return list(re.finditer(rf"(?<![\w]){role}(<[^;(]*>)?\((?!const )", kernel))


@pytest.mark.parametrize("name", sorted(ROLES))
def test_a_producer_waits_for_its_last_copies_however_it_left(name):
    kernel = kernel_of(name)
    calls = calls_of(kernel, "producer")
    assert len(calls) == ROLES[name]
    for call in calls:
        assert kernel[:call.start()].rstrip()[-1] in ";{}", "what follows depends on its result"
        after = body(kernel, call.start())
        assert re.search(r"drain\w*\(", after.split(";", 1)[1]), "it leaves without waiting for its copies"


def test_tree_loaders_wait_for_their_last_copies_when_any_warp_gave_up():
    """Behind the last barrier, where the flag that any warp raises is final, and not by what the loader
    itself returned."""
    kernel = kernel_of("decode_tree_tc.cu")
    for role in ("loader", "raw_loader"):
        (call,) = calls_of(kernel, role)
        assert kernel[:call.start()].rstrip()[-1] in ";{}" and "filled)" in kernel[call.start():].split(";", 1)[0]
    end = body(kernel, kernel.rindex("__syncthreads();"))
    assert re.search(r"if \(\*c\.abort_flag && filled\) \{\s*if constexpr \(E4M3\) drain<Z::kOwnRaw>\(&c\.bar\[c\.kRawFull"
                     r"[^;]*filled\);\s*else drain<Z::kSlots>\(&c\.bar\[c\.kFull\], filled\);", end)
