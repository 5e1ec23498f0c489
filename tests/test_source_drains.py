"""Copies in flight when a CTA gives up, in the source (on a GPU the fault cannot be shown without causing
it).  A warp that copies tiles by TMA may have issued all of its share, fitting the ring, before the warps
that would wait for them give up: so it waits for its last copies however it left its loop, and a call of
its role is followed by those waits unconditionally."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parent.parent / "sliding_window_attention_router_gb300" / "csrc"
ROLES = {"decode_tree_tc.cu": ("loader", "raw_loader"), "attn_prefill.cu": ("producer",), "attn_dual.cu": ("producer",),
         "attn_bwd.cu": ("producer", "producer")}   # two kernels


def body(text, at):
    """From the brace before `at` to the one that closes it."""
    depth, i = 0, at
    while depth >= 0:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i]


@pytest.mark.parametrize("name", sorted(ROLES))
def test_a_copying_warp_waits_for_its_last_copies_however_it_left(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    kernel = text[text.index("__global__"):]
    for role in set(ROLES[name]):
        calls = list(re.finditer(rf"(?<![\w]){role}(<[^;(]*>)?\((?!const )", kernel))   # and not its definition
        assert len(calls) == ROLES[name].count(role)
        for call in calls:
            before = kernel[:call.start()].rstrip()
            assert before[-1] in ";{}", f"{name}: what follows {role} depends on its result"
            after = body(kernel, call.start())
            waits = re.findall(r"drain\w*(?:<[^;(]*>)?\(", after.split(";", 1)[1])
            assert waits, f"{name}: {role} leaves without waiting for its copies"
