"""Every kernel that the library launches as a programmatic dependent waits for the grid before it
(griddepcontrol.wait), so that a grid's completion means that of all grids before it on the stream,
and the next programmatic dependent, which waits for one grid, finds all their results.  Read from
the sources; no GPU."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parent.parent / "sliding_window_attention_router_gb300" / "csrc"


def dependents():
    found = []
    for path in sorted(CSRC.glob("*.cu")):
        text = path.read_text()
        for name in re.findall(r"cudaLaunchKernelEx\(&cfg,\s*(?:\w+::)*(\w+)", text):
            found.append((path.name, name))
    return sorted(set(found))


@pytest.mark.parametrize("source,kernel", dependents())
def test_programmatic_dependents_wait_for_the_grid_before_them(source, kernel):
    text = (CSRC / source).read_text()
    bodies = re.findall(r"__global__[^;{]*?\b%s\(.*?\n}\n" % kernel, text, re.S)
    assert len(bodies) == 1, (source, kernel, len(bodies))
    assert "griddepcontrol.wait" in bodies[0]


def test_all_programmatic_launches_are_seen():
    names = {k for _, k in dependents()}
    assert {"prefill_kernel", "dkdv_kernel", "dq_kernel", "decode_combine_kernel", "dual_epilogue_parts_kernel",
            "rotate_kernel", "decode_e4m3_split_kernel", "decode_e4m3_join_kernel"} <= names
