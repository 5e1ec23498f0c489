"""Host-side refusals of lengths written over the parents that other blocks read (no GPU)."""
import pytest

from test_abi_cache import BF16, BIG, EINVAL, FAKE, lib  # noqa: F401


def accept(lib, parents, T=9, B=3, out=1 << 20):  # noqa: F811
    return lib.swiattn_accept_tree(FAKE, BIG, None, None, 0x10000, 0x20000, 0x30000, parents, 0x40000, out, 1, T, B, 4, 16,
                                   12, 2, 128, BF16, None)


@pytest.mark.parametrize("off", [0, 8, -32, -4])
def test_accepted_lengths_over_the_parents_are_refused(lib, off):  # noqa: F811
    assert accept(lib, (1 << 20) + off) == EINVAL


def test_as_many_parents_as_there_are_tokens(lib):  # noqa: F811
    assert accept(lib, (1 << 20) - 4 * 100, T=101) == EINVAL
