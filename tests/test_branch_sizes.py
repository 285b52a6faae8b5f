"""Sizes next to 2^31 that the drafted-tree entry points refuse, before any launch."""
from .test_branch_abi import accept, keep
from .test_paged_abi import kv, lib  # noqa: F401

MOST = 2 ** 31 - 4096


def test_accept_and_keep_refuse_what_their_steps_would_carry_past_32_bits(lib):
    """Nodes and places of a path are walked 32 and 256 at a time."""
    for size in (MOST + 1, 2 ** 31 - 33, 2 ** 31 - 1):
        assert accept(tokens=size) == 5
        assert accept(width=size) == 5
        assert keep(kv(), width=size) == 5
