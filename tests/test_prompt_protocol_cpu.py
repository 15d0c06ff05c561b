"""What the prompt kernel does once a bounded wait has run out, checked without a GPU: no run can
make that happen in an orderly way, so its parts are checked from the source and on the host."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "self_speculative_sparse_paged_gb300", "csrc")


def _block(text, at):
    """The braces' contents that begin at or after `at`, and where they end."""
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i + 1:j], j + 1
    raise AssertionError("unbalanced braces")


def test_the_softmax_warps_leave_their_items_only_by_a_common_vote():
    """A group's four warps share barriers without a time limit: one that left alone after its
    own wait ran out would keep the other three waiting for ever."""
    with open(os.path.join(CSRC, "prompt_attn.cu")) as f:
        text = f.read()
    role = text.index("softmax of tile X")
    loop, _ = _block(text, text.index("while (", role))
    tile = loop.index("for (int t = kbeg")           # its own breaks end the tile loop only
    _, end = _block(loop, tile)
    items = loop[:tile] + loop[end:]
    exits = [m.start() for m in re.finditer(r"\bbreak;", items)]
    assert exits
    for at in exits:
        assert "named_bar_any(1 + x, 128" in items[max(0, at - 80):at], items[max(0, at - 120):at + 6]
    assert "while (true)" in text[role:text.index("for (int t = kbeg", role)]
