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


def test_each_warpgroup_sets_its_registers_by_one_instruction():
    """setmaxnreg wants all warps of a warpgroup at the same instruction, and the shares together
    may not pass what the block was launched with, or the taking ones would wait for ever."""
    with open(os.path.join(CSRC, "prompt_attn.cu")) as f:
        text = f.read()
    leave = [int(x) for x in re.findall(r"leave_registers<(\d+)>\(\)", text)]
    take = [int(x) for x in re.findall(r"take_registers<(\d+)>\(\)", text)]
    assert len(leave) == 1 and len(take) == 1          # warps 8-11; warps 0-3 and 4-7
    threads = int(re.search(r"kPThreads = (\d+)", text).group(1))
    assert threads == 384
    launch = 65536 // threads // 8 * 8                 # registers a thread of the only CTA of an SM
    assert 128 * leave[0] + 256 * take[0] <= threads * launch
