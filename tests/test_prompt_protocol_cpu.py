"""What the prompt kernel does once a bounded wait has run out, checked without a GPU: no run can
make that happen in an orderly way, so its parts are checked from the source and on the host."""
import os
import re
import subprocess

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


TICKETS = r"""
#include <cstdio>
#include "ticket.h"
using namespace vegas;
// Every order of the arrivals of n CTAs: 0 leaves its state, 1 looks first and takes the join
// itself when all the others have arrived, 2 gives the item up.
int n, kinds[5], bad = 0; long orders = 0;
void go(int ticket, const int* stage, int left, int joins) {
  bool any = false;
  for (int i = 0; i < n; ++i) {
    if (stage[i] == 2) continue;
    any = true;
    int st[5], t = ticket, l = left, j = joins;
    for (int k = 0; k < n; ++k) st[k] = stage[k];
    if (kinds[i] == 1 && stage[i] == 0) {
      st[i] = 1;
      if (t == n - 1) {                     // all the others: no arrival of its own
        st[i] = 2;
        bad += l != n - 1;
        ++j, t = 0;
      }
    } else {
      st[i] = 2;
      const bool up = kinds[i] == 2;
      const TicketTurn turn = ticket_turn(t, n, up);
      t += up ? kTicketGivenUp : kTicketLeft;
      l += !up;
      if (turn.join) bad += l != n, ++j;
      if (turn.last) t = 0;
    }
    go(t, st, l, j);
  }
  if (any) return;
  ++orders;
  bool whole = true;
  for (int i = 0; i < n; ++i) whole = whole && kinds[i] != 2;
  bad += ticket != 0 || joins != (whole ? 1 : 0);
}
int main() {
  for (n = 2; n <= 4; ++n)
    for (int c = 0, all = n == 2 ? 9 : n == 3 ? 27 : 81; c < all; ++c) {
      for (int i = 0, v = c; i < n; ++i, v /= 3) kinds[i] = v % 3;
      const int none[5] = {};
      go(0, none, 0, 0);
    }
  printf("%d of %ld\n", bad, orders);
  return bad != 0;
}
"""


def test_a_ticket_is_zero_after_every_order_of_arrivals(tmp_path):
    src = tmp_path / "tickets.cpp"
    src.write_text(TICKETS)
    exe = tmp_path / "tickets"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0 and int(run.stdout.split()[-1]) > 1000, run.stdout


def test_every_shared_item_is_arrived_on_or_given_up():
    """The kernel's end settles the items that a CTA owes an arrival, and every arrival is noted."""
    with open(os.path.join(CSRC, "prompt_attn.cu")) as f:
        text = f.read()
    assert len(re.findall(r"atomicAdd\(ticket, kTicketLeft\)", text)) == 1
    assert len(re.findall(r"\*arrived = 1;", text)) == 2           # that one, and the join without it
    end = text[text.index("after a wait that ran out: the shared items"):]
    assert "__syncthreads();" in text[:text.index(end)][-120:]     # when all warps are done
    assert "kTicketGivenUp" in end[:600]
    assert "while (walk.next(q, d, w)) owe();" in text             # the walk goes on without its items
