// The ticket of an item that several CTAs share: an int in the workspace, zero between calls.
//
// Every CTA that shares the item arrives on it exactly once: when it has left its state for
// the others, or, if a wait of it ran out, when it gives the item up.  The last one to arrive
// sets the ticket back to zero, and joins the states if all of them are there.  So the next
// call finds zeros whatever became of this one.
#pragma once

#ifdef __CUDACC__
#define VEGAS_HD __host__ __device__ __forceinline__
#else
#define VEGAS_HD inline
#endif

namespace vegas {

// What an arrival adds: the low half counts arrivals (at most one a CTA), the high half those
// without a state.
constexpr int kTicketLeft = 1;
constexpr int kTicketGivenUp = (1 << 16) + 1;

struct TicketTurn {
  bool last;   // set the ticket back to zero
  bool join;   // every other state is there
};

// The turn of an arrival that found `before`, among `arrivals`.
VEGAS_HD TicketTurn ticket_turn(int before, int arrivals, bool given_up) {
  TicketTurn t;
  t.last = (before & 0xffff) == arrivals - 1;
  t.join = !given_up && before == arrivals - 1;
  return t;
}

}  // namespace vegas
