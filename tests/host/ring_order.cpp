// The ring's arithmetic (csrc/ringorder.h) behind C symbols, for tests/test_ring_order.py.
#include "ringorder.h"

extern "C" {

// slot and phase packed as 2 * slot + phase
int ring_step(int at, int slots) {
  sga::Place p = {at >> 1, static_cast<uint32_t>(at & 1)};
  sga::step(p, slots);
  return 2 * p.slot + static_cast<int>(p.phase);
}

int ring_later(int at, int by, int slots) {
  const sga::Place p = sga::later({at >> 1, static_cast<uint32_t>(at & 1)}, by, slots);
  return 2 * p.slot + static_cast<int>(p.phase);
}

int ring_loads(int stages, int slots, int kept) { return sga::num_loads(stages, slots, kept != 0); }
int ring_arrivals(int warps) { return sga::ring_arrivals(warps); }
int ring_sum_arrivals(int load, int stages, int slots) {
  return sga::sum_arrivals(load, stages, slots);
}

}  // extern "C"
