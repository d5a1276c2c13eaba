// ringorder.h -- in which order the loads of a row's piece take the slots of a ring
// (rowring.cuh), and who frees a slot.  Plain arithmetic, for the kernels and for a
// model of them on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SGA_BOTH __host__ __device__ __forceinline__
#else
#define SGA_BOTH inline
#endif

namespace sga {
namespace {

// A load's place: its slot, and the parity of the slot's use.
struct Place {
  int slot;
  uint32_t phase;
};

SGA_BOTH void step(Place &a, int slots) {
  if (++a.slot == slots) {
    a.slot = 0;
    a.phase ^= 1;
  }
}

SGA_BOTH Place later(const Place &a, int by, int slots) {
  const int s = a.slot + by, q = s / slots;
  return {s - q * slots, a.phase ^ (q & 1)};
}

// Loads of a row's piece: its stages, and (kept) those again that the ring could not keep.
SGA_BOTH int num_loads(int stages, int slots, bool kept) {
  return stages + (kept && stages > slots ? stages - slots : 0);
}

// Arrivals that free a slot of a ring that keeps rows, of `warps` sum warps and as many
// output warps.  All warps that wait for the slot's loads one by one are among them: a
// wait tells only even uses from odd ones, so the next load must not land before each
// of them has seen this one.
SGA_BOTH int ring_arrivals(int warps) { return 2 * warps; }

// Those of a sum warp once it has seen a load (and read it, if it is the first of its
// stage): also the output warp's where the ring cannot keep the stage, and output warps
// see its second load only.
SGA_BOTH int sum_arrivals(int load, int stages, int slots) { return load < stages - slots ? 2 : 1; }

}  // namespace
}  // namespace sga
