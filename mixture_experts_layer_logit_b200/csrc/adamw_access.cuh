// Whether the AdamW step may reach the arrays of a tensor by vectors, decided
// by their addresses.  Written without any CUDA construct: a test compiles it
// for the host and holds it against the widths of the accesses.
#pragma once

#include <stdint.h>

#include "moe.h"

namespace moe {

// Bytes of eight elements of type dt: one access of a lane, which needs that alignment.
inline unsigned lane_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 32u : 16u; }

// 8-bit states: arrays are read by copies of 16 bytes to shared memory; a lane
// writes eight elements of param and master, and eight codes of m and v, at
// once.  32-bit states: a lane reads and writes eight elements at once
// throughout, the gradient's among them.  Otherwise every element is reached on
// its own: 334 us where vectors take 328 (67 M elements with master copies; an
// fp32 gradient on 16 bytes alone, read in two halves, takes 328, too little
// gain for a third way).
inline bool adamw_by_vectors(const moe_adamw_tensor& t) {
  auto on = [](const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
  const bool eight = t.state_bits == 8;
  const unsigned state = eight ? 16u : 32u;
  return on(t.param, lane_bytes(t.param_dtype)) && on(t.grad, eight ? 16u : lane_bytes(t.grad_dtype)) &&
         on(t.master, 32u) && on(t.m, state) && on(t.v, state);
}

}  // namespace moe
