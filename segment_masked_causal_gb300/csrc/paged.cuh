// paged.cuh -- where the rows of a step and the pages of a cache lie (internal).
#pragma once
#include <cstdint>

#include "kernels.h"

namespace pa {

// Rows [a, b) of the step are sequence s's; it has kv tokens, the new ones counted.
// What the device-side arrays hold is brought into range here, once for everybody.
struct SeqRows {
  int a, b, kv;
  __host__ __device__ __forceinline__ int base() const { return kv - (b - a); }  // position of its first new token
};
__host__ __device__ __forceinline__ SeqRows seq_rows(const PagedArgs& p, int s) {
  SeqRows r;
  r.a = min(max(p.q_start[s], 0), p.T);
  r.b = min(max(p.q_start[s + 1], r.a), p.T);
  r.kv = max(p.kv_len[s], 0);
  return r;
}

}  // namespace pa
