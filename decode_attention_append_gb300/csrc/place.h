// Where a new row goes, from the page table's words as they are on the device.  The
// appends read their tables where no host has looked at them: what does not hold there
// must end in a refusal and never in an address.
#pragma once
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

namespace daa {

// New row `row` of the request with rows [a0, a1) and pages [p0, p1) of the first
// pages_end ids, the last page holding last_len tokens: its position and the index of
// its page id; false where the words do not fit together.  Differences are of words
// from zero up, and of at most 2^27 pages, so that nothing leaves 32 bits.
__host__ __device__ inline bool row_place(int32_t row, int32_t a0, int32_t a1, int32_t p0, int32_t p1,
                                          int32_t pages_end, int32_t last_len, int32_t& pos, int32_t& page_at) {
  constexpr uint32_t P = 16;
  const uint32_t n_new = (uint32_t)a1 - (uint32_t)a0, np = (uint32_t)p1 - (uint32_t)p0;
  const uint32_t kv_len = (np - 1) * P + (uint32_t)last_len;
  if (a0 < 0 || row < a0 || row >= a1 || p0 < 0 || p1 <= p0 || p1 > pages_end || np > (1u << 27) || last_len < 1 ||
      last_len > (int32_t)P || kv_len > (uint32_t)INT_MAX || n_new > kv_len)
    return false;
  pos = (int32_t)(kv_len - n_new + (uint32_t)(row - a0));
  page_at = p0 + (int32_t)((uint32_t)pos / P);
  return true;
}

}  // namespace daa
