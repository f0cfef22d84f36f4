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
// its page id; false where the words do not fit together.  Differences in 64 bits: of
// words that are no table they leave 32.
__host__ __device__ inline bool row_place(int32_t row, int32_t a0, int32_t a1, int32_t p0, int32_t p1,
                                          int32_t pages_end, int32_t last_len, int32_t& pos, int32_t& page_at) {
  constexpr int P = 16;
  const int64_t n_new = (int64_t)a1 - a0, kv_len = ((int64_t)p1 - p0 - 1) * P + last_len;
  if (a0 < 0 || row < a0 || row >= a1 || p0 < 0 || p1 <= p0 || p1 > pages_end || last_len < 1 || last_len > P ||
      n_new > kv_len || kv_len > INT_MAX)
    return false;
  pos = (int32_t)(kv_len - n_new + (row - a0));
  page_at = p0 + pos / P;
  return true;
}

}  // namespace daa
