// Host-only harness for tests/test_plan_q4.py: the plan of attention over the
// 4-bit cache for batches read from stdin (the format of plan_check.cpp without
// groups), printed.  Compiled with g++ against the library's planner header; runs
// no CUDA call.
//
// Output, per case: "S status", then
//   "U q_row n_tok pos0 kv_len page_base tok_begin tok_end part part_stride" per unit,
//   "R unit unit_end cls" per range, in launch order,
//   "M q_row part_begin n_parts" per merge item,
//   "D row0 page_base kv_len qo_len tok0 ntok key_lo key_hi" per item of the bf16 requests,
//   "X src" the page_indices place of each scratch page,
//   "L n_parts n_scratch total", and "E".
#include <cstdio>
#include <vector>

#include "planner_q4.h"

namespace {

template <class T>
struct Vec {
  std::vector<T> v;
  bool push_back(const T& x) {
    v.push_back(x);
    return true;
  }
  size_t size() const { return v.size(); }
  T* data() { return v.data(); }
  const T* data() const { return v.data(); }
  void clear() { v.clear(); }
};

bool read_ints(std::vector<int32_t>& a, int n) {
  a.resize(n);
  for (int i = 0; i < n; ++i)
    if (std::scanf("%d", &a[i]) != 1) return false;
  return true;
}

}  // namespace

int main() {
  int Hq, Hkv, d, P, sms, batch;
  long long num_pages;
  daa::Q4Plan<Vec> pl;
  while (std::scanf("%d %d %d %d %lld %d", &Hq, &Hkv, &d, &P, &num_pages, &sms) == 6) {
    std::vector<int32_t> qo, kv, last;
    if (std::scanf("%d", &batch) != 1 || !read_ints(qo, batch + 1) || !read_ints(kv, batch + 1) ||
        !read_ints(last, batch))
      return 2;
    const daa_dims dims{Hq, Hkv, d, P, num_pages};
    const int st = daa::plan_batch_q4(qo.data(), kv.data(), last.data(), batch, dims, sms, pl);
    std::printf("S %d\n", st);
    if (st == 0) {
      for (const auto& u : pl.units.v)
        std::printf("U %d %d %d %d %d %d %d %d %d\n", u.q_row, u.n_tok, u.pos0, u.kv_len, u.page_base,
                    u.tok_begin, u.tok_end, u.part, u.part_stride);
      size_t r = 0;
      for (int c = 0; c < daa::kQ4Classes; ++c)
        for (int i = 0; i < pl.lay.n_ranges[c]; ++i, ++r)
          std::printf("R %d %d %d\n", pl.seg_begin[r], pl.seg_begin[r + 1], c);
      for (const auto& m : pl.merges.v) std::printf("M %d %d %d\n", m.q_row, m.part_begin, m.n_parts);
      for (const auto& t : pl.sub_tiles.v)
        std::printf("D %d %d %d %d %d %d %d %d\n", t.q_row0, t.page_base, t.kv_len, t.qo_len, t.tok0,
                    t.ntok + t.ntok1, t.key_lo, t.key_hi);
      for (int32_t x : pl.src) std::printf("X %d\n", x);
      std::printf("L %d %d %zu\n", pl.lay.n_parts, pl.lay.n_scratch, pl.lay.total);
      // the staged bytes lie inside the workspace
      std::vector<uint8_t> host(pl.lay.plan_bytes + 1, 0xEE);
      daa::plan_stage_q4(pl, host.data());
      if (host[pl.lay.plan_bytes] != 0xEE || pl.lay.plan_bytes > pl.lay.total) return 3;
    }
    std::printf("E\n");
  }
  return 0;
}
