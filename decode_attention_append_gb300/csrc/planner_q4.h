// Host-side plan of attention over the 4-bit cache.
//
// "Disaggregated prefill and decode" (Perplexity), "Prefill vs decode
// performance": a long chunk is bound by the tensor cores, a decode request by
// the K/V bytes.  A request whose packed (token, query head) rows are more than
// kQ4NativeRows reads every key many times, so its pages are turned into bf16
// once, in the workspace, and it runs on the bf16 kernels (their plan, on the
// batch of these requests alone), unless there are so few of them that those
// kernels would leave most of the GPU idle (few_chunks_q4); the others are read
// from the 4-bit pages by the attention_q4 kernel.
#pragma once
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "../../include/daa.h"
#include "launch.h"
#include "planner.h"

namespace daa {

// GB300, 8 kv heads, d = 128, 32 requests of 2500 keys, 4 and 8 heads a kv head: 96
// rows 118 us from the 4-bit pages and 133 to 146 by way of bf16, 128 rows 165 to 168 and
// 134 to 151.
constexpr int kQ4NativeRows = 96;
// Rows a unit holds at most: more would spill the register kernel's sums (GB300, a
// further page on an SM: 52, 74 and 92 ns with 8, 16 and 24 rows).  Where all units of 8
// rows find a free warp, smaller ones end sooner.
constexpr int kQ4UnitRows = 24, kQ4SmallUnitRows = 8;
constexpr int kQ4MinPages = 4;    // pages of a range at least
// What a unit costs beside its pages, in pages, by class (GB300: with 3 for all a second
// unit made 16- and 24-row warps end 2 us after the others; decode of 128 requests of 12
// heads 53.3 us with 3 and 51.4 with 7, verify of 5 tokens 44.4 and 42.7).
constexpr int kQ4UnitPages[kQ4Classes] = {5, 7, 7};

// Whether a batch's long requests are better read from the 4-bit pages, too: few_chunks
// of `warps` (units of kQ4UnitRows rows, times kv heads) over up to `keys` keys.  The
// bf16 kernels give a long chunk's rows to few SMs, each of which walks all keys (11 to
// 13 ns a key); 24-row units read the pages again for every 24 rows, but on every SM.
// Requests of two 128-row tiles at most (`split`) have their keys cut there, too.
// Measured on GB300 at 274 points (rows 128 to 2048, keys 100 to 16000, 1 to 32 kv
// heads, 1 to 8 chunks, with and without decode beside them): taken at 170 of them, 1.83
// times as fast on average there, 9.4 at best (252 rows, 1 kv head of 64 dims, 16000 keys:
// 18.8 us and 176) and 1.01 at worst (126 rows, 5 kv heads, 118 keys: 10.4 and 10.5); 1.45
// over all points.  Where it is not taken it would be 1.35 at best.
inline bool few_chunks_q4(int64_t warps, int64_t keys, bool split, int sms) {
  if (5 * warps <= 3 * (int64_t)sms) return !split || warps * keys <= 150000;
  return !split && warps <= 2 * (int64_t)sms - 160000 / keys;
}

inline int q4_class(int rows) { return (rows - 1) / 8; }  // up to 8, 16, 24 rows
// Warps of the class's kernel on an SM (its shared memory and registers).
inline int q4_warps_per_sm(int cls) { return cls == 0 ? 16 : 8; }

// Sections of the workspace, all worked out from the counts and the layout of
// the bf16 requests' plan.  The first plan_bytes are copied from the host.
struct Q4Layout {
  int n_ranges[kQ4Classes] = {};
  int n_units = 0, n_merges = 0, n_parts = 0, n_scratch = 0;
  PlanLayout sub;
  size_t off_units, off_ranges, off_merges, off_src, off_ids, off_sub, plan_bytes, off_part_o, off_part_lse,
      off_pool, total;
  int ranges() const { return n_ranges[0] + n_ranges[1] + n_ranges[2]; }
  void finish(const daa_dims& d) {
    size_t off = 0;
    off_units = off;
    off = plan_align_up(off + (size_t)n_units * sizeof(Q4Unit));
    off_ranges = off;
    off = plan_align_up(off + (size_t)ranges() * sizeof(Q4Range));
    off_merges = off;
    off = plan_align_up(off + (size_t)n_merges * sizeof(MergeItem));
    off_src = off;
    off = plan_align_up(off + (size_t)n_scratch * sizeof(int32_t));
    off_ids = off;
    off = plan_align_up(off + (size_t)n_scratch * sizeof(int32_t));
    off_sub = off;
    plan_bytes = off + (sub.total > 0 ? sub.plan_bytes : 0);
    off = plan_align_up(off + sub.total);
    off_part_o = off;
    off = plan_align_up(off + (size_t)n_parts * d.num_qo_heads * d.head_dim * sizeof(float));
    off_part_lse = off;
    off = plan_align_up(off + (size_t)n_parts * d.num_qo_heads * sizeof(float));
    off_pool = off;
    off = plan_align_up(off + (size_t)n_scratch * 2 * d.num_kv_heads * d.page_size * d.head_dim * 2);
    total = n_units == 0 && sub.total == 0 ? 0 : off;
  }
};

// The plan of one batch; `sub_*` are the items of the bf16 requests.
template <template <class> class Vec>
struct Q4Plan {
  Vec<Q4Unit> units;
  Vec<MergeItem> merges;
  Vec<DecodeUnit> sub_units;
  Vec<MergeItem> sub_merges;
  Vec<PrefillTile> sub_tiles;
  std::vector<int32_t> seg_begin;              // [ranges + 1], first unit of each
  std::vector<int32_t> src;                    // scratch page -> index into page_indices
  std::vector<int32_t> req, sub_qo, sub_kv, sub_last;  // the bf16 requests' table
  Q4Layout lay;
};

template <template <class> class Vec>
daa_status plan_batch_q4(const int32_t* qo, const int32_t* kv, const int32_t* last, int32_t batch,
                         const daa_dims& d, int sms, Q4Plan<Vec>& pl) {
  pl.units.clear();
  pl.merges.clear();
  pl.seg_begin.assign(1, 0);
  pl.src.clear();
  pl.req.clear();
  pl.sub_qo.assign(1, 0);
  pl.sub_kv.assign(1, 0);
  pl.sub_last.clear();
  pl.lay = Q4Layout{};
  daa_status st = plan_check_dims(d);
  if (st != DAA_OK) return st;
  if (batch < 0) return DAA_ERR_INVALID_ARG;
  if (batch > 0) {
    if (!qo || !kv || !last) return DAA_ERR_INVALID_ARG;
    if (qo[0] != 0 || kv[0] != 0) return DAA_ERR_SHAPE;
  }
  const int P = d.page_size;
  const int g = d.num_qo_heads / d.num_kv_heads;
  // units of a request at `rows` a unit
  auto units_of = [g](int64_t nq, int rows) {
    const int64_t tokens = std::max(1, rows / g);
    return (nq + tokens - 1) / tokens;
  };
  // what units are cut from: some new tokens of a request, by class
  struct Stream {
    int r, t0, n_tok, pages, n_units, unit0;
  };
  thread_local std::vector<Stream> streams[kQ4Classes];
  for (auto& v : streams) v.clear();
  int64_t chunk_warps = 0, chunk_keys = 1;  // of requests past kQ4NativeRows
  bool chunk_split = false;
  for (int r = 0; r < batch; ++r) {
    const int64_t nq = (int64_t)qo[r + 1] - qo[r];
    const int64_t np = (int64_t)kv[r + 1] - kv[r];
    if (nq < 0 || np < 0) return DAA_ERR_SHAPE;
    if (np > 0 && (last[r] < 1 || last[r] > P)) return DAA_ERR_SHAPE;
    const int64_t kv_len = np > 0 ? (np - 1) * P + last[r] : 0;
    if (nq > kv_len || kv_len > INT32_MAX / 2) return DAA_ERR_SHAPE;
    if (nq * g > kQ4NativeRows) {
      chunk_warps += units_of(nq, kQ4UnitRows) * d.num_kv_heads;
      chunk_keys = std::max(chunk_keys, kv_len);
      chunk_split |= nq <= 2 * (kPrefillTileRows / g);
    }
  }
  const int64_t native_rows = few_chunks_q4(chunk_warps, chunk_keys, chunk_split, sms) ? INT64_MAX : kQ4NativeRows;
  int64_t small_pages = 0;  // pages that units of few rows would read
  for (int r = 0; r < batch; ++r) {
    const int64_t nq = qo[r + 1] - qo[r], np = kv[r + 1] - kv[r];
    if (nq * g > native_rows) {
      if ((int64_t)pl.src.size() + np > INT32_MAX / (2 * d.num_kv_heads)) return DAA_ERR_UNSUPPORTED;
      pl.req.push_back(r);
      pl.sub_qo.push_back(pl.sub_qo.back() + (int32_t)nq);
      pl.sub_kv.push_back(pl.sub_kv.back() + (int32_t)np);
      pl.sub_last.push_back(last[r]);
      for (int64_t p = 0; p < np; ++p) pl.src.push_back((int32_t)(kv[r] + p));
    } else {
      small_pages += np * units_of(nq, kQ4SmallUnitRows);
    }
  }
  const int64_t free_warps = (int64_t)sms * q4_warps_per_sm(0) / d.num_kv_heads;
  const int unit_rows = small_pages <= free_warps * kQ4MinPages ? kQ4SmallUnitRows : kQ4UnitRows;
  for (int r = 0; r < batch; ++r) {
    const int nq = qo[r + 1] - qo[r];
    if (nq == 0 || (int64_t)nq * g > native_rows) continue;
    const int n_units = (int)units_of(nq, unit_rows);
    for (int i = 0, t0 = 0; i < n_units; ++i) {  // as equal as they come
      const int n = (nq - t0 + n_units - i - 1) / (n_units - i);
      streams[q4_class(n * g)].push_back(Stream{r, t0, n, kv[r + 1] - kv[r], 0, 0});
      t0 += n;
    }
  }
  // Ranges: one for every warp that can be resident (over the kv heads), each with
  // the same cost of pages and units, so that all end together and none waits for
  // a second wave; a unit is cut where a range is full.
  // Beside prefill items the ranges are half as long: some warps start when the
  // prefill's SMs become free.
  // Parts: the merge takes longer with more of them, so a stream of n pages has at
  // most about 3 sqrt(n) (0.35 us a page, 0.6 us for 16 parts).
  int n_parts = 0;
  const int waves = pl.req.empty() ? 1 : 2;
  for (int cls = 0; cls < kQ4Classes; ++cls) {
    auto& ss = streams[cls];
    if (ss.empty()) continue;
    int64_t pages = 0, most = 0;
    for (const Stream& s : ss) {
      pages += s.pages;
      most += (int64_t)std::ceil(3. * std::sqrt((double)s.pages));
    }
    int64_t n_ranges = (int64_t)sms * q4_warps_per_sm(cls) * waves / d.num_kv_heads;
    n_ranges = std::max<int64_t>(1, std::min({n_ranges, most, pages / kQ4MinPages}));
    const int first_range = (int)pl.seg_begin.size() - 1;
    int64_t left_pages = pages;  // not yet in a unit
    int64_t left_streams = (int64_t)ss.size();
    // cost of the next range: what is left over the ranges left (each but the last
    // may cut a stream, which costs a unit more)
    const int unit_pages = kQ4UnitPages[cls];
    auto share = [&] {
      const int64_t left = first_range + n_ranges - (int64_t)(pl.seg_begin.size() - 1);
      return (left_pages + unit_pages * (left_streams + left - 1) + left - 1) / left;
    };
    int64_t room = share();  // of the open range
    for (Stream& s : ss) {
      s.unit0 = (int)pl.units.size();
      for (int at = 0; at < s.pages;) {
        const int left = s.pages - at;
        const bool last_range = (int)pl.seg_begin.size() - first_range == (int)n_ranges;
        if (!last_range && room < std::min<int64_t>(left, kQ4MinPages / 2) + unit_pages &&
            (int)pl.units.size() > pl.seg_begin.back()) {
          pl.seg_begin.push_back((int32_t)pl.units.size());
          room = share();
          continue;
        }
        int n = last_range ? left : (int)std::max<int64_t>(1, std::min<int64_t>(left, room - unit_pages));
        if (left - n < kQ4MinPages / 2) n = left;  // no small rest
        Q4Unit u{};
        u.tok_begin = at * P;
        u.tok_end = (at + n) * P;
        if (!pl.units.push_back(u)) return DAA_ERR_WORKSPACE;
        room -= n + unit_pages;
        left_pages -= n;
        at += n;
      }
      --left_streams;
      s.n_units = (int)pl.units.size() - s.unit0;
    }
    pl.seg_begin.push_back((int32_t)pl.units.size());
    pl.lay.n_ranges[cls] = (int)pl.seg_begin.size() - 1 - first_range;
    // the units' requests and partial slots: token t of unit s of a stream writes
    // slot part0 + t * n_units + s, so a token's parts lie side by side
    for (const Stream& s : ss) {
      const int nq = qo[s.r + 1] - qo[s.r];
      const int kv_len = (s.pages - 1) * P + last[s.r];
      const int part0 = s.n_units > 1 ? n_parts : -1;
      if (part0 >= 0) {
        for (int t = 0; t < s.n_tok; ++t)
          if (!pl.merges.push_back(MergeItem{qo[s.r] + s.t0 + t, part0 + t * s.n_units, s.n_units, -1}))
            return DAA_ERR_WORKSPACE;
        n_parts += s.n_units * s.n_tok;
      }
      for (int i = 0; i < s.n_units; ++i) {
        Q4Unit& u = pl.units.data()[s.unit0 + i];
        u.q_row = qo[s.r] + s.t0;
        u.n_tok = s.n_tok;
        u.pos0 = kv_len - nq + s.t0;
        u.kv_len = kv_len;
        u.page_base = kv[s.r];
        u.tok_end = std::min(u.tok_end, kv_len);
        u.part = part0 >= 0 ? part0 + i : -1;
        u.part_stride = s.n_units;
      }
    }
  }
  // the bf16 requests: their own plan, then its query rows moved to their place in the batch
  // (tiles and merges: a request of more rows than a group has heads has several tokens, and
  // those are never CUDA-core units)
  static_assert(kQ4NativeRows >= 16, "the largest group");
  daa_dims sd = d;
  sd.num_pages = std::max<int64_t>(1, (int64_t)pl.src.size());
  st = plan_batch(pl.sub_qo.data(), pl.sub_kv.data(), pl.sub_last.data(), (int32_t)pl.req.size(), sd,
                  sms, pl.sub_units, pl.sub_merges, pl.sub_tiles, pl.lay.sub);
  if (st != DAA_OK) return st;
  auto moved = [&](int32_t row) {
    const int i = (int)(std::upper_bound(pl.sub_qo.begin(), pl.sub_qo.end(), row) - pl.sub_qo.begin()) - 1;
    return row + qo[pl.req[i]] - pl.sub_qo[i];
  };
  for (size_t i = 0; i < pl.sub_merges.size(); ++i) {
    MergeItem& m = pl.sub_merges.data()[i];
    m.q_row = moved(m.q_row);
  }
  for (size_t i = 0; i < pl.sub_tiles.size(); ++i) {
    PrefillTile& t = pl.sub_tiles.data()[i];
    t.q_row0 = moved(t.q_row0);
  }
  pl.lay.n_units = (int)pl.units.size();
  pl.lay.n_parts = n_parts;
  pl.lay.n_merges = (int)pl.merges.size();
  pl.lay.n_scratch = (int)pl.src.size();
  pl.lay.finish(d);
  return DAA_OK;
}

// Copy the plan into a host staging buffer laid out as the workspace head.
template <template <class> class Vec>
void plan_stage_q4(const Q4Plan<Vec>& pl, uint8_t* host) {
  const Q4Layout& lay = pl.lay;
  std::memset(host, 0, lay.plan_bytes);
  if (lay.n_units) {
    std::memcpy(host + lay.off_units, pl.units.data(), lay.n_units * sizeof(Q4Unit));
    Q4Range* ranges = reinterpret_cast<Q4Range*>(host + lay.off_ranges);
    for (size_t i = 0; i + 1 < pl.seg_begin.size(); ++i)
      ranges[i] = Q4Range{pl.units.data()[pl.seg_begin[i]], pl.seg_begin[i], pl.seg_begin[i + 1], 0, 0};
  }
  if (lay.n_merges) std::memcpy(host + lay.off_merges, pl.merges.data(), lay.n_merges * sizeof(MergeItem));
  if (lay.n_scratch) {
    std::memcpy(host + lay.off_src, pl.src.data(), lay.n_scratch * sizeof(int32_t));
    int32_t* ids = reinterpret_cast<int32_t*>(host + lay.off_ids);
    for (int i = 0; i < lay.n_scratch; ++i) ids[i] = i;
  }
  if (lay.sub.total > 0)
    plan_stage(lay.sub, pl.sub_units, pl.sub_merges, pl.sub_tiles, host + lay.off_sub);
}

}  // namespace daa
