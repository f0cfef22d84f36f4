// Host-side plan of attention over the 4-bit cache.
//
// "Disaggregated prefill and decode" (Perplexity), "Prefill vs decode
// performance": a long chunk is bound by the tensor cores, a decode request by
// the K/V bytes.  A request whose packed (token, query head) rows are more than
// kQ4NativeRows reads every key many times, so its pages are turned into bf16
// once, in the workspace, and it runs on the bf16 kernels (their plan, on the
// batch of these requests alone); the others are read from the 4-bit pages by
// the attention_q4 kernel.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <vector>

#include "../../include/daa.h"
#include "launch.h"
#include "planner.h"

namespace daa {

constexpr int kQ4NativeRows = 64;
constexpr int kQ4UnitsPerSm = 16;
constexpr int kQ4MinPages = 16;
constexpr int kQ4UnitRows = 32;  // rows a unit holds at most

// Sections of the workspace, all worked out from the counts and the layout of
// the bf16 requests' plan.  The first plan_bytes are copied from the host.
struct Q4Layout {
  int n_units[kQ4Classes] = {0, 0, 0};
  int n_merges = 0, n_parts = 0, n_scratch = 0;
  PlanLayout sub;
  size_t off_units, off_merges, off_src, off_ids, off_sub, plan_bytes, off_part_o, off_part_lse,
      off_pool, total;
  int units() const { return n_units[0] + n_units[1] + n_units[2]; }
  void finish(const daa_dims& d) {
    size_t off = 0;
    off_units = off;
    off = plan_align_up(off + (size_t)units() * sizeof(Q4Unit));
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
    total = units() == 0 && sub.total == 0 ? 0 : off;
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
  std::vector<int32_t> src;                    // scratch page -> index into page_indices
  std::vector<int32_t> req, sub_qo, sub_kv, sub_last;  // the bf16 requests' table
  Q4Layout lay;
};

template <template <class> class Vec>
daa_status plan_batch_q4(const int32_t* qo, const int32_t* kv, const int32_t* last, int32_t batch,
                         const daa_dims& d, int sms, Q4Plan<Vec>& pl) {
  pl.units.clear();
  pl.merges.clear();
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
  const int tpu = kQ4UnitRows / g;  // tokens of a unit
  int64_t native_pages = 0;         // pages that units read, once per unit of a request's tokens
  for (int r = 0; r < batch; ++r) {
    const int64_t nq = (int64_t)qo[r + 1] - qo[r];
    const int64_t np = (int64_t)kv[r + 1] - kv[r];
    if (nq < 0 || np < 0) return DAA_ERR_SHAPE;
    if (np > 0 && (last[r] < 1 || last[r] > P)) return DAA_ERR_SHAPE;
    const int64_t kv_len = np > 0 ? (np - 1) * P + last[r] : 0;
    if (nq > kv_len || kv_len > INT32_MAX / 2) return DAA_ERR_SHAPE;
    if (nq * g > kQ4NativeRows) {
      if ((int64_t)pl.src.size() + np > INT32_MAX / (2 * d.num_kv_heads)) return DAA_ERR_UNSUPPORTED;
      pl.req.push_back(r);
      pl.sub_qo.push_back(pl.sub_qo.back() + (int32_t)nq);
      pl.sub_kv.push_back(pl.sub_kv.back() + (int32_t)np);
      pl.sub_last.push_back(last[r]);
      for (int64_t p = 0; p < np; ++p) pl.src.push_back((int32_t)(kv[r] + p));
    } else if (nq > 0) {
      native_pages += np * ((nq + tpu - 1) / tpu);
    }
  }
  // Key splits: about kQ4UnitsPerSm units (times kv heads) an SM, so that the
  // longest is a small part of the pass and the parts to join stay few; at least
  // kQ4MinPages pages, a few for each of a CTA's warps.
  int64_t split = (native_pages * d.num_kv_heads + (int64_t)sms * kQ4UnitsPerSm - 1) /
                  ((int64_t)sms * kQ4UnitsPerSm);
  split = std::max<int64_t>(kQ4MinPages, (split + 3) / 4 * 4);
  int n_parts = 0;
  for (int r = 0; r < batch; ++r) {
    const int nq = qo[r + 1] - qo[r];
    if (nq == 0 || nq * g > kQ4NativeRows) continue;
    const int np = kv[r + 1] - kv[r];
    const int kv_len = (np - 1) * P + last[r];
    // splits cut the keys that token 0 sees, so every split starts at a key that
    // each token sees; the last one also takes the tail
    const int64_t vis = (int64_t)kv_len - nq + 1;
    const int nsplit = (int)((vis + split * P - 1) / (split * P));
    int part0 = -1;
    if (nsplit > 1) {
      part0 = n_parts;
      for (int t = 0; t < nq; ++t)
        if (!pl.merges.push_back(MergeItem{qo[r] + t, part0 + t * nsplit, nsplit, -1}))
          return DAA_ERR_WORKSPACE;
      n_parts += nsplit * nq;
    }
    for (int t0 = 0; t0 < nq; t0 += tpu)
      for (int s = 0; s < nsplit; ++s) {
        Q4Unit u{};
        u.q_row = qo[r] + t0;
        u.n_tok = std::min(tpu, nq - t0);
        u.pos0 = kv_len - nq + t0;
        u.kv_len = kv_len;
        u.page_base = kv[r];
        u.tok_begin = (int)(s * split * P);
        u.tok_end = s == nsplit - 1 ? kv_len : (int)((s + 1) * split * P);
        u.part = part0 >= 0 ? part0 + t0 * nsplit + s : -1;
        u.part_stride = nsplit;
        if (!pl.units.push_back(u)) return DAA_ERR_WORKSPACE;
      }
  }
  // by class, then longest first
  auto cls = [g](const Q4Unit& u) { return u.n_tok * g <= 8 ? 0 : (u.n_tok * g <= 16 ? 1 : 2); };
  std::sort(pl.units.data(), pl.units.data() + pl.units.size(), [&](const Q4Unit& x, const Q4Unit& y) {
    if (cls(x) != cls(y)) return cls(x) < cls(y);
    const int a = x.tok_end - x.tok_begin, b = y.tok_end - y.tok_begin;
    return a != b ? a > b : (x.q_row != y.q_row ? x.q_row < y.q_row : x.tok_begin < y.tok_begin);
  });
  for (size_t i = 0; i < pl.units.size(); ++i) ++pl.lay.n_units[cls(pl.units.data()[i])];
  // the bf16 requests: their own plan, then its query rows moved to their place in the batch
  daa_dims sd = d;
  sd.num_pages = std::max<int64_t>(1, (int64_t)pl.src.size());
  st = plan_batch(pl.sub_qo.data(), pl.sub_kv.data(), pl.sub_last.data(), (int32_t)pl.req.size(), sd,
                  sms, pl.sub_units, pl.sub_merges, pl.sub_tiles, pl.lay.sub);
  if (st != DAA_OK) return st;
  auto moved = [&](int32_t row) {
    const int i = (int)(std::upper_bound(pl.sub_qo.begin(), pl.sub_qo.end(), row) - pl.sub_qo.begin()) - 1;
    return row + qo[pl.req[i]] - pl.sub_qo[i];
  };
  for (size_t i = 0; i < pl.sub_units.size(); ++i) {
    DecodeUnit& u = pl.sub_units.data()[i];
    u.q_row = moved(u.q_row);
  }
  for (size_t i = 0; i < pl.sub_merges.size(); ++i) {
    MergeItem& m = pl.sub_merges.data()[i];
    m.q_row = moved(m.q_row);
  }
  for (size_t i = 0; i < pl.sub_tiles.size(); ++i) {
    PrefillTile& t = pl.sub_tiles.data()[i];
    t.q_row0 = moved(t.q_row0);
  }
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
  if (lay.units()) std::memcpy(host + lay.off_units, pl.units.data(), lay.units() * sizeof(Q4Unit));
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
