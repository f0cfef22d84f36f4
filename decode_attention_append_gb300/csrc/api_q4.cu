// C ABI of the step tables and the 4-bit KV cache: argument checks, the plan of
// attention over the 4-bit cache, and the launches.  Host code only.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "../../include/daa.h"
#include "launch.h"
#include "planner_q4.h"
#include "q4.cuh"

namespace daa {
namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <class F>
cudaError_t traced(int32_t id, cudaStream_t s, F&& f) {
  return traced_launch(id, s, [](void* ctx) { return (*static_cast<F*>(ctx))(); }, &f);
}

template <class T>
struct GrowVec {
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
using HostPlanQ4 = Q4Plan<GrowVec>;

HostPlanQ4& host_plan_q4() {
  thread_local HostPlanQ4 p;
  return p;
}

// The plan, with a failed host allocation reported and not thrown.
daa_status make_plan_q4(const int32_t* qo, const int32_t* kv, const int32_t* last, int32_t batch,
                        const daa_dims& d, HostPlanQ4& pl) {
  try {
    return plan_batch_q4(qo, kv, last, batch, d, device_sms(), pl);
  } catch (...) {
    return DAA_ERR_WORKSPACE;
  }
}

// What daa_batch_attention_q4_plan leaves in the caller's daa_plan_info.
struct PlanRecordQ4 {
  int64_t magic;
  int32_t num_qo_heads, num_kv_heads, head_dim, page_size;
  int64_t num_pages;
  int32_t batch, nnz_qo;
  int32_t n_ranges[kQ4Classes], n_units, n_merges, n_parts, n_scratch;
  PlanLayout sub;
};
constexpr int64_t kPlanMagicQ4 = 0x4441415f51345f50LL;
static_assert(sizeof(PlanRecordQ4) <= sizeof(daa_plan_info), "daa_plan_info too small");

daa_status check_pool(const daa_page_pool* p) {
  if (!p) return DAA_ERR_INVALID_ARG;
  if (p->num_slots <= 0 || p->max_pages <= 0 || p->num_pages <= 0) return DAA_ERR_INVALID_ARG;
  if (!p->seq_len || !p->held || !p->block_table || !p->free_pages || !p->counters)
    return DAA_ERR_INVALID_ARG;
  if (p->page_size != kPlanPageSize) return DAA_ERR_UNSUPPORTED;
  if (p->num_slots > DAA_STEP_MAX_SLOTS || p->max_pages > INT32_MAX / kPlanPageSize)
    return DAA_ERR_UNSUPPORTED;
  return DAA_OK;
}

StepTableArgs pool_args(const daa_page_pool& p) {
  StepTableArgs a{};
  a.seq_len = p.seq_len;
  a.held = p.held;
  a.block_table = p.block_table;
  a.free_pages = p.free_pages;
  a.counters = p.counters;
  a.num_slots = p.num_slots;
  a.max_pages = p.max_pages;
  a.num_pages = p.num_pages;
  a.err = device_error_word();
  return a;
}

}  // namespace
}  // namespace daa

using namespace daa;

extern "C" {

daa_status daa_step_table(const daa_page_pool* pool, const int32_t* slots, const int32_t* new_len,
                          int32_t batch, int32_t advance, int32_t* qo_indptr, int32_t* kv_indptr,
                          int32_t* page_indices, int32_t page_capacity, int32_t* last_page_len,
                          int64_t* slot_map, int32_t* positions, int32_t row_capacity,
                          void* stream) {
  daa_status st = check_pool(pool);
  if (st != DAA_OK) return st;
  if (batch < 0 || page_capacity < 0 || row_capacity < 0 || (advance != 0 && advance != 1))
    return DAA_ERR_INVALID_ARG;
  if (batch > DAA_STEP_MAX_BATCH) return DAA_ERR_UNSUPPORTED;
  if (!qo_indptr || !kv_indptr) return DAA_ERR_INVALID_ARG;
  if (batch > 0 && (!slots || !new_len || !last_page_len)) return DAA_ERR_INVALID_ARG;
  if (page_capacity > 0 && !page_indices) return DAA_ERR_INVALID_ARG;
  if (!aligned(slot_map, 8)) return DAA_ERR_ALIGNMENT;
  StepTableArgs a = pool_args(*pool);
  a.slots = slots;
  a.new_len = new_len;
  a.batch = batch;
  a.advance = advance;
  a.qo_indptr = qo_indptr;
  a.kv_indptr = kv_indptr;
  a.page_indices = page_indices;
  a.last_page_len = last_page_len;
  a.slot_map = slot_map;
  a.positions = positions;
  a.page_capacity = page_capacity;
  a.row_capacity = row_capacity;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(kKernelStepTable, s, [&] { return launch_step_table(a, false, device_sms(), !tracer_on(), s); }) ==
                 cudaSuccess
             ? DAA_OK
             : DAA_ERR_CUDA;
}

daa_status daa_release_pages(const daa_page_pool* pool, const int32_t* slots, int32_t batch,
                             void* stream) {
  daa_status st = check_pool(pool);
  if (st != DAA_OK) return st;
  if (batch < 0) return DAA_ERR_INVALID_ARG;
  if (batch > DAA_STEP_MAX_BATCH) return DAA_ERR_UNSUPPORTED;
  if (batch == 0) return DAA_OK;
  if (!slots) return DAA_ERR_INVALID_ARG;
  StepTableArgs a = pool_args(*pool);
  a.slots = slots;
  a.batch = batch;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(kKernelStepTable, s, [&] { return launch_step_table(a, true, device_sms(), !tracer_on(), s); }) ==
                 cudaSuccess
             ? DAA_OK
             : DAA_ERR_CUDA;
}

daa_status daa_kv_append_q4(const void* k_new, const void* v_new, void* kv_pages,
                            const int32_t* kv_exp, const int32_t* append_indptr,
                            const int32_t* page_indices, const int32_t* kv_indptr,
                            const int32_t* last_page_len, int32_t batch, int32_t nnz_new,
                            daa_dims dims, void* stream) {
  daa_status st = plan_check_dims(dims);
  if (st != DAA_OK) return st;
  if (batch < 0 || nnz_new < 0) return DAA_ERR_INVALID_ARG;
  if (nnz_new == 0 || batch == 0) return nnz_new == 0 ? DAA_OK : DAA_ERR_SHAPE;
  if (!k_new || !v_new || !kv_pages || !append_indptr || !page_indices || !kv_indptr ||
      !last_page_len)
    return DAA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(kv_pages, 16)) return DAA_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(kKernelAppendQ4, s, [&] {
           return launch_kv_append_q4(k_new, v_new, kv_pages, kv_exp, append_indptr, page_indices,
                                      kv_indptr, last_page_len, batch, nnz_new, dims.num_kv_heads,
                                      dims.head_dim, dims.num_pages, device_sms(), device_error_word(),
                                      !tracer_on(), s);
         }) == cudaSuccess
             ? DAA_OK
             : DAA_ERR_CUDA;
}

daa_status daa_kv_dequant_q4(const void* kv_pages, const int32_t* kv_exp, const int32_t* page_ids,
                             int32_t n_pages, void* out, daa_dims dims, void* stream) {
  daa_status st = plan_check_dims(dims);
  if (st != DAA_OK) return st;
  if (n_pages < 0) return DAA_ERR_INVALID_ARG;
  if (n_pages == 0) return DAA_OK;
  if (!kv_pages || !page_ids || !out) return DAA_ERR_INVALID_ARG;
  if (!aligned(kv_pages, 16) || !aligned(out, 16)) return DAA_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(kKernelDequantQ4, s, [&] {
           return launch_kv_dequant_q4(kv_pages, kv_exp, page_ids, nullptr, n_pages, dims.num_kv_heads,
                                       dims.head_dim, dims.num_pages, out, device_sms(), device_error_word(),
                                       !tracer_on(), s);
         }) == cudaSuccess
             ? DAA_OK
             : DAA_ERR_CUDA;
}

size_t daa_batch_attention_q4_workspace_size(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                             const int32_t* h_last_page_len, int32_t batch,
                                             daa_dims dims, daa_status* status) {
  HostPlanQ4& pl = host_plan_q4();
  const daa_status st = make_plan_q4(h_qo_indptr, h_kv_indptr, h_last_page_len, batch, dims, pl);
  if (status) *status = st;
  return st == DAA_OK ? pl.lay.total : 0;
}

daa_status daa_batch_attention_q4_plan(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                       const int32_t* h_last_page_len, int32_t batch, daa_dims dims,
                                       void* workspace, size_t workspace_bytes, daa_plan_info* info,
                                       void* stream) {
  if (!info) return DAA_ERR_INVALID_ARG;
  std::memset(info, 0, sizeof(*info));
  HostPlanQ4& pl = host_plan_q4();
  const daa_status st = make_plan_q4(h_qo_indptr, h_kv_indptr, h_last_page_len, batch, dims, pl);
  if (st != DAA_OK) return st;
  const Q4Layout& lay = pl.lay;
  if (lay.total > 0) {
    if (!workspace || workspace_bytes < lay.total) return DAA_ERR_WORKSPACE;
    if (!aligned(workspace, kPlanAlign)) return DAA_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the copy reads a host buffer that the next plan of this thread fills again,
    // so it cannot be replayed from a graph
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) return DAA_ERR_CUDA;
    if (cap != cudaStreamCaptureStatusNone) return DAA_ERR_UNSUPPORTED;
    thread_local std::vector<uint8_t> host;
    try {
      if (host.size() < lay.plan_bytes) host.resize(lay.plan_bytes);
    } catch (...) {
      return DAA_ERR_WORKSPACE;
    }
    plan_stage_q4(pl, host.data());
    if (cudaMemcpyAsync(workspace, host.data(), lay.plan_bytes, cudaMemcpyHostToDevice, s) != cudaSuccess)
      return DAA_ERR_CUDA;
  }
  PlanRecordQ4 rec{};
  rec.magic = kPlanMagicQ4;
  rec.num_qo_heads = dims.num_qo_heads;
  rec.num_kv_heads = dims.num_kv_heads;
  rec.head_dim = dims.head_dim;
  rec.page_size = dims.page_size;
  rec.num_pages = dims.num_pages;
  rec.batch = batch;
  rec.nnz_qo = batch > 0 ? h_qo_indptr[batch] : 0;
  for (int i = 0; i < kQ4Classes; ++i) rec.n_ranges[i] = lay.n_ranges[i];
  rec.n_units = lay.n_units;
  rec.n_merges = lay.n_merges;
  rec.n_parts = lay.n_parts;
  rec.n_scratch = lay.n_scratch;
  rec.sub = lay.sub;
  std::memcpy(info, &rec, sizeof(rec));
  return DAA_OK;
}

daa_status daa_batch_attention_q4_run(const void* q, const void* kv_pages, const int32_t* kv_exp,
                                      const int32_t* page_indices, const daa_plan_info* info,
                                      int32_t causal, float sm_scale, void* out, float* lse_out,
                                      void* workspace, size_t workspace_bytes, daa_dims dims,
                                      void* stream) {
  if (!info) return DAA_ERR_INVALID_ARG;
  PlanRecordQ4 rec;
  std::memcpy(&rec, info, sizeof(rec));
  if (rec.magic != kPlanMagicQ4 || rec.num_qo_heads != dims.num_qo_heads ||
      rec.num_kv_heads != dims.num_kv_heads || rec.head_dim != dims.head_dim ||
      rec.page_size != dims.page_size || rec.num_pages != dims.num_pages)
    return DAA_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return DAA_ERR_INVALID_ARG;
  Q4Layout lay;
  for (int i = 0; i < kQ4Classes; ++i) lay.n_ranges[i] = rec.n_ranges[i];
  lay.n_units = rec.n_units;
  lay.n_merges = rec.n_merges;
  lay.n_parts = rec.n_parts;
  lay.n_scratch = rec.n_scratch;
  lay.sub = rec.sub;
  lay.finish(dims);
  if (lay.total == 0) return DAA_OK;
  if (!q || !kv_pages || !page_indices || !out) return DAA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(out, 16) || !aligned(lse_out, 4))
    return DAA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < lay.total) return DAA_ERR_WORKSPACE;
  if (!aligned(workspace, kPlanAlign)) return DAA_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (lay.n_scratch > 0) {
    cudaError_t e = traced(kKernelDequantQ4, s, [&] {
      return launch_kv_dequant_q4(kv_pages, kv_exp, page_indices,
                                  reinterpret_cast<const int32_t*>(ws + lay.off_src), lay.n_scratch,
                                  dims.num_kv_heads, dims.head_dim, dims.num_pages, ws + lay.off_pool, device_sms(),
                                  device_error_word(), !tracer_on(), s);
    });
    if (e != cudaSuccess) return DAA_ERR_CUDA;
    LaunchSet ls{};
    ls.q = q;
    ls.kv_pages = ws + lay.off_pool;
    ls.page_indices = reinterpret_cast<const int32_t*>(ws + lay.off_ids);
    ls.dims = dims;
    ls.dims.num_pages = lay.n_scratch;
    ls.causal = causal;
    ls.sm_scale = sm_scale;
    ls.nnz_qo = rec.nnz_qo;
    ls.out = out;
    ls.lse_out = lse_out;
    ls.scratch = ws + lay.off_sub;
    ls.err = device_error_word();
    ls.sms = device_sms();
    const daa_status st = launch_all(ls, lay.sub, s, /*trace=*/true, /*after_append=*/false);
    if (st != DAA_OK) return st;
  }
  if (lay.n_units > 0) {
    AttentionQ4Args a{};
    a.q = static_cast<const uint16_t*>(q);
    a.pool = static_cast<const uint8_t*>(kv_pages);
    a.kv_exp = kv_exp;
    a.page_indices = page_indices;
    a.units = reinterpret_cast<const Q4Unit*>(ws + lay.off_units);
    a.ranges = reinterpret_cast<const Q4Range*>(ws + lay.off_ranges);
    a.Hq = dims.num_qo_heads;
    a.Hkv = dims.num_kv_heads;
    a.group = dims.num_qo_heads / dims.num_kv_heads;
    a.head_dim = dims.head_dim;
    a.num_pages = dims.num_pages;
    a.causal = causal ? 1 : 0;
    a.sm_scale = sm_scale;
    a.out = static_cast<uint16_t*>(out);
    a.lse_out = lse_out;
    a.part_o = reinterpret_cast<float*>(ws + lay.off_part_o);
    a.part_lse = reinterpret_cast<float*>(ws + lay.off_part_lse);
    a.err = device_error_word();
    // beside the bf16 requests' kernels (none of which it reads), and its merge
    // behind it; each kernel alone while the tracer times them
    const bool programmatic = !tracer_on();
    if (traced(kKernelAttentionQ4, s, [&] {
          return launch_attention_q4(a, lay.n_ranges, programmatic, programmatic && lay.n_scratch > 0, s);
        }) != cudaSuccess)
      return DAA_ERR_CUDA;
    if (lay.n_merges > 0) {
      MergeArgs m{};
      m.items = reinterpret_cast<const MergeItem*>(ws + lay.off_merges);
      m.n_items = lay.n_merges;
      m.Hq = dims.num_qo_heads;
      m.head_dim = dims.head_dim;
      m.part_o = a.part_o;
      m.part_lse = a.part_lse;
      m.out = a.out;
      m.lse_out = lse_out;
      if (traced(kKernelMerge, s, [&] { return launch_merge_q4(m, lay.n_parts, programmatic, s); }) != cudaSuccess)
        return DAA_ERR_CUDA;
    }
  }
  return DAA_OK;
}

}  // extern "C"
