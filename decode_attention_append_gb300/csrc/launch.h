// Host-side launchers of the CUDA kernels (one translation unit each).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/daa.h"
#include "plan.h"

namespace daa {

// Address of this library's device error word on the current device.
int* device_error_word();

// Launch `kern` on `s`; with `programmatic`, as a programmatic dependent launch
// (its CTAs may start while the previous kernel on the stream is still running
// and must call grid_dep_wait before reading what that kernel writes).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t s, bool programmatic, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = programmatic ? attr : nullptr;
  cfg.numAttrs = programmatic ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Key tiles are 128 keys; with the prefill append fused (fuse_min_qo > 0), a
// request with qo_len >= fuse_min_qo has its new tokens at positions
// >= fused_from(kv_len, qo_len) written by the prefill kernel, not the append.
constexpr int kFuseTileKeys = 128;
__host__ __device__ inline int fused_from(int kv_len, int qo_len) {
  const int c = kv_len - qo_len;
  return (c + kFuseTileKeys - 1) / kFuseTileKeys * kFuseTileKeys;
}

// Appends rows [row_begin, row_begin + n_rows) of k_new / v_new (all rows:
// 0, nnz_new).  fuse_min_qo: 0 appends every row of that span; otherwise rows
// that the prefill kernel writes itself (see fused_from) are skipped.
cudaError_t launch_kv_append(const void* k_new, const void* v_new, void* pool,
                             const int32_t* append_indptr, const int32_t* page_indices,
                             const int32_t* kv_indptr, const int32_t* last_page_len, int batch,
                             int row_begin, int n_rows, int Hkv, int head_dim, int64_t num_pages,
                             int num_sms, int fuse_min_qo, int* err, cudaStream_t stream);

// The span of rows the append kernel of a fused call must cover: every row
// except those the prefill kernels write (a request's new tokens from
// fused_from on when qo_len >= fuse_min_qo).  Host side, from the host copies
// of the lengths; begin == end when there is none.
struct AppendSpan {
  int begin, end;
};
AppendSpan append_span(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                       const int32_t* h_last_page_len, int batch, int page_size, int fuse_min_qo);

struct DecodeArgs {
  const uint16_t* q;            // [nnz_qo][Hq][d]
  const uint16_t* pool;         // [num_pages][2][Hkv][P][d]
  const int32_t* page_indices;
  const DecodeUnit* units;      // device
  int n_units;
  int Hq, Hkv, group;           // group = Hq / Hkv
  int head_dim;
  int64_t num_pages;
  float sm_scale_log2;          // sm_scale * log2(e)
  uint16_t* out;                // [nnz_qo][Hq][d]
  float* lse_out;               // [nnz_qo][Hq] natural log, or null
  float* part_o;                // [n_parts][Hq][d]
  float* part_lse;              // [n_parts][Hq] (log2 domain)
  int* err;
};
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream, bool programmatic);

struct MergeArgs {
  const MergeItem* items;       // device
  int n_items;
  int Hq, head_dim;
  const float* part_o;
  const float* part_lse;
  uint16_t* out;
  float* lse_out;
};
cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream, bool programmatic);

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* pool;
  const int32_t* page_indices;
  const PrefillTile* tiles;     // device: prefill items
  int n_tiles;
  const PrefillTile* short_tiles;  // device: short multi-token items (single-CTA kernel)
  int n_short_tiles;
  const PrefillTile* dec_tiles; // device: decode and verify items
  int n_dec_tiles;
  int Hq, Hkv, group, head_dim;
  int64_t num_pages;
  int nnz_qo;
  int causal;
  float sm_scale_log2;
  uint16_t* out;
  float* lse_out;
  float* part_o;                // split items: [n_parts][Hq][d]
  float* part_lse;              // split items: [n_parts][Hq] (log2 domain)
  const uint32_t* tree_mask;    // draft-tree mask rows [nnz_qo][mask_words], or null
  int mask_words;
  int* err;
  int* dec_counter;             // persistent decode kernel: [0] work counter, [1] CTAs
                                // finished; zero before a launch, reset to zero by it
  int sms;                      // SMs of the device (persistent grid size)
  // Prefill append fused into the prefill kernels (the fused call
  // only; fuse_min_qo == 0 otherwise).  For a prefill item of a request with
  // qo_len >= fuse_min_qo, key tiles from fused_from(kv_len, qo_len) on are
  // read from k_new / v_new (rows laid out like q) instead of the pool, and the
  // item that holds a tile's first new token writes the tile's rows into their
  // pages (pool_w).
  const uint16_t* k_new;        // [nnz_qo][Hkv][d]
  const uint16_t* v_new;
  uint16_t* pool_w;
  int fuse_min_qo;
};
// Rows of packed (token, head) a prefill tile holds.
constexpr int kPrefillTileRows = 128;
// Single-CTA tensor-core kernel over `tiles` (pairs of 128-row Q tiles: the
// prefill items for head_dim 64, the short items for head_dim 128), and the
// decode instantiation over the decode / verify items (one Q tile, two CTAs
// per SM).
cudaError_t launch_prefill(const PrefillArgs& a, const PrefillTile* tiles, int n_tiles,
                           cudaStream_t stream, bool programmatic);
// head_dim 128: prefill items of four Q tiles on clusters of two CTAs
// (tcgen05 cta_group::2); grid (2 * n_tiles, Hkv).
cudaError_t launch_prefill_pair(const PrefillArgs& a, cudaStream_t stream, bool programmatic);
cudaError_t launch_tc_decode(const PrefillArgs& a, cudaStream_t stream, bool programmatic);

// Everything one batch_attention call launches, given its plan in `scratch`
// (the workspace, or the no-allocation entry point's static array).
struct LaunchSet {
  const void* q;
  const void* kv_pages;
  const int32_t* page_indices;
  daa_dims dims;
  int causal;
  float sm_scale;
  int nnz_qo;
  void* out;
  float* lse_out;
  const uint32_t* tree_mask;    // draft-tree mask rows, or null
  int mask_words;
  void* scratch;
  int* err;
  int sms;
  // the fused call's new rows and the fusion threshold (see PrefillArgs)
  const void* k_new;
  const void* v_new;
  int fuse_min_qo;
};
struct PlanLayout;

// ------------------------------------------------------- step tables, 4-bit cache
// These kernels are launched programmatically (unless the tracer times them): each
// lets the next one start its CTAs at once and waits for the kernel before it
// before its first access, so that of two in a row only the launch overlaps.
// Step tables from request lengths (step_table.cu); release: only slots, batch
// and the pool are read.
struct StepTableArgs {
  const int32_t* slots;    // [batch]
  const int32_t* new_len;  // [batch]
  int batch;
  int advance;             // 1: seq_len += new_len
  int32_t* seq_len;        // [num_slots]
  int32_t* held;           // [num_slots]
  int32_t* block_table;    // [num_slots][max_pages]
  int32_t* free_pages;     // [num_pages], a stack
  int32_t* counters;       // [2]: free pages, CTAs finished (0 between calls)
  int num_slots, max_pages;
  int num_pages;
  int32_t* qo_indptr;      // [batch + 1]
  int32_t* kv_indptr;      // [batch + 1]
  int32_t* page_indices;   // [page_capacity]
  int32_t* last_page_len;  // [batch]
  int64_t* slot_map;       // [row_capacity] or null
  int32_t* positions;      // [row_capacity] or null
  int page_capacity, row_capacity;
  int* err;
};
size_t step_table_smem(int batch, int num_slots);
cudaError_t launch_step_table(const StepTableArgs& a, bool release, int sms, bool programmatic,
                              cudaStream_t stream);

// 4-bit cache (append_q4.cu): the quantising append, and pages as bf16.
// kv_exp: [2][Hkv] or null.  dequant: out page i is pool page ids[src ? src[i] : i].
cudaError_t launch_kv_append_q4(const void* k_new, const void* v_new, void* pool,
                                const int32_t* kv_exp, const int32_t* append_indptr,
                                const int32_t* page_indices, const int32_t* kv_indptr,
                                const int32_t* last_page_len, int batch, int nnz_new, int Hkv,
                                int head_dim, int64_t num_pages, int sms, int* err,
                                bool programmatic, cudaStream_t stream);
cudaError_t launch_kv_dequant_q4(const void* pool, const int32_t* kv_exp, const int32_t* ids,
                                 const int32_t* src, int64_t n_pages, int Hkv, int head_dim,
                                 int64_t num_pages, void* out, int sms, int* err, bool programmatic,
                                 cudaStream_t stream);

// Attention over the 4-bit pages (decode_q4.cu); n_ranges per class, in order.
struct AttentionQ4Args {
  const uint16_t* q;       // [nnz_qo][Hq][d]
  const uint8_t* pool;     // [num_pages][Hkv][2][9 d]
  const int32_t* kv_exp;   // [2][Hkv] or null
  const int32_t* page_indices;
  const Q4Unit* units;
  const Q4Range* ranges;
  int n_ranges;            // set by the launch of each class
  int wait_first;          // read nothing before the kernel before has completed
  int Hq, Hkv, group, head_dim;
  int64_t num_pages;
  int causal;
  float sm_scale;
  uint16_t* out;
  float* lse_out;          // or null
  float* part_o;           // [n_parts][Hq][d]
  float* part_lse;         // [n_parts][Hq] (log2 domain)
  int* err;
};
// beside: the kernel before on the stream is of the same call and is not read.
cudaError_t launch_attention_q4(const AttentionQ4Args& a, const int (&n_ranges)[kQ4Classes],
                                bool programmatic, bool beside, cudaStream_t stream);
// softmax_merge of its n_parts parts (items without a prefix part).
cudaError_t launch_merge_q4(const MergeArgs& a, int n_parts, bool programmatic, cudaStream_t stream);

// ------------------------------------------------------- rotary positions (rope.cu)
// Launched programmatically like the kernels above.  Rows of bf16 heads, strides in
// elements.
struct RopeRows {
  uint16_t* p;  // null: there are none
  int64_t row, head;
};
enum RopeTarget { kRopeRows = 0, kRopePages = 1, kRopePagesQ4 = 2 };
struct RopeArgs {
  uint64_t turns[64];      // of pair i: turns a token, in 2^-64 of a turn, modulo one
  RopeRows q, k, v, q_out, k_out;  // v: appends only; k_out: kRopeRows only
  int n_rows, Hq, Hk;      // Hq 0: no query rows; Hk: kv heads
  int rotary_dim, interleaved;
  float magnitude, magnitude_low, eps;  // the magnitude in two parts
  const uint16_t *q_norm, *k_norm;  // [head_dim] or null
  const int32_t* positions;         // [n_rows]; null: those of the page table
  uint8_t* pool;           // bf16 or 4-bit pages
  const int32_t* kv_exp;   // [2][Hk] or null (4-bit)
  const int32_t *append_indptr, *page_indices, *kv_indptr, *last_page_len;
  int batch;
  int64_t num_pages;
  int* err;
  int parts, part_heads;   // of a row, one a warp; set by the launch
};
cudaError_t launch_rope(const RopeArgs& a, int head_dim, RopeTarget target, int sms, bool programmatic,
                        cudaStream_t stream);

// SMs of the current device, and a launch between the tracer's events (api.cu).
int device_sms();
bool tracer_on();
cudaError_t traced_launch(int32_t kernel_id, cudaStream_t s, cudaError_t (*launch)(void*), void* ctx);
// The kernels run in the order prefill, decode, softmax_merge; each after the
// first is a programmatic dependent launch, and so is the first when
// `after_append` (this call's own kv_append kernel precedes it on the stream).
// Ordering contract, kept by the kernels:
//  * every CTA that reads rows the append wrote (all prefill CTAs, the last
//    key split of each decode request) calls grid_dep_wait first; so does
//    every softmax_merge CTA.  The completion of a kernel therefore implies the
//    completion of the kernel before it, and the last kernel's completion (what
//    later stream work waits for) implies that of the whole chain;
//  * the other decode splits read only cached rows and overlap the kernel
//    before them.
daa_status launch_all(const LaunchSet& ls, const PlanLayout& lay, cudaStream_t s, bool trace,
                      bool after_append);

}  // namespace daa
