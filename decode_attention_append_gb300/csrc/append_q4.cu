// The 4-bit cache's append (quantise and scatter) and its read-back as bf16.
//
// "Chunked prefill" (k4i.top), #correctness: after a chunk its k, v vectors
// join the cache; #io-overhead sizes that traffic.  Here a row is stored in 4.5
// bits a value (q4.cuh has the format):
//   y = x * 2^-e,  s = e4m3(clamp(max|y| / 6, 2^-9, 448)),  q = e2m1(y / s),
// both roundings to the nearest value, ties to even.  NaN is stored as zero and
// an infinity as the block's largest value: the cache holds finite numbers only,
// so a key that a mask hides can never spoil a sum with 0 * NaN.
//
// Rounding a quotient without a division: y has the 8 significant bits of a bf16
// and every midpoint of two e2m1 values times s has at most 7, so y / s is either
// exactly a midpoint or at least 2^-9 (relative) away from one.  y * (1 / s), with
// an approximate reciprocal, is off by less than 2^-21, so rounding it to fp16
// (11 bits, a half step of 2^-11 at most) lands on the midpoint exactly when y / s
// does, and the conversion's tie rule then applies to the exact quotient.  max|y| / 6
// is rounded to e4m3 the same way: 6 times a midpoint of two e4m3 values (5
// significant bits) has at most 7.
//
// Bound: HBM (2 + 9/16 bytes a value) and the 11 instructions a value (widen, scale,
// the maximum taken on packed bits, two conversions a pair, addresses): 36,760 tokens
// of 8 heads of 128 dims 37 us on GB300, launch and ramp among them, 5.2 TB/s, 60 % of
// the issue slots; without the stores 35, without the arithmetic 36.  A step of 128
// single tokens is latency: 5.4 us with the launch.
//
// The read-back moves 9/16 + 2 bytes a value at 6.4 TB/s: 8,192 pages of 8
// heads of 128 dims in 106.8 us (with a thread's 16 dims stored side by side, half a
// sector at a time: 110.7 at best).
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace daa {
namespace {

constexpr int kThreads = 128;
// Blocks of 16 dims per thread in flight: two for small appends (a CTA's chain of
// loads is what they wait for, so they are cut fine: a step of 128 tokens 8.3 us with
// its read-back, 10.3 with six), six once the CTAs fill the GPU more than once
// (36,760 tokens, with the read-back 70.4 us; with two 74.2, with eight 75.5; CTAs that
// stay and load the next chunk while they quantise one: 72.4).
constexpr int kSmallU = 2, kLargeU = 6;
constexpr int kMaxBatch = 1023;                 // requests whose indptr a CTA holds

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 32 bytes at once, where the address allows it: the two 16-byte loads of a block
// would each ask for half of every 32-byte sector of the warp's kilobyte.
__device__ __forceinline__ void ld_stream_32(const uint4* p, uint4& a, uint4& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

// The largest |value| of 16 bf16 values as bits, taken two at a time: without a
// sign bf16 values are ordered as their bits, and NaN is above infinity.
__device__ __forceinline__ uint32_t max_abs_bits(const uint32_t (&w)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}

// One block of 16 bf16 values -> 8 code bytes and the scale byte.
__device__ __forceinline__ uint2 quantise_block(const uint4& a, const uint4& b, float two_to_minus_e,
                                                uint8_t& scale) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = max_abs_bits(w);
  if (top > 0x7F80u) {  // a NaN: they count as zeros
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((w[i] & 0x7FFFu) > 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] & 0x7FFF0000u) > 0x7F800000u) w[i] &= 0x0000FFFFu;
    }
    top = max_abs_bits(w);
  }
  const float amax = __uint_as_float(top << 16);
  const float s6 = fminf(fmaxf(amax * two_to_minus_e * (1.f / 6.f), 0.001953125f), 448.f);
  const uint16_t sb = f16x2_to_e4m3x2(f32x2_to_f16x2(s6, 0.f));
  const float r = rcp_approx(f16x2_to_f32x2(e4m3x2_to_f16x2(sb)).x) * two_to_minus_e;
  scale = (uint8_t)(sb & 0xFFu);
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = f32x2_to_f16x2(bf16lo_to_f32(w[i]) * r, bf16hi_to_f32(w[i]) * r);
  const uint32_t lo[4] = {h[0], h[1], h[2], h[3]}, hi[4] = {h[4], h[5], h[6], h[7]};
  return make_uint2(f16x8_to_e2m1x8(lo), f16x8_to_e2m1x8(hi));
}

// Flat blocks (row, head, block of 16 dims) of K (blockIdx.y 0) or V (1), cut
// into equal contiguous ranges, one per CTA; the owner of each row a CTA
// touches is found once by binary search.
template <int D, int kAppendU>
__global__ void __launch_bounds__(kThreads)
kv_append_q4_kernel(const uint4* k_new, const uint4* v_new,
                    uint8_t* __restrict__ pool, const int32_t* kv_exp,
                    const int32_t* append_indptr,
                    const int32_t* page_indices, const int32_t* kv_indptr,
                    const int32_t* last_page_len, int batch, int nnz_new, int Hkv,
                    int step_rows, int step_blocks, int64_t num_pages, int* err) {
  constexpr int P = kQ4Page, NB = D / kQ4Block, SLICE = q4_slice_bytes(D);
  constexpr int kAppendSpan = kThreads * kAppendU;
  constexpr int kMaxRows = kAppendSpan / NB + 2;  // rows a CTA touches (a row has NB blocks or more)
  __shared__ int64_t s_page[kMaxRows];  // page * Hkv of the row, -1: not written
  __shared__ int s_slot[kMaxRows];
  __shared__ int s_indptr[kMaxBatch + 1], s_kv[kMaxBatch + 1], s_last[kMaxBatch + 1];
  grid_dep_launch();
  grid_dep_wait();
  const int kv = blockIdx.y;
  const int per_row = Hkv * NB;
  const int64_t total = (int64_t)nnz_new * per_row;
  const int64_t first = (int64_t)blockIdx.x * kAppendSpan;
  const int64_t last = min(first + kAppendSpan, total);
  const int row0 = (int)(first / per_row);
  const int in_row0 = (int)(first - (int64_t)row0 * per_row);
  const int nrows = (in_row0 + (int)(last - first) - 1) / per_row + 1;
  // the values do not depend on the page table: load them first
  const uint4* src = kv == 0 ? k_new : v_new;
  uint4 a[kAppendU], b[kAppendU];
  if (reinterpret_cast<uintptr_t>(src) % 32 == 0) {
#pragma unroll
    for (int u = 0; u < kAppendU; ++u) {
      const int64_t i = first + u * kThreads + threadIdx.x;
      if (i < last) ld_stream_32(src + 2 * i, a[u], b[u]);
    }
  } else {
#pragma unroll
    for (int u = 0; u < kAppendU; ++u) {
      const int64_t i = first + u * kThreads + threadIdx.x;
      if (i < last) {
        a[u] = ld_stream(src + 2 * i);
        b[u] = ld_stream(src + 2 * i + 1);
      }
    }
  }
  // the search for a row's request and its lengths are a chain of loads: in shared
  // memory where the arrays fit, so that a CTA waits for memory twice and not ten times
  const int32_t *indptr = append_indptr, *kv_begin = kv_indptr, *last_lens = last_page_len;
  if (batch <= kMaxBatch) {
    for (int t = threadIdx.x; t <= batch; t += kThreads) {
      s_indptr[t] = ld_word(append_indptr + t);
      s_kv[t] = ld_word(kv_indptr + t);
      s_last[t] = t < batch ? ld_word(last_page_len + t) : 0;
    }
    __syncthreads();
    indptr = s_indptr;
    kv_begin = s_kv;
    last_lens = s_last;
  }
  for (int t = threadIdx.x; t < nrows; t += kThreads) {
    const int row = row0 + t;
    int lo = 0, hi = batch - 1;  // largest r with indptr[r] <= row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (indptr[mid] <= row) lo = mid; else hi = mid - 1;
    }
    const int a0 = indptr[lo], a1 = indptr[lo + 1];
    const int p0 = kv_begin[lo], np = kv_begin[lo + 1] - p0;
    const int last_len = np > 0 ? last_lens[lo] : 0;
    const int64_t kv_len = np > 0 ? (int64_t)(np - 1) * P + last_len : 0;
    int64_t at = -1;
    int slot = 0;
    if (row < a0 || row >= a1 || a1 - a0 > kv_len || (np > 0 && (last_len < 1 || last_len > P))) {
      set_device_error(err, kDevErrShape);
    } else {
      const int64_t pos = kv_len - (a1 - a0) + (row - a0);
      const int64_t page = ld_word(page_indices + p0 + pos / P);
      slot = (int)(pos % P);
      if (page < 0 || page >= num_pages) set_device_error(err, kDevErrPageRange);
      else at = page * Hkv;
    }
    s_page[t] = at;
    s_slot[t] = slot;
  }
  __syncthreads();
  // a thread's blocks are kThreads = step_rows * per_row + step_blocks apart
  int next_row = (in_row0 + (int)threadIdx.x) / per_row;
  int next_hb = in_row0 + (int)threadIdx.x - next_row * per_row;
#pragma unroll
  for (int u = 0; u < kAppendU; ++u) {
    const int row = next_row, hb = next_hb;
    next_row += step_rows;
    next_hb += step_blocks;
    if (next_hb >= per_row) {
      next_hb -= per_row;
      ++next_row;
    }
    if (first + u * kThreads + threadIdx.x >= last) continue;
    const int h = (int)((unsigned)hb / NB), blk = (int)((unsigned)hb % NB);
    const int64_t page = s_page[row];
    if (page < 0) continue;
    const int slot = s_slot[row];
    const float me = kv_exp ? q4_pow2(-ld_word(kv_exp + kv * Hkv + h)) : 1.f;
    uint8_t sc;
    const uint2 codes = quantise_block(a[u], b[u], me, sc);
    uint8_t* slice = pool + ((page + h) * 2 + kv) * (int64_t)SLICE;
    *reinterpret_cast<uint2*>(slice + slot * (D / 2) + blk * 8) = codes;
    slice[P * (D / 2) + (kv == 0 ? slot * NB + blk : blk * P + slot)] = sc;
  }
}

// Pages -> bf16: a thread takes 8 dims of tokens tok and tok + 8 of a slice (so that
// a warp's 16-byte stores lie side by side), kDeqU slices at a time.  Scratch page i
// comes from pool page ids[src ? src[i] : i].
// Two slices a CTA until the CTAs fill the GPU twice (1,290 of 64 dims: 4.2 us, with four
// 6.1), then four (8,192 pages: 106.8 us, with two 110.3).
constexpr int kDeqSmallU = 2, kDeqLargeU = 4;

template <int D, int kDeqU>
__global__ void __launch_bounds__(D, 2048 / D)
kv_dequant_q4_kernel(const uint8_t* pool, const int32_t* kv_exp,
                     const int32_t* ids, const int32_t* src,
                     int64_t n_slices, int Hkv, int64_t num_pages, uint16_t* __restrict__ out,
                     int* err) {
  constexpr int P = kQ4Page, NB = D / kQ4Block, SLICE = q4_slice_bytes(D);
  grid_dep_launch();
  grid_dep_wait();
  const int tok = threadIdx.x / (D / 8), chunk = threadIdx.x % (D / 8), blk = chunk / 2;
  // slice s0 = blockIdx.x * kDeqU is slice `rem` of page i (32-bit divisions only)
  const int per_page = 2 * Hkv;
  const int64_t s0 = (int64_t)blockIdx.x * kDeqU;
  const int n = (int)min((int64_t)kDeqU, n_slices - s0);
  const unsigned groups = blockIdx.x / (unsigned)per_page;
  const unsigned in_group = (blockIdx.x - groups * per_page) * kDeqU;
  int i = (int)(groups * kDeqU + in_group / (unsigned)per_page);
  int rem = (int)(in_group % (unsigned)per_page);
  // rounds of loads, each of all slices at once: page ids (by way of src), codes
  int page[kDeqU], at[kDeqU];  // at: K (0) or V (Hkv) plus head
#pragma unroll
  for (int u = 0; u < kDeqU; ++u) {
    at[u] = rem;
    page[u] = i;
    if (++rem == per_page) {
      rem = 0;
      ++i;
    }
  }
  if (src) {
#pragma unroll
    for (int u = 0; u < kDeqU; ++u)
      if (u < n) page[u] = ld_word(src + page[u]);
  }
#pragma unroll
  for (int u = 0; u < kDeqU; ++u)
    if (u < n) page[u] = ld_word(ids + page[u]);
  uint32_t codes[kDeqU][2];
  uint32_t sc[kDeqU];
#pragma unroll
  for (int u = 0; u < kDeqU; ++u) {
    codes[u][0] = codes[u][1] = sc[u] = 0;
    if (u >= n) continue;
    if ((uint32_t)page[u] < (uint64_t)num_pages) {  // another one reads as zeros
      const int kv = at[u] >= Hkv, h = kv ? at[u] - Hkv : at[u];
      const uint8_t* slice = pool + (((int64_t)page[u] * Hkv + h) * 2 + kv) * SLICE;
      const uint8_t* row = slice + tok * (D / 2) + chunk * 4;
      codes[u][0] = (uint32_t)ld_word(row);
      codes[u][1] = (uint32_t)ld_word(row + 8 * (D / 2));
      const uint8_t* s8 = slice + P * (D / 2) + (kv == 0 ? tok * NB + blk : blk * P + tok);
      sc[u] = ld_byte(s8) | ld_byte(s8 + (kv == 0 ? 8 * NB : 8)) << 8;
    } else if (threadIdx.x == 0) {
      set_device_error(err, kDevErrPageRange);
    }
  }
#pragma unroll
  for (int u = 0; u < kDeqU; ++u) {
    if (u >= n) break;
    const float two_e = kv_exp ? q4_pow2(ld_word(kv_exp + at[u])) : 1.f;
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)sc[u]);
    uint4* dst = reinterpret_cast<uint4*>(out + ((s0 + u) * P + tok) * D + chunk * 8);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t sj = __byte_perm(s2, s2, j == 0 ? 0x1010 : 0x3232);
      uint32_t h[4], o[4];
      e2m1x8_to_f16x2(codes[u][j], h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = f16x2_to_f32x2(mul_f16x2(h[k], sj));
        o[k] = pack_bf16x2(f.x * two_e, f.y * two_e);
      }
      dst[j * D] = make_uint4(o[0], o[1], o[2], o[3]);  // 8 rows of D / 8 uint4
    }
  }
}

}  // namespace

cudaError_t launch_kv_append_q4(const void* k_new, const void* v_new, void* pool,
                                const int32_t* kv_exp, const int32_t* append_indptr,
                                const int32_t* page_indices, const int32_t* kv_indptr,
                                const int32_t* last_page_len, int batch, int nnz_new, int Hkv,
                                int head_dim, int64_t num_pages, int sms, int* err, bool programmatic,
                                cudaStream_t stream) {
  if (nnz_new <= 0 || batch <= 0) return cudaSuccess;
  const int64_t total = (int64_t)nnz_new * Hkv * (head_dim / kQ4Block);
  const bool large = total >= (int64_t)sms * 16 * kThreads * kSmallU;  // 16 CTAs an SM
  const int span = kThreads * (large ? kLargeU : kSmallU);
  const int64_t grid = (total + span - 1) / span;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = head_dim == 128 ? (large ? kv_append_q4_kernel<128, kLargeU> : kv_append_q4_kernel<128, kSmallU>)
                              : (large ? kv_append_q4_kernel<64, kLargeU> : kv_append_q4_kernel<64, kSmallU>);
  return launch_kernel(kern, dim3((unsigned)grid, 2), dim3(kThreads), 0, stream, programmatic,
                       (const uint4*)k_new, (const uint4*)v_new, (uint8_t*)pool, kv_exp, append_indptr,
                       page_indices, kv_indptr, last_page_len, batch, nnz_new, Hkv,
                       kThreads / (Hkv * (head_dim / kQ4Block)), kThreads % (Hkv * (head_dim / kQ4Block)),
                       num_pages, err);
}

cudaError_t launch_kv_dequant_q4(const void* pool, const int32_t* kv_exp, const int32_t* ids,
                                 const int32_t* src, int64_t n_pages, int Hkv, int head_dim,
                                 int64_t num_pages, void* out, int sms, int* err, bool programmatic,
                                 cudaStream_t stream) {
  if (n_pages <= 0) return cudaSuccess;
  const int64_t n_slices = n_pages * 2 * Hkv;
  const bool large = n_slices * head_dim >= (int64_t)sms * 2048 * kDeqSmallU;
  const int per_cta = large ? kDeqLargeU : kDeqSmallU;
  const int64_t grid = (n_slices + per_cta - 1) / per_cta;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = head_dim == 128 ? (large ? kv_dequant_q4_kernel<128, kDeqLargeU> : kv_dequant_q4_kernel<128, kDeqSmallU>)
                              : (large ? kv_dequant_q4_kernel<64, kDeqLargeU> : kv_dequant_q4_kernel<64, kDeqSmallU>);
  return launch_kernel(kern, dim3((unsigned)grid), dim3(head_dim), 0, stream,
                       programmatic, (const uint8_t*)pool, kv_exp, ids, src, n_slices, Hkv, num_pages,
                       (uint16_t*)out, err);
}

}  // namespace daa
