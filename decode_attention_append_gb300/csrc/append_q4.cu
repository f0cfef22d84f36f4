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
// Rounding y / s without a division per value: y has the 8 significant bits of
// a bf16 and every midpoint of two e2m1 values times s has at most 7, so y / s
// is either exactly a midpoint or at least 2^-9 (relative) away from one.
// y * (1 / s) is off by at most 2^-23, so rounding it to fp16 (11 bits, a half
// step of 2^-11 at most) lands on the midpoint exactly when y / s does, and the
// conversion's tie rule then applies to the exact quotient.
//
// Bound: HBM (2 + 9/16 bytes a value); about four instructions a value (widen,
// scale, the maximum taken on packed bits, two conversions a pair).
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace daa {
namespace {

constexpr int kThreads = 128;
// Blocks of 16 dims per thread in flight: two for small appends (a CTA's chain of
// loads is what they wait for, so they are cut fine), six once the CTAs fill the
// GPU more than once.
constexpr int kSmallU = 2, kLargeU = 6;
constexpr int kMaxBatch = 1023;                 // requests whose indptr a CTA holds

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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
  // clamp(max|y| / 6): a true division, so that its ties are ties
  const float s6 = fminf(fmaxf(__fdiv_rn(amax * two_to_minus_e, 6.f), 0.001953125f), 448.f);
  const uint16_t sb = f32x2_to_e4m3x2(s6, 0.f);
  const float r = __fdiv_rn(1.f, f16x2_to_f32x2(e4m3x2_to_f16x2(sb)).x) * two_to_minus_e;
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
kv_append_q4_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                    uint8_t* __restrict__ pool, const int32_t* __restrict__ kv_exp,
                    const int32_t* __restrict__ append_indptr,
                    const int32_t* __restrict__ page_indices, const int32_t* __restrict__ kv_indptr,
                    const int32_t* __restrict__ last_page_len, int batch, int nnz_new, int Hkv,
                    int64_t num_pages, int* err) {
  constexpr int P = kQ4Page, NB = D / kQ4Block, SLICE = q4_slice_bytes(D);
  constexpr int kAppendSpan = kThreads * kAppendU;
  constexpr int kMaxRows = kAppendSpan / NB + 2;  // rows a CTA touches (a row has NB blocks or more)
  __shared__ int64_t s_page[kMaxRows];  // page * Hkv of the row, -1: not written
  __shared__ int s_slot[kMaxRows];
  __shared__ int s_indptr[kMaxBatch + 1];
  grid_dep_launch();
  grid_dep_wait();
  const int kv = blockIdx.y;
  const int per_row = Hkv * NB;
  const int64_t total = (int64_t)nnz_new * per_row;
  const int64_t first = (int64_t)blockIdx.x * kAppendSpan;
  const int64_t last = min(first + kAppendSpan, total);
  const int row0 = (int)(first / per_row);
  const int in_row0 = (int)(first - (int64_t)row0 * per_row);
  const int nrows = (int)((last - 1) / per_row) - row0 + 1;
  // the values do not depend on the page table: load them first
  const uint4* src = kv == 0 ? k_new : v_new;
  uint4 a[kAppendU], b[kAppendU];
#pragma unroll
  for (int u = 0; u < kAppendU; ++u) {
    const int64_t i = first + u * kThreads + threadIdx.x;
    if (i < last) {
      a[u] = ld_stream(src + 2 * i);
      b[u] = ld_stream(src + 2 * i + 1);
    }
  }
  // the search for a row's request is a chain of loads: in shared memory where the
  // array fits, so that a small append waits for memory three times and not ten
  const int32_t* indptr = append_indptr;
  if (batch <= kMaxBatch) {
    for (int t = threadIdx.x; t <= batch; t += kThreads) s_indptr[t] = __ldg(append_indptr + t);
    __syncthreads();
    indptr = s_indptr;
  }
  for (int t = threadIdx.x; t < nrows; t += kThreads) {
    const int row = row0 + t;
    int lo = 0, hi = batch - 1;  // largest r with indptr[r] <= row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (indptr[mid] <= row) lo = mid; else hi = mid - 1;
    }
    const int a0 = indptr[lo], a1 = indptr[lo + 1];
    const int p0 = __ldg(kv_indptr + lo), np = __ldg(kv_indptr + lo + 1) - p0;
    const int last_len = np > 0 ? __ldg(last_page_len + lo) : 0;
    const int64_t kv_len = np > 0 ? (int64_t)(np - 1) * P + last_len : 0;
    int64_t at = -1;
    int slot = 0;
    if (row < a0 || row >= a1 || a1 - a0 > kv_len || (np > 0 && (last_len < 1 || last_len > P))) {
      set_device_error(err, kDevErrShape);
    } else {
      const int64_t pos = kv_len - (a1 - a0) + (row - a0);
      const int64_t page = __ldg(page_indices + p0 + pos / P);
      slot = (int)(pos % P);
      if (page < 0 || page >= num_pages) set_device_error(err, kDevErrPageRange);
      else at = page * Hkv;
    }
    s_page[t] = at;
    s_slot[t] = slot;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kAppendU; ++u) {
    const int64_t i = first + u * kThreads + threadIdx.x;
    if (i >= last) continue;
    const unsigned rel = (unsigned)(in_row0 + u * kThreads + threadIdx.x);
    const unsigned row = rel / (unsigned)per_row, hb = rel - row * (unsigned)per_row;
    const int h = (int)(hb / NB), blk = (int)(hb % NB);
    const int64_t page = s_page[row];
    if (page < 0) continue;
    const int slot = s_slot[row];
    const float me = kv_exp ? q4_pow2(-__ldg(kv_exp + kv * Hkv + h)) : 1.f;
    uint8_t sc;
    const uint2 codes = quantise_block(a[u], b[u], me, sc);
    uint8_t* slice = pool + ((page + h) * 2 + kv) * (int64_t)SLICE;
    *reinterpret_cast<uint2*>(slice + slot * (D / 2) + blk * 8) = codes;
    slice[P * (D / 2) + (kv == 0 ? slot * NB + blk : blk * P + slot)] = sc;
  }
}

// Pages -> bf16: a thread takes one (token, block of 16 dims) of a slice, kDeqU
// slices at a time.  Scratch page i comes from pool page ids[src ? src[i] : i].
constexpr int kDeqU = 4;

template <int D>
__global__ void __launch_bounds__(kQ4Page * (D / kQ4Block))
kv_dequant_q4_kernel(const uint8_t* __restrict__ pool, const int32_t* __restrict__ kv_exp,
                     const int32_t* __restrict__ ids, const int32_t* __restrict__ src,
                     int64_t n_slices, int Hkv, int64_t num_pages, uint16_t* __restrict__ out,
                     int* err) {
  constexpr int P = kQ4Page, NB = D / kQ4Block, SLICE = q4_slice_bytes(D);
  grid_dep_launch();
  grid_dep_wait();
  const int tok = threadIdx.x / NB, blk = threadIdx.x % NB;
  const int64_t s0 = (int64_t)blockIdx.x * kDeqU;
  uint2 codes[kDeqU];
  uint8_t sc[kDeqU];
  float two_e[kDeqU];
#pragma unroll
  for (int u = 0; u < kDeqU; ++u) {
    const int64_t s = s0 + u;
    codes[u] = make_uint2(0u, 0u);
    sc[u] = 0;
    two_e[u] = 1.f;
    if (s < n_slices) {
      const int64_t i = s / (2 * Hkv);
      const int rem = (int)(s - i * (2 * Hkv));
      const int kv = rem / Hkv, h = rem - kv * Hkv;
      const int64_t page = __ldg(ids + (src ? (int64_t)__ldg(src + i) : i));
      if (page < 0 || page >= num_pages) {
        if (threadIdx.x == 0) set_device_error(err, kDevErrPageRange);  // the page reads as zeros
      } else {
        const uint8_t* slice = pool + ((page * Hkv + h) * 2 + kv) * SLICE;
        codes[u] = __ldg(reinterpret_cast<const uint2*>(slice + tok * (D / 2) + blk * 8));
        sc[u] = __ldg(slice + P * (D / 2) + (kv == 0 ? tok * NB + blk : blk * P + tok));
        if (kv_exp) two_e[u] = q4_pow2(__ldg(kv_exp + kv * Hkv + h));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kDeqU; ++u) {
    const int64_t s = s0 + u;
    if (s >= n_slices) break;
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)(sc[u] * 0x0101u));
    uint4 o[2];
    uint32_t* ow = reinterpret_cast<uint32_t*>(o);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t h[4];
      e2m1x8_to_f16x2(half == 0 ? codes[u].x : codes[u].y, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = f16x2_to_f32x2(mul_f16x2(h[j], s2));
        ow[4 * half + j] = pack_bf16x2(f.x * two_e[u], f.y * two_e[u]);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (s * P + tok) * D + blk * kQ4Block);
    dst[0] = o[0];
    dst[1] = o[1];
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
                       page_indices, kv_indptr, last_page_len, batch, nnz_new, Hkv, num_pages, err);
}

cudaError_t launch_kv_dequant_q4(const void* pool, const int32_t* kv_exp, const int32_t* ids,
                                 const int32_t* src, int64_t n_pages, int Hkv, int head_dim,
                                 int64_t num_pages, void* out, int* err, bool programmatic,
                                 cudaStream_t stream) {
  if (n_pages <= 0) return cudaSuccess;
  const int64_t n_slices = n_pages * 2 * Hkv;
  const int64_t grid = (n_slices + kDeqU - 1) / kDeqU;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = head_dim == 128 ? kv_dequant_q4_kernel<128> : kv_dequant_q4_kernel<64>;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kQ4Page * (head_dim / kQ4Block)), 0, stream,
                       programmatic, (const uint8_t*)pool, kv_exp, ids, src, n_slices, Hkv, num_pages,
                       (uint16_t*)out, err);
}

}  // namespace daa
