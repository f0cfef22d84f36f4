// Rotary positions, alone and on the way into a paged cache.
//
// "Chunked prefill" (k4i.top), #correctness: a chunk's new k, v vectors join the
// cache at their absolute positions, and its queries attend from theirs.  What the
// projections give is not rotated yet: of a token at position p, pair i of a head's
// first rotary_dim dims, (a, b), becomes
//   m (a cos t - b sin t, b cos t + a sin t),   t = p f_i,
// after an optional division of the head by its root mean square over the head_dim
// dims and a product with weights.  Everything is fp32 from the loaded bf16 values
// to one rounding at the end.  (Between the norm and the rotation nothing is
// rounded; a model that keeps bf16 there differs by that rounding, 2^-9.)
//
// Angles.  p f_i grows to 10^5 and more, where fp32 has no digits of the angle left.
// A pair's turns a token are held as a 64-bit fraction of a turn: p times it, modulo
// 2^64, is the angle modulo one turn, exact but for p 2^-65 turns; its upper 32 bits
// (2^-32 turns, 1.5e-9 rad) go through sincospif.  No table of positions is needed,
// nothing is read for it, and no position is too far or negative.
//
// Layout.  A head is D / 16 threads of two 16-byte chunks each: chunks j and
// j + rotary_dim / 16 for the half layout, so that a thread holds whole pairs, and a
// warp's loads and stores are 64 to 128 contiguous bytes a head.  CTAs take equal
// ranges of the flat (row, head) space, q then k then v heads of a row; each range's
// sines (one pair of values a thread and row) are computed once into shared memory
// and read by all heads of the row.
#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace daa {
namespace {

constexpr int kThreads = 256;
constexpr int kP = 16;
constexpr int kMaxBatch = 1023;            // requests whose lengths a CTA holds
constexpr int kMaxAngleBytes = 24 * 1024;  // sines and cosines of a CTA's rows
constexpr int kSmallU = 1, kLargeU = 4;    // heads of a thread in flight

// Where a row's k and v go: page * 16 + slot, or:
constexpr int64_t kNoPage = -1;  // a bad page id: its q is rotated all the same
constexpr int64_t kNoRow = -2;   // a row of no request: nothing of it is written

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void st_16(void* p, const uint32_t* w) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x;
  f[1] = v.y;
  f[2] = v.z;
  f[3] = v.w;
}

// (a, b) -> (a c - b s, b c + a s), each a product and a fused product.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
  b = __fmaf_rn(b, c, __fmul_rn(a, s));
  a = x;
}

// The page, slot and position of new row `row`.
__device__ __forceinline__ int64_t find_place(const RopeArgs& a, const int32_t* indptr, const int32_t* kv_begin,
                                              const int32_t* last_lens, int row, int& pos) {
  pos = 0;
  if (row >= indptr[a.batch]) return kNoRow;  // padding behind the last request
  int lo = 0, hi = a.batch - 1;  // largest r with indptr[r] <= row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (indptr[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int a0 = indptr[lo], a1 = indptr[lo + 1];
  const int p0 = kv_begin[lo], np = kv_begin[lo + 1] - p0;
  const int last_len = np > 0 ? last_lens[lo] : 0;
  const int64_t kv_len = np > 0 ? (int64_t)(np - 1) * kP + last_len : 0;
  if (row < a0 || row >= a1 || a1 - a0 > kv_len || kv_len > INT32_MAX || p0 < 0 || last_len < 1 || last_len > kP) {
    set_device_error(a.err, kDevErrShape);
    return kNoRow;
  }
  pos = (int)kv_len - (a1 - a0) + (row - a0);
  const int64_t page = ld_word(a.page_indices + p0 + pos / kP);
  if (page < 0 || page >= a.num_pages) {
    set_device_error(a.err, kDevErrPageRange);
    return kNoPage;
  }
  return page * kP + pos % kP;
}

template <int D, int TARGET, bool NORM, int U>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int L = D / 16, G = kThreads / L;  // threads of a head, heads of a CTA at a time
  constexpr bool APPEND = TARGET != kRopeRows, Q4 = TARGET == kRopePagesQ4;
  extern __shared__ __align__(16) uint8_t smem[];
  const int hp = a.rotary_dim / 2;
  float* s_cos = reinterpret_cast<float*>(smem);
  float* s_sin = s_cos + a.max_rows * hp;
  float* s_w = s_sin + a.max_rows * hp;  // weights of q, of k
  int64_t* s_at = reinterpret_cast<int64_t*>(s_w + (NORM ? 2 * D : 0));
  int* s_pos = reinterpret_cast<int*>(s_at + a.max_rows);
  int* s_table = s_pos + a.max_rows;

  const int tid = threadIdx.x, group = tid / L, j = tid % L;
  const uint32_t mask = ((L == 8 ? 0xFFu : 0xFu)) << (tid & 31 & ~(L - 1));  // the head's lanes
  const int H = a.Hq + (APPEND ? 2 : 1) * a.Hk;
  const int first = blockIdx.x * a.per_cta;
  const int count = min(a.per_cta, a.n_rows * H - first);
  const int row0 = first / H, in0 = first - row0 * H;
  const int nrows = (in0 + count - 1) / H + 1;
  // chunks of 8 dims of this thread; in a 4-bit cache's rows two side by side, a block
  const int nrot = a.rotary_dim / 16;
  const bool pairs = a.interleaved != 0;
  const int c0 = pairs ? j : j < nrot ? j : 2 * j;
  const int c1 = pairs ? j + L : j < nrot ? j + nrot : 2 * j + 1;
  const int pair = tid % hp, angle_rows = kThreads / hp;  // this thread's share of the sines
  const uint64_t turns = a.turns[pair];
  const int row_a = (in0 + group) / H, head_a = in0 + group - row_a * H;
  grid_dep_launch();
  grid_dep_wait();

  // the values depend on nothing else: load them first
  uint32_t w[U][8];
  {
    int row = row_a, head = head_a;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * G + group < count) {
        const bool is_q = head < a.Hq, is_k = !is_q && head < a.Hq + a.Hk;
        const RopeRows& x = is_q ? a.q : !APPEND || is_k ? a.k : a.v;
        const int h = is_q ? head : head - a.Hq - (!APPEND || is_k ? 0 : a.Hk);
        const bool side = Q4 && !is_q && (pairs || !is_k);
        const uint16_t* p = x.p + (row0 + row) * x.row + h * x.head;
        const uint4 lo = ld_stream(p + 8 * (side ? 2 * j : c0)), hi = ld_stream(p + 8 * (side ? 2 * j + 1 : c1));
        w[u][0] = lo.x, w[u][1] = lo.y, w[u][2] = lo.z, w[u][3] = lo.w;
        w[u][4] = hi.x, w[u][5] = hi.y, w[u][6] = hi.z, w[u][7] = hi.w;
      }
      row += a.step_rows;
      head += a.step_heads;
      if (head >= H) {
        head -= H;
        ++row;
      }
    }
  }
  if (NORM) {
    for (int t = tid; t < 2 * D; t += kThreads) {
      const uint16_t* n = t < D ? a.q_norm : a.k_norm;
      uint16_t b = 0;
      if (n) asm volatile("ld.global.u16 %0, [%1];" : "=h"(b) : "l"(n + t % D));
      s_w[t] = __uint_as_float((uint32_t)b << 16);
    }
  }
  if (APPEND) {
    const int32_t *indptr = a.append_indptr, *kv_begin = a.kv_indptr, *last_lens = a.last_page_len;
    if (a.batch <= kMaxBatch) {
      int* s_kv = s_table + a.batch + 1;
      int* s_last = s_kv + a.batch + 1;
      for (int t = tid; t <= a.batch; t += kThreads) {
        s_table[t] = ld_word(indptr + t);
        s_kv[t] = ld_word(kv_begin + t);
        if (t < a.batch) s_last[t] = ld_word(last_lens + t);
      }
      __syncthreads();
      indptr = s_table;
      kv_begin = s_kv;
      last_lens = s_last;
    }
    for (int t = tid; t < nrows; t += kThreads) {
      int pos;
      s_at[t] = find_place(a, indptr, kv_begin, last_lens, row0 + t, pos);
      s_pos[t] = a.positions ? ld_word(a.positions + row0 + t) : pos;
    }
  } else {
    for (int t = tid; t < nrows; t += kThreads) s_pos[t] = ld_word(a.positions + row0 + t);
  }
  __syncthreads();
  if (tid < angle_rows * hp) {
    for (int r = tid / hp; r < nrows; r += angle_rows) {
      const uint64_t phase = turns * (uint64_t)(int64_t)s_pos[r];
      float s, c;
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
      s_cos[r * hp + pair] = c * a.magnitude;
      s_sin[r * hp + pair] = s * a.magnitude;
    }
  }
  __syncthreads();

  int row = row_a, head = head_a;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = row, hd = head;
    row += a.step_rows;
    head += a.step_heads;
    if (head >= H) {
      head -= H;
      ++row;
    }
    if (u * G + group >= count) continue;
    const int64_t at = APPEND ? s_at[r] : 0;
    if (at == kNoRow) continue;
    const bool is_q = hd < a.Hq, is_k = !is_q && (!APPEND || hd < a.Hq + a.Hk);
    const int h = is_q ? hd : hd - a.Hq - (is_k ? 0 : a.Hk);
    const bool side = Q4 && !is_q && (pairs || !is_k);
    const int d0 = side ? 2 * j : c0, d1 = side ? 2 * j + 1 : c1;
    uint32_t(&v)[8] = w[u];
    if (is_q || is_k) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16lo_to_f32(v[i]);
        x[2 * i + 1] = bf16hi_to_f32(v[i]);
      }
      bool t0 = pairs ? d0 < 2 * nrot : j < nrot, t1 = pairs ? d1 < 2 * nrot : j < nrot;
      float c[8], s[8];
      const float *cr = s_cos + r * hp, *sr = s_sin + r * hp;
      const int i0 = pairs ? 4 * d0 : 8 * j, i1 = pairs ? 4 * d1 : 8 * j + 4;
      if (t0) {
        load4(cr + i0, c);
        load4(sr + i0, s);
      }
      if (t1) {
        load4(cr + i1, c + 4);
        load4(sr + i1, s + 4);
      }
      const bool norm = NORM && (is_q ? a.q_norm : a.k_norm) != nullptr;
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = L / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(mask, ss, m);
        const float k = rsqrtf(ss * (1.f / D) + a.eps);
        const float* wt = s_w + (is_q ? 0 : D);
        float g[16];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          load4(wt + 8 * d0 + i, g + i);
          load4(wt + 8 * d1 + i, g + 8 + i);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * k * g[i];
      }
      if (!pairs) {
        if (t0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) turn(x[i], x[8 + i], c[i], s[i]);
        }
      } else {
        if (t0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
        }
        if (t1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) turn(x[8 + 2 * i], x[9 + 2 * i], c[4 + i], s[4 + i]);
        }
      }
      // dims that are neither normalised nor rotated keep their bits
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (norm || t0) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        if (norm || t1) v[4 + i] = pack_bf16x2(x[8 + 2 * i], x[9 + 2 * i]);
      }
    }
    if (is_q || !APPEND) {
      const RopeRows& y = is_q ? a.q_out : a.k_out;
      uint16_t* p = y.p + (row0 + r) * y.row + h * y.head;
      st_16(p + 8 * d0, v);
      st_16(p + 8 * d1, v + 4);
      continue;
    }
    if (at == kNoPage) continue;
    const int64_t page = at / kP;
    const int slot = (int)(at % kP), kv = is_k ? 0 : 1;
    if (!Q4) {
      uint16_t* p = reinterpret_cast<uint16_t*>(a.pool) + (((page * 2 + kv) * a.Hk + h) * kP + slot) * D;
      st_16(p + 8 * d0, v);
      st_16(p + 8 * d1, v + 4);
    } else {
      uint4 b[2] = {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])};
      if (!side) {
        // chunks 2j and 2j + 1 of the head, from the threads that have them
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 2 * j + i;
          const int from = t < nrot ? t : t < 2 * nrot ? t - nrot : t / 2;
          const bool upper = t < 2 * nrot ? t >= nrot : (t & 1) != 0;
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = __shfl_sync(mask, v[k], from, L), hi = __shfl_sync(mask, v[4 + k], from, L);
            o[k] = upper ? hi : lo;
          }
          b[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      const float me = a.kv_exp ? q4_pow2(-ld_word(a.kv_exp + kv * a.Hk + h)) : 1.f;
      uint8_t scale;
      const uint2 codes = quantise_block(b[0], b[1], me, scale);
      uint8_t* slice = a.pool + ((page * a.Hk + h) * 2 + kv) * (int64_t)q4_slice_bytes(D);
      *reinterpret_cast<uint2*>(slice + slot * (D / 2) + j * 8) = codes;
      slice[kP * (D / 2) + (kv == 0 ? slot * L + j : j * kP + slot)] = scale;
    }
  }
}

template <int D, int TARGET>
cudaError_t launch(RopeArgs a, int sms, bool programmatic, cudaStream_t stream) {
  constexpr int G = kThreads / (D / 16);
  const int H = a.Hq + (TARGET != kRopeRows ? 2 : 1) * a.Hk;
  const int64_t total = (int64_t)a.n_rows * H;
  const bool large = total >= (int64_t)sms * 16 * G;
  const int hp = a.rotary_dim / 2;
  auto rows_of = [&](int items) { return (items + H - 2) / H + 1; };
  a.per_cta = G * (large ? kLargeU : kSmallU);
  const int most = kMaxAngleBytes / (8 * hp);
  if (rows_of(a.per_cta) > most) a.per_cta = (most - 1) * H;
  a.max_rows = rows_of(a.per_cta);
  a.step_rows = G / H;
  a.step_heads = G % H;
  const bool norm = a.q_norm || a.k_norm;
  const size_t smem = (size_t)a.max_rows * (hp * 8 + 12) + (norm ? 2 * D * 4 : 0) +
                      (TARGET != kRopeRows && a.batch <= kMaxBatch ? 12 * ((size_t)a.batch + 1) : 0);
  const int64_t grid = (total + a.per_cta - 1) / a.per_cta;
  auto kern = norm ? (large ? rope_kernel<D, TARGET, true, kLargeU> : rope_kernel<D, TARGET, true, kSmallU>)
                   : (large ? rope_kernel<D, TARGET, false, kLargeU> : rope_kernel<D, TARGET, false, kSmallU>);
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), smem, stream, programmatic, a);
}

template <int TARGET>
cudaError_t launch_d(const RopeArgs& a, int head_dim, int sms, bool programmatic, cudaStream_t stream) {
  return head_dim == 128 ? launch<128, TARGET>(a, sms, programmatic, stream) : launch<64, TARGET>(a, sms, programmatic, stream);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int head_dim, RopeTarget target, int sms, bool programmatic, cudaStream_t stream) {
  return target == kRopeRows    ? launch_d<kRopeRows>(a, head_dim, sms, programmatic, stream)
         : target == kRopePages ? launch_d<kRopePages>(a, head_dim, sms, programmatic, stream)
                                : launch_d<kRopePagesQ4>(a, head_dim, sms, programmatic, stream);
}

}  // namespace daa
