// Attention over the 4-bit cache for requests with few query rows (decode and
// verify steps): split-KV, read straight from the 4-bit pages.
//
// "Disaggregated prefill and decode" (Perplexity), "Prefill vs decode
// performance": decode attention is bound by the K/V bytes, and splits over
// requests and over kv_len; "Chunked prefill" (k4i.top), #correctness: the parts
// are joined by softmax_merge.
//
// Mathematics.  For the rows n (new token, query head) of one kv head and one
// page of 16 keys, with K, V the values of the 4-bit codes (q4.cuh):
//   S^T = K Q^T           [16 keys x rows]     mma.sync m16n8k16, fp16 in, fp32 out
//   P   = 2^(S * f - m)   f: scales of a row, m: its running maximum less 7
//   O^T += V^T P^T        [d x rows]
// Taking the keys (and dims) as the 16-row side of the products lets 8 query rows
// fill one instruction, and the codes turn into A operands in registers: e2m1 *
// e4m3 is exact in fp16, so a thread converts two codes at a time (one cvt),
// multiplies by the scale (one fp16x2 product) and has two elements of its
// fragment.  Nothing is written back to shared memory.  The contraction order is
// free, so each thread takes dims that lie side by side in a row: 16 (d = 128) or
// 8 bytes of a K row in one load, and of V rows the 16 (8) dims of one block,
// whose codes for two keys are interleaved by nibble so that one cvt gives the
// two keys' values of a dim (the pair an A register holds).
//
// Roundings: q is scaled by the power of two that brings its row's largest value
// to [1, 2) and held in fp16: bf16's 8 bits fit, and what is 2^-14 below the
// row's largest loses at most 2^-25 of it.  P is rounded to fp16 (11 bits) after
// a shift by 2^7, so that weights down to 2^-31 of the largest are kept (a sum of
// a million far smaller ones would stay under 2^-11); with the lazy maximum (it
// is raised only when a score passes it by 8) P is at most 2^15.  Sums, maxima
// and O are fp32.
//
// Bound: HBM.  A (page, head) is 18 d bytes; at the measured 6.7 TB/s an SM gets
// one of d = 128 every 52 ns (99 clocks), in which it can issue about 400 warp
// instructions; this loop takes about 200.  Warps work alone: each streams its
// own pages (every fourth of the unit) through its own ring with one bulk copy a
// page (K and V of a head are side by side), so nothing but the end of the unit
// synchronises the CTA.
#include <climits>

#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace daa {
namespace {

constexpr int kP = kQ4Page;
constexpr int kWarps = 4;
constexpr float kBias = 7.f;     // P = 2^(s - m + kBias)
constexpr float kRaise = 8.f;    // the maximum is raised when a score passes it by this

template <int D, int NT>
struct Shape {
  static constexpr int SLICE = q4_slice_bytes(D);
  static constexpr int STAGE = 2 * SLICE;              // K and V of one (page, head)
  static constexpr int NSTAGE = D == 128 ? 5 : 8;
  static constexpr int ROWS = 8 * NT;
  static constexpr int TILES = D / 16;                 // 16-dim tiles of O^T
  static constexpr int KSTEPS = D / 16;
  static constexpr int RING = kWarps * NSTAGE * STAGE;
  static constexpr int MERGE = kWarps * ROWS * (D + 2) * 4;
  static constexpr int BODY = RING > MERGE ? RING : MERGE;
  static constexpr int OFF_BAR = BODY;
  static constexpr int SMEM = OFF_BAR + kWarps * NSTAGE * 8;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 tile of 16-bit elements held as rows over a warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t nibbles(uint32_t lo, uint32_t hi) {  // (lo & 0x0F..) | (hi & 0xF0..)
  return (lo & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u);
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
attention_q4_kernel(const AttentionQ4Args a) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR) + warp * S::NSTAGE;
  uint8_t* ring = smem + warp * (S::NSTAGE * S::STAGE);

  // the heads of a unit side by side: their slices of a page are, too
  const Q4Unit u = a.units[blockIdx.x / a.Hkv];
  const int kvh = blockIdx.x % a.Hkv;
  const int g = a.group;
  const int rows = u.n_tok * g;
  const int key_end = a.causal ? min(u.tok_end, u.pos0 + u.n_tok) : u.tok_end;
  const int pg0 = u.tok_begin / kP + warp;
  const int pg_end = (key_end + kP - 1) / kP;
  const int my_n = pg_end > pg0 ? (pg_end - pg0 + kWarps - 1) / kWarps : 0;

  if (threadIdx.x == 0) grid_dep_launch();  // the merge may launch; it waits for this grid
  if (lane == 0) {
    for (int i = 0; i < S::NSTAGE; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();

  // page ids, 32 of this warp's pages at a time (lane l: page base + l)
  int32_t ids = 0;
  auto load_ids = [&](int k0) {
    const int k = k0 + lane;
    ids = k < my_n ? __ldg(a.page_indices + u.page_base + pg0 + k * kWarps) : 0;
    if (ids < 0 || ids >= a.num_pages) {
      set_device_error(a.err, kDevErrPageRange);
      ids = 0;  // a valid page instead; the output is undefined anyway
    }
  };
  auto issue = [&](int k) {  // whole warp, k < my_n
    const int64_t page = __shfl_sync(0xffffffffu, ids, k & 31);
    if (lane == 0) {
      const int st = k % S::NSTAGE;
      mbar_arrive_expect_tx(&full[st], S::STAGE);
      bulk_g2s(ring + st * S::STAGE, a.pool + (page * a.Hkv + kvh) * S::STAGE, S::STAGE, &full[st]);
    }
    if ((k & 31) == 31) load_ids(k + 1);
  };
  load_ids(0);
  for (int k = 0; k < S::NSTAGE && k < my_n; ++k) issue(k);

  // Q^T fragments: rows n = 8 t + r, this thread's dims [c * D/4, (c + 1) * D/4)
  const float f_k = a.sm_scale_log2 * (a.kv_exp ? q4_pow2(__ldg(a.kv_exp + kvh)) : 1.f);
  uint32_t qf[NT][S::KSTEPS][2];
  float fs[NT][2];       // score factor of rows 8 t + 2 c, + 1
  int lim[NT][2];        // keys of those rows: [0, lim)
  int lim_min = INT_MAX;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = 8 * t + r;
    float x[D / 4];
    float mx = 0.f;
    if (n < rows) {
      const int tok = n / g;
      const uint16_t* src = a.q + ((int64_t)(u.q_row + tok) * a.Hq + kvh * g + (n - tok * g)) * D + c * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + i);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * i + 2 * j] = bf16lo_to_f32(ww[j]);
          x[8 * i + 2 * j + 1] = bf16hi_to_f32(ww[j]);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(x[i]));
    } else {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int ex = mx > 0.f ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -126), 126) : 0;
    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int j = 0; j < S::KSTEPS; ++j) {
      qf[t][j][0] = pack_f16x2(x[4 * j] * down, x[4 * j + 1] * down);
      qf[t][j][1] = pack_f16x2(x[4 * j + 2] * down, x[4 * j + 3] * down);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int m = 8 * t + 2 * c + b;
      const int e = __shfl_sync(0xffffffffu, ex, 4 * (2 * c + b));  // row m's, held by lanes 4 (m % 8) ..
      fs[t][b] = f_k * __uint_as_float((uint32_t)(127 + e) << 23);
      lim[t][b] = a.causal && m < rows ? min(u.pos0 + m / g + 1, u.kv_len) : u.kv_len;
      lim_min = min(lim_min, lim[t][b]);
    }
  }
  // every lane agrees on whether a page needs masks
  lim_min = __reduce_min_sync(0xffffffffu, lim_min);

  float o[NT][S::TILES][4];
  float m_run[NT][2], l_run[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m_run[t][0] = m_run[t][1] = -INFINITY;
    l_run[t][0] = l_run[t][1] = 0.f;
#pragma unroll
    for (int i = 0; i < S::TILES; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
  }
  // the two keys of a pair are swapped in odd threads of a quad (see the V loads)
  const uint32_t pair_sel = (c & 1) ? 0x1032u : 0x3210u;

  constexpr int PPI = 2;  // pages per pass of the loop
  for (int k = 0; k < my_n; k += PPI) {
    // ---- S^T of two pages
    float s[PPI][NT][4];
#pragma unroll
    for (int p = 0; p < PPI; ++p) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[p][t][e] = 0.f;
      if (k + p >= my_n) continue;
      const int st = (k + p) % S::NSTAGE;
      mbar_wait(&full[st], ((k + p) / S::NSTAGE) & 1, a.err);
      const uint8_t* kb = ring + st * S::STAGE;
      constexpr int W = D / 32;  // code words of a thread per key row
      uint32_t w0[W], w1[W];
      uint32_t sc0[2], sc1[2];   // block scales of the thread's dims, keys r and r + 8
      if constexpr (D == 128) {
        const uint4 x0 = *reinterpret_cast<const uint4*>(kb + r * 64 + c * 16);
        const uint4 x1 = *reinterpret_cast<const uint4*>(kb + (r + 8) * 64 + c * 16);
        w0[0] = x0.x; w0[1] = x0.y; w0[2] = x0.z; w0[3] = x0.w;
        w1[0] = x1.x; w1[1] = x1.y; w1[2] = x1.z; w1[3] = x1.w;
        const uint32_t y0 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kb + 1024 + r * 8 + 2 * c));
        const uint32_t y1 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kb + 1024 + (r + 8) * 8 + 2 * c));
        sc0[0] = __byte_perm(y0, y0, 0x1010); sc0[1] = __byte_perm(y0, y0, 0x3232);
        sc1[0] = __byte_perm(y1, y1, 0x1010); sc1[1] = __byte_perm(y1, y1, 0x3232);
      } else {
        const uint2 x0 = *reinterpret_cast<const uint2*>(kb + r * 32 + c * 8);
        const uint2 x1 = *reinterpret_cast<const uint2*>(kb + (r + 8) * 32 + c * 8);
        w0[0] = x0.x; w0[1] = x0.y;
        w1[0] = x1.x; w1[1] = x1.y;
        // one block a thread: keys r and r + 8 in one conversion
        const uint32_t y = e4m3x2_to_f16x2((uint16_t)(kb[512 + r * 4 + c] | (kb[512 + (r + 8) * 4 + c] << 8)));
        sc0[0] = sc0[1] = __byte_perm(y, y, 0x1010);
        sc1[0] = sc1[1] = __byte_perm(y, y, 0x3232);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t h0[4], h1[4];
        e2m1x8_to_f16x2(w0[w], h0);
        e2m1x8_to_f16x2(w1[w], h1);
        const uint32_t z0 = sc0[(2 * w) / W], z1 = sc1[(2 * w) / W];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h0[i] = mul_f16x2(h0[i], z0);
          h1[i] = mul_f16x2(h1[i], z1);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma_f16(s[p][t], h0[0], h1[0], h0[1], h1[1], qf[t][2 * w][0], qf[t][2 * w][1]);
          mma_f16(s[p][t], h0[2], h1[2], h0[3], h1[3], qf[t][2 * w + 1][0], qf[t][2 * w + 1][1]);
        }
      }
    }

    // ---- scores in the log2 domain, hidden keys at -inf
    bool raise = false;
#pragma unroll
    for (int p = 0; p < PPI; ++p) {
      const int key = (pg0 + (k + p) * kWarps) * kP + r;  // of s[..][0], [1]; + 8 of [2], [3]
      const bool masked = k + p >= my_n || key - r + kP > lim_min;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[p][t][e] * fs[t][e & 1];
          if (masked && (k + p >= my_n || key + (e >= 2 ? 8 : 0) >= lim[t][e & 1])) x = -INFINITY;
          s[p][t][e] = x;
          raise |= x > m_run[t][e & 1] + kRaise;
        }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float mx = m_run[t][b];
#pragma unroll
          for (int p = 0; p < PPI; ++p) mx = fmax3(mx, s[p][t][b], s[p][t][b + 2]);
#pragma unroll
          for (int m = 4; m <= 16; m <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
          const float alpha = mx == -INFINITY ? 1.f : ex2_approx(m_run[t][b] - mx);
          m_run[t][b] = mx;
          l_run[t][b] *= alpha;
#pragma unroll
          for (int i = 0; i < S::TILES; ++i) {
            o[t][i][b] *= alpha;
            o[t][i][b + 2] *= alpha;
          }
        }
    }

    // ---- P (fp16), transposed into the B operand of O^T += V^T P^T
    uint32_t pb[PPI][NT][2];
#pragma unroll
    for (int p = 0; p < PPI; ++p)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = m_run[t][i & 1];
          // a row with no visible key yet keeps m = -inf: its scores are -inf too
          e[i] = ex2_approx(s[p][t][i] - (m == -INFINITY ? 0.f : m - kBias));
        }
        l_run[t][0] += e[0] + e[2];
        l_run[t][1] += e[1] + e[3];
        pb[p][t][0] = __byte_perm(transpose8(pack_f16x2(e[0], e[1])), 0u, pair_sel);
        pb[p][t][1] = __byte_perm(transpose8(pack_f16x2(e[2], e[3])), 0u, pair_sel);
      }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int p = 0; p < PPI; ++p) {
      if (k + p >= my_n) continue;
      const int st = (k + p) % S::NSTAGE;
      const uint8_t* vb = ring + st * S::STAGE + S::SLICE;
      constexpr int W = D / 64;        // code words of a thread per key
      constexpr int BPR = D / 16;      // bytes of a thread per key
      // Keys 2c, 2c + 1 (pair 0) and 2c + 8, 2c + 9 (pair 1) of the page.  Key rows
      // of one parity share their banks (d = 128), so odd threads of a quad read
      // the pair's second key first; P and the scales are swapped to match.
      uint32_t w[2][2][W];
#pragma unroll
      for (int pr = 0; pr < 2; ++pr)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* row = vb + (8 * pr + 2 * c + (h ^ (c & 1))) * (D / 2) + r * BPR;
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(row);
            w[pr][h][0] = x.x;
            w[pr][h][W - 1] = x.y;
          } else {
            w[pr][h][0] = *reinterpret_cast<const uint32_t*>(row);
          }
        }
      const int blk = D == 128 ? r : r >> 1;
      uint32_t sc[2];
      const int key0 = (pg0 + (k + p) * kWarps) * kP;
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        sc[pr] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vb + 8 * D + blk * kP + 8 * pr + 2 * c));
        // slots past the last key may hold anything: their scales count as zero
        const int over = key0 + 8 * pr + 2 * c - u.kv_len;  // >= 0: both keys, -1: the second
        if (over >= -1) sc[pr] = over >= 0 ? 0u : sc[pr] & 0xFFFFu;
        sc[pr] = __byte_perm(sc[pr], 0u, pair_sel);
      }
#pragma unroll
      for (int x = 0; x < W; ++x) {
        uint32_t lo[2][4], hi[2][4];  // dims 2i, 2i + 1 of tile 4 x + j, for the two pairs
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          e2m1x8_to_f16x2(nibbles(w[pr][0][x], w[pr][1][x] << 4), lo[pr]);
          e2m1x8_to_f16x2(nibbles(w[pr][0][x] >> 4, w[pr][1][x]), hi[pr]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo[pr][j] = mul_f16x2(lo[pr][j], sc[pr]);
            hi[pr][j] = mul_f16x2(hi[pr][j], sc[pr]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_f16(o[t][4 * x + j], lo[0][j], hi[0][j], lo[1][j], hi[1][j], pb[p][t][0], pb[p][t][1]);
      }
    }
    __syncwarp();  // both pages have been read
#pragma unroll
    for (int p = 0; p < PPI; ++p)
      if (k + p + S::NSTAGE < my_n) issue(k + p + S::NSTAGE);
  }

  // ---- join the four warps in shared memory (the rings are free), then write
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int m = 4; m <= 16; m <<= 1) l_run[t][b] += __shfl_xor_sync(0xffffffffu, l_run[t][b], m);
  __syncthreads();
  float* mo = reinterpret_cast<float*>(smem);        // [warp][row][D]
  float* mm = mo + kWarps * S::ROWS * D;             // [warp][row]
  float* ml = mm + kWarps * S::ROWS;                 // [warp][row]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int n = 8 * t + 2 * c + b;
      if (n >= rows) continue;
      float* dst = mo + (warp * S::ROWS + n) * D + r * (D / 8);
#pragma unroll
      for (int i = 0; i < S::TILES; i += 2)
        *reinterpret_cast<float4*>(dst + 2 * i) =
            make_float4(o[t][i][b], o[t][i][b + 2], o[t][i + 1][b], o[t][i + 1][b + 2]);
      if (r == 0) {
        mm[warp * S::ROWS + n] = m_run[t][b];
        ml[warp * S::ROWS + n] = l_run[t][b];
      }
    }
  __syncthreads();
  const float f_v = a.kv_exp ? q4_pow2(__ldg(a.kv_exp + a.Hkv + kvh)) : 1.f;
  for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kWarps) {
    const int n = i / (D / 4), d0 = (i - n * (D / 4)) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mm[w * S::ROWS + n]);
    float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float m = mm[w * S::ROWS + n];
      const float wt = m == -INFINITY ? 0.f : ex2_approx(m - M);
      const float4 v = *reinterpret_cast<const float4*>(mo + (w * S::ROWS + n) * D + d0);
      L += wt * ml[w * S::ROWS + n];
      acc[0] += wt * v.x;
      acc[1] += wt * v.y;
      acc[2] += wt * v.z;
      acc[3] += wt * v.w;
    }
    const float inv = L > 0.f ? f_v / L : 0.f;  // no visible key: zero, lse -inf
    const float lse2 = M - kBias + __log2f(L);
    const int tok = n / g;
    const int hq = kvh * g + (n - tok * g);
    if (u.part < 0) {
      const int64_t row = (int64_t)(u.q_row + tok) * a.Hq + hq;
      uint2 pk;
      pk.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
      pk.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
      *reinterpret_cast<uint2*>(a.out + row * D + d0) = pk;
      if (d0 == 0 && a.lse_out) a.lse_out[row] = lse2 * 0.69314718055994531f;
    } else {
      const int64_t row = ((int64_t)u.part + (int64_t)tok * u.part_stride) * a.Hq + hq;
      *reinterpret_cast<float4*>(a.part_o + row * D + d0) =
          make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      if (d0 == 0) a.part_lse[row] = lse2;
    }
  }
}

template <int D, int NT>
cudaError_t launch_t(const AttentionQ4Args& a, int n_units, cudaStream_t stream) {
  using S = Shape<D, NT>;
  auto kern = attention_q4_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  if ((int64_t)a.Hkv * n_units > INT32_MAX) return cudaErrorInvalidValue;
  kern<<<a.Hkv * n_units, 32 * kWarps, S::SMEM, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(AttentionQ4Args a, const int (&n_units)[kQ4Classes], cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < kQ4Classes && e == cudaSuccess; ++i) {
    if (n_units[i] == 0) continue;
    e = i == 0 ? launch_t<D, 1>(a, n_units[i], stream)
               : (i == 1 ? launch_t<D, 2>(a, n_units[i], stream) : launch_t<D, 4>(a, n_units[i], stream));
    a.units += n_units[i];
  }
  return e;
}

}  // namespace

cudaError_t launch_attention_q4(const AttentionQ4Args& a, const int (&n_units)[kQ4Classes],
                                cudaStream_t stream) {
  return a.head_dim == 128 ? launch_d<128>(a, n_units, stream) : launch_d<64>(a, n_units, stream);
}

}  // namespace daa
