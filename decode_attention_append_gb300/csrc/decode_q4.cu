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
// Bound: HBM for 8 rows; for more, the instructions at the pace that two warps a scheduler
// (221 and 255 registers) can issue them.  A (page, head) is 18 d bytes; at
// the measured 6.7 TB/s an SM gets one of d = 128 every 52 ns (about 99 clocks), in
// which it can issue 400 warp instructions.  A page takes 280 of them with 8 rows, 309
// with 16 and 389 with 24: 64 conversions and 64 products of the codes, 16 mma for
// every 8 rows, the rest loads, scales, exponents and the ring.  Measured (GB300): each
// further page of long contexts takes an SM 52 ns with 8 rows (the bytes' time), 74 with
// 16 and 92 with 24; about 3.5 us go by before the first pages are there, and 0.5 to 2
// for writing a range's last unit.  Kernels: 32 requests of 0.5k to 4k tokens, 32 heads
// on 32, 56 us (5.7 TB/s); 128 of 1k to 32k, 12 heads on 1, 44.7 us (4.0 TB/s); verify of
// 5 tokens, 32 heads on 8, 35 us (2.8 TB/s); issue slots used 64, 49 and 43 %.  The loads
// alone take 49, 34 and 26 us.
//
// Warps work alone: each streams a range of pages of its own (the units of one kv
// head, cut so that every resident warp has the same cost) through its own ring with
// one bulk copy a page (K and V of a head are side by side), over the ends of
// requests, and writes its own parts; nothing in a CTA is synchronised.  Measured and
// not faster: two warps to a range that share its pages and split the dims, so that
// 16 and 24 rows have 16 warps an SM, too (58 us for 48 and 51 for 39.5: 460
// instructions a page); 12 warps of 168 registers for 16 rows (51 for 48); the scores of a
// pair beside the products of the one before it (52 for 48); tcgen05 with the codes
// converted into TMEM and shared memory (79 for 47); a unit's rows written by way of
// shared memory (47 us for 44.9 with the merge).
#include <cfloat>
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
constexpr float kNoMax = -1e37f;  // `off` of a row that has seen no key
constexpr int kHidden = 0x40000000;  // a key position past every request

template <int D, int NT>
struct Shape {
  static constexpr int SLICE = q4_slice_bytes(D);
  static constexpr int PAGE = 2 * SLICE;               // K and V of one (page, head)
  static constexpr int CTAS = NT == 1 ? 4 : 2;         // meant to share an SM: 128 and 255 registers
  // Ring, in pairs of pages.  Deeper ones measured slower: at the start every warp's
  // further pages queue in front of other warps' first ones (24 rows, contexts of 4k:
  // 53.8 us with two, 55.4 with three; 16 rows 50.9 and 50.4).
  static constexpr int PAIRS = (NT == 2 ? 3 : 2) * (D == 128 ? 1 : 2);
  static constexpr int STAGE = 2 * PAGE;
  static constexpr int TILES = D / 16;                 // 16-dim tiles of O^T
  static constexpr int KWORDS = D / 32;                // code words of a thread per key row
  static constexpr int Q_WARP = NT * KWORDS * 32 * 16; // Q^T fragments of a warp
  static constexpr int OFF_Q = kWarps * PAIRS * STAGE;
  static constexpr int OFF_BAR = OFF_Q + kWarps * Q_WARP;
  static constexpr int SMEM = OFF_BAR + kWarps * PAIRS * 8;
  static_assert(CTAS * (SMEM + 1024) <= 233472, "shared memory of the CTAs of an SM");
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

// (lo & 0x0F0F0F0F) | (hi & 0xF0F0F0F0) in one instruction (two masks would take two)
__device__ __forceinline__ uint32_t nibbles(uint32_t lo, uint32_t hi) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, 0x0F0F0F0F, 0xE4;" : "=r"(d) : "r"(lo), "r"(hi));
  return d;
}

// sm_scale * log2(e) * 2^e for |e| <= 158, cut to fp32's normal numbers: a factor of zero (or
// infinity) would turn the -inf of a hidden key (or the score 0) into NaN.  2^e comes in two
// halves, so nothing on the way is out of range when the result is not.  Below FLT_MIN every
// weight is 1 to within 2^-100 (before it a score is under 2^20) and the cut changes nothing.
__device__ __forceinline__ float score_factor(float sm_scale, int e) {
  const int half = e / 2;
  const float f = sm_scale * __int_as_float((127 + half) << 23) * __int_as_float((127 + e - half) << 23);
  return fminf(fmaxf(f * 1.4426950408889634f, FLT_MIN), FLT_MAX);
}

// A sector at once (p on a 32-byte boundary): with 16-byte stores, half a sector each,
// the parts of 24-row units cost 1.5 us more (verify of 5 tokens 42.8 us, 41.3).
__device__ __forceinline__ void st_32(float* p, float a, float b, float c, float d, float e, float f, float g,
                                      float h) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d),
               "f"(e), "f"(f), "f"(g), "f"(h)
               : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, Shape<D, NT>::CTAS)
attention_q4_kernel(const AttentionQ4Args a) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR) + warp * S::PAIRS;
  uint8_t* ring = smem + warp * (S::PAIRS * S::STAGE);
  uint4* q_frag = reinterpret_cast<uint4*>(smem + S::OFF_Q + warp * S::Q_WARP);

  // the heads of a range in warps side by side: their slices of a page are, too
  const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
  const int range = (int)(id / a.Hkv);
  if (range >= a.n_ranges) return;
  const int kvh = (int)(id - (int64_t)range * a.Hkv);
  const int g = a.group;
  const uint32_t inv_g = 65536u / (uint32_t)g + 1;  // n / g = n * inv_g >> 16, a row's token (n < 64)
  auto token_of = [&](int n) { return (int)((uint32_t)n * inv_g >> 16); };
  const Q4Range rec = a.ranges[range];  // of the plan: copied long before the kernel ahead of this one
  if (lane == 0) {
    for (int i = 0; i < S::PAIRS; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // The next kernel may start its CTAs, but not before this one may read: the next
  // class's launch does not wait by itself.
  if (a.wait_first) grid_dep_wait();
  grid_dep_launch();
  const int e_k = a.kv_exp ? q4_exp(ld_word(a.kv_exp + kvh)) : 0;
  const float f_v = a.kv_exp ? q4_pow2(ld_word(a.kv_exp + a.Hkv + kvh)) : 1.f;
  auto pages_of = [&](const Q4Unit& u) {
    const int key_end = a.causal ? min(u.tok_end, u.pos0 + u.n_tok) : u.tok_end;
    return max(0, (key_end + kP - 1) / kP - u.tok_begin / kP);
  };

  // The loads run ahead of the products by the ring's depth, over the end of a
  // unit into the next ones: in_unit, in_j, in_n are the unit, page and page count
  // of the next pair to load; lane l holds the id of page in_j - in_j % 32 + l.
  int in_unit = rec.unit, in_j = 0, in_n = pages_of(rec.first);
  const int32_t* in_ids = a.page_indices + rec.first.page_base + rec.first.tok_begin / kP;
  int32_t ids = 0;
  const uint8_t* head = a.pool + (int64_t)kvh * S::PAGE;
  const uint32_t page_stride = (uint32_t)a.Hkv * S::PAGE;
  auto load_ids = [&]() {
    ids = in_j + lane < in_n ? ld_word(in_ids + in_j + lane) : 0;
    if (ids < 0 || ids >= a.num_pages) {
      set_device_error(a.err, kDevErrPageRange);
      ids = 0;  // a valid page instead; the output is undefined anyway
    }
  };
  auto load_next = [&](int st) {  // whole warp
    while (in_j >= in_n) {
      if (in_unit + 1 >= rec.unit_end) return;
      const Q4Unit u = a.units[++in_unit];
      in_n = pages_of(u);
      in_ids = a.page_indices + u.page_base + u.tok_begin / kP;
      in_j = 0;
      load_ids();
    }
    const uint32_t id0 = (uint32_t)__shfl_sync(0xffffffffu, ids, in_j & 31);
    const uint32_t id1 = (uint32_t)__shfl_sync(0xffffffffu, ids, (in_j + 1) & 31);
    if (lane == 0) {
      const bool two = in_j + 1 < in_n;
      uint8_t* dst = ring + st * S::STAGE;
      mbar_arrive_expect_tx(&full[st], two ? 2 * S::PAGE : S::PAGE);
      bulk_g2s(dst, head + (uint64_t)id0 * page_stride, S::PAGE, &full[st]);
      if (two) bulk_g2s(dst + S::PAGE, head + (uint64_t)id1 * page_stride, S::PAGE, &full[st]);
    }
    in_j += 2;
    if ((in_j & 31) == 0) load_ids();
  };
  load_ids();
  load_next(0);

  // Key of row r of S^T: the keys of a pair change places in odd threads of a
  // quad, so that the V rows a quad reads at once lie in different banks.
  const int key_r = r ^ ((r >> 1) & 1);
  const int key_v = 2 * c + (c & 1);                   // first key of a thread's pair of V rows
  const uint32_t pair_sel = (c & 1) ? 0x1032u : 0x3210u;
  const int k_off = key_r * (D / 2) + c * (D / 8);     // K codes of the thread, key row r
  const int v_off = S::SLICE + key_v * (D / 2) + r * (D / 16);
  const int v_step = (c & 1) ? -(D / 2) : D / 2;       // to the pair's other key
  const int sv_off = S::SLICE + 8 * D + (D == 128 ? r : r >> 1) * kP + 2 * c;

  int st = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int unit = rec.unit; unit < rec.unit_end; ++unit) {
  const Q4Unit u = unit == rec.unit ? rec.first : a.units[unit];
  const int rows = u.n_tok * g;
  const int n_pages = pages_of(u);

  // Q^T fragments: rows n = 8 t + r, this thread's dims [c * D/4, (c + 1) * D/4)
  float fs[NT][2];       // score factor of rows 8 t + 2 c, + 1
  int lim[NT][2];        // keys of those rows: [0, lim)
  int lim_min = INT_MAX;
  uint4 q_row[NT][D / 32];  // all loads at once; a row past the last is another one, set to zero
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = min(8 * t + r, rows - 1), tok = token_of(n);
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + ((int64_t)(u.q_row + tok) * a.Hq + kvh * g + (n - tok * g)) * D + c * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) q_row[t][i] = ld_16(src + i);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float x[D / 4];
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 w = q_row[t][i];
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = 8 * t + r < rows ? ww[j] : 0u;
        x[8 * i + 2 * j] = bf16lo_to_f32(v);
        x[8 * i + 2 * j + 1] = bf16hi_to_f32(v);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(x[i]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int ex = mx > 0.f ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -126), 126) : 0;
    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int w = 0; w < S::KWORDS; ++w)  // a lane reads what it writes here
      q_frag[(t * S::KWORDS + w) * 32 + lane] =
          make_uint4(pack_f16x2(x[8 * w] * down, x[8 * w + 1] * down),
                     pack_f16x2(x[8 * w + 2] * down, x[8 * w + 3] * down),
                     pack_f16x2(x[8 * w + 4] * down, x[8 * w + 5] * down),
                     pack_f16x2(x[8 * w + 6] * down, x[8 * w + 7] * down));
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int m = 8 * t + 2 * c + b;
      const int e = __shfl_sync(0xffffffffu, ex, 4 * (2 * c + b));  // row m's, held by lanes 4 (m % 8) ..
      fs[t][b] = score_factor(a.sm_scale, e + e_k);
      lim[t][b] = a.causal && m < rows ? min(u.pos0 + token_of(m) + 1, u.kv_len) : u.kv_len;
      lim_min = min(lim_min, lim[t][b]);
    }
  }
  // The rest of the ring once the first unit's rows are here: asked for at once by
  // every warp, it would queue in front of other warps' first pages.
  if (unit == rec.unit) {
#pragma unroll 1
    for (int i = 1; i < S::PAIRS; ++i) load_next(i);
  }
  // every lane agrees on whether a page needs masks
  lim_min = __reduce_min_sync(0xffffffffu, lim_min);

  float o[NT][S::TILES][4];
  // weights are 2^(s * fs - off), off = running maximum - kBias; before the first
  // visible key off is so low that any score raises it, and hidden ones (-inf)
  // weigh nothing
  float off[NT][2], l_run[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    off[t][0] = off[t][1] = kNoMax;
    l_run[t][0] = l_run[t][1] = 0.f;
#pragma unroll
    for (int i = 0; i < S::TILES; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
  }
#pragma unroll 1
  for (int j = 0; j < n_pages; j += 2) {
    mbar_wait(&full[st], phase, a.err);
    // the second page of a last single one is whatever the slot holds, with every
    // key hidden
    const uint8_t* stage = ring + st * S::STAGE;
    const int key0[2] = {u.tok_begin + j * kP, j + 1 < n_pages ? u.tok_begin + (j + 1) * kP : kHidden};

    // ---- S^T of the two pages
    float s[2][NT][4];
    constexpr int W = S::KWORDS;
    uint32_t kw[2][2][W];              // [page][key rows r, r + 8]
    uint32_t ks[2][2][2];              // block scales of the thread's dims
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[p][t][e] = 0.f;
      const uint8_t* kb = stage + p * S::PAGE + k_off;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(kb + h * (8 * 64));
          kw[p][h][0] = x.x; kw[p][h][1] = x.y; kw[p][h][2] = x.z; kw[p][h][3] = x.w;
          const uint8_t* sb = stage + p * S::PAGE + 1024 + key_r * 8 + 2 * c;
          const uint32_t y = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sb + 64 * h));
          ks[p][h][0] = __byte_perm(y, y, 0x1010);
          ks[p][h][1] = __byte_perm(y, y, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(kb + h * (8 * 32));
          kw[p][h][0] = x.x; kw[p][h][1] = x.y;
        }
      }
      if constexpr (D == 64) {
        // one block a thread: key rows r and r + 8 in one conversion
        const uint8_t* sb = stage + p * S::PAGE + 512 + key_r * 4 + c;
        const uint32_t y = e4m3x2_to_f16x2((uint16_t)(sb[0] | (sb[32] << 8)));
        ks[p][0][0] = ks[p][0][1] = __byte_perm(y, y, 0x1010);
        ks[p][1][0] = ks[p][1][1] = __byte_perm(y, y, 0x3232);
      }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint4 qw[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) qw[t] = q_frag[(t * W + w) * 32 + lane];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t h0[4], h1[4];
        e2m1x8_to_f16x2(kw[p][0][w], h0);
        e2m1x8_to_f16x2(kw[p][1][w], h1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h0[i] = mul_f16x2(h0[i], ks[p][0][(2 * w) / W]);
          h1[i] = mul_f16x2(h1[i], ks[p][1][(2 * w) / W]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma_f16(s[p][t], h0[0], h1[0], h0[1], h1[1], qw[t].x, qw[t].y);
          mma_f16(s[p][t], h0[2], h1[2], h0[3], h1[3], qw[t].z, qw[t].w);
        }
      }
    }
    const bool tail = max(key0[0], key0[1]) + kP > lim_min;  // some row does not see some key
    if (tail) {
      __syncwarp();  // a branch of its own: predicated, these would be issued for every pair
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0[p] + key_r + (e >= 2 ? 8 : 0) >= lim[t][e & 1]) s[p][t][e] = -INFINITY;
    }

    // ---- exponents; the maximum is raised when one passes it by kRaise
    float x[2][NT][4];
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[p][t][e] = fmaf(s[p][t][e], fs[t][e & 1], -off[t][e & 1]);
        top = fmax3(top, x[p][t][0], x[p][t][1]);
        top = fmax3(top, x[p][t][2], x[p][t][3]);
      }
    }
    if (__any_sync(0xffffffffu, top > kRaise + kBias)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float mx = fmax3(s[0][t][b], s[0][t][b + 2], fmaxf(s[1][t][b], s[1][t][b + 2]));
#pragma unroll
          for (int m = 4; m <= 16; m <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
          const float raised = fmaxf(off[t][b], mx * fs[t][b] - kBias);
          const float alpha = ex2_approx(off[t][b] - raised);  // 0 from kNoMax
          off[t][b] = raised;
          l_run[t][b] *= alpha;
#pragma unroll
          for (int i = 0; i < S::TILES; ++i) {
            o[t][i][b] *= alpha;
            o[t][i][b + 2] *= alpha;
          }
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            x[p][t][b] = fmaf(s[p][t][b], fs[t][b], -off[t][b]);
            x[p][t][b + 2] = fmaf(s[p][t][b + 2], fs[t][b], -off[t][b]);
          }
        }
    }

    // ---- P (fp16), transposed into the B operand of O^T += V^T P^T
    uint32_t pf[2][NT][2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = ex2_approx(x[p][t][i]);
        l_run[t][0] += e[0] + e[2];
        l_run[t][1] += e[1] + e[3];
        pf[p][t][0] = transpose8(pack_f16x2(e[0], e[1]));
        pf[p][t][1] = transpose8(pack_f16x2(e[2], e[3]));
      }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      constexpr int W = D / 64;        // code words of a thread per key
      uint32_t w[2][2][W];             // [pair of keys][key][word]
      uint32_t sc[2];
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        const uint8_t* row = stage + p * S::PAGE + v_off + pr * (4 * D);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (D == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(row + h * v_step);
            w[pr][h][0] = y.x;
            w[pr][h][W - 1] = y.y;
          } else {
            w[pr][h][0] = *reinterpret_cast<const uint32_t*>(row + h * v_step);
          }
        }
        sc[pr] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(stage + p * S::PAGE + sv_off + 8 * pr));
      }
      if (tail) {
        __syncwarp();
        // slots past the last key may hold anything: their scales count as zero
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          const int over = key0[p] + 8 * pr + 2 * c - u.kv_len;  // >= 0: both keys, -1: the second
          if (over >= -1) sc[pr] = over >= 0 ? 0u : sc[pr] & 0xFFFFu;
        }
      }
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) sc[pr] = __byte_perm(sc[pr], 0u, pair_sel);
#pragma unroll
      for (int y = 0; y < W; ++y) {
        uint32_t lo[2][4], hi[2][4];  // dims 2i, 2i + 1 of tile 4 y + i, for the two pairs
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          e2m1x8_to_f16x2(nibbles(w[pr][0][y], w[pr][1][y] << 4), lo[pr]);
          e2m1x8_to_f16x2(nibbles(w[pr][0][y] >> 4, w[pr][1][y]), hi[pr]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[pr][i] = mul_f16x2(lo[pr][i], sc[pr]);
            hi[pr][i] = mul_f16x2(hi[pr][i], sc[pr]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_f16(o[t][4 * y + i], lo[0][i], hi[0][i], lo[1][i], hi[1][i], pf[p][t][0], pf[p][t][1]);
      }
    }
    __syncwarp();  // both pages have been read
    load_next(st);
    if (++st == S::PAIRS) {
      st = 0;
      phase ^= 1u;
    }
  }

  // ---- write: a thread has D/8 dims in a row of two rows (2c, 2c + 1) a tile
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float L = l_run[t][b];
#pragma unroll
      for (int m = 4; m <= 16; m <<= 1) L += __shfl_xor_sync(0xffffffffu, L, m);
      const int n = 8 * t + 2 * c + b;
      if (n >= rows) continue;
      const float inv = L > 0.f || L != L ? f_v / L : 0.f;  // no visible key: zero, lse -inf
      const float lse2 = off[t][b] + __log2f(L);            // a weight is 2^(s - off)
      const int tok = token_of(n);
      const int hq = kvh * g + (n - tok * g);
      if (u.part < 0) {
        const int64_t row = (int64_t)(u.q_row + tok) * a.Hq + hq;
        uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + r * (D / 8));
#pragma unroll
        for (int i = 0; i < S::TILES; i += 4) {
          uint4 pk;
          pk.x = pack_bf16x2(o[t][i][b] * inv, o[t][i][b + 2] * inv);
          pk.y = pack_bf16x2(o[t][i + 1][b] * inv, o[t][i + 1][b + 2] * inv);
          pk.z = pack_bf16x2(o[t][i + 2][b] * inv, o[t][i + 2][b + 2] * inv);
          pk.w = pack_bf16x2(o[t][i + 3][b] * inv, o[t][i + 3][b + 2] * inv);
          dst[i / 4] = pk;
        }
        if (r == 0 && a.lse_out) a.lse_out[row] = lse2 * 0.69314718055994531f;
      } else {
        const int64_t row = ((int64_t)u.part + (int64_t)tok * u.part_stride) * a.Hq + hq;
        float* dst = a.part_o + row * D + r * (D / 8);
#pragma unroll
        for (int i = 0; i < S::TILES; i += 4)
          st_32(dst + 2 * i, o[t][i][b] * inv, o[t][i][b + 2] * inv, o[t][i + 1][b] * inv,
                o[t][i + 1][b + 2] * inv, o[t][i + 2][b] * inv, o[t][i + 2][b + 2] * inv,
                o[t][i + 3][b] * inv, o[t][i + 3][b + 2] * inv);
        if (r == 0) a.part_lse[row] = lse2;
      }
    }
  }
  // This grid reads nothing of the one before it in the call; its completion
  // still has to imply that one's, for what follows on the stream.
  if (blockIdx.x == 0) grid_dep_wait();
}

// softmax_merge of the parts of a (token, query head): weights 2^(lse - M) with M the
// running maximum of lse, their sum and the weighted sum of the parts (lse in the
// log2 domain).  Bound: latency (a part and its lse are loaded together, kMergeLoads
// parts at a time).  W warps share a row: one where rows have few parts, so that a
// wave of CTAs holds as many rows as it can; four where they have many (GB300, decode
// of 128 requests, 12 heads, 15 parts on average and 47 at most: 12.5 us with one, 7
// with four; 160 tokens, 32 heads, 6 parts: 7 us and 10).
constexpr int kMergeWarps = 4;
constexpr int kMergeLoads = 6;
constexpr int kMergeWideParts = 10;  // parts of a token, on average, from which four warps share it

template <int D, int W>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_q4_kernel(const MergeArgs a) {
  constexpr int EPL = D / 32;  // dims of a lane
  __shared__ float s_acc[W > 1 ? W : 1][W > 1 ? D : 1];
  __shared__ float s_sum[W], s_max[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MergeItem it = a.items[blockIdx.x];
  const int hq = blockIdx.y * (kMergeWarps / W) + warp / W;
  const int share = warp % W;
  if (hq >= a.Hq) return;  // W == 1 only
  const float* lse = a.part_lse + (int64_t)it.part_begin * a.Hq + hq;
  const float* part = a.part_o + ((int64_t)it.part_begin * a.Hq + hq) * D + lane * EPL;
  const int64_t stride = (int64_t)a.Hq * D;
  grid_dep_wait();  // the parts come from the kernel launched before
  // a share's weights are relative to its own maximum, M, raised as it goes
  float acc[EPL], sum = 0.f, M = -FLT_MAX;
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  for (int p0 = share; p0 < it.n_parts; p0 += W * kMergeLoads) {
    float w[kMergeLoads], v[kMergeLoads][EPL];
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) {
      const int p = p0 + i * W;
      w[i] = p < it.n_parts ? lse[(int64_t)p * a.Hq] : -INFINITY;
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = 0.f;
      if (p < it.n_parts) {
        if constexpr (EPL == 4) {
          const float4 x = *reinterpret_cast<const float4*>(part + p * stride);
          v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(part + p * stride);
          v[i][0] = x.x; v[i][1] = x.y;
        }
      }
    }
    float raised = M;
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) raised = fmaxf(raised, w[i]);
    const float alpha = ex2_approx(M - raised);
    M = raised;
    sum *= alpha;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] *= alpha;
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) {
      const float x = ex2_approx(w[i] - M);
      sum += x;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = fmaf(x, v[i][e], acc[e]);
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) s_acc[warp][lane * EPL + e] = acc[e];
    if (lane == 0) {
      s_sum[warp] = sum;
      s_max[warp] = M;
    }
    __syncthreads();
    if (warp > 0) return;
    const float M0 = M;
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, s_max[w]);
    const float alpha = ex2_approx(M0 - M);
    sum *= alpha;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] *= alpha;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float x = ex2_approx(s_max[w] - M);
      sum = fmaf(x, s_sum[w], sum);
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = fmaf(x, s_acc[w][lane * EPL + e], acc[e]);
    }
  }
  const float inv = 1.f / sum;
  const int64_t row = (int64_t)it.q_row * a.Hq + hq;
  uint16_t* dst = a.out + row * D + lane * EPL;
  if constexpr (EPL == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0 && a.lse_out) a.lse_out[row] = (M + __log2f(sum)) * 0.69314718055994531f;
}

template <int D, int NT>
cudaError_t launch_t(AttentionQ4Args a, int n_ranges, bool programmatic, bool beside, cudaStream_t stream) {
  using S = Shape<D, NT>;
  a.n_ranges = n_ranges;
  a.wait_first = !beside;
  auto kern = attention_q4_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)a.Hkv * n_ranges;
  return launch_kernel(kern, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(32 * kWarps), S::SMEM,
                       stream, programmatic, a);
}

template <int D>
cudaError_t launch_d(AttentionQ4Args a, const int (&n_ranges)[kQ4Classes], bool programmatic, bool beside,
                     cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < kQ4Classes && e == cudaSuccess; ++i) {
    if (n_ranges[i] == 0) continue;
    e = i == 0   ? launch_t<D, 1>(a, n_ranges[i], programmatic, beside, stream)
        : i == 1 ? launch_t<D, 2>(a, n_ranges[i], programmatic, beside, stream)
                 : launch_t<D, 3>(a, n_ranges[i], programmatic, beside, stream);
    beside = programmatic;
    a.ranges += n_ranges[i];
  }
  return e;
}

}  // namespace

cudaError_t launch_attention_q4(const AttentionQ4Args& a, const int (&n_ranges)[kQ4Classes],
                                bool programmatic, bool beside, cudaStream_t stream) {
  return a.head_dim == 128 ? launch_d<128>(a, n_ranges, programmatic, beside, stream)
                           : launch_d<64>(a, n_ranges, programmatic, beside, stream);
}

cudaError_t launch_merge_q4(const MergeArgs& a, int n_parts, bool programmatic, cudaStream_t stream) {
  if (a.n_items <= 0) return cudaSuccess;
  const bool wide = n_parts >= kMergeWideParts * a.n_items;
  const dim3 grid(a.n_items, wide ? a.Hq : (a.Hq + kMergeWarps - 1) / kMergeWarps), block(32 * kMergeWarps);
  void (*kern)(MergeArgs) = a.head_dim == 128 ? (wide ? merge_q4_kernel<128, 4> : merge_q4_kernel<128, 1>)
                                              : (wide ? merge_q4_kernel<64, 4> : merge_q4_kernel<64, 1>);
  return launch_kernel(kern, grid, block, 0, stream, programmatic, a);
}

}  // namespace daa
