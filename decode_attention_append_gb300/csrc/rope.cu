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
// rounded; a model that keeps bf16 there differs by that rounding, 2^-8.)
//
// Angles.  p f_i grows to 10^5 and more, where fp32 has no digits of the angle left.
// A pair's turns a token are held as a 64-bit fraction of a turn: p times it, modulo
// 2^64, is the angle modulo one turn, exact but for p 2^-65 turns.  Its upper 8 bits,
// rounded, name a table entry (sine and cosine of n / 256 turns); the rest, at most
// 2^-9 turns, goes through short series and the addition theorems (cos_sin).  No table
// of positions is needed, and no position is too far or negative.
//
// Layout.  A warp takes a row, or a part of its heads where rows are few.  It finds
// the row's request and place, works out the row's sines once (one pair a lane, by way
// of shared memory), and then streams heads: a head is D / 16 lanes of two 16-byte
// chunks each, chunks j and j + rotary_dim / 16 for the half layout, so that a lane
// holds whole pairs and keeps its eight sines and cosines in registers.  Loads run
// kAhead heads ahead of their use, the first ones ahead of the search.  Warps share
// nothing but constants: no barrier behind the first.  Each layout has kernels of its
// own (keys into 4 bits with one for all: 153 us where interleaved heads take 119 and
// parts of heads 116); many rotated rows share one (kEitherRounds).
//   With the sines of a CTA's rows in shared memory and two barriers: 297 us for the first
// case below, 249 instructions a warp of heads where this takes 126.
//   Four rows a warp, 32,800 rows: into bf16 pages 24 us for 3 heads a row where LEAN takes
// 28, but 31 and 30 for 6, 49 and 44 for 14; into 4 bits, which has no such form, 35 us
// where a row a warp takes 45, 45 and 51 for 6, 58 and 59 for 14, 69 and 66 for 20.  Not
// built: a second set of kernels for rows of very few heads.
//
// Bound, and times on GB300 (graph replays; bytes at 6,785 GB/s, a copy's rate):
//   32,832 rows of 80 heads of 128 dims appended   HBM: 200 us, 99 % of that rate
//   16,416 rows of 72 heads rotated                HBM and the last wave: 96 us, 93 %
//   36,760 rows of 48 heads into 4 bits            147 us, 77 %: instructions (55 % of the
//       issue slots) and latency at 18 warps an SM.  Keys rotated as queries are would
//       take 11 us less of it, and stray from the definition at one code in some 10^6.
//   16,416 rows of 48 heads (8 of keys) with norms into 4 bits 101 us, 52 %, of 96 (32)
//       222 us, 41 %: instructions (4,118 a row of 48, 57 % of the issue slots at 18 warps
//       an SM).  Every key is normalised and turned in two parts, for the few that need it.
//   128 rows of 14 heads, 32 of 64                 2.8 and 1.6 us: a launch, and two or
//       three dependent loads
//   32,800 rows of 10 heads appended 38 us, 66 %, of 14 44 us, 79 %, rotated (9 and 13)
//       32 and 41 us, 70 and 79 %, into 4 bits 53 and 60 us, 44 and 55 %: what a row
//       costs before its heads (search, place, sines: about 450 instructions a warp of
//       1,264 a row of 10 heads into 4 bits).
#include <algorithm>

#include "launch.h"
#include "place.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace daa {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
enum Layout { kPart, kWhole, kInterleaved, kEither };  // pairs of halves of a part or all of the head; neighbours; by a look
constexpr int kP = 16;
// Heads of a lane in flight, and CTAs of an SM that registers are left for.  Rows are
// bound by HBM and want warps: 16,416 rows of 72 heads 96 us with two and 7 CTAs, 104
// with 6, 98 with 8 (spills).  Pages want loads in flight: 32,832 rows of 80 heads 200
// us with five heads and 4 CTAs, 205 with two and 7; a chunk beside decodes 3.9 and 4.8.
// But where rows are many and of few heads, what comes before a row's heads is most of
// it, and more warps do that at a time (LEAN: two heads and 7 CTAs): 32,800 rows of 14
// heads 44 us and not 53, of 10 38 and 47, of 20 56 and 60, of 32 no difference; of 64
// dims, where as many rounds are twice the heads, of 10 30 and 40, of 28 46 and 53, of 48
// 69 and 71, of 64 (past kLeanRounds) 87 and 89.  The 4-bit append is bound by
// instructions and latency: 36,760 rows of 48 heads 147 us with three heads and 5 CTAs,
// 155 with two, 159 with 4 CTAs.  With norms 96 registers hold it for whole heads only
// (16,416 rows of 48: 101 us, 105 with 4 CTAs; interleaved 113, 108).  Without, interleaved
// heads spill 56 bytes at 96 registers, and neither count is best for all of them: 16,416
// rows of 48 heads of 128 dims 78.6 us with 5 CTAs and 77.5 with 4, of 96 165 and 155, 544
// rows of 48 6.0 and 4.9; but of 14 heads 32.5 and 34.5, of 36 57.0 and 59.7, 1,332 rows
// of 32 6.3 and 7.2, of 28 heads of 64 dims 35.5 and 36.9.
constexpr int ahead_of(int target, bool norm, bool lean) {
  return target == kRopeRows || lean ? 2 : target == kRopePages ? 5 : norm ? 2 : 3;
}
constexpr int ctas_of(int target, bool norm, int layout, bool lean) {
  return target == kRopeRows    ? (norm ? 5 : 7)
         : target == kRopePages ? (lean ? 7 : 4)
                                : (norm && layout != kWhole ? 4 : 5);
}
constexpr int kLeanRounds = 6;  // of a warp's heads at a time, a row
// Rows without norms of heads that are not turned whole: one kernel that looks at the layout,
// where a warp has so many rounds of heads and rows are many (16,416 rows of 72 heads, half of
// each turned 96.8 us, 99.8 with the layout's own kernel; interleaved 95.7 and 97.2; of 13
// 22.8 and 23.7).  Below, and where rows share warps, the layout's own: of 9 heads 18.5 and
// 18.6, of 5 12.3 and 13.2; 632 rows of 64 interleaved heads 4.3 and 4.6.  Heads of 64 dims
// change over at the same rounds (24 heads 20.8 and 21.5, 36 28.7 and 28.5, 72 51.5 and 50.9).
constexpr int kEitherRounds = 4;

// ------------------------------------------------------------------- angles
// Sine and cosine of n / 256 turns, each as the sum of two fp32 numbers.
constexpr int kSteps = 256;
constexpr double kTwoPi = 6.283185307179586;

struct __align__(16) SineTable {
  float v[kSteps][4];  // cosine: upper, lower; sine: upper, lower
};

constexpr double series(double x, int first) {  // Taylor's, of sine (1) or cosine (0), |x| <= pi / 4
  double term = first ? x : 1.0, sum = term;
  for (int n = first + 1; n < 24; n += 2) {
    term *= -x * x / (n * (n + 1.0));
    sum += term;
  }
  return sum;
}

constexpr SineTable make_table() {
  SineTable t{};
  for (int n = 0; n < kSteps; ++n) {
    const int quarter = n / 64, r = n % 64;
    const double a = (r <= 32 ? r : 64 - r) * (kTwoPi / kSteps);
    const double x = series(a, r <= 32 ? 0 : 1), y = series(a, r <= 32 ? 1 : 0);  // cosine, sine within the quarter
    const double c = quarter == 0 ? x : quarter == 1 ? -y : quarter == 2 ? -x : y;
    const double s = quarter == 0 ? y : quarter == 1 ? x : quarter == 2 ? -y : -x;
    t.v[n][0] = (float)c;
    t.v[n][1] = (float)(c - t.v[n][0]);
    t.v[n][2] = (float)s;
    t.v[n][3] = (float)(s - t.v[n][2]);
  }
  return t;
}

__device__ constexpr SineTable g_sines = make_table();

// Two fp32 numbers in one instruction, each rounded by itself; below, T is float or F2.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 both(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void apart(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 neg(F2 a) { return F2{a.v ^ 0x8000000080000000ull}; }
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, both(-1.f, -1.f), a); }
__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ float neg(float a) { return -a; }
__device__ __forceinline__ float sub(float a, float b) { return __fsub_rn(a, b); }
__device__ __forceinline__ F2 same(float a) { return both(a, a); }

// a + b = s + e exactly.
template <class T>
__device__ __forceinline__ void two_sum(T a, T b, T& s, T& e) {
  s = add(a, b);
  const T t = sub(s, a);
  e = add(sub(a, sub(s, t)), sub(b, t));
}
// a b = p + e exactly.
template <class T>
__device__ __forceinline__ void two_prod(T a, T b, T& p, T& e) {
  p = mul(a, b);
  e = fma(a, b, neg(p));
}

// m cos and m sin of two phases of 2^-64 turns, each the sum of two fp32 numbers, good to
// 2^-35 of m.
struct CosSin {
  F2 ch, cl, sh, sl;
};
__device__ __forceinline__ CosSin cos_sin(uint64_t phase0, uint64_t phase1, const float4* table, float mh, float ml) {
  // d = dh + dl in 2^-40 turns beside the table's angle, |d| <= 1 / 512 turns
  auto split = [&](uint64_t phase, float4& t, float& dh, float& dl) {
    const uint32_t n = (uint32_t)((phase + (1ull << 55)) >> 56);
    const int32_t r = (int32_t)((int64_t)(phase - ((uint64_t)n << 56)) >> 24);
    t = table[n];
    dh = (float)r;
    dl = (float)(r - (int32_t)dh);
  };
  float4 t0, t1;
  float dh0, dl0, dh1, dl1;
  split(phase0, t0, dh0, dl0);
  split(phase1, t1, dh1, dl1);
  const F2 C = both(t0.x, t1.x), Cl = both(t0.y, t1.y), S = both(t0.z, t1.z), Sl = both(t0.w, t1.w);
  const F2 dh = both(dh0, dh1), dl = both(dl0, dl1);
  // in radians vh + vl, |d| <= pi / 256
  constexpr double unit = kTwoPi / 1099511627776.0;
  constexpr float kh = (float)unit, kl = (float)(unit - kh);
  F2 vh, vl;
  two_prod(dh, same(kh), vh, vl);
  vl = add(vl, fma(dh, same(kl), mul(dl, same(kh))));
  // cos d - 1 = u + ul, sin d = vh + sl:  d^2 / 2 <= 2^-13.7, d^3 / 6 <= 2^-21.6
  F2 z, zl;
  two_prod(vh, vh, z, zl);
  const F2 half = same(-0.5f), u = mul(z, half);
  const F2 ul = fma(mul(z, z), same(1.f / 24), fma(neg(vh), vl, mul(zl, half)));
  const F2 sl = fma(mul(vh, z), fma(z, same(1.f / 120), same(-1.f / 6)), vl);
  // cos (t + d) = C + C u - S v,  sin (t + d) = S + S u + C v
  auto turned = [&](F2 A, F2 Al, F2 B, F2 Bl, F2& h, F2& low) {
    F2 a, ae, b, be, d, de, g, ge;
    two_prod(A, u, a, ae);
    two_prod(B, vh, b, be);
    two_sum(a, b, d, de);
    two_sum(A, d, g, ge);
    low = add(add(ge, de), add(ae, be));
    low = add(low, fma(A, ul, fma(B, sl, fma(Bl, vh, fma(Al, u, Al)))));
    h = add(g, low);
    low = sub(low, sub(h, g));
  };
  auto scaled = [&](F2 h, F2 l, F2& oh, F2& ol) {
    F2 a, ae;
    two_prod(h, same(mh), a, ae);
    ae = add(ae, fma(h, same(ml), mul(l, same(mh))));
    oh = add(a, ae);
    ol = sub(ae, sub(oh, a));
  };
  CosSin o;
  F2 h, l;
  turned(C, Cl, neg(S), neg(Sl), h, l);
  scaled(h, l, o.ch, o.cl);
  turned(S, Sl, C, Cl, h, l);
  scaled(h, l, o.sh, o.sl);
  return o;
}

// ----------------------------------------------------------------- rotations
// (a, b) -> (a c - b s, b c + a s), each a product and a fused product.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
  b = __fmaf_rn(b, c, __fmul_rn(a, s));
  a = x;
}

// a c + b s = d + e, to 2^-40 of |a| + |b|, with c and s in 16 bits and the rest.
// Of a and b of 8 bits the upper products are exact; of 16 bits (LONG) they are not.
template <bool LONG, class T>
__device__ __forceinline__ void sum_of_products(T a, T c, T cl, T b, T s, T sl, T& d, T& e) {
  T low;
  if (LONG) {
    T p, pe, q, qe;
    two_prod(a, c, p, pe);
    two_prod(b, s, q, qe);
    two_sum(p, q, d, e);
    low = fma(a, cl, fma(b, sl, add(pe, qe)));
  } else {
    two_sum(mul(a, c), mul(b, s), d, e);
    low = fma(a, cl, mul(b, sl));
  }
  e = add(e, low);
}

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

// ------------------------------------------------------------- a row's place
// New row `row`: its position in its request and the index of its page id, or false for
// a row of which nothing is written.  A warp's lanes together.
__device__ __forceinline__ bool find_place(const RopeArgs& a, int row, int lane, int& pos, int& page_at) {
  // the last request r with append_indptr[r] <= row: narrowed to 256 by probes, then counted
  int lo = 0, n = a.batch;
  while (n > 256) {
    const int step = (n + 31) / 32;
    const bool below = lane * step < n && ld_word(a.append_indptr + lo + lane * step) <= row;
    const int k = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  int r = lo - 1;
  {
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = INT32_MAX;
      if (32 * i < n && 32 * i + lane < n) v[i] = ld_word(a.append_indptr + lo + 32 * i + lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) r += __popc(__ballot_sync(0xffffffffu, v[i] <= row));
  }
  r = max(r, 0);
  const int32_t* p = lane == 0   ? a.append_indptr + r
                     : lane == 1 ? a.append_indptr + r + 1
                     : lane == 2 ? a.kv_indptr + r
                     : lane == 3 ? a.kv_indptr + r + 1
                     : lane == 4 ? a.last_page_len + r
                     : lane == 5 ? a.append_indptr + a.batch
                                 : a.kv_indptr + a.batch;
  const int word = lane < 7 ? ld_word(p) : 0;
  const int a0 = __shfl_sync(0xffffffffu, word, 0), a1 = __shfl_sync(0xffffffffu, word, 1);
  const int p0 = __shfl_sync(0xffffffffu, word, 2), p1 = __shfl_sync(0xffffffffu, word, 3);
  const int last_len = __shfl_sync(0xffffffffu, word, 4), rows_end = __shfl_sync(0xffffffffu, word, 5);
  const int pages_end = __shfl_sync(0xffffffffu, word, 6);
  if (row >= rows_end) return false;  // padding behind the last request
  if (!row_place(row, a0, a1, p0, p1, pages_end, last_len, pos, page_at)) {
    set_device_error(a.err, kDevErrShape);
    return false;
  }
  return true;
}

template <int D, int TARGET, bool NORM, int LAYOUT, bool LEAN>
__global__ void __launch_bounds__(kThreads, ctas_of(TARGET, NORM, LAYOUT, LEAN)) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int L = D / 16, G = 32 / L;  // lanes of a head, heads of a warp at a time
  constexpr bool APPEND = TARGET != kRopeRows, Q4 = TARGET == kRopePagesQ4;
  constexpr bool FULL = LAYOUT == kWhole;
  constexpr int kAhead = ahead_of(TARGET, NORM, LEAN);
  __shared__ float4 s_table[kSteps];
  __shared__ uint64_t s_turns[64];
  // a row's cosines and sines; of both, 16 bits and what these leave
  __shared__ __align__(16) float s_angle[kWarps][Q4 ? 6 : 2][64];
  __shared__ __align__(16) float s_w[NORM ? 2 : 1][D];  // norm weights of q and k

  const bool pairs = LAYOUT == kInterleaved || (LAYOUT == kEither && a.interleaved != 0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, group = lane / L, j = lane % L;
  const uint32_t mask = (L == 8 ? 0xFFu : 0xFu) << (lane & ~(L - 1));  // the head's lanes
  grid_dep_launch();
  for (int t = tid; t < kSteps; t += kThreads) s_table[t] = *reinterpret_cast<const float4*>(g_sines.v[t]);
  if (tid < 64) s_turns[tid] = a.turns[tid];
  __syncthreads();
  grid_dep_wait();
  // norm weights: asked for now, in shared memory once the first heads are asked for too
  constexpr int kWeights = NORM ? 2 * D / kThreads : 0;
  uint16_t weight[NORM ? kWeights : 1];
#pragma unroll
  for (int i = 0; i < kWeights; ++i) {
    const int t = tid + i * kThreads;
    const uint16_t* n = t < D ? a.q_norm : a.k_norm;
    weight[i] = 0;
    if (n) asm volatile("ld.global.u16 %0, [%1];" : "=h"(weight[i]) : "l"(n + t % D));
  }

  const int task = blockIdx.x * kWarps + warp;
  const int row = task / a.parts, first = (task - row * a.parts) * a.part_heads;
  const bool live = row < a.n_rows;
  const int H = a.Hq + (APPEND ? 2 : 1) * a.Hk;
  const int end = live ? min(first + a.part_heads, H) : 0;
  // chunks of 8 dims of this lane; in a 4-bit cache's rows two side by side, a block
  const int nrot = FULL ? L : a.rotary_dim / 16;
  const int c0 = FULL || pairs || j < nrot ? j : 2 * j;
  const int c1 = FULL || pairs ? j + L : j < nrot ? j + nrot : 2 * j + 1;
  const uint16_t* q_row = a.q.p + row * a.q.row;
  const uint16_t* k_row = a.k.p + row * a.k.row;
  const uint16_t* v_row = a.v.p + row * a.v.row;
  auto side_by_side = [&](int head) { return Q4 && head >= a.Hq && (pairs || head >= a.Hq + a.Hk); };
  auto load = [&](int head, uint32_t (&w)[8]) {
    const int h = head - a.Hq;
    const uint16_t* p = h < 0 ? q_row + head * a.q.head : !APPEND || h < a.Hk ? k_row + h * a.k.head : v_row + (h - a.Hk) * a.v.head;
    const bool side = side_by_side(head);
    const uint4 lo = ld_stream(p + 8 * (side ? 2 * j : c0)), hi = ld_stream(p + 8 * (side ? 2 * j + 1 : c1));
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
    w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
  };
  uint32_t w[kAhead][8];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (first + u * G + group < end) load(first + u * G + group, w[u]);

  int given = 0;
  if (live && a.positions) given = ld_word(a.positions + row);
  if (NORM) {
#pragma unroll
    for (int i = 0; i < kWeights; ++i)
      s_w[(tid + i * kThreads) / D][(tid + i * kThreads) % D] = __uint_as_float((uint32_t)weight[i] << 16);
    __syncthreads();
  }
  if (!live) return;
  int place = 0, page_at = 0, page = 0;
  if (APPEND) {
    if (!find_place(a, row, lane, place, page_at)) return;
    page = ld_word(a.page_indices + page_at);
  }
  const int pos = a.positions ? given : place, slot = place % kP;
  float(&angle)[Q4 ? 6 : 2][64] = s_angle[warp];
  {
    // pairs lane and lane + 32 (where there are so many)
    const CosSin x = cos_sin(s_turns[lane] * (uint64_t)(int64_t)pos, s_turns[lane + 32] * (uint64_t)(int64_t)pos, s_table,
                             a.magnitude, a.magnitude_low);
    auto put = [&](int i, F2 y) { apart(y, angle[i][lane], angle[i][lane + 32]); };
    put(0, x.ch);
    put(1, x.sh);
    if (Q4) {
      const F2 ch{x.ch.v & 0xFFFFFF00FFFFFF00ull}, sh{x.sh.v & 0xFFFFFF00FFFFFF00ull};
      put(Q4 ? 2 : 0, ch);
      put(Q4 ? 3 : 0, add(sub(x.ch, ch), x.cl));
      put(Q4 ? 4 : 0, sh);
      put(Q4 ? 5 : 0, add(sub(x.sh, sh), x.sl));
    }
  }
  __syncwarp();
  // this lane's pairs: whether its two chunks turn, and by what
  auto turns = [&](int chunk) { return FULL || (pairs ? chunk < 2 * nrot : j < nrot); };
  auto sines_of = [&](int d0, int d1, float (&c)[8], float (&s)[8]) {
    const int i0 = pairs ? 4 * d0 : 8 * j, i1 = pairs ? 4 * d1 : 8 * j + 4;
    if (turns(d0)) {
      load4(angle[0] + i0, c);
      load4(angle[1] + i0, s);
    }
    if (turns(d1)) {
      load4(angle[0] + i1, c + 4);
      load4(angle[1] + i1, s + 4);
    }
  };
  float lane_c[8], lane_s[8];  // of chunks c0 and c1
  sines_of(c0, c1, lane_c, lane_s);

  // normalised, turned by c and s, rounded: chunks d0 and d1
  auto rotate = [&](uint32_t (&v)[8], bool is_q, int d0, int d1, const float (&c)[8], const float (&s)[8]) {
    const bool t0 = turns(d0), t1 = turns(d1);
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = bf16lo_to_f32(v[i]);
      x[2 * i + 1] = bf16hi_to_f32(v[i]);
    }
    const bool norm = NORM && (is_q ? a.q_norm : a.k_norm) != nullptr;
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = __fmaf_rn(x[i], x[i], ss);
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(mask, ss, m);
      const float k = rsqrtf(ss * (1.f / D) + a.eps);
      const float* wt = s_w[is_q ? 0 : NORM];
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
  };

  // The same of k that is quantised, in two parts: a code changes by up to a third where a key
  // falls on the other side of a border, so it is the definition that decides and not
  // the order of fp32 operations.  As above, to the nearest fp32 and then to bf16.
  auto rotate_exactly = [&](uint32_t (&v)[8], int d0, int d1) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = bf16lo_to_f32(v[i]);
      x[2 * i + 1] = bf16hi_to_f32(v[i]);
    }
    const bool norm = NORM && a.k_norm != nullptr;
    float r = 1.f, rl = 0.f;
    if (norm) {
      float ss = 0.f, sl = 0.f, e;  // the squares are exact
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        two_sum(ss, __fmul_rn(x[i], x[i]), ss, e);
        sl = __fadd_rn(sl, e);
      }
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) {
        two_sum(ss, __shfl_xor_sync(mask, ss, m), ss, e);
        sl = __fadd_rn(__fadd_rn(sl, __shfl_xor_sync(mask, sl, m)), e);
      }
      two_sum(ss * (1.f / D), a.eps, ss, e);
      sl = __fmaf_rn(sl, 1.f / D, e);
      // one step of Newton's from r: 1 / sqrt(ss + sl) = r (1 + t / 2), t = 1 - (ss + sl) r^2
      r = rsqrtf(ss);
      float rr, re;
      two_prod(r, r, rr, re);
      const float t = __fsub_rn(__fmaf_rn(-ss, rr, 1.f), __fmaf_rn(ss, re, __fmul_rn(sl, rr)));
      // r's power of two goes to the values ahead of the weights: their products stay near the
      // outputs' size, whatever the head's and the weights' are
      const float two = __uint_as_float(__float_as_uint(r) & 0x7F800000u);
      r = __uint_as_float((__float_as_uint(r) & 0x007FFFFFu) | 0x3F800000u);
      rl = isfinite(t) ? 0.5f * r * t : 0.f;
      const float* wt = s_w[NORM];
      float g[16];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        load4(wt + 8 * d0 + i, g + i);
        load4(wt + 8 * d1 + i, g + 8 + i);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], two), g[i]);  // 16 bits: exact
    }
    auto scaled = [&](float d, float e) {  // (d + e) (r + rl)
      if (!NORM || !norm) return __fadd_rn(d, e);
      float h, he;
      two_prod(d, r, h, he);
      return __fadd_rn(h, __fadd_rn(he, __fmaf_rn(d, rl, __fmul_rn(e, r))));
    };
    const bool z0 = turns(d0), z1 = turns(d1);
    const int e0 = pairs ? 4 * d0 : 8 * j, e1 = pairs ? 4 * d1 : 8 * j + 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // half layout: pairs 4 half + i of the two chunks; else those of this half's chunk
      if (half ? z1 : z0) {
        const int at_pair = half ? e1 : e0;
        float ch[4], cl[4], sh[4], sl[4];
        load4(angle[Q4 ? 2 : 0] + at_pair, ch);
        load4(angle[Q4 ? 3 : 0] + at_pair, cl);
        load4(angle[Q4 ? 4 : 0] + at_pair, sh);
        load4(angle[Q4 ? 5 : 0] + at_pair, sl);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float p, pe, q, qe;
          if (pairs) {
            float &u = x[8 * half + 2 * i], &w = x[8 * half + 2 * i + 1];
            sum_of_products<NORM>(u, ch[i], cl[i], -w, sh[i], sl[i], p, pe);
            sum_of_products<NORM>(w, ch[i], cl[i], u, sh[i], sl[i], q, qe);
            u = scaled(p, pe);
            w = scaled(q, qe);
          } else {
            float &u = x[4 * half + i], &w = x[4 * half + i + 8];
            sum_of_products<NORM>(u, ch[i], cl[i], -w, sh[i], sl[i], p, pe);
            sum_of_products<NORM>(w, ch[i], cl[i], u, sh[i], sl[i], q, qe);
            u = scaled(p, pe);
            w = scaled(q, qe);
          }
        }
      } else if (norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (pairs) {
            x[8 * half + 2 * i] = scaled(x[8 * half + 2 * i], 0.f);
            x[8 * half + 2 * i + 1] = scaled(x[8 * half + 2 * i + 1], 0.f);
          } else {
            x[4 * half + i] = scaled(x[4 * half + i], 0.f);
            x[4 * half + i + 8] = scaled(x[4 * half + i + 8], 0.f);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (norm || z0) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      if (norm || z1) v[4 + i] = pack_bf16x2(x[8 + 2 * i], x[9 + 2 * i]);
    }
  };

  uint16_t* q_out = a.q_out.p + row * a.q_out.row;
  const bool no_page = APPEND && (page < 0 || page >= a.num_pages);  // its q is rotated all the same
  if (no_page) set_device_error(a.err, kDevErrPageRange);
  auto finish = [&](int head, uint32_t (&v)[8]) {
    const int h = head - a.Hq;  // of k, then of v
    const bool is_q = h < 0, is_k = !is_q && (!APPEND || h < a.Hk);
    const bool side = side_by_side(head);
    const int d0 = side ? 2 * j : c0, d1 = side ? 2 * j + 1 : c1;
    if (Q4 && is_k) {
      // past 2^100 products leave fp32's range, and their small parts are no numbers
      if ((NORM && a.k_norm) || max_abs_bits(v) < 0x7180u) {
        rotate_exactly(v, d0, d1);
      } else {
        float c[8], s[8];
        sines_of(d0, d1, c, s);
        rotate(v, false, d0, d1, c, s);
      }
    } else if (is_q || is_k) {
      rotate(v, is_q, c0, c1, lane_c, lane_s);
    }
    if (is_q || !APPEND) {
      uint16_t* p = is_q ? q_out + head * a.q_out.head : a.k_out.p + row * a.k_out.row + h * a.k_out.head;
      st_16(p + 8 * c0, v);
      st_16(p + 8 * c1, v + 4);
    } else if (no_page) {
    } else if (!Q4) {
      // a page is [2][Hk][16][D]: v's heads follow k's
      uint16_t* p = reinterpret_cast<uint16_t*>(a.pool) + (((int64_t)page * 2 * a.Hk + h) * kP + slot) * D;
      st_16(p + 8 * c0, v);
      st_16(p + 8 * c1, v + 4);
    } else {
      uint4 b[2] = {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])};
      if (!side) {
        // chunks 2j and 2j + 1 of the head, from the lanes that have them
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 2 * j + i;
          const int from = t < nrot ? t : FULL || t < 2 * nrot ? t - nrot : t / 2;
          const bool upper = FULL || t < 2 * nrot ? t >= nrot : (t & 1) != 0;
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = __shfl_sync(mask, v[k], from, L), hi = __shfl_sync(mask, v[4 + k], from, L);
            o[k] = upper ? hi : lo;
          }
          b[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      const int kv = is_k ? 0 : 1, hk = h - kv * a.Hk;
      const float me = a.kv_exp ? q4_pow2(-ld_word(a.kv_exp + h)) : 1.f;
      uint8_t scale;
      const uint2 codes = quantise_block(b[0], b[1], me, scale);
      uint8_t* slice = a.pool + (((int64_t)page * a.Hk + hk) * 2 + kv) * q4_slice_bytes(D);
      *reinterpret_cast<uint2*>(slice + slot * (D / 2) + j * 8) = codes;
      slice[kP * (D / 2) + (kv == 0 ? slot * L + j : j * kP + slot)] = scale;
    }
  };

  for (int base = first + group; base < end; base += kAhead * G) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int head = base + u * G;
      if (head < end) {
        finish(head, w[u]);
        if (head + kAhead * G < end) load(head + kAhead * G, w[u]);
      }
    }
  }
}

template <int D, int TARGET, bool LEAN, bool NORM>
auto kernel_of(int layout) {
  if constexpr (TARGET == kRopeRows && !NORM) {
    if (layout == kEither) return rope_kernel<D, TARGET, NORM, kEither, LEAN>;
  }
  return layout == kWhole         ? rope_kernel<D, TARGET, NORM, kWhole, LEAN>
         : layout == kInterleaved ? rope_kernel<D, TARGET, NORM, kInterleaved, LEAN>
                                  : rope_kernel<D, TARGET, NORM, kPart, LEAN>;
}
template <int D, int TARGET, bool LEAN>
auto kernel_of(bool norm, int layout) {
  return norm ? kernel_of<D, TARGET, LEAN, true>(layout) : kernel_of<D, TARGET, LEAN, false>(layout);
}

template <int D, int TARGET>
cudaError_t launch(RopeArgs a, int sms, bool programmatic, cudaStream_t stream) {
  constexpr int G = 32 / (D / 16);
  const int H = a.Hq + (TARGET != kRopeRows ? 2 : 1) * a.Hk;
  const int rounds = (H + G - 1) / G;
  const bool norm = a.q_norm || a.k_norm;
  int layout = a.interleaved ? kInterleaved : a.rotary_dim == D ? kWhole : kPart;
  // few rows: their heads over more warps, as many as the GPU starts at once
  const int64_t want = (int64_t)sms * kWarps * ctas_of(TARGET, norm, layout, false);
  const int parts = (int)std::min<int64_t>(rounds, std::max<int64_t>(1, want / a.n_rows));
  a.part_heads = (rounds + parts - 1) / parts * G;
  a.parts = (H + a.part_heads - 1) / a.part_heads;
  if (TARGET == kRopeRows && !norm && layout != kWhole && parts == 1 && rounds >= kEitherRounds) layout = kEither;
  const int64_t tasks = (int64_t)a.n_rows * a.parts, grid = (tasks + kWarps - 1) / kWarps;
  const bool lean = TARGET == kRopePages && parts == 1 && rounds <= kLeanRounds;
  auto kern = lean ? kernel_of<D, TARGET, TARGET == kRopePages>(norm, layout) : kernel_of<D, TARGET, false>(norm, layout);
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), 0, stream, programmatic, a);
}

template <int TARGET>
cudaError_t launch_d(const RopeArgs& a, int head_dim, int sms, bool programmatic, cudaStream_t stream) {
  return head_dim == 128 ? launch<128, TARGET>(a, sms, programmatic, stream) : launch<64, TARGET>(a, sms, programmatic, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int head_dim, RopeTarget target, int sms, bool programmatic,
                        cudaStream_t stream) {
  return target == kRopeRows    ? launch_d<kRopeRows>(a, head_dim, sms, programmatic, stream)
         : target == kRopePages ? launch_d<kRopePages>(a, head_dim, sms, programmatic, stream)
                                : launch_d<kRopePagesQ4>(a, head_dim, sms, programmatic, stream);
}

}  // namespace daa
