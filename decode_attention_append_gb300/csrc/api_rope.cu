// C ABI of the rotary positions and the appends that apply them: the rotation's
// record, argument checks and the launches.  Host code only.
#include <cmath>
#include <cstring>

#include "../../include/daa.h"
#include "launch.h"
#include "planner.h"

namespace daa {
namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <class F>
cudaError_t traced(int32_t id, cudaStream_t s, F&& f) {
  return traced_launch(id, s, [](void* ctx) { return (*static_cast<F*>(ctx))(); }, &f);
}

bool head_dim_ok(int32_t d) { return d == 64 || d == 128; }

// 2^64 times the turns a token of a pair that turns by f radians, modulo 2^64, rounded
// once.  1 / 2 pi in two parts, so that the product is good to 2^-100 of f.
uint64_t turns_of(double f) {
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double p = f * hi, rest = std::fma(f, hi, -p) + f * lo;
  // exact: below one turn either way, then half a turn, then whole units and less than one
  double t = std::ldexp(p - std::trunc(p), 64);
  if (t >= 0x1p63) t -= 0x1p64;
  if (t < -0x1p63) t += 0x1p64;
  const double whole = std::trunc(t);
  return (uint64_t)(int64_t)whole + (uint64_t)std::llrint((t - whole) + std::ldexp(rest, 64));
}

daa_status check_rope(const daa_rope* r) {
  if (!r) return DAA_ERR_INVALID_ARG;
  if (!head_dim_ok(r->head_dim) || r->rotary_dim < 16 || r->rotary_dim > r->head_dim || r->rotary_dim % 16 != 0)
    return DAA_ERR_UNSUPPORTED;
  if ((r->interleaved != 0 && r->interleaved != 1) || !(r->magnitude >= DAA_ROPE_MIN_MAGNITUDE) ||
      !(r->magnitude <= DAA_ROPE_MAX_MAGNITUDE))
    return DAA_ERR_INVALID_ARG;
  return DAA_OK;
}

// Elements from the first to one past the last, or -1 for strides that no tensor has.
constexpr int64_t kMaxStride = (int64_t)1 << 40;
int64_t span_of(const daa_rows& x, int64_t rows, int64_t heads, int64_t d) {
  const int64_t rs = rows > 1 ? x.row_stride : 0, hs = heads > 1 ? x.head_stride : 0;
  if (rs < 0 || hs < 0 || rs > kMaxStride || hs > kMaxStride) return -1;
  const __int128 n = (__int128)(rows - 1) * rs + (__int128)(heads - 1) * hs + d;
  return n > ((__int128)1 << 60) ? -1 : (int64_t)n;
}

daa_status check_rows(const daa_rows& x, int64_t rows, int64_t heads, int64_t d) {
  if (!x.data || span_of(x, rows, heads, d) < 0) return DAA_ERR_INVALID_ARG;
  if (!aligned(x.data, 16) || (rows > 1 && x.row_stride % 8 != 0) || (heads > 1 && x.head_stride % 8 != 0))
    return DAA_ERR_ALIGNMENT;
  return DAA_OK;
}

// Rows that are written: no two of them share an element, whichever of rows and heads
// is the outer one.
daa_status check_out(const daa_rows& x, int64_t rows, int64_t heads, int64_t d) {
  const daa_status st = check_rows(x, rows, heads, d);
  if (st != DAA_OK) return st;
  const int64_t rs = rows > 1 ? x.row_stride : kMaxStride * 4, hs = heads > 1 ? x.head_stride : kMaxStride * 4;
  const bool rows_outer = (heads == 1 || hs >= d) && rs >= span_of(x, 1, heads, d);
  const bool heads_outer = (rows == 1 || rs >= d) && hs >= span_of(x, rows, 1, d);
  return rows_outer || heads_outer ? DAA_OK : DAA_ERR_INVALID_ARG;
}

bool same_rows(const daa_rows& a, const daa_rows& b, int64_t rows, int64_t heads) {
  return a.data == b.data && (rows == 1 || a.row_stride == b.row_stride) &&
         (heads == 1 || a.head_stride == b.head_stride);
}

bool ranges_meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// Whether `a` and `b` may share an element.  Their ranges may meet where they are
// column blocks of one matrix (views of a projection's rows), or heads that lie
// between one another in the same order.
bool may_meet(const daa_rows& a, int64_t a_heads, const daa_rows& b, int64_t b_heads, int64_t rows, int64_t d) {
  if (!ranges_meet(a.data, 2 * span_of(a, rows, a_heads, d), b.data, 2 * span_of(b, rows, b_heads, d))) return false;
  auto apart = [](int64_t offset, int64_t period, int64_t a_len, int64_t b_len) {
    offset = (offset % period + period) % period;
    return offset >= a_len && offset + b_len <= period;
  };
  const int64_t offset =
      ((int64_t)reinterpret_cast<uintptr_t>(b.data) - (int64_t)reinterpret_cast<uintptr_t>(a.data)) / 2;
  const int64_t rs = a.row_stride, hs = a.head_stride;
  const bool same_rs = rows == 1 || (rs == b.row_stride && rs > 0);
  if (same_rs && rows > 1 && apart(offset, rs, span_of(a, 1, a_heads, d), span_of(b, 1, b_heads, d))) return false;
  const bool same_hs = hs > 0 && hs == b.head_stride && (rows == 1 || rs % hs == 0);
  return !(same_rs && same_hs && apart(offset, hs, d, d));
}

RopeRows rows_of(const daa_rows& x) {
  return RopeRows{static_cast<uint16_t*>(x.data), x.row_stride, x.head_stride};
}

// What every call checks, and the kernel's arguments but for the target.  heads: of q
// and of k (and v, of an append); q may be missing from an append.
daa_status common_args(const daa_rope* rope, const daa_rope_rows* io, int64_t q_heads, int64_t k_heads, bool append,
                       RopeArgs& a) {
  const daa_status st = check_rope(rope);
  if (st != DAA_OK) return st;
  if (!io || io->num_rows < 0) return DAA_ERR_INVALID_ARG;
  const int64_t n = io->num_rows, d = rope->head_dim;
  if ((io->q_norm || io->k_norm) && !(std::isfinite(io->eps) && io->eps >= 0.f)) return DAA_ERR_INVALID_ARG;
  if (!aligned(io->q_norm, 2) || !aligned(io->k_norm, 2) || !aligned(io->positions, 4)) return DAA_ERR_ALIGNMENT;
  if (n == 0) return DAA_OK;
  if (q_heads > DAA_ROPE_MAX_HEADS || k_heads > DAA_ROPE_MAX_HEADS ||
      n * (q_heads + (append ? 2 : 1) * k_heads) > DAA_ROPE_MAX_HEADS)
    return DAA_ERR_UNSUPPORTED;
  struct One {
    const daa_rows* x;
    int64_t heads;
  };
  One in[3], out[2];
  int n_in = 0, n_out = 0;
  if (q_heads > 0) {
    in[n_in++] = {&io->q, q_heads};
    out[n_out++] = {&io->q_out, q_heads};
  }
  if (k_heads > 0) {
    in[n_in++] = {&io->k, k_heads};
    if (append) in[n_in++] = {&io->v, k_heads};
    else out[n_out++] = {&io->k_out, k_heads};
  }
  for (int i = 0; i < n_in; ++i)
    if (daa_status e = check_rows(*in[i].x, n, in[i].heads, d); e != DAA_OK) return e;
  for (int i = 0; i < n_out; ++i)
    if (daa_status e = check_out(*out[i].x, n, out[i].heads, d); e != DAA_OK) return e;
  // an output is its own input (in place) or shares nothing with any of them
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i) {
      const bool its_own = i == o && (!append || o == 0);
      if (its_own && same_rows(*out[o].x, *in[i].x, n, in[i].heads)) continue;
      if (may_meet(*out[o].x, out[o].heads, *in[i].x, in[i].heads, n, d)) return DAA_ERR_INVALID_ARG;
    }
  }
  for (int o = 0; o < n_out; ++o) {
    auto covers = [&](const void* p, int64_t bytes) {
      return p && ranges_meet(out[o].x->data, 2 * span_of(*out[o].x, n, out[o].heads, d), p, bytes);
    };
    if (covers(io->positions, 4 * n) || covers(io->q_norm, 2 * d) || covers(io->k_norm, 2 * d))
      return DAA_ERR_INVALID_ARG;
  }
  if (n_out == 2 && may_meet(*out[0].x, out[0].heads, *out[1].x, out[1].heads, n, d)) return DAA_ERR_INVALID_ARG;
  std::memcpy(a.turns, rope->turns, sizeof(a.turns));
  a.rotary_dim = rope->rotary_dim;
  a.interleaved = rope->interleaved;
  a.magnitude = (float)rope->magnitude;
  a.magnitude_low = (float)(rope->magnitude - a.magnitude);
  a.n_rows = io->num_rows;
  a.Hq = (int)q_heads;
  a.Hk = (int)k_heads;
  if (q_heads > 0) {
    a.q = rows_of(io->q);
    a.q_out = rows_of(io->q_out);
    a.q_norm = static_cast<const uint16_t*>(io->q_norm);
  }
  if (k_heads > 0) {
    a.k = rows_of(io->k);
    if (append) a.v = rows_of(io->v);
    else a.k_out = rows_of(io->k_out);
    a.k_norm = static_cast<const uint16_t*>(io->k_norm);
  }
  a.eps = io->eps;
  a.positions = io->positions;
  a.err = device_error_word();
  return DAA_OK;
}

daa_status append(const daa_rope* rope, const daa_rope_rows* io, void* kv_pages, const int32_t* kv_exp,
                  const int32_t* append_indptr, const int32_t* page_indices, const int32_t* kv_indptr,
                  const int32_t* last_page_len, int32_t batch, const daa_dims& dims, RopeTarget target,
                  void* stream) {
  daa_status st = plan_check_dims(dims);
  if (st != DAA_OK) return st;
  if (batch < 0 || !io) return DAA_ERR_INVALID_ARG;
  if (rope && rope->head_dim != dims.head_dim && head_dim_ok(rope->head_dim)) return DAA_ERR_INVALID_ARG;
  const int64_t q_heads = io->q.data ? dims.num_qo_heads : 0;
  if (!io->q.data && io->q_out.data) return DAA_ERR_INVALID_ARG;
  RopeArgs a{};
  st = common_args(rope, io, q_heads, dims.num_kv_heads, true, a);
  if (st != DAA_OK) return st;
  if (io->num_rows == 0) return DAA_OK;
  if (batch == 0) return DAA_ERR_SHAPE;
  if (batch > DAA_ROPE_MAX_HEADS) return DAA_ERR_UNSUPPORTED;
  if (!kv_pages || !append_indptr || !page_indices || !kv_indptr || !last_page_len) return DAA_ERR_INVALID_ARG;
  if (!aligned(kv_pages, 16) || !aligned(kv_exp, 4) || !aligned(append_indptr, 4) || !aligned(page_indices, 4) ||
      !aligned(kv_indptr, 4) || !aligned(last_page_len, 4))
    return DAA_ERR_ALIGNMENT;
  const int64_t n = io->num_rows, d = dims.head_dim;
  const int64_t slice = target == kRopePagesQ4 ? 9 * d : 2 * d * kPlanPageSize;
  const int64_t pool_bytes = dims.num_pages * 2 * dims.num_kv_heads * slice;
  auto in_pool = [&](const daa_rows& x, int64_t heads) {
    return ranges_meet(x.data, 2 * span_of(x, n, heads, d), kv_pages, pool_bytes);
  };
  if (in_pool(io->k, dims.num_kv_heads) || in_pool(io->v, dims.num_kv_heads) ||
      (q_heads > 0 && (in_pool(io->q, q_heads) || in_pool(io->q_out, q_heads))))
    return DAA_ERR_INVALID_ARG;
  const struct {
    const void* p;
    int64_t bytes;
  } also_read[] = {{io->positions, 4 * n},          {io->q_norm, 2 * d},
                   {io->k_norm, 2 * d},             {kv_exp, 8 * (int64_t)dims.num_kv_heads},
                   {append_indptr, 4 * (int64_t)batch + 4}, {kv_indptr, 4 * (int64_t)batch + 4},
                   {last_page_len, 4 * (int64_t)batch},     {page_indices, 4}};  // of these, the number is on the device
  for (const auto& x : also_read)
    if (x.p && (ranges_meet(x.p, x.bytes, kv_pages, pool_bytes) ||
                (q_heads > 0 && ranges_meet(x.p, x.bytes, io->q_out.data, 2 * span_of(io->q_out, n, q_heads, d)))))
      return DAA_ERR_INVALID_ARG;
  a.pool = static_cast<uint8_t*>(kv_pages);
  a.kv_exp = kv_exp;
  a.append_indptr = append_indptr;
  a.page_indices = page_indices;
  a.kv_indptr = kv_indptr;
  a.last_page_len = last_page_len;
  a.batch = batch;
  a.num_pages = dims.num_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(target == kRopePagesQ4 ? kKernelAppendRopeQ4 : kKernelAppendRope, s, [&] {
           return launch_rope(a, dims.head_dim, target, device_sms(), !tracer_on(), s);
         }) == cudaSuccess
             ? DAA_OK
             : DAA_ERR_CUDA;
}

}  // namespace
}  // namespace daa

using namespace daa;

extern "C" {

daa_status daa_rope_init(daa_rope* rope, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
                         const double* radians, double magnitude) {
  if (!rope || !radians) return DAA_ERR_INVALID_ARG;
  daa_rope r{};
  r.head_dim = head_dim;
  r.rotary_dim = rotary_dim;
  r.interleaved = interleaved;
  r.magnitude = magnitude;
  const daa_status st = check_rope(&r);
  if (st != DAA_OK) return st;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (!(std::fabs(radians[i]) <= DAA_ROPE_MAX_RADIANS)) return DAA_ERR_INVALID_ARG;
    r.turns[i] = turns_of(radians[i]);
  }
  *rope = r;
  return DAA_OK;
}

daa_status daa_apply_rope(const daa_rope* rope, const daa_rope_rows* rows, int32_t num_q_heads, int32_t num_k_heads,
                          void* stream) {
  if (num_q_heads < 1 || num_k_heads < 0) return DAA_ERR_INVALID_ARG;
  RopeArgs a{};
  const daa_status st = common_args(rope, rows, num_q_heads, num_k_heads, false, a);
  if (st != DAA_OK) return st;
  if (rows->num_rows == 0) return DAA_OK;
  if (!rows->positions) return DAA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(kKernelRope, s, [&] {
           return launch_rope(a, rope->head_dim, kRopeRows, device_sms(), !tracer_on(), s);
         }) == cudaSuccess
             ? DAA_OK
             : DAA_ERR_CUDA;
}

daa_status daa_append_rope(const daa_rope* rope, const daa_rope_rows* rows, void* kv_pages,
                           const int32_t* append_indptr, const int32_t* page_indices, const int32_t* kv_indptr,
                           const int32_t* last_page_len, int32_t batch, daa_dims dims, void* stream) {
  return append(rope, rows, kv_pages, nullptr, append_indptr, page_indices, kv_indptr, last_page_len, batch, dims,
                kRopePages, stream);
}

daa_status daa_append_rope_q4(const daa_rope* rope, const daa_rope_rows* rows, void* kv_pages, const int32_t* kv_exp,
                              const int32_t* append_indptr, const int32_t* page_indices, const int32_t* kv_indptr,
                              const int32_t* last_page_len, int32_t batch, daa_dims dims, void* stream) {
  return append(rope, rows, kv_pages, kv_exp, append_indptr, page_indices, kv_indptr, last_page_len, batch, dims,
                kRopePagesQ4, stream);
}

}  // extern "C"
