// Step tables built on the GPU from request lengths, and pages given back.
//
// "Accelerating Sonar through speculation" (Perplexity), "Inference with
// speculative decoding": a step's KV page information is prepared on the host
// and copied to the GPU.  Here the page lists stay on the GPU (a block table row
// per slot, a stack of free pages) and one kernel turns the step's lengths into
// the CSR arrays that the append and the attention read:
//   kv_r = len_r + new_r, pages_r = ceil(kv_r / 16), take_r = max(0, pages_r - held_r)
//   qo_indptr, kv_indptr, T = exclusive sums of new, pages, take
//   page p of request r = block_table[slot_r][p]            (p < held_r)
//                         free[count - 1 - (T_r + p - held_r)]  otherwise
//   row i of request r: position len_r + i, slot_map = page * 16 + position % 16
// The free stack is read by position, so every CTA can work out any page alone
// and results do not depend on the order in which CTAs run.
//
// Bound: 8 bytes per page id and 12 per new row; a launch, three dependent loads and
// the scans for all but the longest batches.  Measured on GB300: 7.2 us for 64
// requests of 1k to 4k tokens, 10.7 for 512 of 4k to 128k (1.2 million pages; 1.4 us
// of bytes) as graph replays; with the ticket taken behind the page work and page ids
// stored one at a time 8.2 and 14.2.  Each CTA does the sums over the whole
// batch itself (a few KB from L2) instead of waiting for another kernel, then
// takes its share of the pages and rows; the CTA that is the last to have read the
// batch (a ticket) writes the lengths, page counts and free count back.  Nothing is changed when the step cannot be made (a bad or doubled
// slot, lengths past a row, more pages or rows than the buffers hold or the pool
// has): the tables then describe an empty step and the error word says why.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace daa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kP = 16;
constexpr int kDevErrNoPages = 4;  // beside ptx.cuh's codes: a step needs more pages than are free

// Shared memory: exclusive sums [batch + 1] each, then per request slot, pages
// held, cached length; the scan's warp sums; the bitmap of the slots seen.
struct Layout {
  int batch, words;
  __host__ __device__ constexpr size_t bytes() const {
    return 8 * (size_t)(3 * kWarps) + 4 * ((size_t)6 * batch + 3 + words);
  }
};

constexpr size_t kMaxSmem = Layout{DAA_STEP_MAX_BATCH, DAA_STEP_MAX_SLOTS / 32}.bytes();

struct Smem {
  long long* warp_sums;  // [3][kWarps]
  int *kp, *qo, *tp, *slot, *held, *len;
  uint32_t* seen;
  __device__ Smem(uint8_t* base, const Layout& l) {
    warp_sums = reinterpret_cast<long long*>(base);
    kp = reinterpret_cast<int*>(warp_sums + 3 * kWarps);
    qo = kp + l.batch + 1;
    tp = qo + l.batch + 1;
    slot = tp + l.batch + 1;
    held = slot + l.batch;
    len = held + l.batch;
    seen = reinterpret_cast<uint32_t*>(len + l.batch);
  }
};

// W: 64-bit sums, for batches whose longest possible step passes 32 bits.
template <bool W>
struct Sums {
  using T = typename std::conditional<W, long long, int>::type;
  T pages, rows, take;
};

// Inclusive sums over the block's threads of three values at once; `total`
// gets the block's sums.
template <bool W>
__device__ __forceinline__ Sums<W> block_scan(Sums<W> v, long long* sums, Sums<W>& total) {
  using T = typename Sums<W>::T;
  T* ws = reinterpret_cast<T*>(sums);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const T a = __shfl_up_sync(0xffffffffu, v.pages, m);
    const T b = __shfl_up_sync(0xffffffffu, v.rows, m);
    const T c = __shfl_up_sync(0xffffffffu, v.take, m);
    if (lane >= m) {
      v.pages += a;
      v.rows += b;
      v.take += c;
    }
  }
  if (lane == 31) {
    ws[warp] = v.pages;
    ws[kWarps + warp] = v.rows;
    ws[2 * kWarps + warp] = v.take;
  }
  __syncthreads();
  total = Sums<W>{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const T a = ws[w], b = ws[kWarps + w], c = ws[2 * kWarps + w];
    if (w < warp) {
      v.pages += a;
      v.rows += b;
      v.take += c;
    }
    total.pages += a;
    total.rows += b;
    total.take += c;
  }
  __syncthreads();
  return v;
}

// Index of the entry of the exclusive sums s[0 .. n] that holds item i < s[n]:
// the largest r with s[r] <= i (never an empty one).
__device__ __forceinline__ int find_owner(const int* s, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Reads the batch and leaves its sums in shared memory.  RELEASE: the pages of a
// slot are those it holds, and there are no rows.  Returns the error code that
// every CTA works out alike (0: none).
template <bool RELEASE, bool W>
__device__ int read_batch(const StepTableArgs& a, const Smem& s, const Layout& l, int& free_count) {
  free_count = a.counters[0];
  for (int i = threadIdx.x; i < l.words; i += kThreads) s.seen[i] = 0;
  __syncthreads();
  Sums<W> sum{0, 0, 0};
  int bad = 0;
  for (int base = 0; base < a.batch; base += kThreads) {
    const int i = base + threadIdx.x;
    Sums<W> v{0, 0, 0};
    int slot = -1, held = 0, len = 0;
    if (i < a.batch) {
      slot = ld_word(a.slots + i);
      const int n = RELEASE ? 0 : ld_word(a.new_len + i);
      if (slot < 0 || slot >= a.num_slots || n < 0) {
        bad = 1;
        slot = 0;
      } else {
        const uint32_t bit = 1u << (slot & 31);
        bad |= (atomicOr(&s.seen[slot >> 5], bit) & bit) != 0;
        // plain loads: the last CTA of this kernel writes these
        held = a.held[slot];
        len = RELEASE ? 0 : a.seq_len[slot];
        const long long kv = (long long)len + n;
        if (held < 0 || held > a.max_pages || len < 0 || kv > (long long)a.max_pages * kP) {
          bad = 1;
        } else {
          const int pages = RELEASE ? held : (int)((kv + kP - 1) / kP);
          v.pages = pages;
          v.rows = n;
          v.take = RELEASE ? 0 : max(0, pages - held);
        }
      }
    }
    Sums<W> total;
    const Sums<W> inc = block_scan<W>(v, s.warp_sums, total);
    if (i < a.batch) {
      s.kp[i] = (int)(sum.pages + inc.pages - v.pages);
      s.qo[i] = (int)(sum.rows + inc.rows - v.rows);
      s.tp[i] = (int)(sum.take + inc.take - v.take);
      s.slot[i] = slot;
      s.held[i] = held;
      s.len[i] = len;
    }
    sum.pages += total.pages;
    sum.rows += total.rows;
    sum.take += total.take;
  }
  if (threadIdx.x == 0) {
    s.kp[a.batch] = (int)sum.pages;
    s.qo[a.batch] = (int)sum.rows;
    s.tp[a.batch] = (int)sum.take;
  }
  bad |= free_count < 0 || free_count > a.num_pages;
  if (__syncthreads_or(bad)) return kDevErrShape;
  if (RELEASE) return sum.pages > a.num_pages - free_count ? kDevErrShape : 0;
  if (sum.pages > a.page_capacity || sum.rows > a.row_capacity) return kDevErrShape;
  return sum.take > free_count ? kDevErrNoPages : 0;
}

// Thread 0, once the CTA has read all it needs of the lengths and counts (each
// value is used before read_batch's last barrier): its number among the CTAs.  The
// answer is asked for at the end only, so the atomic runs beside the page work.
__device__ __forceinline__ int take_ticket(int* ticket) {
  if (threadIdx.x != 0 || gridDim.x == 1) return 0;
  __threadfence();
  return atomicAdd(ticket, 1);
}

// True in every thread of the CTA whose ticket is the last: no CTA reads the lengths
// and counts any more.
__device__ __forceinline__ bool is_last(int ticket) {
  __shared__ int s_last;
  if (threadIdx.x == 0) {
    s_last = ticket == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  return s_last != 0;
}

template <bool W>
__global__ void __launch_bounds__(kThreads) step_table_kernel(const StepTableArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Layout l{a.batch, (a.num_slots + 31) / 32};
  const Smem s(smem, l);
  grid_dep_launch();
  grid_dep_wait();
  int free_count;
  const int err = read_batch<false, W>(a, s, l, free_count);
  const int n = a.batch;
  if (err != 0) {
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) set_device_error(a.err, err);
      for (int i = threadIdx.x; i <= n; i += kThreads) {
        a.qo_indptr[i] = 0;
        a.kv_indptr[i] = 0;
        if (i < n) a.last_page_len[i] = 0;
      }
    }
    return;
  }
  const int ticket = take_ticket(a.counters + 1);
  auto fresh_page = [&](int r, int p) {
    return ld_word(a.free_pages + (free_count - 1 - (s.tp[r] + p - s.held[r])));
  };
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= n; i += kThreads) {
      a.qo_indptr[i] = s.qo[i];
      a.kv_indptr[i] = s.kp[i];
      if (i < n) {
        const int pages = s.kp[i + 1] - s.kp[i];
        const int kv = s.len[i] + (s.qo[i + 1] - s.qo[i]);
        a.last_page_len[i] = pages > 0 ? kv - (pages - 1) * kP : 0;
      }
    }
  }
  // page ids, four consecutive ones per thread (one search; a warp taking 128 in a
  // row, lane by lane, measured slower: 18 us and 14 for 1.2 million pages); new
  // pages also enter their row of the block table
  const int n_pages = s.kp[n], n_rows = s.qo[n];
  const int stride = (int)gridDim.x * kThreads;
  const bool wide_store = reinterpret_cast<uintptr_t>(a.page_indices) % 16 == 0;
  for (int64_t p0 = 4ll * (blockIdx.x * kThreads + threadIdx.x); p0 < n_pages; p0 += 4ll * stride) {
    int r = find_owner(s.kp, n, (int)p0);
    int id[4];
    const int p = (int)p0 - s.kp[r];
    if (p0 + 4 <= s.kp[r + 1] && p + 4 <= s.held[r]) {  // one request's, all held
      const int* row = a.block_table + (int64_t)s.slot[r] * a.max_pages + p;
#pragma unroll
      for (int u = 0; u < 4; ++u) id[u] = row[u];
    } else {
      int row_r[4], row_p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = p0 + u;
        row_r[u] = -1;
        id[u] = 0;
        if (i < n_pages) {
          while (i >= s.kp[r + 1]) ++r;
          row_p[u] = (int)i - s.kp[r];
          const bool old = row_p[u] < s.held[r];
          id[u] = old ? a.block_table[(int64_t)s.slot[r] * a.max_pages + row_p[u]] : fresh_page(r, row_p[u]);
          row_r[u] = old ? -1 : r;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (row_r[u] >= 0) a.block_table[(int64_t)s.slot[row_r[u]] * a.max_pages + row_p[u]] = id[u];
    }
    if (wide_store && p0 + 4 <= n_pages) {
      *reinterpret_cast<int4*>(a.page_indices + p0) = make_int4(id[0], id[1], id[2], id[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p0 + u < n_pages) a.page_indices[p0 + u] = id[u];
    }
  }
  if (a.slot_map || a.positions) {
    for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < n_rows; i += stride) {
      const int r = find_owner(s.qo, n, (int)i);
      const int pos = s.len[r] + ((int)i - s.qo[r]);
      if (a.positions) a.positions[i] = pos;
      if (a.slot_map) {
        const int p = pos / kP;
        const int id = p < s.held[r] ? a.block_table[(int64_t)s.slot[r] * a.max_pages + p] : fresh_page(r, p);
        a.slot_map[i] = (int64_t)id * kP + pos % kP;
      }
    }
  }
  if (!is_last(ticket)) return;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int pages = s.kp[i + 1] - s.kp[i];
    if (pages > s.held[i]) a.held[s.slot[i]] = pages;
    if (a.advance) a.seq_len[s.slot[i]] = s.len[i] + (s.qo[i + 1] - s.qo[i]);
  }
  if (threadIdx.x == 0) {
    a.counters[0] = free_count - s.tp[n];
    a.counters[1] = 0;
  }
}

// The pages of the batch's slots go back on the stack in the reverse of the
// order in which a step would take them, so releasing what was just taken
// restores the stack.
template <bool W>
__global__ void __launch_bounds__(kThreads) release_pages_kernel(const StepTableArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Layout l{a.batch, (a.num_slots + 31) / 32};
  const Smem s(smem, l);
  grid_dep_launch();
  grid_dep_wait();
  int free_count;
  const int err = read_batch<true, W>(a, s, l, free_count);
  if (err != 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_device_error(a.err, err);
    return;
  }
  const int ticket = take_ticket(a.counters + 1);
  const int n = a.batch, n_pages = s.kp[n];
  const int stride = (int)gridDim.x * kThreads;
  for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < n_pages; i += stride) {
    const int r = find_owner(s.kp, n, (int)i);
    a.free_pages[free_count + n_pages - 1 - i] =
        a.block_table[(int64_t)s.slot[r] * a.max_pages + ((int)i - s.kp[r])];
  }
  if (!is_last(ticket)) return;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    a.held[s.slot[i]] = 0;
    a.seq_len[s.slot[i]] = 0;
  }
  if (threadIdx.x == 0) {
    a.counters[0] = free_count + n_pages;
    a.counters[1] = 0;
  }
}

}  // namespace

size_t step_table_smem(int batch, int num_slots) { return Layout{batch, (num_slots + 31) / 32}.bytes(); }

cudaError_t launch_step_table(const StepTableArgs& a, bool release, int sms, bool programmatic,
                              cudaStream_t stream) {
  const size_t smem = step_table_smem(a.batch, a.num_slots);
  // sums of pages and of tokens: at most max_pages * 16 a request
  const bool wide = (int64_t)a.batch * a.max_pages * kP > INT32_MAX;
  auto kern = release ? (wide ? release_pages_kernel<true> : release_pages_kernel<false>)
                      : (wide ? step_table_kernel<true> : step_table_kernel<false>);
  // The kernel's limit, always the same one: with each call's own size, a smaller step
  // prepared in another thread could lower it between this call and the launch.
  static_assert(kMaxSmem <= 227 * 1024, "a step's shared memory");
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  // the host knows only upper bounds of the work: a CTA per 2048 pages or 512
  // rows of the buffers (what a release returns is at most the pool)
  const int64_t pages = release ? a.num_pages : a.page_capacity;
  const int64_t rows = !release && (a.slot_map || a.positions) ? a.row_capacity : 0;
  const int64_t want = std::max<int64_t>((pages + 4 * kThreads - 1) / (4 * kThreads),
                                         (rows + kThreads - 1) / kThreads);
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(want, 1), sms);
  return launch_kernel(kern, dim3(grid), dim3(kThreads), smem, stream, programmatic, a);
}

}  // namespace daa
