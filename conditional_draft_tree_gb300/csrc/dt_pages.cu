// dt_pages.cu -- page tables and slot maps of the paged cache, built on the device from
// the requests' lengths.
//
// The free pages and, behind them, the pages that this call's requests give back form one
// sequence V; what is taken comes from V's end, what is left of V is the new stack. Counted
// from V's end, the w-th page that is given back is the w-th in the order of requests and of
// their tables, so the g-th page taken is the g-th one given back, or, behind those, the g-th from
// the end of the old stack. Hence no entry of the stack is both read and written, every table entry
// that is given back is read and cleared by the one thread that places its page, and the
// whole call is one parallel pass.
#include <algorithm>
#include <cstdint>

#include "dt_cache.cuh"
#include "dt_internal.h"

namespace dt {

int check_cache(const dt_cache *c);

namespace {

constexpr int kThreads = 512;
constexpr int kMaxBatch = 16384;

struct ReserveArgs {
  CacheView c;
  int32_t *table;
  int32_t *held, *free_pages, *state;
  const int32_t *lengths;
  int batch;
};

// request whose part of the running sums `s` (s[0] = 0) holds place `at`
__device__ __forceinline__ int owner(const int32_t *s, int batch, int at) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int saturated(int64_t v) {
  return static_cast<int>(min(v, int64_t{0x7fffffff}));
}

struct Wants {
  int held, need;        // need = held: nothing
  bool over;             // more than its table has room for
};
__device__ __forceinline__ Wants wants(const ReserveArgs &a, int b) {
  Wants w;
  w.held = min(max(a.held[b], 0), a.c.width);
  const int64_t rows = max(a.lengths[b], 0), page = int64_t{1} << a.c.shift;
  const int64_t need = (rows + page - 1) >> a.c.shift;
  w.over = need > a.c.width;
  w.need = w.over ? w.held : static_cast<int>(need);
  return w;
}

// Every block adds up the requests' wants for itself (the running sums of pages taken and
// given back in shared memory) and places its share of the pages; the last block to finish writes
// what the others read. Bound by latency: three dependent reads and two scans, a call
// 2.9 us for 32 requests and 5.6 for 512 with pages of 16 rows (means of three calls).
__global__ void __launch_bounds__(kThreads) cache_reserve_kernel(const __grid_constant__ ReserveArgs a) {
  extern __shared__ int32_t s_sums[];                 // [batch + 1] taken, [batch + 1] given back
  __shared__ int64_t s_warp[2][kThreads / 32];
  __shared__ int s_last;
  int32_t *s_take = s_sums, *s_back = s_sums + a.batch + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  int64_t take = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    const Wants w = wants(a, b);
    take += max(w.need - w.held, 0);
    back += max(w.held - w.need, 0);
  }
  int64_t upto[2] = {take, back};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = static_cast<int64_t>(shfl64_up(static_cast<uint64_t>(upto[k]), d));
      if (lane >= d) upto[k] += o;
    }
    if (lane == 31) s_warp[k][warp] = upto[k];
  }
  __syncthreads();
  int64_t all[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) upto[k] += s_warp[k][w];
      all[k] += s_warp[k][w];
    }
  const int64_t count = min(max(a.state[0], 0), a.c.pages);
  const int64_t there = count + all[1];               // pages of V
  take = upto[0] - take;
  back = upto[1] - back;
  for (int b = b0; b < b1; ++b) {
    const Wants w = wants(a, b);
    s_take[b] = saturated(take);
    s_back[b] = saturated(back);
    take += max(w.need - w.held, 0);
    back += max(w.held - w.need, 0);
  }
  if (tid == 0) {
    s_take[a.batch] = saturated(all[0]);
    s_back[a.batch] = saturated(all[1]);
    s_last = 1;
  }
  __syncthreads();
  // pages that can be taken: those of the requests before the first that does not fit
  int64_t taken = all[0];
  if (taken > there) {
    const int first = owner(s_take, a.batch + 1, saturated(there));    // the last sum <= there
    taken = s_take[first];
  }
  // the w-th page that is given back; its table entry is cleared
  auto given = [&](int64_t w) {
    const int b = owner(s_back, a.batch, static_cast<int>(w));
    const Wants k = wants(a, b);
    int32_t *entry = a.table + static_cast<int64_t>(b) * a.c.width + k.need + (w - s_back[b]);
    const int page = *entry;
    *entry = -1;
    if (page < 0 || page >= a.c.pages) cache_fault(a.c, b);
    return page;
  };
  const int64_t kept = max(all[1] - taken, int64_t{0});      // given back and not taken again
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + tid; g < taken + kept; g += step) {
    if (g < taken) {
      const int page = g < all[1] ? given(g) : a.free_pages[there - 1 - g];
      const int b = owner(s_take, a.batch, static_cast<int>(g));
      const Wants k = wants(a, b);
      a.table[static_cast<int64_t>(b) * a.c.width + k.held + (g - s_take[b])] = page;
    } else {
      const int64_t w = g, at = there - 1 - w;               // its place in V
      const int page = given(w);
      if (at < a.c.pages) a.free_pages[at] = page;
    }
  }
  if (gridDim.x > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      s_last = atomicAdd(&a.state[1], 1) == static_cast<int>(gridDim.x) - 1;
      if (s_last) a.state[1] = 0;
    }
  }
  __syncthreads();
  if (!s_last) return;
  for (int b = b0; b < b1; ++b) {
    const Wants w = wants(a, b);
    if (w.over) cache_fault(a.c, b);
    if (w.need > w.held && s_take[b] + static_cast<int64_t>(w.need - w.held) > taken)
      a.c.status[b] = DT_ERR_NO_PAGES;
    else if (w.need != a.held[b])
      a.held[b] = w.need;
  }
  if (tid == 0) a.state[0] = static_cast<int>(min(there - taken, static_cast<int64_t>(a.c.pages)));
}

struct SlotArgs {
  CacheView c;
  const int32_t *first, *counts;
  int64_t *slots;
  int32_t *positions;
  int n, row_blocks;
};

// A thread a row; bound by latency (131080 rows 2.2 us).
__global__ void __launch_bounds__(256) cache_slots_kernel(const __grid_constant__ SlotArgs a) {
  const int b = blockIdx.x / a.row_blocks;
  const int i = static_cast<int>(blockIdx.x % a.row_blocks) * 256 + threadIdx.x;
  if (i >= a.n) return;
  const int count = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  int64_t slot = -1, at = -1;
  if (i < count) {
    at = static_cast<int64_t>(a.first[b]) + i;
    if (at >= 0 && (at >> a.c.shift) < a.c.width) {
      const int page = a.c.table[static_cast<int64_t>(b) * a.c.width + (at >> a.c.shift)];
      if (page >= 0 && page < a.c.pages)
        slot = (static_cast<int64_t>(page) << a.c.shift) + (at & ((1 << a.c.shift) - 1));
    }
    if (slot < 0) cache_fault(a.c, b);
  }
  const int64_t to = static_cast<int64_t>(b) * a.n + i;
  if (a.slots) a.slots[to] = slot;
  if (a.positions) a.positions[to] = static_cast<int32_t>(at);
}

bool aligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) == 0; }

}  // namespace

}  // namespace dt

extern "C" {

int dt_cache_reserve(const dt_cache *c, const dt_page_pool *pool, const int32_t *lengths,
                     void *stream) {
  if (dt::check_cache(c) || !pool || !pool->held || !pool->free_pages || !pool->state || !lengths ||
      !dt::aligned(pool->held, 4) || !dt::aligned(pool->free_pages, 4) || !dt::aligned(pool->state, 4) ||
      !dt::aligned(lengths, 4) || c->batch > dt::kMaxBatch)
    return DT_ERR_INVALID_ARG;
  int sms, smem;
  const int rc = dt::device_sm_count(&sms, &smem);
  if (rc) return rc;
  dt::ReserveArgs a;
  a.c = dt::cache_view(*c);
  a.table = const_cast<int32_t *>(c->table);
  a.held = pool->held; a.free_pages = pool->free_pages; a.state = pool->state;
  a.lengths = lengths;
  a.batch = c->batch;
  const size_t bytes = 2 * sizeof(int32_t) * (c->batch + 1);
  if (bytes > 40000) {
    const cudaError_t e = cudaFuncSetAttribute(dt::cache_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               2 * sizeof(int32_t) * (dt::kMaxBatch + 1));
    if (e != cudaSuccess) return DT_ERR_CUDA;
  }
  // a block for every 4096 entries that the tables have room for
  const int64_t room = static_cast<int64_t>(c->batch) * c->table_width;
  const int64_t grid = std::min<int64_t>(sms, (room + 4095) / 4096);
  dt::cache_reserve_kernel<<<static_cast<unsigned>(grid), dt::kThreads, bytes, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

int dt_cache_slots(const dt_cache *c, int n, const int32_t *first, const int32_t *counts,
                   int64_t *slots, int32_t *positions, void *stream) {
  if (dt::check_cache(c) || n < 1 || !first || !dt::aligned(first, 4) || !dt::aligned(counts, 4) ||
      (!slots && !positions) || !dt::aligned(slots, 8) || !dt::aligned(positions, 4))
    return DT_ERR_INVALID_ARG;
  const int64_t row_blocks = (static_cast<int64_t>(n) + 255) / 256, grid = row_blocks * c->batch;
  if (grid > 0x7fffffff) return DT_ERR_INVALID_ARG;
  dt::SlotArgs a;
  a.c = dt::cache_view(*c);
  a.first = first; a.counts = counts; a.slots = slots; a.positions = positions;
  a.n = n; a.row_blocks = static_cast<int>(row_blocks);
  dt::cache_slots_kernel<<<static_cast<unsigned>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // extern "C"
