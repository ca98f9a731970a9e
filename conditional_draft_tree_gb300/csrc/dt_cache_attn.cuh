// dt_cache_attn.cuh -- attention over the paged cache: what its kernels share
// (arguments, the cut of the work over blocks, visibility, partial results).
//
// A unit of work is (request, key/value head, tile of BM query rows); the H / Hkv
// query heads that share a key/value head are stacked token by token, row
// r = i G + g, so K and V are read once for all of them. A unit's keys come in
// tiles of T. Units lie one after another on a line, each `lead` long (what it costs to
// begin and end one) and then `weight` for each of its key tiles; the line is cut into
// equal parts, one a block, and a block has the tiles that begin in its part. Lengths
// differ from request to request and are known on the device only, and this keeps every
// block about equally busy for any mix of them. A block writes a unit that it holds
// whole; a unit cut over blocks leaves partial results (unnormalised output, reference
// maximum, sum) in the workspace, at most two a block, and a second launch joins them in
// block order: the result does not depend on timing.
#pragma once

#include <atomic>
#include <cuda.h>

#include "dt_cache.cuh"

namespace dt {

struct AttnArgs {
  CacheView c;
  const char *q;
  char *out;
  int64_t qb, qh, qr, ob, oh, orow;   // strides in bytes
  const int32_t *prefix, *counts;
  const uint8_t *mask;
  float *part;           // [grid][2][2][slot]: [BM][DH] of O, [BM] maxima, [BM] sums, of a
                         // block's first or last unit, and of one of its two groups of
                         // warps where these share a unit's rows; behind it [grid][2][slot],
                         // which passes one group's part to the other
  int odd;               // the last row tile's units are shared so
  int64_t slot;          // fp32 numbers of one part, a multiple of 8
  float scale_log2;      // scale times log2(e)
  int batch, n, G, row_tiles, grid, min_tiles;
  int weight, last_weight, lead;      // of a key tile, of one of the last row tile, of a unit
  int4 *cut;             // [grid][2]: the unit that a block's part of the line begins within
};

struct Request {         // one request's sizes, clamped to its table
  int64_t pre;           // rows before the query rows
  int count;             // query rows
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, int b) {
  Request r;
  const int64_t cap = static_cast<int64_t>(a.c.width) << a.c.shift;
  r.pre = min(max(static_cast<int64_t>(a.prefix[b]), int64_t{0}), cap);
  r.count = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  return r;
}

// end of the keys that row tile rt (of bm rows) may see (a tile of dead rows sees none)
__device__ __forceinline__ int64_t tile_end(const AttnArgs &a, const Request &r, int rt, int bm) {
  const int i0 = rt * bm / a.G;
  if (i0 >= r.count) return 0;
  if (a.mask) return r.pre + r.count;
  return r.pre + min(r.count, (rt * bm + bm - 1) / a.G + 1);
}

// key tiles of the unit; at least one, whose block writes the unit's rows
__device__ __forceinline__ int unit_tiles(const AttnArgs &a, const Request &r, int rt, int bm, int T) {
  const int64_t e = tile_end(a, r, rt, bm);
  return e > T ? static_cast<int>((e + T - 1) / T) : 1;
}

__device__ __forceinline__ int tile_weight(const AttnArgs &a, int rt) {
  return rt == a.row_tiles - 1 ? a.last_weight : a.weight;
}

// length of the units of one head before row tile `upto`
__device__ __forceinline__ int64_t length_before(const AttnArgs &a, const Request &r, int upto, int bm,
                                                 int T) {
  int64_t len = static_cast<int64_t>(upto) * a.lead;
  if (a.mask) {   // every live row tile sees the same keys
    const int live = min(upto, (r.count * a.G + bm - 1) / bm);
    int64_t tiles = upto - live;
    if (live) tiles += static_cast<int64_t>(live) * unit_tiles(a, r, 0, bm, T);
    len += tiles * a.weight;
    if (upto == a.row_tiles)
      len -= static_cast<int64_t>(a.weight - a.last_weight) * unit_tiles(a, r, upto - 1, bm, T);
  } else {
    for (int rt = 0; rt < upto; ++rt)
      len += static_cast<int64_t>(unit_tiles(a, r, rt, bm, T)) * tile_weight(a, rt);
  }
  return len;
}

// inclusive sum over the block's threads (THREADS a multiple of 32); *total gets all
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *s_warp, int64_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = static_cast<int64_t>(shfl64_up(static_cast<uint64_t>(v), d));
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return v + before;
}

// The cut of the line over the blocks. All threads of the block call plan() and find();
// s_scan: THREADS / 32 + 2 numbers of shared memory. Up to 128 requests every warp adds up
// for itself, four requests a lane: a block begins a few microseconds earlier than by way of
// shared memory and barriers.
template <int THREADS>
struct Schedule {
  int64_t total, chunk;
  int64_t before;        // length before this lane's first request (up to 128 requests)
  int64_t len[4];        // its requests' lengths
  __device__ int64_t request_length(const AttnArgs &a, int b, int bm, int T) {
    return b < a.batch ? a.c.Hkv * length_before(a, request_of(a, b), a.row_tiles, bm, T) : 0;
  }
  // sizes of the whole launch
  __device__ void plan(const AttnArgs &a, int bm, int T, int64_t *s_scan) {
    const int lane = threadIdx.x & 31;
    if (a.batch <= 128) {
      int64_t sum = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        len[q] = request_length(a, 4 * lane + q, bm, T);
        sum += len[q];
      }
      int64_t upto = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = static_cast<int64_t>(shfl64_up(static_cast<uint64_t>(upto), d));
        if (lane >= d) upto += o;
      }
      before = upto - sum;
      total = static_cast<int64_t>(shfl64(static_cast<uint64_t>(upto), 31));
    } else {
      total = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
        int64_t all;
        block_scan<THREADS>(request_length(a, b0 + threadIdx.x, bm, T), s_scan, &all);
        total += all;
      }
    }
    const int64_t least = static_cast<int64_t>(a.min_tiles) * a.weight + a.lead;
    chunk = max((total + a.grid - 1) / a.grid, least);
  }
  // request that holds place `at` (below total), and the place where it begins
  __device__ void find(const AttnArgs &a, int bm, int T, int64_t at, int64_t *s_scan, int *b,
                       int64_t *start) {
    if (a.batch <= 128) {
      int mine = -1;
      int64_t from = before, place = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (at >= from && at < from + len[q]) {
          mine = q;
          place = from;
        }
        from += len[q];
      }
      const int src = __ffs(__ballot_sync(kFull, mine >= 0)) - 1;
      *b = 4 * src + __shfl_sync(kFull, mine, src);
      *start = static_cast<int64_t>(shfl64(static_cast<uint64_t>(place), src));
      return;
    }
    int64_t *s_found = s_scan + THREADS / 32, sum = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
      const int64_t w = request_length(a, b0 + threadIdx.x, bm, T);
      int64_t all;
      const int64_t u = sum + block_scan<THREADS>(w, s_scan, &all);
      if (at >= u - w && at < u) {
        s_found[0] = b0 + threadIdx.x;
        s_found[1] = u - w;
      }
      sum += all;
    }
    __syncthreads();
    *b = static_cast<int>(s_found[0]);
    *start = s_found[1];
    __syncthreads();
  }
};

// the head whose units, `per` long together, hold place `at` of a request's: a 64-bit
// division only where a number needs it (2^24 stacked rows over a million keys pass 2^32)
__host__ __device__ __forceinline__ int head_at(int64_t at, int64_t per) {
  return (at | per) >> 32 ? static_cast<int>(at / per)
                          : static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(per));
}

// One unit's part that falls to a block: key tiles [t0, t1) of its `tiles`.
struct Segment {
  int b, hk, rt, t0, t1, tiles;
  Request rq;
  int64_t end;           // end of the unit's keys
  int64_t place;         // of the unit's first tile
};

// Walks a block's part [at, stop) of the line, unit by unit.
struct Walk {
  int64_t at, stop, base;
  int b;
  __device__ bool next(const AttnArgs &a, int bm, int T, Segment *s) {
    while (at < stop) {
      s->rq = request_of(a, b);
      int64_t per = length_before(a, s->rq, a.row_tiles, bm, T);
      while (at - base >= a.c.Hkv * per) {
        base += a.c.Hkv * per;
        s->rq = request_of(a, ++b);
        per = length_before(a, s->rq, a.row_tiles, bm, T);
      }
      s->b = b;
      s->hk = head_at(at - base, per);
      int64_t unit = base + s->hk * per;
      int weight, len;
      for (s->rt = 0;; ++s->rt) {
        s->tiles = unit_tiles(a, s->rq, s->rt, bm, T);
        weight = tile_weight(a, s->rt);
        len = a.lead + s->tiles * weight;
        if (at < unit + len) break;
        unit += len;
      }
      // the tiles that begin in [at, stop)
      s->place = unit + a.lead;
      s->t0 = at <= s->place ? 0 : static_cast<int>((at - s->place + weight - 1) / weight);
      s->t1 = stop <= s->place ? 0
                               : static_cast<int>(min(static_cast<int64_t>(s->tiles),
                                                      (stop - s->place + weight - 1) / weight));
      s->end = tile_end(a, s->rq, s->rt, bm);
      at = unit + len;
      if (s->t0 < s->t1) return true;
    }
    return false;
  }
  // what the join has to know of the unit that the block's part begins within
  __device__ void note_cut(const AttnArgs &a, int64_t chunk, bool any, const Segment &s) {
    int4 unit = make_int4(-1, 0, 0, 0), blocks = make_int4(0, 0, 0, 0);
    if (any && s.t0 > 0) {
      unit = make_int4(s.b, s.hk, s.rt, 0);
      const int64_t last = s.place + static_cast<int64_t>(s.tiles - 1) * tile_weight(a, s.rt);
      blocks = make_int4(static_cast<int>(s.place / chunk), static_cast<int>(last / chunk), 0, 0);
    }
    a.cut[2 * blockIdx.x] = unit;
    a.cut[2 * blockIdx.x + 1] = blocks;
  }
};

// whether query row i sees cache row j (j < pre + count)
__device__ __forceinline__ bool sees(const AttnArgs &a, const Request &r, int b, int i, int64_t j) {
  if (j < r.pre) return true;
  const int t = static_cast<int>(j - r.pre);
  if (t >= r.count) return false;
  return a.mask ? a.mask[(static_cast<int64_t>(b) * a.n + i) * a.n + t] != 0 : t <= i;
}

// 2^x, 2 ulp, 0 for -inf
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A ring of places that steps are copied into and taken from in order: where the next step
// goes and comes from, and the parity of the phase that ends its copies. A warp that gives
// up a wait takes no further step, issues none, and waits for the ones in flight before it
// ends.
struct StepRing {
  uint32_t in, out, parity;
  __host__ __device__ void issued(uint32_t places) {
    if (++in == places) in = 0;
  }
  __host__ __device__ void taken(uint32_t places) {
    if (++out == places) {
      out = 0;
      parity ^= 1u;
    }
  }
  // steps in flight when step k of `steps` has not been taken
  __host__ __device__ static int flying(int k, int steps, int places) {
    return steps - k < places ? steps - k : places;
  }
};

struct AttnPlan {        // resolved on the host from sizes alone
  enum { kAny, kWide, kFew } kind;     // dt_cache_attn.cu, dt_cache_wide.cu, dt_cache_few.cu
  int bm, dhp, row_tiles, grid;
  int odd, ring, raw;    // dt_cache_wide.cu: the last unit is half a one; tiles, raw tiles in flight
  size_t smem, bytes;
};
// Opts a kernel into the device's whole shared memory, once a device (the call costs about
// as much as a launch; always the same size, so that calls on several threads agree).
template <auto Kernel>
cudaError_t allow_smem() {
  static std::atomic<bool> allowed[64] = {};
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && allowed[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes f;
  e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&f, Kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most - static_cast<int>(f.sharedSizeBytes));
  if (e == cudaSuccess && dev < 64) allowed[dev].store(true, std::memory_order_release);
  return e;
}

constexpr int kWideKeys = 128;         // keys of a tile of dt_cache_wide.cu
constexpr int kWideLead = 4;           // a unit's begin and end, in half key tiles of a full unit
constexpr int kFewRows = 16, kFewKeys = 64;   // rows of dt_cache_few.cu, keys of its tiles
bool wide_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p);
bool few_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p);
bool page_map(const dt_cache &c, const void *base, int box_rows, CUtensorMap *map);
cudaError_t launch_few(const dt_cache &c, const AttnArgs &a, int dtype, const AttnPlan &p,
                       cudaStream_t st);
cudaError_t launch_wide(const dt_cache &c, const AttnArgs &a, int dtype, const AttnPlan &p,
                        cudaStream_t st);

}  // namespace dt
