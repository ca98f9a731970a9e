// dt_cache_attn.cuh -- attention over the paged cache: what its kernels share
// (arguments, the cut of the work over blocks, visibility, partial results).
//
// A unit of work is (request, key/value head, tile of BM query rows); the H / Hkv
// query heads that share a key/value head are stacked token by token, row
// r = i G + g, so K and V are read once for all of them. A unit's keys come in
// tiles of T. All units' tiles, in order, are cut into equal contiguous ranges,
// one a block: lengths differ from request to request and are known on the device
// only, and this keeps every block equally busy for any mix of them. A block writes
// a unit that it holds whole; a unit cut over blocks leaves partial results
// (unnormalised output, reference maximum, sum) in the workspace, at most two a
// block, and a second launch joins them in block order: the result does not
// depend on timing.
#pragma once

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
  int64_t slot;          // fp32 numbers of one part, a multiple of 4
  float scale_log2;      // scale times log2(e)
  int batch, n, H, G, row_tiles, grid, min_tiles;
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

// the units of one head before row tile `upto`
__device__ __forceinline__ int64_t tiles_before(const AttnArgs &a, const Request &r, int upto, int bm,
                                                int T) {
  int64_t w = 0;
  if (a.mask) {   // every live row tile sees the same keys
    const int live = min(upto, (r.count * a.G + bm - 1) / bm);
    w = upto - live;
    if (live) w += static_cast<int64_t>(live) * unit_tiles(a, r, 0, bm, T);
  } else {
    for (int rt = 0; rt < upto; ++rt) w += unit_tiles(a, r, rt, bm, T);
  }
  return w;
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

// The cut of all work tiles over the blocks. All threads of the block call plan() and
// find(); s_scan: THREADS / 32 + 2 numbers of shared memory.
template <int THREADS>
struct Schedule {
  int64_t total, chunk;
  int64_t one;           // this thread's request's tiles where one scan covers the batch
  int64_t upto;          // inclusive sum to it
  __device__ int64_t request_tiles(const AttnArgs &a, int b, int bm, int T) {
    return b < a.batch ? a.c.Hkv * tiles_before(a, request_of(a, b), a.row_tiles, bm, T) : 0;
  }
  // sizes of the whole launch
  __device__ void plan(const AttnArgs &a, int bm, int T, int64_t *s_scan) {
    total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
      one = request_tiles(a, b0 + threadIdx.x, bm, T);
      int64_t all;
      upto = block_scan<THREADS>(one, s_scan, &all);
      total += all;
    }
    chunk = (total + a.grid - 1) / a.grid;
    if (chunk < a.min_tiles) chunk = a.min_tiles;
  }
  // request that holds work tile `at`, and the first work tile of that request
  __device__ void find(const AttnArgs &a, int bm, int T, int64_t at, int64_t *s_scan, int *b,
                       int64_t *start) {
    int64_t *s_found = s_scan + THREADS / 32;
    if (a.batch <= THREADS) {
      if (at >= upto - one && at < upto) {
        s_found[0] = threadIdx.x;
        s_found[1] = upto - one;
      }
    } else {
      int64_t before = 0;
      for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
        const int64_t w = request_tiles(a, b0 + threadIdx.x, bm, T);
        int64_t all;
        const int64_t u = before + block_scan<THREADS>(w, s_scan, &all);
        if (at >= u - w && at < u) {
          s_found[0] = b0 + threadIdx.x;
          s_found[1] = u - w;
        }
        before += all;
      }
    }
    __syncthreads();
    *b = static_cast<int>(s_found[0]);
    *start = s_found[1];
    __syncthreads();
  }
  // first work tile of request b
  __device__ int64_t first_of(const AttnArgs &a, int bm, int T, int b, int64_t *s_scan) {
    int64_t *s_found = s_scan + THREADS / 32;
    if (a.batch <= THREADS) {
      if (threadIdx.x == b) s_found[0] = upto - one;
    } else {
      int64_t mine = 0, all;
      for (int x = threadIdx.x; x < b; x += THREADS) mine += request_tiles(a, x, bm, T);
      block_scan<THREADS>(mine, s_scan, &all);
      if (threadIdx.x == 0) s_found[0] = all;
    }
    __syncthreads();
    return s_found[0];
  }
};

// One unit's part that falls to a block: key tiles [t0, t1) of its `tiles`.
struct Segment {
  int b, hk, rt, t0, t1, tiles;
  Request rq;
  int64_t end;           // end of the unit's keys
};

// Walks the work tiles [at, stop) of a block, unit by unit.
struct Walk {
  int64_t at, stop, base;
  int b;
  __device__ bool next(const AttnArgs &a, int bm, int T, Segment *s) {
    if (at >= stop) return false;
    s->rq = request_of(a, b);
    int64_t per = tiles_before(a, s->rq, a.row_tiles, bm, T);
    while (at - base >= a.c.Hkv * per) {
      base += a.c.Hkv * per;
      s->rq = request_of(a, ++b);
      per = tiles_before(a, s->rq, a.row_tiles, bm, T);
    }
    s->b = b;
    // a 64-bit division only where it is needed
    s->hk = (at - base) >> 31 ? static_cast<int>((at - base) / per)
                              : static_cast<int>(static_cast<uint32_t>(at - base) / static_cast<uint32_t>(per));
    int64_t in_head = (at - base) - s->hk * per;
    s->rt = 0;
    s->tiles = unit_tiles(a, s->rq, 0, bm, T);
    while (in_head >= s->tiles) {
      in_head -= s->tiles;
      s->tiles = unit_tiles(a, s->rq, ++s->rt, bm, T);
    }
    s->t0 = static_cast<int>(in_head);
    s->t1 = static_cast<int>(min(static_cast<int64_t>(s->tiles), in_head + (stop - at)));
    s->end = tile_end(a, s->rq, s->rt, bm);
    at += s->t1 - s->t0;
    return true;
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

struct AttnPlan {        // resolved on the host from sizes alone
  int wide;              // dt_cache_wide.cu, else the mma.sync kernel
  int bm, dhp, row_tiles, grid;
  int odd, ring, raw;    // dt_cache_wide.cu: the last unit is half a one; operand, raw tiles
  size_t smem, bytes;
};
constexpr int kWideKeys = 128;         // keys of a tile of dt_cache_wide.cu
constexpr int kFewRows = 16;           // rows up to which the other kernel is used
bool wide_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p);
cudaError_t launch_wide(const dt_cache &c, const AttnArgs &a, int dtype, const AttnPlan &p,
                        cudaStream_t st);

}  // namespace dt
