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
  float *part;           // [grid][2][BM][DH + 2]
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

// end of the keys that row tile rt may see (a tile of dead rows sees none)
template <int BM>
__device__ __forceinline__ int64_t tile_end(const AttnArgs &a, const Request &r, int rt) {
  const int i0 = rt * BM / a.G;
  if (i0 >= r.count) return 0;
  if (a.mask) return r.pre + r.count;
  return r.pre + min(r.count, (rt * BM + BM - 1) / a.G + 1);
}

// key tiles of the unit; at least one, whose block writes the unit's rows
template <int BM, int T>
__device__ __forceinline__ int unit_tiles(const AttnArgs &a, const Request &r, int rt) {
  const int64_t e = tile_end<BM>(a, r, rt);
  return e > T ? static_cast<int>((e + T - 1) / T) : 1;
}

template <int BM, int T>
__device__ __forceinline__ int64_t head_tiles(const AttnArgs &a, const Request &r) {
  int64_t w = 0;
  if (a.mask) {   // every live row tile sees the same keys
    const int live = min(a.row_tiles, (r.count * a.G + BM - 1) / BM);
    w = a.row_tiles - live;
    if (live) w += static_cast<int64_t>(live) * unit_tiles<BM, T>(a, r, 0);
  } else {
    for (int rt = 0; rt < a.row_tiles; ++rt) w += unit_tiles<BM, T>(a, r, rt);
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

// The block's place in the work. All threads of the block call both functions.
template <int BM, int T, int THREADS>
struct Schedule {
  int64_t total, chunk;
  int64_t one;           // this thread's request's tiles where one scan covers the batch
  int64_t upto;          // inclusive sum to it
  // sizes of the whole launch
  __device__ void plan(const AttnArgs &a, int64_t *s_warp) {
    total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
      const int b = b0 + threadIdx.x;
      one = b < a.batch ? a.c.Hkv * head_tiles<BM, T>(a, request_of(a, b)) : 0;
      int64_t all;
      upto = block_scan<THREADS>(one, s_warp, &all);
      total += all;
    }
    chunk = (total + a.grid - 1) / a.grid;
    if (chunk < a.min_tiles) chunk = a.min_tiles;
  }
  // request that holds work tile `at`, and the first work tile of that request
  __device__ void find(const AttnArgs &a, int64_t at, int64_t *s_warp, int64_t *s_found, int *b,
                       int64_t *start) {
    if (a.batch <= THREADS) {
      if (at >= upto - one && at < upto) {
        s_found[0] = threadIdx.x;
        s_found[1] = upto - one;
      }
    } else {
      int64_t before = 0;
      for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
        const int t = b0 + threadIdx.x;
        const int64_t w = t < a.batch ? a.c.Hkv * head_tiles<BM, T>(a, request_of(a, t)) : 0;
        int64_t all;
        const int64_t u = before + block_scan<THREADS>(w, s_warp, &all);
        if (at >= u - w && at < u) {
          s_found[0] = t;
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
  int wide;              // the tensor-core kernel for many rows
  int bm, dhp, row_tiles, grid;
  size_t bytes;
};
int attn_plan(const dt_cache &c, int H, int n, AttnPlan *p);

}  // namespace dt
