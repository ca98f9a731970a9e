// dt_cache.cu -- rotary positions and the paged key/value cache: rows written
// (turned and quantised on the way), read back, and compacted onto an accepted
// path. All of it moves bytes: each value is read once and written once.
//
// Turning: y_a = m (x_a cos - x_b sin), y_b = m (x_a sin + x_b cos). The angle of pair
// i at position p is frac(p f_i / 2 pi) turns; f_i / 2 pi is a 64-bit fraction of
// a turn, and p times it modulo 2^64 is exact, where a product in fp32 would be off by
// p 2^-25 turns: what is left is the table's own error, below p 2^-55 (it is computed in
// double precision). The upper 32 bits, as a signed number in units of 2^-31 half turns,
// go to sincospif.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dt_cache.cuh"
#include "dt_internal.h"

namespace dt {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                     // lanes of one head row
constexpr int kGroups = kThreads / kLanes;    // head rows in flight per block
constexpr int kBlockTokens = 32;               // tokens of a block, at most
constexpr int kMaxHalf = 128;                 // pairs of a head, at most

struct View {            // one of up to three tensors of a launch
  const char *in;
  char *out;             // null: the cache
  int64_t ib, ih, ir, ob, oh, orow;   // strides in bytes
  int heads, turned, to_v;
};

struct RowArgs {
  View t[3];
  int nt, heads;         // tensors, and their heads together
  CacheView c;           // where a tensor goes to the cache
  const int32_t *first, *counts, *positions;
  const uint64_t *turns;
  float mag;
  int batch, n, dh, rot, interleaved, gradient;
  int tokens_block, heads_block, head_blocks;
};

__device__ __forceinline__ int clamped_count(const int32_t *counts, int b, int n) {
  return counts ? min(max(counts[b], 0), n) : n;
}

// N fp32 numbers of shared memory (on a boundary of 4 N bytes, or of 16)
template <int N>
__device__ __forceinline__ void load_f32(const float *p, float *x) {
  if (N % 4 == 0) {
#pragma unroll
    for (int e = 0; e < N / 4; ++e)
      *reinterpret_cast<float4 *>(x + 4 * e) = reinterpret_cast<const float4 *>(p)[e];
  } else {
    *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(p);
  }
}

// Head rows from the tensors t[] to views or to the cache. A block takes
// tokens_block tokens and heads_block heads of each: a token's angles and its place
// in the cache are found once for all of them. Eight lanes own a row; a lane holds
// chunks of VEC values two at a time, chunk c of the turned part with its partner
// (halves: the pair's other half, so a lane reads both before it writes either and a
// tensor can be turned in place; interleaved: any other chunk). 8-bit rows need the
// row's largest magnitude before the first code, so a lane keeps its values in
// registers. Bound by memory: a lane's next row is loaded (its first one before the
// angles are known) while the one before it is turned and written. Measured, dh 128: two
// prompts of 4099 tokens, 40 heads, fp16, 64 of 128 values turned, 33 us, 5.1 TB/s; 15009
// tokens of 16 heads to 8-bit rows 25 us, 3.7 TB/s (scaling and packing take half of the
// issue slots); 8 tokens 4.2 us.
template <int DT, bool QUANT, int VEC, int ITEMS>
__global__ void __launch_bounds__(kThreads) cache_rows_kernel(const __grid_constant__ RowArgs a) {
  extern __shared__ __align__(16) float s_cs[];      // [tokens_block][2][rot / 2]
  __shared__ int64_t s_row[kBlockTokens];            // of head 0; -1: no place, or no such token
  const int tid = threadIdx.x, lane = tid & (kLanes - 1), grp = tid / kLanes;
  const int64_t all = static_cast<int64_t>(a.batch) * a.n;
  const int64_t tk0 = static_cast<int64_t>(blockIdx.x / a.head_blocks) * a.tokens_block;
  const int h0 = static_cast<int>(blockIdx.x % a.head_blocks) * a.heads_block;
  const int nh = min(a.heads_block, a.heads - h0);
  const int ntok = static_cast<int>(min(static_cast<int64_t>(a.tokens_block), all - tk0));
  const int half = a.rot >> 1, chunks = a.dh / VEC;
  const int b0 = static_cast<int>(tk0 / a.n), i0 = static_cast<int>(tk0 - static_cast<int64_t>(b0) * a.n);
  // the request and the row of token tk0 + t
  auto place = [&](int t, int *b, int *i) {
    *b = b0;
    *i = i0 + t;
    while (*i >= a.n) {
      *i -= a.n;
      ++*b;
    }
  };
  // Row r of the block: its token, its tensor and head there, its chunks.
  struct Row {
    int t, k, h, pairs, rest2, items;
  };
  int rt = 0, rh = grp;                // token and head (of the block's) of the row to load
  while (rh >= nh) {
    rh -= nh;
    ++rt;
  }
  uint32_t w[ITEMS][2][VEC / 2];
  auto load = [&](Row *row) {
    row->t = rt;
    int h = h0 + rh, k = 0;
    while (k + 1 < a.nt && h >= a.t[k].heads) h -= a.t[k++].heads;
    const View &vw = a.t[k];
    row->k = k;
    row->h = h;
    row->pairs = vw.turned ? a.rot / (2 * VEC) : 0;           // chunk pairs of the turned part
    const int rest = chunks - 2 * row->pairs;
    row->rest2 = (rest + 1) >> 1;
    row->items = row->pairs + row->rest2;
    if (rt >= ntok) return;
    int b, i;
    place(rt, &b, &i);
    const char *in = vw.in + b * vw.ib + h * vw.ih + i * vw.ir;
    const bool read = vw.out || i < clamped_count(a.counts, b, a.n);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int m = lane + it * kLanes;
      const int c0 = m < row->pairs ? m : 2 * row->pairs + (m - row->pairs);
      const int c1 = m < row->pairs ? m + row->pairs : c0 + row->rest2;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int c = z ? c1 : c0;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) w[it][z][e] = 0u;
        if (read && m < row->items && c < chunks) {
          if (VEC == 8) *reinterpret_cast<uint4 *>(w[it][z]) = *reinterpret_cast<const uint4 *>(in + c * 16);
          else *reinterpret_cast<uint2 *>(w[it][z]) = *reinterpret_cast<const uint2 *>(in + c * 8);
        }
      }
    }
    rh += kGroups;
    while (rh >= nh) {
      rh -= nh;
      ++rt;
    }
  };
  Row next;
  load(&next);
  if (tid < ntok && a.c.table) {
    int b, i;
    place(tid, &b, &i);
    int64_t row = -1;
    if (i < clamped_count(a.counts, b, a.n)) {
      row = cache_row(a.c, b, static_cast<int64_t>(a.first[b]) + i, 0);
      if (row < 0) cache_fault(a.c, b);
    }
    s_row[tid] = row;
  }
  for (int u = tid; u < ntok * half; u += kThreads) {
    const int t = u / half, i = u - t * half;
    const int64_t p = a.positions[tk0 + t];
    const uint64_t frac = static_cast<uint64_t>(p) * a.turns[i];   // modulo one turn
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f, &s, &c);
    if (a.gradient) s = -s;
    s_cs[(2 * t) * half + i] = a.mag * c;
    s_cs[(2 * t + 1) * half + i] = a.mag * s;
  }
  __syncthreads();
  while (next.t < ntok) {
    const Row cur = next;
    const View &vw = a.t[cur.k];
    const int pairs = cur.pairs, rest2 = cur.rest2, items = cur.items;
    float x[ITEMS][2][VEC];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 f = Half16<DT>::unpack(w[it][z][e]);
          x[it][z][2 * e] = f.x;
          x[it][z][2 * e + 1] = f.y;
        }
    load(&next);
    char *out = vw.out;
    uint8_t *expo = nullptr;
    if (out) {
      int b, i;
      place(cur.t, &b, &i);
      out += b * vw.ob + cur.h * vw.oh + i * vw.orow;
    } else {
      if (s_row[cur.t] < 0) continue;
      const int64_t row = s_row[cur.t] + (static_cast<int64_t>(cur.h) << a.c.shift);
      out = static_cast<char *>(vw.to_v ? a.c.v : a.c.k) + row * a.dh * (QUANT ? 1 : 2);
      if (QUANT) expo = (vw.to_v ? a.c.v_exp : a.c.k_exp) + row;
    }
    const float *cs = s_cs + 2 * cur.t * half;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int m = lane + it * kLanes;
      if (m >= pairs) continue;
      if (!a.interleaved) {
        float co[VEC], si[VEC];
        load_f32<VEC>(cs + m * VEC, co);
        load_f32<VEC>(cs + half + m * VEC, si);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xa = x[it][0][e], xb = x[it][1][e];
          x[it][0][e] = xa * co[e] - xb * si[e];
          x[it][1][e] = xa * si[e] + xb * co[e];
        }
      } else {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float co[VEC / 2], si[VEC / 2];
          const int p = (z ? m + pairs : m) * (VEC / 2);
          load_f32<VEC / 2>(cs + p, co);
          load_f32<VEC / 2>(cs + half + p, si);
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) {
            const float xa = x[it][z][2 * e], xb = x[it][z][2 * e + 1];
            x[it][z][2 * e] = xa * co[e] - xb * si[e];
            x[it][z][2 * e + 1] = xa * si[e] + xb * co[e];
          }
        }
      }
    }
    const bool quant = QUANT && !vw.out;
    float scale = 1.0f;
    bool whole = true;
    if (quant) {
      uint32_t mx = 0;   // of magnitude bits: NaN > infinity > finite
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e)
          mx = max(mx, __float_as_uint(x[it][e / VEC][e % VEC]) & 0x7fffffffu);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1)
        mx = max(mx, __shfl_xor_sync(0xffu << (threadIdx.x & 24), mx, d));
      whole = mx < 0x7f800000u;
      const int e = row_exponent(__uint_as_float(mx));
      scale = exp2i(-e);
      if (e == 120) {               // 256 2^120 is no finite bf16 number
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
#pragma unroll
          for (int y = 0; y < 2 * VEC; ++y) {
            float &f = x[it][y / VEC][y % VEC];
            f = fminf(fmaxf(f, -240.0f * 0x1p120f), 240.0f * 0x1p120f);
          }
      }
      if (lane == 0) *expo = static_cast<uint8_t>(whole ? e + 127 : 255);
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int m = lane + it * kLanes;
      const int c0 = m < pairs ? m : 2 * pairs + (m - pairs);
      const int c1 = m < pairs ? m + pairs : c0 + rest2;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int c = z ? c1 : c0;
        if (m >= items || c >= chunks) continue;
        const float *f = x[it][z];
        if (quant) {
          uint32_t w[VEC / 4];
#pragma unroll
          for (int e = 0; e < VEC; e += 4) {
            const uint32_t y = e4m3_pack2(f[e] * scale, f[e + 1] * scale) |
                               (e4m3_pack2(f[e + 2] * scale, f[e + 3] * scale) << 16);
            w[e / 4] = whole ? y : 0x7f7f7f7fu;
          }
          if (VEC == 8) *reinterpret_cast<uint2 *>(out + c * 8) = make_uint2(w[0], w[VEC / 4 - 1]);
          else *reinterpret_cast<uint32_t *>(out + c * 4) = w[0];
        } else {
          uint32_t w[VEC / 2];
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) w[e] = Half16<DT>::pack(f[2 * e], f[2 * e + 1]);
          if (VEC == 8) *reinterpret_cast<uint4 *>(out + c * 16) = *reinterpret_cast<uint4 *>(w);
          else *reinterpret_cast<uint2 *>(out + c * 8) = *reinterpret_cast<uint2 *>(w);
        }
      }
    }
  }
}

struct ReadArgs {
  CacheView c;
  const int32_t *first, *counts;
  char *k, *v;
  int64_t kb, kh, kr, vb, vh, vr;    // strides in bytes
  int n, row_blocks;
};

constexpr int kReadRows = 64;        // rows of a block, of one head

// Rows of the cache to dense views. A block takes 64 rows of one (request, head):
// their places once into shared memory, then 8 values a lane, four rows of K and
// of V in flight a lane. Bound by memory: 8 requests of 9000 to 16385 rows, 8 heads, dh 128,
// from 8-bit rows to bf16 119 us, 6.3 TB/s.
template <int DT, bool QUANT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadArgs a) {
  __shared__ int64_t s_row[kReadRows];
  const int tid = threadIdx.x, dh = a.c.dh, chunks = dh >> 3;
  const int bh = blockIdx.x / a.row_blocks;
  const int i0 = static_cast<int>(blockIdx.x % a.row_blocks) * kReadRows;
  const int b = bh / a.c.Hkv, hk = bh - b * a.c.Hkv;
  const int count = clamped_count(a.counts, b, a.n), rows = min(kReadRows, a.n - i0);
  if (tid < rows) {
    int64_t row = -1;
    if (i0 + tid < count) {
      row = cache_row(a.c, b, static_cast<int64_t>(a.first[b]) + i0 + tid, hk);
      if (row < 0) cache_fault(a.c, b);
    }
    s_row[tid] = row;
  }
  __syncthreads();
  // lanes a row: the power of two at or above its 8-value chunks
  const int lsh = chunks <= 8 ? 3 : chunks <= 16 ? 4 : 5;
  const int c = tid & ((1 << lsh) - 1), step = kThreads >> lsh;
  if (c >= chunks) return;
  constexpr int kUnroll = 4;
  for (int r0 = tid >> lsh; r0 < rows; r0 += kUnroll * step) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const char *pool = static_cast<const char *>(which ? a.c.v : a.c.k);
      const uint8_t *expo = which ? a.c.v_exp : a.c.k_exp;
      char *out = which ? a.v + b * a.vb + hk * a.vh : a.k + b * a.kb + hk * a.kh;
      const int64_t stride = which ? a.vr : a.kr;
      uint4 w[kUnroll];
      float scale[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * step;
        const int64_t row = r < rows ? s_row[r] : -1;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        scale[u] = 0.0f;
        if (row >= 0) {
          if (QUANT) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(pool + row * dh) + c);
            w[u].x = q.x;
            w[u].y = q.y;
            scale[u] = row_scale(expo[row]);
          } else {
            w[u] = __ldcs(reinterpret_cast<const uint4 *>(pool + row * dh * 2) + c);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * step;
        if (r >= rows) break;
        uint4 o = w[u];
        if (QUANT) {
          o.x = e4m3_to16<DT>(w[u].x & 0xffffu, scale[u]);
          o.y = e4m3_to16<DT>(w[u].x >> 16, scale[u]);
          o.z = e4m3_to16<DT>(w[u].y & 0xffffu, scale[u]);
          o.w = e4m3_to16<DT>(w[u].y >> 16, scale[u]);
        }
        __stcs(reinterpret_cast<uint4 *>(out + (i0 + r) * stride) + c, o);
      }
    }
  }
}

struct CommitArgs {
  CacheView c;
  const int32_t *first, *path, *lengths;
  int width, n, row_bytes;
};

constexpr int kMaxPath = DT_MAX_D + 1;

// One block per (request, head, K or V): all rows of the path into shared memory,
// a barrier, then to their new places. Paths rise, but nothing relies on it.
// Bound by latency: 16 KB or less a block; 32 paths of up to 17 rows 4.4 us, 128 16 us with
// the rows read back.
__global__ void __launch_bounds__(kThreads) cache_commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int64_t s_from[kMaxPath], s_to[kMaxPath];
  __shared__ uint8_t s_exp[kMaxPath];
  extern __shared__ __align__(16) unsigned char s_rows[];   // [width][row_bytes]
  const int tid = threadIdx.x;
  const int which = blockIdx.x & 1, bh = blockIdx.x >> 1;
  const int b = bh / a.c.Hkv, hk = bh - b * a.c.Hkv;
  const int len = min(max(a.lengths[b], 0), a.width);
  char *pool = static_cast<char *>(which ? a.c.v : a.c.k);
  uint8_t *expo = which ? a.c.v_exp : a.c.k_exp;
  if (tid < len) {
    const int p = a.path[static_cast<int64_t>(b) * a.width + tid];
    const int64_t first = a.first[b];
    int64_t from = -1, to = -1;
    if (p >= 0 && p < a.n && first >= 0) {
      from = cache_row(a.c, b, first + p, hk);
      to = cache_row(a.c, b, first + tid, hk);
    }
    const bool fine = from >= 0 && to >= 0;
    if (!fine) cache_fault(a.c, b);
    s_from[tid] = fine && from != to ? from : -1;
    s_to[tid] = to;
    if (expo && fine) s_exp[tid] = expo[from];
  }
  __syncthreads();
  const int units = a.row_bytes >> 4;
  for (int u = tid; u < len * units; u += kThreads) {
    const int j = u / units, c = u - j * units;
    if (s_from[j] >= 0)
      reinterpret_cast<uint4 *>(s_rows)[u] =
          reinterpret_cast<const uint4 *>(pool + s_from[j] * a.row_bytes)[c];
  }
  __syncthreads();
  for (int u = tid; u < len * units; u += kThreads) {
    const int j = u / units, c = u - j * units;
    if (s_from[j] >= 0)
      reinterpret_cast<uint4 *>(pool + s_to[j] * a.row_bytes)[c] =
          reinterpret_cast<const uint4 *>(s_rows)[u];
  }
  if (expo && tid < len && s_from[tid] >= 0) expo[s_to[tid]] = s_exp[tid];
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <int DT, bool QUANT>
cudaError_t launch_rows(const RowArgs &a, cudaStream_t st) {
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.n;
  const int64_t grid = (tokens + a.tokens_block - 1) / a.tokens_block * a.head_blocks;
  const size_t smem = sizeof(float) * a.tokens_block * a.rot;
  // 8-value chunks where a turned half is made of them, else 4 (rot = 8 mod 16)
  const bool wide = a.rot % 16 == 0;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a);
    return cudaGetLastError();
  };
  if (wide)
    return a.dh <= 128 ? go(cache_rows_kernel<DT, QUANT, 8, 1>) : go(cache_rows_kernel<DT, QUANT, 8, 2>);
  return a.dh <= 128 ? go(cache_rows_kernel<DT, QUANT, 4, 2>) : go(cache_rows_kernel<DT, QUANT, 4, 4>);
}

// Tokens and heads of a block: where there are too few head rows to fill the GPU with
// blocks of 32 rows (one for each group of lanes), one token's heads are cut over blocks;
// else a block takes as many tokens (up to 32) as let all blocks run at once, four an SM,
// so that angles and places are found once for a token and no SM waits for a last block.
// (Measured at four, five and six an SM, the latter two at fewer registers: the prompts
// above 33, 33 and 41 us, the 8-bit rows 25.3, 26.0 and 30.5 us. Four tokens a block
// whatever the size: 37 and 30 us.)
int split_rows(RowArgs *a) {
  const int64_t rows = static_cast<int64_t>(a->batch) * a->n * a->heads;
  a->tokens_block = 1;
  a->heads_block = a->heads;
  if (rows < static_cast<int64_t>(kGroups) * 2048) {
    a->heads_block = a->heads < kGroups ? a->heads : kGroups;
  } else {
    int sms, smem;
    const int rc = device_sm_count(&sms, &smem);
    if (rc) return rc;
    const int64_t tokens = static_cast<int64_t>(a->batch) * a->n, at_once = int64_t{4} * sms;
    a->tokens_block = static_cast<int>(std::min<int64_t>(kBlockTokens, (tokens + at_once - 1) / at_once));
  }
  a->head_blocks = (a->heads + a->heads_block - 1) / a->heads_block;
  return DT_OK;
}

bool set_in(View *v, const dt_heads *x) {
  v->in = static_cast<const char *>(x->data);
  v->ib = 2 * x->stride_batch; v->ih = 2 * x->stride_head; v->ir = 2 * x->stride_row;
  v->heads = x->heads;
  return true;
}
void set_out(View *v, const dt_heads *x) {
  v->out = static_cast<char *>(x->data);
  v->ob = 2 * x->stride_batch; v->oh = 2 * x->stride_head; v->orow = 2 * x->stride_row;
}

bool set_rotation(RowArgs *a, const dt_rotation *rot, const int32_t *positions, int dh) {
  if (!rot || !positions || !al4(positions) || !rot->turns ||
      (reinterpret_cast<uintptr_t>(rot->turns) & 7u) || rot->rot < 8 || rot->rot > dh ||
      rot->rot % 8 || !std::isfinite(rot->magnitude))
    return false;
  a->turns = rot->turns;
  a->rot = rot->rot;
  a->interleaved = rot->interleaved != 0;
  a->mag = rot->magnitude;
  a->positions = positions;
  return true;
}

constexpr int64_t kMaxTokens = int64_t{1} << 28;   // keeps every grid below 2^31

}  // namespace

// sizes, alignment and strides of a [batch][heads][n][dh] view
bool heads_ok(const dt_heads *x) {
  return x && x->data && al16(x->data) && x->heads >= 1 && x->heads <= 4096 &&
         x->stride_batch % 8 == 0 && x->stride_head % 8 == 0 && x->stride_row % 8 == 0;
}

int check_cache(const dt_cache *c) {
  if (!c || !c->k || !c->v || !c->table || !c->status || !al16(c->k) || !al16(c->v) ||
      !al4(c->table) || !al4(c->status))
    return DT_ERR_INVALID_ARG;
  if (!(c->page == 16 || c->page == 32 || c->page == 64 || c->page == 128) || c->pages < 1 ||
      c->Hkv < 1 || c->Hkv > 4096 || c->dh < 16 || c->dh > 256 || c->dh % 16 || c->batch < 1 ||
      c->batch > 65535 || c->table_width < 1 || c->table_width > (1 << 24) / 16 ||
      static_cast<int64_t>(c->pages) * c->Hkv > 0x7fffffff)     // a tensor map's third coordinate
    return DT_ERR_INVALID_ARG;
  if (!(c->dtype == DT_BF16 || c->dtype == DT_F16 || c->dtype == DT_E4M3))
    return DT_ERR_INVALID_ARG;
  if (!al16(c->k_exp) || !al16(c->v_exp) || (c->dtype == DT_E4M3) != (c->k_exp != nullptr) || (c->dtype == DT_E4M3) != (c->v_exp != nullptr))
    return DT_ERR_INVALID_ARG;
  return DT_OK;
}

// the type of tensors around the cache: its own, or a 16-bit one for 8-bit rows
bool cache_dtype_ok(const dt_cache *c, int dtype) {
  return (dtype == DT_BF16 || dtype == DT_F16) && (c->dtype == DT_E4M3 || c->dtype == dtype);
}

}  // namespace dt

extern "C" {

int dt_rotary_table(const dt_rotary_params *p, uint64_t *turns, double *magnitude) {
  if (!p || !turns || !magnitude) return DT_ERR_INVALID_ARG;
  if (p->rot < 8 || p->rot > 2 * dt::kMaxHalf || p->rot % 8 || !std::isfinite(p->base) ||
      !(p->base > 1.0) || !std::isfinite(p->factor) || !(p->factor >= 1.0) ||
      p->scaling < DT_ROTARY_NONE || p->scaling > DT_ROTARY_PARTS)
    return DT_ERR_INVALID_ARG;
  const bool parts = p->scaling == DT_ROTARY_PARTS;
  if (parts && (!std::isfinite(p->trained) || !(p->trained >= 1.0) || !std::isfinite(p->beta_fast) ||
                !std::isfinite(p->beta_slow) || !(p->beta_fast > p->beta_slow)))
    return DT_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  double base = p->base;
  if (p->scaling == DT_ROTARY_BASE) base *= std::pow(p->factor, p->rot / (p->rot - 2.0));
  if (!std::isfinite(base)) return DT_ERR_INVALID_ARG;
  for (int i = 0; i < p->rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / p->rot);
    if (p->scaling == DT_ROTARY_LINEAR) f /= p->factor;
    if (parts) {
      double g = (p->trained * f / two_pi - p->beta_slow) / (p->beta_fast - p->beta_slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f *= g + (1.0 - g) / p->factor;
    }
    turns[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);   // f / 2 pi < 1/6
  }
  *magnitude = parts ? 1.0 + 0.1 * std::log(p->factor) : 1.0;
  return DT_OK;
}

int dt_rotary(const dt_rotation *rot, const int32_t *positions, int batch, int n, int dh,
              int dtype, const dt_heads *x0, const dt_heads *out0, const dt_heads *x1,
              const dt_heads *out1, int gradient, void *stream) {
  if (batch < 1 || batch > 65535 || n < 1 || static_cast<int64_t>(batch) * n > dt::kMaxTokens ||
      dh < 16 || dh > 256 || dh % 16 || !(dtype == DT_BF16 || dtype == DT_F16))
    return DT_ERR_INVALID_ARG;
  if (!dt::heads_ok(x0) || !dt::heads_ok(out0) || x0->heads != out0->heads || !x1 != !out1)
    return DT_ERR_INVALID_ARG;
  if (x1 && (!dt::heads_ok(x1) || !dt::heads_ok(out1) || x1->heads != out1->heads))
    return DT_ERR_INVALID_ARG;
  dt::RowArgs a = {};
  if (!dt::set_rotation(&a, rot, positions, dh)) return DT_ERR_INVALID_ARG;
  a.gradient = gradient != 0;
  a.batch = batch; a.n = n; a.dh = dh;
  a.nt = x1 ? 2 : 1;
  for (int i = 0; i < a.nt; ++i) {
    dt::set_in(&a.t[i], i ? x1 : x0);
    dt::set_out(&a.t[i], i ? out1 : out0);
    a.t[i].turned = 1;
    a.heads += a.t[i].heads;
  }
  const int rc = dt::split_rows(&a);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DT_BF16 ? dt::launch_rows<DT_BF16, false>(a, st)
                                         : dt::launch_rows<DT_F16, false>(a, st);
  return e == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

int dt_cache_write(const dt_cache *c, const dt_heads *k, const dt_heads *v, int n, int dtype,
                   const int32_t *first, const int32_t *counts, const dt_rotation *rot,
                   const int32_t *positions, const dt_heads *q, const dt_heads *q_out,
                   void *stream) {
  if (dt::check_cache(c) || !dt::cache_dtype_ok(c, dtype) || !dt::heads_ok(k) || !dt::heads_ok(v) ||
      k->heads != c->Hkv || v->heads != c->Hkv || n < 1 ||
      static_cast<int64_t>(c->batch) * n > dt::kMaxTokens || !first || !dt::al4(first) ||
      !dt::al4(counts) || !rot != !positions || !q != !q_out || (q && !rot))
    return DT_ERR_INVALID_ARG;
  if (q && (!dt::heads_ok(q) || !dt::heads_ok(q_out) || q->heads != q_out->heads))
    return DT_ERR_INVALID_ARG;
  dt::RowArgs a = {};
  if (rot && !dt::set_rotation(&a, rot, positions, c->dh)) return DT_ERR_INVALID_ARG;
  a.c = dt::cache_view(*c);
  a.first = first; a.counts = counts;
  a.batch = c->batch; a.n = n; a.dh = c->dh;
  a.nt = q ? 3 : 2;
  dt::set_in(&a.t[0], k);
  a.t[0].turned = rot != nullptr;
  dt::set_in(&a.t[1], v);
  a.t[1].to_v = 1;
  a.heads = 2 * c->Hkv;
  if (q) {
    dt::set_in(&a.t[2], q);
    dt::set_out(&a.t[2], q_out);
    a.t[2].turned = 1;
    a.heads += q->heads;
  }
  const int rc = dt::split_rows(&a);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool quant = c->dtype == DT_E4M3;
  const cudaError_t e =
      dtype == DT_BF16 ? (quant ? dt::launch_rows<DT_BF16, true>(a, st) : dt::launch_rows<DT_BF16, false>(a, st))
                       : (quant ? dt::launch_rows<DT_F16, true>(a, st) : dt::launch_rows<DT_F16, false>(a, st));
  return e == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

int dt_cache_read(const dt_cache *c, int n, int dtype, const int32_t *first,
                  const int32_t *counts, const dt_heads *k, const dt_heads *v, void *stream) {
  if (dt::check_cache(c) || !dt::cache_dtype_ok(c, dtype) || !dt::heads_ok(k) || !dt::heads_ok(v) ||
      k->heads != c->Hkv || v->heads != c->Hkv || n < 1 || !first || !dt::al4(first) ||
      !dt::al4(counts))
    return DT_ERR_INVALID_ARG;
  const int64_t row_blocks = (static_cast<int64_t>(n) + dt::kReadRows - 1) / dt::kReadRows;
  const int64_t grid = row_blocks * c->batch * c->Hkv;
  if (grid > 0x7fffffff) return DT_ERR_INVALID_ARG;
  dt::ReadArgs a;
  a.c = dt::cache_view(*c);
  a.first = first; a.counts = counts;
  a.k = static_cast<char *>(k->data); a.v = static_cast<char *>(v->data);
  a.kb = 2 * k->stride_batch; a.kh = 2 * k->stride_head; a.kr = 2 * k->stride_row;
  a.vb = 2 * v->stride_batch; a.vh = 2 * v->stride_head; a.vr = 2 * v->stride_row;
  a.n = n; a.row_blocks = static_cast<int>(row_blocks);
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), dt::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ERR_CUDA;
  };
  if (c->dtype != DT_E4M3) return go(dt::cache_read_kernel<DT_BF16, false>);   // a copy
  return dtype == DT_BF16 ? go(dt::cache_read_kernel<DT_BF16, true>)
                          : go(dt::cache_read_kernel<DT_F16, true>);
}

int dt_cache_commit(const dt_cache *c, const int32_t *first, const int32_t *path,
                    const int32_t *lengths, int width, int n, void *stream) {
  if (dt::check_cache(c) || !first || !path || !lengths || !dt::al4(first) || !dt::al4(path) ||
      !dt::al4(lengths) || width < 1 || width > dt::kMaxPath || n < 1 || n > DT_MAX_N + 1)
    return DT_ERR_INVALID_ARG;
  const int64_t grid = 2ll * c->batch * c->Hkv;
  dt::CommitArgs a;
  a.c = dt::cache_view(*c);
  a.first = first; a.path = path; a.lengths = lengths;
  a.width = width; a.n = n;
  a.row_bytes = c->dh * (c->dtype == DT_E4M3 ? 1 : 2);
  dt::cache_commit_kernel<<<static_cast<unsigned>(grid), dt::kThreads, width * a.row_bytes,
                            static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // extern "C"
