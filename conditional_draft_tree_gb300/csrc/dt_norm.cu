// dt_norm.cu -- root-mean-square norm of rows with the residual's addition, to 16 bits and
// to 8-bit rows, and rows to 8 bits alone.
//
// t = x + residual, y_i = t_i g_i / sqrt(mean(t^2) + eps), g = offset + weight. A group of
// threads owns a row and keeps it in registers, so each value is read once and each result
// written once. One reduction gives both the sum of squares and the largest |t_i g_i|:
// multiplying by a positive number keeps the order of fp32 numbers, so that
// the largest |y| is that product's, rounded the same way, and the 8-bit row's exponent needs no
// second one.
//
// Bound by memory where rows lie on 16-byte boundaries: 262336 heads of 128 fp16 values 25.5 us, 5.3
// TB/s; 8192 rows of 4096 with their sum 41.8 us, 6.4 TB/s; 2080 of them, much of them in L2, 9.4 us,
// to 16 and 8 bits 12.0; eight 2.3. Rows to 8 bits alone: 8192 of 4096 25.8 us, 3.9 TB/s, 2080 8.1. Rows off such
// boundaries: 4099 of 5001 values 56 us, 2.9 TB/s, where loads and stores of single values took 163. Instructions
// (shifts, shuffles, the ends) and latency bound them together: 62 a value, which at full rate would be 32 us, issued
// in 53 % of the cycles by 22 warps an SM (two blocks, by registers, without a row ahead) that wait for
// results and loads most, for barriers and shared memory next; DRAM is 28 % busy. Forms of more than two chunks a thread
// in few registers spill: aligned rows above 16384 values 2500 of 16392 108 us, 3.0 TB/s, 1300 of 32768 88, 3.9
// (16384: 54 us, 6.1 TB/s); off boundaries above 15864, 2500 of 15871 182 us, 1.75 TB/s (15863: 106, 3.0), 1300
// of 32767 189.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "dt_cache.cuh"
#include "dt_internal.h"

namespace dt {

namespace {

constexpr int kBlock = 0;      // a row's group of threads: the whole block

struct NormArgs {
  const char *x, *res, *weight;
  char *total, *out;
  uint8_t *codes, *exps;
  int64_t xo, xi, ro, ri, to, ti, oo, oi;   // strides in bytes
  const char *x_lo, *x_hi, *res_lo, *res_hi;   // where the views begin and end
  float offset, eps, inv_d;
  int rows, inner, d, norm;
};

// the larger magnitude (with some sign), NaN above all
__device__ __forceinline__ float top_abs(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// the sum and, TOP, the largest magnitude over the group's threads; whole blocks go through shared
// memory, one slot a warp, twice so that a row's are not overwritten before all have read
// the row before it
template <int GROUP>
__device__ __forceinline__ void reduce(float &sum, float &top, bool with_top, float (*s_sum)[32],
                                       float (*s_top)[32], int &turn) {
  constexpr bool kWhole = GROUP == kBlock || GROUP > 32;
  constexpr int kIn = kWhole ? 32 : GROUP;
  const int lane = threadIdx.x & 31;
  const unsigned mask = kIn == 32 ? kFull : ((1u << kIn) - 1u) << (lane & ~(kIn - 1));
  auto across = [&](int from, unsigned among) {
#pragma unroll
    for (int m = from; m; m >>= 1) sum += __shfl_xor_sync(among, sum, m);
    if (with_top)
#pragma unroll
      for (int m = from; m; m >>= 1) top = top_abs(top, __shfl_xor_sync(among, top, m));
  };
  across(kIn / 2, mask);
  if (kWhole) {
    const int warp = threadIdx.x >> 5, warps = (GROUP == kBlock ? blockDim.x : GROUP) >> 5;
    if (lane == 0) {
      s_sum[turn][warp] = sum;
      s_top[turn][warp] = top;
    }
    __syncthreads();
    const bool there = lane < warps;
    sum = there ? s_sum[turn][lane] : 0.0f;
    top = there ? s_top[turn][lane] : 0.0f;
    turn ^= 1;
    across(16, kFull);
  }
}

// Sixteen bytes at g (on a 16-byte boundary), those outside [lo, hi) as zeros or left as they are: where
// a tensor, or a row that is written, does not begin or end on such a boundary.
__device__ __noinline__ uint4 load_end(const char *g, const char *lo, const char *hi) {
  uint32_t w[4] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (g + 2 * e >= lo && g + 2 * e < hi)
      w[e / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(g + 2 * e)) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Granules that lie partly outside [lo, hi), those of the lanes that say so: one after the other, a
// lane an element (a loop of one lane over its eight is as long as the rest of a row's work).
__device__ __forceinline__ void store_ends(bool mine, char *g, const char *lo, const char *hi, const uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 31;
  for (unsigned left = __ballot_sync(kFull, mine); left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __shfl_sync(kFull, w[e], from);
    char *to = reinterpret_cast<char *>(shfl64(reinterpret_cast<uint64_t>(g), from)) + 2 * lane;
    const uint32_t word = lane & 4 ? (lane & 2 ? v[3] : v[2]) : (lane & 2 ? v[1] : v[0]);
    if (lane < 8 && to >= lo && to < hi)
      *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(word >> (16 * (lane & 1)));
  }
}
__device__ __forceinline__ void store_codes_ends(bool mine, uint8_t *g, const uint8_t *lo, const uint8_t *hi, uint64_t w) {
  const int lane = threadIdx.x & 31;
  for (unsigned left = __ballot_sync(kFull, mine); left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    const uint64_t v = shfl64(w, from);
    uint8_t *to = reinterpret_cast<uint8_t *>(shfl64(reinterpret_cast<uint64_t>(g), from)) + lane;
    if (lane < 8 && to >= lo && to < hi) *to = static_cast<uint8_t>(v >> (8 * (lane & 7)));
  }
}

// the 16 bytes that begin `off` bytes (even, below 16; the same for a row's threads) into the 32 of a and
// b. (Branches that the compiler keeps: as selections this takes three times the instructions.)
__device__ __forceinline__ void shifted(const uint32_t *a, const uint32_t *b, int off, uint32_t (&r)[4]) {
  const uint32_t w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  const int half = off & 2 ? 16 : 0;
  auto from = [&](auto k) {
    asm volatile("");
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(w[k.value + i], w[k.value + i + 1], half);
  };
  switch (off >> 2) {
    case 0: from(std::integral_constant<int, 0>{}); break;
    case 1: from(std::integral_constant<int, 1>{}); break;
    case 2: from(std::integral_constant<int, 2>{}); break;
    default: from(std::integral_constant<int, 3>{}); break;
  }
}

__device__ __forceinline__ uint32_t up_one(uint32_t v) { return __shfl_up_sync(kFull, v, 1); }

template <int DT>
__device__ __forceinline__ uint64_t unpack2(uint32_t u) {
  const float2 f = Half16<DT>::unpack(u);
  return pair(f.x, f.y);
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  unpair(v, &lo, &hi);
  return Half16<DT>::pack(lo, hi);
}

constexpr int kSmall = 256;    // threads of a block whose rows have fewer than 32

// GROUP threads a row (kBlock: those that the block has), each with ITEMS chunks of 8 values. WIDE: all
// rows lie on 16-byte boundaries, chunks are loads and stores. Else each tensor's rows begin anywhere:
// a chunk is cut from the two 16-byte granules that it lies in, and a granule of a result put together
// from a thread's chunk and its left neighbour's; a warp's first lane has the chunk of the warp before
// it once more for that (31 new chunks a warp). (Chunks that follow x's own boundaries, one granule
// each, were no faster: 57 us for 56.) AHEAD: the next row is on its way while this one is worked on. Values
// go in pairs through the two-wide fp32 instructions: one by one, some 25 instructions a value
// bounded the kernel (heads 43 us, 5000 wide 53 us; now 25.5 and 28).
template <int DT, bool WIDE, int GROUP, int ITEMS, bool AHEAD, int REGS>
__global__ void __maxnreg__(REGS) rms_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr bool kWhole = GROUP == kBlock || GROUP > 32;      // a row a block
  constexpr int kRows = kWhole ? 1 : kSmall / (kWhole ? 1 : GROUP);   // of a block at a time
  constexpr int kWords = WIDE ? 4 : 8;                        // of a chunk's loads
  constexpr bool kPacked = ITEMS > 2;                         // the weights stay in 16 bits
  __shared__ float s_sum[2][32], s_top[2][32];
  const int group = GROUP == kBlock ? blockDim.x : GROUP;
  const int lane = kWhole ? threadIdx.x : threadIdx.x % (kWhole ? 1 : GROUP);
  const int mine = kWhole ? 0 : threadIdx.x / (kWhole ? 1 : GROUP);   // row of the block's
  int turn = 0;
  // chunk number of an item; -1: none (the first lane of a row's first warp)
  auto chunk = [&](int it) {
    return WIDE ? it * group + lane : (it * (group >> 5) + (lane >> 5)) * 31 + (lane & 31) - 1;
  };
  const bool again = !WIDE && (lane & 31) == 0;               // its chunk counts for the warp before
  const int chunks = (a.d + 7) >> 3;
  // Granules that hold some of the row's values are read, and no others: memory between the rows need not be there.
  // (What else lies in them is dropped by words(); the tensor's first and last ones are read by value.)
  auto load = [&](const char *p, const char *lo, const char *hi, bool there, uint32_t (&w)[ITEMS][kWords]) {
    const int off = WIDE ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
    const bool inside = p - 16 >= lo && p + 2 * a.d + 32 <= hi;      // (all rows but the first and the last)
    const bool after = 16 * chunks - off < 2 * a.d;       // the last chunk ends behind its first granule
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const int c = chunk(it);
      uint4 v = make_uint4(0u, 0u, 0u, 0u), z = v;
      if (there && c >= 0 && c < chunks) {
        const char *g = p + 16 * c - off;
        if (WIDE) {
          v = *reinterpret_cast<const uint4 *>(g);
        } else if (inside) {
          v = *reinterpret_cast<const uint4 *>(g);
          if (c + 1 < chunks || after) z = *reinterpret_cast<const uint4 *>(g + 16);
        } else {
          v = load_end(g, lo, hi);
          z = load_end(g + 16, lo, hi);
        }
      }
      w[it][0] = v.x; w[it][1] = v.y; w[it][2] = v.z; w[it][3] = v.w;
      if (!WIDE) {
        w[it][kWords - 4] = z.x; w[it][kWords - 3] = z.y; w[it][kWords - 2] = z.z; w[it][kWords - 1] = z.w;
      }
    }
  };
  // a chunk's four words, zeros behind the row's end
  auto words = [&](int it, const uint32_t (&w)[kWords], const char *p, uint32_t (&r)[4]) {
    if (WIDE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = w[e];
    } else {
      shifted(w, w + kWords - 4, static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u), r);
      const int left = a.d - 8 * chunk(it);
      if (left < 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = left > 2 * e + 1 ? r[e] : left > 2 * e ? r[e] & 0xffffu : 0u;
      }
    }
  };
  auto store = [&](char *p, int it, const uint32_t (&r)[4]) {
    const int c = chunk(it);
    if (WIDE) {
      if (c < chunks) *reinterpret_cast<uint4 *>(p + 16 * c) = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
      const uint32_t left[4] = {up_one(r[0]), up_one(r[1]), up_one(r[2]), up_one(r[3])};
      uint32_t g[4];
      shifted(left, r, (16 - off) & 15, g);
      const bool none = again || c > chunks || (c == chunks && !off), whole = c > 0 && c + 1 < chunks;
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = off ? g[e] : r[e];
      char *to = p + 16 * c - off;
      if (!none && whole) *reinterpret_cast<uint4 *>(to) = make_uint4(g[0], g[1], g[2], g[3]);
      store_ends(!none && !whole, to, p, p + 2 * a.d, g);
    }
  };
  // eight codes: bytes begin anywhere, a granule has eight
  auto store8 = [&](uint8_t *p, int it, uint32_t lo, uint32_t hi) {
    const int c = chunk(it);
    if (WIDE) {
      if (c < chunks) *reinterpret_cast<uint2 *>(p + 8 * c) = make_uint2(lo, hi);
    } else {
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 7u);
      const uint64_t left = up_one(lo) | (static_cast<uint64_t>(up_one(hi)) << 32);
      const uint64_t mine = lo | (static_cast<uint64_t>(hi) << 32);
      const bool none = again || c > chunks || (c == chunks && !off), whole = c > 0 && c + 1 < chunks;
      const uint64_t g = off ? (left >> (64 - 8 * off)) | (mine << (8 * off)) : mine;
      uint8_t *to = p + 8 * c - off;
      if (!none && whole) *reinterpret_cast<uint64_t *>(to) = g;
      store_codes_ends(!none && !whole, to, p, p + a.d, g);
    }
  };
  // the group's row, and where it lies; rows follow at a fixed distance, without a division for each
  struct Row {
    int at, o, i;
  };
  const int stride = gridDim.x * kRows, outer_step = stride / a.inner, inner_step = stride - outer_step * a.inner;
  auto next_of = [&](Row r) {
    r.at += stride;
    r.o += outer_step;
    r.i += inner_step;
    if (r.i >= a.inner) {
      r.i -= a.inner;
      ++r.o;
    }
    return r;
  };
  Row row;
  row.at = blockIdx.x * kRows + mine;
  row.o = row.at / a.inner;
  row.i = row.at - row.o * a.inner;
  uint32_t wx[ITEMS][kWords], wr[ITEMS][kWords], wg[ITEMS][4];
  uint64_t gains[ITEMS][4];
  auto place = [&](const char *p, int64_t outer, int64_t inner, const Row &r) { return p + r.o * outer + r.i * inner; };
  auto fetch = [&](const Row &r) {
    const bool there = r.at < a.rows;
    load(place(a.x, a.xo, a.xi, r), a.x_lo, a.x_hi, there, wx);
    if (a.res) load(place(a.res, a.ro, a.ri, r), a.res_lo, a.res_hi, there, wr);
  };
  if (AHEAD) fetch(row);
  const uint64_t offset = pair(a.offset, a.offset);
  auto gain = [&](int it, int e) { return kPacked && a.weight ? add2(unpack2<DT>(wg[it][e]), offset) : gains[kPacked ? 0 : it][kPacked ? 0 : e]; };
  {
    uint32_t w[ITEMS][kWords];
    if (a.weight) load(a.weight, a.weight, a.weight + 2 * a.d, true, w);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      if (a.weight) words(it, w[it], a.weight, wg[it]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        gains[it][e] = a.weight ? add2(unpack2<DT>(wg[it][e]), offset)
                       : a.norm ? add2(pair(1.0f, 1.0f), offset) : pair(1.0f, 1.0f);
    }
  }
  // the threads of a block go through as many rows each: the last ones may be none
  for (; row.at - mine < a.rows; row = next_of(row)) {
    if (!AHEAD) fetch(row);
    uint64_t t[ITEMS][4];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      uint32_t w[4];
      words(it, wx[it], place(a.x, a.xo, a.xi, row), w);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[it][e] = unpack2<DT>(w[e]);
    }
    if (a.res) {                       // (without one -0 stays -0)
      char *total = const_cast<char *>(place(a.total, a.to, a.ti, row));
      uint32_t w[ITEMS][4];
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        words(it, wr[it], place(a.res, a.ro, a.ri, row), w[it]);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[it][e] = add2(t[it][e], unpack2<DT>(w[it][e]));
      }
      if (AHEAD) fetch(next_of(row));
      // the sum may take the place of x or the residual: for wide rows each thread writes what it alone
      // has read, others' granules are written behind the reduction
      if (WIDE && row.at < a.rows) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[it][e] = pack2<DT>(t[it][e]);
          store(total, it, w[it]);
        }
      }
    } else if (AHEAD) {
      fetch(next_of(row));
    }
    const bool live = row.at < a.rows;
    float sum, top;
    auto reduce_row = [&]() {
      uint64_t s = 0;
      top = 0.0f;
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fma2(t[it][e], t[it][e], s);
      if (a.codes) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo, hi;
            unpair(mul2(t[it][e], gain(it, e)), &lo, &hi);
            top = top_abs(top_abs(top, lo), hi);
          }
      }
      float lo, hi;
      unpair(s, &lo, &hi);
      sum = again ? 0.0f : lo + hi;
      reduce<GROUP>(sum, top, a.codes != nullptr, s_sum, s_top, turn);
    };
    reduce_row();
    if (a.res && !WIDE && live) {
      char *total = const_cast<char *>(place(a.total, a.to, a.ti, row));
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack2<DT>(t[it][e]);
        store(total, it, w);
      }
    }
    float scale = 1.0f;
    if (a.norm) {
      if (!(sum <= 0x1p100f)) {          // squares that leave fp32: the row times 2^-80
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[it][e] = mul2(t[it][e], pair(0x1p-80f, 0x1p-80f));
        reduce_row();
        scale = rsqrtf(sum * a.inv_d);   // eps 2^-160 is nothing beside a mean above 2^-75
      } else {
        scale = rsqrtf(sum * a.inv_d + a.eps);
      }
    }
    if (!live) continue;                 // a whole group: no other lane of it is left behind
    const uint64_t scales = pair(scale, scale);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[it][e] = mul2(mul2(t[it][e], gain(it, e)), scales);
    if (a.out) {
      char *out = const_cast<char *>(place(a.out, a.oo, a.oi, row));
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack2<DT>(t[it][e]);
        store(out, it, w);
      }
    }
    if (a.codes) {
      const uint32_t most = __float_as_uint(fabsf(top) * scale) & 0x7fffffffu;
      const bool whole = most < 0x7f800000u;
      const int ex = row_exponent(__uint_as_float(most));
      const float down = exp2i(-ex);
      if (lane == 0) a.exps[row.at] = static_cast<uint8_t>(whole ? ex + 127 : 255);
      uint8_t *codes = a.codes + static_cast<int64_t>(row.at) * a.d;
      const bool clamp = ex == 120;      // 256 2^120 is no finite bf16 number
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          unpair(mul2(t[it][e], pair(down, down)), &lo, &hi);
          if (clamp) {
            lo = fminf(fmaxf(lo, -240.0f), 240.0f);
            hi = fminf(fmaxf(hi, -240.0f), 240.0f);
          }
          y[e] = e4m3_pack2(lo, hi);
        }
        store8(codes, it, whole ? y[0] | (y[1] << 16) : 0x7f7f7f7fu, whole ? y[2] | (y[3] << 16) : 0x7f7f7f7fu);
      }
    }
  }
}

template <int DT, bool WIDE>
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t st) {
  // as many blocks as run at once (65536 registers an SM), or fewer
  auto go = [&](auto kernel, int threads, int rows, int regs) {
    const int64_t blocks = (static_cast<int64_t>(a.rows) + rows - 1) / rows;
    const int64_t most = static_cast<int64_t>(sms) * std::max(1, std::min(16, 65536 / (threads * regs)));
    kernel<<<static_cast<unsigned>(std::min(blocks, most)), threads, 0, st>>>(a);
    return cudaGetLastError();
  };
  const int chunks = (a.d + 7) / 8;
  if constexpr (WIDE) {
    if (chunks <= 8) return go(rms_norm_kernel<DT, true, 8, 1, true, 48>, kSmall, kSmall / 8, 48);
    if (chunks <= 16) return go(rms_norm_kernel<DT, true, 16, 1, true, 48>, kSmall, kSmall / 16, 48);
    if (chunks <= 32) return go(rms_norm_kernel<DT, true, 32, 1, true, 48>, kSmall, kSmall / 32, 48);
    if (chunks <= 64) return go(rms_norm_kernel<DT, true, 32, 2, true, 80>, kSmall, kSmall / 32, 80);
    // Blocks of as many threads as the row needs; where that is a power of two, or nearly, of a number
    // that the compiler knows (2080 rows of 4096 with their sum 10.4 to 9.5 us, to 8 bits too 13.9 to
    // 12.2).
    auto nearly = [&](int threads) { return chunks <= 2 * threads && chunks > 2 * threads * 7 / 8; };
    if (nearly(64)) return go(rms_norm_kernel<DT, true, 64, 2, true, 80>, 64, 1, 80);
    if (nearly(128)) return go(rms_norm_kernel<DT, true, 128, 2, true, 80>, 128, 1, 80);
    if (nearly(256)) return go(rms_norm_kernel<DT, true, 256, 2, true, 80>, 256, 1, 80);
    if (nearly(512)) return go(rms_norm_kernel<DT, true, 512, 2, true, 80>, 512, 1, 80);
    if (chunks <= 1024) return go(rms_norm_kernel<DT, true, kBlock, 2, true, 80>, (chunks + 63) / 64 * 32, 1, 80);
    if (chunks <= 2048) return go(rms_norm_kernel<DT, true, kBlock, 4, true, 128>, (chunks + 127) / 128 * 32, 1, 128);
    return go(rms_norm_kernel<DT, true, kBlock, 4, false, 64>, (chunks + 127) / 128 * 32, 1, 64);
  } else {
    // 31 chunks a warp and item, and one for a row's last granule
    const int need = chunks + 1;
    if (need <= 31) return go(rms_norm_kernel<DT, false, 32, 1, true, 64>, kSmall, kSmall / 32, 64);
    if (need <= 62) return go(rms_norm_kernel<DT, false, 32, 2, true, 112>, kSmall, kSmall / 32, 112);
    if (need <= 992) return go(rms_norm_kernel<DT, false, kBlock, 2, false, 80>, (need + 61) / 62 * 32, 1, 80);
    if (need <= 1984) return go(rms_norm_kernel<DT, false, kBlock, 4, false, 128>, (need + 123) / 124 * 32, 1, 128);
    return go(rms_norm_kernel<DT, false, kBlock, 5, false, 64>, (need + 154) / 155 * 32, 1, 64);
  }
}

bool al2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// the bytes that a view of rows of d values spans
void view_span(const dt_rows *v, int outer, int inner, int d, const char **lo, const char **hi) {
  const int64_t o = 2 * v->stride_outer * (outer - 1), i = 2 * v->stride_inner * (inner - 1), zero = 0;
  const char *p = static_cast<const char *>(v->data);
  *lo = p + std::min(o, zero) + std::min(i, zero);
  *hi = p + std::max(o, zero) + std::max(i, zero) + 2 * static_cast<int64_t>(d);
}

// strides into bytes; whether the view's rows lie on 16-byte boundaries
bool view_wide(const dt_rows *v, int64_t *outer, int64_t *inner) {
  *outer = 2 * v->stride_outer;
  *inner = 2 * v->stride_inner;
  return (reinterpret_cast<uintptr_t>(v->data) & 15u) == 0 && v->stride_outer % 8 == 0 &&
         v->stride_inner % 8 == 0;
}

int norm_rows(const dt_rows *x, const dt_rows *residual, const dt_rows *total, const dt_rows *out,
              uint8_t *codes, uint8_t *exps, const void *weight, float offset, float eps, int outer,
              int inner, int d, int dtype, int norm, void *stream) {
  if (!x || !x->data || !al2(x->data) || !residual != !total || (!out && !codes) || !codes != !exps ||
      outer < 1 || inner < 1 || static_cast<int64_t>(outer) * inner > (int64_t{1} << 30) || d < 1 ||
      d > 32768 || !(dtype == DT_BF16 || dtype == DT_F16) || !al2(weight))
    return DT_ERR_INVALID_ARG;
  if (norm && (!(eps >= 1e-30f) || !std::isfinite(eps) || !std::isfinite(offset)))
    return DT_ERR_INVALID_ARG;
  for (const dt_rows *v : {residual, total, out})
    if (v && (!v->data || !al2(v->data))) return DT_ERR_INVALID_ARG;
  if (total && out && total->data == out->data) return DT_ERR_INVALID_ARG;      // one of the two would be lost
  NormArgs a = {};
  a.x = static_cast<const char *>(x->data);
  bool wide = view_wide(x, &a.xo, &a.xi) && d % 8 == 0 &&
              (reinterpret_cast<uintptr_t>(weight) & 15u) == 0 && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0;
  view_span(x, outer, inner, d, &a.x_lo, &a.x_hi);
  if (residual) {
    view_span(residual, outer, inner, d, &a.res_lo, &a.res_hi);
    a.res = static_cast<const char *>(residual->data);
    a.total = static_cast<char *>(total->data);
    wide = view_wide(residual, &a.ro, &a.ri) && wide;
    wide = view_wide(total, &a.to, &a.ti) && wide;
  }
  if (out) {
    a.out = static_cast<char *>(out->data);
    wide = view_wide(out, &a.oo, &a.oi) && wide;
  }
  a.codes = codes;
  a.exps = exps;
  a.weight = static_cast<const char *>(weight);
  a.offset = offset;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(d);
  a.rows = outer * inner;
  a.inner = inner;
  a.d = d;
  a.norm = norm;
  int sms, smem;
  const int rc = device_sm_count(&sms, &smem);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == DT_BF16 ? (wide ? launch_norm<DT_BF16, true>(a, sms, st) : launch_norm<DT_BF16, false>(a, sms, st))
                       : (wide ? launch_norm<DT_F16, true>(a, sms, st) : launch_norm<DT_F16, false>(a, sms, st));
  return e == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // namespace

}  // namespace dt

extern "C" {

int dt_rms_norm(const dt_rows *x, const dt_rows *residual, const dt_rows *total,
                const dt_rows *out, uint8_t *codes, uint8_t *exps, const void *weight,
                float offset, float eps, int outer, int inner, int d, int dtype, void *stream) {
  return dt::norm_rows(x, residual, total, out, codes, exps, weight, offset, eps, outer, inner, d,
                       dtype, 1, stream);
}

int dt_quantize_rows(const dt_rows *x, uint8_t *codes, uint8_t *exps, int outer, int inner, int d,
                     int dtype, void *stream) {
  return dt::norm_rows(x, nullptr, nullptr, nullptr, codes, exps, nullptr, 0.0f, 1.0f, outer, inner,
                       d, dtype, 0, stream);
}

}  // extern "C"
