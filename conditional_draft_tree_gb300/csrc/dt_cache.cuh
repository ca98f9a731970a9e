// dt_cache.cuh -- the paged key/value cache: addressing and the 8-bit row format,
// shared by the kernels that write, read, compact and attend over it.
//
// Row `index` of request b (0 = the request's first token) lies in page
// table[b][index / page], slot index % page; a page holds, for each key/value
// head, its slots' rows one after another: [Hkv][page][dh].
//
// 8-bit rows: e4m3 codes and one exponent byte E a row, value = code 2^(E - 127).
// E - 127 is the least e in [-117, 120] with amax <= 448 2^e, so nothing is
// clipped (but values above 248 2^120, which become 240 2^120), scaling is exact
// and every value is exact in bf16: 4 significant bits, and the least one,
// 2^-9 2^-117, is a normal bf16 number. A row that holds a NaN or an infinity
// cannot be scaled: E = 255, codes 0x7f, and it reads back as NaN.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dt_common.cuh"
#include "../../include/dt.h"

namespace dt {

struct CacheView {
  void *k, *v;
  uint8_t *k_exp, *v_exp;
  const int32_t *table;
  int32_t *status;
  int pages, shift, Hkv, dh, width;   // page = 1 << shift
  int64_t page_rows;                  // Hkv << shift
};

inline CacheView cache_view(const dt_cache &c) {
  CacheView v;
  v.k = c.k; v.v = c.v; v.k_exp = c.k_exp; v.v_exp = c.v_exp;
  v.table = c.table; v.status = c.status;
  v.pages = c.pages; v.Hkv = c.Hkv; v.dh = c.dh; v.width = c.table_width;
  v.shift = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
  v.page_rows = static_cast<int64_t>(c.Hkv) << v.shift;
  return v;
}

// head row number of (request b, row index, head hk), or -1 where the index is
// outside the request's table or its page outside the pool (64-bit: a pool may
// hold more than 2^31 elements)
__host__ __device__ __forceinline__ int64_t cache_row(const CacheView &c, int b, int64_t index,
                                                      int hk) {
  if (index < 0 || (index >> c.shift) >= c.width) return -1;
  const int page = c.table[static_cast<int64_t>(b) * c.width + (index >> c.shift)];
  if (page < 0 || page >= c.pages) return -1;
  return page * c.page_rows + (static_cast<int64_t>(hk) << c.shift) +
         (index & ((1 << c.shift) - 1));
}

__device__ __forceinline__ void cache_fault(const CacheView &c, int b) {
  c.status[b] = DT_ERR_BAD_PAGE;   // several threads may store the same code
}

// ------------------------------------------------------------ 16-bit types

template <int DT> struct Half16;   // DT_BF16 or DT_F16 bits <-> fp32
template <> struct Half16<DT_BF16> {
  __device__ static float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  __device__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <> struct Half16<DT_F16> {
  __device__ static float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
  }
  __device__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// largest magnitudes of two pairs of 16-bit values (signs are not kept), NaN above all
template <int DT>
__device__ __forceinline__ uint32_t top_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == DT_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ------------------------------------------------------------- 8-bit rows

// 2^e as fp32, e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// exponent of a row whose largest magnitude is `amax` (finite)
__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = 1.m 2^k <= 448 2^e = 1.75 2^(8 + e)
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return min(max(e, -117), 120);
}

// two values, already scaled to |x| <= 448, as e4m3 codes (round to nearest even);
// lo in the low byte
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two codes (low 16 bits) as two exact fp16 values
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
// row scale of an exponent byte; NaN for 255 (0 and 254 are never written, and
// read as the powers of two that fp32 has next to them)
__device__ __forceinline__ float row_scale(uint32_t E) {
  return E == 255u ? __uint_as_float(0x7fc00000u)
                   : __uint_as_float((E == 0u ? 1u : E) << 23);
}
// two codes times the row's scale, in the 16-bit type (fp16 saturates at 65504)
template <int DT>
__device__ __forceinline__ uint32_t e4m3_to16(uint32_t two, float scale) {
  const float2 f = Half16<DT_F16>::unpack(e4m3_f16x2(two));
  float a = f.x * scale, b = f.y * scale;
  if (DT == DT_F16) {   // comparisons keep a NaN
    a = a > 65504.0f ? 65504.0f : a < -65504.0f ? -65504.0f : a;
    b = b > 65504.0f ? 65504.0f : b < -65504.0f ? -65504.0f : b;
  }
  return Half16<DT>::pack(a, b);
}

}  // namespace dt
