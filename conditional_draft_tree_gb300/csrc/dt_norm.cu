// dt_norm.cu -- root-mean-square norm of rows with the residual's addition, to 16 bits and
// to 8-bit rows, and rows to 8 bits alone.
//
// t = x + residual, y_i = t_i g_i / sqrt(mean(t^2) + eps), g = offset + weight. A group of
// threads owns a row and keeps it in registers, so each value is read once and each result
// written once. One reduction gives both the sum of squares and the largest |t_i g_i|:
// multiplying by a positive number keeps the order of fp32 numbers, so that
// the largest |y| is that product's, rounded the same way, and the 8-bit row's exponent needs no
// second one.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dt_cache.cuh"
#include "dt_internal.h"

namespace dt {

namespace {

struct NormArgs {
  const char *x, *res, *weight;
  char *total, *out;
  uint8_t *codes, *exps;
  int64_t xo, xi, ro, ri, to, ti, oo, oi;   // strides in bytes
  float offset, eps, inv_d;
  int rows, inner, d, norm;
};

// sums and largest magnitude bits over the group's threads; whole blocks go through shared
// memory, one slot a warp, twice so that a row's are not overwritten before all have read
// the row before it
template <int GROUP>
__device__ __forceinline__ void reduce(float &sum, uint32_t &top, float (*s_sum)[32],
                                       uint32_t (*s_top)[32], int &turn) {
  constexpr int kIn = GROUP < 32 ? GROUP : 32;
  const int lane = threadIdx.x & 31;
  const unsigned mask = kIn == 32 ? kFull : ((1u << kIn) - 1u) << (lane & ~(kIn - 1));
#pragma unroll
  for (int m = kIn / 2; m; m >>= 1) {
    sum += __shfl_xor_sync(mask, sum, m);
    top = max(top, __shfl_xor_sync(mask, top, m));
  }
  if (GROUP > 32) {
    constexpr int kWarps = GROUP / 32;
    const int warp = threadIdx.x >> 5;
    if (lane == 0) {
      s_sum[turn][warp] = sum;
      s_top[turn][warp] = top;
    }
    __syncthreads();
    sum = lane < kWarps ? s_sum[turn][lane] : 0.0f;
    top = lane < kWarps ? s_top[turn][lane] : 0u;
    turn ^= 1;
#pragma unroll
    for (int m = (kWarps > 1 ? 16 : 0); m; m >>= 1) {
      sum += __shfl_xor_sync(kFull, sum, m);
      top = max(top, __shfl_xor_sync(kFull, top, m));
    }
  }
}

// GROUP threads a row, each with ITEMS chunks of 8 values: 16 bytes at a time (WIDE), or
// value by value, neighbours in neighbouring threads.
template <int DT, bool WIDE, int GROUP, int ITEMS>
__global__ void __launch_bounds__(GROUP < 256 ? 256 : GROUP)
rms_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = GROUP < 256 ? 256 / GROUP : 1;        // rows of a block at a time
  __shared__ float s_sum[2][32];
  __shared__ uint32_t s_top[2][32];
  const int lane = threadIdx.x % GROUP;
  int turn = 0;
  auto at = [&](int it, int e) { return WIDE ? (it * GROUP + lane) * 8 + e : (it * 8 + e) * GROUP + lane; };
  auto load = [&](const char *p, uint32_t (&w)[ITEMS][4]) {
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      if (WIDE) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (p && at(it, 0) < a.d) v = *reinterpret_cast<const uint4 *>(p + 2 * at(it, 0));
        w[it][0] = v.x; w[it][1] = v.y; w[it][2] = v.z; w[it][3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t lo = 0, hi = 0;
          if (p && at(it, 2 * e) < a.d) lo = *reinterpret_cast<const uint16_t *>(p + 2 * at(it, 2 * e));
          if (p && at(it, 2 * e + 1) < a.d) hi = *reinterpret_cast<const uint16_t *>(p + 2 * at(it, 2 * e + 1));
          w[it][e] = lo | (hi << 16);
        }
      }
    }
  };
  auto store = [&](char *p, const float (&f)[ITEMS][8]) {
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = Half16<DT>::pack(f[it][2 * e], f[it][2 * e + 1]);
      if (WIDE) {
        if (at(it, 0) < a.d) *reinterpret_cast<uint4 *>(p + 2 * at(it, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at(it, e) < a.d)
            *reinterpret_cast<uint16_t *>(p + 2 * at(it, e)) = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
      }
    }
  };
  const int stride = gridDim.x * kRows;
  int row = blockIdx.x * kRows + threadIdx.x / GROUP;
  uint32_t wx[ITEMS][4], wr[ITEMS][4], wg[ITEMS][4];
  auto fetch = [&](int r) {
    const int o = r / a.inner, i = r - o * a.inner;
    load(r < a.rows ? a.x + o * a.xo + i * a.xi : nullptr, wx);
    load(a.res && r < a.rows ? a.res + o * a.ro + i * a.ri : nullptr, wr);
  };
  fetch(row);
  load(a.weight, wg);
  // the threads of a block go through as many rows each: the last ones may be none
  for (; row - static_cast<int>(threadIdx.x / GROUP) < a.rows; row += stride) {
    float t[ITEMS][8], p[ITEMS][8];
    float sum = 0.0f;
    uint32_t top = 0;
    // power: the rows of values whose squares leave fp32 are taken times 2^-80
    auto products = [&](float power) {
      sum = 0.0f;
      top = 0;
#pragma unroll
      for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = t[it][e] * power;
          float g = 1.0f;
          if (a.weight) {
            const float2 f = Half16<DT>::unpack(wg[it][e / 2]);
            g = a.offset + (e & 1 ? f.y : f.x);
          } else {
            g = a.norm ? a.offset + 1.0f : 1.0f;
          }
          p[it][e] = v * g;
          sum += v * v;
          top = max(top, __float_as_uint(p[it][e]) & 0x7fffffffu);
        }
    };
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = Half16<DT>::unpack(wx[it][e]), r = Half16<DT>::unpack(wr[it][e]);
        t[it][2 * e] = a.res ? x.x + r.x : x.x;      // (-0 stays -0)
        t[it][2 * e + 1] = a.res ? x.y + r.y : x.y;
      }
    const int here = row;
    fetch(row + stride);
    products(1.0f);
    reduce<GROUP>(sum, top, s_sum, s_top, turn);
    float scale = 1.0f;
    if (a.norm) {
      if (!(sum <= 0x1p100f)) {
        products(0x1p-80f);
        reduce<GROUP>(sum, top, s_sum, s_top, turn);
        scale = rsqrtf(sum * a.inv_d);     // eps 2^-160 is nothing beside a mean above 2^-75
      } else {
        scale = rsqrtf(sum * a.inv_d + a.eps);
      }
    }
    if (here >= a.rows) continue;
    const int o = here / a.inner, i = here - o * a.inner;
    if (a.total) store(a.total + o * a.to + i * a.ti, t);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
      for (int e = 0; e < 8; ++e) p[it][e] *= scale;
    if (a.out) store(a.out + o * a.oo + i * a.oi, p);
    if (!a.codes) continue;
    const uint32_t most = __float_as_uint(__uint_as_float(top) * scale) & 0x7fffffffu;
    const bool whole = most < 0x7f800000u;
    const int ex = row_exponent(__uint_as_float(most));
    const float down = exp2i(-ex);
    if (lane == 0) a.exps[here] = static_cast<uint8_t>(whole ? ex + 127 : 255);
    uint8_t *codes = a.codes + static_cast<int64_t>(here) * a.d;
    const float bound = ex == 120 ? 240.0f * 0x1p120f : __int_as_float(0x7f800000);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        float f[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) f[z] = fminf(fmaxf(p[it][e + z], -bound), bound) * down;
        const uint32_t y = e4m3_pack2(f[0], f[1]) | (e4m3_pack2(f[2], f[3]) << 16);
        w[e / 4] = whole ? y : 0x7f7f7f7fu;
      }
      if (WIDE) {
        if (at(it, 0) < a.d) *reinterpret_cast<uint2 *>(codes + at(it, 0)) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at(it, e) < a.d) codes[at(it, e)] = static_cast<uint8_t>(w[e / 4] >> (8 * (e & 3)));
      }
    }
  }
}

template <int DT, bool WIDE>
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t st) {
  auto go = [&](auto kernel, int group) {
    const int threads = group < 256 ? 256 : group, rows = threads / group;
    const int64_t blocks = (static_cast<int64_t>(a.rows) + rows - 1) / rows;
    const int64_t most = static_cast<int64_t>(sms) * (1024 / threads);
    kernel<<<static_cast<unsigned>(std::min(blocks, most)), threads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (a.d <= 64) return go(rms_norm_kernel<DT, WIDE, 8, 1>, 8);
  if (a.d <= 128) return go(rms_norm_kernel<DT, WIDE, 16, 1>, 16);
  if (a.d <= 256) return go(rms_norm_kernel<DT, WIDE, 32, 1>, 32);
  if (a.d <= 512) return go(rms_norm_kernel<DT, WIDE, 32, 2>, 32);
  if (a.d <= 2048) return go(rms_norm_kernel<DT, WIDE, 256, 1>, 256);
  if (a.d <= 4096) return go(rms_norm_kernel<DT, WIDE, 256, 2>, 256);
  if (a.d <= 8192) return go(rms_norm_kernel<DT, WIDE, 512, 2>, 512);
  if (a.d <= 16384) return go(rms_norm_kernel<DT, WIDE, 1024, 2>, 1024);
  return go(rms_norm_kernel<DT, WIDE, 1024, 4>, 1024);
}

bool al2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

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
  NormArgs a = {};
  a.x = static_cast<const char *>(x->data);
  bool wide = view_wide(x, &a.xo, &a.xi) && d % 8 == 0 &&
              (reinterpret_cast<uintptr_t>(weight) & 15u) == 0 && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0;
  if (residual) {
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
