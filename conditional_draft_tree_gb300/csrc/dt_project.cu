// dt_project.cu -- a projection that many requests share, with low-rank adapters of their
// own beside it: y = x W^T + scale_a (x A_a^T) B_a^T for the rows of a request with adapter a.
#include <algorithm>
#include <cstdint>

#include "dt_cache.cuh"
#include "dt_internal.h"

namespace dt {

namespace {

struct ProjectArgs {
  const char *w, *x, *x16, *down, *up;
  const uint8_t *w_exps, *x_exps;
  const float *scale;
  const int32_t *index;
  char *y;
  uint16_t *u;           // [rows][rank]: scale x A^T, rounded
  int32_t *status;
  int64_t ldw, ldx, ldx16, ldy;    // in bytes
  int rows, n, O, K, count, rank;
};

template <int DT>
__device__ __forceinline__ float value16(const char *p, int64_t i) {
  const uint32_t v = *reinterpret_cast<const uint16_t *>(p + 2 * i);
  return Half16<DT>::unpack(v).x;
}
__device__ __forceinline__ float value8(const char *p, int64_t i) {
  return Half16<DT_F16>::unpack(e4m3_f16x2(*reinterpret_cast<const uint8_t *>(p + i))).x;
}

// u = scale x A^T of a row, a warp for each of the adapter's ranks in turn.
template <int DT>
__global__ void __launch_bounds__(256) adapter_down_kernel(const __grid_constant__ ProjectArgs a) {
  const int row = blockIdx.x, lane = threadIdx.x & 31;
  const int at = a.index[row / a.n];
  if (at >= a.count && threadIdx.x == 0) *a.status = DT_ERR_BAD_INDEX;
  if (at < 0 || at >= a.count) return;
  const char *x = a.x16 + row * a.ldx16;
  for (int j = threadIdx.x >> 5; j < a.rank; j += 8) {
    const char *d = a.down + 2 * (static_cast<int64_t>(at) * a.rank + j) * a.K;
    float s = 0.0f;
    for (int k = lane; k < a.K; k += 32) s += value16<DT>(x, k) * value16<DT>(d, k);
    s = warp_sum(s) * (a.scale ? a.scale[at] : 1.0f);
    if (lane == 0) a.u[static_cast<int64_t>(row) * a.rank + j] = static_cast<uint16_t>(Half16<DT>::pack(s, 0.0f));
  }
}

// 64 rows x 64 outputs a block, 4 x 4 a thread, 32 values of K at a time.
template <int DT, bool E8>
__global__ void __launch_bounds__(256) project_kernel(const __grid_constant__ ProjectArgs a) {
  __shared__ float s_x[32][65], s_w[32][65];
  const int tid = threadIdx.x, r0 = blockIdx.y * 64, o0 = blockIdx.x * 64;
  const int ty = tid / 16, tx = tid % 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    for (int i = tid; i < 64 * 32; i += 256) {
      const int r = i / 32, k = i % 32;
      float x = 0.0f, w = 0.0f;
      if (k0 + k < a.K && r0 + r < a.rows) {
        const char *p = a.x + (r0 + r) * a.ldx;
        x = E8 ? value8(p, k0 + k) : value16<DT>(p, k0 + k);
      }
      if (k0 + k < a.K && o0 + r < a.O) {
        const char *p = a.w + (o0 + r) * a.ldw;
        w = E8 ? value8(p, k0 + k) : value16<DT>(p, k0 + k);
      }
      s_x[k][r] = x;
      s_w[k][r] = w;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += s_x[k][ty + 16 * i] * s_w[k][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty + 16 * i, o = o0 + tx + 16 * j;
      if (r >= a.rows || o >= a.O) continue;
      float y = acc[i][j];
      if (E8) y = y * row_scale(a.x_exps[r]) * row_scale(a.w_exps[o]);
      const int at = a.index ? a.index[r / a.n] : -1;
      if (at >= 0 && at < a.count) {
        const char *up = a.up + 2 * (static_cast<int64_t>(at) * a.O + o) * a.rank;
        for (int k = 0; k < a.rank; ++k)
          y += value16<DT>(reinterpret_cast<const char *>(a.u + static_cast<int64_t>(r) * a.rank), k) * value16<DT>(up, k);
      }
      *reinterpret_cast<uint16_t *>(a.y + r * a.ldy + 2 * o) = static_cast<uint16_t>(Half16<DT>::pack(y, 0.0f));
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int DT>
cudaError_t launch_project(const ProjectArgs &a, bool e8, cudaStream_t st) {
  if (a.index) {
    adapter_down_kernel<DT><<<a.rows, 256, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((a.O + 63) / 64, (a.rows + 63) / 64);
  if (grid.y > 65535) return cudaErrorInvalidConfiguration;
  if (e8) project_kernel<DT, true><<<grid, 256, 0, st>>>(a);
  else project_kernel<DT, false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

}  // namespace dt

extern "C" {

size_t dt_project_workspace_bytes(int batch, int n, int rank) {
  if (batch < 1 || batch > 65535 || n < 1 || static_cast<int64_t>(batch) * n > (1 << 24) || rank < 16 ||
      rank > 128 || rank % 16)
    return 0;
  return (static_cast<size_t>(batch) * n * rank * 2 + 255) / 256 * 256;
}

int dt_project(const dt_matrix *w, const void *x, int64_t ldx, const uint8_t *x_exps, int batch,
               int n, int dtype, const dt_adapters *adapters, const int32_t *index,
               const void *x16, int64_t ldx16, void *y, int64_t ldy, int32_t *status,
               void *workspace, size_t workspace_bytes, void *stream) {
  if (!w || !w->data || !x || !y || !status || !dt::al16(w->data) || !dt::al16(x) ||
      (reinterpret_cast<uintptr_t>(y) & 1u) || (reinterpret_cast<uintptr_t>(status) & 3u) ||
      batch < 1 || batch > 65535 || n < 1 || static_cast<int64_t>(batch) * n > (1 << 24) ||
      !(dtype == DT_BF16 || dtype == DT_F16) || !(w->dtype == dtype || w->dtype == DT_E4M3) ||
      w->K < 16 || w->K > 65536 || w->K % 16 || w->O < 1 || w->O > (1 << 24))
    return DT_ERR_INVALID_ARG;
  const bool e8 = w->dtype == DT_E4M3;
  const int64_t size = e8 ? 1 : 2, rows = static_cast<int64_t>(batch) * n, most = int64_t{1} << 32;
  if (w->ld < w->K || w->ld * size % 16 || w->ld > most || ldx < w->K || ldx * size % 16 || ldx > most ||
      ldy < w->O || ldy > most || e8 != (w->exps != nullptr) || e8 != (x_exps != nullptr))
    return DT_ERR_INVALID_ARG;
  if (!adapters != !index || (!adapters || !e8) != !x16) return DT_ERR_INVALID_ARG;
  dt::ProjectArgs a = {};
  a.w = static_cast<const char *>(w->data);
  a.x = static_cast<const char *>(x);
  a.y = static_cast<char *>(y);
  a.w_exps = w->exps;
  a.x_exps = x_exps;
  a.status = status;
  a.ldw = w->ld * size;
  a.ldx = ldx * size;
  a.ldy = 2 * ldy;
  a.rows = static_cast<int>(rows);
  a.n = n;
  a.O = w->O;
  a.K = w->K;
  if (adapters) {
    if (!adapters->down || !adapters->up || !dt::al16(adapters->down) || !dt::al16(adapters->up) ||
        (reinterpret_cast<uintptr_t>(adapters->scale) & 3u) || adapters->count < 1 ||
        adapters->count > (1 << 20) || adapters->rank < 16 || adapters->rank > 128 || adapters->rank % 16 ||
        (reinterpret_cast<uintptr_t>(index) & 3u) || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < dt_project_workspace_bytes(batch, n, adapters->rank) ||
        static_cast<int64_t>(adapters->count) * w->O > 0x7fffffff)
      return DT_ERR_INVALID_ARG;
    if (e8 && (!dt::al16(x16) || ldx16 < w->K || ldx16 % 8 || ldx16 > most)) return DT_ERR_INVALID_ARG;
    a.x16 = e8 ? static_cast<const char *>(x16) : a.x;
    a.ldx16 = e8 ? 2 * ldx16 : a.ldx;
    a.down = static_cast<const char *>(adapters->down);
    a.up = static_cast<const char *>(adapters->up);
    a.scale = adapters->scale;
    a.index = index;
    a.count = adapters->count;
    a.rank = adapters->rank;
    a.u = static_cast<uint16_t *>(workspace);
  }
  int sms, smem;
  const int rc = dt::device_sm_count(&sms, &smem);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DT_BF16 ? dt::launch_project<DT_BF16>(a, e8, st)
                                         : dt::launch_project<DT_F16>(a, e8, st);
  return e == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // extern "C"
