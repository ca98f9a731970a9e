// dt_cache_attn.cu -- attention of tree, chain and single-token rows over the paged
// cache: the kernel for head sizes above 128 (whose operands do not fit the others'
// tiles), the launch that joins partial results, and the entry points.
//
// One pass over the keys with a running maximum: per key tile S = Q K^T, x = S scale
// log2(e) (-inf where the row does not see the key), m' = max(m, max x),
// p = 2^(x - m'), l = l 2^(m - m') + sum p, O = O 2^(m - m') + p V; out = O / l. Sums, m, l
// and O are fp32; p is rounded to the 16-bit type for the product with V (bf16:
// relative 2^-8; fp16 2^-11, p scaled by 2^12 so that small weights stay normal
// numbers; fp16 over 8-bit rows two bf16 terms), l sums the unrounded p.
//
// Products are mma.sync m16n8k16, a warp's 16 rows by the tile's keys, and the copies of
// the next tile run during this one's. Measured at head size 256, 16 requests at 4096 keys,
// 16 / 4 heads: single tokens 92 us (2.9 TB/s of bf16 rows; 8-bit rows 158 us, with fp16
// queries, whose weights are two products, 205 us), trees of 16 rows 242 us, of 65 rows 0.97 ms
// (72 TFLOP/s; 8-bit rows 1.20 ms, 1.53 ms). Bound by latency: four warps a block, one block
// an SM at this head size, and 8-bit rows converted in between.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dt_cache_attn.cuh"
#include "dt_internal.h"
#include "dt_umma.cuh"

namespace dt {

bool heads_ok(const dt_heads *x);
int check_cache(const dt_cache *c);
bool cache_dtype_ok(const dt_cache *c, int dtype);

namespace {

constexpr int kNThreads = 128;
constexpr int kJoinThreads = 512;      // 8 rows of 256 values, 4 each
constexpr int kT = 64;                 // keys of a tile

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <int DT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (DT == DT_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// byte offset of 16-byte chunk c of row r in a tile of DH 16-bit values a row: chunks
// are permuted by the row so that eight rows' same chunk lie in eight bank groups
template <int DH>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * (DH * 2) + ((c ^ (r & 7)) << 4));
}

// non-finite 16-bit values of either type
template <int DT>
__device__ __forceinline__ uint32_t odd16(uint32_t w) {
  const uint32_t e = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
  return ((w & e) == e ? 0xffffu : 0u) | (((w >> 16) & e) == e ? 0xffff0000u : 0u);
}

template <int DH, bool QUANT>
constexpr int narrow_smem(int bm) {
  // two stages of K and V as they are stored, for 8-bit rows the 16-bit tiles too, Q
  return 2 * 2 * kT * DH * (QUANT ? 1 : 2) + (QUANT ? 2 * kT * DH * 2 : 0) + bm * DH * 2;
}

// Four warps: 4 / WK row groups of 16 query rows, the keys of a tile cut over WK warps
// of each (few rows: WK = 4, so that no warp idles and single tokens read their keys
// with all four).
template <int DT, bool QUANT, int DH, int WK>
__global__ void __launch_bounds__(kNThreads)
cache_attention_kernel(const __grid_constant__ AttnArgs a) {
  // fp16 rows over 8-bit ones: V's values (as many as 2^137 apart) in bf16, where they are
  // exact, against the weights in two bf16 terms; K's in fp16, rounded as dt_cache_read does
  constexpr bool TWO = QUANT && DT == DT_F16;
  constexpr int VDT = TWO ? DT_BF16 : DT;
  constexpr int BM = 64 / WK, NK = kT / WK, C8 = DH / 8;
  constexpr int RB = DH * (QUANT ? 1 : 2);      // bytes of a stored row (padded)
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ int64_t s_scan[kNThreads / 32 + 2];
  __shared__ int s_bad, s_odd;
  __shared__ uint8_t s_exp[2][2][kT];
  unsigned char *sStage = sm;                                  // [2][K, V][kT][RB]
  unsigned char *sDeq = sStage + 4 * kT * RB;                  // [K, V][kT][DH] 16-bit
  unsigned char *sQ = sDeq + (QUANT ? 2 * kT * DH * 2 : 0);    // [BM][DH]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wr = warp / WK, wk = warp % WK, g = lane >> 2, t4 = lane & 3;
  const float ninf = -__int_as_float(0x7f800000);
  constexpr float kShift = VDT == DT_F16 ? 12.0f : 0.0f;
  const int dh = a.c.dh;

  Schedule<kNThreads> sch;
  sch.plan(a, BM, kT, s_scan);
  Walk walk;
  Segment sg;
  walk.at = blockIdx.x * sch.chunk;
  walk.stop = min(walk.at + sch.chunk, sch.total);
  if (walk.at < walk.stop) sch.find(a, BM, kT, walk.at, s_scan, &walk.b, &walk.base);
  bool more = walk.next(a, BM, kT, &sg);
  if (tid == 0) walk.note_cut(a, sch.chunk, more, sg);

  for (; more; more = walk.next(a, BM, kT, &sg)) {
    const int b = sg.b, hk = sg.hk, rt = sg.rt, t0 = sg.t0, t1 = sg.t1;
    const Request rq = sg.rq;
    const int64_t end = sg.end;
    const int rows = a.n * a.G;

    // (s_bad was last read before the barrier that ended the last unit's last tile; cleared
    // before this one, it cannot be cleared after a warp's stage() has set it)
    if (tid == 0) s_bad = 0;
    __syncthreads();   // the last unit's shared memory is free
    if (tid == 0 && a.prefix[b] != rq.pre) cache_fault(a.c, b);
    for (int u = tid; u < BM * C8; u += kNThreads) {
      const int r = u / C8, c = u - r * C8, gr = rt * BM + r;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (gr < rows && c * 8 < dh) {
        const int i = gr / a.G, h = hk * a.G + gr % a.G;
        x = *reinterpret_cast<const uint4 *>(a.q + b * a.qb + h * a.qh + i * a.qr + c * 16);
      }
      *reinterpret_cast<uint4 *>(sQ + swz<DH>(r, c)) = x;
    }
    // this thread's two query rows
    int tok[2];
    bool live[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int gr = rt * BM + wr * 16 + g + 8 * y;
      tok[y] = gr / a.G;
      live[y] = gr < rows && tok[y] < rq.count;
    }
    // A warp copies 16 rows of the tile, kRows at a time: lane k < 16 looks the k-th of them
    // up, and (8-bit rows) loads its exponents, which note() leaves in shared memory.
    constexpr int CR = RB / 16, kRows = 32 / CR;         // 16-byte chunks of a row
    auto row_of = [&](int k) { return (kNThreads / 32 * (k / kRows) + warp) * kRows + k % kRows; };
    uint32_t ek = 127u, ev = 127u;
    auto stage = [&](int t) {
      unsigned char *sk = sStage + (t & 1) * 2 * kT * RB, *sv = sk + kT * RB;
      const int64_t j = static_cast<int64_t>(t) * kT + row_of(lane & 15);
      int64_t mine = -1;
      if (j < end) {
        mine = cache_row(a.c, b, j, hk);
        if (mine < 0) {
          s_bad = 1;
          cache_fault(a.c, b);
        }
      }
      if (QUANT) {
        ek = mine < 0 ? 127u : a.c.k_exp[mine];
        ev = mine < 0 ? 127u : a.c.v_exp[mine];
      }
      const int c = lane % CR;
      const bool column = c * 16 < dh * (QUANT ? 1 : 2);
#pragma unroll
      for (int i = 0; i < 16 / kRows; ++i) {
        const int k = i * kRows + lane / CR, r = row_of(k);
        const int64_t row = __shfl_sync(kFull, mine, k);
        const bool read = row >= 0 && column;
        const int64_t off = read ? row * dh * (QUANT ? 1 : 2) + c * 16 : 0;
        const uint32_t n16 = read ? 16u : 0u;
        const uint32_t to = QUANT ? static_cast<uint32_t>(r * RB + c * 16) : swz<DH>(r, c);
        cp_async16(sk + to, static_cast<const char *>(a.c.k) + off, n16);
        cp_async16(sv + to, static_cast<const char *>(a.c.v) + off, n16);
      }
      cp_async_commit();
    };
    auto note = [&](int t) {
      if (QUANT && lane < 16) {
        s_exp[t & 1][0][row_of(lane)] = static_cast<uint8_t>(ek);
        s_exp[t & 1][1][row_of(lane)] = static_cast<uint8_t>(ev);
      }
    };

    float o[DH / 8][4];
#pragma unroll
    for (int x = 0; x < DH / 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[x][y] = 0.0f;
    float m[2] = {ninf, ninf}, l[2] = {0.0f, 0.0f};

    stage(t0);
    note(t0);
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) {
        stage(t + 1);
        cp_async_wait_group<1>();
      } else {
        cp_async_wait_all();
      }
      if (tid == 0) s_odd = 0;
      __syncthreads();
      unsigned char *sK = sStage + (t & 1) * 2 * kT * RB, *sV = sK + kT * RB;
      const int64_t j0 = static_cast<int64_t>(t) * kT;
      if (QUANT) {   // codes to 16-bit values
        // (a row that is not there, or a column past dh, has codes of zero)
#pragma unroll 4
        for (int u = tid; u < 2 * kT * C8; u += kNThreads) {
          const int which = u / (kT * C8), r = (u / C8) % kT, c = u % C8;
          const float sc = row_scale(s_exp[t & 1][which][r]);
          const uint2 q = *reinterpret_cast<const uint2 *>((which ? sV : sK) + r * RB + c * 8);
          auto to16 = [&](uint32_t two) {
            return TWO && which ? e4m3_to16<VDT>(two, sc) : e4m3_to16<DT>(two, sc);
          };
          uint4 w;
          w.x = to16(q.x & 0xffffu);
          w.y = to16(q.x >> 16);
          w.z = to16(q.y & 0xffffu);
          w.w = to16(q.y >> 16);
          *reinterpret_cast<uint4 *>(sDeq + which * kT * DH * 2 + swz<DH>(r, c)) = w;
        }
        __syncthreads();
        sK = sDeq;
        sV = sDeq + kT * DH * 2;
      }
      const bool tree = j0 + kT > rq.pre;   // the tile holds rows that not every row sees
      if (tree) {
        // a weight of zero times a value that is not finite is NaN: such values
        // leave the tile and are added, below, to the rows that see them
        for (int u = tid; u < kT * C8; u += kNThreads) {
          uint32_t *w = reinterpret_cast<uint32_t *>(sV + u * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t odd = odd16<VDT>(w[e]);
            if (odd) {
              w[e] &= ~odd;
              s_odd = 1;
            }
          }
        }
        __syncthreads();
      }
      const bool bad = s_bad != 0;
      auto visible = [&](int y, int key) {
        const int64_t j = j0 + key;
        return live[y] && j < end && (!tree || sees(a, rq, b, tok[y], j)) &&
               (!bad || cache_row(a.c, b, j, hk) >= 0);
      };

      float s[NK / 8][4];
#pragma unroll
      for (int x = 0; x < NK / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][y] = 0.0f;
      const uint32_t q_at = smem_u32(sQ), k_at = smem_u32(sK), v_at = smem_u32(sV);
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
        uint32_t qa[4];
        ldsm4(qa, q_at + swz<DH>(wr * 16 + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
        for (int x = 0; x < NK / 16; ++x) {
          uint32_t kb[4];   // keys 0-7 / 8-15 by dims 0-7 / 8-15 of the slice
          ldsm4(kb, k_at + swz<DH>(wk * NK + 16 * x + (lane & 7) + ((lane >> 4) << 3),
                                   2 * k + ((lane >> 3) & 1)));
          mma16816<DT>(s[2 * x], qa, kb[0], kb[1]);
          mma16816<DT>(s[2 * x + 1], qa, kb[2], kb[3]);
        }
      }
      const bool all = !tree && !bad && j0 + kT <= end;
      float mx[2] = {ninf, ninf};
#pragma unroll
      for (int x = 0; x < NK / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const bool v = all ? live[y >> 1] : visible(y >> 1, wk * NK + 8 * x + 2 * t4 + (y & 1));
          s[x][y] = v ? s[x][y] * a.scale_log2 : ninf;
          mx[y >> 1] = fmaxf(mx[y >> 1], s[x][y]);
        }
      float f[2], ref[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        mx[y] = fmaxf(mx[y], __shfl_xor_sync(kFull, mx[y], 1));
        mx[y] = fmaxf(mx[y], __shfl_xor_sync(kFull, mx[y], 2));
        const float mn = fmaxf(m[y], mx[y]);
        f[y] = mn == ninf ? 1.0f : fast_exp2(m[y] - mn);   // nothing seen yet: all is zero
        ref[y] = mn == ninf ? 0.0f : mn - kShift;
        m[y] = mn;
        l[y] *= f[y];
      }
#pragma unroll
      for (int x = 0; x < NK / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          s[x][y] = fast_exp2(s[x][y] - ref[y >> 1]);
          l[y >> 1] += s[x][y];
        }
#pragma unroll
      for (int x = 0; x < DH / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[x][y] *= f[y >> 1];
#pragma unroll
      for (int kb = 0; kb < NK / 16; ++kb) {
        uint32_t pa[4], pl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = s[2 * kb + (e >> 1)][2 * (e & 1)], p1 = s[2 * kb + (e >> 1)][2 * (e & 1) + 1];
          pa[e] = Half16<VDT>::pack(p0, p1);
          if (TWO) {
            const float2 hi = Half16<VDT>::unpack(pa[e]);
            pl[e] = Half16<VDT>::pack(p0 - hi.x, p1 - hi.y);
          }
        }
#pragma unroll
        for (int x = 0; x < DH / 16; ++x) {
          uint32_t vb[4];
          ldsm4t(vb, v_at + swz<DH>(wk * NK + 16 * kb + (lane & 15), 2 * x + (lane >> 4)));
          mma16816<VDT>(o[2 * x], pa, vb[0], vb[1]);
          mma16816<VDT>(o[2 * x + 1], pa, vb[2], vb[3]);
          if (TWO) {
            mma16816<VDT>(o[2 * x], pl, vb[0], vb[1]);
            mma16816<VDT>(o[2 * x + 1], pl, vb[2], vb[3]);
          }
        }
      }
      if (tree && s_odd) {
        for (int key = wk * NK; key < (wk + 1) * NK; ++key) {
          const int64_t row = j0 + key < end ? cache_row(a.c, b, j0 + key, hk) : -1;
          if (row < 0) continue;
          const bool v0 = visible(0, key), v1 = visible(1, key);
#pragma unroll
          for (int x = 0; x < DH / 8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int col = 8 * x + 2 * t4 + y;
              if (col >= dh) continue;
              float v;
              if (QUANT) {
                v = row_scale(a.c.v_exp[row]);     // NaN, or the row is finite
              } else {
                const uint16_t w = static_cast<const uint16_t *>(a.c.v)[row * dh + col];
                v = odd16<DT>(w) & 0xffffu ? Half16<DT>::unpack(w).x : 0.0f;
              }
              if (v - v != 0.0f || v != v) {
                if (v0) o[x][y] += v;
                if (v1) o[x][2 + y] += v;
              }
            }
        }
      }
      if (t + 1 < t1) note(t + 1);
      __syncthreads();   // the stage is free
    }

    // the warps' results through shared memory: [BM][WK] maxima and sums, [WK][BM][DH]
    float *sO = reinterpret_cast<float *>(sm);
    __shared__ float s_m[64], s_l[64];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] += __shfl_xor_sync(kFull, l[y], 1);
      l[y] += __shfl_xor_sync(kFull, l[y], 2);
      const int r = wr * 16 + g + 8 * y;
      if (t4 == 0) {
        s_m[wk * BM + r] = m[y];
        s_l[wk * BM + r] = l[y];
      }
#pragma unroll
      for (int x = 0; x < DH / 8; ++x)
        *reinterpret_cast<float2 *>(sO + (wk * BM + r) * DH + 8 * x + 2 * t4) =
            make_float2(o[x][2 * y], o[x][2 * y + 1]);
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == sg.tiles;
    float *pp = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (t0 > 0 ? 0 : 1)) * 2 * a.slot;
    constexpr int C4 = DH / 8;
    for (int u = tid; u < BM * C4; u += kNThreads) {
      const int r = u / C4, c = u - r * C4, gr = rt * BM + r;
      float mm = ninf, ll = 0.0f, w[WK], acc[8];
#pragma unroll
      for (int k = 0; k < WK; ++k) mm = fmaxf(mm, s_m[k * BM + r]);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        // A row that saw nothing has -inf and 0, and its values may be anything: a row past
        // the count has a weight of zero for every key of the prefix, zero times a value
        // that is not finite is NaN. (A sum that is NaN is not nothing.)
        if (s_m[k * BM + r] == ninf && s_l[k * BM + r] == 0.0f) continue;
        w[k] = fast_exp2(s_m[k * BM + r] - mm);
        ll += w[k] * s_l[k * BM + r];
        const float *src = sO + (k * BM + r) * DH + c * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += w[k] * src[e];
      }
      if (!whole) {
        *reinterpret_cast<float4 *>(pp + r * DH + c * 8) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4 *>(pp + r * DH + c * 8 + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c == 0) {
          pp[BM * DH + r] = mm;
          pp[BM * DH + BM + r] = ll;
        }
      } else if (gr < rows && c * 8 < dh) {
        const float inv = ll > 0.0f ? 1.0f / ll : ll == ll ? 0.0f : ll;
        uint4 x;
        x.x = Half16<DT>::pack(acc[0] * inv, acc[1] * inv);
        x.y = Half16<DT>::pack(acc[2] * inv, acc[3] * inv);
        x.z = Half16<DT>::pack(acc[4] * inv, acc[5] * inv);
        x.w = Half16<DT>::pack(acc[6] * inv, acc[7] * inv);
        const int i = gr / a.G, h = hk * a.G + gr % a.G;
        *reinterpret_cast<uint4 *>(a.out + b * a.ob + h * a.oh + i * a.orow + c * 16) = x;
      }
    }
  }
}

// Joins the partial results of units that were cut over blocks. A block for kJoinRows
// rows of the unit that block blockIdx.x's part of the line begins within, if it is the
// first to continue it: a thread has 4 values of a row, all parts' weights before all
// parts' values, so that the loads wait for each other twice, not once a part.
// Launched early, it waits on the device for the first kernel's end: 24.8 us to 22.7 us
// for one tree of 33 rows, 2 to 3 us a call at any size.
constexpr int kJoinRows = 8;
template <int DT>
__global__ void __launch_bounds__(kJoinThreads)
cache_attention_join_kernel(const __grid_constant__ AttnArgs a, int BM, int DH) {
  cudaGridDependencySynchronize();
  const int4 unit = a.cut[2 * blockIdx.x], blocks = a.cut[2 * blockIdx.x + 1];
  if (unit.x < 0 || blocks.x + 1 != static_cast<int>(blockIdx.x)) return;
  const int b = unit.x, hk = unit.y, rt = unit.z;
  const float ninf = -__int_as_float(0x7f800000);
  const int C4 = DH / 4, r = blockIdx.y * kJoinRows + threadIdx.x / C4, c = threadIdx.x % C4;
  const int gr = rt * BM + r;
  if (r >= min(BM, static_cast<int>(blockIdx.y + 1) * kJoinRows) || gr >= a.n * a.G || c * 4 >= a.c.dh) return;
  // a shared unit has a part of either group of warps in a block; a block's last unit is
  // in its second place, the one that it began within in its first
  const int per = a.odd && rt == a.row_tiles - 1 ? 2 : 1, parts = (blocks.y - blocks.x + 1) * per;
  auto part = [&](int x) {
    const int k = blocks.x + (per == 2 ? x >> 1 : x), g = per == 2 ? x & 1 : 0;
    return a.part + ((static_cast<int64_t>(k) * 2 + (k > blocks.x ? 0 : 1)) * 2 + g) * a.slot;
  };
  float m = ninf;
#pragma unroll 4
  for (int x = 0; x < parts; ++x) m = fmaxf(m, part(x)[BM * DH + r]);
  float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int x = 0; x < parts; ++x) {
    const float *pp = part(x);
    const float pm = pp[BM * DH + r], pl = pp[BM * DH + BM + r];
    const float4 po = *reinterpret_cast<const float4 *>(pp + r * DH + c * 4);
    if (pm == ninf && pl == 0.0f) continue;     // saw nothing; its values are not written
    const float e = fast_exp2(pm - m);
    l += pl * e;
    o[0] += po.x * e;
    o[1] += po.y * e;
    o[2] += po.z * e;
    o[3] += po.w * e;
  }
  const float inv = l > 0.0f ? 1.0f / l : l == l ? 0.0f : l;
  const int i = gr / a.G, h = hk * a.G + gr - i * a.G;
  *reinterpret_cast<uint2 *>(a.out + b * a.ob + h * a.oh + i * a.orow + c * 8) =
      make_uint2(Half16<DT>::pack(o[0] * inv, o[1] * inv), Half16<DT>::pack(o[2] * inv, o[3] * inv));
}

template <int DT, bool QUANT, int DH, int WK>
cudaError_t launch_narrow(const AttnArgs &a, cudaStream_t st) {
  constexpr int BM = 64 / WK;
  const int smem = narrow_smem<DH, QUANT>(BM);
  const cudaError_t e = allow_smem<cache_attention_kernel<DT, QUANT, DH, WK>>();
  if (e != cudaSuccess) return e;
  cache_attention_kernel<DT, QUANT, DH, WK><<<a.grid, kNThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_join(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
  // launched while the first kernel still runs; waits for its end on the device
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(a.grid, (p.bm + kJoinRows - 1) / kJoinRows);
  config.blockDim = dim3(kJoinRows * p.dhp / 4);
  config.stream = st;
  config.attrs = &early;
  config.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&config, cache_attention_join_kernel<DT>, a, p.bm, p.dhp);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int DT, bool QUANT>
cudaError_t launch_any(const AttnArgs &a, int bm, cudaStream_t st) {
  return bm == 16   ? launch_narrow<DT, QUANT, 256, 4>(a, st)
         : bm == 32 ? launch_narrow<DT, QUANT, 256, 2>(a, st)
                    : launch_narrow<DT, QUANT, 256, 1>(a, st);
}

int64_t slot_floats(const AttnPlan &p) {
  return (static_cast<int64_t>(p.bm) * (p.dhp + 2) + 7) / 8 * 8;
}
size_t plan_bytes(const AttnPlan &p) {
  return static_cast<size_t>(p.grid) * (2 * sizeof(int4) + 6 * slot_floats(p) * sizeof(float));
}

bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

// What a call launches, from its sizes and types alone.
int attn_plan(const dt_cache &c, int H, int n, AttnPlan *p) {
  int sms = 0, smem = 0;
  const int rc = device_sm_count(&sms, &smem);
  if (rc) return rc;
  const int64_t rows = static_cast<int64_t>(n) * (H / c.Hkv);
  *p = {};
  if (!few_plan(c, rows, sms, smem, p) && !wide_plan(c, rows, sms, smem, p)) {
    *p = {};
    p->dhp = 256;
    p->bm = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    p->row_tiles = static_cast<int>((rows + p->bm - 1) / p->bm);
    p->grid = sms;
  }
  p->bytes = plan_bytes(*p);
  return DT_OK;
}

}  // namespace dt

extern "C" {

size_t dt_cache_attention_workspace_bytes(const dt_cache *c, int H, int n) {
  dt::AttnPlan p;
  if (dt::check_cache(c) || H < 1 || H % c->Hkv || n < 1 || n > 65536 || dt::attn_plan(*c, H, n, &p))
    return 0;
  // Units of two row tiles are as long as the rows divide: 65 x 4 stacked rows take units of
  // 174, 64 x 4 take 256. The size is that of the largest that so many rows or fewer take, so
  // that a workspace serves every smaller call.
  if (p.kind == dt::AttnPlan::kWide)
    p.bm = 2 * static_cast<int>(std::min<int64_t>(static_cast<int64_t>(n) * (H / c->Hkv), 128));
  return dt::plan_bytes(p);
}

int dt_cache_attention(const dt_cache *c, const dt_heads *q, int n, int dtype,
                       const int32_t *prefix_len, const int32_t *counts, const uint8_t *mask,
                       float scale, const dt_heads *out, void *workspace, size_t workspace_bytes,
                       void *stream) {
  if (dt::check_cache(c) || !dt::cache_dtype_ok(c, dtype) || !dt::heads_ok(q) || !dt::heads_ok(out) ||
      q->heads != out->heads || q->heads % c->Hkv || n < 1 || n > (mask ? DT_MAX_N + 1 : 65536) ||
      !prefix_len || !dt::al4(prefix_len) || !dt::al4(counts) || !std::isfinite(scale) ||
      !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return DT_ERR_INVALID_ARG;
  const int G = q->heads / c->Hkv;
  dt::AttnPlan p;
  const int rc = dt::attn_plan(*c, q->heads, n, &p);
  if (rc) return rc;
  if (static_cast<int64_t>(n) * G > (1 << 24) ||
      static_cast<int64_t>(c->batch) * c->Hkv * p.row_tiles > 0x7fffffff || workspace_bytes < p.bytes)
    return DT_ERR_INVALID_ARG;
  dt::AttnArgs a = {};
  a.c = dt::cache_view(*c);
  a.q = static_cast<const char *>(q->data);
  a.out = static_cast<char *>(out->data);
  a.qb = 2 * q->stride_batch; a.qh = 2 * q->stride_head; a.qr = 2 * q->stride_row;
  a.ob = 2 * out->stride_batch; a.oh = 2 * out->stride_head; a.orow = 2 * out->stride_row;
  a.prefix = prefix_len; a.counts = counts; a.mask = mask;
  a.cut = static_cast<int4 *>(workspace);
  a.part = reinterpret_cast<float *>(a.cut + 2 * p.grid);
  // (a scale of zero: all weights equal, and -inf times it still -inf)
  a.scale_log2 = scale == 0.0f ? 1e-38f : scale * 1.4426950408889634f;
  a.batch = c->batch; a.n = n; a.G = G;
  a.row_tiles = p.row_tiles; a.grid = p.grid; a.min_tiles = 2;
  a.slot = dt::slot_floats(p);
  a.odd = p.odd;
  const bool wide = p.kind == dt::AttnPlan::kWide;
  a.weight = wide ? 2 : 1;
  a.last_weight = wide && p.odd ? 1 : a.weight;
  a.lead = wide ? dt::kWideLead : 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool quant = c->dtype == DT_E4M3;
  cudaError_t e =
      wide ? dt::launch_wide(*c, a, dtype, p, st)
      : p.kind == dt::AttnPlan::kFew ? dt::launch_few(*c, a, dtype, p, st)
      : dtype == DT_BF16 ? (quant ? dt::launch_any<DT_BF16, true>(a, p.bm, st) : dt::launch_any<DT_BF16, false>(a, p.bm, st))
                         : (quant ? dt::launch_any<DT_F16, true>(a, p.bm, st) : dt::launch_any<DT_F16, false>(a, p.bm, st));
  if (e == cudaSuccess)
    e = dtype == DT_BF16 ? dt::launch_join<DT_BF16>(a, p, st) : dt::launch_join<DT_F16>(a, p, st);
  return e == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // extern "C"
