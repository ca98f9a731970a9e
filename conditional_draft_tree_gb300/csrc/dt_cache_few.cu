// dt_cache_few.cu -- attention over the paged cache for a few rows (single tokens, short
// chains: G heads x rows <= 16) and head sizes up to 128: bound by the cache's bytes.
//
// Each of twelve warps of a block streams keys of its own, 16 at a time (8-bit rows 32),
// through a ring of its own, filled by TMA through a 128-byte swizzled tensor map (16 rows
// lie in one page): no warp waits for another before the unit's end, and about 140 KB of an SM's shared
// memory are in flight (its share of the memory's bandwidth times latency is 45 KB). The
// products are mma.sync m16n8k16 with the query rows on the M side; the softmax is online,
// its reference renewed only when the maximum has grown by 2^8 (fp16: 2^4).
//
// 8-bit rows become operands in registers. The product with K sums over dimensions in any
// order that both sides share, so a thread takes 16 codes of a key at once, and e4m3 codes
// are exact in fp16: one conversion a pair, K's scale and the row's own (bf16 query rows are
// scaled to fp16 by a power of two: their values lose less than 2^-24 of the row's largest)
// multiply the score. V's codes come transposed from shared memory (8-bit ldmatrix: four
// consecutive keys of a column), are set in bf16 fields as they are, which makes them their
// value times 2^-120, and 2^120 and V's scale are part of the weight: p 2^(e - ref + 60),
// ref the largest exponent e so far (within 2^40), which keeps both in bf16's range; the
// result has that power of two taken out. fp16 results need weights of more than bf16's 8
// bits: two terms.
#include <cmath>
#include <cstdint>
#include <cuda.h>

#include "dt_cache_attn.cuh"
#include "dt_internal.h"
#include "dt_umma.cuh"

namespace dt {

namespace {

constexpr int kFWarps = 12, kFThreads = 32 * kFWarps;
template <bool QUANT> constexpr int kSub = QUANT ? 32 : 16;      // keys of a warp's step
constexpr int kT = kFewKeys;           // keys of a tile of the cut
constexpr int kMaxStages = 4;
constexpr int kMergeCols = 32;
constexpr long long kFWaitCycles = 4000000000ll;   // about 2 s

struct FewSmall {
  uint64_t full[kFWarps][kMaxStages];
  uint8_t exps[kFWarps][kMaxStages][2 * kSub<true>];     // K's and V's
  float m[kFWarps][16], l[kFWarps][16];
  float out[kFWarps][16][kMergeCols];
  int64_t scan[kFThreads / 32 + 2];
};

// bytes of a step's K (V) rows: blocks of 16 rows of 128 bytes
template <int DH, bool QUANT> constexpr int kHalfStage = QUANT ? 4096 : DH / 64 * 2048;

__device__ __forceinline__ bool few_wait(uint64_t *bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    if (done) return true;
    const long long t = clock64();
    if (it == 0) t0 = t;
    else if (t - t0 > kFWaitCycles) return false;
  }
}
__device__ __forceinline__ void few_tma(void *dst, const CUtensorMap *map, int x, int y, int z,
                                        uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

template <int DT>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

template <int DT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  const uint32_t e = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
  return ((w & e) == e ? 0xffffu : 0u) | (((w >> 16) & e) == e ? 0xffff0000u : 0u);
}

// a word's codes (0: lower two, 1: upper two) in bf16 fields: their values times 2^-120
template <int HALF>
__device__ __forceinline__ uint32_t codes_low(uint32_t w) {
  uint32_t r;   // byte, its sign eight times; twice
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(HALF ? 0xb3a2 : 0x9180));
  return (r << 4) & 0x87f087f0u;
}

template <int DT, bool QUANT, int DH, int RY>   // RY: rows of a thread, 1 for up to 8 rows, else 2
__global__ void __launch_bounds__(kFThreads, 1)
cache_attention_few_kernel(const __grid_constant__ AttnArgs a, int stages,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  constexpr int HS = kHalfStage<DH, QUANT>, BM = 16, SUB = kSub<QUANT>, NG = SUB / 16, QDT = QUANT ? DT_F16 : DT;
  constexpr float kShift = !QUANT && DT == DT_F16 ? 8.0f : 0.0f;
  constexpr float kGrow = !QUANT && DT == DT_F16 ? 4.0f : 8.0f;
  extern __shared__ __align__(1024) unsigned char sm[];
  FewSmall &ss = *reinterpret_cast<FewSmall *>(sm + kFWarps * stages * 2 * HS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int dh = a.c.dh;
  const float ninf = -__int_as_float(0x7f800000);
  unsigned char *ring = sm + warp * stages * 2 * HS;
  uint64_t *full = ss.full[warp];
  if (lane == 0)
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
  __syncwarp();

  Schedule<kFThreads> sch;
  sch.plan(a, BM, kT, ss.scan);
  Walk walk;
  Segment sg;
  walk.at = blockIdx.x * sch.chunk;
  walk.stop = min(walk.at + sch.chunk, sch.total);
  if (walk.at < walk.stop) sch.find(a, BM, kT, walk.at, ss.scan, &walk.b, &walk.base);
  bool more = walk.next(a, BM, kT, &sg);
  if (tid == 0) walk.note_cut(a, sch.chunk, more, sg);

  const int rows = a.n * a.G;
  uint32_t stage_in = 0, stage_out = 0, parity_out = 0;     // places in the ring
  bool failed = false;
  uint32_t there_in = 0;               // bit NG i + h: group h of 16 keys of place i is on a good page
  // the warp's step k of a segment: keys from t0 T + SUB (warp + 12 k); the number of its steps
  auto step_key = [&](const Segment &s, int k) { return s.t0 * kT + SUB * (warp + kFWarps * k); };
  auto seg_end = [&](const Segment &s) { return static_cast<int>(min(static_cast<int64_t>(s.t1) * kT, s.end)); };
  auto step_count = [&](const Segment &s) {
    const int left = seg_end(s) - step_key(s, 0);
    return left <= 0 ? 0 : (left + SUB * kFWarps - 1) / (SUB * kFWarps);
  };
  auto issue = [&](const Segment &s, int k) {
    const int j = step_key(s, k), end = seg_end(s);
    const int32_t *table = a.c.table + static_cast<int64_t>(s.b) * a.c.width;
    int entry[NG];
    uint32_t good = 0u;
#pragma unroll
    for (int h = 0; h < NG; ++h) {
      const int page = (j + 16 * h) >> a.c.shift;
      entry[h] = j + 16 * h < end ? (page < a.c.width ? table[page] : -1) : -2;
    }
#pragma unroll
    for (int h = 0; h < NG; ++h)
      if (static_cast<uint32_t>(entry[h]) < static_cast<uint32_t>(a.c.pages)) good |= 1u << h;
    there_in = (there_in & ~(((1u << NG) - 1u) << (NG * stage_in))) | good << (NG * stage_in);
    if (lane == 0) {
      uint64_t *bar = &full[stage_in];
      unsigned char *dst = ring + stage_in * 2 * HS;
      mbar_expect_tx(bar, __popc(good) * (2 * HS / NG + (QUANT ? 32 : 0)));
#pragma unroll
      for (int h = 0; h < NG; ++h) {
        if (!((good >> h) & 1u)) {
          if (entry[h] != -2) cache_fault(a.c, s.b);
          continue;
        }
        const int z = entry[h] * a.c.Hkv + s.hk, y = (j + 16 * h) & ((1 << a.c.shift) - 1);
#pragma unroll
        for (int kb = 0; kb < HS / NG / 2048; ++kb) {
          few_tma(dst + (h + kb) * 2048, &kmap, 64 * kb, y, z, bar);
          few_tma(dst + HS + (h + kb) * 2048, &vmap, 64 * kb, y, z, bar);
        }
        if (QUANT) {
          const int64_t row = (static_cast<int64_t>(z) << a.c.shift) + y;
          uint8_t *e = ss.exps[warp][stage_in] + 16 * h;
          bulk_g2s(e, a.c.k_exp + row, 16, bar);
          bulk_g2s(e + SUB, a.c.v_exp + row, 16, bar);
        }
      }
    }
    if (++stage_in == static_cast<uint32_t>(stages)) stage_in = 0;
  };
  if (more)
    for (int k = 0; k < min(stages, step_count(sg)); ++k) issue(sg, k);

  while (more) {
    const Request rq = sg.rq;
    const int b = sg.b, hk = sg.hk, pre = static_cast<int>(rq.pre), end = seg_end(sg);
    const int steps = step_count(sg);
    if (tid == 0 && a.prefix[b] != rq.pre) cache_fault(a.c, b);
    // this thread's query rows, and its part of them
    int tok[RY], head[RY];
    bool live[RY];
    float row_mul[RY];
    uint32_t q[DH / 16][4];
#pragma unroll
    for (int y = 0; y < RY; ++y) {
      const int r = g + 8 * y;
      tok[y] = r / a.G;
      head[y] = hk * a.G + r - tok[y] * a.G;
      live[y] = r < rows && tok[y] < rq.count;
      row_mul[y] = a.scale_log2;
      const char *src = a.q + b * a.qb + head[y] * a.qh + tok[y] * a.qr;
      uint32_t w[DH / 8];
      // 16 bytes at dimension 32 c + 8 t (a key's chunk c, t of 8 values), or 32 bytes at 64 c + 16 t
#pragma unroll
      for (int c = 0; c < DH / 32; ++c) {
        const int d = QUANT ? 64 * (c >> 1) + 16 * t4 + 8 * (c & 1) : 32 * c + 8 * t4;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows && d < dh) x = *reinterpret_cast<const uint4 *>(src + 2 * d);
        w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
      }
      if (QUANT && DT == DT_BF16) {
        // to fp16, the row's largest value in [1, 2) (a row that is not finite: as it is)
        uint32_t mx = 0u;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) mx = max(mx, max(w[c] & 0x7fffu, (w[c] >> 16) & 0x7fffu));
        mx = max(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = max(mx, __shfl_xor_sync(kFull, mx, 2));
        const int e = mx >= 0x7f80u || mx < 0x80u ? 0 : static_cast<int>(mx >> 7) - 127;
        const float down = exp2i(max(-e, -126)), up = e == 127 ? 0x1p126f : exp2i(max(e, -126));
        row_mul[y] *= up;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) {
          const float2 f = Half16<DT_BF16>::unpack(w[c]);
          w[c] = Half16<DT_F16>::pack(f.x * down, f.y * down);
        }
      }
      // k step s takes values 4 s' .. 4 s' + 3 of a chunk: pairs (a0, a2) of row g, (a1, a3) of g + 8
#pragma unroll
      for (int s = 0; s < DH / 16; ++s) {
        q[s][y] = w[2 * s];
        q[s][2 + y] = w[2 * s + 1];
        if (RY == 1) q[s][1] = q[s][3] = 0u;
      }
    }
    float o[DH / 8][4];
#pragma unroll
    for (int x = 0; x < DH / 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[x][y] = 0.0f;
    float m[RY], l[RY];
#pragma unroll
    for (int y = 0; y < RY; ++y) {
      m[y] = ninf;
      l[y] = 0.0f;
    }
    int vref = -1000;                  // V's reference exponent
    const int whole_end = min(pre, end);
    // the thread's keys of a step, 4 of each group of 16, in the order of its scores' columns
    auto key_of = [&](int x) {
      return 16 * (x >> 2) + (QUANT ? 4 * t4 + (x & 3) : 8 * ((x >> 1) & 1) + 2 * t4 + (x & 1));
    };

#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      const int j0 = step_key(sg, k);
      const uint32_t good = (there_in >> (NG * stage_out)) & ((1u << NG) - 1u);
      if (!failed && !few_wait(&full[stage_out], parity_out)) {
        failed = true;
        a.c.status[b] = DT_ERR_TIMEOUT;
      }
      __syncwarp();
      const unsigned char *sK = ring + stage_out * 2 * HS, *sV = sK + HS;
      const bool masked = j0 + SUB > whole_end || good != (1u << NG) - 1u;
      auto there = [&](int x) { return j0 + key_of(x) < end && ((good >> (x >> 2)) & 1u); };
      // ------------------------------------------------------------ scores
      float s[2 * NG][4];
#pragma unroll
      for (int x = 0; x < 2 * NG; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][y] = 0.0f;
      if (QUANT) {
#pragma unroll
        for (int h = 0; h < DH / 64; ++h) {
          uint4 c[2 * NG];
#pragma unroll
          for (int x = 0; x < 2 * NG; ++x) {
            const int key = 4 * (g >> 1) + (g & 1) + 2 * (x & 1);
            c[x] = *reinterpret_cast<const uint4 *>(sK + (x >> 1) * 2048 + key * 128 +
                                                    (((4 * h + t4) ^ (key & 7)) << 4));
          }
#pragma unroll
          for (int z = 0; z < 4; ++z)
#pragma unroll
            for (int x = 0; x < 2 * NG; ++x) {
              const uint32_t w = z == 0 ? c[x].x : z == 1 ? c[x].y : z == 2 ? c[x].z : c[x].w;
              mma16<QDT>(s[x], q[4 * h + z], e4m3_f16x2(w & 0xffffu), e4m3_f16x2(w >> 16));
            }
        }
      } else {
#pragma unroll
        for (int h = 0; h < DH / 32; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = g + 8 * x;
            const uint4 c = *reinterpret_cast<const uint4 *>(
                sK + (h >> 1) * 2048 + key * 128 + (((4 * (h & 1) + t4) ^ (key & 7)) << 4));
            mma16<QDT>(s[x], q[2 * h], c.x, c.y);
            mma16<QDT>(s[x], q[2 * h + 1], c.z, c.w);
          }
      }
      uint32_t ve[NG];
      float kmul[4 * NG];
#pragma unroll
      for (int h = 0; h < NG; ++h) {
        if (QUANT) {
          const uint32_t ke = *reinterpret_cast<const uint32_t *>(ss.exps[warp][stage_out] + 16 * h + 4 * t4);
          ve[h] = *reinterpret_cast<const uint32_t *>(ss.exps[warp][stage_out] + SUB + 16 * h + 4 * t4);
#pragma unroll
          for (int x = 0; x < 4; ++x) kmul[4 * h + x] = row_scale((ke >> (8 * x)) & 255u);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) kmul[4 * h + x] = 1.0f;
        }
      }
      uint32_t see[RY];                // bits: keys x that row y sees
      float mx[RY];
#pragma unroll
      for (int y = 0; y < RY; ++y) {
        see[y] = live[y] ? (1u << (4 * NG)) - 1u : 0u;
        if (masked) {
          see[y] = 0u;
#pragma unroll
          for (int x = 0; x < 4 * NG; ++x)
            if (live[y] && there(x) && sees(a, rq, b, tok[y], j0 + key_of(x))) see[y] |= 1u << x;
        }
        mx[y] = ninf;
      }
#pragma unroll
      for (int y = 0; y < RY; ++y)
#pragma unroll
        for (int x = 0; x < 4 * NG; ++x) {
          float &v = s[x >> 1][2 * y + (x & 1)];
          v *= row_mul[y] * kmul[x];
          if (masked) v = (see[y] >> x) & 1u ? v : ninf;
          mx[y] = fmaxf(mx[y], v);
        }
      bool grow = false;
#pragma unroll
      for (int y = 0; y < RY; ++y) {
        mx[y] = fmaxf(mx[y], __shfl_xor_sync(kFull, mx[y], 1));
        mx[y] = fmaxf(mx[y], __shfl_xor_sync(kFull, mx[y], 2));
        if (!live[y]) mx[y] = ninf;
        grow |= mx[y] > m[y] + kGrow || (m[y] == ninf && mx[y] != ninf);
      }
      // V's reference: the step's largest exponent of a key that is there
      float vmul = 1.0f;               // of O, for a new reference
      if (QUANT) {
        int top = -1000;
#pragma unroll
        for (int x = 0; x < 4 * NG; ++x) {
          const int e = static_cast<int>((ve[x >> 2] >> (8 * (x & 3))) & 255u);
          if (e != 255 && (!masked || there(x))) top = max(top, e - 127);
        }
        top = __reduce_max_sync(kFull, top);
        if (top > vref + 40) {
          vmul = vref == -1000 ? 0.0f : exp2i(max(vref - top, -126));
          vref = top;
          grow = true;
        }
      }
      if (__any_sync(kFull, grow)) {
        float f[2] = {1.0f, 1.0f};
#pragma unroll
        for (int y = 0; y < RY; ++y) {
          const bool up = mx[y] > m[y] + kGrow || (m[y] == ninf && mx[y] != ninf);
          f[y] = !up ? 1.0f : m[y] == ninf ? 0.0f : fast_exp2(m[y] - mx[y]);
          if (up) m[y] = mx[y];
          l[y] *= f[y];
          f[y] *= vmul;
        }
#pragma unroll
        for (int x = 0; x < DH / 8; ++x)
#pragma unroll
          for (int y = 0; y < 2 * RY; ++y) o[x][y] *= f[y >> 1];
      }
      // ----------------------------------------------------------- weights
      float p[2][4 * NG];
#pragma unroll
      for (int y = 0; y < RY; ++y) {
        const float ref = m[y] == ninf ? 0.0f : m[y] - kShift;
#pragma unroll
        for (int x = 0; x < 4 * NG; ++x) {
          p[y][x] = fast_exp2(s[x >> 1][2 * y + (x & 1)] - ref);
          l[y] += p[y][x];
        }
      }
      if (QUANT) {
#pragma unroll
        for (int x = 0; x < 4 * NG; ++x) {
          const uint32_t E = (ve[x >> 2] >> (8 * (x & 3))) & 255u;
          // 2^(e - ref + 60), e at most 40 above ref; NaN rows NaN
          const float f = E == 255u ? row_scale(E)
                                    : exp2i(max(static_cast<int>(E) - 127 - vref + 60, -126));
#pragma unroll
          for (int y = 0; y < RY; ++y) {
            p[y][x] *= f;
            if (masked) p[y][x] = (see[y] >> x) & 1u ? p[y][x] : 0.0f;
          }
        }
      }
      uint32_t odd = 0u;
      const uint32_t v_at = smem_u32(sV);
      constexpr int PDT = QUANT ? DT_BF16 : DT;
#pragma unroll
      for (int h = 0; h < NG; ++h) {
        uint32_t pa[4], pl[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          pa[z] = pl[z] = 0u;
          if ((z & 1) >= RY) continue;
          const float p0 = p[z & 1][4 * h + 2 * (z >> 1)], p1 = p[z & 1][4 * h + 2 * (z >> 1) + 1];
          pa[z] = Half16<PDT>::pack(p0, p1);
          if (QUANT && DT == DT_F16) {   // second term
            const float2 hi = Half16<PDT>::unpack(pa[z]);
            pl[z] = Half16<PDT>::pack(p0 - hi.x, p1 - hi.y);
          }
        }
        // ------------------------------------------------------------ values
#pragma unroll
        for (int c = 0; c < DH / 32; ++c) {
          if (QUANT) {
            uint32_t r[4];   // columns 32 c + g + 8 i: keys 4 t .. 4 t + 3
            const int key = lane & 15, chunk = 2 * c + (lane >> 4);
            asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                         : "r"(v_at + h * 2048 + key * 128 + ((chunk ^ (key & 7)) << 4)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = codes_low<0>(r[i]), b1 = codes_low<1>(r[i]);
              mma16<PDT>(o[4 * c + i], pa, b0, b1);
              if (DT == DT_F16) mma16<PDT>(o[4 * c + i], pl, b0, b1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t r[4];
              const int key = lane & 15, chunk = 4 * (c & 1) + 2 * i + (lane >> 4);
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                           : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                           : "r"(v_at + (c >> 1) * 2048 + key * 128 + ((chunk ^ (key & 7)) << 4)));
              if (masked) {      // zero times a value that is not finite is NaN: see below
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const uint32_t x = not_finite<DT>(r[z]);
                  odd |= x;
                  r[z] &= ~x;
                }
              }
              mma16<PDT>(o[4 * c + 2 * i], pa, r[0], r[1]);
              mma16<PDT>(o[4 * c + 2 * i + 1], pa, r[2], r[3]);
            }
          }
        }
      }
      if (!QUANT && masked && __any_sync(kFull, odd != 0u)) {
        // values that are not finite, for the rows that see them
#pragma unroll 1
        for (int key = 0; key < SUB && j0 + key < end && good; ++key) {
          bool v[RY];
#pragma unroll
          for (int y = 0; y < RY; ++y) v[y] = live[y] && sees(a, rq, b, tok[y], j0 + key);
#pragma unroll
          for (int x = 0; x < DH / 8; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = 8 * x + 2 * t4 + e;
              const uint16_t w = *reinterpret_cast<const uint16_t *>(
                  sV + (col >> 6) * 2048 + key * 128 + ((((col & 63) >> 3) ^ (key & 7)) << 4) + (col & 7) * 2);
              if (col < dh && (not_finite<DT>(w) & 0xffffu))
#pragma unroll
                for (int y = 0; y < RY; ++y)
                  if (v[y]) o[x][2 * y + e] += Half16<DT>::unpack(w).x;
            }
        }
      }
      __syncwarp();                    // the place is read
      if (++stage_out == static_cast<uint32_t>(stages)) {
        stage_out = 0;
        parity_out ^= 1u;
      }
      if (k + stages < steps) issue(sg, k + stages);
    }

    // The next segment's first steps are on their way while this one's end is written.
    const Segment done = sg;
    more = walk.next(a, BM, kT, &sg);
    if (more)
      for (int k = 0; k < min(stages, step_count(sg)); ++k) issue(sg, k);

    // the warps' results together, 32 columns at a time
#pragma unroll
    for (int y = 0; y < RY; ++y) {
      if (!live[y]) l[y] = 0.0f;       // (m is -inf: the row's O is not looked at)
      l[y] += __shfl_xor_sync(kFull, l[y], 1);
      l[y] += __shfl_xor_sync(kFull, l[y], 2);
      if (t4 == 0) {
        ss.m[warp][g + 8 * y] = m[y];
        ss.l[warp][g + 8 * y] = l[y];
      }
    }
    const float out_mul = QUANT ? 0x1p60f : 1.0f, out_mul2 = QUANT && vref > -1000 ? exp2i(vref) : 1.0f;
    const bool whole = done.t0 == 0 && done.t1 == done.tiles;
    float *pp = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (done.t0 > 0 ? 0 : 1)) * 2 * a.slot;
    // a thread: row r, columns 4 c of a round
    const int r = tid / (kMergeCols / 4), c = tid % (kMergeCols / 4);
    const bool mine = r < rows && r < 8 * RY;
    float w[kFWarps], inv = 0.0f;
#pragma unroll
    for (int round = 0; round < DH / kMergeCols; ++round) {
#pragma unroll
      for (int x = 0; x < kMergeCols / 8; ++x)
#pragma unroll
        for (int y = 0; y < RY; ++y)
          *reinterpret_cast<float2 *>(&ss.out[warp][g + 8 * y][8 * x + 2 * t4]) =
              make_float2(o[kMergeCols / 8 * round + x][2 * y] * out_mul * out_mul2,
                          o[kMergeCols / 8 * round + x][2 * y + 1] * out_mul * out_mul2);
      __syncthreads();
      if (mine) {
        if (round == 0) {
          float mm = ninf, ll = 0.0f;
#pragma unroll
          for (int z = 0; z < kFWarps; ++z) mm = fmaxf(mm, ss.m[z][r]);
#pragma unroll
          for (int z = 0; z < kFWarps; ++z) {
            // (nothing seen: m is -inf; a sum that is NaN is not nothing)
            w[z] = ss.m[z][r] == ninf && ss.l[z][r] == 0.0f ? 0.0f : fast_exp2(ss.m[z][r] - mm);
            ll += w[z] * ss.l[z][r];
          }
          inv = whole ? (ll > 0.0f ? 1.0f / ll : ll == ll ? 0.0f : ll) : 1.0f;
          if (!whole && c == 0) {
            pp[BM * DH + r] = mm;
            pp[BM * DH + BM + r] = ll;
          }
        }
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int z = 0; z < kFWarps; ++z) {
          const float4 x = *reinterpret_cast<const float4 *>(&ss.out[z][r][4 * c]);
          if (w[z] != 0.0f) {
            acc[0] += w[z] * x.x; acc[1] += w[z] * x.y; acc[2] += w[z] * x.z; acc[3] += w[z] * x.w;
          }
        }
        const int col = kMergeCols * round + 4 * c;
        if (!whole) {
          *reinterpret_cast<float4 *>(pp + r * DH + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        } else if (col < dh) {
          const int i = r / a.G, h = done.hk * a.G + r - i * a.G;
          *reinterpret_cast<uint2 *>(a.out + done.b * a.ob + h * a.oh + i * a.orow + 2 * col) =
              make_uint2(Half16<DT>::pack(acc[0] * inv, acc[1] * inv), Half16<DT>::pack(acc[2] * inv, acc[3] * inv));
        }
      }
      __syncthreads();
    }
  }
}

template <int DT, bool QUANT, int DH, int RY>
cudaError_t go_rows(const AttnArgs &a, const AttnPlan &p, const CUtensorMap &k, const CUtensorMap &v,
                    cudaStream_t st) {
  const cudaError_t e = allow_smem<cache_attention_few_kernel<DT, QUANT, DH, RY>>();
  if (e != cudaSuccess) return e;
  cache_attention_few_kernel<DT, QUANT, DH, RY><<<a.grid, kFThreads, p.smem, st>>>(a, p.ring, k, v);
  return cudaGetLastError();
}

template <int DT, bool QUANT, int DH>
cudaError_t go(const AttnArgs &a, const AttnPlan &p, const CUtensorMap &k, const CUtensorMap &v,
               cudaStream_t st) {
  return a.n * a.G <= 8 ? go_rows<DT, QUANT, DH, 1>(a, p, k, v, st) : go_rows<DT, QUANT, DH, 2>(a, p, k, v, st);
}

template <int DT, bool QUANT>
cudaError_t go_dh(const AttnArgs &a, const AttnPlan &p, const CUtensorMap &k, const CUtensorMap &v,
                  cudaStream_t st) {
  return p.dhp == 64 ? go<DT, QUANT, 64>(a, p, k, v, st) : go<DT, QUANT, 128>(a, p, k, v, st);
}

}  // namespace

// For units of one row tile of at most 16 rows. False where the kernel does not apply.
bool few_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p) {
  if (c.dh > 128 || rows > kFewRows || static_cast<int64_t>(c.pages) * c.Hkv > 0x7fffffff) return false;
  p->kind = AttnPlan::kFew;
  p->bm = 16;
  p->row_tiles = 1;
  p->dhp = c.dh <= 64 ? 64 : 128;
  const int stage = 2 * (c.dtype == DT_E4M3 ? 4096 : p->dhp / 64 * 2048);
  p->ring = (smem - static_cast<int>(sizeof(FewSmall))) / (kFWarps * stage);
  if (p->ring > kMaxStages) p->ring = kMaxStages;
  if (p->ring < 2) return false;
  p->smem = static_cast<size_t>(p->ring) * kFWarps * stage + sizeof(FewSmall);
  p->grid = sms;
  return true;
}

cudaError_t launch_few(const dt_cache &c, const AttnArgs &a, int dtype, const AttnPlan &p,
                       cudaStream_t st) {
  CUtensorMap k = {}, v = {};
  if (!page_map(c, c.k, 16, &k) || !page_map(c, c.v, 16, &v)) return cudaErrorInvalidValue;
  const bool quant = c.dtype == DT_E4M3;
  if (dtype == DT_BF16) return quant ? go_dh<DT_BF16, true>(a, p, k, v, st) : go_dh<DT_BF16, false>(a, p, k, v, st);
  return quant ? go_dh<DT_F16, true>(a, p, k, v, st) : go_dh<DT_F16, false>(a, p, k, v, st);
}

}  // namespace dt
