// dt_cache_few.cu -- attention over the paged cache for a few rows (single tokens, short
// chains: G heads x rows <= 16) and head sizes up to 128: bound by the cache's bytes.
//
// Each of twelve warps of a block streams keys of its own, 16 at a time (8-bit rows 32),
// through a ring of its own, filled by TMA through a 128-byte swizzled tensor map (16 rows
// lie in one page): no warp waits for another before the unit's end, and about 140 KB of an SM's shared
// memory are in flight (its share of the memory's bandwidth times latency is 45 KB). The
// products are mma.sync m16n8k16, taken transposed: S^T = K Q^T and O^T += V^T P^T, so that
// keys and dimensions fill the M side and eight rows are one N tile, not half an M side
// (half the products and half the accumulators for up to eight rows; P^T becomes an operand
// by an 8x8 transpose between lanes). The softmax is online, its reference renewed only
// when the maximum has grown by 2^8 (fp16: 2^4).
//
// 8-bit rows become operands in registers. The product with K sums over dimensions in any
// order that both sides share, so a thread takes 16 codes of a key at once, and e4m3 codes
// are exact in fp16: one conversion a pair, K's scale and the row's own (bf16 query rows are
// scaled to fp16 by a power of two: their values lose less than 2^-24 of the row's largest)
// multiply the score. (fp16 query rows: where a value is no fp16 number, K is rounded or
// saturated as dt_cache_read does, so that a key's score does not depend on the number of
// rows.) V's codes come transposed from shared memory (8-bit ldmatrix: four consecutive
// keys of a column) and are set in bf16 fields as they are, which makes them their value
// times 2^-120. V's scale 2^e is part of the weight: 2^(x + e - M + 60) for a score x (a
// power of two's exponent, as the references are), where M = m + a whole number is a
// reference of the row's own for x + e, as m is for x: the largest term of O is near it
// however scores and scales are mixed, and keys that a row does not see leave its result
// alone. (One reference exponent a warp, of all its keys, lost what was 2^-80 of it: a row of
// 2^100 that nobody saw made the others' results zero. The second exponential costs no time:
// 32 tokens at 8192 keys 135 us before, 133 us now.) The result has that power of two taken
// out. fp16 results need weights of more than bf16's 8 bits: two terms.
//
// Measured, 32 / 8 heads, dh 128, 32 single tokens at 8192 keys: 8-bit rows 133 us, 4.1 TB/s
// of cache rows; 16-bit rows 205 us, 5.2 TB/s (of 6.8 that a copy reaches). For 8-bit rows a
// scheduler's three warps take about 1800 cycles for their steps of 32 keys, where memory
// would deliver them in 1400: conversions and products wait on each other; short caches are bound by a launch, its cut and the
// merge of a block's warps: 22 us for one request at 300 keys.
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

template <int DT, bool QUANT, int DH, int RN>   // RN: N tiles of 8 rows
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
  StepRing places = {0u, 0u, 0u};
  int given_up = 0;                    // steps in flight behind a wait that ran out
  uint32_t there_in = 0;               // bit NG i + h: group h of 16 keys of place i is on a good page
  // the warp's step k of a segment: keys from t0 T + SUB (warp + 12 k); the number of its steps
  auto step_key = [&](const Segment &s, int k) { return s.t0 * kT + SUB * (warp + kFWarps * k); };
  auto seg_end = [&](const Segment &s) { return static_cast<int>(min(static_cast<int64_t>(s.t1) * kT, s.end)); };
  auto step_count = [&](const Segment &s) {
    const int left = seg_end(s) - step_key(s, 0);
    return left <= 0 ? 0 : (left + SUB * kFWarps - 1) / (SUB * kFWarps);
  };
  auto issue = [&](const Segment &s, int k) {
    const uint32_t stage_in = places.in;
    const int j = step_key(s, k), end = seg_end(s);
    const int32_t *table = a.c.table + static_cast<int64_t>(s.b) * a.c.width;
    int entry[NG];
    uint32_t good = 0u;
#pragma unroll
    for (int h = 0; h < NG; ++h) {
      const int page = (j + 16 * h) >> a.c.shift;
      entry[h] = j + 16 * h < end && page < a.c.width ? table[page] : -1;
    }
#pragma unroll
    for (int h = 0; h < NG; ++h)
      if (static_cast<uint32_t>(entry[h]) < static_cast<uint32_t>(a.c.pages)) good |= 1u << h;
    there_in = (there_in & ~(((1u << NG) - 1u) << (NG * stage_in))) | good << (NG * stage_in);
    uint64_t *bar = &full[stage_in];
    if (lane == 0) {
      mbar_expect_tx(bar, __popc(good) * (2 * HS / NG + (QUANT ? 32 : 0)));
#pragma unroll
      for (int h = 0; h < NG; ++h)
        if (j + 16 * h < end && !((good >> h) & 1u)) cache_fault(a.c, s.b);
    }
    __syncwarp();
    // a lane a copy: boxes of K, of V (four of 16-bit rows, or two for each of two groups),
    // then the exponents
    constexpr int kBoxes = HS / NG / 2048;     // of a group's K
    const int which = lane & 1, u = lane >> 1;
    unsigned char *dst = ring + stage_in * 2 * HS + which * HS;
    if (u < NG * kBoxes) {
      const int h = u / kBoxes, kb = u % kBoxes;
      if ((good >> h) & 1u)
        few_tma(dst + u * 2048, which ? &vmap : &kmap, 64 * kb, (j + 16 * h) & ((1 << a.c.shift) - 1),
                (NG == 1 || h == 0 ? entry[0] : entry[NG - 1]) * a.c.Hkv + s.hk, bar);
    } else if (QUANT && u < 2 * NG) {
      const int h = u - NG;
      if ((good >> h) & 1u) {
        const int64_t row = (static_cast<int64_t>((h == 0 ? entry[0] : entry[NG - 1]) * a.c.Hkv + s.hk) << a.c.shift) +
                            ((j + 16 * h) & ((1 << a.c.shift) - 1));
        bulk_g2s(ss.exps[warp][stage_in] + which * SUB + 16 * h, (which ? a.c.v_exp : a.c.k_exp) + row, 16, bar);
      }
    }
    places.issued(stages);
  };
  if (more)
    for (int k = 0; k < min(stages, step_count(sg)); ++k) issue(sg, k);

  while (more) {
    const Request rq = sg.rq;
    const int b = sg.b, hk = sg.hk, pre = static_cast<int>(rq.pre), end = seg_end(sg);
    const int steps = given_up ? 0 : step_count(sg);
    if (tid == 0 && a.prefix[b] != rq.pre) cache_fault(a.c, b);
    // Q^T: this thread's part of row 8 z + g; its scores are of rows 8 z + 2 t, 8 z + 2 t + 1
    uint32_t q[DH / 16][RN][2];
    float row_mul[RN][2];
    int tok[RN][2];
    bool live[RN][2];
#pragma unroll
    for (int z = 0; z < RN; ++z) {
      const int r = 8 * z + g, i = r / a.G;
      const char *src = a.q + b * a.qb + (hk * a.G + r - i * a.G) * a.qh + i * a.qr;
      float mul = a.scale_log2;
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
        mul *= up;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) {
          const float2 f = Half16<DT_BF16>::unpack(w[c]);
          w[c] = Half16<DT_F16>::pack(f.x * down, f.y * down);
        }
      }
      // k step s takes four values of a chunk: two pairs
#pragma unroll
      for (int s = 0; s < DH / 16; ++s) {
        q[s][z][0] = w[2 * s];
        q[s][z][1] = w[2 * s + 1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * z + 2 * t4 + e;
        tok[z][e] = row / a.G;
        live[z][e] = row < rows && tok[z][e] < rq.count;
        row_mul[z][e] = __shfl_sync(kFull, mul, 4 * (2 * t4 + e));
      }
    }
    float o[DH / 16][RN][4];           // dimensions 16 x + g, 16 x + g + 8 of those two rows
#pragma unroll
    for (int x = 0; x < DH / 16; ++x)
#pragma unroll
      for (int z = 0; z < RN; ++z)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[x][z][y] = 0.0f;
    // references and sums; (8-bit rows) O's reference is m + od, od a whole number
    float m[RN][2], l[RN][2], od[RN][2];
#pragma unroll
    for (int z = 0; z < RN; ++z)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[z][e] = ninf;
        l[z][e] = od[z][e] = 0.0f;
      }
    const int whole_end = min(pre, end);
    // the thread's two keys of a group of 16, as rows g and g + 8 of the product
    const int key0 = QUANT ? 4 * (g >> 1) + (g & 1) : g, key1 = key0 + (QUANT ? 2 : 8);

#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      const int j0 = step_key(sg, k);
      const uint32_t stage_out = places.out;
      const uint32_t good = (there_in >> (NG * stage_out)) & ((1u << NG) - 1u);
      if (!__all_sync(kFull, few_wait(&full[stage_out], places.parity))) {
        given_up = StepRing::flying(k, steps, stages);
        a.c.status[b] = DT_ERR_TIMEOUT;
        break;
      }
      const unsigned char *sK = ring + stage_out * 2 * HS, *sV = sK + HS;
      const bool masked = j0 + SUB > whole_end || good != (1u << NG) - 1u;
      auto key_at = [&](int x) { return j0 + 16 * (x >> 1) + (x & 1 ? key1 : key0); };    // x: 2 h + which
      auto there = [&](int x) { return key_at(x) < end && ((good >> (x >> 1)) & 1u); };
      // ------------------------------------------------------------ scores
      // (in two sums each, so that half as many products wait for one another)
      float s[NG][RN][4], s2[NG][RN][4];
#pragma unroll
      for (int h = 0; h < NG; ++h)
#pragma unroll
        for (int z = 0; z < RN; ++z)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[h][z][y] = s2[h][z][y] = 0.0f;
#pragma unroll
      for (int d = 0; d < (QUANT ? DH / 64 : DH / 32); ++d) {
        uint4 c[NG][2];
#pragma unroll
        for (int h = 0; h < NG; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = x ? key1 : key0;
            c[h][x] = *reinterpret_cast<const uint4 *>(
                sK + (QUANT ? h : d >> 1) * 2048 + key * 128 +
                (((QUANT ? 4 * d + t4 : 4 * (d & 1) + t4) ^ (key & 7)) << 4));
          }
#pragma unroll
        for (int i = 0; i < (QUANT ? 4 : 2); ++i)
#pragma unroll
          for (int h = 0; h < NG; ++h) {
            uint32_t ka[4];            // rows g, g + 8; four values each
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 &v = c[h][x];
              if (QUANT) {
                const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
                ka[x] = e4m3_f16x2(w & 0xffffu);
                ka[2 + x] = e4m3_f16x2(w >> 16);
              } else {
                ka[x] = i ? v.z : v.x;
                ka[2 + x] = i ? v.w : v.y;
              }
            }
#pragma unroll
            for (int z = 0; z < RN; ++z) {
              const uint32_t(&qb)[2] = q[(QUANT ? 4 : 2) * d + i][z];
              mma16<QDT>(i & 1 ? s2[h][z] : s[h][z], ka, qb[0], qb[1]);
            }
          }
      }
      uint32_t ve[2 * NG];             // V's exponent bytes of the thread's keys
      float kmul[2 * NG];
#pragma unroll
      for (int h = 0; h < NG; ++h) {
        if (QUANT) {
          const uint8_t *e = ss.exps[warp][stage_out] + 16 * h + key0;
          const uint32_t w = *reinterpret_cast<const uint32_t *>(e - (g & 1)) >> (8 * (g & 1));
          const uint32_t v = *reinterpret_cast<const uint32_t *>(e + SUB - (g & 1)) >> (8 * (g & 1));
          kmul[2 * h] = row_scale(w & 255u);
          kmul[2 * h + 1] = row_scale((w >> 16) & 255u);
          ve[2 * h] = v & 255u;
          ve[2 * h + 1] = (v >> 16) & 255u;
        } else {
          kmul[2 * h] = kmul[2 * h + 1] = 1.0f;
          ve[2 * h] = ve[2 * h + 1] = 0u;
        }
      }
      if (QUANT && DT == DT_F16) {
        // Scales of which fp16 rounds or saturates a value: the scores of the keys as
        // dt_cache_read gives them, in a short loop that reads Q again. (One token at 300 keys
        // takes 22 us, 21 without this, 26 with a second copy of the products above.)
        bool odd = false;
#pragma unroll
        for (int x = 0; x < 2 * NG; ++x) odd |= kmul[x] < 0x1p-15f || kmul[x] > 0x1p7f;
        if (__any_sync(kFull, odd)) {
          odd = false;
#pragma unroll
          for (int x = 0; x < 2 * NG; ++x) {
            if (kmul[x] < 0x1p-33f) kmul[x] = 0.0f;      // below half of fp16's least step: zeros
            odd |= kmul[x] > 0.0f && (kmul[x] < 0x1p-15f || kmul[x] > 0x1p7f);
          }
          if (__any_sync(kFull, odd)) {
#pragma unroll
            for (int h = 0; h < NG; ++h)
#pragma unroll
              for (int z = 0; z < RN; ++z)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[h][z][y] = s2[h][z][y] = 0.0f;
#pragma unroll 1
            for (int k16 = 0; k16 < DH / 16; ++k16) {    // four values of each of four lanes
              const int at = 64 * (k16 >> 2) + 16 * t4 + 4 * (k16 & 3);
              uint2 qw[RN];
#pragma unroll
              for (int z = 0; z < RN; ++z) {
                const int r = 8 * z + g, i = r / a.G;
                qw[z] = make_uint2(0u, 0u);
                if (r < rows && at < dh)
                  qw[z] = *reinterpret_cast<const uint2 *>(a.q + b * a.qb + (hk * a.G + r - i * a.G) * a.qh +
                                                           i * a.qr + 2 * at);
              }
#pragma unroll
              for (int h = 0; h < NG; ++h) {
                uint32_t ka[4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int key = x ? key1 : key0;
                  const uint32_t w = *reinterpret_cast<const uint32_t *>(
                      sK + h * 2048 + key * 128 + (((at >> 4) ^ (key & 7)) << 4) + (at & 15));
                  ka[x] = e4m3_to16<DT_F16>(w & 0xffffu, kmul[2 * h + x]);
                  ka[2 + x] = e4m3_to16<DT_F16>(w >> 16, kmul[2 * h + x]);
                }
#pragma unroll
                for (int z = 0; z < RN; ++z) mma16<DT_F16>(s[h][z], ka, qw[z].x, qw[z].y);
              }
            }
#pragma unroll
            for (int x = 0; x < 2 * NG; ++x) kmul[x] = 1.0f;
          }
        }
      }
      uint32_t see = ~0u;              // bit (2 h + x) 2 RN + 2 z + e: the row sees the key
      if (masked) {
        see = 0u;
#pragma unroll
        for (int x = 0; x < 2 * NG; ++x)
#pragma unroll
          for (int z = 0; z < RN; ++z)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (live[z][e] && there(x) && sees(a, rq, b, tok[z][e], key_at(x)))
                see |= 1u << (2 * RN * x + 2 * z + e);
      }
      // V's exponents as numbers (a row of 255: NaN), which go to the weights' exponents
      float vx[2 * NG];
#pragma unroll
      for (int x = 0; x < 2 * NG; ++x)
        vx[x] = ve[x] == 255u ? row_scale(255u) : static_cast<float>(static_cast<int>(ve[x]) - 127);
      // largest scores, and largest sums of a score and its V's exponent
      float mx[RN][2], mo[RN][2];
#pragma unroll
      for (int z = 0; z < RN; ++z)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[z][e] = mo[z][e] = ninf;
#pragma unroll
          for (int x = 0; x < 2 * NG; ++x) {
            float &v = s[x >> 1][z][2 * (x & 1) + e];
            // (one scale after the other: their product may be no fp32 number where the score is)
            v = (v + s2[x >> 1][z][2 * (x & 1) + e]) * row_mul[z][e];
            if (QUANT) v *= kmul[x];
            if (masked) v = (see >> (2 * RN * x + 2 * z + e)) & 1u ? v : ninf;
            mx[z][e] = fmaxf(mx[z][e], v);
            if (QUANT) mo[z][e] = fmaxf(mo[z][e], v + vx[x]);
          }
        }
      // Does a row's maximum grow past its reference, or that sum past O's? Each lane asks
      // for its own keys; only then are they taken across lanes.
      bool grow = false;
#pragma unroll
      for (int z = 0; z < RN; ++z)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!live[z][e]) mx[z][e] = mo[z][e] = ninf;
          grow |= mx[z][e] > m[z][e] + kGrow || (m[z][e] == ninf && mx[z][e] != ninf);
          if (QUANT) grow |= mo[z][e] > m[z][e] + od[z][e] + kGrow;
        }
      if (__any_sync(kFull, grow)) {
#pragma unroll
        for (int z = 0; z < RN; ++z)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = mx[z][e], to = mo[z][e];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              t = fmaxf(t, __shfl_xor_sync(kFull, t, x));
              if (QUANT) to = fmaxf(to, __shfl_xor_sync(kFull, to, x));
            }
            const bool first = m[z][e] == ninf, up = t > m[z][e] + kGrow || (first && t != ninf);
            const float old = m[z][e], shift = up ? old - t : 0.0f;
            if (up) m[z][e] = t;
            float f = first ? 0.0f : fast_exp2(shift);
            l[z][e] *= f;
            if (QUANT) {
              // (within 180 for any scores and exponents that are numbers)
              const float from = old + od[z][e], ref = first || to > from + kGrow ? to : from;
              const float dn = fminf(fmaxf(rintf(ref - m[z][e]), -180.0f), 180.0f);
              f = first ? 0.0f : fast_exp2(shift + (od[z][e] - dn));
              od[z][e] = dn;
            }
#pragma unroll
            for (int x = 0; x < DH / 16; ++x) {
              o[x][z][e] *= f;
              o[x][z][2 + e] *= f;
            }
          }
      }
      // ----------------------------------------------------------- weights
      // p^T of 8 keys x 8 rows a register, transposed between lanes: keys 2 t, 2 t + 1 of row g
      constexpr int PDT = QUANT ? DT_BF16 : DT;
      uint32_t pb[NG][RN][2], pl[NG][RN][2];
#pragma unroll
      for (int x = 0; x < 2 * NG; ++x) {
#pragma unroll
        for (int z = 0; z < RN; ++z) {
          float p[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[z][e] == ninf ? 0.0f : m[z][e] - kShift;
            const float a2 = s[x >> 1][z][2 * (x & 1) + e] - ref;
            p[e] = fast_exp2(a2);
            l[z][e] += p[e];
            if (QUANT) p[e] = fast_exp2(a2 + (vx[x] - od[z][e] + 60.0f));
            if (QUANT && masked) p[e] = (see >> (2 * RN * x + 2 * z + e)) & 1u ? p[e] : 0.0f;
          }
          const uint32_t hi = Half16<PDT>::pack(p[0], p[1]);
          asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[x >> 1][z][x & 1]) : "r"(hi));
          if (QUANT && DT == DT_F16) {   // second term
            const float2 h2 = Half16<PDT>::unpack(hi);
            const uint32_t lo = Half16<PDT>::pack(p[0] - h2.x, p[1] - h2.y);
            asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pl[x >> 1][z][x & 1]) : "r"(lo));
          }
        }
      }
      // ------------------------------------------------------------ values
      uint32_t odd = 0u;
      const uint32_t v_at = smem_u32(sV);
#pragma unroll
      for (int h = 0; h < NG; ++h) {
#pragma unroll
        for (int c = 0; c < DH / 32; ++c) {
          uint32_t va[2][4];           // dimensions 32 c + 16 i + g, + 8; the 16 keys
          if (QUANT) {
            uint32_t r[4];             // columns 32 c + g + 8 i: keys 4 t .. 4 t + 3
            const int key = lane & 15, chunk = 2 * c + (lane >> 4);
            asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                         : "r"(v_at + h * 2048 + key * 128 + ((chunk ^ (key & 7)) << 4)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              va[i >> 1][i & 1] = codes_low<0>(r[i]);
              va[i >> 1][2 + (i & 1)] = codes_low<1>(r[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int key = (lane & 7) + ((lane >> 4) << 3), chunk = 4 * (c & 1) + 2 * i + ((lane >> 3) & 1);
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                           : "=r"(va[i][0]), "=r"(va[i][1]), "=r"(va[i][2]), "=r"(va[i][3])
                           : "r"(v_at + (c >> 1) * 2048 + key * 128 + ((chunk ^ (key & 7)) << 4)));
              if (masked) {      // zero times a value that is not finite is NaN: see below
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const uint32_t x = not_finite<DT>(va[i][z]);
                  odd |= x;
                  va[i][z] &= ~x;
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int z = 0; z < RN; ++z) {
              mma16<PDT>(o[2 * c + i][z], va[i], pb[h][z][0], pb[h][z][1]);
              if (QUANT && DT == DT_F16) mma16<PDT>(o[2 * c + i][z], va[i], pl[h][z][0], pl[h][z][1]);
            }
        }
      }
      if (!QUANT && masked && __any_sync(kFull, odd != 0u)) {
        // values that are not finite, for the rows that see them
#pragma unroll 1
        for (int key = 0; key < SUB && j0 + key < end && good; ++key)
#pragma unroll
          for (int z = 0; z < RN; ++z)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (!live[z][e] || !sees(a, rq, b, tok[z][e], j0 + key)) continue;
#pragma unroll
              for (int x = 0; x < DH / 16; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int d = 16 * x + g + 8 * y;
                  const uint16_t w = *reinterpret_cast<const uint16_t *>(
                      sV + (d >> 6) * 2048 + key * 128 + ((((d & 63) >> 3) ^ (key & 7)) << 4) + (d & 7) * 2);
                  if (d < dh && (not_finite<DT>(w) & 0xffffu)) o[x][z][2 * y + e] += Half16<DT>::unpack(w).x;
                }
            }
      }
      __syncwarp();                    // the place is read
      places.taken(stages);
      if (k + stages < steps) issue(sg, k + stages);
    }

    // The next segment's first steps are on their way while this one's end is written.
    const Segment done = sg;
    more = walk.next(a, BM, kT, &sg);
    if (more && !given_up)
      for (int k = 0; k < min(stages, step_count(sg)); ++k) issue(sg, k);

    // the warps' results together, 32 columns at a time
#pragma unroll
    for (int z = 0; z < RN; ++z)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (!live[z][e]) l[z][e] = 0.0f;       // (m is -inf: the row's O is not looked at)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[z][e] += __shfl_xor_sync(kFull, l[z][e], x);
        if (g == 0) {
          ss.m[warp][8 * z + 2 * t4 + e] = m[z][e];
          ss.l[warp][8 * z + 2 * t4 + e] = l[z][e];
        }
      }
    // (8-bit rows) 2^(60 + d) in two factors
    float mul0[RN][2], mul1[RN][2];
#pragma unroll
    for (int z = 0; z < RN; ++z)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int dn = static_cast<int>(od[z][e]), part = dn / 2;
        mul0[z][e] = QUANT ? exp2i(30 + part) : 1.0f;
        mul1[z][e] = QUANT ? exp2i(30 + dn - part) : 1.0f;
      }
    const bool whole = done.t0 == 0 && done.t1 == done.tiles;
    float *pp = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (done.t0 > 0 ? 0 : 1)) * 2 * a.slot;
    // a thread: row r, columns 4 c of a round
    const int r = tid / (kMergeCols / 4), c = tid % (kMergeCols / 4);
    const bool mine = r < rows && r < 8 * RN;
    float w[kFWarps], inv = 0.0f;
#pragma unroll
    for (int round = 0; round < DH / kMergeCols; ++round) {
#pragma unroll
      for (int x = 0; x < kMergeCols / 16; ++x)
#pragma unroll
        for (int z = 0; z < RN; ++z)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            ss.out[warp][8 * z + 2 * t4 + (y & 1)][16 * x + g + 8 * (y >> 1)] =
                o[kMergeCols / 16 * round + x][z][y] * mul0[z][y & 1] * mul1[z][y & 1];
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
  // No copy may be in flight when the block ends: after a wait that ran out, wait (bounded
  // again) for those behind it.
  for (; given_up > 0; --given_up) {
    few_wait(&full[places.out], places.parity);
    places.taken(stages);
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
// Sixteen, measured against the tcgen05 kernel (us, that one second; single tokens of G
// heads, 8 key/value heads; requests x keys; head size), with the ratio of the two in the mean:
//                              1 x 300  1 x 32768  8 x 2048  32 x 8192  128 x 1024
//   bf16, 16-bit  64,  G 8     14  31    37  51     29  37   122  152     86  121   0.68
//                 64,  G 16    29  31    45  57     32  37   123  152    103  121   0.85
//                 128, G 8     22  33    57  68     39  44   205  199    124  150   0.85
//                 128, G 9     43  35    70  70     45  45   214  200    158  152   1.07
//                 128, G 16    25  35    70  72     45  45   217  202    161  156   0.95
//   bf16, 8-bit   64,  G 16    27  37    49  62     38  43   141  201    125  176   0.76
//                 128, G 8     22  41    51  62     37  45   131  204    114  195   0.67
//                 128, G 9     39  41    71  64     53  45   197  206    180  200   1.01
//                 128, G 16    39  41    70  68     53  47   197  206    182  204   0.99
//   fp16, 8-bit   128, G 8     22  45    51  71     37  51   134  248    115  255   0.58
//                 128, G 16    37  47    76  76     55  53   237  250    204  269   0.90
// (fp16 over 16-bit rows as bf16.) Nine to sixteen rows at head sizes above 64 are about
// even: their second N tile spills 160 to 480 bytes a thread. More rows would need a third.
bool few_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p) {
  if (c.dh > 128 || rows > kFewRows) return false;
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
