// dt_cache_wide.cu -- attention over the paged cache on the tcgen05 tensor cores
// (head sizes up to 128).
//
// Both products are taken transposed, so that the query rows are the MMA's N side,
// which comes in steps of 16 where the M side is 128: the rows of a unit (G heads x
// tree rows, 4 to 192 of them) are padded to the next 16, not 128, and one kernel
// serves single tokens and wide trees. Per tile of 128 keys and group of up to 112
// rows: S^T = K Q^T (M = keys, K-major K tile and Q), p = 2^(x - m) by one thread a
// key, which finds its key's scores for all rows in its TMEM lane, P^T to shared
// memory ([key][row], the N side MN-major), O^T += V^T P^T (M = head dimension: the V
// tile as it is stored, MN-major). Neither K nor V is transposed anywhere.
//
// The running maximum runs along the lanes of S^T, and is not taken for every tile:
// a row's reference m stays until one of its weights passes 2^10 (fp16: 2^15, from
// weights that start at 2^8), which a thread sees from its own weights; only then
// (and for a unit's first tile) are the tile's maxima taken across lanes, O^T and the
// sums rescaled. Any reference at most that far below the maximum gives the same
// quotient; sums and O are fp32. Each thread sums its keys' weights row by row in
// registers, joined across lanes once a unit.
//
// Two warpgroups (A, B) take weights, so that the tensor cores work for one meanwhile.
// Up to 96 rows: both have all rows, A the even and B the odd key tiles, and A or the
// join adds them up (an MMA takes 32 + N / 4 cycles at least, the first term for
// reading its 128 keys: one MMA over all rows beats two over half). More rows: each
// has half the rows, and every tile, so that a tile is read, and an 8-bit one
// converted, once for up to 192 rows. K and V tiles alternate in a ring in the order
// in which they are consumed (K0 K1 V0 K2 V1 ...), filled by TMA, page by page,
// through a 128-byte swizzled tensor map; tiles of 8-bit rows land in a raw ring by
// plain bulk copies and a third warpgroup writes their bf16 or fp16 values into the
// operand ring.
#include <cmath>
#include <cstdint>
#include <cuda.h>

#include "dt_cache_attn.cuh"
#include "dt_internal.h"
#include "dt_umma.cuh"

namespace dt {

namespace {

constexpr int kW = kWideKeys;
constexpr int kBlk = kW * 128;         // bytes of 128 rows of 64 16-bit values
constexpr int kMaxRing = 8;
constexpr int kSegs = 4;
constexpr int kMaxCols = 96;           // rows of a group: one sum of each in a thread's registers

// Warpgroups: two for weights, two (8-bit rows) that convert, one whose warps load, issue
// the products, find segments. Registers at launch times threads is what setmaxnreg
// shares out: 640 x 96 >= 256 x 176 + 384 x 40, and 384 x 168 >= 256 x 200 + 128 x 96.
template <bool QUANT> constexpr int kWThreads = QUANT ? 640 : 384;
template <bool QUANT> constexpr int kWeightRegs = QUANT ? 176 : 200;
template <bool QUANT> constexpr int kOtherRegs = QUANT ? 40 : 96;
template <int N> __device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int kOddWords = (DT_MAX_N + 32) / 32;
constexpr long long kWaitCycles = 4000000000ll;   // about 2 s

struct WideShape {
  int bm, na, nb, alt, ring, raw, nblk, raw_bytes;
  int off_q, off_pa, off_pb, off_raw, off_small;
};

struct Small {                          // behind the big buffers
  float neg_m[2][128];                  // minus the reference of each row (plus the fp16 shift)
  float fac[2][128];
  uint64_t full[kMaxRing], empty[kMaxRing], raw_full[kMaxRing], raw_empty[kMaxRing];
  uint64_t q_full, q_free, s_full[2], p_full[2], pv_done[2];
  int64_t scan[640 / 32 + 2];
  Segment seg[kSegs];                   // the next segments; b < 0: no more
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t odd[2][kOddWords + 1];      // tree rows whose V is not all finite; the last word: any
  uint32_t tmem;
  int fail;
};

// Bounded wait for a phase. The limit is in SM cycles: a read of the clock register
// costs a few cycles, of the global timer about a microsecond, which every wait that
// is not over at once would pay.
__device__ __forceinline__ bool mbar_wait_cycles(uint64_t *bar, uint32_t parity) {
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
    else if (t - t0 > kWaitCycles) return false;
  }
}

// 128-byte swizzled operand descriptor; its address field counts 16-byte units, so an
// operand further on is a plain addition
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return umma_desc(addr, lbo, sbo) | (2ull << 61);
}

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                       uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// 16 fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}

// barrier of one warpgroup (id 1, 2); the second form also ORs a predicate
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %2, 0;\n"
      "barrier.cta.red.or.pred q, %1, 128, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r) : "r"(id), "r"(static_cast<uint32_t>(p)) : "memory");
  return r != 0;
}
// both warpgroups: a part of one unit handed from B to A through global memory
__device__ __forceinline__ void pair_sync() {
  __threadfence_block();
  asm volatile("barrier.cta.sync 3, 256;" ::: "memory");
}

// packed pairs of fp32
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float *lo, float *hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int DT>
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {   // a number beats a NaN
  uint32_t r;
  if (DT == DT_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// largest magnitudes of two pairs of 16-bit values (signs are not kept), NaN above all
template <int DT>
__device__ __forceinline__ uint32_t top_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == DT_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 weights of key gt into the group's P^T tile
__device__ __forceinline__ void put_weights(unsigned char *sP, int gt, int c, const uint32_t (&y)[8]) {
  unsigned char *p = sP + (c >> 2) * kBlk + gt * 128;
  const int ch = (c & 3) * 2;
  *reinterpret_cast<uint4 *>(p + ((ch ^ (gt & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<uint4 *>(p + (((ch + 1) ^ (gt & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
}

// sets bits [lo, hi) of a 128-bit set
__device__ __forceinline__ void set_run(uint64_t (&bits)[2], int lo, int hi) {
  if (lo >= hi) return;
  const int n = hi - lo;
  const uint64_t run = n >= 64 ? ~0ull : (1ull << n) - 1;
  if (lo < 64) {
    bits[0] |= run << lo;
    if (hi > 64) bits[1] |= hi >= 128 ? ~0ull : (1ull << (hi - 64)) - 1;
  } else {
    bits[1] |= run << (lo - 64);
  }
}

// Reduces 16 columns across the 32 lanes of a warp (MAX: maximum, else sum): lanes
// 2 c and 2 c + 1 end with column c.
template <bool MAX>
__device__ __forceinline__ float reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8, m = 16; half >= 1; half >>= 1, m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < half) {
        const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
        const float got = __shfl_xor_sync(kFull, give, m);
        v[i] = MAX ? fmaxf(keep, got) : keep + got;
      }
  }
  const float got = __shfl_xor_sync(kFull, v[0], 1);
  return MAX ? fmaxf(v[0], got) : v[0] + got;
}

// Sums of 8 row pairs [pair][128 keys][2] over the keys into out[16].
__device__ __forceinline__ void sum_chunk(const float *part, float *out, int gt, int bar_id) {
  group_sync(bar_id);
  // 16 lanes a row pair, 8 keys each
  const float4 *src = reinterpret_cast<const float4 *>(part + ((gt >> 4) * 128) * 2) + (gt & 15);
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 x = src[16 * k];
    a += x.x + x.z;
    b += x.y + x.w;
  }
#pragma unroll
  for (int m = 8; m; m >>= 1) {
    a += __shfl_xor_sync(kFull, a, m);
    b += __shfl_xor_sync(kFull, b, m);
  }
  if ((gt & 15) == 0) {
    out[2 * (gt >> 4)] = a;
    out[2 * (gt >> 4) + 1] = b;
  }
  group_sync(bar_id);
}

// New references of a group's rows: the larger of the old one and the tile's maximum,
// taken across lanes (scores that do not count are -inf there). fac: what earlier sums
// are to be scaled by.
__device__ __forceinline__ void new_refs(uint32_t t_s, int n, float *wred, int gt, int lane, int bar_id,
                                         float scale, float shift, float *neg_m, float *fac, float *m) {
  const float ninf = -__int_as_float(0x7f800000);
#pragma unroll 1
  for (int c = 0; c * 16 < n; ++c) {
    float v[16];
    tmem_ld16(t_s + 16 * c, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] *= scale;
    const float r = reduce16<true>(v, lane);
    if (!(lane & 1)) wred[(gt >> 5) * 128 + 16 * c + (lane >> 1)] = r;
  }
  group_sync(bar_id);
  if (gt < n) {
    float mn = fmaxf(fmaxf(wred[gt], wred[128 + gt]), fmaxf(wred[256 + gt], wred[384 + gt]));
    mn = fmaxf(mn, *m);
    fac[gt] = mn == ninf ? 1.0f : fast_exp2(*m - mn);
    // a row that has seen nothing yet: any score passes the limit
    neg_m[gt] = mn == ninf ? 1e30f : shift - mn;
    *m = mn;
  }
  group_sync(bar_id);
}

// instruction descriptor of kind::f16, M = 128, fp32 accumulation; mn: both operands
// MN-major
template <int DT>
__device__ __forceinline__ uint32_t idesc16(int N, bool mn) {
  const uint32_t f = DT == DT_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (mn ? 3u << 15 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | ((128u >> 4) << 24);
}

// two of a word's four e4m3 codes (0: the lower two) as sign-extended half words
template <int HALF>
__device__ __forceinline__ uint32_t spread_codes(uint32_t w) {
  uint32_t r;   // byte, its sign eight times; twice
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(HALF ? 0xb3a2 : 0x9180));
  return r;
}
// two codes spread over half words as bf16 values times 2^-120 times `mul` (bf16 pair): the
// code's exponent and mantissa bits, set in the bf16 fields, are the value times 2^-120
// exactly, subnormal codes included
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t spread, uint32_t mul) {
  const uint32_t r = (spread << 4) & 0x87f087f0u;
  uint32_t o;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(r), "r"(mul));
  return o;
}
// 16 values of row r into an operand tile, swizzled
__device__ __forceinline__ void put_operand(unsigned char *row, int r, int c, const uint32_t (&y)[8]) {
  unsigned char *to = row + (c >> 2) * kBlk;
  const int z = (c & 3) * 2;
  *reinterpret_cast<uint4 *>(to + ((z ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<uint4 *>(to + (((z + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
}

// a place in a ring of `size` tiles, and the parity of its barriers' phase
struct Place {
  uint32_t at, parity;
  __device__ void step(uint32_t size) {
    if (++at == size) {
      at = 0;
      parity ^= 1u;
    }
  }
};

template <int DT, bool QUANT>
__global__ void __launch_bounds__(kWThreads<QUANT>, 1)
cache_attention_wide_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ WideShape w,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Small &ss = *reinterpret_cast<Small *>(sm + w.off_small);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int dh = a.c.dh, tile_bytes = w.nblk * kBlk;
  const float ninf = -__int_as_float(0x7f800000);

  if (tid == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&ss.full[i], QUANT ? 256 : 1);
      mbar_init(&ss.empty[i], 1);
      mbar_init(&ss.raw_full[i], 1);
      mbar_init(&ss.raw_empty[i], 256);
    }
    mbar_init(&ss.q_full, w.alt ? 128 : 256);
    mbar_init(&ss.q_free, 128);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&ss.seg_full[i], 1);
      mbar_init(&ss.seg_empty[i], QUANT ? 18 : 10);   // the warps that take segments
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ss.s_full[x], 1);
      mbar_init(&ss.p_full[x], 128);
      mbar_init(&ss.pv_done[x], 1);
    }
    ss.fail = 0;
  }
  // rows that are padding keep a reference that gives them weight 0
  for (int i = tid; i < 256; i += kWThreads<QUANT>) (&ss.neg_m[0][0])[i] = ninf;
  if (warp == 0) tmem_alloc(&ss.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = ss.tmem;

  Schedule<kWThreads<QUANT>> sch;
  sch.plan(a, w.bm, kW, ss.scan);
  Walk walk;
  walk.at = blockIdx.x * sch.chunk;
  walk.stop = min(walk.at + sch.chunk, sch.total);
  walk.b = 0;
  walk.base = 0;
  if (walk.at < walk.stop) sch.find(a, w.bm, kW, walk.at, ss.scan, &walk.b, &walk.base);
  Segment sg;
  sg.b = 0;
  volatile int *fail = &ss.fail;
  // Every wait is bounded. One that runs out ends the block's loads and products; the
  // weights' warpgroups, which meet at barriers of their own, go through the rest of
  // their steps without waiting.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (*fail) return false;
    if (mbar_wait_cycles(bar, parity)) return true;
    *fail = 1;
    a.c.status[sg.b] = DT_ERR_TIMEOUT;
    return false;
  };
  // the same for a converged warp: all lanes go on together
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(kFull, wait(bar, parity)) != 0;
  };
  // The block's next segment. One warp finds them ahead of time (its code is long and its
  // loads depend on each other) and ends with b < 0, in any case: every warp sees the
  // same segments, whatever has failed.
  uint32_t seg = 0;
  auto next_segment = [&]() {
    const uint32_t i = seg % kSegs, parity = (seg / kSegs) & 1;
    bool there = false;
    for (int k = 0; k < 4 && !there; ++k) there = mbar_wait_cycles(&ss.seg_full[i], parity);
    __syncwarp();
    if (!there) return false;
    sg = ss.seg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ss.seg_empty[i]);
    ++seg;
    return sg.b >= 0;
  };
  // operand tiles of a segment of T key tiles, in ring order: K0 K1 V0 K2 V1 ... V(T-1)
  auto op_tile = [](int op, int T, bool *is_v) {
    if (op == 0) { *is_v = false; return 0; }
    if (op == 2 * T - 1) { *is_v = true; return T - 1; }
    *is_v = (op & 1) == 0;
    return *is_v ? op / 2 - 1 : (op + 1) / 2;
  };

  if (warp < 8) {
    // ------------------------------------------------ weights: groups A and B
    more_regs<kWeightRegs<QUANT>>();
    const int X = warp >> 2, gt = tid & 127, bar_id = 1 + X;   // gt: key, lane and row of the group
    const int n = !w.alt && X ? w.nb : w.na, col0 = !w.alt && X ? w.na : 0;
    const int tstep = w.alt ? 2 : 1, tfirst = w.alt ? X : 0;
    unsigned char *sP = sm + (X ? w.off_pb : w.off_pa);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 128 * X + lane_off, t_o = tmem + 256 + 128 * X + lane_off;
    float *neg_m = ss.neg_m[X], *fac = ss.fac[X];
    // while P is not in use: [4][128] of the warps, row places [128], [128] factors of B's part
    float *wred = reinterpret_cast<float *>(sP);
    int64_t *row_off = reinterpret_cast<int64_t *>(sP + 2048);
    float *fac_b = reinterpret_cast<float *>(sP + 3072);
    constexpr float kShift = DT == DT_F16 ? 8.0f : 0.0f;
    const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
    // a score that counts for nothing: -inf after the scaling (0 scale: see below)
    const float lowest = a.scale_log2 < 0.0f ? -ninf : ninf;
    uint32_t mine = 0, ring_op = 0;            // tiles of this group, ring places
    int slot = 0;
    while (next_segment()) {
      const uint32_t si = seg - 1;
      const Request rq = sg.rq;
      const int T = sg.t1 - sg.t0, rows = a.n * a.G, row0 = sg.rt * w.bm + col0;
      const int live_rows = min(min(n, w.bm - col0), rows - row0);    // of this group
      if (tid == 0 && a.prefix[sg.b] != rq.pre) cache_fault(a.c, sg.b);
      // keys before `pre` are seen by every (live) row of the unit
      // (row numbers fit 32 bits: a table has at most 2^20 pages of at most 128 rows)
      const int pre = static_cast<int>(a.mask ? rq.pre : rq.pre + sg.rt * w.bm / a.G);
      const int end = static_cast<int>(sg.end);
      const int32_t *table = a.c.table + static_cast<int64_t>(sg.b) * a.c.width;
      uint32_t *odd = ss.odd[si & 1];
      if (X == 0)
        for (int i = gt; i < kOddWords + 1; i += 128) odd[i] = 0u;
      // the rows of Q, K-major, 128-byte swizzle: a thread has one chunk of every
      // eighth (sixteenth) row, eight in flight
      if (!w.alt || X == 0) {
        if (w.alt && si > 0) wait(&ss.q_free, (si - 1) & 1);   // B's last scores are taken
        const int c = gt & (w.nblk * 8 - 1), step = 128 / (w.nblk * 8);
        const char *src = a.q + sg.b * a.qb + sg.hk * a.G * a.qh + c * 16;
        unsigned char *dst = sm + w.off_q + (c >> 3) * (w.na + w.nb) * 128 + col0 * 128;
#pragma unroll 1
        for (int r0 = gt / (w.nblk * 8); r0 < n; r0 += 8 * step) {
          uint4 x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = r0 + e * step;
            x[e] = make_uint4(0u, 0u, 0u, 0u);
            if (r < live_rows && c * 8 < dh) {
              const int i = (row0 + r) / a.G, g = row0 + r - i * a.G;
              x[e] = *reinterpret_cast<const uint4 *>(src + g * a.qh + i * a.qr);
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = r0 + e * step;
            if (r < n) *reinterpret_cast<uint4 *>(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x[e];
          }
        }
        fence_async_smem();
        mbar_arrive(&ss.q_full);
      } else {
        // B goes on once A has: A waits for q_free segment by segment, and a second
        // arrival of B before that would pass the phase that A waits for
        wait(&ss.q_full, si & 1);
      }
      float m = ninf;                 // reference of row gt of the group
      uint64_t l[kMaxCols / 2];       // sums of this thread's keys' weights, two rows each
#pragma unroll
      for (int c = 0; c < kMaxCols / 2; ++c) l[c] = 0ull;
      // whether this thread's key of tile t is there, on a good page
      auto key_there = [&](int t) {
        const int j = (sg.t0 + t) * kW + gt, page = j >> a.c.shift;
        return t < T && j < end && page < a.c.width &&
               static_cast<uint32_t>(table[page]) < static_cast<uint32_t>(a.c.pages);
      };
      bool valid = key_there(tfirst);

      for (int t = tfirst; t < T; t += tstep, ++mine) {
        const int j = (sg.t0 + t) * kW + gt;
        const bool first = t == tfirst;
        const bool masked = __any_sync(kFull, !valid || j >= pre);
        uint64_t bits[2] = {0ull, 0ull};          // the rows that see this thread's key
        if (masked && valid) {
          if (j < pre) {
            bits[0] = bits[1] = ~0ull;
          } else {
            // tree row j - rq.pre: eight tokens' loads in flight, then each token's run of rows
            const int tr = j - static_cast<int>(rq.pre), i0 = row0 / a.G;
            const uint8_t *mk =
                a.mask ? a.mask + (static_cast<int64_t>(sg.b) * a.n + i0) * a.n + tr : nullptr;
            const int tokens = min((row0 + live_rows - 1) / a.G + 1, rq.count) - i0;
            for (int i = 0; i < tokens; i += 8) {
              uint32_t v = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const bool in = i + e < tokens;
                v |= (in && (mk ? mk[static_cast<int64_t>(i + e) * a.n] != 0 : tr <= i0 + i + e) ? 1u : 0u) << e;
              }
#pragma unroll 1
              for (; v; v &= v - 1) {
                const int e = i0 + i + __ffs(v) - 1;
                set_run(bits, max(e * a.G - row0, 0), min((e + 1) * a.G - row0, live_rows));
              }
            }
          }
        }
        wait(&ss.s_full[X], mine & 1);
        if (!first) wait(&ss.pv_done[X], (mine - 1) & 1);   // P is free, O is whole
        __syncwarp();
        tmem_fence_after();
        if (w.alt && X == 1 && t + 2 >= T) mbar_arrive(&ss.q_free);
        if ((w.alt || X == 0) && masked) {
          // V rows that nobody sees become zeros, and so do values that are not finite in
          // tree rows (zero times them is NaN): the rows that see those get them below.
          // (The slot's tile before this one is consumed by now, K(t) at the latest with
          // three places and V(t - 1) with two, so this parity is this tile's.)
          const uint32_t vop = ring_op + (t < T - 1 ? 2 * t + 2 : 2 * T - 1);
          const uint32_t turn = vop / w.ring, vslot = vop - turn * w.ring;
          wait(&ss.full[vslot], turn & 1);
          unsigned char *v = sm + vslot * tile_bytes + gt * 128;
          bool found = false;
          if (!valid) {
#pragma unroll 4
            for (int c = 0; c < 8 * w.nblk; ++c)
              *reinterpret_cast<uint4 *>(v + (c >> 3) * kBlk + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          } else if (j >= pre) {
            uint32_t top = 0u;          // largest magnitudes, a NaN above all
#pragma unroll 4
            for (int c = 0; c < 8 * w.nblk; ++c) {
              const uint4 x = *reinterpret_cast<const uint4 *>(v + (c >> 3) * kBlk + (((c & 7) ^ (gt & 7)) << 4));
              top = top_abs<DT>(top_abs<DT>(top, x.x), top_abs<DT>(x.y, top_abs<DT>(x.z, x.w)));
            }
            const uint32_t ex = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
            if ((top & ex) == ex || ((top >> 16) & ex) == ex) {
              found = true;
#pragma unroll 1
              for (int c = 0; c < 64 * w.nblk; ++c) {
                uint16_t *x = reinterpret_cast<uint16_t *>(v + (c >> 6) * kBlk) + (c & 63);
                if ((*x & ex) == ex) *x = 0;
              }
            }
          }
          if (found) {
            // (a mask's rows, or the at most 192 that a causal unit's rows see in part)
            atomicOr(&odd[(j - pre) >> 5], 1u << ((j - pre) & 31));
            odd[kOddWords] = 1u;
          }
        }
        if (masked) {
          // scores that do not count become -inf in place; nothing below asks again
#pragma unroll 1
          for (int c = 0; c * 16 < n; ++c) {
            float v[16];
            tmem_ld16(t_s + 16 * c, v);
            tmem_wait_ld();
            const uint32_t b16 = static_cast<uint32_t>((c >= 4 ? bits[1] : bits[0]) >> ((c & 3) * 16));
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = (b16 >> e) & 1u ? v[e] : lowest;
            tmem_st16(t_s + 16 * c, v);
          }
          tmem_wait_st();
        }
        valid = key_there(t + tstep);
        if (first) new_refs(t_s, n, wred, gt, lane, bar_id, a.scale_log2, kShift, neg_m, fac, &m);
        uint32_t top = 0u;            // largest weights
        {
          float s0[16], s1[16];
          tmem_ld16(t_s, s0);
#pragma unroll
          for (int c = 0; c < kMaxCols / 16; ++c) {
            if (16 * c < n) {
              float *v = c & 1 ? s1 : s0;
              const ulonglong2 *r = reinterpret_cast<const ulonglong2 *>(neg_m + 16 * c);
              tmem_wait_ld();
              if (16 * c + 16 < n) {
                if (c & 1) tmem_ld16(t_s + 16 * c + 16, s0);
                else tmem_ld16(t_s + 16 * c + 16, s1);
              }
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float p0, p1;
                unpair(fma2(pair(v[2 * e], v[2 * e + 1]), scale2, e & 1 ? r[e >> 1].y : r[e >> 1].x), &p0, &p1);
                p0 = fast_exp2(p0);
                p1 = fast_exp2(p1);
                l[8 * c + e] = add2(l[8 * c + e], pair(p0, p1));
                y[e] = Half16<DT>::pack(p0, p1);
                top = max16x2<DT>(top, y[e]);
              }
              put_weights(sP, gt, c, y);
            }
          }
        }
        // weights are not negative: their bits order them (2^10; fp16 2^15)
        const uint32_t lim = DT == DT_BF16 ? 0x4480u : 0x7800u;
        if (group_any(bar_id, (top & 0xffffu) > lim || (top >> 16) > lim)) {
          // Rare. New references; what was summed so far is scaled to them, this tile's
          // weights are written anew. A sum past 2^100 is this tile's (what came before
          // it is below 2^-60 of it) and may have overflowed: it starts again.
          new_refs(t_s, n, wred, gt, lane, bar_id, a.scale_log2, kShift, neg_m, fac, &m);
#pragma unroll
          for (int c = 0; c < kMaxCols / 16; ++c) {
            if (16 * c < n) {
              float v[16];
              if (!first) {
                tmem_ld16(t_o + 16 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= fac[16 * c + e];
                tmem_st16(t_o + 16 * c, v);
              }
              tmem_ld16(t_s + 16 * c, v);
              tmem_wait_ld();
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float p0 = fast_exp2(fmaf(v[2 * e], a.scale_log2, neg_m[16 * c + 2 * e]));
                const float p1 = fast_exp2(fmaf(v[2 * e + 1], a.scale_log2, neg_m[16 * c + 2 * e + 1]));
                float l0, l1;
                unpair(l[8 * c + e], &l0, &l1);
                l0 = l0 > 0x1p100f ? p0 : l0 * fac[16 * c + 2 * e];
                l1 = l1 > 0x1p100f ? p1 : l1 * fac[16 * c + 2 * e + 1];
                l[8 * c + e] = pair(l0, l1);
                y[e] = Half16<DT>::pack(p0, p1);
              }
              put_weights(sP, gt, c, y);
            }
          }
          tmem_wait_st();
        }
        fence_async_smem();
        tmem_fence_before();
        mbar_arrive(&ss.p_full[X]);
      }
      if (w.alt && X == 1 && T < 2) mbar_arrive(&ss.q_free);
      // The unit's end: sums across lanes, then O^T, a lane's dimension of every row.
      const bool some = tfirst < T;
      if (some) wait(&ss.pv_done[X], (mine - 1) & 1);
      __syncwarp();
      tmem_fence_after();
      // (16 rows at a time through P's place: 16 lanes add up a pair of rows)
      float *part = reinterpret_cast<float *>(sP + 4096);
#pragma unroll
      for (int c = 0; c < kMaxCols / 16; ++c) {
        if (16 * c < n) {
#pragma unroll
          for (int e = 0; e < 8; ++e) *reinterpret_cast<uint64_t *>(part + (e * 128 + gt) * 2) = l[8 * c + e];
          sum_chunk(part, wred + 16 * c, gt, bar_id);
        }
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.tiles, both = w.alt && whole;
      const bool leave = !whole || (both && X == 1);      // a part for the join or for A
      const int DH = 64 * w.nblk;
      float *pp = a.part + (both ? (4ll * a.grid + 2 * blockIdx.x + (si & 1)) * a.slot
                                 : ((2ll * blockIdx.x + slot) * a.parts + (w.alt ? X : 0)) * a.slot);
      if (gt < live_rows) {
        const float sum = wred[gt];
        const int gr = row0 + gt, i = gr / a.G;
        const bool live = i < rq.count;
        if (leave) {
          fac[gt] = live ? 1.0f : 0.0f;
          pp[w.bm * DH + col0 + gt] = live ? m : ninf;
          pp[w.bm * (DH + 1) + col0 + gt] = live ? sum : 0.0f;
        } else {
          row_off[gt] = sg.b * a.ob + (sg.hk * a.G + (gr - i * a.G)) * a.oh + i * a.orow;
          if (both) {      // joined with B's part below
            fac[gt] = m;
            wred[gt] = sum;
          } else {
            fac[gt] = !live ? 0.0f : sum > 0.0f ? 1.0f / sum : sum == sum ? 0.0f : sum;
          }
        }
      }
      if (both && X == 0) {
        pair_sync();
        if (gt < live_rows) {
          const float ma = fac[gt], sa = wred[gt];
          const float mb = pp[w.bm * DH + gt], sb = pp[w.bm * (DH + 1) + gt], mm = fmaxf(ma, mb);
          const float fa = ma == ninf && sa == 0.0f ? 0.0f : fast_exp2(ma - mm);
          const float fb = mb == ninf && sb == 0.0f ? 0.0f : fast_exp2(mb - mm);
          const float all = sa * fa + sb * fb;
          const float inv = (row0 + gt) / a.G >= rq.count ? 0.0f
                            : all > 0.0f ? 1.0f / all : all == all ? 0.0f : all;
          fac[gt] = fa * inv;
          fac_b[gt] = fb * inv;
        }
      }
      group_sync(bar_id);
      const bool any_odd = odd[kOddWords] != 0u;
      const int d = (warp & 3) * 32 + lane;
#pragma unroll 1
      for (int c = 0; some && c * 16 < live_rows; ++c) {
        float o[16];
        tmem_ld16(t_o + 16 * c, o);
        tmem_wait_ld();
        if (any_odd && d < dh) {       // rare: values that are not finite
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            const int i = (row0 + 16 * c + e) / a.G;
            if (16 * c + e >= live_rows || i >= rq.count) continue;
            float add = 0.0f;
            for (int x = 0; x < 32 * kOddWords; ++x) {
              const int key = pre + x, kt = key / kW - sg.t0;
              if (!((odd[x >> 5] >> (x & 31)) & 1u) || key >= end || kt < tfirst || kt >= T ||
                  (w.alt && (kt & 1) != X) || !sees(a, rq, sg.b, i, key))
                continue;
              const int64_t row = cache_row(a.c, sg.b, key, sg.hk);
              if (row < 0) continue;
              const float v = QUANT ? row_scale(a.c.v_exp[row])
                                    : Half16<DT>::unpack(static_cast<const uint16_t *>(a.c.v)[row * dh + d]).x;
              if (v - v != 0.0f) add += v;
            }
#pragma unroll
            for (int z = 0; z < 16; ++z)
              if (z == e) o[z] += add;
          }
        }
        __syncwarp();
        // a dead row's O may hold anything: zero whatever it is
        if (d < dh) {
          // (all reads before the first store: it might, for all the compiler knows, change them)
          if (!leave) {
            float f[16];
            int64_t at[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              f[e] = fac[16 * c + e];
              at[e] = row_off[16 * c + e];
            }
            if (both) {
              const float *ob = pp + 16 * c * DH + d;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                o[e] = f[e] == 0.0f ? 0.0f : o[e] * f[e];
                f[e] = 1.0f;
                const float fb = 16 * c + e < live_rows ? fac_b[16 * c + e] : 0.0f;
                if (fb != 0.0f) o[e] += ob[e * DH] * fb;
              }
            }
            char *out = a.out + 2 * d;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (16 * c + e < live_rows)
                *reinterpret_cast<uint16_t *>(out + at[e]) =
                    static_cast<uint16_t>(Half16<DT>::pack(f[e] == 0.0f ? 0.0f : o[e] * f[e], 0.0f));
          } else {
            float *out = pp + (col0 + 16 * c) * DH + d;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fac[16 * c + e] == 0.0f ? 0.0f : o[e];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (16 * c + e < live_rows) out[e * DH] = o[e];
          }
        }
        __syncwarp();
      }
      tmem_fence_before();
      if (both && X == 1) pair_sync();
      group_sync(bar_id);            // wred, row_off and O are free
      ring_op += 2 * T;
      slot = 1;
    }
  } else if (QUANT && warp < 16) {
    fewer_regs<kOtherRegs<QUANT>>();
    {
      // ------------------------------- 8-bit rows to the operand tiles
      // two threads a row
      const int ct = tid & 127, half = (tid >> 7) & 1;
      Place r = {0, 0}, o = {0, 1};     // (an operand place starts free)
      bool stop = false;
      while (!stop && next_segment()) {
        const int T = sg.t1 - sg.t0;
#pragma unroll 1
        for (int x = 0; x < 2 * T; ++x) {
          const uint32_t rs = r.at, os = o.at;
          if (!wait(&ss.raw_full[rs], r.parity) || !wait(&ss.empty[os], o.parity)) {
            stop = true;
            break;
          }
          r.step(w.raw);
          o.step(w.ring);
          const unsigned char *raw = sm + w.off_raw + rs * w.raw_bytes;
          // Two threads have a row (its scale once), 16 codes at a time, chunks starting at a
          // place of the row's own so that eight lanes' chunks lie in eight bank groups, in
          // the raw tile and, swizzled as K's and V's always, in the operand tile.
          const uint32_t E = raw[kW * dh + ct];
          const unsigned char *src = raw + ct * dh;
          unsigned char *row = sm + os * tile_bytes + ct * 128;
          uint4 q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = (4 * half + i + ct) & 7;
            if (c < dh >> 4) q[i] = *reinterpret_cast<const uint4 *>(src + c * 16);
          }
          if (DT == DT_BF16 && (E <= 134u || E == 255u)) {
            // 2^(E - 127) 2^120 as a bf16 pair
            uint32_t mul = E == 255u ? 0x7fc0u : (E + 120u) << 7;
            mul |= mul << 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = (4 * half + i + ct) & 7;
              if (c >= dh >> 4) continue;
              const uint32_t qw[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[2 * e] = codes_bf16x2(spread_codes<0>(qw[e]), mul);
                y[2 * e + 1] = codes_bf16x2(spread_codes<1>(qw[e]), mul);
              }
              put_operand(row, ct, c, y);
            }
          } else {
            const float sc = row_scale(E);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = (4 * half + i + ct) & 7;
              if (c >= dh >> 4) continue;
              const uint32_t qw[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[2 * e] = e4m3_to16<DT>(qw[e] & 0xffffu, sc);
                y[2 * e + 1] = e4m3_to16<DT>(qw[e] >> 16, sc);
              }
              put_operand(row, ct, c, y);
            }
          }
          mbar_arrive(&ss.raw_empty[rs]);
          fence_async_smem();
          mbar_arrive(&ss.full[os]);
        }
      }
    }
  } else {
    fewer_regs<kOtherRegs<QUANT>>();
    const int role = warp - (QUANT ? 16 : 8);
    if (role == 0) {
      // ---------------------------------------------------------- loads
      Place r = {0, 1};
      uint32_t issued = 0;
      bool stop = false;
      const int slots = QUANT ? w.raw : w.ring;
      const int page = 1 << a.c.shift, pages = kW >> a.c.shift;
      uint64_t *full = QUANT ? ss.raw_full : ss.full, *empty = QUANT ? ss.raw_empty : ss.empty;
      while (!stop && next_segment()) {
        const int T = sg.t1 - sg.t0;
#pragma unroll 1
        for (int x = 0; x < 2 * T; ++x) {
          bool is_v;
          const int t = sg.t0 + op_tile(x, T, &is_v);
          const uint32_t s = r.at;
          if (!wait_warp(&empty[s], r.parity)) {
            stop = true;
            break;
          }
          r.step(slots);
          ++issued;
          // lane i: page i of the tile
          const int64_t j = static_cast<int64_t>(t) * kW + (static_cast<int64_t>(lane) << a.c.shift);
          int64_t row = -1;
          if (lane < pages && j < sg.end) {
            row = cache_row(a.c, sg.b, j, sg.hk);
            if (row < 0) cache_fault(a.c, sg.b);
          }
          const int have = __popc(__ballot_sync(kFull, row >= 0));
          if (lane == 0)
            mbar_expect_tx(&full[s], static_cast<uint32_t>(have) *
                                         (QUANT ? page * dh + page : page * 128 * w.nblk));
          __syncwarp();
          if (row >= 0) {
            if (QUANT) {
              unsigned char *dst = sm + w.off_raw + s * w.raw_bytes;
              bulk_g2s(dst + lane * page * dh, static_cast<const char *>(is_v ? a.c.v : a.c.k) + row * dh,
                       page * dh, &full[s]);
              bulk_g2s(dst + kW * dh + lane * page, (is_v ? a.c.v_exp : a.c.k_exp) + row, page, &full[s]);
            } else {
              unsigned char *dst = sm + s * tile_bytes + lane * page * 128;
              for (int kb = 0; kb < w.nblk; ++kb)
                tma_3d(dst + kb * kBlk, is_v ? &vmap : &kmap, 64 * kb, 0,
                       static_cast<int>(row >> a.c.shift), &full[s]);
            }
          }
        }
      }
      // no copy may be in flight when the block ends: wait (bounded) for the last ones
      for (int k = 0; k < slots; ++k, r.step(slots))
        if (issued >= static_cast<uint32_t>(slots) || r.at < issued)
          mbar_wait_cycles(&full[r.at], r.at < issued % slots ? (issued / slots) & 1
                                                              : (issued / slots - 1) & 1);
    } else if (role == 1) {
      // --------------------------------------------------------- products
      // The warp stays converged and one elected lane issues: descriptors are then
      // uniform values that need no move for each MMA.
      Place kp = {0, 0}, vp;            // the next operand tile; a V tile
      const uint32_t base = smem_u32(sm), q_blk = (w.na + w.nb) * 128;
      const uint64_t k0 = desc128(base, 16, 1024), v0 = desc128(base, w.nblk > 1 ? kBlk : 0, 1024);
      const int ks = dh >> 4, ng = w.alt ? 1 : 2;
      bool stop = false;
      auto scores = [&](int X, uint32_t s, uint64_t *free) {
        const bool second = !w.alt && X;      // the rows' second half
        const uint64_t kd = k0 + ((s * tile_bytes) >> 4);
        const uint64_t qd = k0 + ((w.off_q + (second ? w.na * 128 : 0)) >> 4);
        const uint32_t id = idesc16<DT>(second ? w.nb : w.na, false), to = tmem + 128 * X;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < ks)
              umma_bf16(to, kd + (k >> 2) * (kBlk >> 4) + (k & 3) * 2,
                        qd + (k >> 2) * (q_blk >> 4) + (k & 3) * 2, id, k > 0);
          umma_commit(&ss.s_full[X]);
          if (free) umma_commit(free);
        }
        __syncwarp();
      };
      auto values = [&](int X, uint32_t s, bool more, uint64_t *free) {
        const uint64_t vd = v0 + ((s * tile_bytes) >> 4);
        const uint64_t pd = desc128(base + (X ? w.off_pb : w.off_pa), kBlk, 1024);
        const uint32_t id = idesc16<DT>(!w.alt && X ? w.nb : w.na, true), to = tmem + 256 + 128 * X;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kW / 16; ++k) umma_bf16(to, vd + k * 128, pd + k * 128, id, more || k > 0);
          umma_commit(&ss.pv_done[X]);
          if (free) umma_commit(free);
        }
        __syncwarp();
      };
      uint32_t taken_a = 0, taken_b = 0;      // tiles of each group
      while (!stop && next_segment()) {
        const int T = sg.t1 - sg.t0;
        if (!wait_warp(&ss.q_full, (seg - 1) & 1) || !wait_warp(&ss.full[kp.at], kp.parity)) break;
        tmem_fence_after();
#pragma unroll 1
        for (int X = 0; X < ng; ++X) scores(X, kp.at, X == ng - 1 ? &ss.empty[kp.at] : nullptr);
        kp.step(w.ring);
#pragma unroll 1
        for (int t = 0; t < T && !stop; ++t) {
          const bool next = t + 1 < T;
          const Place k = kp;
          if (next) kp.step(w.ring);
          vp = kp;
          kp.step(w.ring);
          if (next && !wait_warp(&ss.full[k.at], k.parity)) { stop = true; break; }
          if (w.alt && next) scores((t + 1) & 1, k.at, &ss.empty[k.at]);
#pragma unroll 1
          for (int Y = 0; Y < ng; ++Y) {
            const int X = w.alt ? t & 1 : Y;
            const bool last = Y == ng - 1;
            if (!wait_warp(&ss.p_full[X], (X ? taken_b++ : taken_a++) & 1)) { stop = true; break; }
            tmem_fence_after();
            if (!w.alt && next) scores(X, k.at, last ? &ss.empty[k.at] : nullptr);
            if (Y == 0 && !wait_warp(&ss.full[vp.at], vp.parity)) { stop = true; break; }
            values(X, vp.at, t >= (w.alt ? 2 : 1), last ? &ss.empty[vp.at] : nullptr);
          }
        }
      }
    } else if (role == 2 && lane == 0) {
      // -------------------------------------------------------- segments
      Segment found;
      bool more = true;
      for (uint32_t i = 0; more; ++i) {
        more = !*fail && walk.next(a, w.bm, kW, &found);
        if (!more) found.b = -1;
        // (after a failure the others go through their segments without waiting)
        if (!mbar_wait_cycles(&ss.seg_empty[i % kSegs], ((i / kSegs) & 1) ^ 1)) *fail = 1;
        ss.seg[i % kSegs] = found;
        mbar_arrive(&ss.seg_full[i % kSegs]);
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's encoder, through the runtime (the library does not link the driver)
EncodeTiled encoder() {
  static EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) !=
            cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// pages as [pages * Hkv][page][dh], a box of 64 values x one page, 128-byte swizzled
bool make_map(const dt_cache &c, const void *base, CUtensorMap *map) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.dh), static_cast<cuuint64_t>(c.page),
                              static_cast<cuuint64_t>(c.pages) * c.Hkv};
  const cuuint64_t strides[2] = {2ull * c.dh, 2ull * c.dh * c.page};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(c.page), 1}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

WideShape wide_shape(const dt_cache &c, const AttnPlan &p) {
  WideShape w;
  w.bm = p.bm; w.na = p.na; w.nb = p.nb; w.alt = p.parts == 2; w.ring = p.ring; w.raw = p.raw;
  w.nblk = c.dh > 64 ? 2 : 1;
  w.raw_bytes = kW * c.dh + kW;
  w.off_q = p.ring * w.nblk * kBlk;
  w.off_pa = (w.off_q + (p.na + p.nb) * 128 * w.nblk + 1023) & ~1023;
  w.off_pb = w.off_pa + (p.na + 63) / 64 * kBlk;
  w.off_raw = w.off_pb + ((w.alt ? p.na : p.nb) + 63) / 64 * kBlk;
  w.off_small = w.off_raw + p.raw * w.raw_bytes;
  return w;
}

template <int DT, bool QUANT>
cudaError_t go(const AttnArgs &a, const WideShape &w, const AttnPlan &p, const CUtensorMap &k,
               const CUtensorMap &v, cudaStream_t st) {
  auto *kernel = cache_attention_wide_kernel<DT, QUANT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(p.smem));
  if (e != cudaSuccess) return e;
  kernel<<<a.grid, kWThreads<QUANT>, p.smem, st>>>(a, w, k, v);
  return cudaGetLastError();
}

}  // namespace

// Units of at most 96 rows (both groups the same) or, from 97 rows on, 192 (half the
// rows each), as equal as they come. False where the kernel does not apply.
bool wide_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p) {
  if (c.dh > 128 || static_cast<int64_t>(c.pages) * c.Hkv > 0x7fffffff) return false;
  const bool quant = c.dtype == DT_E4M3;
  p->parts = rows <= kMaxCols ? 2 : 1;
  const int64_t units = (rows + 2 * kMaxCols - 1) / (2 * kMaxCols);
  p->bm = static_cast<int>((rows + units - 1) / units);
  p->row_tiles = static_cast<int>((rows + p->bm - 1) / p->bm);
  if (p->parts == 2) {
    p->na = (p->bm + 15) & ~15;
    p->nb = 0;
  } else {
    p->na = ((p->bm + 1) / 2 + 15) & ~15;
    p->nb = (p->bm - p->na + 15) & ~15;
  }
  p->ring = p->raw = 0;
  const WideShape w = wide_shape(c, *p);
  const int tile = w.nblk * kBlk;
  const int room = smem - w.off_small - static_cast<int>(sizeof(Small));
  if (quant) {
    // three operand tiles (two where the rows leave no room), the rest for raw ones
    p->ring = p->parts == 2 || room >= 3 * tile + 2 * w.raw_bytes ? 3 : 2;
    p->raw = (room - p->ring * tile) / w.raw_bytes;
    if (p->raw > kMaxRing) p->raw = kMaxRing;
    if (p->raw < 2) return false;
  } else {
    p->ring = room / tile < kMaxRing ? room / tile : kMaxRing;
    if (p->ring < 3) return false;
  }
  p->dhp = 64 * w.nblk;
  p->grid = sms;
  p->smem = wide_shape(c, *p).off_small + sizeof(Small);
  p->wide = 1;
  return true;
}

cudaError_t launch_wide(const dt_cache &c, const AttnArgs &a, int dtype, const AttnPlan &p,
                        cudaStream_t st) {
  const WideShape w = wide_shape(c, p);
  CUtensorMap k = {}, v = {};
  const bool quant = c.dtype == DT_E4M3;
  if (!quant && (!make_map(c, c.k, &k) || !make_map(c, c.v, &v))) return cudaErrorInvalidValue;
  if (dtype == DT_BF16) return quant ? go<DT_BF16, true>(a, w, p, k, v, st) : go<DT_BF16, false>(a, w, p, k, v, st);
  return quant ? go<DT_F16, true>(a, w, p, k, v, st) : go<DT_F16, false>(a, w, p, k, v, st);
}

}  // namespace dt
