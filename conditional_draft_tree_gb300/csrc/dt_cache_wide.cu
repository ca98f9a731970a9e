// dt_cache_wide.cu -- attention over the paged cache on the tcgen05 tensor cores, for
// more than a few rows and head sizes up to 128.
//
// The rows of a (request, key/value head), G heads x tree rows, are cut into tiles of at
// most 128 rows, as equal as they come; a unit is two of them (A and B), which share each
// K and V tile of 128 keys, or the one that is left over. Per tile: S = Q K^T (Q and K
// K-major in shared memory, S in TMEM, a thread a row), x = S scale log2(e) in one pass for
// the row's maximum and one for its weights p = 2^(x - m), which go back to TMEM as the
// first operand of O += P V (V as it is stored, MN-major). Maximum, sum and weights of a
// row stay in its thread: no shuffle, no barrier, no shared memory. m follows the
// maximum only when that has grown by 2^8 (fp16: 2^4), and only then are O and the sum
// rescaled; any reference at most that far below the maximum gives the same quotient.
//
// What bounds it is the shared memory's 128 bytes a cycle as much as the tensor cores: an
// MMA of 128 x 128 x 16 takes 64 cycles and reads 4 KB of each operand that is there. P
// from TMEM halves that for the second product. (A version with both products transposed,
// rows on the N side in steps of 16 and P^T through shared memory, was bound by it: 1.0 ms
// where this one takes 0.58 ms for 8 trees of 129 rows over 16384 to 32768 8-bit rows.)
// Measured, 32 / 8 heads, dh 128: 8 trees of 129 rows over 32768 bf16 rows 0.63 ms, 880
// TFLOP/s (0.46 of what a large matrix product reaches), 8-bit rows 0.75 ms, with fp16
// queries, whose weights are two products, 1.06 ms; 32 trees of 65 rows over 512 to 1024
// rows 0.10 ms. There a block has two or three units, and their beginnings (Q, masks) and
// ends (O to memory), some 15 thousand cycles each, are as long as their products.
//
// While one group takes its weights the tensor cores work for the other. In a unit of a
// single tile both groups have the same rows, A the even key tiles and B the odd ones,
// and A or the join adds them up. K and V tiles pass through a ring in the order in which
// they are consumed, filled by TMA, page by page, through a 128-byte
// swizzled tensor map; tiles of 8-bit rows land in a raw ring by plain bulk copies and two
// warpgroups write their bf16 or fp16 values into the operand ring.
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
constexpr int kOddWords = (DT_MAX_N + 32) / 32;
constexpr long long kWaitCycles = 4000000000ll;   // about 2 s

// Warpgroups: two for weights, two (8-bit rows) that convert, one whose warps load, issue
// the products and find segments. Registers at launch times threads is what setmaxnreg
// shares out: 640 x 96 >= 256 x 144 + 384 x 64.
template <bool QUANT> constexpr int kWThreads = QUANT ? 640 : 384;

struct WideShape {
  int tr, odd, ring, raw, nblk, raw_bytes;   // rows of a tile; whether the last unit is one tile
  int off_q, off_raw, off_small;
};

struct Small {                          // behind the big buffers
  uint64_t full[kMaxRing], empty[kMaxRing], raw_full[kMaxRing], raw_empty[kMaxRing];
  uint64_t q_full, q_free, s_full[2], p_full[2], o_done[2], idle;
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

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 bytes (aligned) of global memory
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// both warpgroups: a part of one unit handed from B to A through global memory
__device__ __forceinline__ void pair_sync() {
  __threadfence_block();
  asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
}
// one warpgroup
__device__ __forceinline__ void group_sync(int X) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + X) : "memory");
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
// largest magnitudes of two pairs of 16-bit values (signs are not kept), NaN above all
template <int DT>
__device__ __forceinline__ uint32_t top_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == DT_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// instruction descriptor of kind::f16, M = 128, fp32 accumulation; mn: B is MN-major
template <int DT>
__device__ __forceinline__ uint32_t idesc16(int N, bool mn) {
  const uint32_t f = DT == DT_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | ((128u >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]^T
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
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
  // fp16 rows over 8-bit ones: V's values (as many as 2^137 apart) in bf16, where they are
  // exact, against the weights in two bf16 terms; K's in fp16, rounded as dt_cache_read does
  constexpr bool TWO = QUANT && DT == DT_F16;
  constexpr int VDT = TWO ? DT_BF16 : DT;
  extern __shared__ __align__(1024) unsigned char sm[];
  Small &ss = *reinterpret_cast<Small *>(sm + w.off_small);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int dh = a.c.dh, tile_bytes = w.nblk * kBlk, bm = 2 * w.tr;
  const float ninf = -__int_as_float(0x7f800000);

  if (tid == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&ss.full[i], QUANT ? 128 : 1);
      mbar_init(&ss.empty[i], 1);
      mbar_init(&ss.raw_full[i], 1);
      mbar_init(&ss.raw_empty[i], 128);
    }
    mbar_init(&ss.q_full, 256);
    mbar_init(&ss.q_free, 1);
    mbar_init(&ss.idle, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&ss.seg_full[i], 1);
      mbar_init(&ss.seg_empty[i], QUANT ? 18 : 10);   // the warps that take segments
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ss.s_full[x], 1);
      mbar_init(&ss.p_full[x], 128);
      mbar_init(&ss.o_done[x], 1);
    }
    ss.fail = 0;
  }
  if (warp == 0) tmem_alloc(&ss.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = ss.tmem;

  Schedule<kWThreads<QUANT>> sch;
  sch.plan(a, bm, kW, ss.scan);
  Walk walk;
  walk.at = blockIdx.x * sch.chunk;
  walk.stop = min(walk.at + sch.chunk, sch.total);
  walk.b = 0;
  walk.base = 0;
  if (walk.at < walk.stop) sch.find(a, bm, kW, walk.at, ss.scan, &walk.b, &walk.base);
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
  // a unit of a single tile of rows
  auto single = [&]() { return w.odd && sg.rt == a.row_tiles - 1; };
  // Operand tiles of a segment of T key tiles in ring order, which is the order in which
  // they are consumed: K0 V0 K1 V1 ... in a unit of two row tiles, and K0 K1 V0 K2 V1 ...
  // V(T-1) in a unit of one, where a tile's scores are taken before the weights of the one
  // before it. (That a tile is consumed then says the same of all before it, on which the
  // waits below rely: a barrier's parity tells two phases apart, not three.)
  auto op_tile = [&](int op, int T, bool *is_v) {
    if (!single()) {
      *is_v = op & 1;
      return op >> 1;
    }
    if (op == 0) { *is_v = false; return 0; }
    if (op == 2 * T - 1) { *is_v = true; return T - 1; }
    *is_v = (op & 1) == 0;
    return *is_v ? op / 2 - 1 : (op + 1) / 2;
  };

  if (warp < 8) {
    // ------------------------------------------------ weights: groups A and B
    if (QUANT) asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int X = warp >> 2, gt = tid & 127;      // gt: the group's row, TMEM lane (and key)
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 128 * X + lane_off, t_o = tmem + 256 + 128 * X + lane_off;
    // fp16 weights are scaled by 2^8, so that small ones stay normal numbers
    constexpr float kShift = VDT == DT_F16 ? 8.0f : 0.0f;
    constexpr float kGrow = VDT == DT_F16 ? 4.0f : 8.0f;
    const float scale = fabsf(a.scale_log2);
    const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;   // the scale's sign goes to Q
    const uint64_t scale2 = pair(scale, scale);
    const int DH = 64 * w.nblk;
    uint32_t mine = 0, segs_mine = 0, ring_op = 0;  // tiles, segments of this group, ring places
    while (next_segment()) {
      const uint32_t si = seg - 1;
      const Request rq = sg.rq;
      const bool alt = single();
      const int T = sg.t1 - sg.t0, tstep = alt ? 2 : 1, tfirst = alt ? X : 0;
      const int col0 = alt ? 0 : X * w.tr, row = sg.rt * bm + col0 + gt;     // stacked query row
      const int tok = row / a.G, head = sg.hk * a.G + row - tok * a.G;
      const bool real = gt < w.tr && row < a.n * a.G, live = real && tok < rq.count;
      if (tid == 0 && a.prefix[sg.b] != rq.pre) cache_fault(a.c, sg.b);
      // keys before `pre` are seen by every (live) row of the unit
      // (row numbers fit 32 bits: a table has at most 2^20 pages of at most 128 rows)
      const int pre = static_cast<int>(a.mask ? rq.pre : rq.pre + sg.rt * bm / a.G);
      const int end = static_cast<int>(sg.end), whole_end = min(pre, end);
      const int32_t *table = a.c.table + static_cast<int64_t>(sg.b) * a.c.width;
      uint32_t *odd = ss.odd[si & 1];
      if (X == 0)
        for (int i = gt; i < kOddWords + 1; i += 128) odd[i] = 0u;
      if (si > 0) wait(&ss.q_free, (si - 1) & 1);
      // the thread's row of Q, K-major, 128-byte swizzle
      if (real && (!alt || X == 0)) {
        const char *src = a.q + sg.b * a.qb + head * a.qh + tok * a.qr;
        unsigned char *dst = sm + w.off_q + (alt ? 0 : X * tile_bytes) + gt * 128;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          uint4 x[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (kb < w.nblk && 64 * kb + 8 * c < dh) x[c] = reinterpret_cast<const uint4 *>(src)[8 * kb + c];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (kb < w.nblk && 64 * kb + 8 * c < dh) {
              x[c].x ^= flip; x[c].y ^= flip; x[c].z ^= flip; x[c].w ^= flip;
              *reinterpret_cast<uint4 *>(dst + kb * kBlk + ((c ^ (gt & 7)) << 4)) = x[c];
            }
        }
      }
      fence_async_smem();
      mbar_arrive(&ss.q_full);
      float m = ninf;                       // reference of this thread's row
      uint64_t l2[2] = {0ull, 0ull};        // its sum, in four parts
      // page number `lane` of key tile t, 0 in lanes that have none, -1 outside the table;
      // loaded a tile ahead of its use
      const int pages = kW >> a.c.shift;
      auto page_of = [&](int t) {
        const int page = (((sg.t0 + t) * kW) >> a.c.shift) + lane;
        if (t >= T || lane >= pages || (page << a.c.shift) >= end) return 0;
        return page < a.c.width ? table[page] : -1;
      };
      int entry = page_of(tfirst);

#pragma unroll 1
      for (int t = tfirst; t < T; t += tstep, ++mine) {
        const int j0 = (sg.t0 + t) * kW;
        const uint32_t bad_pages =
            __ballot_sync(kFull, static_cast<uint32_t>(entry) >= static_cast<uint32_t>(a.c.pages));
        const bool masked = bad_pages != 0u || j0 + kW > whole_end;
        entry = page_of(t + tstep);
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};     // keys of the tile that the row sees
        if (masked) {
          // the warp's rows' tokens, four at a time, a lane a key of each of four words
          const int lo = __shfl_sync(kFull, tok, 0), hi = min(__shfl_sync(kFull, tok, 31), rq.count - 1);
          const int pre0 = static_cast<int>(rq.pre);
          bool there[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            there[q] = j0 + 32 * q + lane < end && !((bad_pages >> ((32 * q + lane) >> a.c.shift)) & 1u);
            see[q] = __ballot_sync(kFull, there[q]);
          }
#pragma unroll 1
          for (int i = lo; i <= hi; i += 4) {
            uint32_t v = 0u;      // bit 4 q + e: key of word q seen by token i + e
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int tr = j0 + 32 * q + lane - pre0;
              const bool tree = there[q] && tr >= 0 && tr < rq.count;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                bool x = there[q] && tr < 0;
                if (tree && i + e <= hi)
                  x = a.mask ? a.mask[(static_cast<int64_t>(sg.b) * a.n + i + e) * a.n + tr] != 0 : tr <= i + e;
                v |= x ? 1u << (4 * q + e) : 0u;
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t x = __ballot_sync(kFull, (v >> (4 * q + e)) & 1u);
                if (tok == i + e) see[q] = x;
              }
          }
          if (!live) see[0] = see[1] = see[2] = see[3] = 0u;
        }
        wait(&ss.s_full[X], mine & 1);
        __syncwarp();
        tmem_fence_after();
        if (masked && (alt || X == 0)) {
          // V rows that nobody sees become zeros, and so do values that are not finite in
          // tree rows (zero times them is NaN): the rows that see those get them below. The
          // thread takes the row of key gt. (S of tile t is complete, and with it every
          // product issued before; the ring has at least three places, so the tile that was
          // in this one is consumed and the parity waited for is this tile's.)
          const uint32_t vop = ring_op + (!alt ? 2 * t + 1 : t < T - 1 ? 2 * t + 2 : 2 * T - 1);
          const uint32_t turn = vop / w.ring, vslot = vop - turn * w.ring;
          wait(&ss.full[vslot], turn & 1);
          unsigned char *v = sm + vslot * tile_bytes + gt * 128;
          const int j = j0 + gt;
          if (j >= end || ((bad_pages >> (gt >> a.c.shift)) & 1u)) {
#pragma unroll 4
            for (int c = 0; c < 8 * w.nblk; ++c)
              *reinterpret_cast<uint4 *>(v + (c >> 3) * kBlk + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          } else if (j >= pre) {
            uint32_t top = 0u;          // largest magnitudes, a NaN above all
#pragma unroll 4
            for (int c = 0; c < 8 * w.nblk; ++c) {
              const uint4 x = *reinterpret_cast<const uint4 *>(v + (c >> 3) * kBlk + (((c & 7) ^ (gt & 7)) << 4));
              top = top_abs<VDT>(top_abs<VDT>(top, x.x), top_abs<VDT>(x.y, top_abs<VDT>(x.z, x.w)));
            }
            const uint32_t ex = VDT == DT_BF16 ? 0x7f80u : 0x7c00u;
            if ((top & ex) == ex || ((top >> 16) & ex) == ex) {
#pragma unroll 1
              for (int c = 0; c < 64 * w.nblk; ++c) {
                uint16_t *x = reinterpret_cast<uint16_t *>(v + (c >> 6) * kBlk) + (c & 63);
                if ((*x & ex) == ex) *x = 0;
              }
              // (a mask's rows, or the at most 256 that a causal unit's rows see in part)
              atomicOr(&odd[(j - pre) >> 5], 1u << ((j - pre) & 31));
              odd[kOddWords] = 1u;
            }
          }
          fence_async_smem();
        }
        if (masked) {
          // scores that do not count become -inf in place; nothing below asks again
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (__all_sync(kFull, see[q] == ~0u)) continue;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              float v[16];
              tmem_ld16(t_s + 32 * q + 16 * h, v);
              tmem_wait_ld();
              const uint32_t b16 = see[q] >> (16 * h);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = (b16 >> e) & 1u ? v[e] : ninf;
              tmem_st16(t_s + 32 * q + 16 * h, v);
            }
          }
          tmem_wait_st();
        }
        // the row's maximum
        float top = ninf;
        {
          float s0[16], s1[16];
          tmem_ld16(t_s, s0);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float *v = c & 1 ? s1 : s0;
            tmem_wait_ld();
            if (c < 7) {
              if (c & 1) tmem_ld16(t_s + 16 * c + 16, s0);
              else tmem_ld16(t_s + 16 * c + 16, s1);
            }
            float x = fmaxf(v[0], v[1]), y = fmaxf(v[2], v[3]);    // 3-input maxima
#pragma unroll
            for (int e = 4; e < 16; e += 4) {
              x = fmaxf(fmaxf(x, v[e]), v[e + 1]);
              y = fmaxf(fmaxf(y, v[e + 2]), v[e + 3]);
            }
            top = fmaxf(fmaxf(top, x), y);
          }
        }
        top *= scale;
        const bool grow = live && (top > m + kGrow || (m == ninf && top != ninf));
        if (__any_sync(kFull, grow)) {
          const float f = grow ? (m == ninf ? 0.0f : fast_exp2(m - top)) : 1.0f;
          if (grow) m = top;
          float a0, a1, b0, b1;
          unpair(l2[0], &a0, &a1);
          unpair(l2[1], &b0, &b1);
          l2[0] = pair(a0 * f, a1 * f);
          l2[1] = pair(b0 * f, b1 * f);
          if (t != tfirst) {
#pragma unroll 1
            for (int c = 0; c < dh; c += 16) {
              float o[16];
              tmem_ld16(t_o + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tmem_st16(t_o + c, o);
            }
            tmem_wait_st();
          }
        }
        // the weights, written over the scores: 8 columns a chunk from the first on, or, of two
        // terms, over the chunk's own 16 columns
        {
          const float nm = m == ninf ? 0.0f : kShift - m;
          const uint64_t nm2 = pair(nm, nm);
          float s0[16], s1[16];
          tmem_ld16(t_s, s0);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float *v = c & 1 ? s1 : s0;
            tmem_wait_ld();
            if (c < 7) {
              if (c & 1) tmem_ld16(t_s + 16 * c + 16, s0);
              else tmem_ld16(t_s + 16 * c + 16, s1);
            }
            uint32_t y[8], lo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float p0, p1;
              unpair(fma2(pair(v[2 * e], v[2 * e + 1]), scale2, nm2), &p0, &p1);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              l2[e & 1] = add2(l2[e & 1], pair(p0, p1));
              y[e] = Half16<VDT>::pack(p0, p1);
              if (TWO) {
                const float2 hi = Half16<VDT>::unpack(y[e]);
                lo[e] = Half16<VDT>::pack(p0 - hi.x, p1 - hi.y);
              }
            }
            // (the next chunk's scores are being read: columns 16 c + 16 on)
            tmem_st8(t_s + (TWO ? 16 : 8) * c, y);
            if (TWO) tmem_st8(t_s + 16 * c + 8, lo);
          }
          tmem_wait_st();
        }
        tmem_fence_before();
        mbar_arrive(&ss.p_full[X]);
      }
      // The unit's end: O of this thread's row.
      const bool some = tfirst < T;
      if (some) wait(&ss.o_done[X], segs_mine++ & 1);
      __syncwarp();
      tmem_fence_after();
      float sum;
      {
        float a0, a1, b0, b1;
        unpair(l2[0], &a0, &a1);
        unpair(l2[1], &b0, &b1);
        sum = (a0 + a1) + (b0 + b1);
      }
      if (!live) {
        m = ninf;
        sum = 0.0f;
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.tiles, both = alt && whole;
      const bool leave = !whole || (both && X == 1);      // a part for the join or for A
      float *pp = a.part + (both ? (4ll * a.grid + 2 * blockIdx.x + (si & 1)) * a.slot
                                 : ((2ll * blockIdx.x + (sg.t0 > 0 ? 0 : 1)) * 2 + (alt ? X : 0)) * a.slot);
      if (leave && real) {
        pp[bm * DH + col0 + gt] = m;
        pp[bm * (DH + 1) + col0 + gt] = sum;
      }
      float f = leave ? 1.0f : 0.0f, fb = 0.0f;           // factors of O and of B's part
      if (both && X == 0) {
        pair_sync();
        if (live) {
          const float mb = pp[bm * DH + gt], sb = pp[bm * (DH + 1) + gt], mm = fmaxf(m, mb);
          const float fa = m == ninf && sum == 0.0f ? 0.0f : fast_exp2(m - mm);
          fb = mb == ninf && sb == 0.0f ? 0.0f : fast_exp2(mb - mm);
          const float all = sum * fa + sb * fb;
          const float inv = all > 0.0f ? 1.0f / all : all == all ? 0.0f : all;
          f = fa * inv;
          fb *= inv;
        }
      } else if (!leave && live) {
        f = sum > 0.0f ? 1.0f / sum : sum == sum ? 0.0f : sum;
      }
      if (!live) f = 0.0f;
      group_sync(X);                        // odd[] is complete
      const bool any_odd = odd[kOddWords] != 0u;
      char *out = a.out + sg.b * a.ob + head * a.oh + tok * a.orow;
      float *po = pp + (col0 + gt) * DH;
#pragma unroll 1
      for (int c = 0; c < dh; c += 16) {
        float o[16];
        tmem_ld16(t_o + c, o);
        tmem_wait_ld();
        if (any_odd && live && some) {        // rare: values that are not finite
#pragma unroll 1
          for (int x = 0; x < 32 * kOddWords; ++x) {
            const int key = pre + x, kt = key / kW - sg.t0;
            if (!((odd[x >> 5] >> (x & 31)) & 1u) || key >= end || kt < tfirst || kt >= T ||
                (alt && (kt & 1) != X) || !sees(a, rq, sg.b, tok, key))
              continue;
            const int64_t at = cache_row(a.c, sg.b, key, sg.hk);
            if (at < 0) continue;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float v = QUANT ? row_scale(a.c.v_exp[at])
                                    : Half16<DT>::unpack(static_cast<const uint16_t *>(a.c.v)[at * dh + c + e]).x;
              if (v - v != 0.0f) o[e] += v;
            }
          }
        }
        // a dead row's O may hold anything: zero whatever it is
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = f == 0.0f || !some ? 0.0f : o[e] * f;
        if (real && leave) {
          store32(po + c, reinterpret_cast<uint32_t(&)[8]>(o[0]));
          store32(po + c + 8, reinterpret_cast<uint32_t(&)[8]>(o[8]));
        } else if (real) {
          if (fb != 0.0f) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 x = *reinterpret_cast<const float4 *>(po + c + e);
              o[e] += x.x * fb; o[e + 1] += x.y * fb; o[e + 2] += x.z * fb; o[e + 3] += x.w * fb;
            }
          }
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = Half16<DT>::pack(o[2 * e], o[2 * e + 1]);
          if (((reinterpret_cast<uintptr_t>(a.out) | a.ob | a.oh | a.orow) & 31) == 0) {   // whole sectors
            store32(out + 2 * c, y);
          } else {
            *reinterpret_cast<uint4 *>(out + 2 * c) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4 *>(out + 2 * c + 16) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
        __syncwarp();
      }
      tmem_fence_before();
      if (both && X == 1) pair_sync();
      ring_op += 2 * T;
    }
  } else if (QUANT && warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    {
      // ------------------------------- 8-bit rows to the operand tiles
      // one warpgroup the K tiles, the other the V tiles: a tile's waits and fences pass
      // while the other is converted
      const int ct = tid & 127;
      const bool mine_v = (tid >> 7) & 1;
      Place r = {0, 0}, o = {0, 1};     // (an operand place starts free)
      bool stop = false;
      while (!stop && next_segment()) {
        const int T = sg.t1 - sg.t0;
#pragma unroll 1
        for (int x = 0; x < 2 * T; ++x) {
          bool is_v;
          op_tile(x, T, &is_v);
          const Place rp = r, op = o;
          const uint32_t rs = rp.at, os = op.at;
          r.step(w.raw);
          o.step(w.ring);
          if (is_v != mine_v) continue;
          // First the operand's place: it is free once the tile three before this one is
          // consumed, which has been converted then, and all before it, so that the raw
          // place's phase is this tile's (there are at least three raw places).
          if (!wait(&ss.empty[os], op.parity) || !wait(&ss.raw_full[rs], rp.parity)) {
            stop = true;
            break;
          }
          const unsigned char *raw = sm + w.off_raw + rs * w.raw_bytes;
          // A thread has a row (its scale once), 16 codes at a time, chunks starting at a
          // place of the row's own so that eight lanes' chunks lie in eight bank groups, in
          // the raw tile and, swizzled as K's and V's always, in the operand tile.
          const uint32_t E = raw[kW * dh + ct];
          const unsigned char *src = raw + ct * dh;
          unsigned char *row = sm + os * tile_bytes + ct * 128;
          if ((DT == DT_BF16 || mine_v) && (E <= 134u || E == 255u)) {
            // 2^(E - 127) 2^120 as a bf16 pair
            uint32_t mul = E == 255u ? 0x7fc0u : (E + 120u) << 7;
            mul |= mul << 16;
#pragma unroll 4
            for (int i = 0; i < 8; ++i) {
              const int c = (i + ct) & 7;
              if (c >= dh >> 4) continue;
              const uint4 q = *reinterpret_cast<const uint4 *>(src + c * 16);
              const uint32_t y[8] = {
                  codes_bf16x2(spread_codes<0>(q.x), mul), codes_bf16x2(spread_codes<1>(q.x), mul),
                  codes_bf16x2(spread_codes<0>(q.y), mul), codes_bf16x2(spread_codes<1>(q.y), mul),
                  codes_bf16x2(spread_codes<0>(q.z), mul), codes_bf16x2(spread_codes<1>(q.z), mul),
                  codes_bf16x2(spread_codes<0>(q.w), mul), codes_bf16x2(spread_codes<1>(q.w), mul)};
              put_operand(row, ct, c, y);
            }
          } else if (DT == DT_F16 && !mine_v && E >= 103u && E <= 134u) {
            // 2^(E - 127) and the codes are fp16 numbers, and no product is above 448 2^7: one
            // multiplication rounds as dt_cache_read does
            uint32_t mul = E >= 113u ? (E - 112u) << 10 : 1u << (E - 103u);
            mul |= mul << 16;
            const __half2 mul2 = *reinterpret_cast<const __half2 *>(&mul);
            auto times = [&](uint32_t two) {
              const uint32_t f = e4m3_f16x2(two);
              const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&f), mul2);
              return *reinterpret_cast<const uint32_t *>(&r);
            };
#pragma unroll 4
            for (int i = 0; i < 8; ++i) {
              const int c = (i + ct) & 7;
              if (c >= dh >> 4) continue;
              const uint4 q = *reinterpret_cast<const uint4 *>(src + c * 16);
              const uint32_t y[8] = {times(q.x & 0xffffu), times(q.x >> 16), times(q.y & 0xffffu), times(q.y >> 16),
                                     times(q.z & 0xffffu), times(q.z >> 16), times(q.w & 0xffffu), times(q.w >> 16)};
              put_operand(row, ct, c, y);
            }
          } else {
            const float sc = row_scale(E);
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
              const int c = (i + ct) & 7;
              if (c >= dh >> 4) continue;
              const uint4 q = *reinterpret_cast<const uint4 *>(src + c * 16);
              const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[2 * e] = mine_v ? e4m3_to16<VDT>(qw[e] & 0xffffu, sc) : e4m3_to16<DT>(qw[e] & 0xffffu, sc);
                y[2 * e + 1] = mine_v ? e4m3_to16<VDT>(qw[e] >> 16, sc) : e4m3_to16<DT>(qw[e] >> 16, sc);
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
    if (QUANT) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
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
      const uint32_t base = smem_u32(sm);
      const uint64_t k0 = desc128(base, 16, 1024), v0 = desc128(base, kBlk, 1024);
      const uint32_t id_s = idesc16<DT>(kW, false), id_o = idesc16<VDT>(dh, true);
      const int ks = dh >> 4;
      Place op = {0, 0};               // the next operand tile
      uint32_t taken_a = 0, taken_b = 0;      // tiles of each group
      bool stop = false;
      // S of group X from K tile s; `free`, `q_free`: the last reader of that tile, of Q
      auto scores = [&](int X, bool second, uint32_t s, bool free, bool q_free) {
        const uint64_t kd = k0 + ((s * tile_bytes) >> 4);
        const uint64_t qd = k0 + ((w.off_q + (second ? tile_bytes : 0)) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < ks) {
              const int at = (k >> 2) * (kBlk >> 4) + (k & 3) * 2;
              umma_bf16(tmem + 128 * X, qd + at, kd + at, id_s, k > 0);
            }
          umma_commit(&ss.s_full[X]);
          if (free) umma_commit(&ss.empty[s]);
          if (q_free) umma_commit(&ss.q_free);
        }
        __syncwarp();
      };
      auto values = [&](int X, uint32_t s, bool more, bool free, bool last) {
        const uint64_t vd = v0 + ((s * tile_bytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kW / 16; ++k)
            umma_ts(tmem + 256 + 128 * X, tmem + 128 * X + (TWO ? 16 : 8) * k, vd + k * 128, id_o, more || k > 0);
          if (TWO)
#pragma unroll
            for (int k = 0; k < kW / 16; ++k)
              umma_ts(tmem + 256 + 128 * X, tmem + 128 * X + 16 * k + 8, vd + k * 128, id_o, true);
          if (last) umma_commit(&ss.o_done[X]);
          if (free) umma_commit(&ss.empty[s]);
        }
        __syncwarp();
      };
      while (!stop && next_segment()) {
        const bool alt = single();
        const int T = sg.t1 - sg.t0;
        Place k = op, v;
        op.step(w.ring);
        if (!wait_warp(&ss.q_full, (seg - 1) & 1) || !wait_warp(&ss.full[k.at], k.parity)) break;
        tmem_fence_after();
        scores(0, false, k.at, alt, alt && T == 1);
        if (!alt) scores(1, true, k.at, true, T == 1);
        // `k`: the K tile of step t + 1, whose scores of groups A, B (of alternating groups:
        // group B's, already) are issued in step t
        for (int t = 0; t < T && !stop; ++t) {
          const bool next = t + 1 < T;
          if (alt) {
            k = op;
            if (next) op.step(w.ring);
            v = op;
            op.step(w.ring);
            // S of tile t + 1 has a group of its own: before the weights of tile t
            if (next) {
              if (!wait_warp(&ss.full[k.at], k.parity)) { stop = true; break; }
              // (from tile 2 on behind the group's last product, which read its weights)
              scores((t + 1) & 1, false, k.at, true, t + 2 == T);
            }
            const int X = t & 1;
            if (!wait_warp(&ss.p_full[X], (X ? taken_b++ : taken_a++) & 1) ||
                !wait_warp(&ss.full[v.at], v.parity)) { stop = true; break; }
            tmem_fence_after();
            values(X, v.at, t >= 2, true, t + 2 >= T);
          } else {
            v = op;
            op.step(w.ring);
            k = op;
            if (next) op.step(w.ring);
            for (int X = 0; X < 2; ++X) {
              if (!wait_warp(&ss.p_full[X], (X ? taken_b++ : taken_a++) & 1) ||
                  (X == 0 && !wait_warp(&ss.full[v.at], v.parity)) ||
                  (X == 0 && next && !wait_warp(&ss.full[k.at], k.parity))) { stop = true; break; }
              tmem_fence_after();
              values(X, v.at, t > 0, X == 1, !next);
              if (next) scores(X, X == 1, k.at, X == 1, X == 1 && t + 2 == T);
            }
          }
        }
      }
      // No product may be under way when the block gives back its tensor memory and ends,
      // also after a wait that ran out: the last arrival follows all of them (bounded).
      if (elect_one()) umma_commit(&ss.idle);
      __syncwarp();
      mbar_wait_cycles(&ss.idle, 0);
    } else if (role == 2 && lane == 0) {
      // -------------------------------------------------------- segments
      Segment found;
      bool more = true;
      for (uint32_t i = 0; more; ++i) {
        more = !*fail && walk.next(a, bm, kW, &found);
        if (i == 0) walk.note_cut(a, sch.chunk, more, found);
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

WideShape wide_shape(const dt_cache &c, const AttnPlan &p) {
  WideShape w;
  w.tr = p.bm / 2; w.odd = p.odd; w.ring = p.ring; w.raw = p.raw;
  w.nblk = c.dh > 64 ? 2 : 1;
  w.raw_bytes = kW * c.dh + kW;
  w.off_q = p.ring * w.nblk * kBlk;
  w.off_raw = w.off_q + (p.odd && p.row_tiles == 1 ? 1 : 2) * w.nblk * kBlk;
  w.off_small = w.off_raw + p.raw * w.raw_bytes;
  return w;
}

template <int DT, bool QUANT>
cudaError_t go(const AttnArgs &a, const WideShape &w, const AttnPlan &p, const CUtensorMap &k,
               const CUtensorMap &v, cudaStream_t st) {
  const cudaError_t e = allow_smem<cache_attention_wide_kernel<DT, QUANT>>();
  if (e != cudaSuccess) return e;
  cache_attention_wide_kernel<DT, QUANT><<<a.grid, kWThreads<QUANT>, p.smem, st>>>(a, w, k, v);
  return cudaGetLastError();
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

}  // namespace

// pages as [pages * Hkv][page][dh], a box of 128 bytes of `box_rows` rows, swizzled
bool page_map(const dt_cache &c, const void *base, int box_rows, CUtensorMap *map) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.dh), static_cast<cuuint64_t>(c.page),
                              static_cast<cuuint64_t>(c.pages) * c.Hkv};
  const cuuint64_t size = c.dtype == DT_E4M3 ? 1 : 2;
  const cuuint64_t strides[2] = {size * c.dh, size * c.dh * c.page};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row tiles of at most 128 rows, two a unit. False where the kernel does not apply. (The
// kernel for any size took 0.28 ms for 32 trees of 65 rows over 512 to 1024 rows where this
// one takes 0.10 ms, and 6.2 ms for 8 of 129 over up to 32768 8-bit rows: 0.58 ms.)
bool wide_plan(const dt_cache &c, int64_t rows, int sms, int smem, AttnPlan *p) {
  if (c.dh > 128) return false;
  const bool quant = c.dtype == DT_E4M3;
  const int64_t tiles = (rows + 127) / 128;
  p->bm = 2 * static_cast<int>((rows + tiles - 1) / tiles);
  p->row_tiles = static_cast<int>((tiles + 1) / 2);
  p->odd = static_cast<int>(tiles & 1);
  p->ring = p->raw = 0;
  const WideShape w = wide_shape(c, *p);
  const int tile = w.nblk * kBlk;
  const int room = smem - w.off_small - static_cast<int>(sizeof(Small));
  if (quant) {
    p->ring = 3;
    p->raw = (room - p->ring * tile) / w.raw_bytes;
    if (p->raw > kMaxRing) p->raw = kMaxRing;
    if (p->raw < 3) return false;
  } else {
    p->ring = room / tile < kMaxRing ? room / tile : kMaxRing;
    if (p->ring < 3) return false;
  }
  p->dhp = 64 * w.nblk;
  p->grid = sms;
  p->smem = wide_shape(c, *p).off_small + sizeof(Small);
  p->kind = AttnPlan::kWide;
  return true;
}

cudaError_t launch_wide(const dt_cache &c, const AttnArgs &a, int dtype, const AttnPlan &p,
                        cudaStream_t st) {
  const WideShape w = wide_shape(c, p);
  CUtensorMap k = {}, v = {};
  const bool quant = c.dtype == DT_E4M3;
  if (!quant && (!page_map(c, c.k, c.page, &k) || !page_map(c, c.v, c.page, &v))) return cudaErrorInvalidValue;
  if (dtype == DT_BF16) return quant ? go<DT_BF16, true>(a, w, p, k, v, st) : go<DT_BF16, false>(a, w, p, k, v, st);
  return quant ? go<DT_F16, true>(a, w, p, k, v, st) : go<DT_F16, false>(a, w, p, k, v, st);
}

}  // namespace dt
