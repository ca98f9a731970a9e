// dt_project.cu -- a projection that many requests share, with low-rank adapters of their
// own beside it, on the tcgen05 tensor cores: y = x W^T + scale_a (x A_a^T) B_a^T for the rows of
// a request with adapter a.
//
// The MMA's M side is 128 rows of W (256 in a pair of blocks), its N side a tile of up to 256 token
// rows, so that one form serves single tokens and long prompts. K goes by in slabs of 128
// bytes a row (64 16-bit values or 128 codes) through a ring that TMA fills. The adapters are more of
// K: for the distinct adapters of a tile's rows one after the other, B_a beside W and, beside x, the
// rows u = scale x A_a^T with zeros in the rows of other requests, so the shared and the own
// products meet in one accumulator and B_a is read once a tile, however its requests lie. (8-bit
// rows: in an accumulator of their own, as the shared one is scaled at the end.) u comes from a
// launch before, which stacks the A_a of a tile's adapters on the M side; the projection begins
// beside it and waits for it only where it reads u. u is a sum in 32 bits, and the tensor cores take 16: it goes
// as two terms, the rounded value and what the rounding left, two products with the same B_a. Results are then as
// far from sums in fp32 in another order as without adapters (trees 1.5e-4 of y's norm, most of it y's own
// rounding falling to the other side), with one term eight times as far (1.2e-3). The second term costs 2 to 3
// us: with one the trees below take 69 us for 71, the 8-bit tokens 22 for 25.
//
// Measured on the GPU, inputs in rotation (K 4096): 32 trees of 65 rows to 6144 outputs, eight adapters
// of rank 16, bf16, 71 to 72 us, 1.46 PFLOP/s (62 to 63 us without adapters; the tensor pipe 72 % active with
// cold caches); two prompts of 4099 rows to 4001, rank 64, fp16, 190 to 196 us, 1.4 PFLOP/s; 8224 rows of
// 8-bit codes to 6144 120 us, 3.45 PFLOP/s; one token of 8 requests to 6144 16 us, of which W's
// 50 MB from memory are 8; of 128 requests with 64 adapters of rank 32, 8-bit, to 4096 25.4 us. These are
// bursts of a few ms at 2070 MHz. Calls of 2 s in a row come to the power limit (1250 to 1290 W): trees 79 us
// at 1770 MHz, prompts 208 at 1650, 8-bit rows 139 at 1477; the small cases keep the clock and their times.
// Large cases are bound by the tensor cores, at the clock that power leaves them, and by tiles that
// do not fill a last round. A pair's slab (128 bytes of K), with one tile a pair and from the
// times of K = 2048, 4096 and 8192: 256 rows 282 to 295 ns with 8-bit codes and 275 to 305 with
// 16 bits, where 2.25 and 4.5 PFLOP/s would be 283; 128 rows 183 to 186 and 181 to 210, where
// they would be 142, so that short tiles pay for more than their products. Two pairs that share
// their rows of x by multicast were built: 8-bit rows 117 us for 119, the trees 76 for 67. Small
// cases are bound by what stands before the first product (launch, barriers,
// first copy: 3 us) and behind the last (a cluster's sum: 3 us).
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "dt_cache_attn.cuh"
#include "dt_internal.h"
#include "dt_umma.cuh"

namespace dt {

namespace {

constexpr int kOuts = 128;             // rows of W of a block's tile: lanes of TMEM
constexpr int kSlabA = kOuts * 128;    // bytes of a slab of them
constexpr int kMaxTokens = 256;        // rows of x of a tile
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;           // blocks that share a tile's K: a cluster
constexpr int kGroups = 2;             // warpgroups that empty an accumulator, 16 columns in turn
constexpr int kDrain = 128 * kGroups;  // their threads; behind them the warps of TMA and products

struct ProjectArgs {
  const uint8_t *w_exps, *x_exps;
  const float *scale;
  const int32_t *index;
  char *y;
  uint16_t *u;           // [terms][rows][rank]: scale x A^T, rounded, and what the rounding left, rounded
  int32_t *status;
  int64_t ldy;           // in bytes
  uint32_t limit;        // SM cycles after which a wait is given up
  int rows, n, O, K, count, rank, terms;
};

struct ProjectShape {
  int nt, stages;                 // rows of x of a tile; places of the ring
  int tiles_o, tiles, split;      // tiles along the outputs, all; blocks that share a tile
  int outs, piece;                // rows of W of a block's tile; values of B_a's rows of one copy
  int off_small;
};

// The distinct adapters of a tile's requests, in the order in which they first occur.
struct AdapterList {
  int count, first;               // first: the request of the tile's first row
  int ids[kMaxTokens];
  int16_t slot[kMaxTokens];       // place in ids of each request's, -1: it has none
};

struct ListScratch {
  int4 ad[kMaxTokens / 4];
  int counts[8];
};

struct Small {                    // behind the ring
  uint64_t full[kMaxStages], empty[kMaxStages], u_go[kMaxStages], up_full[kMaxStages], u_full[kMaxStages];
  uint64_t acc_full[2], acc_empty[2], list_full[2], list_empty[2], idle;
  AdapterList list[2];
  uint32_t odd[2][kOuts][kMaxTokens / 32];   // of each row of W's tile: adapters whose B row is not all finite
  int any_odd[2];
  ListScratch scratch;
  int16_t token_slot[kMaxTokens];
  alignas(16) int xexp[4 * kGroups][kMaxTokens];   // exponents of the tile's rows of x, as bits of fp32; one copy a warp
  uint32_t tmem;
  int fail, peer_fail;            // a wait ran out in this block; in the other one of its pair
  // how far the copies have come, for what follows on a wait that ran out: the ring's turns; stages whose
  // last turn is one of W and x; stages with a copy of B_a that up_full counts, and its phases
  uint32_t turns, mains, flying, ups;
  uint32_t peer_turns, peer_mains;
};

// ------------------------------------------------------------ clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// the address of block `rank`'s copy of a shared variable
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_peer(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void arrive_peer(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ------------------------------------------------- one block, or a pair (CG = 2)

template <int CG>
__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t *dst) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, 512);
  }
}
template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t taddr) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
  else
    tmem_dealloc(taddr, 512);
}

// D[tmem] (+)= A[smem] * B[smem]^T; E8: e4m3 operands, 32 values of K, else 16
template <int CG, bool E8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
#define DT_MMA(group, kind)                                                                      \
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"                                       \
               "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n}\n" ::"r"(d), \
               "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))                       \
               : "memory")
  if (CG == 2) {
    if (E8) DT_MMA("2", "f8f6f4");
    else DT_MMA("2", "f16");
  } else {
    if (E8) DT_MMA("1", "f8f6f4");
    else DT_MMA("1", "f16");
  }
#undef DT_MMA
}

// one arrival on the barrier (in a pair: on both blocks') once all products so far are done
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}

// counts bytes as arrived on a barrier
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// instruction descriptor: fp32 accumulation, both operands K-major
template <int DT, bool E8>
__device__ __forceinline__ uint32_t descriptor(int M, int N) {
  const uint32_t f = !E8 && DT == DT_BF16 ? 1u : 0u;     // e4m3 and fp16: 0
  return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// operands in rows of 128 bytes, or fewer, swizzled by as much
__device__ __forceinline__ uint64_t rows128(uint32_t addr) { return umma_desc(addr, 16, 1024) | (2ull << 61); }
// rows of `values` 16-bit values: 64, 32 or 16
__device__ __forceinline__ uint64_t rows_of(uint32_t addr, int values) {
  return umma_desc(addr, 16, 16 * values) | ((values == 64 ? 2ull : values == 32 ? 4ull : 6ull) << 61);
}

// 16 fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void load16(uint32_t taddr, float (&v)[16]) {
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

// Waits of a converged warp. The lanes agree by votes, so that the compiler knows a warp's loops to be
// uniform and keeps addresses and descriptors where TMA and MMA instructions take them from (with
// one lane in a loop of its own a slab took 310 ns, whatever its size).
template <bool SLEEP>
__device__ __forceinline__ bool passed(uint64_t *bar, uint32_t parity) {
  uint32_t done;
#define DT_PASSED(op)                                                                    \
  asm volatile("{\n.reg .pred p;\nmbarrier." op ".parity.shared::cta.b64 p, [%1], %2;\n" \
               "selp.u32 %0, 1, 0, p;\n}\n"                                              \
               : "=r"(done)                                                              \
               : "r"(smem_u32(bar)), "r"(parity)                                         \
               : "memory")
  if (SLEEP) DT_PASSED("try_wait");
  else DT_PASSED("test_wait");
#undef DT_PASSED
  return __all_sync(kFull, done);
}
// Bounded. False when the wait ran out, here or (where this one is not over) in another warp. With a limit of a
// test's the warp does not sleep, which may take longer than that. (Norm and 8-bit trees 67.7 us a call
// for 66.2 without that branch, one token and 16-bit trees the same.)
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *fail, int32_t *status,
                                          uint32_t limit) {
  if (passed<false>(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
  const bool sleep = limit >= static_cast<uint32_t>(kWaitCycles);
  for (;;) {
    if (sleep ? passed<true>(bar, parity) : passed<false>(bar, parity)) return true;
    if (__any_sync(kFull, *fail != 0)) return false;
    if (__any_sync(kFull, static_cast<uint32_t>(clock()) - t0 > limit)) {
      *fail = 1;
      *status = DT_ERR_TIMEOUT;
      return false;
    }
  }
}

// a place in a ring of `size` stages, and the parity of its barriers' phase
struct Place {
  uint32_t at, parity;
  __device__ void step(uint32_t size) {
    if (++at == size) {
      at = 0;
      parity ^= 1u;
    }
  }
};

// The list for the rows [t0, t1), by 128 threads that meet at barrier `bar`. A request's adapter is
// compared with those of the tile's requests before it (256 at most), four at a time.
__device__ void list_adapters(const ProjectArgs &a, int t0, int t1, AdapterList &list, ListScratch &z, int tid,
                              int bar) {
  const int b0 = t0 / a.n, nb = (t1 - 1) / a.n - b0 + 1, lane = tid & 31, warp = tid >> 5;
  int *ad = reinterpret_cast<int *>(z.ad);
  auto meet = [&]() { asm volatile("barrier.cta.sync %0, 128;" ::"r"(bar) : "memory"); };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + 128 * k;
    int at = -1;
    if (i < nb) {
      at = a.index[b0 + i];
      if (at >= a.count) {
        *a.status = DT_ERR_BAD_INDEX;
        at = -1;
      }
    }
    ad[i] = at < 0 ? -1 : at;
  }
  meet();
  int same[2];
  unsigned votes[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + 128 * k, at = ad[i];
    int j = i;                                  // the first request with this adapter
    if (at >= 0)
#pragma unroll 4
      for (int q = i / 4; q >= 0; --q) {
        const int4 v = z.ad[q];
        if (v.w == at && 4 * q + 3 <= i) j = 4 * q + 3;
        if (v.z == at && 4 * q + 2 <= i) j = 4 * q + 2;
        if (v.y == at && 4 * q + 1 <= i) j = 4 * q + 1;
        if (v.x == at && 4 * q <= i) j = 4 * q;
      }
    same[k] = at < 0 ? -1 : j;
    votes[k] = __ballot_sync(kFull, same[k] == i);
    if (lane == 0) z.counts[4 * k + warp] = __popc(votes[k]);
  }
  meet();
  int slot[2] = {-1, -1};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + 128 * k;
    if (same[k] == i) {
      slot[k] = __popc(votes[k] & ((1u << lane) - 1u));
      for (int w = 0; w < 4 * k + warp; ++w) slot[k] += z.counts[w];
      list.ids[slot[k]] = ad[i];
      list.slot[i] = static_cast<int16_t>(slot[k]);
    } else if (same[k] < 0) {
      list.slot[i] = -1;
    }
  }
  if (tid == 0) {
    int all = 0;
    for (int w = 0; w < 8; ++w) all += z.counts[w];
    list.count = all;
    list.first = b0;
  }
  meet();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + 128 * k;
    if (same[k] >= 0 && same[k] != i) list.slot[i] = list.slot[same[k]];
  }
  meet();
}

// Slabs of a stage. Two halve what its waits and issuing take, for tiles whose products take less (a
// single block's: 8 tokens 17.4 to 15.9 us); a pair's tiles of 256 rows have a shallower ring
// then (two prompts, u in one term, 178 to 187 us).
__host__ __device__ constexpr int deep_of(int cg) { return cg == 1 ? 2 : 1; }
// Sixteens of B_a's ranks in a stage, whose place of x takes each row's values of u in `terms` terms.
__host__ __device__ constexpr int fill_of(int cg, int terms) { return cg == 2 && terms == 2 ? 2 : 4; }

// Sums over the blocks of a cluster that share a tile's K. Each block owns a share of the tile's columns:
// the others write their terms into its shared memory (where the ring was: all blocks have passed a
// cluster barrier), [block][column of the share][128 lanes]; behind a second barrier it adds them up
// in the blocks' order. (Writes to another block do not wait for each other, as reads would.)
struct Shares {
  uint32_t base;         // of the memory, in this block
  int width, split, rank, lane;
  __device__ Shares(const void *memory, int columns, int split_, int rank_, int lane_)
      : base(smem_u32(memory)), width(share_width(columns, split_)), split(split_), rank(rank_), lane(lane_) {}
  // columns of a share: whole sixteens, so that those that are read together have one owner
  __host__ __device__ static int share_width(int columns, int split) {
    return ((columns + 16 * split - 1) / (16 * split)) * 16;
  }
  // the i-th sixteen columns that this block sends: the blocks begin with different owners
  __device__ __forceinline__ int turn(int i, int columns) const {
    return split > 1 ? (16 * i + rank * width) % columns : 16 * i;
  }
  // the terms of columns c .. c + 15
  __device__ __forceinline__ void push(int c, const float (&v)[16]) {
    const int owner = c / width;
    const uint32_t to = peer_address(base, owner) + ((rank * width + c - owner * width) * 128 + lane) * 4;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 512 * e), "f"(v[e]) : "memory");
  }
  // put(column, its eight sums), by one of `groups` warpgroups
  template <typename Put>
  __device__ __forceinline__ void sum(const unsigned char *memory, int columns, int group, int groups, Put put) {
    const int c0 = rank * width, end = min(c0 + width, columns);
    for (int c = c0 + 8 * group; c < end; c += 8 * groups) {
      const float *own = reinterpret_cast<const float *>(memory) + (c - c0) * 128 + lane;
      float v[8] = {};
      for (int q = 0; q < split; ++q, own += width * 128)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += own[e * 128];
      put(c, v);
    }
  }
};

// 16 bytes, or zeros, without a branch
__device__ __forceinline__ uint4 load_if(const void *p, bool there) {
  uint4 v;
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %5, 0;\nmov.u32 %0, 0;\nmov.u32 %1, 0;\nmov.u32 %2, 0;\nmov.u32 %3, 0;\n"
      "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<int>(there))
      : "memory");
  return v;
}

// whether one of two pairs' halves has all exponent bits set (of magnitudes; `m` of top_abs)
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t m) {
  constexpr uint32_t kExp = DT == DT_BF16 ? 0x7f807f80u : 0x7c007c00u, kOne = DT == DT_BF16 ? 0x00800080u : 0x04000400u;
  return (((m & kExp) + kOne) & 0x80008000u) != 0u;       // a full exponent carries into the sign's place
}
// such values set to zero
template <int DT>
__device__ __noinline__ void make_finite(uint4 *p) {
  constexpr uint32_t kExp = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
  uint32_t *w = reinterpret_cast<uint32_t *>(p);
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & kExp) == kExp) w[i] &= 0xffff0000u;
    if (((w[i] >> 16) & kExp) == kExp) w[i] &= 0xffffu;
  }
}

template <int DT>
__device__ __forceinline__ uint16_t round16(float v) {
  return static_cast<uint16_t>(Half16<DT>::pack(v, 0.0f));
}

// scale x A^T of a row and a rank: one 16-bit term, or two
template <int DT>
__device__ __forceinline__ void store_u(const ProjectArgs &a, uint16_t *to, float v) {
  const uint16_t first = round16<DT>(v);
  *to = first;
  if (a.terms == 2) {
    const float at = Half16<DT>::unpack(first).x;
    to[static_cast<int64_t>(a.rows) * a.rank] = round16<DT>(isfinite(at) ? v - at : 0.0f);
  }
}

// v 2^e for any e in [-254, 256], without overflow or underflow on the way
__device__ __noinline__ float times_power(float v, int e) {
  const int h = e >> 1;
  return v * __uint_as_float(static_cast<uint32_t>(h + 127) << 23) *
         __uint_as_float(static_cast<uint32_t>(e - h + 127) << 23);
}

// u = scale x A^T: 128 stacked rows of A_a (the slots [m spt, m spt + spt) of a token tile's list)
// times nt rows of x, K shared by the blocks of a cluster. Warps 0-7: the list (0-3),
// and the accumulator's rows to u; 8: TMA; 9: products.
template <int DT>
__global__ void __launch_bounds__(kDrain + 64, 1)
adapter_down_kernel(const __grid_constant__ ProjectArgs a, const __grid_constant__ ProjectShape w,
                    const __grid_constant__ CUtensorMap dmap, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Small &ss = *reinterpret_cast<Small *>(sm + w.off_small);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = w.split, rank = static_cast<int>(blockIdx.x) % split, tile = blockIdx.x / split;
  const int spt = kOuts / a.rank, m = tile % w.tiles_o;
  const int t0 = tile / w.tiles_o * w.nt, t1 = min(t0 + w.nt, a.rows);
  AdapterList &list = ss.list[0];
  const int steps = (2 * a.K + 127) / 128, k0 = steps * rank / split, k1 = steps * (rank + 1) / split;
  const int stage = kSlabA + w.nt * 128;
  volatile int *fail = &ss.fail;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, fail, a.status, a.limit); };
  const bool issuer = elect_one();
  // the rows of x need no list: the ring's first round of them is on its way before there is one
  auto load_x = [&](int s, uint32_t at) {
    mbar_expect_tx(&ss.full[at], w.nt * 128);
    tma_2d<1>(sm + at * stage + kSlabA, &xmap, s * 64, t0, smem_u32(&ss.full[at]));
  };
  const int ahead = min(w.stages, k1 - k0);
  if (warp == kDrain / 32 && lane == 0) {
    for (int i = 0; i < w.stages; ++i) {
      mbar_init(&ss.full[i], 2);
      mbar_init(&ss.empty[i], 1);
    }
    mbar_init(&ss.acc_full[0], 1);
    ss.fail = 0;
    fence_async_smem();
    for (int i = 0; i < ahead; ++i) load_x(k0 + i, i);
  }
  if (warp == kDrain / 32 + 1) tmem_alloc(&ss.tmem, 256);
  if (warp < 4) {
    list_adapters(a, t0, t1, list, ss.scratch, tid, 1);
    for (int t = t0 + tid; t < t0 + w.nt; t += 128)
      ss.token_slot[t - t0] = t < t1 ? list.slot[t / a.n - list.first] : static_cast<int16_t>(-1);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // The projection may begin now and not before: one of its blocks on this SM takes all columns of TMEM
  // and keeps them until every block of this launch has ended, so each of these has to own its columns first.
  cudaTriggerProgrammaticLaunchCompletion();
  const uint32_t tmem = ss.tmem;
  const int slots = min(list.count - m * spt, spt);
  if (slots <= 0) {                             // all blocks of the cluster alike
    if (warp == kDrain / 32 && lane == 0)
      for (int i = 0; i < ahead; ++i) {         // (an arrival without bytes ends the phase with the copies)
        mbar_arrive(&ss.full[i]);
        mbar_wait_cycles(&ss.full[i], 0);
      }
    if (warp == kDrain / 32 + 1) tmem_dealloc(tmem, 256);
    return;
  }
  Place p = {0, 0};
  if (warp == kDrain / 32) {
    int s = k0;
    for (; s < k1 && wait(&ss.empty[p.at], p.parity ^ 1u); ++s) {
      if (issuer) {
        if (s >= k0 + ahead) load_x(s, p.at);
        mbar_expect_tx(&ss.full[p.at], slots * a.rank * 128);
        for (int i = 0; i < slots; ++i)
          tma_2d<1>(sm + p.at * stage + i * a.rank * 128, &dmap, s * 64, list.ids[m * spt + i] * a.rank,
                    smem_u32(&ss.full[p.at]));
      }
      p.step(w.stages);
    }
    if (lane == 0) ss.turns = s - k0;
  } else if (warp == kDrain / 32 + 1) {
    const uint32_t idesc = descriptor<DT, false>(kOuts, w.nt);
    for (int s = k0; s < k1 && wait(&ss.full[p.at], p.parity); ++s) {
      tmem_fence_after();
      const uint32_t at = smem_u32(sm) + p.at * stage;
      const uint64_t da = rows128(at), db = rows128(at + kSlabA);
      const int parts = min(4, (a.K - s * 64 + 15) / 16);
      if (issuer) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < parts) mma<1, false>(tmem, da + 2 * i, db + 2 * i, idesc, s > k0 || i > 0);
        commit<1>(&ss.empty[p.at]);
      }
      p.step(w.stages);
    }
    if (issuer) commit<1>(&ss.acc_full[0]);
  }
  if (tid < kDrain) {
    __syncwarp();
    const int row = tid & 127, group = tid >> 7;
    const int slot = row / a.rank, j = row - slot * a.rank;
    const bool live = slot < slots;
    const int want = live ? m * spt + slot : -2;
    const float scale = live && a.scale ? a.scale[list.ids[want]] : 1.0f;
    const bool go = wait(&ss.acc_full[0], 0);
    tmem_fence_after();
    auto put = [&](int c, const auto &v) {
      uint16_t *to = a.u + static_cast<int64_t>(t0 + c) * a.rank + j;
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(v) / sizeof(float)); ++e)
        if (ss.token_slot[c + e] == want) store_u<DT>(a, to + e * a.rank, v[e] * scale);
    };
    if (split > 1) cluster_sync();
    Shares shares(sm, w.nt, split, rank, row);
#pragma unroll 1
    for (int i = group; i < w.nt / 16 && go; i += kGroups) {
      const int c = shares.turn(i, w.nt);
      float v[16];
      load16(tmem + (static_cast<uint32_t>(warp & 3) << 21) + c, v);
      tmem_wait_ld();
      if (split == 1) put(c, v);
      else shares.push(c, v);
    }
    tmem_fence_before();
    if (split > 1) {
      cluster_sync();
      shares.sum(sm, w.nt, group, kGroups, put);
    }
  } else if (split > 1) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  __syncthreads();
  if (ss.fail) {       // a wait ran out: no copy may land, and no product read, where the block has ended
    if (warp == kDrain / 32 && lane == 0) {
      int i = static_cast<int>(ss.turns);
      for (; i < ahead; ++i) mbar_arrive(&ss.full[i]);      // (ends a phase that has its rows of x alone)
      for (int k = max(i - w.stages, 0); k < i; ++k) mbar_wait_cycles(&ss.full[k % w.stages], (k / w.stages) & 1);
    }
    if (warp == kDrain / 32 + 1 && lane == 0) mbar_wait_cycles(&ss.acc_full[0], 0);
    __syncthreads();
  }
  if (split > 1) cluster_sync();                // its sums have been read
  tmem_fence_after();
  if (warp == kDrain / 32 + 1) tmem_dealloc(tmem, 256);
}

// The same for few rows: a block takes a row and four ranks, its warps share K. No list, no cluster, and
// nothing that a projection's block would have to wait for; A_a is read once a row, from L2 for all but
// the first.
template <int DT>
__global__ void __launch_bounds__(256) adapter_rows_kernel(const __grid_constant__ ProjectArgs a, const char *x,
                                                           int64_t ldx, const char *down) {
  __shared__ float s_sum[8][4];
  const int fours = a.rank >> 2, row = blockIdx.x / fours, j0 = (blockIdx.x - row * fours) * 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cudaTriggerProgrammaticLaunchCompletion();
  const int at = a.index[row / a.n];
  if (at >= a.count && threadIdx.x == 0) *a.status = DT_ERR_BAD_INDEX;
  if (at < 0 || at >= a.count) return;
  const char *d = down + 2 * (static_cast<int64_t>(at) * a.rank + j0) * a.K;
  x += row * ldx;
  float v[4] = {};
#pragma unroll 2
  for (int k = threadIdx.x * 8; k < a.K; k += 256 * 8) {
    const uint4 p = *reinterpret_cast<const uint4 *>(x + 2 * k);
    const uint32_t xs[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 q = __ldg(reinterpret_cast<const uint4 *>(d + 2 * (static_cast<int64_t>(j) * a.K + k)));
      const uint32_t ds[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Half16<DT>::unpack(xs[e]), g = Half16<DT>::unpack(ds[e]);
        v[j] += f.x * g.x;
        v[j] += f.y * g.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = warp_sum(v[j]);
    if (lane == 0) s_sum[warp][j] = v[j];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) all += s_sum[w][threadIdx.x];
    store_u<DT>(a, a.u + static_cast<int64_t>(row) * a.rank + j0 + threadIdx.x, all * (a.scale ? a.scale[at] : 1.0f));
  }
}

// The projection. Warps 0-7: accumulators to y (a thread an output, two for each); 8: TMA; 9: products; 10-13
// (AD): the adapters' list, and their u rows into the ring. In a pair (CG = 2) each block holds its 128
// rows of W and half of the tile's rows of x, and the first one issues the products of both. Two
// accumulators: one is emptied while the next tile's products run; of 8-bit rows a third, for
// adapters.
template <int DT, bool E8, int AD, int CG>
__global__ void __launch_bounds__(AD ? kDrain + 192 : kDrain + 64, 1)
project_kernel(const __grid_constant__ ProjectArgs a, const __grid_constant__ ProjectShape w,
               const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
               const __grid_constant__ CUtensorMap umap) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Small &ss = *reinterpret_cast<Small *>(sm + w.off_small);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = CG == 2 ? 2 : w.split;                 // blocks of a cluster
  const int crank = size > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int split = CG == 2 ? 1 : w.split, rank = CG == 2 ? 0 : crank;
  const int pair = CG == 2 ? crank : 0;
  const int mine = w.nt / CG;                             // rows of x in this block's memory
  constexpr int deep = deep_of(CG);
  const int slab_x = deep * kSlabA, stage = deep * (kSlabA + mine * 128);   // x behind W in a stage
  const int first = blockIdx.x / size, step = gridDim.x / size;
  const int kbytes = E8 ? a.K : 2 * a.K, steps = (kbytes + 127) / 128;
  const int k0 = steps * rank / split, k1 = steps * (rank + 1) / split;
  constexpr int kValues = E8 ? 128 : 64;                  // of a slab's row

  if (tid == 0) {
    for (int i = 0; i < w.stages; ++i) {
      mbar_init(&ss.full[i], 1);
      mbar_init(&ss.empty[i], 1);
      mbar_init(&ss.u_go[i], 1);
      mbar_init(&ss.up_full[i], 1);
      mbar_init(&ss.u_full[i], 128 * CG);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ss.acc_full[i], 1);
      mbar_init(&ss.acc_empty[i], kDrain * CG);
      mbar_init(&ss.list_full[i], 128);
      mbar_init(&ss.list_empty[i], 2 + kDrain / 32);
      ss.any_odd[i] = 0;
    }
    mbar_init(&ss.idle, 1);
    ss.fail = ss.peer_fail = 0;
  }
  if (AD)
    for (int i = tid; i < 2 * kOuts * (kMaxTokens / 32); i += blockDim.x) (&ss.odd[0][0][0])[i] = 0u;
  if (warp == kDrain / 32 + 1) tmem_take<CG>(&ss.tmem);
  tmem_fence_before();
  __syncthreads();
  if (size > 1) cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = ss.tmem;
  volatile int *fail = &ss.fail;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, fail, a.status, a.limit); };
  const bool issuer = elect_one();
  // the barrier of the block that issues the products
  auto first_block = [&](uint64_t *bar) { return CG == 2 ? peer_address(smem_u32(bar), 0) : smem_u32(bar); };
  auto arrive_first = [&](uint64_t *bar) {
    if (CG == 2) arrive_peer(first_block(bar));
    else mbar_arrive(bar);
  };
  // The adapters' part of K in sixteens, `fill` a stage; this block's stages of them. The second terms of u lie behind
  // the first ones, in the place of a second slab of x (single blocks) or of its second half.
  constexpr int fill = fill_of(CG, AD);
  const int second = fill * mine * 32;
  auto sixteens_of = [&](const AdapterList &l) { return l.count * (a.rank >> 4); };
  auto share = [&](int all, int *q0, int *q1) {
    const int n = (all + fill - 1) / fill;
    *q0 = n * rank / split;
    *q1 = n * (rank + 1) / split;
  };

  if (warp == kDrain / 32) {
    Place p = {0, 0};
    uint32_t issued = 0, mains = 0, ups = 0, flying = 0;
    bool go = true;
    for (int t = first, i = 0; t < w.tiles && go; t += step, ++i) {
      const int o0 = (t % w.tiles_o * CG + pair) * w.outs, x0 = t / w.tiles_o * w.nt + pair * mine;
      for (int s = k0; s < k1 && go; s += deep) {
        if (!(go = wait(&ss.empty[p.at], p.parity ^ 1u))) break;
        unsigned char *to = sm + p.at * stage;
        const uint32_t bar = first_block(&ss.full[p.at]);
        const int here = min(deep, k1 - s);
        if (issuer) {
          if (pair == 0) mbar_expect_tx(&ss.full[p.at], CG * here * (w.outs + mine) * 128);
          tma_2d<CG>(to, &wmap, s * kValues, o0, bar);
          tma_2d<CG>(to + slab_x, &xmap, s * kValues, x0, bar);
          if (deep > 1 && here > 1) {
            tma_2d<CG>(to + kSlabA, &wmap, (s + 1) * kValues, o0, bar);
            tma_2d<CG>(to + slab_x + mine * 128, &xmap, (s + 1) * kValues, x0, bar);
          }
        }
        flying &= ~(1u << p.at);
        mains |= 1u << p.at;
        p.step(w.stages);
        ++issued;
      }
      if (!AD || !go) continue;
      if (!(go = wait(&ss.list_full[i & 1], (i >> 1) & 1))) break;
      const AdapterList &l = ss.list[i & 1];
      const int all = sixteens_of(l), per = a.rank >> 4, wide = w.piece >> 4;
      int q0, q1;
      share(all, &q0, &q1);
      int u = fill * q0 / per, j = fill * q0 - u * per;  // adapter, and the sixteen of its rank
      for (int q = q0; q < q1; ++q) {
        if (!(go = wait(&ss.empty[p.at], p.parity ^ 1u))) break;
        if (issuer) mbar_arrive(&ss.u_go[p.at]);
        unsigned char *to = sm + p.at * stage;
        const uint32_t bar = smem_u32(&ss.up_full[p.at]);
        const int here = min(fill, all - fill * q);
        if (issuer) {
          if (pair == 0) mbar_arrive(&ss.full[p.at]);     // (it counts the ring's turns)
          mbar_expect_tx(&ss.up_full[p.at], here * w.outs * 32);
        }
        for (int k = 0; k < here; k += wide) {
          if (issuer) tma_2d<CG>(to + k * kOuts * 32, &umap, 16 * j, l.ids[u] * a.O + o0, bar);
          if ((j += wide) == per) j = 0, ++u;
        }
        ups ^= 1u << p.at;
        flying |= 1u << p.at;
        mains &= ~(1u << p.at);
        p.step(w.stages);
        ++issued;
      }
      __syncwarp();
      if (issuer) mbar_arrive(&ss.list_empty[i & 1]);
    }
    if (lane == 0) {
      ss.turns = issued;
      ss.mains = mains;
      ss.flying = flying;
      ss.ups = ups;
    }
  } else if (warp == kDrain / 32 + 1) {
    const uint32_t idesc = descriptor<DT, E8>(kOuts * CG, w.nt), idesc16 = descriptor<DT, false>(kOuts * CG, w.nt);
    Place p = {0, 0};
    uint32_t phases = 0;                       // of u_full, a bit a stage
    bool go = true;
    for (int t = first, i = 0; t < w.tiles && go; t += step, ++i) {
      const int buf = i & 1, turn = i >> 1;
      const uint32_t acc = tmem + buf * w.nt;
      if (pair == 0) {
        if (!(go = wait(&ss.acc_empty[buf], (turn & 1) ^ 1))) break;
        tmem_fence_after();
        for (int s = k0; s < k1; s += deep) {
          if (!(go = wait(&ss.full[p.at], p.parity))) break;
          tmem_fence_after();
          const uint32_t at = smem_u32(sm) + p.at * stage;
          const uint64_t da = rows128(at), db = rows128(at + slab_x);
          const int parts = min(4, (kbytes - s * 128 + 31) / 32);
          const int more = deep > 1 && k1 - s > 1 ? min(4, (kbytes - s * 128 - 97) / 32) : 0;   // of the next slab
          if (issuer) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < parts) mma<CG, E8>(acc, da + 2 * k, db + 2 * k, idesc, s > k0 || k > 0);
            if (deep > 1)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < more)
                  mma<CG, E8>(acc, da + kSlabA / 16 + 2 * k, db + mine * 8 + 2 * k, idesc, true);
            commit<CG>(&ss.empty[p.at]);
          }
          p.step(w.stages);
        }
        if (!go) break;
      }
      if (AD) {
        if (!(go = wait(&ss.list_full[i & 1], (i >> 1) & 1))) break;
        const int all = sixteens_of(ss.list[i & 1]), wide = w.piece >> 4;
        int q0, q1;
        share(all, &q0, &q1);
        if (pair == 0) {
          // the adapters' own accumulator is the only one: the tile before has to have read it
          if (E8 && i > 0 && q0 < q1) {
            if (!(go = wait(&ss.acc_empty[(i - 1) & 1], ((i - 1) >> 1) & 1))) break;
            tmem_fence_after();
          }
          const uint32_t to = E8 ? tmem + 2 * w.nt : acc;
          for (int q = q0; q < q1; ++q) {
            if (!(go = wait(&ss.full[p.at], p.parity) && wait(&ss.u_full[p.at], (phases >> p.at) & 1u))) break;
            phases ^= 1u << p.at;
            tmem_fence_after();
            const uint32_t at = smem_u32(sm) + p.at * stage;
            const int here = min(fill, all - fill * q);
            const uint64_t da = rows_of(at, w.piece), db = rows_of(at + slab_x, w.piece);
            if (issuer) {
#pragma unroll
              for (int k = 0; k < fill; ++k) {
                const int first_of = k & ~(wide - 1), in = 2 * (k - first_of);     // of its piece; 32 bytes on
                const uint64_t dw = da + first_of * kOuts * 2 + in, du = db + first_of * mine * 2 + in;
                if (k < here) mma<CG, false>(to, dw, du, idesc16, !E8 || q > q0 || k > 0);
                if (AD == 2 && k < here) mma<CG, false>(to, dw, du + second / 16, idesc16, true);
              }
              commit<CG>(&ss.empty[p.at]);
            }
            p.step(w.stages);
          }
          if (!go) break;
        }
        __syncwarp();              // every lane has read the list's count
        if (issuer) mbar_arrive(&ss.list_empty[i & 1]);
      }
      if (pair == 0 && issuer) commit<CG>(&ss.acc_full[buf]);
    }
  } else if (AD && tid >= kDrain + 64) {
    const int id = tid - kDrain - 64;
    uint32_t at = 0, phases = 0;               // stage of the ring; phases of u_go
    bool marked[2] = {false, false};           // this thread's row of ss.odd has something
    // Where a thread's sixteens lie in a stage, as offsets of their first halves (the second ones 16 bytes
    // away, before or behind): of row `id` of the rows u (there are 128 at most), and of B_a's.
    const int row_bytes = 2 * w.piece, chunks = w.piece >> 3;      // of a piece's row
    const int shift = w.piece == 64 ? 0 : w.piece == 32 ? 1 : 2;   // rows of one swizzle
    int u_at[fill], b_at[fill];
#pragma unroll
    for (int z = 0; z < fill; ++z) {
      const int c = 2 * z & (chunks - 1), in = id * row_bytes + 16 * (c ^ ((id >> shift) & (chunks - 1)));
      u_at[z] = slab_x + (2 * z - c) * mine * 16 + in;
      b_at[z] = (2 * z - c) * kOuts * 16 + in;
    }
    // (these warps meet for the lists: they go through all tiles, whatever has failed)
    for (int t = first, i = 0; t < w.tiles; t += step, ++i) {
      AdapterList &l = ss.list[i & 1];
      const int tt = t / w.tiles_o * w.nt, x0 = tt + pair * mine;
      bool go = wait(&ss.list_empty[i & 1], ((i >> 1) & 1) ^ 1);
      if (marked[i & 1]) {
        for (int k = 0; k < kMaxTokens / 32; ++k) ss.odd[i & 1][id][k] = 0u;
        ss.any_odd[i & 1] = 0;
        marked[i & 1] = false;
      }
      list_adapters(a, tt, min(tt + w.nt, a.rows), l, ss.scratch, id, 1);
      mbar_arrive(&ss.list_full[i & 1]);
      if (i == 0) cudaGridDependencySynchronize();        // u is there
      const int all = sixteens_of(l), per = a.rank >> 4;
      int q0, q1;
      share(all, &q0, &q1);
      const int row = x0 + id, slot = id < mine && row < a.rows ? l.slot[row / a.n - l.first] : -1;
      const uint16_t *u[2];                    // the terms
      u[0] = a.u + static_cast<int64_t>(row) * a.rank;
      u[1] = u[0] + static_cast<int64_t>(a.rows) * a.rank;
      at = (at + (k1 - k0 + deep - 1) / deep) % w.stages;
      uint4 v[2][fill][2];
      int of = fill * q0 / per, j = fill * q0 - of * per, whose[fill];   // adapter and sixteen of its rank to be fetched
      auto fetch = [&](int q) {                // loads of the next stage's rows, before there is room
#pragma unroll
        for (int z = 0; z < fill; ++z) {
          whose[z] = fill * q + z < all ? of : -2;
#pragma unroll
          for (int k = 0; k < AD; ++k) {
            v[k][z][0] = load_if(u[k] + 16 * j, whose[z] == slot);
            v[k][z][1] = load_if(u[k] + 16 * j + 8, whose[z] == slot);
          }
          if (++j == per) j = 0, ++of;
        }
      };
      if (q0 < q1) fetch(q0);
      for (int q = q0; q < q1 && go; ++q) {
        const uint32_t parity = (phases >> at) & 1u;
        if (!(go = wait(&ss.u_go[at], parity))) break;
        phases ^= 1u << at;
        unsigned char *const place = sm + at * stage;
#pragma unroll
        for (int k = 0; k < AD; ++k) {
          if (id >= mine) break;
#pragma unroll
          for (int z = 0; z < fill; ++z) {
            const int to = u_at[z] + k * second;
            *reinterpret_cast<uint4 *>(place + to) = v[k][z][0];
            *reinterpret_cast<uint4 *>(place + (to ^ 16)) = v[k][z][1];
          }
        }
        int looked[fill];
#pragma unroll
        for (int z = 0; z < fill; ++z) looked[z] = whose[z];
        __syncwarp();
        if (q + 1 < q1) fetch(q + 1);          // (on its way while this stage's B_a is looked through)
        // B_a's rows stand beside zeros of other requests' rows: what is not finite there would reach them.
        // A thread looks through a row, takes such values out, and notes whose they are; the
        // output is NaN for the rows with that adapter.
        go = wait(&ss.up_full[at], parity);
        if (go && id < w.outs) {
          uint32_t most[4] = {};
#pragma unroll
          for (int z = 0; z < fill; ++z) {
            const uint4 lo = *reinterpret_cast<const uint4 *>(place + b_at[z]);
            const uint4 hi = *reinterpret_cast<const uint4 *>(place + (b_at[z] ^ 16));
            most[z] = top_abs<DT>(top_abs<DT>(top_abs<DT>(lo.x, lo.y), top_abs<DT>(lo.z, lo.w)),
                                  top_abs<DT>(top_abs<DT>(hi.x, hi.y), top_abs<DT>(hi.z, hi.w)));
          }
          if (not_finite<DT>(top_abs<DT>(top_abs<DT>(most[0], most[1]), top_abs<DT>(most[2], most[3])))) {
#pragma unroll
            for (int z = 0; z < fill; ++z)
              if (looked[z] >= 0 && not_finite<DT>(most[z])) {
                make_finite<DT>(reinterpret_cast<uint4 *>(place + b_at[z]));
                make_finite<DT>(reinterpret_cast<uint4 *>(place + (b_at[z] ^ 16)));
                ss.odd[i & 1][id][looked[z] >> 5] |= 1u << (looked[z] & 31);
                ss.any_odd[i & 1] = 1;
                marked[i & 1] = true;
              }
          }
        }
        __syncwarp();
        fence_async_smem();
        arrive_first(&ss.u_full[at]);
        __syncwarp();
        if (++at == static_cast<uint32_t>(w.stages)) at = 0;
      }
    }
  } else if (tid < kDrain) {
    const int row = tid & 127, group = tid >> 7;
    bool go = true;
    for (int t = first, i = 0; t < w.tiles && go; t += step, ++i) {
      const int buf = i & 1, turn = i >> 1;
      const int o = row < w.outs ? (t % w.tiles_o * CG + pair) * w.outs + row : a.O, t0 = t / w.tiles_o * w.nt;
      bool both = false;                       // the adapters have something in their accumulator
      __syncwarp();                            // (all lanes have read the last tile's exponents)
      if (AD && E8) {
        go = wait(&ss.list_full[i & 1], (i >> 1) & 1);
        int q0 = 0, q1 = 0;
        if (go) share(sixteens_of(ss.list[i & 1]), &q0, &q1);
        both = q0 < q1;
      }
      const int rows = min(w.nt, a.rows - t0);
      // 8-bit rows: 2^wexp of this output times 2^xexp of the rows of x, in one number where that
      // cannot leave fp32's range on the way
      const int wexp = E8 && o < a.O ? a.w_exps[o] - 127 : 0;
      bool far = false;
      if (E8) {
        far = abs(wexp) > 60;
        for (int c = lane; c < w.nt; c += 32) {
          const int e = c < rows ? a.x_exps[t0 + c] - 127 : 0;
          far |= abs(e) > 60;
          ss.xexp[warp][c] = e << 23;
        }
        far = __any_sync(kFull, far);          // (also orders the writes before the reads below)
      }
      const int wbits = (wexp + 127) << 23;
      __syncwarp();
      go = go && wait(&ss.acc_full[buf], turn & 1);
      tmem_fence_after();
      const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
      Shares shares(sm, w.nt, split, rank, row);
      if (split > 1) cluster_sync();
      char *y = a.y + static_cast<int64_t>(t0) * a.ldy + 2 * static_cast<int64_t>(o);
      const bool inside = o < a.O;
      const uint32_t ldy = static_cast<uint32_t>(a.ldy);
      auto put = [&](int c, const auto &v) {
        if (!inside) return;
        char *at = y + c * a.ldy;
        const int live = rows - c;
#pragma unroll
        for (int e = 0; e < static_cast<int>(sizeof(v) / sizeof(float)); e += 2) {
          const uint32_t two = Half16<DT>::pack(v[e], v[e + 1]);
          if (e < live) *reinterpret_cast<uint16_t *>(at + static_cast<uint64_t>(e * ldy)) = static_cast<uint16_t>(two);
          if (e + 1 < live)
            *reinterpret_cast<uint16_t *>(at + static_cast<uint64_t>((e + 1) * ldy)) = static_cast<uint16_t>(two >> 16);
        }
      };
      float v[16], z[16], next[16], next_z[16];
      auto fetch = [&](int c) {
        load16(lanes + buf * w.nt + c, next);
        if (AD && E8 && both) load16(lanes + 2 * w.nt + c, next_z);
      };
      // 16 columns are on their way from TMEM while the 16 before them are written. (One copy of this
      // code, as short as it comes: a warp issues an instruction every six cycles here, and its
      // instructions have to fit their cache.)
      const int sixteens = w.nt / 16;
      if (go && group < sixteens) fetch(shares.turn(group, w.nt));
#pragma unroll 1
      for (int part = group; part < sixteens && go; part += kGroups) {
        const int c = shares.turn(part, w.nt);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          v[e] = next[e];
          if (AD && E8) z[e] = next_z[e];
        }
        if (part + kGroups < sixteens) fetch(shares.turn(part + kGroups, w.nt));
        if (E8) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const int4 x = *reinterpret_cast<const int4 *>(&ss.xexp[warp][c + e]);
            const int bits[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (__builtin_expect(far, 0)) v[e + k] = times_power(v[e + k], wexp + (bits[k] >> 23));
              else v[e + k] *= __int_as_float(wbits + bits[k]);
              if (AD && both) v[e + k] += z[e + k];
            }
          }
        }
        if (AD && __builtin_expect(ss.any_odd[i & 1], 0)) {
          const AdapterList &l = ss.list[i & 1];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int of = c + e < rows ? l.slot[(t0 + c + e) / a.n - l.first] : -1;
            if (of >= 0 && ((ss.odd[i & 1][row][of >> 5] >> (of & 31)) & 1u)) v[e] = __int_as_float(0x7fffffff);
          }
        }
        if (split > 1) shares.push(c, v);
        else put(c, v);
      }
      tmem_fence_before();
      arrive_first(&ss.acc_empty[buf]);
      if (AD) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.list_empty[i & 1]);
      }
      if (split > 1) {
        cluster_sync();
        shares.sum(sm, w.nt, group, kGroups, put);
      }
    }
  }
  if (split > 1 && tid >= kDrain) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  __syncthreads();
  if (CG == 2 && ss.fail && tid == 0) store_peer(peer_address(smem_u32(&ss.peer_fail), pair ^ 1), 1u);
  if (size > 1) cluster_sync();          // no block ends while another may still read or signal it
  if (__builtin_expect(ss.fail | ss.peer_fail, 0)) {
    // A wait ran out (for a pair: in either block). No copy may land, and no product read or write, where a block
    // has ended.
    if (warp == kDrain / 32 + 1) {
      if (pair == 0 && issuer) commit<CG>(&ss.idle);
      if (lane == 0) mbar_wait_cycles(&ss.idle, 0);
    }
    if (warp == kDrain / 32 && lane == 0) {
      if (pair == 1) {
        store_peer(peer_address(smem_u32(&ss.peer_turns), 0), ss.turns);
        store_peer(peer_address(smem_u32(&ss.peer_mains), 0), ss.mains);
      }
      for (int k = 0; k < w.stages; ++k)
        if ((ss.flying >> k) & 1u) mbar_wait_cycles(&ss.up_full[k], ((ss.ups >> k) & 1u) ^ 1u);
    }
    if (CG == 2) cluster_sync();
    if (warp == kDrain / 32 && lane == 0 && pair == 0) {
      // full counts the copies of both blocks of a pair, which may have come differently far
      const uint32_t stages = w.stages, bytes = (w.outs + mine) * 128;
      const uint32_t own = ss.turns, peer = CG == 2 ? ss.peer_turns : own, all = max(own, peer);
      for (uint32_t k = all > stages ? all - stages : 0; k < all; ++k) {
        const uint32_t at = k % stages;
        if (k >= peer && ((ss.mains >> at) & 1u)) mbar_complete_tx(&ss.full[at], bytes);     // that never come
        if (k >= own) {
          if (!((ss.peer_mains >> at) & 1u)) continue;
          mbar_expect_tx(&ss.full[at], bytes);
        }
        mbar_wait_cycles(&ss.full[at], (k / stages) & 1u);
      }
    }
    __syncthreads();
    if (CG == 2) cluster_sync();
  }
  tmem_fence_after();
  if (warp == kDrain / 32 + 1) tmem_give<CG>(tmem);
}

// ------------------------------------------------------------ plans

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }
int stages_of(int smem, int stage) { return std::min(kMaxStages, (smem - static_cast<int>(sizeof(Small)) - 1024) / stage); }

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct ProjectPlan {
  int cg;
  ProjectShape s;
  int blocks, idle;      // blocks; how many of the GPU's places have a tile less to do than others
  double tile;           // cycles of a tile
  size_t smem;
};

// clusters of each size that run at once, one block an SM (an SM whose cluster is not complete
// stays idle); [1]: SMs
struct Rooms {
  int of[kMaxSplit + 1];
};

int rooms(int sms, Rooms *r) {
  static std::atomic<int> known[64][kMaxSplit + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DT_ERR_CUDA;
  constexpr auto kernel = adapter_down_kernel<DT_BF16>;
  r->of[0] = 0;
  r->of[1] = sms;
  for (int size = 2; size <= kMaxSplit; ++size) {
    int n = dev < 64 ? known[dev][size].load(std::memory_order_relaxed) : 0;
    if (!n) {
      if (allow_smem<kernel>() != cudaSuccess) return DT_ERR_CUDA;
      cudaLaunchAttribute cluster = {};
      cluster.id = cudaLaunchAttributeClusterDimension;
      cluster.val.clusterDim.x = size;
      cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
      cudaLaunchConfig_t config = {};
      config.gridDim = dim3(sms / size * size);
      config.blockDim = dim3(kDrain + 64);
      config.dynamicSmemBytes = 200 * 1024;
      config.attrs = &cluster;
      config.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &config) != cudaSuccess) return DT_ERR_CUDA;
      n = std::max(n, 0);
      if (dev < 64) known[dev][size].store(n ? n : -1, std::memory_order_relaxed);
    }
    r->of[size] = std::max(n, 0);
  }
  return DT_OK;
}

constexpr double kCopyRate = 55.0;     // bytes a cycle into an SM's shared memory
constexpr double kRowsRate = 4000.0;   // bytes a cycle that adapter_rows_kernel reads
constexpr double kMemoryRate = 3500.0; // bytes a cycle from memory

// Cycles that a slab takes in a block: its products, its bytes on the way in, and what waits and
// issuing take whatever its size.
double slab_cycles(int outs, int nt, int cg) {
  return std::max(std::max(2.0 * nt, 330.0), (outs + nt / cg) * 128 / kCopyRate);
}

// The tile, and the blocks that share one, of the least estimated time: whole rounds of tiles over the
// clusters that the GPU has room for, or memory's time, and what a tile's end takes. A pair of blocks
// (cg = 2) loads half of the rows of x each. Where one round does, tiles have as few rows of W as keep
// all SMs busy. Only the order of the estimates matters. Both sides measured: pairs of 256 rows against
// single blocks of 144 (with adapters 128), trees 72 and 93 us, 8-bit stress rows 120 and 151, prompts 190 and
// 236; one token of 8 requests by two blocks a tile and by one, 16.3 and 18.3 us; of 128 requests in tiles of
// 128 rows by four blocks, of 64 by two and of 32 by one, 25.2, 24.6 and 25.4 us. The adapters' stages are
// not in the estimates: how many distinct adapters a tile's requests have the host does not know. With a small
// K and many adapters of a high rank they are most of a tile's time, and the plan is that of their absence.
void choose(const ProjectArgs &a, bool e8, bool ad, const Rooms &room, int smem, ProjectPlan *p) {
  const int size = e8 ? 1 : 2, steps = ceil_div(static_cast<int64_t>(a.K) * size, 128);
  // of a pair; with adapters three accumulators instead of two. Of a single block: three stages; with adapters a thread
  // a row of u
  const int most[3] = {0, ad ? 128 : 144, ad && e8 ? 160 : kMaxTokens};
  const double memory = (static_cast<double>(a.O) + a.rows) * a.K * size / kMemoryRate;
  double best = 1e300;
  for (int cg = 1; cg <= 2; ++cg)
    for (int nt = 16 * cg; nt <= most[cg]; nt += 16 * cg) {
      const int tiles_t = ceil_div(a.rows, nt);
      for (int split = 1; split <= (cg == 2 ? 1 : std::min(kMaxSplit, steps)); ++split) {
        const int places = room.of[cg == 2 ? 2 : split];
        if (places < 1) continue;
        int outs = kOuts;
        if (cg == 1 && places >= tiles_t)
          outs = std::min(kOuts, (ceil_div(a.O, places / tiles_t) + 7) / 8 * 8);
        const int tiles_o = ceil_div(a.O, outs * cg);
        const int64_t tiles = static_cast<int64_t>(tiles_o) * tiles_t;
        if (split > 1 && tiles > places) continue;
        const int rounds = ceil_div(tiles, places);
        const double tile = ceil_div(steps, split) * slab_cycles(outs, nt, cg);
        const double cost = std::max(rounds * tile, memory) + 16.0 * nt + (split > 1 ? 3000.0 + 16.0 * nt : 0.0);
        if (cost < best) {
          best = cost;
          p->cg = cg;
          p->tile = tile;
          p->s.nt = nt;
          p->s.split = split;
          p->s.outs = outs;
          p->s.tiles_o = tiles_o;
          p->s.tiles = static_cast<int>(tiles);
          const int clusters = static_cast<int>(std::min<int64_t>(tiles, places)), members = cg == 2 ? 2 : split;
          p->blocks = clusters * members;
          p->idle = room.of[1] - p->blocks + static_cast<int>(static_cast<int64_t>(rounds) * clusters - tiles) * members;
        }
      }
      if (nt >= a.rows) break;
    }
  const int stage = deep_of(p->cg) * (kSlabA + p->s.nt / p->cg * 128);
  p->s.stages = stages_of(smem, stage);
  p->s.off_small = p->s.stages * stage;
  p->s.piece = a.rank % 64 == 0 ? 64 : a.rank % 32 == 0 ? 32 : 16;
  p->s.piece = std::min(p->s.piece, 16 * fill_of(p->cg, a.terms));
  p->smem = p->s.off_small + sizeof(Small);
}

// The launch before: a block a row and four ranks while all that they read (from L2) takes less time
// than the other kernel adds (s->tiles = 0: 128 tokens of rank 32 25.4 us instead of 30, but the trees
// 93 instead of 72); else blocks that fit the places which have a tile less to do cost nothing as long as
// they end within the others' first tile (the trees: 24 blocks of 152 places;
// 72 us, 66 where no request has an adapter, 63 without any); else the shortest.
void choose_down(const ProjectArgs &a, const ProjectPlan &p, const Rooms &room, int smem, ProjectShape *s) {
  const int steps = ceil_div(2 * a.K, 128), spt = kOuts / a.rank;
  double best = 1e300;
  for (int nt = 16; nt <= kMaxTokens; nt += 16) {
    const int requests = std::min(nt, (nt + a.n - 2) / a.n + 1);        // of a tile, at most
    const int tiles_o = ceil_div(std::min(requests, a.count), spt);
    const int64_t tiles = static_cast<int64_t>(tiles_o) * ceil_div(a.rows, nt);
    for (int split = 1; split <= std::min(kMaxSplit, steps); split *= 2) {
      if (room.of[split] < 1 || (split > 1 && tiles > room.of[split])) continue;
      const double rounds = ceil_div(tiles, room.of[split]);
      const double time = rounds * (ceil_div(steps, split) * slab_cycles(kOuts, nt, 1) + 10000.0 +
                                    (split > 1 ? 3000.0 + 16.0 * nt : 16.0 * nt));
      const double cost = (tiles * split <= p.idle ? std::max(0.0, time - p.tile) : time) + 1e-3 * time;
      if (cost < best) {
        best = cost;
        s->nt = nt;
        s->tiles_o = tiles_o;
        s->tiles = static_cast<int>(tiles);
        s->split = split;
      }
    }
    if (nt >= a.rows) break;
  }
  if (4000.0 + 2.0 * a.rows * a.rank * a.K / kRowsRate < best) {
    s->tiles = 0;
    return;
  }
  const int stage = kSlabA + s->nt * 128;
  s->stages = std::min(stages_of(smem, stage),
                       std::max(ceil_div(steps, s->split),
                                ceil_div(s->split * Shares::share_width(s->nt, s->split) * 512, stage)));
  s->off_small = s->stages * stage;
}

// Blocks of a cluster wait for one another, each with its columns of TMEM. Were two such launches (of two streams)
// to share SMs, a block of each could wait for columns that the other one's peer holds, without end. So a
// cluster's blocks ask for all shared memory (`most`) but these bytes, less than any block here has.
constexpr int kLeave = 32 * 1024;
static_assert(sizeof(Small) + kSlabA + 16 * 128 > kLeave);

template <auto Kernel, typename... Args>
cudaError_t launch_cluster(int blocks, int threads, size_t smem, int most, int cluster, bool early, cudaStream_t st,
                           const Args &...args) {
  if (cluster > 1) smem = std::max(smem, static_cast<size_t>(most - kLeave));
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(blocks);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = st;
  config.attrs = attr;
  config.numAttrs = early ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&config, Kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT>
cudaError_t launch_down(const ProjectArgs &a, const ProjectShape &s, const dt_adapters &ad, const void *x16,
                        int64_t ldx16, int smem, cudaStream_t st) {
  if (s.tiles == 0) {
    adapter_rows_kernel<DT><<<a.rows * (a.rank / 4), 256, 0, st>>>(a, static_cast<const char *>(x16), ldx16,
                                                                   static_cast<const char *>(ad.down));
    return cudaGetLastError();
  }
  const cudaError_t e = allow_smem<adapter_down_kernel<DT>>();
  if (e != cudaSuccess) return e;
  CUtensorMap down, x;
  if (!matrix_map(ad.down, 2, a.K, static_cast<int64_t>(a.count) * a.rank, 2 * a.K, 64, a.rank, &down) ||
      !matrix_map(x16, 2, a.K, a.rows, ldx16, 64, s.nt, &x))
    return cudaErrorUnknown;
  return launch_cluster<adapter_down_kernel<DT>>(s.tiles * s.split, kDrain + 64, s.off_small + sizeof(Small), smem, s.split,
                                                 false, st, a, s, down, x);
}

template <int DT, bool E8, int AD, int CG>
cudaError_t launch_main(const ProjectArgs &a, const ProjectPlan &p, const CUtensorMap &w, const CUtensorMap &x,
                        const CUtensorMap &up, int smem, cudaStream_t st) {
  constexpr auto kernel = project_kernel<DT, E8, AD, CG>;
  const cudaError_t e = allow_smem<kernel>();
  if (e != cudaSuccess) return e;
  return launch_cluster<kernel>(p.blocks, AD ? kDrain + 192 : kDrain + 64, p.smem, smem, CG == 2 ? 2 : p.s.split, AD, st,
                                a, p.s, w, x, up);
}

template <int DT, bool E8, int AD>
cudaError_t launch_project(const ProjectArgs &a, const dt_matrix &m, const void *x, int64_t ldx,
                           const dt_adapters *ad, const void *x16, int64_t ldx16, const Rooms &room, int smem,
                           cudaStream_t st) {
  ProjectPlan p = {};
  choose(a, E8, AD, room, smem, &p);
  CUtensorMap w, xm, up = {};
  const int size = E8 ? 1 : 2;
  if (!matrix_map(m.data, size, a.K, a.O, m.ld * size, 128 / size, p.s.outs, &w) ||
      !matrix_map(x, size, a.K, a.rows, ldx, 128 / size, p.s.nt / p.cg, &xm))
    return cudaErrorUnknown;
  if (AD) {
    if (!matrix_map(ad->up, 2, a.rank, static_cast<int64_t>(a.count) * a.O, 2 * a.rank, p.s.piece, p.s.outs, &up))
      return cudaErrorUnknown;
    ProjectShape down = {};
    choose_down(a, p, room, smem, &down);
    const cudaError_t e = launch_down<DT>(a, down, *ad, x16, ldx16, smem, st);
    if (e != cudaSuccess) return e;
  }
  return p.cg == 2 ? launch_main<DT, E8, AD, 2>(a, p, w, xm, up, smem, st)
                   : launch_main<DT, E8, AD, 1>(a, p, w, xm, up, smem, st);
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
      w->K < 16 || w->K > 65536 || w->K % 16 || w->O < 1 || w->O > (1 << 24) ||
      w->wait_cycles < 0 || static_cast<int64_t>(batch) * n * w->O > (int64_t{1} << 38))
    return DT_ERR_INVALID_ARG;
  const bool e8 = w->dtype == DT_E4M3;
  const int64_t size = e8 ? 1 : 2, rows = static_cast<int64_t>(batch) * n, most = int64_t{1} << 32;
  if (w->ld < w->K || w->ld * size % 16 || w->ld > most || ldx < w->K || ldx * size % 16 || ldx > most ||
      ldy < w->O || ldy > (1 << 26) || e8 != (w->exps != nullptr) || e8 != (x_exps != nullptr))
    return DT_ERR_INVALID_ARG;
  if (!adapters != !index || (!adapters || !e8) != !x16) return DT_ERR_INVALID_ARG;
  dt::ProjectArgs a = {};
  a.y = static_cast<char *>(y);
  a.w_exps = w->exps;
  a.x_exps = x_exps;
  a.status = status;
  a.ldy = 2 * ldy;
  a.limit = w->wait_cycles ? w->wait_cycles : static_cast<uint32_t>(dt::kWaitCycles);
  a.rows = static_cast<int>(rows);
  a.n = n;
  a.O = w->O;
  a.K = w->K;
  if (adapters) {
    if (!adapters->down || !adapters->up || !dt::al16(adapters->down) || !dt::al16(adapters->up) ||
        (reinterpret_cast<uintptr_t>(adapters->scale) & 3u) || adapters->count < 1 ||
        adapters->count > (1 << 20) || adapters->terms < 0 || adapters->terms > 2 ||
        adapters->rank < 16 || adapters->rank > 128 || adapters->rank % 16 ||
        (reinterpret_cast<uintptr_t>(index) & 3u) || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < std::max(adapters->terms, 1) * dt_project_workspace_bytes(batch, n, adapters->rank) ||
        static_cast<int64_t>(adapters->count) * w->O > 0x7fffff00 ||
        static_cast<int64_t>(adapters->count) * adapters->rank > 0x7fffff00)
      return DT_ERR_INVALID_ARG;
    if (e8 && (!dt::al16(x16) || ldx16 < w->K || ldx16 % 8 || ldx16 > most)) return DT_ERR_INVALID_ARG;
    if (!e8) {
      x16 = x;
      ldx16 = ldx;
    }
    a.scale = adapters->scale;
    a.index = index;
    a.count = adapters->count;
    a.rank = adapters->rank;
    a.terms = std::max(adapters->terms, 1);
    a.u = static_cast<uint16_t *>(workspace);
  }
  int sms, smem;
  const int rc = dt::device_sm_count(&sms, &smem);
  if (rc) return rc;
  dt::Rooms room;
  if (dt::rooms(sms, &room)) return DT_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto type, auto eight, auto with) {
    return dt::launch_project<decltype(type)::value, decltype(eight)::value, decltype(with)::value>(
        a, *w, x, ldx * size, adapters, x16, 2 * ldx16, room, smem, st);
  };
  auto typed = [&](auto type) {
    auto with = [&](auto terms) { return e8 ? go(type, std::true_type{}, terms) : go(type, std::false_type{}, terms); };
    return a.terms == 2   ? with(std::integral_constant<int, 2>{})
           : a.terms == 1 ? with(std::integral_constant<int, 1>{})
                          : with(std::integral_constant<int, 0>{});
  };
  const cudaError_t e = dtype == DT_BF16 ? typed(std::integral_constant<int, DT_BF16>{})
                                         : typed(std::integral_constant<int, DT_F16>{});
  return e == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // extern "C"
