// The products of wide experts and of 8-bit integers on the 5th-generation
// tensor cores.
//
// Every product is D[j, i] = sum_k B[j, k] A[i, k] over the tiles of a group:
//   forward, 8-bit: j a product row, i an output channel, k an input channel;
//   dx:             j a product row, i an input channel, k an output channel;
//   dW:             j an output channel, i an input channel, k a product row.
// i, the axis that is contiguous in the result, takes the MMA's M (128 per
// CTA: a TMEM lane each, so a warp's stores are contiguous); j takes its N,
// which is as wide as the group's rows need in steps of 16 per CTA.  A group
// that ends inside a tile then costs no idle products, and a decode batch's
// few rows per expert are an MMA of N = 16 or 32 over the streamed weights.
//
// Operands come by TMA in 128-byte-swizzled tiles of 128 bytes of k (K-major)
// or of 64 x 64 (the transposed operands of dx and dW, MN-major); rows of x
// taken by token come by cp.async from four warps (a TMA row gather costs
// about 77 cycles per four rows of 128 bytes, five times the products of the
// tile they feed).  Rows past a group's end that a load brings along only
// reach columns that are not stored; dW, whose sum runs over the rows, zeroes
// the last block's in shared memory before its products.
// CTAS = 2 pairs two CTAs on one 256-wide tile: each holds its half of A and
// of B, and the pair's first CTA issues the MMAs.
// Warps 0-7 drain the accumulators, warp 8 issues the TMA loads, warp 9 the
// MMAs, warps 12-15 gather (10 and 11 fill their warpgroup); two TMEM accumulators alternate, so a tile is
// stored while the next is summed.
//
// PIECES: the tensor core's fp32 sums cut every addition towards zero, an
// error of about 1.1e-9 of the result per term of k.  bf16 results do not
// show it; fp32 results are summed in pieces of 512 terms, which the draining
// warps add up in registers, rounded to nearest.
#include "linear.cuh"
#include "tc_common.cuh"

namespace omni {
namespace {

using namespace tc;

constexpr int kBM = 128;            // i per CTA
constexpr int kABytes = kBM * 128;  // a k-block's A tile: 128 bytes of k per row
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;
constexpr int kLoadWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kRowWarp = kEpiWarps + 4;
constexpr int kRowWarps = 4, kRowThreads = 32 * kRowWarps;
constexpr int kThreads = 32 * (kEpiWarps + 4 + kRowWarps);
// Registers: 512 threads start with 128 each; the two draining warpgroups
// (128 sums a thread) go to 184, the other two to 72: 2 * 184 + 2 * 72 = 4 * 128.
constexpr int kLaunchRegs = 128, kEpiRegs = 184, kOtherRegs = 72;
static_assert(2 * kEpiRegs + 2 * kOtherRegs == 4 * kLaunchRegs && kThreads == 512, "");
// dW's tiles leave through shared memory: per half of the draining warps two
// buffers of 16 columns of 128 fp32
constexpr int kOutCols = 16, kOutBytes = kOutCols * kBM * 4;
constexpr int kPiece = 512;         // terms of k in a piece
constexpr size_t kSmemLimit = 227 * 1024;

// ---- instructions --------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// the address of the first CTA's copy of a shared-memory location of this one
__device__ __forceinline__ uint32_t leader_addr(uint32_t a) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}

// bar: an mbarrier of this CTA, or with CTAS == 2 of either
template <int CTAS>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0,
                                        int c1) {
  if constexpr (CTAS == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(c0),
        "r"(c1)
        : "memory");
}
template <int CTAS>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0,
                                        int c1, int c2) {
  if constexpr (CTAS == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(c0), "r"(c1),
        "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(c0),
        "r"(c1), "r"(c2)
        : "memory");
}
// 16 bytes from global to shared memory; zeros without `valid`
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
// arrive on bar (one of its expected arrivals) when this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// arrive on an mbarrier of either CTA of a pair
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// barrier of one half (four warps) of the draining warps
__device__ __forceinline__ void half_sync(int half) {
  if (half == 0) asm volatile("bar.sync 2, 128;" ::: "memory");
  else asm volatile("bar.sync 3, 128;" ::: "memory");
}

// shared memory -> a box of dW: written, or added
__device__ __forceinline__ void store_3d(const CUtensorMap* m, uint32_t src, int c0, int c1,
                                         int c2, bool add) {
  if (add)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
        " [%0, {%2, %3, %4}], [%1];" ::"l"(m), "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group"
        " [%0, {%2, %3, %4}], [%1];" ::"l"(m), "r"(src), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

template <int CTAS, bool I8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (CTAS == 1 && !I8)
    umma_bf16(d, a, b, idesc, accumulate);
  else if constexpr (!I8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// arrive on bar (of both CTAs of a pair) once the MMAs issued so far are done
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CTAS == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  if constexpr (CTAS == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}

// SiLU for a bf16 result: the fast exponential and reciprocal are off by at
// most 2^-17 of the result (the rounding of z / ln 2, |z| < 89), where the
// rounding to bf16 that follows is off by up to 2^-8.
__device__ __forceinline__ float silu_fast(float z) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-z)));
  return z * r;
}

__device__ __forceinline__ void zero16(uint32_t dst) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}

// mbar_wait for barriers that the other CTA of a pair arrives on too
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
template <int CTAS>
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, int32_t* status) {
  if (CTAS == 1) return mbar_wait(bar, parity, status);
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t polls = 1; !try_wait_cluster(bar, parity); ++polls) {
    if (polls >= kWaitMaxPolls || global_ns() - t0 > kWaitLimitNs) {
      raise_status(status, OMNI_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
// the same by a whole warp: the outcome is the same in every lane
template <int CTAS>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, wait_one<CTAS>(bar, parity, status));
}

// One lane of a converged warp.  tcgen05 and TMA instructions take their
// operands from uniform registers: behind elect.sync the compiler knows that
// one lane is left and issues them straight, behind `lane == 0` it wraps
// each in a loop over the lanes (610 cycles per stage for four MMAs).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Shared-memory descriptors without their start address.  Of a K-major tile
// with 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 bytes apart.
constexpr uint64_t kDescK = (1ull << 16) | (1024ull >> 4 << 32) | (1ull << 46) | (2ull << 61);
// Of an MN-major tile with 128-byte swizzle: 64 of the operand's M or N (128
// bytes) per k, 8-k groups 1024 bytes apart, chunks of 64 along M or N one
// [64 k x 128 bytes] box, 8192 bytes, apart.
constexpr uint64_t kDescMn =
    (8192ull >> 4 << 16) | (1024ull >> 4 << 32) | (1ull << 46) | (2ull << 61);

// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- the kernel ------------------------------------------------------------------

struct Maps {
  CUtensorMap a, b;  // boxes of the two operands (a: W, or x for dW)
  CUtensorMap out;   // dW
};

template <Product P, int CTAS, int BN, bool PIECES>
struct Cfg {
  static constexpr bool kI8 = P == Product::kInt8;
  static constexpr bool kGradW = P == Product::kGradW, kGradX = P == Product::kGradX;
  static constexpr bool kMnA = kGradW || kGradX, kMnB = kGradW;
  static constexpr int kBlockK = kI8 ? 128 : 64;  // k of 128 bytes
  // k-blocks per stage: two where a block's products are short, which halves
  // what a stage costs its waits and commits (about 250 cycles)
  static constexpr int kSub = CTAS == 1 && BN <= 64 ? 2 : 1;
  static constexpr int kStageK = kBlockK * kSub;
  static constexpr int kMmaK = kI8 ? 32 : 16;
  static constexpr int kNb = BN / CTAS;           // j per CTA
  static constexpr int kBox = kGradW ? 64 : kNb < 32 ? kNb : 32;  // j of one B load
  static constexpr int kBBytes = kNb * 128;  // of a k-block
  static constexpr int kStageA = kSub * kABytes, kStageB = kSub * kBBytes;
  static constexpr int kStage = kStageA + kStageB;
  static constexpr int kOut = kGradW ? 4 * kOutBytes : 0;  // dW's way out
  static constexpr int kCols = 2 * BN;            // TMEM columns
  static_assert(!kGradW || kNb % 64 == 0, "dW's B tile is made of 64-wide boxes");
};

// One tile: columns j0 .. j0 + n - 1 of a group, i from i0.
struct Tile {
  int i0, j0, n, row0, id, K;
};

template <class C, int CTAS, int BN>
struct TileWalk {
  const LinearArgs& a;
  const GroupTab* tab;
  int groups, mt, c = 0;
  __device__ __forceinline__ Tile at(int t) {
    while (c + 1 < groups && tab[c + 1].begin <= t) ++c;
    const GroupTab g = tab[c];
    const int local = t - g.begin;
    Tile r;
    r.i0 = (local % mt) * (kBM * CTAS);
    r.j0 = (local / mt) * BN;
    const int J = C::kGradW ? a.out : g.rows;
    r.n = J - r.j0 < BN ? J - r.j0 : BN;
    r.row0 = g.row0;
    r.id = g.id;
    r.K = C::kGradW ? g.rows : C::kGradX ? a.out : a.in;
    return r;
  }
};

template <Product P, int CTAS, int BN, bool PIECES>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ Maps maps, const __grid_constant__ LinearArgs a,
                int stages) {
  using C = Cfg<P, CTAS, BN, PIECES>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kMaxStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ GroupScratch scratch;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sA = smem_u32(smem), sB = sA + stages * C::kStageA;
  GroupTab* tab = reinterpret_cast<GroupTab*>(smem + stages * C::kStage + C::kOut);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages;
  const uint32_t tfull0 = empty0 + 8 * kMaxStages, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = CTAS == 2 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

  const bool gathers = !C::kGradX && a.rows != nullptr;
  // Where a half needs more than its TMA loads (gathered rows, rows to zero),
  // each CTA of a pair waits for its own and the second tells the first;
  // else the loads of both report to the first.
  const bool halves = C::kGradW || gathers;
  if (threadIdx.x == 32 * kLoadWarp) {
    prefetch_map(&maps.a);
    prefetch_map(&maps.b);
    // a stage is full after its loads' expect, its gathered rows, and in a
    // pair's first CTA the second's word that its half is ready
    const int arrivals =
        1 + (gathers ? kRowThreads : 0) + (halves && CTAS == 2 && rank == 0 ? 1 : 0);
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, arrivals);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kEpiWarps * CTAS);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  const int I = C::kMnA ? a.in : a.out;
  const int mt = (I + kBM * CTAS - 1) / (kBM * CTAS);
  // dW behind dx: dx lets it start once dx's own wait is over (a.follows), so
  // everything dW reads is there; it waits for dx at its end, before the
  // kernels behind it may start
  if (!a.follows) pdl_wait();
  if (a.leads) pdl_trigger();
  if (warp < kGroupWarps) {
    build_groups(
        a.g,
        [&](int rows) {
          if (C::kGradW) return rows > 0 || !a.accumulate ? mt * ((a.out + BN - 1) / BN) : 0;
          return mt * ((rows + BN - 1) / BN);
        },
        tab, &scratch, blockIdx.x == 0 ? a.status : nullptr);
  } else if (warp == kMmaWarp) {
    tmem_alloc<CTAS>(smem_u32(&tmem_slot), C::kCols);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  if (CTAS == 2) cluster_sync();
  else __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const int tiles = scratch.total_tiles;
  const uint32_t tmem = tmem_slot;
  TileWalk<C, CTAS, BN> walk{a, tab, scratch.total_groups, mt};
  auto n_mma = [](const Tile& t) { return (t.n + 16 * CTAS - 1) / (16 * CTAS) * (16 * CTAS); };

  if (warp < kEpiWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ---- results: TMEM lane = i, column = j; a warp takes 32 lanes and every
    // other chunk of 32 columns
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t sOut = sB + stages * C::kStageB;
    uint32_t acc_no = 0, out_buf = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile tl = walk.at(t);
      const int i = tl.i0 + rank * kBM + 32 * quarter + lane;
      const int pieces = PIECES ? (tl.K + kPiece - 1) / kPiece : 1;
      float ws = 0.0f;
      if (C::kI8 && i < I) ws = a.Ws[static_cast<int64_t>(tl.id) * a.out + i];

      auto wait_full = [&]() -> bool {
        const bool got =
            __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * (acc_no & 1), (acc_no >> 1) & 1, a.status));
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        return got;
      };
      auto drained = [&]() {  // this warp has read its part of the accumulator
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = tempty0 + 8 * (acc_no & 1);
          if (CTAS == 2) arrive_cluster(leader_addr(bar));
          else mbar_arrive(bar);
        }
        ++acc_no;
      };
      // dW: 16 columns from c to shared memory, and from there by TMA, while the
      // next 16 go to the other buffer
      auto leave = [&](int c, const float* v) {
        const bool issues = quarter == 0 && lane == 0;
        const uint32_t buf = sOut + (2 * half + out_buf) * kOutBytes;
        if (issues) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        half_sync(half);
#pragma unroll
        for (int q = 0; q < kOutCols; ++q)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(buf + (q * kBM + 32 * quarter + lane) * 4),
                       "f"(v[q])
                       : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        half_sync(half);
        if (issues)
          store_3d(&maps.out, buf, tl.i0 + rank * kBM, tl.j0 + c, tl.id, a.accumulate != 0);
        out_buf ^= 1;
      };
      // columns c .. c + 31 of this lane's i
      auto store = [&](int c, const float* v) {
        const int n = tl.n - c;  // columns that exist
        {
          const int64_t at = static_cast<int64_t>(tl.row0 + tl.j0 + c) * I;
          float z[32];
          float xs = 0.0f;
          if (C::kI8 && lane < n) {
            const int r = tl.row0 + tl.j0 + c + lane;
            int xr = r;
            if (a.rows != nullptr) {
              xr = a.rows[r];
              if (xr < 0 || xr >= a.T) xr = 0;
            }
            xs = a.xs[xr];
          }
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            z[q] = v[q];
            if constexpr (C::kI8)
              z[q] = static_cast<float>(__float_as_int(v[q])) *
                     __shfl_sync(0xffffffffu, xs, q) * ws;
          }
          if (a.silu) {
            if (a.out_f32) {
#pragma unroll
              for (int q = 0; q < 32; ++q) z[q] = silu(z[q]);
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q) z[q] = silu_fast(z[q]);
            }
          }
          if (a.out_f32) {
            float* o = static_cast<float*>(a.o) + at + i;
            if (i < I) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q < n) o[static_cast<int64_t>(q) * I] = z[q];
            }
          } else {
            // two lanes trade so that each stores two neighbours of one column
            const bool odd = lane & 1;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + at + (i & ~1);
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, odd ? z[q] : z[q + 1], 1);
              const __nv_bfloat162 w =
                  odd ? __floats2bfloat162_rn(got, z[q + 1]) : __floats2bfloat162_rn(z[q], got);
              if (i < I && q + (odd ? 1 : 0) < n)
                *reinterpret_cast<__nv_bfloat162*>(o + static_cast<int64_t>(q + (odd ? 1 : 0)) * I) = w;
            }
          }
        }
      };

      if constexpr (PIECES) {
        constexpr int kAcc = BN > 32 ? BN / 2 : 32;  // columns of this warp
        float sum[kAcc];
#pragma unroll
        for (int q = 0; q < kAcc; ++q) sum[q] = 0.0f;
        for (int p = 0; p < pieces && ok; ++p) {
          ok = wait_full();
          if (!ok) break;
#pragma unroll
          for (int u = 0; u < kAcc / 32; ++u) {
            const int c = (2 * u + half) * 32;
            if (c < tl.n) {
#pragma unroll
              for (int w = 0; w < 32; w += 16) {
                uint32_t v[16];
                tmem_ld16(tmem + lanes + (acc_no & 1) * BN + c + w, v);
#pragma unroll
                for (int q = 0; q < 16; ++q) sum[u * 32 + w + q] += __uint_as_float(v[q]);
              }
            }
          }
          drained();
        }
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < kAcc / 32; ++u) {
          const int c = (2 * u + half) * 32;
          if constexpr (C::kGradW) {
#pragma unroll
            for (int w = 0; w < 32; w += kOutCols)
              if (c + w < tl.n && tl.i0 + rank * kBM < I) leave(c + w, sum + u * 32 + w);
          } else {
            if (c < tl.n) store(c, sum + u * 32);
          }
        }
      } else {
        ok = wait_full();
        if (!ok) break;
        for (int c = half * 32; c < tl.n; c += 64) {
          uint32_t v[32];
          tmem_ld32(tmem + lanes + (acc_no & 1) * BN + c, v);
          store(c, reinterpret_cast<const float*>(v));
        }
        drained();
      }
    }
    if (C::kGradW)  // this thread's stores are done
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ---- TMA loads
      if (elect_one()) {
        int s = 0;
        uint32_t ph = 0, issued = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = walk.at(t);
          const int nb = n_mma(tl) / CTAS;  // j of this CTA: j0 + rank * nb ..
          const int i0 = tl.i0 + rank * kBM, j0 = tl.j0 + rank * nb;
          const int boxes = (nb + C::kBox - 1) / C::kBox;
          const uint32_t bytes = (C::kGradW && gathers ? 0 : kABytes) +
                                 (!C::kGradW && gathers ? 0 : boxes * C::kBox * 128);
          for (int k0 = 0; k0 < tl.K; k0 += C::kStageK) {
            const uint32_t own = full0 + 8 * s;
            const uint32_t bar = CTAS == 2 && !halves ? leader_addr(own) : own;
            if (!mbar_wait(empty0 + 8 * s, ph ^ 1, a.status)) {
              ok = false;
              break;
            }
            const int subs = C::kSub == 1 || tl.K - k0 <= C::kBlockK ? 1 : 2;
            if (halves)
              mbar_expect_tx(own, subs * bytes);
            else if (rank == 0)
              mbar_expect_tx(own, CTAS * subs * bytes);
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) {
              if (u >= subs) break;
              const uint32_t da = sA + s * C::kStageA + u * kABytes;
              const uint32_t db = sB + s * C::kStageB + u * C::kBBytes;
              const int k = k0 + u * C::kBlockK;
              if constexpr (C::kGradW) {
                if (!gathers)
                  for (int h = 0; h < 2; ++h)
                    load_2d<1>(da + h * 8192, &maps.a, bar, i0 + 64 * h, tl.row0 + k);
                for (int h = 0; h < boxes; ++h)
                  load_2d<1>(db + h * 8192, &maps.b, bar, j0 + 64 * h, tl.row0 + k);
              } else {
                if constexpr (C::kGradX) {
                  for (int h = 0; h < 2; ++h)
                    load_3d<CTAS>(da + h * 8192, &maps.a, bar, i0 + 64 * h, k, tl.id);
                } else {
                  load_3d<CTAS>(da, &maps.a, bar, k, i0, tl.id);
                }
                if (!gathers)
                  for (int q = 0; q < boxes; ++q)
                    load_2d<CTAS>(db + q * C::kBox * 128, &maps.b, bar, k,
                                  tl.row0 + j0 + q * C::kBox);
              }
            }
            ++issued;
            if (++s == stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        if (!ok) {
          // a wait timed out: the loads in flight land (each wait bounded again)
          // before the CTA exits
          if (rank == 0 || halves)
            for (uint32_t k = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
                 k < issued; ++k)
              mbar_wait(full0 + 8 * (k % stages), (k / stages) & 1, a.status);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---- products: issued by one lane of the pair's first CTA.  dW keeps the
      // whole warp in step, to zero rows.
      constexpr bool kWarp = C::kGradW;
      if ((rank == 0 || halves) && (kWarp || elect_one())) {
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
          if (kWarp) return wait_warp<CTAS>(bar, parity, a.status);
          return wait_one<CTAS>(bar, parity, a.status);
        };
        int s = 0;
        uint32_t ph = 0, acc_no = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = walk.at(t);
          const uint32_t idesc =
              (C::kI8 ? (2u << 4) : (1u << 4)) | (1u << 7) | (1u << 10) |
              (C::kMnA ? 1u << 15 : 0u) | (C::kMnB ? 1u << 16 : 0u) |
              (static_cast<uint32_t>(n_mma(tl) >> 3) << 17) |
              (static_cast<uint32_t>(kBM * CTAS >> 4) << 24);
          uint32_t acc = 0;
          for (int k0 = 0; k0 < tl.K; k0 += C::kStageK) {
            const int left = tl.K - k0;
            const bool starts = k0 % (PIECES ? kPiece : 1 << 30) == 0;
            const bool ends =
                left <= C::kStageK || (PIECES && (k0 + C::kStageK) % kPiece == 0);
            if (starts && rank == 0) {
              const uint32_t b = acc_no & 1;
              ok = wait(tempty0 + 8 * b, ((acc_no >> 1) & 1) ^ 1);
              if (!ok) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              acc = tmem + b * BN;
            }
            const uint32_t da = sA + s * C::kStageA, db = sB + s * C::kStageB;
            ok = wait(full0 + 8 * s, ph);
            if (!ok) break;
            if constexpr (C::kGradW) {
              // rows past the group's end, up to the last product's 16: zeros (of
              // both operands: what is there may be infinite)
              if (left < C::kBlockK && (left & 15) != 0) {
                const int rows = 16 - (left & 15), nb = n_mma(tl) / CTAS;
                for (int g = lane; g < rows * 8; g += 32) {
                  const uint32_t at = (left + (g >> 3)) * 128 + (g & 7) * 16;
                  if (!gathers)
                    for (int h = 0; h < 2; ++h) zero16(da + h * 8192 + at);
                  for (int h = 0; h < (nb + 63) / 64; ++h) zero16(db + h * 8192 + at);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              }
            }
            // rows copied by threads, before the tensor core reads them
            if (gathers) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (kWarp) __syncwarp();
            if (rank != 0) {  // this half is ready
              if (!kWarp || lane == 0) arrive_cluster(leader_addr(full0 + 8 * s));
            } else if (!kWarp || elect_one()) {
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              const int steps = left >= C::kStageK ? C::kStageK / C::kMmaK
                                                   : (left + C::kMmaK - 1) / C::kMmaK;
              const uint64_t ad = (C::kMnA ? kDescMn : kDescK) | (da >> 4);
              const uint64_t bd = (C::kMnB ? kDescMn : kDescK) | (db >> 4);
              // a step of k: 32 bytes along K-major rows, 16 rows of an MN-major tile
              constexpr int kPer = C::kBlockK / C::kMmaK;  // steps of a k-block
              constexpr int sa = (C::kMnA ? 2048 : 32) >> 4, sb = (C::kMnB ? 2048 : 32) >> 4;
              mma<CTAS, C::kI8>(acc, ad, bd, idesc, starts ? 0u : 1u);
#pragma unroll
              for (int kk = 1; kk < C::kStageK / C::kMmaK; ++kk)
                if (kk < steps)
                  mma<CTAS, C::kI8>(acc, ad + kk / kPer * (kABytes >> 4) + kk % kPer * sa,
                                    bd + kk / kPer * (C::kBBytes >> 4) + kk % kPer * sb, idesc, 1u);
              commit<CTAS>(empty0 + 8 * s);
              if (ends) commit<CTAS>(tfull0 + 8 * (acc_no & 1));
            }
            if (kWarp) __syncwarp();
            if (ends) ++acc_no;
            if (++s == stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        if (!ok) {
          // the MMAs in flight end (bounded) before TMEM is freed
          if (rank == 0 && (!kWarp || elect_one())) {
            commit<CTAS>(drain);
            mbar_wait(drain, 0, a.status);
          }
        }
      }
    } else if (warp >= kRowWarp) {
      // ---- x's rows by token: 16 bytes a copy, eight copies to a row's 128 bytes
      if (gathers) {
        constexpr int kRows = C::kGradW ? 64 : C::kNb;         // of a stage
        constexpr int kMine = (kRows + kRowThreads / 8 - 1) / (kRowThreads / 8);
        const int tid = threadIdx.x - 32 * kRowWarp;
        const int r0 = tid >> 3, piece = tid & 7;
        const uint32_t place = static_cast<uint32_t>((piece ^ (r0 & 7)) * 16);  // swizzled
        const int64_t pitch = static_cast<int64_t>(a.in) * (C::kI8 ? 1 : 2);
        const char* x = static_cast<const char*>(a.x);
        auto checked = [&](int v) -> int {  // a row number as the caller gave it
          if (v >= 0 && v < a.T) return v;
          raise_status(a.status, OMNI_DEV_BAD_INDEX);
          return 0;
        };
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = walk.at(t);
          const int nb = n_mma(tl) / CTAS;
          const int i0 = tl.i0 + rank * kBM;
          const int mine = tl.n - rank * nb;  // dW: unused; else rows of this CTA
          const int row0 = C::kGradW ? tl.row0 : tl.row0 + tl.j0 + rank * nb;
          // dW takes other rows every block: each lane reads two of the block's
          // 64 row numbers, three blocks ahead
          int2 ahead[3];
          auto fetch = [&](int kb) -> int2 {
            const int r = kb * 64 + lane;
            return make_int2(r < tl.K ? a.rows[row0 + r] : -1,
                             r + 32 < tl.K ? a.rows[row0 + r + 32] : -1);
          };
          const char* src[kMine];
          if constexpr (C::kGradW) {
#pragma unroll
            for (int q = 0; q < 3; ++q) ahead[q] = fetch(q);
          } else {
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
              const int r = r0 + q * (kRowThreads / 8);
              // (past the group's end any row will do: its column is not stored)
              const int row = r < mine && r < kRows ? checked(a.rows[row0 + r]) : 0;
              src[q] = x + row * pitch + 16 * piece;
            }
          }
          for (int k0 = 0; k0 < tl.K; k0 += C::kStageK) {
            ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * s, ph ^ 1, a.status));
            if (!ok) break;
            if constexpr (C::kGradW) {
              const int left = tl.K - k0;
              const int2 v = make_int2(lane < left ? checked(ahead[0].x) : -1,
                                       lane + 32 < left ? checked(ahead[0].y) : -1);
              ahead[0] = ahead[1];
              ahead[1] = ahead[2];
              ahead[2] = fetch(k0 / 64 + 3);
              const uint32_t da = sA + s * C::kStageA + r0 * 128 + place;
              const int c = i0 + 8 * piece;
              const char* xc = x + static_cast<int64_t>(c) * 2;
              const bool whole = left >= 64 && i0 + kBM <= a.in;
              auto row_of = [&](int q) -> int {
                return __shfl_sync(0xffffffffu, q < kMine / 2 ? v.x : v.y,
                                   (r0 + q * (kRowThreads / 8)) & 31);
              };
              if (whole) {
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
                  const char* p = xc + row_of(q) * pitch;
                  copy16(da + q * (kRowThreads / 8) * 128, p);
                  copy16(da + q * (kRowThreads / 8) * 128 + 8192, p + 128);
                }
              } else {
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
                  const int row = row_of(q);
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const bool in = row >= 0 && c + 64 * h < a.in;
                    copy16_or_zero(da + q * (kRowThreads / 8) * 128 + h * 8192,
                                   in ? xc + row * pitch + 128 * h : x, in);
                  }
                }
              }
            } else {
              const uint32_t db = sB + s * C::kStageB + r0 * 128 + place;
#pragma unroll
              for (int u = 0; u < C::kSub; ++u) {
                const int k = k0 + u * C::kBlockK;
                if (k >= tl.K) break;
                const int64_t c = static_cast<int64_t>(k) * (C::kI8 ? 1 : 2);  // bytes
                const bool whole = k + C::kBlockK <= tl.K, in = c + 16 * piece < pitch;
                const uint32_t to = db + u * C::kBBytes;
                if (whole) {
#pragma unroll
                  for (int q = 0; q < kMine; ++q)
                    if (q * (kRowThreads / 8) < nb) copy16(to + q * (kRowThreads / 8) * 128, src[q] + c);
                } else {
#pragma unroll
                  for (int q = 0; q < kMine; ++q)
                    if (q * (kRowThreads / 8) < nb)
                      copy16_or_zero(to + q * (kRowThreads / 8) * 128, in ? src[q] + c : x, in);
                }
              }
            }
            copies_arrive(full0 + 8 * s);
            if (++s == stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  // a pair's CTAs read each other's shared memory and barriers to the end
  if (CTAS == 2) cluster_sync();
  else __syncthreads();
  if (a.follows) pdl_wait();
  if (!a.leads) pdl_trigger();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<CTAS>(tmem, C::kCols);
  }
}

// ---- host --------------------------------------------------------------------------

// A tensor map of a packed array: dims innermost first.
bool make_map_nd(CUtensorMap* m, const void* base, CUtensorMapDataType type, int esize, int nd,
                 const int64_t* dim, const int* box,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3], es[3] = {1, 1, 1};
  int64_t bytes = esize;
  for (int q = 0; q < nd; ++q) {
    d[q] = static_cast<cuuint64_t>(dim[q]);
    bx[q] = static_cast<cuuint32_t>(box[q]);
    bytes *= dim[q];
    if (q + 1 < nd) st[q] = static_cast<cuuint64_t>(bytes);
  }
  return fn(m, type, nd, const_cast<void*>(base), d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Product P, int CTAS, int BN, bool PIECES>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
  using C = Cfg<P, CTAS, BN, PIECES>;
  Maps m{};
  const int64_t W[3] = {a.in, a.out, a.g.E}, X[2] = {a.in, a.T}, Y[2] = {a.out, a.g.M};
  const int kb = C::kBlockK, esize = C::kI8 ? 1 : 2;
  const CUtensorMapDataType type =
      C::kI8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int box_w[3] = {kb, C::kMnA ? 64 : kBM, 1}, box_r[2] = {kb, C::kBox};
  const int box_64[2] = {64, 64};
  bool ok = true;
  if (a.g.M > 0) {
    if (C::kGradW) {
      ok = make_map_nd(&m.a, a.x, type, esize, 2, X, box_64) &&
           make_map_nd(&m.b, a.dy, type, esize, 2, Y, box_64);
    } else {
      ok = make_map_nd(&m.a, a.W, type, esize, 3, W, box_w) &&
           make_map_nd(&m.b, C::kGradX ? a.dy : a.x, type, esize, 2, C::kGradX ? Y : X, box_r);
    }
  }
  if (C::kGradW) {
    const int box_o[3] = {kBM, kOutCols, 1};
    ok = ok && make_map_nd(&m.out, a.o, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, 3, W, box_o,
                           CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  if (!ok) return cudaErrorInvalidValue;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const size_t fixed = 1024 + C::kOut + sizeof(GroupTab) * static_cast<size_t>(a.g.G);
  const size_t statics = sizeof(GroupScratch) + (2 * kMaxStages + 5) * 8 + 64;
  int stages = static_cast<int>((kSmemLimit - statics - fixed) / C::kStage);
  if (stages > kMaxStages) stages = kMaxStages;
  const size_t smem = fixed + static_cast<size_t>(stages) * C::kStage;
  auto kernel = k_linear_tc<P, CTAS, BN, PIECES>;
  OMNI_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem)));
  // no more pairs (or CTAs) than there can be tiles
  const int64_t mt = ((C::kMnA ? a.in : a.out) + kBM * CTAS - 1) / (kBM * CTAS);
  const int64_t live = a.g.G < a.g.M ? a.g.G : a.g.M;
  int64_t most = C::kGradW ? mt * ((a.out + BN - 1) / BN) * a.g.G : mt * (a.g.M / BN + live);
  if (most > sms / CTAS) most = sms / CTAS;
  if (most < 1) most = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most * CTAS));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS == 2 ? 2 : 1;
  OMNI_TRY(cudaLaunchKernelEx(&cfg, kernel, m, a, stages));
  return cudaGetLastError();
}

template <Product P, bool PIECES>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  const int64_t live = a.g.G < a.g.M ? a.g.G : a.g.M;
  const int64_t each = (a.g.M + live - 1) / live;  // rows of a group, on average
  const int rule = each <= 32 ? 32 : each <= 64 ? 64 : each <= 128 ? 128 : 256;
  int v = rule;
  if (v == 32) return launch<P, 1, 32, PIECES>(a, s);
  if (v == 64) return launch<P, 1, 64, PIECES>(a, s);
  if (v == 128) return launch<P, 1, 128, PIECES>(a, s);
  return launch<P, 2, 256, PIECES>(a, s);
}

}  // namespace

cudaError_t launch_linear(Product p, const LinearArgs& a, cudaStream_t s) {
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  const bool f32 = a.out_f32 != 0;
  switch (p) {
    case Product::kForward:
      return f32 ? pick<Product::kForward, true>(a, s) : pick<Product::kForward, false>(a, s);
    case Product::kGradX:
      return f32 ? pick<Product::kGradX, true>(a, s) : pick<Product::kGradX, false>(a, s);
    case Product::kGradW:
      return launch<Product::kGradW, 2, 256, true>(a, s);
    default: return pick<Product::kInt8, false>(a, s);
  }
}

}  // namespace omni
