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
// taken by token come by cp.async from four warps (TMA row gathers, four rows
// an instruction, took 211 us against 189 for 16384 rows of 2048 to 4096).
// Rows past a group's end that a load brings along only reach columns that
// are not stored; dW, whose sum runs over the rows, zeroes the last block's in
// shared memory before its products.
// CTAS = 2 pairs two CTAs on one 256-wide tile: each holds its half of A and
// of B, and the pair's first CTA issues the MMAs.
// Warps 0-7 drain the accumulators, warps 8 and 10 issue the TMA loads of A
// and of B, warp 9 the MMAs, warps 12-15 gather (11 fills its warpgroup); two
// TMEM accumulators alternate, so a tile is stored while the next is summed.
//
// Pieces: the tensor core's fp32 sums cut every addition towards zero, an
// error of about 1.1e-9 of the result per term of k.  bf16 results do not
// show it; fp32 results are summed in pieces of 512 terms, which the draining
// warps add up in registers, rounded to nearest.  Within a piece the cuts
// remain, all one way: 3e-7 to 5e-7 from 64 bits, about twice what fp32 sums
// rounded to nearest are off by (1.2e-7 to 2.5e-7).
//
// Bounds and measurements (kernel times on one B200, short bursts).  Long
// groups: the tensor pipe; 16384 rows, 2048 to 4096: forward 172-180 us (1530
// to 1600 TFLOP/s of a measured 1673), gathered 187-190, dx 175-180, 8-bit
// 90-100 (2750 to 3060 TOP/s).  Decode: HBM; 512 rows on 64 experts of 2048 to
// 1024 read 268 MB in 46 us (5.8 TB/s).  dW of short groups: its own writes;
// 64 matrices of 4096 x 2048 in fp32 take 391-403 us for 16 rows each (5.3 to
// 5.5 TB/s), 425-440 for 256.  Single tokens: latency, 5 us for the smallest
// call.
#include <atomic>

#include "linear.cuh"
#include "linear_plan.h"
#include "tc_common.cuh"

namespace omni {
namespace {

using namespace tc;

constexpr int kABytes = kBM * 128;  // a k-block's A tile: 128 bytes of k per row
constexpr int kMaxStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kLoadWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kLoadWarpB = kEpiWarps + 2;
constexpr int kRowWarp = kEpiWarps + 4;
constexpr int kRowWarps = 4;
constexpr int kThreads = 32 * (kEpiWarps + 4 + kRowWarps);
// Registers: 512 threads start with 128 each; the two draining warpgroups
// (128 sums a thread) go to 184, the other two to 72: 2 * 184 + 2 * 72 = 4 * 128.
constexpr int kLaunchRegs = 128, kEpiRegs = 184, kOtherRegs = 72;
static_assert(2 * kEpiRegs + 2 * kOtherRegs == 4 * kLaunchRegs && kThreads == 512, "");
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
// Arrive on an mbarrier of either CTA of a pair, without a release at cluster
// scope.  What the arrival reports has been observed by this thread (a
// completed barrier phase, a fence, a finished TMEM load), and lies in this
// CTA's shared memory or TMEM, where the tensor core reads or writes it in
// place.  That the other CTA's products see it is an assumption: PTX promises
// it for an arrival with .release.cluster only, which costs some 2000 cycles
// (558 against 206 us for dW of 16384 x 2048 x 4096 with one per stage).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// barrier of one half (four warps) of the draining warps
__device__ __forceinline__ void half_sync(int half) {
  if (half == 0) asm volatile("bar.sync 2, 128;" ::: "memory");
  else asm volatile("bar.sync 3, 128;" ::: "memory");
}

// shared memory -> a box of y or dx
__device__ __forceinline__ void store_2d(const CUtensorMap* m, uint32_t src, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m),
      "r"(src), "r"(c0), "r"(c1)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
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

// SiLU, z / (1 + e^-z).  For an fp32 result: the exponential is within 2^-23 of
// its value, the sum within 2^-24, the reciprocal within 2^-23 and the product
// within 2^-24.  (A division costs 16 columns of a warp about a microsecond.)
__device__ __forceinline__ float rcp_near(float y) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}
__device__ __forceinline__ float silu_f32(float z) { return z * rcp_near(1.0f + expf(-z)); }
// For a bf16 result: the fast exponential is off by at most 2^-17 of it (the
// rounding of z / ln 2, |z| < 89), where the rounding to bf16 that follows is
// off by up to 2^-8.
__device__ __forceinline__ float silu_fast(float z) { return z * rcp_near(1.0f + __expf(-z)); }

__device__ __forceinline__ void zero16(uint32_t dst) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}

// The bounded wait of this kernel: a try suspends its warp in hardware until
// the phase ends or the hint (nanoseconds) runs out, so that the warps that
// wait leave the issue slots to the warps that work; time-outs as mbar_wait.
// CLUSTER: for barriers that the other CTA of a pair arrives on too.
template <bool CLUSTER>
__device__ __forceinline__ bool try_wait_for(uint32_t bar, uint32_t parity) {
  constexpr uint32_t kHint = 20000;
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kHint)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kHint)
        : "memory");
  return ok != 0;
}
// (times: how many limits the wait may last)
template <bool CLUSTER>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, int32_t* status,
                                         uint32_t times = 1) {
  if (try_wait_for<CLUSTER>(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint64_t polls = 1; !try_wait_for<CLUSTER>(bar, parity); ++polls) {
    if (polls >= uint64_t(kWaitMaxPolls) * times || global_ns() - t0 > kWaitLimitNs * times) {
      raise_status(status, OMNI_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
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
}
__device__ __forceinline__ void tmem_wait() {  // for the loads so far
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- the kernel ------------------------------------------------------------------

struct Maps {
  CUtensorMap a, b;  // boxes of the two operands (a: W, or x for dW)
  CUtensorMap whole;  // B in one box, where a tile has all its columns
  CUtensorMap out;    // the result
};

template <Product P, int CTAS, int BN, bool F32>
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
  static constexpr bool kPieces = F32 && !kI8;
  // Narrow tiles, where a CTA has several: each half of the draining warps takes
  // every other tile (and so always the same accumulator) whole, since a
  // tile's fixed costs, not its columns, bound short sums (1 to 4 % of most
  // small products).  With one tile both halves share it.
  static constexpr bool kAlternate = BN <= 64 && !kPieces;
  static constexpr int kOutSize = F32 ? 4 : 2, kOutBytes = kOutCols * kBM * kOutSize;
  // chunks each half of the draining warps may have on the way out (dW of
  // 16384 x 2048 x 4096 by 8 experts: 220 us with one, 214 with two, 209 with
  // four; narrow tiles have one chunk per half or two, and stages to keep)
  static constexpr int kOutBufs = BN >= 128 ? 4 : BN == 64 && !F32 ? 2 : 1;
  static constexpr int kOut = 2 * kOutBufs * kOutBytes;
  static constexpr int kCols = 2 * BN;            // TMEM columns
  static_assert((kSmemLimit - 600 - 1024 - kOut - OMNI_MAX_GROUPS * sizeof(GroupTab)) / kStage >=
                    kRowWarps,
                "the row warps' turns need as many stages");
  static_assert((kSmemLimit - 1024 - kOut) / kStage <= kMaxStages, "a barrier for each stage");
  static_assert(!kGradW || kNb % 64 == 0, "dW's B tile is made of 64-wide boxes");
};

// Whether dW's block of k with `left` rows to its group's end holds rows past
// it that its last product (16 rows) would read.
__device__ __forceinline__ bool has_tail(int left) { return left < 64 && (left & 15) != 0; }

// One tile: columns j0 .. j0 + n - 1 of a group, i from i0.
struct Tile {
  int i0, j0, n, row0, id, K;
};

template <class C, int CTAS, int BN>
struct TileWalk {
  const LinearArgs& a;
  const GroupTab* tab;
  int groups, mt;
  uint32_t inv;  // (2^32 - 1) / mt: a quotient by it is right or one too small
  int c = 0;
  __device__ __forceinline__ Tile at(int t) {
    while (c + 1 < groups && tab[c + 1].begin <= t) ++c;
    const GroupTab g = tab[c];
    const int local = t - g.begin;
    int q = static_cast<int>(__umulhi(static_cast<uint32_t>(local), inv));
    if (local - q * mt >= mt) ++q;
    Tile r;
    r.i0 = (local - q * mt) * (kBM * CTAS);
    r.j0 = q * BN;
    const int J = C::kGradW ? a.out : g.rows;
    r.n = J - r.j0 < BN ? J - r.j0 : BN;
    r.row0 = g.row0;
    r.id = g.id;
    r.K = C::kGradW ? g.rows : C::kGradX ? a.out : a.in;
    return r;
  }
};

template <Product P, int CTAS, int BN, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ Maps maps, const __grid_constant__ LinearArgs a,
                int stages, int mt, uint32_t mt_inv) {
  using C = Cfg<P, CTAS, BN, F32>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[3 * kMaxStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ GroupScratch scratch;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sA = smem_u32(smem), sB = sA + stages * C::kStageA;
  GroupTab* tab = reinterpret_cast<GroupTab*>(smem + stages * C::kStage + C::kOut);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages;
  const uint32_t tail0 = empty0 + 8 * kMaxStages;  // dW: a stage with rows to zero has landed
  const uint32_t tfull0 = tail0 + 8 * kMaxStages, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = CTAS == 2 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

  const bool gathers = !C::kGradX && a.rows != nullptr;
  // With gathered rows each CTA of a pair waits for its own half and the
  // second tells the first; else the loads of both report to the first.
  const bool halves = gathers;
  if (threadIdx.x == 32 * kLoadWarp) {
    if (a.g.M > 0) {  // (dW of no rows has no operands)
      prefetch_map(&maps.a);
      if (C::kGradW) prefetch_map(&maps.b);
      else if (!gathers) prefetch_map(&maps.whole);
    }
    // A stage is full after its loads' two expects.  With gathered rows it is
    // one expect, the threads of one row warp, and in a pair's first CTA the
    // second's word that its half is ready.  Where dW has rows to zero, the
    // row warps take the place of the expects.
    const int arrivals = gathers ? 1 + 32 + (CTAS == 2 && rank == 0 ? 1 : 0) : 2;
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, arrivals);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(tail0 + 8 * s, gathers ? 1 : 2);
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
  // dW behind dx (LinearArgs::follows) starts without a wait of its own, and
  // waits for dx at its end, before the kernels behind it may start
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
  TileWalk<C, CTAS, BN> walk{a, tab, scratch.total_groups, mt, mt_inv};
  auto n_mma = [](const Tile& t) { return (t.n + 16 * CTAS - 1) / (16 * CTAS) * (16 * CTAS); };

  if (warp < kEpiWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ---- results: TMEM lane = i, column = j; a warp takes 32 lanes and every
    // other chunk of 16 columns
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t sOut = sB + stages * C::kStageB + half * C::kOutBufs * C::kOutBytes;
    const bool issues = quarter == 0 && lane == 0;  // this half's stores
    uint32_t acc_no = 0, out_buf = 0;
    const bool alternate = C::kAlternate && tiles > step;
    // this warp's chunks of columns: from first_c, gap columns apart
    const int gap = alternate ? kOutCols : 2 * kOutCols, first_c = alternate ? 0 : half * kOutCols;
    const DrainRule rule{C::kGradW, !F32 && C::kOutBufs >= 2, gap};
    bool ok = true;
    int t = first;
    for (; t < tiles; t += step) {
      if (alternate && static_cast<int>(acc_no & 1) != half) {
        ++acc_no;
        continue;
      }
      const Tile tl = walk.at(t);
      const int ic = tl.i0 + rank * kBM, i = ic + 32 * quarter + lane;
      float ws = 0.0f;
      if (C::kI8 && i < I) ws = a.Ws[static_cast<int64_t>(tl.id) * a.out + i];

      auto wait_full = [&]() -> bool {
        const bool got = __all_sync(
            0xffffffffu, wait_for<false>(tfull0 + 8 * (acc_no & 1), (acc_no >> 1) & 1, a.status));
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
          if (alternate) mbar_arrive(bar);  // for the other half's warp
        }
        ++acc_no;
      };
      // columns c .. c + 15 of this lane's i leave.  A whole chunk goes through
      // shared memory and from there by TMA, which writes full lines and clips
      // i (the warps' own stores, 64 or 128 bytes each, cost about 10 cycles
      // apiece and bounded short sums); columns cut by a group's end are
      // stored one by one.  dW's columns end with the matrix, where TMA clips.
      auto stage_chunk = [&](uint32_t buf, const float* z) {
        const uint32_t to = buf + (32 * quarter + lane) * C::kOutSize;
#pragma unroll
        for (int q = 0; q < kOutCols; q += 2) {
          if constexpr (F32) {
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + q * kBM * 4), "f"(z[q]) : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + (q + 1) * kBM * 4), "f"(z[q + 1])
                         : "memory");
          } else {
            const __nv_bfloat162 w = __floats2bfloat162_rn(z[q], z[q + 1]);
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + q * kBM * 2),
                         "h"(__bfloat16_as_ushort(w.x))
                         : "memory");
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + (q + 1) * kBM * 2),
                         "h"(__bfloat16_as_ushort(w.y))
                         : "memory");
          }
        }
      };
      auto send_chunk = [&](uint32_t buf, int c) {
        if constexpr (C::kGradW)
          store_3d(&maps.out, buf, ic, tl.j0 + c, tl.id, a.accumulate != 0);
        else
          store_2d(&maps.out, buf, ic, tl.row0 + tl.j0 + c);
      };
      auto next_buf = [&]() -> uint32_t {
        const uint32_t buf = sOut + out_buf * C::kOutBytes;
        if (++out_buf == C::kOutBufs) out_buf = 0;
        return buf;
      };
      auto leave = [&](int c, const float* z) {
        const int n = tl.n - c;
        if (ic >= I) return;
        if (rule.whole(n)) {
          const uint32_t buf = next_buf();
          if (issues)
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(C::kOutBufs - 1) : "memory");
          half_sync(half);
          stage_chunk(buf, z);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          half_sync(half);
          if (issues) send_chunk(buf, c);
        } else if (i < I) {
          const int64_t at = static_cast<int64_t>(tl.row0 + tl.j0 + c) * I + i;
#pragma unroll
          for (int q = 0; q < kOutCols; ++q)
            if (q < n) {
              if constexpr (F32)
                static_cast<float*>(a.o)[at + static_cast<int64_t>(q) * I] = z[q];
              else
                static_cast<__nv_bfloat16*>(a.o)[at + static_cast<int64_t>(q) * I] =
                    __float2bfloat16_rn(z[q]);
            }
        }
      };
      // Two chunks, gap apart, for the barriers of one where both are whole:
      // 16384 x 256 x 4096 in bf16 56 -> 45 us.  Not of fp32, whose stores bound
      // the way out and then wait for two free buffers (dW of 64 experts, 2048 x
      // 4096: 441 -> 485 us).
      auto leave_two = [&](int c, const float* z0, const float* z1) {
        if (ic < I && rule.two(tl.n - c)) {
          const uint32_t b0 = next_buf(), b1 = next_buf();
          if (issues)
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(
                             C::kOutBufs >= 2 ? C::kOutBufs - 2 : 0)
                         : "memory");
          half_sync(half);
          stage_chunk(b0, z0);
          stage_chunk(b1, z1);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          half_sync(half);
          if (issues) {
            send_chunk(b0, c);
            send_chunk(b1, c + gap);
          }
        } else {
          leave(c, z0);
          leave(c + gap, z1);
        }
      };
      // the scales of the 16 columns from c (lanes 0 .. 15) and of the next chunk's
      auto token_scale = [&](int c) -> float {
        const int j = c + lane + (lane < 16 ? 0 : gap - kOutCols);
        if (!C::kI8 || j >= tl.n) return 0.0f;
        const int r = tl.row0 + tl.j0 + j;
        if (a.rows == nullptr) return a.xs[r];
        const int v = a.rows[r];
        return a.xs[v >= 0 && v < a.T ? v : 0];
      };
      auto finish = [&](float* z, float xs, int from) {
        if constexpr (C::kI8) {
#pragma unroll
          for (int q = 0; q < kOutCols; ++q)
            z[q] = static_cast<float>(__float_as_int(z[q])) *
                   __shfl_sync(0xffffffffu, xs, from + q) * ws;
        }
        if (!C::kGradW && a.silu) {
#pragma unroll
          for (int q = 0; q < kOutCols; ++q) z[q] = F32 ? silu_f32(z[q]) : silu_fast(z[q]);
        }
      };

      if constexpr (C::kPieces) {
        constexpr int kMine = BN / 32;  // chunks of this warp
        float sum[kMine][kOutCols];
#pragma unroll
        for (int u = 0; u < kMine; ++u)
#pragma unroll
          for (int q = 0; q < kOutCols; ++q) sum[u][q] = 0.0f;
        for (int k0 = 0; k0 < tl.K; k0 += kPiece) {
          ok = wait_full();
          if (!ok) break;
#pragma unroll
          for (int u = 0; u < kMine; ++u) {
            const int c = (2 * u + half) * kOutCols;
            if (c < tl.n) {
              uint32_t v[kOutCols];
              tmem_ld16(tmem + lanes + (acc_no & 1) * BN + c, v);
              tmem_wait();
#pragma unroll
              for (int q = 0; q < kOutCols; ++q) sum[u][q] += __uint_as_float(v[q]);
            }
          }
          drained();
        }
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < kMine; u += 2) {
          const int c = (2 * u + half) * kOutCols;
          if (c >= tl.n) continue;
          finish(sum[u], 0.0f, 0);
          if (kMine > 1 && c + 2 * kOutCols < tl.n) {
            constexpr int kNext = kMine > 1 ? 1 : 0;
            finish(sum[u + kNext], 0.0f, 0);
            leave_two(c, sum[u], sum[u + kNext]);
          } else {
            leave(c, sum[u]);
          }
        }
      } else {
        // two chunks at a time
        float xs = token_scale(first_c);
        ok = wait_full();
        if (!ok) break;
        const uint32_t acc = tmem + lanes + (acc_no & 1) * BN;
        for (int c = first_c; c < tl.n; c += 2 * gap) {
          uint32_t v[2][kOutCols];
          tmem_ld16(acc + c, v[0]);
          const bool both = gap < BN && c + gap < tl.n;
          if (both) tmem_ld16(acc + c + gap, v[1]);
          tmem_wait();
          const float scale = xs;
          if (c + 2 * gap < tl.n) xs = token_scale(c + 2 * gap);
          else drained();
          float *z0 = reinterpret_cast<float*>(v[0]), *z1 = reinterpret_cast<float*>(v[1]);
          finish(z0, scale, 0);
          if (both) {
            finish(z1, scale, 16);
            leave_two(c, z0, z1);
          } else {
            leave(c, z0);
          }
        }
        if (first_c >= tl.n) drained();
      }
    }
    // A wait ran out.  The half's barriers have no limit and take all four
    // warps, whose waits need not run out alike: this warp still comes to the
    // barriers of the tile that it was waiting for and of all behind it.  It
    // frees no accumulator any more, so the products stop and the other warps'
    // waits run out in turn.
    if (!ok)
      for (; t < tiles; t += step) {
        if (alternate && static_cast<int>(acc_no++ & 1) != half) continue;
        const Tile tl = walk.at(t);
        if (tl.i0 + rank * kBM >= I) continue;
        for (int q = rule.barriers(tl.n, first_c); q > 0; --q) half_sync(half);
      }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // this thread's stores are done
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp || warp == kLoadWarpB) {
      // ---- TMA loads: one warp for each operand that is not gathered (a load
      // costs its thread about 70 cycles, a stage's products 512)
      const bool loads_a = warp == kLoadWarp;
      if (!(gathers && loads_a == C::kGradW) && elect_one()) {
        int s = 0;
        uint32_t ph = 0, issued = 0;
        uint32_t tails = 0;  // dW: parity of each stage's uses of its tail barrier
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = walk.at(t);
          const int nb = n_mma(tl) / CTAS;  // j of this CTA: j0 + rank * nb ..
          const int i0 = tl.i0 + rank * kBM, j0 = tl.j0 + rank * nb;
          const int boxes = (nb + C::kBox - 1) / C::kBox;
          const uint32_t bytes = loads_a ? kABytes : boxes * C::kBox * 128;
          for (int k0 = 0; k0 < tl.K; k0 += C::kStageK) {
            const uint32_t own = full0 + 8 * s;
            if (!wait_for<false>(empty0 + 8 * s, ph ^ 1, a.status)) {
              ok = false;
              break;
            }
            const int subs = C::kSub == 1 || tl.K - k0 <= C::kBlockK ? 1 : 2;
            uint32_t bar = CTAS == 2 && !halves ? leader_addr(own) : own;
            if (C::kGradW && has_tail(tl.K - k0)) {
              // the row warps see these loads first, zero rows, and fill the stage
              bar = tail0 + 8 * s;
              mbar_expect_tx(bar, bytes);
              tails ^= 1u << s;
              if (gathers) mbar_arrive(own);
            } else if (halves) {
              mbar_expect_tx(own, subs * bytes);
            } else if (rank == 0) {
              mbar_expect_tx(own, CTAS * subs * bytes);
            }
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) {
              if (u >= subs) break;
              const uint32_t da = sA + s * C::kStageA + u * kABytes;
              const uint32_t db = sB + s * C::kStageB + u * C::kBBytes;
              const int k = k0 + u * C::kBlockK;
              if (loads_a) {
                if constexpr (C::kGradW) {
                  for (int h = 0; h < 2; ++h)
                    load_2d<CTAS>(da + h * 8192, &maps.a, bar, i0 + 64 * h, tl.row0 + k);
                } else if constexpr (C::kGradX) {
                  for (int h = 0; h < 2; ++h)
                    load_3d<CTAS>(da + h * 8192, &maps.a, bar, i0 + 64 * h, k, tl.id);
                } else {
                  load_3d<CTAS>(da, &maps.a, bar, k, i0, tl.id);
                }
              } else if constexpr (C::kGradW) {
                for (int h = 0; h < boxes; ++h)
                  load_2d<CTAS>(db + h * 8192, &maps.b, bar, j0 + 64 * h, tl.row0 + k);
              } else if (C::kBox == C::kNb || nb == C::kNb) {
                load_2d<CTAS>(db, &maps.whole, bar, k, tl.row0 + j0);
              } else {
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
        if (ok) {
          // every MMA's arrival on a stage's barrier has come, the other CTA's
          // too, before this CTA may exit
          for (uint32_t k = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
               k < issued; ++k)
            wait_for<false>(empty0 + 8 * (k % stages), (k / stages) & 1, a.status);
        } else {
          // a wait timed out: the loads in flight land (each wait bounded again)
          // before the CTA exits
          if (C::kGradW)
            for (int q = 0; q < stages; ++q)
              wait_for<false>(tail0 + 8 * q, ((tails >> q) & 1) ^ 1, a.status);
          if (rank == 0 || halves)
            for (uint32_t k = issued > static_cast<uint32_t>(stages) ? issued - stages : 0u;
                 k < issued; ++k)
              wait_for<false>(full0 + 8 * (k % stages), (k / stages) & 1, a.status);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---- products: issued by one lane of the pair's first CTA
      if ((rank == 0 || halves) && elect_one()) {
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
            const bool starts = k0 % (C::kPieces ? kPiece : 1 << 30) == 0;
            const bool ends =
                left <= C::kStageK || (C::kPieces && (k0 + C::kStageK) % kPiece == 0);
            if (starts && rank == 0) {
              const uint32_t b = acc_no & 1;
              ok = wait_for<CTAS == 2>(tempty0 + 8 * b, ((acc_no >> 1) & 1) ^ 1, a.status);
              if (!ok) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              acc = tmem + b * BN;
            }
            const uint32_t da = sA + s * C::kStageA, db = sB + s * C::kStageB;
            ok = wait_for<CTAS == 2>(full0 + 8 * s, ph, a.status);
            if (!ok) break;
            // rows copied by threads, before the tensor core reads them
            if (gathers) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (rank != 0) {  // this half is ready
              arrive_cluster(leader_addr(full0 + 8 * s));
            } else {
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
            if (ends) ++acc_no;
            if (++s == stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        if (!ok) {
          // the MMAs in flight end (bounded) before TMEM is freed
          if (rank == 0) {
            commit<CTAS>(drain);
            wait_for<false>(drain, 0, a.status);
          }
        }
      }
    } else if (warp >= kRowWarp) {
      // ---- x's rows by token, and dW's rows past a group's end.  The warps take
      // the stages in turn, one each: a stage costs a warp some 650 cycles of
      // waits, arrival and bookkeeping beside its copies (16 bytes a thread,
      // eight threads to a row's 128 bytes, four rows at a time).
      // (Two warps to a stage, which halves the time from a free stage to its last
      // copy, is slower: 216 against 187 us at 16384 x 2048 x 4096.)
      const int mine = warp - kRowWarp;
      const int sub = lane >> 3, piece = lane & 7;
      // where the copy of row 4 q + sub goes: even and odd q (swizzled)
      const uint32_t even = static_cast<uint32_t>(sub * 128 + ((piece ^ sub) * 16));
      const uint32_t odd = even ^ 64u;
      const int64_t pitch = static_cast<int64_t>(a.in) * (C::kI8 ? 1 : 2);
      const char* x = static_cast<const char*>(a.x);
      auto checked = [&](int v) -> int {  // a row number as the caller gave it
        if (v >= 0 && v < a.T) return v;
        raise_status(a.status, OMNI_DEV_BAD_INDEX);
        return 0;
      };
      // Stage number no.  A warp waits for every kRowWarps-th stage only; with at
      // least that many stages in the ring, the wait before told it that the
      // barrier is at most one phase behind, so the parity is not mistaken.
      auto wait_empty = [&](uint32_t no, int* s) -> bool {
        *s = static_cast<int>(no % stages);
        const uint32_t ph = (no / stages) & 1;
        return __all_sync(0xffffffffu, wait_for<false>(empty0 + 8 * *s, ph ^ 1, a.status));
      };
      uint32_t no = 0;  // of the tile's first stage
      bool ok = true;
      if constexpr (C::kGradW) {
        uint32_t tails = 0;
        WaitSpan span;
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = walk.at(t);
          const int blocks = (tl.K + 63) / 64, last = tl.K - 64 * (blocks - 1);
          const bool tail = blocks > 0 && has_tail(last);
          const int tail_s = static_cast<int>((no + blocks - 1) % stages);
          // zeroes the rows past the group's end up to the last product's 16, of
          // both operands: what is there may be infinite
          span.tile(blocks);
          auto zero_tail = [&]() {
            // (with gathered rows this warp has just taken the same stage)
            ok = __all_sync(0xffffffffu,
                            wait_for<false>(tail0 + 8 * tail_s, (tails >> tail_s) & 1, a.status,
                                            gathers ? 1 : span.limits()));
            if (!ok) return;
            span.waited();
            const uint32_t da = sA + tail_s * C::kStageA, db = sB + tail_s * C::kStageB;
            const int chunks = (n_mma(tl) / CTAS + 63) / 64;
            for (int g = lane; g < (16 - (last & 15)) * 8; g += 32) {
              const uint32_t at = (last + (g >> 3)) * 128 + (g & 7) * 16;
              if (!gathers)
                for (int h = 0; h < 2; ++h) zero16(da + h * 8192 + at);
              for (int h = 0; h < chunks; ++h) zero16(db + h * 8192 + at);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          };
          if (gathers) {
            const int c = tl.i0 + rank * kBM + 8 * piece;  // column of x
            const char* xc = x + static_cast<int64_t>(c) * 2;
            const bool wide = tl.i0 + rank * kBM + kBM <= a.in;
            auto fetch = [&](int kb) -> int2 {  // a block's 64 row numbers
              const int r = 64 * kb + lane;
              return make_int2(r < tl.K ? fresh(a.rows + tl.row0 + r) : 0,
                               r + 32 < tl.K ? fresh(a.rows + tl.row0 + r + 32) : 0);
            };
            int kb = static_cast<int>((mine - no) & (kRowWarps - 1));
            int2 ahead = fetch(kb);
            for (; kb < blocks; kb += kRowWarps) {
              const int left = tl.K - 64 * kb;
              const int lo = lane < left ? checked(ahead.x) : -1;
              const int hi = lane + 32 < left ? checked(ahead.y) : -1;
              ahead = fetch(kb + kRowWarps);
              int s;
              ok = wait_empty(no + kb, &s);
              if (!ok) break;
              const uint32_t to = sA + s * C::kStageA;
              if (wide && left >= 64) {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                  const int row = __shfl_sync(0xffffffffu, q < 8 ? lo : hi, (4 * q + sub) & 31);
                  const char* p = xc + row * pitch;
                  copy16(to + q * 512 + (q & 1 ? odd : even), p);
                  copy16(to + q * 512 + (q & 1 ? odd : even) + 8192, p + 128);
                }
              } else {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                  const int row = __shfl_sync(0xffffffffu, q < 8 ? lo : hi, (4 * q + sub) & 31);
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const bool in = row >= 0 && c + 64 * h < a.in;
                    copy16_or_zero(to + q * 512 + (q & 1 ? odd : even) + h * 8192,
                                   in ? xc + row * pitch + 128 * h : x, in);
                  }
                }
              }
              if (tail && kb == blocks - 1) {
                zero_tail();
                if (!ok) break;
              }
              copies_arrive(full0 + 8 * s);
            }
          } else if (tail && mine == 0) {
            // one warp takes every such block, in order: it is then never more
            // than one phase from a tail barrier's, and its parity says which
            zero_tail();
            __syncwarp();
            if (ok && lane == 0) {  // in place of the loads' two expects
              if (CTAS == 2) {
                arrive_cluster(leader_addr(full0 + 8 * tail_s));
              } else {
                mbar_arrive(full0 + 8 * tail_s);
                mbar_arrive(full0 + 8 * tail_s);
              }
            }
          }
          if (tail) tails ^= 1u << tail_s;
          no += blocks;
        }
      } else if (gathers) {
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = walk.at(t);
          const int nb = n_mma(tl) / CTAS;
          const int there = tl.n - rank * nb, row0 = tl.row0 + tl.j0 + rank * nb;
          const int blocks = (tl.K + C::kStageK - 1) / C::kStageK;
          // the tile's row numbers, 32 to a register of the warp (past the
          // group's end any row will do: its column is not stored)
          int at[(C::kNb + 31) / 32];
#pragma unroll
          for (int h = 0; h < (C::kNb + 31) / 32; ++h)
            at[h] = 32 * h + lane < there ? checked(a.rows[row0 + 32 * h + lane]) : 0;
          for (int kb = static_cast<int>((mine - no) & (kRowWarps - 1)); kb < blocks; kb += kRowWarps) {
            int s;
            ok = wait_empty(no + kb, &s);
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) {
              const int k = kb * C::kStageK + u * C::kBlockK;
              if (k >= tl.K) break;
              const uint32_t to = sB + s * C::kStageB + u * C::kBBytes;
              const int64_t c = static_cast<int64_t>(k) * (C::kI8 ? 1 : 2) + 16 * piece;  // bytes
              const char* xc = x + c;
              if (k + C::kBlockK <= tl.K && nb == C::kNb) {
#pragma unroll
                for (int q = 0; q < C::kNb / 4; ++q) {
                  const int row = __shfl_sync(0xffffffffu, at[q / 8], (4 * q + sub) & 31);
                  copy16(to + q * 512 + (q & 1 ? odd : even), xc + row * pitch);
                }
              } else if (k + C::kBlockK <= tl.K) {
#pragma unroll
                for (int q = 0; q < C::kNb / 4; ++q)
                  if (4 * q < nb) {
                    const int row = __shfl_sync(0xffffffffu, at[q / 8], (4 * q + sub) & 31);
                    copy16(to + q * 512 + (q & 1 ? odd : even), xc + row * pitch);
                  }
              } else {
                const bool in = c < pitch;
#pragma unroll
                for (int q = 0; q < C::kNb / 4; ++q)
                  if (4 * q < nb) {
                    const int row = __shfl_sync(0xffffffffu, at[q / 8], (4 * q + sub) & 31);
                    copy16_or_zero(to + q * 512 + (q & 1 ? odd : even),
                                   in ? xc + row * pitch : x, in);
                  }
              }
            }
            copies_arrive(full0 + 8 * s);
          }
          no += blocks;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
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

template <Product P, int CTAS, int BN, bool F32>
cudaError_t launch(const LinearArgs& a, int sms, cudaStream_t s) {
  using C = Cfg<P, CTAS, BN, F32>;
  Maps m{};
  const int64_t W[3] = {a.in, a.out, a.g.E}, X[2] = {a.in, a.T}, Y[2] = {a.out, a.g.M};
  const int kb = C::kBlockK, esize = C::kI8 ? 1 : 2;
  const CUtensorMapDataType type =
      C::kI8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int box_w[3] = {kb, C::kMnA ? 64 : kBM, 1}, box_r[2] = {kb, C::kBox};
  const int box_b[2] = {kb, C::kNb}, box_64[2] = {64, 64};
  bool ok = true;
  if (a.g.M > 0) {
    if (C::kGradW) {
      ok = make_map_nd(&m.a, a.x, type, esize, 2, X, box_64) &&
           make_map_nd(&m.b, a.dy, type, esize, 2, Y, box_64);
    } else {
      // (gathered rows need no map; a box of all of a tile's columns and one of
      // some are the same where tiles are narrow)
      ok = make_map_nd(&m.a, a.W, type, esize, 3, W, box_w);
      if (C::kGradX || a.rows == nullptr) {
        const void* b = C::kGradX ? a.dy : a.x;
        const int64_t* dim = C::kGradX ? Y : X;
        ok = ok && make_map_nd(&m.whole, b, type, esize, 2, dim, box_b);
        if (C::kBox < C::kNb) ok = ok && make_map_nd(&m.b, b, type, esize, 2, dim, box_r);
      }
    }
  }
  const int box_o[3] = {kBM, kOutCols, 1};
  const int64_t O[2] = {C::kGradX ? a.in : a.out, a.g.M};
  if (C::kGradW || a.g.M >= kOutCols)  // (fewer rows have no whole chunk)
    ok = ok && make_map_nd(&m.out, a.o,
                           F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           C::kOutSize, C::kGradW ? 3 : 2, C::kGradW ? W : O, box_o,
                           CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!ok) return cudaErrorInvalidValue;
  const size_t fixed = 1024 + C::kOut + sizeof(GroupTab) * static_cast<size_t>(a.g.G);
  const size_t statics = sizeof(GroupScratch) + (3 * kMaxStages + 5) * 8 + 64;
  const int stages = static_cast<int>((kSmemLimit - statics - fixed) / C::kStage);
  const size_t smem = fixed + static_cast<size_t>(stages) * C::kStage;
  auto kernel = k_linear_tc<P, CTAS, BN, F32>;
  int dev = 0;
  cudaGetDevice(&dev);
  // once per device (of a bit each; later devices are asked every time)
  static std::atomic<uint64_t> allowed{0};
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if ((allowed.load(std::memory_order_relaxed) & bit) == 0) {
    OMNI_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(kSmemLimit - statics)));
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
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
  OMNI_TRY(cudaLaunchKernelEx(&cfg, kernel, m, a, stages, static_cast<int>(mt),
                              0xffffffffu / static_cast<uint32_t>(mt)));
  return cudaGetLastError();
}

template <Product P, bool F32>
cudaError_t pick(const LinearArgs& a, int sms, cudaStream_t s) {
  switch (pick_shape(P == Product::kGradX ? a.in : a.out, a.g.M, a.g.G, sms)) {
    case 0: return launch<P, 1, 32, F32>(a, sms, s);
    case 1: return launch<P, 1, 64, F32>(a, sms, s);
    case 2: return launch<P, 1, 128, F32>(a, sms, s);
    default: return launch<P, 2, 256, F32>(a, sms, s);
  }
}

cudaError_t pick_grad_w(const LinearArgs& a, int sms, cudaStream_t s) {
  return grad_w_pairs(a.in, a.out, a.g.M, a.g.G, sms)
             ? launch<Product::kGradW, 2, 256, true>(a, sms, s)
             : launch<Product::kGradW, 1, 128, true>(a, sms, s);
}

}  // namespace

cudaError_t launch_linear(Product p, const LinearArgs& a, cudaStream_t s) {
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const bool f32 = a.out_f32 != 0;
  switch (p) {
    case Product::kForward:
      return f32 ? pick<Product::kForward, true>(a, sms, s)
                 : pick<Product::kForward, false>(a, sms, s);
    case Product::kGradX:
      return f32 ? pick<Product::kGradX, true>(a, sms, s)
                 : pick<Product::kGradX, false>(a, sms, s);
    case Product::kGradW: return pick_grad_w(a, sms, s);
    default:
      return f32 ? pick<Product::kInt8, true>(a, sms, s) : pick<Product::kInt8, false>(a, sms, s);
  }
}

}  // namespace omni
