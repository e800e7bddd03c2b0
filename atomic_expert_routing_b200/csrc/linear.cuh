// Grouped products (the wide experts and the 8-bit products): what a launch
// gets, and the group table every CTA builds from the caller's device arrays.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace omni {

// One group as the kernels see it: its first tile, rows and matrix.
struct __align__(16) GroupTab {
  int32_t begin;  // tiles of all earlier groups
  int32_t row0;   // first product row
  int32_t rows;
  int32_t id;     // matrix
};

// The group arrays of a call (device pointers, see include/omnimoe.h).
struct Groups {
  int64_t M;
  int32_t E, G;
  const int32_t* off;       // nullptr: one group of all M rows
  const int32_t* ids;       // nullptr: matrix g
  const int32_t* n_groups;  // nullptr: G
};

// Shared memory of build_groups beside the table: per-warp partial results
// and the totals.
constexpr int kGroupWarps = 8;
struct GroupScratch {
  int32_t off_max[kGroupWarps], id_max[kGroupWarps], tiles[kGroupWarps], used[kGroupWarps];
  int32_t total_tiles, total_groups;
};

// An entry of a caller's array, read from L2.  dW behind dx of the same call
// may start before it has waited for the kernels ahead itself (LinearArgs), and
// so reads nothing through L1, which might hold what was there before them.
__device__ __forceinline__ int32_t fresh(const int32_t* p) { return __ldcg(p); }

// Builds the table of the groups that have tiles, in order, with the CTA's
// first kGroupWarps warps (the caller's barrier makes it visible).
// tiles_of(rows): tiles of a group of that many rows, 0 to leave it out.  A
// group counts only if its first offset is the largest entry so far, its end
// is neither before that nor past M, and its id lies in [0, E) above every
// earlier id: no two listed groups then share a row or a matrix, whatever
// the arrays hold (G <= E, so without ids group g's is g).  status: where the
// bad-index bit goes (one CTA passes it, the others nullptr).
// The first round's entries are loaded beside the group count, and up to 32
// groups need no exchange between warps: the table is the latency of one
// load and some twenty shuffles, on the path of every call.
template <class TilesOf>
__device__ __forceinline__ void build_groups(const Groups& P, const TilesOf& tiles_of,
                                             GroupTab* tab, GroupScratch* sh, int32_t* status) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kThreads = 32 * kGroupWarps;
  if (P.off == nullptr) {
    if (tid == 0) {
      const int32_t rows = static_cast<int32_t>(P.M);
      tab[0] = GroupTab{0, 0, rows, 0};
      sh->total_tiles = tiles_of(rows);
      sh->total_groups = sh->total_tiles > 0 ? 1 : 0;
    }
    return;
  }
  int n = P.G;
  bool bad = false;
  int32_t a = 0, b = 0, id = -1;
  auto load = [&](int g) {  // G entries exist whatever the count says
    const bool there = g < P.G;
    a = there ? fresh(P.off + g) : 0;
    b = there ? fresh(P.off + g + 1) : 0;
    id = !there ? -1 : P.ids != nullptr ? fresh(P.ids + g) : g;
  };
  load(tid);
  if (P.n_groups != nullptr) {
    const int v = fresh(P.n_groups);
    bad = v < 0 || v > n;
    n = v < 0 ? 0 : (v > n ? n : v);
  }
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  int32_t carry_off = 0, carry_id = -1, carry_tiles = 0, carry_used = 0;
  for (int g0 = 0; g0 < n; g0 += kThreads) {
    const int g = g0 + tid;
    const bool in = g < n;
    if (g0 > 0) load(g);
    const int warps = n - g0 > 32 * (kGroupWarps - 1) ? kGroupWarps : (n - g0 + 31) / 32;
    if (warps == 1 && warp > 0) break;  // the last round is the first warp's
    // running maxima of the offsets (inclusive) and ids (exclusive)
    int32_t mo = in ? a : 0, mi = in ? id : -1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t po = __shfl_up_sync(0xffffffffu, mo, o);
      const int32_t pi = __shfl_up_sync(0xffffffffu, mi, o);
      if (lane >= o) {
        mo = po > mo ? po : mo;
        mi = pi > mi ? pi : mi;
      }
    }
    int32_t mi_before = __shfl_up_sync(0xffffffffu, mi, 1);
    if (lane == 0) mi_before = -1;
    int32_t before_off = carry_off, before_id = carry_id;
    if (warps > 1) {
      if (lane == 31) {
        sh->off_max[warp] = mo;
        sh->id_max[warp] = mi;
      }
      sync();
      for (int w = 0; w < warps; ++w) {
        if (w == warp) {
          before_off = carry_off;
          before_id = carry_id;
        }
        carry_off = sh->off_max[w] > carry_off ? sh->off_max[w] : carry_off;
        carry_id = sh->id_max[w] > carry_id ? sh->id_max[w] : carry_id;
      }
    }
    mo = before_off > mo ? before_off : mo;
    mi_before = before_id > mi_before ? before_id : mi_before;
    const bool ok = in && a >= 0 && a == mo && b >= a && b <= P.M && id >= 0 && id < P.E &&
                    id > mi_before;
    bad |= in && !ok;
    // places in the table; a bad group whose matrix is known is one without rows
    const int32_t rows = ok ? b - a : 0;
    const int32_t mine = ok || (in && P.ids == nullptr) ? tiles_of(rows) : 0;
    const unsigned with = __ballot_sync(0xffffffffu, mine > 0);
    int32_t st = mine, before_t = 0, before_u = __popc(with & lanemask_lt());
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t pt = __shfl_up_sync(0xffffffffu, st, o);
      if (lane >= o) st += pt;
    }
    int32_t all_t = 0, all_u = 0;
    if (warps > 1) {
      if (lane == 31) {
        sh->tiles[warp] = st;
        sh->used[warp] = __popc(with);
      }
      sync();
      int32_t u = 0;
      for (int w = 0; w < warps; ++w) {
        if (w == warp) {
          before_t = all_t;
          u = all_u;
        }
        all_t += sh->tiles[w];
        all_u += sh->used[w];
      }
      before_u += u;
    } else {
      all_t = __shfl_sync(0xffffffffu, st, 31);
      all_u = __popc(with);
    }
    if (mine > 0)
      tab[carry_used + before_u] = GroupTab{carry_tiles + before_t + st - mine, a, rows, id};
    carry_tiles += all_t;
    carry_used += all_u;
    // the next round writes the maxima before its first barrier and the sums
    // after it: every thread is past its reads of both by then
  }
  if (tid == 0) {
    sh->total_tiles = carry_tiles;
    sh->total_groups = carry_used;
  }
  if (bad) raise_status(status, OMNI_DEV_BAD_INDEX);
}

// What the products of one launch read and write.
struct LinearArgs {
  Groups g;
  int64_t T;
  int32_t in, out;
  int32_t out_f32, silu, accumulate;
  // dx (leads) and dW (follows) of one call may run side by side: dx lets dW
  // start once its own wait for the kernels ahead is over.  Their writes are
  // complete by then, in the L2; that a kernel which has not waited itself sees
  // them there is an assumption beyond what the programming model states for
  // dependent launches, so dW reads x, dy, rows and the group arrays from L2
  // only (TMA, cp.async.cg, fresh()).
  int32_t leads, follows;
  const int32_t* rows;  // nullable
  const void* x;        // [T x in]
  const void* W;        // [E x out x in]
  const void* dy;       // [M x out]
  const float* xs;      // [T] (8-bit products)
  const float* Ws;      // [E x out]
  void* o;              // y [M x out], dx [M x in] or dW [E x out x in]
  int32_t* status;
};

enum class Product { kForward, kGradX, kGradW, kInt8 };

cudaError_t launch_linear(Product p, const LinearArgs& a, cudaStream_t s);
cudaError_t launch_quantize_rows(int64_t n, int64_t width, bool f32, const void* src, int8_t* q,
                                 float* scale, cudaStream_t s);

}  // namespace omni
