// Persistent tcgen05 GEMM engine on CTA pairs (cta_group::2) for bf16 operands with fp32
// accumulation in TMEM:  D[256 x W] = A[256 x K] * B[W x K]^T per tile, W <= 256.
//
// Two CTAs of a cluster (two SMs) work on one tile.  Each holds 128 rows of A and W/2 rows of
// B in its own shared memory and the accumulator of its 128 rows in its own TMEM; one
// tcgen05.mma of the even CTA reads both.  An SM therefore stages 32 KiB per 64-wide k-block
// for 128 x 256 x 64 products, a third less than a CTA alone on a 128 x 256 tile (48 KiB),
// which is what the L2 -> SM path has to carry.
//
//   warp 0     producer (both CTAs): one lane streams its CTA's halves of A and B through a
//              ring of stages; their bytes count on the even CTA's full barrier
//   warp 1     MMA issuer (even CTA; allocates TMEM in both): commits every stage back to both
//              producers and every finished tile to both epilogues
//   warps 2-9  epilogue (both CTAs): warp w reads TMEM lanes [32 (w & 3), +32); warps 2-5 take
//              the even 64-column pieces of the tile, 6-9 the odd ones.  Two 256-column
//              accumulators, so a tile's epilogue runs beside the next tile's products.
//
// Operand layouts are those of tc_gemm.cuh (128-byte swizzle; K-major rows of 64 k, or MN-major
// blocks of 64 x 64).  Loads carry no multicast.  Every wait is bounded (tc_common.cuh); on
// expiry a CTA leaves its loops, its peer does the same on its own budget, and both meet at the
// final cluster barrier.
#pragma once

#include "tc_gemm.cuh"

namespace pkm {
namespace tc {

constexpr int kPairM = 256;                  // rows of a tile: 128 per CTA
constexpr int kPairHalf = 128;               // rows of A, and at most of B, per CTA
constexpr int kPairStage = 2 * kPairHalf * kBK * 2;  // 32 KiB: A half, then B half
constexpr int kPairThreads = 320;
// The shared memory that an epilogue's staging leaves goes into stages of the ring.
constexpr int kPairSmemMost = 232448 - 1024 - 512;
template <class Prob>
constexpr int pair_stages() {
  return (kPairSmemMost - 8 * Prob::kStg) / kPairStage;
}
template <class Prob>
constexpr size_t pair_smem() {
  return 1024 + (size_t)pair_stages<Prob>() * kPairStage + 8 * Prob::kStg;
}

// Operands and outputs.  A K-major B has a second map with low boxes for narrow tiles.  An
// MN-major operand whose columns are whole blocks of 64 is mapped as blocks (a3, b3), so that one
// load brings two of them.
struct PairMaps {
  CUtensorMap a[3], b[2], low[2], o[3];
  bool a3, b3[2];
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Shared-memory address of the same variable in the even CTA of the pair.
__device__ __forceinline__ uint32_t even_cta_addr(const void* p) {
  return smem_u32(p) & 0xFEFFFFFFu;
}
__device__ __forceinline__ void pair_load_2d(void* smem_dst, const CUtensorMap* map, int x, int y,
                                             uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(even_cta_addr(bar))
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y,
                                             int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(even_cta_addr(bar))
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Arrive on this barrier of both CTAs once every product issued so far is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void arrive_even_cta(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   even_cta_addr(bar))
               : "memory");
}

// ------------------------------------------------------------------ the walk over tiles
// Column tiles of `width` and one narrower for the rest; every pair of CTAs takes one tile of a
// round.  Wide tiles fill whole rounds first.  What is left then is short: the remaining wide
// tiles, each cut into `split` column pieces, and after them the narrow ones, which go round in
// turns of alternating direction, so that a pair with a wide piece is the last to get another.
constexpr int kBand = 8;
struct PairWalk {
  int m_tiles;  // row tiles (all kinds together)
  int full_n;   // column tiles of full width
  int width;    // a multiple of 64
  int rest;     // width of the last column tile, a multiple of 64, or 0
  int whole;    // wide tiles in whole rounds
  int split;    // column pieces of each remaining wide tile
  int total;
};
struct WalkTile {
  int mt, n0, w;
};
// Wide tiles go in bands of kBand row tiles, all column tiles of a band before the next, so that
// the tiles in flight share rows of A and of B in L2.
__device__ __forceinline__ WalkTile walk_tile(const PairWalk& W, int u) {
  const int wide = W.m_tiles * W.full_n;
  int part = 0, i = u, w = W.width;
  if (u >= W.whole) {
    const int v = u - W.whole, left = (wide - W.whole) * W.split;
    if (v >= left) return WalkTile{v - left, W.full_n * W.width, W.rest};
    i = W.whole + v / W.split;
    part = v % W.split;
    w = W.width / W.split;
  }
  const int per = kBand * W.full_n, b = i / per, r = i % per;
  const int rows = min(kBand, W.m_tiles - b * kBand);
  return WalkTile{b * kBand + r % rows, r / rows * W.width + part * w, w};
}
// The tile of CTA pair `pair` in round r.
__device__ __forceinline__ int tile_of_round(int r, int pair, int pairs, int whole) {
  const bool back = r * pairs >= whole && ((r - whole / pairs) & 1);
  return r * pairs + (back ? pairs - 1 - pair : pair);
}

// What an epilogue call works with: the tile, its accumulator, the warp's place.
struct PairEpi {
  const PairMaps* maps;
  uint32_t taddr;      // TMEM address of the accumulator's column 0 on this warp's lanes
  unsigned char* stg;  // the warp's staging bytes (1024-byte aligned)
  int row0;            // first row of the warp's 32, relative to the tile
  int set;             // 0: even pieces, 1: odd
  int lane;
};

// A problem provides
//   kAMN, kBMN          operand layouts (0 K-major, 1 MN-major)
//   kStg                staging bytes of an epilogue warp (a multiple of 1024)
//   Params              with int* status
//   Tile, tile(P, u)    the u-th tile; Tile::w is its MMA width (a multiple of 64)
//   num_tiles(P), num_kblocks(P)
//   load(P, maps, t, kb, rank, sa, sb, bar)   load_bytes(maps, t) bytes per CTA
//   prefetch(P, t, epi, early)     loads into registers that the epilogue of t begins with
//   epilogue(P, t, epi, early)
template <class Prob>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    tc_pair_kernel(const __grid_constant__ PairMaps maps, const typename Prob::Params P) {
  constexpr int S = pair_stages<Prob>();
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], tfull_bar[2], tempty_bar[2],
      drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  // both CTAs have the same layout, so the aligned base is at the same offset in each
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 16);  // 8 epilogue warps of each CTA
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  int* status = P.status;
  const int ntiles = Prob::num_tiles(P);
  const int nk = Prob::num_kblocks(P);

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int r = 0; r * pairs < ntiles && ok; ++r) {
        const int u = tile_of_round(r, pair, pairs, P.walk.whole);
        if (u >= ntiles) continue;
        const typename Prob::Tile t = Prob::tile(P, u);
        const uint32_t bytes = 2 * Prob::load_bytes(maps, t);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag, status)) {
            ok = false;
            break;
          }
          unsigned char* sa = smem + (size_t)stage * kPairStage;
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], bytes);
          Prob::load(P, maps, t, kb, (int)rank, sa, sa + kPairStage / 2, &full_bar[stage]);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // loads still in flight land before the CTA exits: their completion cannot be waited
        // for in both CTAs after an expired wait, so give them a fixed, generous time
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitBudgetCycles / 16) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int r = 0; r * pairs < ntiles && ok; ++r) {
        const int u = tile_of_round(r, pair, pairs, P.walk.whole);
        if (u >= ntiles) continue;
        const typename Prob::Tile t = Prob::tile(P, u);
        const uint32_t idesc = idesc_bf16(kPairM, t.w, Prob::kAMN, Prob::kBMN);
        if (!mbar_wait(&tempty_bar[acc], ((acc_phase >> acc) & 1u) ^ 1u, &abort_flag, status))
          break;
        tc_fence_after();
        const uint32_t dt = tmem_base + (uint32_t)acc * kBN;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full_bar[stage], phase, &abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + (size_t)stage * kPairStage);
          const uint32_t sb = sa + kPairStage / 2;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t da = Prob::kAMN ? desc_mnmajor_sw128(sa + 2048u * k, 8192u, 1024u)
                                           : desc_kmajor_sw128(sa) + (uint64_t)(2 * k);
            const uint64_t db = Prob::kBMN ? desc_mnmajor_sw128(sb + 2048u * k, 8192u, 1024u)
                                           : desc_kmajor_sw128(sb) + (uint64_t)(2 * k);
            pair_mma(dt, da, db, idesc, (kb | k) != 0 ? 1u : 0u);
          }
          issued = true;
          pair_commit(&empty_bar[stage]);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        pair_commit(&tfull_bar[acc]);
        acc_phase ^= 1u << acc;
        acc ^= 1;
      }
      if (issued) pair_commit(&drain_bar);
    }
    // every product, and every arrival its commits send to either CTA, is done before TMEM and
    // shared memory are given up
    if (lane == 0 && pair < ntiles && !abort_flag) {
      const long long t0 = clock64();
      while (!mbar_try_wait_sleep(&drain_bar, 0, 2000u) && !abort_flag &&
             clock64() - t0 < kWaitBudgetCycles) {
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;
    PairEpi epi;
    epi.maps = &maps;
    epi.stg = smem + (size_t)S * kPairStage + (size_t)(warp - 2) * Prob::kStg;
    epi.row0 = (int)rank * kPairHalf + quarter * 32;
    epi.set = (warp - 2) >> 2;
    epi.lane = lane;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int r = 0; r * pairs < ntiles; ++r) {
      const int u = tile_of_round(r, pair, pairs, P.walk.whole);
      if (u >= ntiles) continue;
      const typename Prob::Tile t = Prob::tile(P, u);
      typename Prob::Early early;
      Prob::prefetch(P, t, epi, early);
      // warp-uniform: lane 0 waits, so the warp reaches the .sync.aligned TMEM loads together
      int got = 0;
      if (lane == 0)
        got = mbar_wait(&tfull_bar[acc], (acc_phase >> acc) & 1u, &abort_flag, status) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      tc_fence_after();
      epi.taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)acc * kBN;
      Prob::epilogue(P, t, epi, early);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_even_cta(&tempty_bar[acc]);
      acc_phase ^= 1u << acc;
      acc ^= 1;
    }
    if (lane == 0) bulk_wait_all();  // tile stores complete before the CTA exits
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols)
                 : "memory");
  }
}

}  // namespace tc
}  // namespace pkm
