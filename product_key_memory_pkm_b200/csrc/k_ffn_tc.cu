// The gated feed-forward block on tensor cores (bf16 storage), on the CTA-pair engine.
//
//   forward    gate   h = act(x Wg^T) * (x Wu^T): one tile holds 128 columns of both projections
//                     (the even CTA stages Wg's rows, the odd one Wu's), so the epilogue has g
//                     and u of an element in one thread and neither reaches memory unless kept
//              down   y = h Wd^T
//   backward   dh     dy Wd, whose epilogue reads the kept projections and writes h, dg and du
//              weights  dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//              dx     dg Wg + du Wu, one accumulator over both products
//
// h, dg and du are rounded to bf16: they are operands of bf16 products.
#include <algorithm>
#include <atomic>

#include "ffn_internal.cuh"
#include "tc_pair.cuh"

namespace pkm {
namespace {

using namespace tc;
using bf = __nv_bfloat16;

// ------------------------------------------------------------------ device helpers
// Fast forms: 2^x and the reciprocal are good to ~2^-22, far inside the bf16 rounding that
// every result of them gets.  (The .ftz forms: the others spend as many instructions again on
// subnormal operands, which here only arise where the result is 0 or 1 to fp32.)
__device__ __forceinline__ float sigmoid_fast(float v) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}
// Phi(v), and e = exp(-v^2 / 2) for the slope, from one exponential and one reciprocal: with
// t = 1 / (1 + 0.2 sqrt(2) |v|), Phi(-|v|) = e t p(t), where t p(t) stands for
// erfcx(|v| / sqrt(2)) / 2.  p is a degree-8 fit to that function on 0 < t <= 1 for the least
// largest relative error (1.3e-7; iteratively reweighted least squares); with fp32 arithmetic
// Phi is good to 1.4e-6 of itself for v > -5 and 4e-6 for v > -9, so the tail keeps its accuracy.
__device__ __forceinline__ float normal_cdf_fast(float v, float* e) {
  const float a = fabsf(v);
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.282842712474619f, a, 1.f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(*e) : "f"(v * v * -0.7213475204444817f));
  float p = 0.025132272392511368f;
  p = fmaf(p, t, -0.09145597368478775f);
  p = fmaf(p, t, 0.08455199748277664f);
  p = fmaf(p, t, -0.0028124095406383276f);
  p = fmaf(p, t, 0.07072025537490845f);
  p = fmaf(p, t, 0.08426965773105621f);
  p = fmaf(p, t, 0.1039215549826622f);
  p = fmaf(p, t, 0.11283478885889053f);
  p = fmaf(p, t, 0.11283793300390244f);
  const float q = p * t * *e;
  return v < 0.f ? q : 1.f - q;
}
template <int ACT>
__device__ __forceinline__ float act_fast(float v) {
  float e;
  return v * (ACT == PKM_ACT_GELU ? normal_cdf_fast(v, &e) : sigmoid_fast(v));
}
// act(v) and act'(v).  GELU's slope is Phi(v) + v phi(v); SiLU's s (1 + v (1 - s)), with a = v s
// as s + (a - a s).
template <int ACT>
__device__ __forceinline__ void act_and_slope_fast(float v, float* a, float* slope) {
  if (ACT == PKM_ACT_GELU) {
    float e;
    const float c = normal_cdf_fast(v, &e);
    *a = v * c;
    *slope = fmaf(v * kInvSqrt2Pi, e, c);
    return;
  }
  const float s = sigmoid_fast(v);
  *a = v * s;
  *slope = s + fmaf(-*a, s, *a);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Columns [32 half, +32) of a warp's 32 x 64 bf16 piece into a 4 KiB staging tile (row = lane,
// 128-byte swizzle: 16-byte chunk v of row r sits at chunk v ^ (r & 7)), so that a store's rows
// are whole 128-byte lines.
__device__ __forceinline__ void stage_bf16(unsigned char* stg, int lane, int half,
                                           const uint32_t (&p)[16]) {
  uint4* s = reinterpret_cast<uint4*>(stg) + lane * 8;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    s[(half * 4 + v) ^ (lane & 7)] =
        make_uint4(p[4 * v], p[4 * v + 1], p[4 * v + 2], p[4 * v + 3]);
}
// The 32 columns alone, rows of 64 bytes (64-byte swizzle), 2 KiB: for the epilogues of three
// outputs, where the 48 KiB this saves are a fifth stage of the ring (16384 x 1600 x 6400: gate with
// kept projections 841 -> 763 thousand cycles, dh 530 -> 493; the waits for operands shrink).
__device__ __forceinline__ void stage_bf16_32(unsigned char* stg, int lane, const uint32_t (&p)[16]) {
  uint4* s = reinterpret_cast<uint4*>(stg) + lane * 4;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    s[v ^ ((lane >> 1) & 3)] = make_uint4(p[4 * v], p[4 * v + 1], p[4 * v + 2], p[4 * v + 3]);
}
// A warp's 32 x 32 fp32 piece, the same way.
__device__ __forceinline__ void stage_f32(unsigned char* stg, int lane, const uint32_t (&r)[32]) {
  uint4* s = reinterpret_cast<uint4*>(stg) + lane * 8;
#pragma unroll
  for (int v = 0; v < 8; ++v)
    s[v ^ (lane & 7)] = make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
}
// A 32 x 32 piece transposed: its column j becomes row j of the staged tile, 32 lanes side by
// side (64-byte swizzle for bf16, 128-byte for fp32).
template <bool F32>
__device__ __forceinline__ void stage_transposed(unsigned char* stg, int lane,
                                                 const uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (F32)
      *reinterpret_cast<uint32_t*>(stg + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) +
                                   (lane & 3) * 4) = r[j];
    else
      *reinterpret_cast<bf*>(stg + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) +
                             (lane & 7) * 2) = __float2bfloat16_rn(__uint_as_float(r[j]));
  }
}
// Shared -> global tile addition in fp32 (every output element has one writer per call).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::
          "l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y)
      : "memory");
}
// The warp's earlier stores have read its staging bytes.
__device__ __forceinline__ void staging_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}
__device__ __forceinline__ void staging_ready() {
  fence_proxy_async_smem();
  __syncwarp();
}

// A CTA's 128 rows of A.  K-major: one box of 128 rows x 64 k; MN-major: two blocks of 64
// columns x 64 k.
template <int MN>
__device__ __forceinline__ void load_a(const PairMaps& m, const CUtensorMap* map, void* s, int row,
                                       int k, uint64_t* bar) {
  if (!MN) {
    pair_load_2d(s, map, k, row, bar);
  } else if (m.a3) {
    pair_load_3d(s, map, 0, k, row >> 6, bar);
  } else {
    pair_load_2d(s, map, row, k, bar);
    pair_load_2d(static_cast<unsigned char*>(s) + 8192, map, row + 64, k, bar);
  }
}
// `rows` <= 128 rows of B from `row`.  K-major: one box for 128 rows (a box of 32 at a time cost
// 10% there), else as many low ones as the tile needs.  MN-major as A; blocks start at multiples
// of 64 only where tiles do, so a narrow tile's blocks come one by one from the flat map.
constexpr int kLowBox = 32;
template <int MN>
__device__ __forceinline__ uint32_t b_bytes(int rows) {
  const int box = MN ? 64 : kLowBox;
  return (uint32_t)((rows + box - 1) / box * box * kBK * 2);
}
template <int MN>
__device__ __forceinline__ void load_b(const PairMaps& m,
                                       int which, void* s, int row, int rows, int k,
                                       uint64_t* bar) {
  const CUtensorMap* low = &m.low[which];
  unsigned char* d = static_cast<unsigned char*>(s);
  if (rows == kPairHalf && (!MN || m.b3[which])) {
    if (MN)
      pair_load_3d(s, &m.b[which], 0, k, row >> 6, bar);
    else
      pair_load_2d(s, &m.b[which], k, row, bar);
    return;
  }
  constexpr int box = MN ? 64 : kLowBox;
  for (int r = 0; r < rows; r += box, d += box * kBK * 2) {
    if (MN)
      pair_load_2d(d, low, row + r, k, bar);
    else
      pair_load_2d(d, low, k, row + r, bar);
  }
}

struct NoEarly {};

// Three staged pieces of 32 columns to the three outputs.
__device__ __forceinline__ void store3(const PairEpi& e, int c, int y, int cols) {
  staging_ready();
  if (e.lane == 0 && c < cols) {
#pragma unroll
    for (int i = 0; i < 3; ++i) tma_store_2d(&e.maps->o[i], e.stg + 2048 * i, c, y);
    bulk_commit();
  }
  __syncwarp();
}

// 32 bytes of global memory that nothing else reads, one whole sector (ALIGNED32), or as two
// 16-byte loads.
__device__ __forceinline__ void load32(const uint4* p, bool aligned32, uint4& a, uint4& b) {
  if (aligned32) {
    asm volatile(
        "ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
        : "l"(p));
  } else {
    a = __ldg(p);
    b = __ldg(p + 1);
  }
}

// ------------------------------------------------------------------ gate
template <int ACT, bool KEEP, bool CKPT8>
struct GateProb {
  static constexpr int kAMN = 0, kBMN = 0;
  static constexpr int kStg = KEEP && !CKPT8 ? 3 * 2048 : 4096;
  struct Params {
    int* status;
    PairWalk walk;  // a tile of width w holds w / 2 columns of g and the same of u
    int64_t N, runs;
    int f, nk;
    int8_t *cg, *cu;
    float *sg, *su;
  };
  struct Tile {
    int m0, f0, w;
  };
  using Early = NoEarly;
  __device__ static void prefetch(const Params&, const Tile&, const PairEpi&, Early&) {}
  __device__ static int num_tiles(const Params& P) { return P.walk.total; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    const WalkTile t = walk_tile(P.walk, u);
    return Tile{t.mt * kPairM, t.n0 / 2, t.w};
  }
  __device__ static uint32_t load_bytes(const PairMaps&, const Tile& t) {
    return kPairStage / 2 + b_bytes<0>(t.w / 2);
  }
  __device__ static void load(const Params&, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    load_a<0>(m, &m.a[0], sa, t.m0 + rank * kPairHalf, kb * kBK, bar);
    load_b<0>(m, rank, sb, t.f0, t.w / 2, kb * kBK, bar);
  }
  __device__ static void keep8(const Params& P, const uint32_t (&r)[32], int64_t run_idx,
                               int8_t* codes, float* scale) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) top = max(top, r[j] & 0x7fffffffu);
    const CkptScale s = ckpt_scale<false>(top);
    float a[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) a[j] = __uint_as_float(r[j]);
    uint32_t w[8];
    ckpt_codes<false>(a, s, w);
    uint4* d = reinterpret_cast<uint4*>(codes + run_idx * kCkptRun);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    scale[run_idx] = s.scale;
  }
  __device__ static void epilogue(const Params& P, const Tile& t, const PairEpi& e, const Early&) {
    const int y0 = t.m0 + e.row0;
    const int64_t row = (int64_t)y0 + e.lane;
    if (y0 >= P.N) return;  // warp-uniform
    for (int piece = e.set; piece * 128 < t.w; piece += 2) {
      const int c0 = t.f0 + piece * 64;
      if (c0 >= P.f) break;  // warp-uniform
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t g[32], u[32], p[16];
        tmem_ld32(e.taddr + piece * 64 + half * 32, g);
        tmem_ld32(e.taddr + t.w / 2 + piece * 64 + half * 32, u);
        tmem_wait_ld(g);
        tmem_wait_ld(u);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          p[j] = pack_bf16(
              act_fast<ACT>(__uint_as_float(g[2 * j])) * __uint_as_float(u[2 * j]),
              act_fast<ACT>(__uint_as_float(g[2 * j + 1])) * __uint_as_float(u[2 * j + 1]));
        if (KEEP && !CKPT8) {
          staging_free(e.lane);
          stage_bf16_32(e.stg, e.lane, p);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            p[j] = pack_bf16(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
          stage_bf16_32(e.stg + 2048, e.lane, p);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            p[j] = pack_bf16(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
          stage_bf16_32(e.stg + 4096, e.lane, p);
          store3(e, c0 + half * 32, y0, P.f);
        } else {
          if (half == 0) staging_free(e.lane);
          stage_bf16(e.stg, e.lane, half, p);
        }
        if (KEEP && CKPT8 && row < P.N && c0 + half * 32 < P.f) {
          const int64_t run = row * P.runs + (c0 >> 5) + half;
          keep8(P, g, run, P.cg, P.sg);
          keep8(P, u, run, P.cu, P.su);
        }
      }
      if (KEEP && !CKPT8) continue;
      staging_ready();
      if (e.lane == 0) {
        tma_store_2d(&e.maps->o[0], e.stg, c0, y0);
        bulk_commit();
      }
      __syncwarp();
    }
  }
};

// ------------------------------------------------------------------ dh
// The accumulator is dh; the thread's row of the kept projections is requested one piece ahead.
template <int ACT, bool CKPT8>
struct GateGradProb {
  static constexpr int kAMN = 0, kBMN = 1;
  static constexpr int kStg = 3 * 2048;
  struct Params {
    int* status;
    PairWalk walk;
    int64_t N, runs;
    int f, nk;
    bool aligned32;     // rows of g and u start on 32-byte boundaries
    const void *g, *u;  // bf16 values or int8 codes
    const float *sg, *su;
  };
  struct Tile {
    int m0, n0, w;
  };
  struct Early {
    uint4 g[CKPT8 ? 2 : 4], u[CKPT8 ? 2 : 4];
    float sg, su;
  };
  __device__ static int num_tiles(const Params& P) { return P.walk.total; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    const WalkTile t = walk_tile(P.walk, u);
    return Tile{t.mt * kPairM, t.n0, t.w};
  }
  __device__ static uint32_t load_bytes(const PairMaps&, const Tile& t) {
    return kPairStage / 2 + b_bytes<1>(t.w / 2);
  }
  __device__ static void load(const Params&, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    load_a<0>(m, &m.a[0], sa, t.m0 + rank * kPairHalf, kb * kBK, bar);
    load_b<1>(m, 0, sb, t.n0 + rank * (t.w / 2), t.w / 2, kb * kBK, bar);
  }
  __device__ static void fetch(const Params& P, int64_t row, int c0, Early& k) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool in = row < P.N && c0 < P.f;
    const uint4 *g = static_cast<const uint4*>(P.g), *u = static_cast<const uint4*>(P.u);
    if (CKPT8) {
      const int64_t run = in ? row * P.runs + (c0 >> 5) : 0;
      k.g[0] = k.g[1] = k.u[0] = k.u[1] = zero;
      k.sg = k.su = 0.f;
      if (in) {
        load32(g + run * 2, P.aligned32, k.g[0], k.g[1]);
        load32(u + run * 2, P.aligned32, k.u[0], k.u[1]);
        k.sg = __ldg(P.sg + run);
        k.su = __ldg(P.su + run);
      }
    } else {
      const int64_t at = in ? (row * P.f + c0) >> 3 : 0;
#pragma unroll
      for (int v = 0; v < 4; v += 2) {
        k.g[v] = k.g[v + 1] = k.u[v] = k.u[v + 1] = zero;
        if (in && c0 + 8 * v + 8 < P.f) {
          load32(g + at + v, P.aligned32, k.g[v], k.g[v + 1]);
          load32(u + at + v, P.aligned32, k.u[v], k.u[v + 1]);
        } else if (in && c0 + 8 * v < P.f) {  // the row ends after 8 columns
          k.g[v] = __ldg(g + at + v);
          k.u[v] = __ldg(u + at + v);
        }
      }
    }
  }
  __device__ static void prefetch(const Params& P, const Tile& t, const PairEpi& e, Early& k) {
    fetch(P, (int64_t)t.m0 + e.row0 + e.lane, t.n0 + e.set * 64, k);
  }
  // Columns 4j .. 4j + 3 of the piece.
  __device__ static void four_of(const uint4* q, float scale, int j, float (&v)[4]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(q);
    if (CKPT8) {
      ckpt_floats4(w[j], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= scale;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[2 * i] = __uint_as_float(w[2 * j + i] << 16);
        v[2 * i + 1] = __uint_as_float(w[2 * j + i] & 0xffff0000u);
      }
    }
  }
  __device__ static void epilogue(const Params& P, const Tile& t, const PairEpi& e, Early& k) {
    const int y0 = t.m0 + e.row0;
    const int64_t row = (int64_t)y0 + e.lane;
    if (y0 >= P.N) return;  // warp-uniform
    for (int piece = e.set; piece * 64 < t.w; piece += 2) {
      const int c0 = t.n0 + piece * 64;
      if (c0 >= P.f) break;  // warp-uniform
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t d[32], ph[16], pg[16], pu[16];
        tmem_ld32(e.taddr + piece * 64 + half * 32, d);
        const Early now = k;
        // the next half, or the first of the set's next piece
        if (half == 0)
          fetch(P, row, c0 + 32, k);
        else if ((piece + 2) * 64 < t.w)
          fetch(P, row, c0 + 128, k);
        tmem_wait_ld(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float g[4], u[4], hh[4], dg[4], du[4];
          four_of(now.g, now.sg, j, g);
          four_of(now.u, now.su, j, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float dh = __uint_as_float(d[4 * j + i]);
            float a, slope;
            act_and_slope_fast<ACT>(g[i], &a, &slope);
            hh[i] = a * u[i];
            dg[i] = dh * u[i] * slope;
            du[i] = dh * a;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ph[2 * j + i] = pack_bf16(hh[2 * i], hh[2 * i + 1]);
            pg[2 * j + i] = pack_bf16(dg[2 * i], dg[2 * i + 1]);
            pu[2 * j + i] = pack_bf16(du[2 * i], du[2 * i + 1]);
          }
        }
        staging_free(e.lane);
        stage_bf16_32(e.stg, e.lane, ph);
        stage_bf16_32(e.stg + 2048, e.lane, pg);
        stage_bf16_32(e.stg + 4096, e.lane, pu);
        store3(e, c0 + half * 32, y0, P.f);
      }
    }
  }
};

// ------------------------------------------------------------------ plain products
// A warp's 32 x 64 accumulator columns to the output: bf16 rows in one store, fp32 (ADD: +=) or
// a transposed piece in two of 32 columns.
template <bool ADD>
__device__ __forceinline__ void write_piece(const CUtensorMap* out, const PairEpi& e,
                                            uint32_t taddr, bool trans, int c0, int y0, int cols) {
  constexpr int kHalf = ADD ? 4096 : 2048;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t r[32];
    tmem_ld32(taddr + half * 32, r);
    tmem_wait_ld(r);
    if (half == 0) staging_free(e.lane);
    if (trans) {
      stage_transposed<ADD>(e.stg + half * kHalf, e.lane, r);
    } else if (ADD) {
      stage_f32(e.stg + half * kHalf, e.lane, r);
    } else {
      uint32_t p[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        p[j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      stage_bf16(e.stg, e.lane, half, p);
    }
  }
  staging_ready();
  if (e.lane == 0) {
    for (int half = 0; half < (trans || ADD ? 2 : 1); ++half) {
      const int c = c0 + half * 32;
      if (c >= cols) break;
      const int x = trans ? y0 : c, y = trans ? c : y0;
      if (ADD)
        tma_add_2d(out, e.stg + half * kHalf, x, y);
      else
        tma_store_2d(out, e.stg + half * kHalf, x, y);
    }
    bulk_commit();
  }
  __syncwarp();
}

// Token rows: out[rows x cols] = A[0] B[0]^T, and for k-blocks from nk0 on A[1] B[1]^T into the
// same accumulator (y, dx).  SPLIT: so few tiles that k is cut into parts, which are row tiles of
// their own (part i: k-blocks [i * nk, +nk), past the end zeros) and write fp32 partial
// results [part][rows][cols]; sum_parts_kernel adds them in order.
template <int BMN, bool SPLIT>
struct RowsProb {
  static constexpr int kAMN = 0, kBMN = BMN;
  static constexpr int kStg = SPLIT ? 2 * 4096 : 4096;
  struct Params {
    int* status;
    PairWalk walk;
    int64_t rows;
    int cols, m_each, nk, nk0;
  };
  struct Tile {
    int m0, n0, w, part;
  };
  using Early = NoEarly;
  __device__ static void prefetch(const Params&, const Tile&, const PairEpi&, Early&) {}
  __device__ static int num_tiles(const Params& P) { return P.walk.total; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    const WalkTile t = walk_tile(P.walk, u);
    const int part = SPLIT ? t.mt / P.m_each : 0;
    return Tile{(t.mt - part * P.m_each) * kPairM, t.n0, t.w, part};
  }
  __device__ static uint32_t load_bytes(const PairMaps&, const Tile& t) {
    return kPairStage / 2 + b_bytes<BMN>(t.w / 2);
  }
  __device__ static void load(const Params& P, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    if (SPLIT) kb += t.part * P.nk;
    const int second = kb >= P.nk0;
    const int k = (second ? kb - P.nk0 : kb) * kBK;
    load_a<0>(m, &m.a[second], sa, t.m0 + rank * kPairHalf, k, bar);
    load_b<BMN>(m, second, sb, t.n0 + rank * (t.w / 2), t.w / 2, k, bar);
  }
  __device__ static void epilogue(const Params& P, const Tile& t, const PairEpi& e, const Early&) {
    const int y0 = t.m0 + e.row0;
    if (y0 >= P.rows) return;  // warp-uniform
    for (int piece = e.set; piece * 64 < t.w; piece += 2) {
      const int c0 = t.n0 + piece * 64;
      if (c0 >= P.cols) break;  // warp-uniform
      if (!SPLIT) {
        write_piece<false>(&e.maps->o[0], e, e.taddr + piece * 64, false, c0, y0, P.cols);
        continue;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t r[32];
        tmem_ld32(e.taddr + piece * 64 + half * 32, r);
        tmem_wait_ld(r);
        if (half == 0) staging_free(e.lane);
        stage_f32(e.stg + half * 4096, e.lane, r);
      }
      staging_ready();
      if (e.lane == 0) {
        for (int half = 0; half < 2 && c0 + half * 32 < P.cols; ++half)
          tma_store_3d(&e.maps->o[0], e.stg + half * 4096, c0 + half * 32, y0, t.part);
        bulk_commit();
      }
      __syncwarp();
    }
  }
};

// out = sum of the parts in order, rounded to bf16.  A thread has 8 columns.
__global__ void __launch_bounds__(256) sum_parts_kernel(int64_t chunks, int64_t part_stride,
                                                        int parts, const float* src, bf* dst) {
  grid_dependency_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= chunks) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; ++p) {
    const float4* s = reinterpret_cast<const float4*>(src + p * part_stride + i * 8);
    const float4 a = s[0], b = s[1];
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
  reinterpret_cast<uint4*>(dst)[i] =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7]));
}

// Weight gradients: D[d_ff rows x cols] = A^T B over the tokens, up to three kinds of row tiles:
// dg^T x (dWg), du^T x (dWu) and h^T dy, which is stored transposed (dWd [d_out][d_ff]): d_ff is
// what fills row tiles in all of them.  One launch for all of a width, so their last tiles share
// a round.  ADD: fp32, +=; else bf16, overwritten.
template <bool ADD>
struct WeightProb {
  static constexpr int kAMN = 1, kBMN = 1;
  static constexpr int kStg = ADD ? 2 * 4096 : 4096;
  struct Params {
    int* status;
    PairWalk walk;
    int rows, cols, m_each, nk;
    int which[3];  // of the kinds present, in order: 0 dWg, 1 dWu, 2 dWd
  };
  struct Tile {
    int m0, n0, w, which;
  };
  using Early = NoEarly;
  __device__ static void prefetch(const Params&, const Tile&, const PairEpi&, Early&) {}
  __device__ static int num_tiles(const Params& P) { return P.walk.total; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    const WalkTile t = walk_tile(P.walk, u);
    const int kind = t.mt / P.m_each;
    return Tile{(t.mt - kind * P.m_each) * kPairM, t.n0, t.w,
                kind == 0 ? P.which[0] : kind == 1 ? P.which[1] : P.which[2]};
  }
  __device__ static uint32_t load_bytes(const PairMaps&, const Tile& t) {
    return kPairStage / 2 + b_bytes<1>(t.w / 2);
  }
  __device__ static void load(const Params&, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    load_a<1>(m, &m.a[t.which], sa, t.m0 + rank * kPairHalf, kb * kBK, bar);
    load_b<1>(m, t.which == 2, sb, t.n0 + rank * (t.w / 2), t.w / 2, kb * kBK, bar);
  }
  __device__ static void epilogue(const Params& P, const Tile& t, const PairEpi& e, const Early&) {
    const int y0 = t.m0 + e.row0;
    if (y0 >= P.rows) return;  // warp-uniform
    for (int piece = e.set; piece * 64 < t.w; piece += 2) {
      const int c0 = t.n0 + piece * 64;
      if (c0 >= P.cols) break;  // warp-uniform
      write_piece<ADD>(&e.maps->o[t.which], e, e.taddr + piece * 64, t.which == 2, c0, y0, P.cols);
    }
  }
};

// ------------------------------------------------------------------ host
template <class Prob>
cudaError_t launch_pair(const FfnPlan& p, const PairMaps& maps, const typename Prob::Params& P,
                        int64_t tiles, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set (64 at most)
  const uint64_t bit = (uint64_t)1 << p.dev;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        tc_pair_kernel<Prob>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)pair_smem<Prob>());
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  if (tiles <= 0) return cudaSuccess;
  const int pairs = (int)std::min<int64_t>(tiles, p.sm_count / 2);
  tc_pair_kernel<Prob><<<2 * pairs, kPairThreads, pair_smem<Prob>(), st>>>(maps, P);
  PKM_COUNT(1);
  return cudaGetLastError();
}

// [rows][cols] bf16 as an operand whose K runs along the row ...
bool map_kmajor(CUtensorMap* m, const void* base, int64_t rows, int cols, int box) {
  return make_tmap_bf16_2d(m, base, cols, rows, (uint64_t)cols * 2, kBK, box);
}
// ... or down the rows: flat (64 columns x 64 k), or in blocks of 64 columns, two to a load.
bool map_mnmajor(CUtensorMap* m, const void* base, int64_t rows, int cols) {
  return make_tmap_bf16_2d(m, base, cols, rows, (uint64_t)cols * 2, 64, kBK);
}
bool map_blocks(CUtensorMap* m, const void* base, int64_t rows, int cols) {
  const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)cols / 64};
  const uint64_t strides[2] = {(uint64_t)cols * 2, 128};
  const uint32_t box[3] = {64, kBK, 2};
  return make_tmap_store(m, false, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_a_mn(PairMaps* m, int i, const void* base, int64_t rows, int cols) {
  m->a3 = cols % 64 == 0;
  return m->a3 ? map_blocks(&m->a[i], base, rows, cols) : map_mnmajor(&m->a[i], base, rows, cols);
}
bool map_b_mn(PairMaps* m, int i, const void* base, int64_t rows, int cols) {
  m->b3[i] = cols % 64 == 0;
  return map_mnmajor(&m->low[i], base, rows, cols) &&
         (!m->b3[i] || map_blocks(&m->b[i], base, rows, cols));
}
bool map_b_k(PairMaps* m, int i, const void* base, int64_t rows, int cols) {
  return map_kmajor(&m->b[i], base, rows, cols, kPairHalf) &&
         map_kmajor(&m->low[i], base, rows, cols, kLowBox);
}
// An output in boxes of 32 rows x `wide` columns (32 fp32, 64 bf16, or 32 bf16 transposed).
bool map_out(CUtensorMap* m, bool fp32, void* base, int64_t rows, int cols, uint32_t wide) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * (fp32 ? 4 : 2)};
  const uint32_t box[2] = {wide, 32};
  return make_tmap_store(m, fp32, 2, base, dims, strides, box,
                         wide * (fp32 ? 4 : 2) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                      : CU_TENSOR_MAP_SWIZZLE_64B);
}

int64_t tiles_of(int64_t rows, int w) { return (rows + w - 1) / w; }

// Time of a tile of width w in units of the products of one column: the products themselves, or
// the operand bytes of a k-block (A's 128 rows and B's w / 2 per CTA at the rate at which 128
// rows of B would just keep up), whichever is longer.
int tile_cost(int w) { return std::max(w, 128 + w / 2); }

// The rounds that are left after the whole ones: n1 tiles of cost c1, then n2 of cost c2, as
// tile_of_round deals them out.  The longest share is that of the first or the last pair or of one
// beside the place where the tiles change or end.
int64_t tail_cost(int64_t n1, int c1, int64_t n2, int c2, int pairs) {
  const int64_t n = n1 + n2;
  const auto share = [&](int64_t p) {
    int64_t sum = 0;
    for (int64_t r = 0; r * pairs < n; ++r) {
      const int64_t u = r * pairs + (r & 1 ? pairs - 1 - p : p);
      if (u < n) sum += u < n1 ? c1 : c2;
    }
    return sum;
  };
  int64_t most = std::max(share(0), share(pairs - 1));
  for (const int64_t end : {n1, n})
    for (int64_t u = std::max<int64_t>(end - 1, 0); u <= end; ++u) {
      const int64_t i = u % pairs;
      most = std::max(most, std::max(share(i), share(pairs - 1 - i)));
    }
  return most;
}

// The walk of least cost over tile widths and cuts of the remaining wide tiles.  Widths below
// 192 lose more to operand bytes than they gain in balance; every width is a multiple of the
// epilogue's pieces (step: 64, for the gate 128, 64 of each projection).
PairWalk make_walk(int64_t m_tiles, int64_t cols, int pairs, int step) {
  PairWalk best{};
  int64_t least = -1;
  for (int w = 256; w >= 192; w -= 64) {
    if (w % step) continue;
    PairWalk k{};
    k.m_tiles = (int)m_tiles;
    k.width = w;
    k.full_n = (int)(cols / w);
    k.rest = (int)((cols % w + step - 1) / step * step);
    const int64_t wide = m_tiles * k.full_n;
    k.whole = (int)(wide / pairs * pairs);
    for (int s = 1; s <= 4; s *= 2) {
      if (w % (s * step)) continue;
      k.split = s;
      const int64_t left = (wide - k.whole) * s, narrow = k.rest ? m_tiles : 0;
      k.total = (int)(k.whole + left + narrow);
      const int64_t cost = (int64_t)k.whole / pairs * tile_cost(w) +
                           tail_cost(left, tile_cost(w / s), narrow, tile_cost(k.rest), pairs);
      if (least < 0 || cost < least) {
        least = cost;
        best = k;
      }
    }
  }
  return best;
}

#define FFN_TRY(...)                  \
  do {                                \
    const cudaError_t _e = (__VA_ARGS__); \
    if (_e != cudaSuccess) return _e; \
  } while (0)
#define FFN_MAP(expr)                            \
  do {                                           \
    if (!(expr)) return cudaErrorInvalidValue;   \
  } while (0)

template <int ACT, bool KEEP, bool CKPT8>
cudaError_t run_gate(const FfnPlan& p, const PairMaps& m, const pkm_ffn_saved* s, cudaStream_t st) {
  using G = GateProb<ACT, KEEP, CKPT8>;
  typename G::Params P{};
  P.status = p.status;
  P.N = p.N;
  P.runs = p.runs;
  P.f = p.d_ff;
  P.walk = make_walk(tiles_of(p.N, kPairM), 2 * (int64_t)p.d_ff, p.sm_count / 2, 128);
  P.nk = (int)tiles_of(p.d_in, kBK);
  if (KEEP && CKPT8) {
    P.cg = static_cast<int8_t*>(s->g);
    P.cu = static_cast<int8_t*>(s->u);
    P.sg = s->g_scale;
    P.su = s->u_scale;
  }
  return launch_pair<G>(p, m, P, P.walk.total, st);
}

template <int ACT, bool CKPT8>
cudaError_t run_gate_grad(const FfnPlan& p, const PairMaps& m, const pkm_ffn_saved& s,
                          cudaStream_t st) {
  using G = GateGradProb<ACT, CKPT8>;
  typename G::Params P{};
  P.status = p.status;
  P.N = p.N;
  P.runs = p.runs;
  P.f = p.d_ff;
  P.walk = make_walk(tiles_of(p.N, kPairM), p.d_ff, p.sm_count / 2, 64);
  P.nk = (int)tiles_of(p.d_out, kBK);
  P.g = s.g;
  P.u = s.u;
  P.aligned32 = (((uintptr_t)s.g | (uintptr_t)s.u) & 31) == 0 && (CKPT8 || p.d_ff % 16 == 0);
  P.sg = s.g_scale;
  P.su = s.u_scale;
  return launch_pair<G>(p, m, P, P.walk.total, st);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Parts of k for a product of few tiles: as many as leave a pair of SMs to each and 16 k-blocks
// to every part.  (Planned for 74 pairs wherever it runs, so that the workspace depends on the
// sizes alone.)  Backward of 64 tokens, 1600 x 6400 x 1600: 66 us, in one part 116; forward 30
// against 52; of 1024 tokens, 1024 x 4096 x 1024: 72 against 98.
int parts_of(int64_t rows, int cols, int64_t nk) {
  constexpr int kPairs = 74, kMostParts = 8;
  const int64_t tiles = tiles_of(rows, kPairM) * tiles_of(cols, 256);
  if (2 * tiles > kPairs || nk < 32) return 1;
  return (int)std::min<int64_t>({kMostParts, kPairs / tiles, nk / 16});
}
size_t part_bytes(int64_t rows, int cols, int64_t nk) {
  const int parts = parts_of(rows, cols, nk);
  return parts > 1 ? align256((size_t)parts * rows * cols * 4) : 0;
}

// out [p.N][cols] bf16 over k of length K, once or with a second pair of operands after the
// first.  scratch: part_bytes.
template <int BMN>
cudaError_t run_rows(const FfnPlan& p, PairMaps& m, void* out, int cols, int64_t K, bool twice,
                     void* scratch, cudaStream_t st) {
  const int64_t nk0 = tiles_of(K, kBK), nk = twice ? 2 * nk0 : nk0;
  const int parts = parts_of(p.N, cols, nk);
  const int m_each = (int)tiles_of(p.N, kPairM);
  const auto fill = [&](auto& P) {
    P.status = p.status;
    P.rows = p.N;
    P.cols = cols;
    P.m_each = m_each;
    P.walk = make_walk((int64_t)m_each * parts, cols, p.sm_count / 2, 64);
    P.nk0 = twice ? (int)nk0 : INT32_MAX;  // without a second pair nothing may read its maps
    P.nk = (int)tiles_of(nk, parts);
  };
  if (parts == 1) {
    using G = RowsProb<BMN, false>;
    typename G::Params P{};
    fill(P);
    FFN_MAP(map_out(&m.o[0], false, out, p.N, cols, 64));
    return launch_pair<G>(p, m, P, P.walk.total, st);
  }
  using G = RowsProb<BMN, true>;
  typename G::Params P{};
  fill(P);
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)p.N, (uint64_t)parts};
  const uint64_t strides[2] = {(uint64_t)cols * 4, (uint64_t)cols * p.N * 4};
  const uint32_t box[3] = {32, 32, 1};
  FFN_MAP(make_tmap_store(&m.o[0], true, 3, scratch, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B));
  FFN_TRY(launch_pair<G>(p, m, P, P.walk.total, st));
  const int64_t chunks = p.N * cols / 8;
  const cudaError_t e = launch_dependent(
      sum_parts_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, st, chunks,
      p.N * cols, parts, static_cast<const float*>(scratch), static_cast<bf*>(out));
  PKM_COUNT(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The weight gradients among `kinds` (of which[0 ..]); operands and outputs are mapped.
template <bool ADD>
cudaError_t run_weights(const FfnPlan& p, const PairMaps& m, const int* which, int kinds, int cols,
                        cudaStream_t st) {
  using G = WeightProb<ADD>;
  typename G::Params P{};
  P.status = p.status;
  P.rows = p.d_ff;
  P.cols = cols;
  P.m_each = (int)tiles_of(p.d_ff, kPairM);
  P.walk = make_walk((int64_t)P.m_each * kinds, cols, p.sm_count / 2, 64);
  P.nk = (int)tiles_of(p.N, kBK);
  for (int i = 0; i < kinds; ++i) P.which[i] = which[i];
  return launch_pair<G>(p, m, P, P.walk.total, st);
}

}  // namespace

// Forward: h.  Backward: h, dg, du.  All [N][d_ff] bf16; then the parts of y or dx.
size_t ffn_tc_workspace(const FfnPlan& p, bool backward) {
  const size_t each = align256((size_t)p.N * p.d_ff * 2);
  const int64_t nk = tiles_of(p.d_ff, kBK);
  return backward ? 3 * each + part_bytes(p.N, p.d_in, 2 * nk) : each + part_bytes(p.N, p.d_out, nk);
}

cudaError_t launch_ffn_fwd_tc(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                              const void* Wd, void* y, const pkm_ffn_saved* s, void* ws,
                              cudaStream_t st) {
  PairMaps m{};
  FFN_MAP(map_kmajor(&m.a[0], x, p.N, p.d_in, kPairHalf));
  FFN_MAP(map_b_k(&m, 0, Wg, p.d_ff, p.d_in));
  FFN_MAP(map_b_k(&m, 1, Wu, p.d_ff, p.d_in));
  const bool three = s && !p.ckpt8;
  FFN_MAP(map_out(&m.o[0], false, ws, p.N, p.d_ff, three ? 32 : 64));
  if (three) {
    FFN_MAP(map_out(&m.o[1], false, s->g, p.N, p.d_ff, 32));
    FFN_MAP(map_out(&m.o[2], false, s->u, p.N, p.d_ff, 32));
  }
#define FFN_GATE(ACT)                                                              \
  FFN_TRY(!s ? run_gate<ACT, false, false>(p, m, s, st)                            \
             : p.ckpt8 ? run_gate<ACT, true, true>(p, m, s, st)                    \
                       : run_gate<ACT, true, false>(p, m, s, st))
  if (p.act == PKM_ACT_GELU) FFN_GATE(PKM_ACT_GELU); else FFN_GATE(PKM_ACT_SILU);
#undef FFN_GATE
  PairMaps d{};
  FFN_MAP(map_kmajor(&d.a[0], ws, p.N, p.d_ff, kPairHalf));
  FFN_MAP(map_b_k(&d, 0, Wd, p.d_out, p.d_ff));
  char* scratch = static_cast<char*>(ws) + align256((size_t)p.N * p.d_ff * 2);
  return run_rows<0>(p, d, y, p.d_out, p.d_ff, false, scratch, st);
}

cudaError_t launch_ffn_bwd_tc(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                              const void* Wd, const pkm_ffn_saved& s, const void* dy, void* dx,
                              void* dWg, void* dWu, void* dWd, void* ws, cudaStream_t st) {
  if (!dx && !dWg && !dWu && !dWd) return cudaSuccess;
  const size_t each = align256((size_t)p.N * p.d_ff * 2);
  char* h = static_cast<char*>(ws);
  char* dg = h + each;
  char* du = dg + each;
  PairMaps m{};
  FFN_MAP(map_kmajor(&m.a[0], dy, p.N, p.d_out, kPairHalf));
  FFN_MAP(map_b_mn(&m, 0, Wd, p.d_out, p.d_ff));
  FFN_MAP(map_out(&m.o[0], false, h, p.N, p.d_ff, 32));
  FFN_MAP(map_out(&m.o[1], false, dg, p.N, p.d_ff, 32));
  FFN_MAP(map_out(&m.o[2], false, du, p.N, p.d_ff, 32));
#define FFN_GRAD(ACT)                                              \
  FFN_TRY(p.ckpt8 ? run_gate_grad<ACT, true>(p, m, s, st)          \
                  : run_gate_grad<ACT, false>(p, m, s, st))
  if (p.act == PKM_ACT_GELU) FFN_GRAD(PKM_ACT_GELU); else FFN_GRAD(PKM_ACT_SILU);
#undef FFN_GRAD
  if (dWg || dWu || dWd) {
    const bool add = !p.grad_bf16;
    PairMaps w{};
    int which[3], kinds = 0;
    if (dWg) {
      FFN_MAP(map_a_mn(&w, 0, dg, p.N, p.d_ff));
      FFN_MAP(map_out(&w.o[0], add, dWg, p.d_ff, p.d_in, add ? 32 : 64));
      which[kinds++] = 0;
    }
    if (dWu) {
      FFN_MAP(map_a_mn(&w, 1, du, p.N, p.d_ff));
      FFN_MAP(map_out(&w.o[1], add, dWu, p.d_ff, p.d_in, add ? 32 : 64));
      which[kinds++] = 1;
    }
    if (kinds) FFN_MAP(map_b_mn(&w, 0, x, p.N, p.d_in));
    if (dWd) {
      FFN_MAP(map_a_mn(&w, 2, h, p.N, p.d_ff));
      FFN_MAP(map_b_mn(&w, 1, dy, p.N, p.d_out));
      FFN_MAP(map_out(&w.o[2], add, dWd, p.d_out, p.d_ff, 32));
      which[kinds++] = 2;
    }
    const auto run = add ? run_weights<true> : run_weights<false>;
    if (p.d_in == p.d_out || kinds == 1 || !dWd) {
      FFN_TRY(run(p, w, which, kinds, dWd ? p.d_out : p.d_in, st));
    } else {
      FFN_TRY(run(p, w, which, kinds - 1, p.d_in, st));
      FFN_TRY(run(p, w, which + kinds - 1, 1, p.d_out, st));
    }
  }
  if (dx) {
    PairMaps w{};
    FFN_MAP(map_kmajor(&w.a[0], dg, p.N, p.d_ff, kPairHalf));
    FFN_MAP(map_kmajor(&w.a[1], du, p.N, p.d_ff, kPairHalf));
    FFN_MAP(map_b_mn(&w, 0, Wg, p.d_ff, p.d_in));
    FFN_MAP(map_b_mn(&w, 1, Wu, p.d_ff, p.d_in));
    FFN_TRY(run_rows<1>(p, w, dx, p.d_in, p.d_ff, true, du + each, st));
  }
  return cudaSuccess;
}

}  // namespace pkm
