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
// Fast forms: exp and the quotient are good to ~2^-21, far inside the bf16 rounding that
// every result of them gets.
template <int ACT>
__device__ __forceinline__ float act_fast(float v) {
  if (ACT == PKM_ACT_GELU) return act_fn<ACT>(v);
  return __fdividef(v, 1.f + __expf(-v));
}
template <int ACT>
__device__ __forceinline__ void act_and_slope_fast(float v, float* a, float* slope) {
  if (ACT == PKM_ACT_GELU) return act_and_slope<ACT>(v, a, slope);
  const float s = __fdividef(1.f, 1.f + __expf(-v));
  *a = v * s;
  *slope = s * fmaf(v, 1.f - s, 1.f);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A warp's 32 x 32 bf16 piece into a 2 KiB staging tile (row = lane, 64-byte swizzle: 16-byte
// chunk v of row r sits at chunk v ^ ((r >> 1) & 3)).
__device__ __forceinline__ void stage_bf16(unsigned char* stg, int lane, const uint32_t (&p)[16]) {
  uint4* s = reinterpret_cast<uint4*>(stg) + lane * 4;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    s[v ^ ((lane >> 1) & 3)] = make_uint4(p[4 * v], p[4 * v + 1], p[4 * v + 2], p[4 * v + 3]);
}
__device__ __forceinline__ void stage_f32(unsigned char* stg, int lane, const uint32_t (&r)[32]) {
  uint4* s = reinterpret_cast<uint4*>(stg) + lane * 8;
#pragma unroll
  for (int v = 0; v < 8; ++v)
    s[v ^ (lane & 7)] = make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
}
// Shared -> global tile addition in fp32 (every output element has one writer per call).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::
          "l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y)
      : "memory");
}
// The staging bytes may be written again: the warp's earlier stores have read them.
__device__ __forceinline__ void staging_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}
__device__ __forceinline__ void staging_ready() {
  fence_proxy_async_smem();
  __syncwarp();
}

// Tiles walk the output in bands of kBand row tiles, all column tiles of a band before the
// next, so the tiles in flight at one time share rows of A and of B in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void band_tile(int u, int m_tiles, int n_tiles, int* mt, int* nt) {
  const int per = kBand * n_tiles, b = u / per, r = u % per;
  const int rows = min(kBand, m_tiles - b * kBand);
  *mt = b * kBand + r % rows;
  *nt = r / rows;
}

// K-major operand half: 128 rows from `row`; MN-major: two 64 x 64 boxes from column `row`.
template <int MN>
__device__ __forceinline__ void load_half(const CUtensorMap* map, void* s, int row, int k,
                                          uint64_t* bar) {
  if (MN) {
    pair_load_2d(s, map, row, k, bar);
    pair_load_2d(static_cast<unsigned char*>(s) + 8192, map, row + 64, k, bar);
  } else {
    pair_load_2d(s, map, k, row, bar);
  }
}

struct NoEarly {};

// ------------------------------------------------------------------ gate
template <int ACT, bool KEEP, bool CKPT8>
struct GateProb {
  static constexpr int kAMN = 0, kBMN = 0;
  struct Params {
    int* status;
    int64_t N, runs;
    int f, m_tiles, n_tiles, nk;
    int8_t *cg, *cu;
    float *sg, *su;
  };
  struct Tile {
    int m0, f0, w;
  };
  using Early = NoEarly;
  __device__ static void prefetch(const Params&, const Tile&, const PairEpi&, Early&) {}
  __device__ static int num_tiles(const Params& P) { return P.m_tiles * P.n_tiles; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    int mt, nt;
    band_tile(u, P.m_tiles, P.n_tiles, &mt, &nt);
    return Tile{mt * kPairM, nt * kPairHalf, 256};
  }
  __device__ static void load(const Params&, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    load_half<0>(&m.a0, sa, t.m0 + rank * kPairHalf, kb * kBK, bar);
    load_half<0>(rank ? &m.b1 : &m.b0, sb, t.f0, kb * kBK, bar);
  }
  __device__ static void keep8(const Params& P, const uint32_t (&r)[32], int64_t run_idx,
                               int8_t* codes, float* scale) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) top = max(top, r[j] & 0x7fffffffu);
    const CkptScale s = ckpt_scale(top);
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
    for (int piece = e.set; piece < 4; piece += 2) {
      const int c0 = t.f0 + piece * 32;
      if (c0 >= P.f) break;  // warp-uniform
      uint32_t g[32], u[32], p[16];
      tmem_ld32(e.taddr + piece * 32, g);
      tmem_ld32(e.taddr + kPairHalf + piece * 32, u);
      tmem_wait_ld(g);
      tmem_wait_ld(u);
      staging_free(e.lane);
      if (KEEP && !CKPT8) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          p[j] = pack_bf16(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
        stage_bf16(e.stg + 2048, e.lane, p);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          p[j] = pack_bf16(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
        stage_bf16(e.stg + 4096, e.lane, p);
      }
      if (KEEP && CKPT8 && row < P.N) {
        const int64_t run = row * P.runs + (c0 >> 5);
        keep8(P, g, run, P.cg, P.sg);
        keep8(P, u, run, P.cu, P.su);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
        p[j] = pack_bf16(
            act_fast<ACT>(__uint_as_float(g[2 * j])) * __uint_as_float(u[2 * j]),
            act_fast<ACT>(__uint_as_float(g[2 * j + 1])) * __uint_as_float(u[2 * j + 1]));
      stage_bf16(e.stg, e.lane, p);
      staging_ready();
      if (e.lane == 0) {
        tma_store_2d(&e.maps->o0, e.stg, c0, y0);
        if (KEEP && !CKPT8) {
          tma_store_2d(&e.maps->o1, e.stg + 2048, c0, y0);
          tma_store_2d(&e.maps->o2, e.stg + 4096, c0, y0);
        }
        bulk_commit();
      }
    }
  }
};

// ------------------------------------------------------------------ dh
// The accumulator is dh; the thread's row of the kept projections is requested one piece ahead.
template <int ACT, bool CKPT8>
struct GateGradProb {
  static constexpr int kAMN = 0, kBMN = 1;
  struct Params {
    int* status;
    int64_t N, runs;
    int f, m_tiles, n_tiles, nk, w;
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
  __device__ static int num_tiles(const Params& P) { return P.m_tiles * P.n_tiles; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    int mt, nt;
    band_tile(u, P.m_tiles, P.n_tiles, &mt, &nt);
    return Tile{mt * kPairM, nt * P.w, P.w};
  }
  __device__ static void load(const Params&, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    load_half<0>(&m.a0, sa, t.m0 + rank * kPairHalf, kb * kBK, bar);
    load_half<1>(&m.b0, sb, t.n0 + rank * (t.w / 2), kb * kBK, bar);
  }
  __device__ static void fetch(const Params& P, int64_t row, int c0, Early& k) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool in = row < P.N && c0 < P.f;
    if (CKPT8) {
      const int64_t run = in ? row * P.runs + (c0 >> 5) : 0;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        k.g[v] = in ? __ldg(static_cast<const uint4*>(P.g) + run * 2 + v) : zero;
        k.u[v] = in ? __ldg(static_cast<const uint4*>(P.u) + run * 2 + v) : zero;
      }
      k.sg = in ? __ldg(P.sg + run) : 0.f;
      k.su = in ? __ldg(P.su + run) : 0.f;
    } else {
      const int64_t at = in ? (row * P.f + c0) >> 3 : 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const bool has = in && c0 + 8 * v < P.f;
        k.g[v] = has ? __ldg(static_cast<const uint4*>(P.g) + at + v) : zero;
        k.u[v] = has ? __ldg(static_cast<const uint4*>(P.u) + at + v) : zero;
      }
    }
  }
  __device__ static void prefetch(const Params& P, const Tile& t, const PairEpi& e, Early& k) {
    fetch(P, (int64_t)t.m0 + e.row0 + e.lane, t.n0 + e.set * 32, k);
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
    for (int piece = e.set; piece * 32 < t.w; piece += 2) {
      const int c0 = t.n0 + piece * 32;
      if (c0 >= P.f) break;  // warp-uniform
      uint32_t d[32], ph[16], pg[16], pu[16];
      tmem_ld32(e.taddr + piece * 32, d);
      const Early now = k;
      if ((piece + 2) * 32 < t.w) fetch(P, row, c0 + 64, k);
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
      stage_bf16(e.stg, e.lane, ph);
      stage_bf16(e.stg + 2048, e.lane, pg);
      stage_bf16(e.stg + 4096, e.lane, pu);
      staging_ready();
      if (e.lane == 0) {
        tma_store_2d(&e.maps->o0, e.stg, c0, y0);
        tma_store_2d(&e.maps->o1, e.stg + 2048, c0, y0);
        tma_store_2d(&e.maps->o2, e.stg + 4096, c0, y0);
        bulk_commit();
      }
    }
  }
};

// ------------------------------------------------------------------ plain products
// out[rows x cols] = A B^T.  A second product may follow the first in the same accumulator
// (k-blocks from nk0 on read a1 and b1), or stand beside it as further tiles (kinds == 2: the
// second half of the tiles read a1 and write o1).  ADD: fp32 output, +=; else bf16, overwritten.
template <int AMN, int BMN, bool ADD>
struct PlainProb {
  static constexpr int kAMN = AMN, kBMN = BMN;
  struct Params {
    int* status;
    int64_t rows;
    int cols, m_tiles, n_tiles, kinds, nk, nk0, w;
  };
  struct Tile {
    int m0, n0, w, kind;
  };
  using Early = NoEarly;
  __device__ static void prefetch(const Params&, const Tile&, const PairEpi&, Early&) {}
  __device__ static int num_tiles(const Params& P) { return P.m_tiles * P.n_tiles * P.kinds; }
  __device__ static int num_kblocks(const Params& P) { return P.nk; }
  __device__ static Tile tile(const Params& P, int u) {
    int mt, nt;
    const int each = P.m_tiles * P.n_tiles;
    band_tile(u % each, P.m_tiles, P.n_tiles, &mt, &nt);
    return Tile{mt * kPairM, nt * P.w, P.w, u / each};
  }
  __device__ static void load(const Params& P, const PairMaps& m, const Tile& t, int kb, int rank,
                              void* sa, void* sb, uint64_t* bar) {
    const bool second = kb >= P.nk0;
    const int k = (second ? kb - P.nk0 : kb) * kBK;
    load_half<AMN>(second || t.kind ? &m.a1 : &m.a0, sa, t.m0 + rank * kPairHalf, k, bar);
    load_half<BMN>(second ? &m.b1 : &m.b0, sb, t.n0 + rank * (t.w / 2), k, bar);
  }
  __device__ static void epilogue(const Params& P, const Tile& t, const PairEpi& e, const Early&) {
    const int y0 = t.m0 + e.row0;
    if (y0 >= P.rows) return;  // warp-uniform
    const CUtensorMap* out = t.kind ? &e.maps->o1 : &e.maps->o0;
    for (int piece = e.set; piece * 32 < t.w; piece += 2) {
      const int c0 = t.n0 + piece * 32;
      if (c0 >= P.cols) break;  // warp-uniform
      uint32_t r[32];
      tmem_ld32(e.taddr + piece * 32, r);
      tmem_wait_ld(r);
      staging_free(e.lane);
      if (ADD) {
        stage_f32(e.stg, e.lane, r);
      } else {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          p[j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        stage_bf16(e.stg, e.lane, p);
      }
      staging_ready();
      if (e.lane == 0) {
        if (ADD) tma_add_2d(out, e.stg, c0, y0); else tma_store_2d(out, e.stg, c0, y0);
        bulk_commit();
      }
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
        tc_pair_kernel<Prob>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  if (tiles <= 0) return cudaSuccess;
  const int pairs = (int)std::min<int64_t>(tiles, p.sm_count / 2);
  tc_pair_kernel<Prob><<<2 * pairs, kPairThreads, kPairSmem, st>>>(maps, P);
  PKM_COUNT(1);
  return cudaGetLastError();
}

// [rows][cols] bf16 as an operand whose K runs along the row (boxes of 64 k x 128 rows) or
// down the rows (64 columns x 64 k).
bool map_kmajor(CUtensorMap* m, const void* base, int64_t rows, int cols) {
  return make_tmap_bf16_2d(m, base, cols, rows, (uint64_t)cols * 2, kBK, kPairHalf);
}
bool map_mnmajor(CUtensorMap* m, const void* base, int64_t rows, int cols) {
  return make_tmap_bf16_2d(m, base, cols, rows, (uint64_t)cols * 2, 64, kBK);
}
bool map_out(CUtensorMap* m, bool fp32, void* base, int64_t rows, int cols) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * (fp32 ? 4 : 2)};
  const uint32_t box[2] = {32, 32};
  return make_tmap_store(m, fp32, 2, base, dims, strides, box,
                         fp32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

int64_t tiles_of(int64_t rows, int w) { return (rows + w - 1) / w; }

// Output-tile width: the multiple of 32 whose rounds over the SM pairs times width is least;
// ties go to the wider tile, which reads fewer operand bytes per product.
int pair_width(int64_t m_tiles, int cols, int pairs) {
  int best = 256;
  int64_t cost = -1;
  for (int w = 256; w >= 128; w -= 32) {
    const int64_t c = tiles_of(m_tiles * tiles_of(cols, w), pairs) * w;
    if (cost < 0 || c < cost) {
      cost = c;
      best = w;
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
  P.m_tiles = (int)tiles_of(p.N, kPairM);
  P.n_tiles = (int)tiles_of(p.d_ff, kPairHalf);
  P.nk = (int)tiles_of(p.d_in, kBK);
  if (KEEP && CKPT8) {
    P.cg = static_cast<int8_t*>(s->g);
    P.cu = static_cast<int8_t*>(s->u);
    P.sg = s->g_scale;
    P.su = s->u_scale;
  }
  return launch_pair<G>(p, m, P, (int64_t)P.m_tiles * P.n_tiles, st);
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
  P.m_tiles = (int)tiles_of(p.N, kPairM);
  P.w = pair_width(P.m_tiles, p.d_ff, p.sm_count / 2);
  P.n_tiles = (int)tiles_of(p.d_ff, P.w);
  P.nk = (int)tiles_of(p.d_out, kBK);
  P.g = s.g;
  P.u = s.u;
  P.sg = s.g_scale;
  P.su = s.u_scale;
  return launch_pair<G>(p, m, P, (int64_t)P.m_tiles * P.n_tiles, st);
}

// out (+)= A B^T with k of length K (or K0 then K more).
template <int AMN, int BMN, bool ADD>
cudaError_t run_plain(const FfnPlan& p, const PairMaps& m, int64_t rows, int cols, int64_t K,
                      int kinds, bool twice, cudaStream_t st) {
  using G = PlainProb<AMN, BMN, ADD>;
  typename G::Params P{};
  P.status = p.status;
  P.rows = rows;
  P.cols = cols;
  P.kinds = kinds;
  P.m_tiles = (int)tiles_of(rows, kPairM);
  P.w = pair_width((int64_t)P.m_tiles * kinds, cols, p.sm_count / 2);
  P.n_tiles = (int)tiles_of(cols, P.w);
  P.nk0 = (int)tiles_of(K, kBK);
  P.nk = twice ? 2 * P.nk0 : P.nk0;
  return launch_pair<G>(p, m, P, (int64_t)P.m_tiles * P.n_tiles * kinds, st);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// Forward: h.  Backward: h, dg, du.  All [N][d_ff] bf16.
size_t ffn_tc_workspace(const FfnPlan& p, bool backward) {
  return align256((size_t)p.N * p.d_ff * 2) * (backward ? 3 : 1);
}

cudaError_t launch_ffn_fwd_tc(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                              const void* Wd, void* y, const pkm_ffn_saved* s, void* ws,
                              cudaStream_t st) {
  PairMaps m{};
  FFN_MAP(map_kmajor(&m.a0, x, p.N, p.d_in));
  FFN_MAP(map_kmajor(&m.b0, Wg, p.d_ff, p.d_in));
  FFN_MAP(map_kmajor(&m.b1, Wu, p.d_ff, p.d_in));
  FFN_MAP(map_out(&m.o0, false, ws, p.N, p.d_ff));
  if (s && !p.ckpt8) {
    FFN_MAP(map_out(&m.o1, false, s->g, p.N, p.d_ff));
    FFN_MAP(map_out(&m.o2, false, s->u, p.N, p.d_ff));
  }
#define FFN_GATE(ACT)                                                              \
  FFN_TRY(!s ? run_gate<ACT, false, false>(p, m, s, st)                            \
             : p.ckpt8 ? run_gate<ACT, true, true>(p, m, s, st)                    \
                       : run_gate<ACT, true, false>(p, m, s, st))
  if (p.act == PKM_ACT_GELU) FFN_GATE(PKM_ACT_GELU); else FFN_GATE(PKM_ACT_SILU);
#undef FFN_GATE
  PairMaps d{};
  FFN_MAP(map_kmajor(&d.a0, ws, p.N, p.d_ff));
  FFN_MAP(map_kmajor(&d.b0, Wd, p.d_out, p.d_ff));
  FFN_MAP(map_out(&d.o0, false, y, p.N, p.d_out));
  return run_plain<0, 0, false>(p, d, p.N, p.d_out, p.d_ff, 1, false, st);
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
  FFN_MAP(map_kmajor(&m.a0, dy, p.N, p.d_out));
  FFN_MAP(map_mnmajor(&m.b0, Wd, p.d_out, p.d_ff));
  FFN_MAP(map_out(&m.o0, false, h, p.N, p.d_ff));
  FFN_MAP(map_out(&m.o1, false, dg, p.N, p.d_ff));
  FFN_MAP(map_out(&m.o2, false, du, p.N, p.d_ff));
#define FFN_GRAD(ACT)                                              \
  FFN_TRY(p.ckpt8 ? run_gate_grad<ACT, true>(p, m, s, st)          \
                  : run_gate_grad<ACT, false>(p, m, s, st))
  if (p.act == PKM_ACT_GELU) FFN_GRAD(PKM_ACT_GELU); else FFN_GRAD(PKM_ACT_SILU);
#undef FFN_GRAD
  const bool add = !p.grad_bf16;
  if (dWd) {
    PairMaps w{};
    FFN_MAP(map_mnmajor(&w.a0, dy, p.N, p.d_out));
    FFN_MAP(map_mnmajor(&w.b0, h, p.N, p.d_ff));
    FFN_MAP(map_out(&w.o0, add, dWd, p.d_out, p.d_ff));
    FFN_TRY(add ? run_plain<1, 1, true>(p, w, p.d_out, p.d_ff, p.N, 1, false, st)
                : run_plain<1, 1, false>(p, w, p.d_out, p.d_ff, p.N, 1, false, st));
  }
  if (dWg || dWu) {
    PairMaps w{};
    void* first = dWg ? dWg : dWu;
    FFN_MAP(map_mnmajor(&w.a0, dWg ? dg : du, p.N, p.d_ff));
    FFN_MAP(map_mnmajor(&w.a1, du, p.N, p.d_ff));
    FFN_MAP(map_mnmajor(&w.b0, x, p.N, p.d_in));
    FFN_MAP(map_out(&w.o0, add, first, p.d_ff, p.d_in));
    if (dWg && dWu) FFN_MAP(map_out(&w.o1, add, dWu, p.d_ff, p.d_in));
    const int kinds = dWg && dWu ? 2 : 1;
    FFN_TRY(add ? run_plain<1, 1, true>(p, w, p.d_ff, p.d_in, p.N, kinds, false, st)
                : run_plain<1, 1, false>(p, w, p.d_ff, p.d_in, p.N, kinds, false, st));
  }
  if (dx) {
    PairMaps w{};
    FFN_MAP(map_kmajor(&w.a0, dg, p.N, p.d_ff));
    FFN_MAP(map_kmajor(&w.a1, du, p.N, p.d_ff));
    FFN_MAP(map_mnmajor(&w.b0, Wg, p.d_ff, p.d_in));
    FFN_MAP(map_mnmajor(&w.b1, Wu, p.d_ff, p.d_in));
    FFN_MAP(map_out(&w.o0, false, dx, p.N, p.d_in));
    FFN_TRY((run_plain<0, 1, false>(p, w, p.N, p.d_in, p.d_ff, 1, true, st)));
  }
  return cudaSuccess;
}

}  // namespace pkm
