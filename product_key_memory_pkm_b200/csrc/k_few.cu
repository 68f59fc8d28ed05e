// Products of a few tokens with a large matrix, y[n][o] = sum_i x[n][i] W[o][i], for 4-bit and
// bf16 weights, and the gated block made of them (decoding).
//
// Bound by reading the weights once.  They go straight from global memory into the registers
// that mma.sync takes them in: a row's codes are the A operand's rows, tokens the B operand's 8
// columns, and since a sum over k may run in any order, "k" inside an instruction is whichever 16
// columns the lanes happen to hold after wide loads of consecutive bytes.  The tensor cores do
// the products because their cost then does not grow with the tokens (up to 8 per
// instruction), not for their rate; a CTA-wide tcgen05 tile would have to put the weights
// through shared memory first.
//
//   4-bit   a lane's 8 codes are bytes of one row; (w >> 4j) & 0x000f000f is the pair of codes
//           (j, j + 4), and 0x4300 | code is the bf16 number 128 + code, from which 136 is
//           taken (exact).  Products of codes with bf16 x are exact, a unit of 64 columns is
//           summed in fp32 and then scaled by its group's scale in fp32.
//   bf16    a lane's 16 bytes are 8 columns of one row.
//
// A CTA's 8 warps split k for 16 output rows and add up through shared memory; where the rows
// are too few to fill the SMs, 2 or 4 CTAs of a cluster split k further and add up through
// distributed shared memory.  Every sum has a fixed order.
#include <algorithm>
#include <atomic>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

using bf = __nv_bfloat16;

constexpr int kWarps = 8, kTpb = 32 * kWarps;
constexpr int kRows = 16;   // output rows of a CTA
constexpr int kBatch = 4;   // units a warp has in flight

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes (j, j + 4) of a word as bf16 numbers code - 8.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int j) {
  const uint32_t m = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), off);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The products of a unit start from zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// 8 columns of a token in the order a word's codes come out in: (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ uint4 w4_order(const uint4& q) {
  return make_uint4(__byte_perm(q.x, q.z, 0x5410), __byte_perm(q.x, q.z, 0x7632),
                    __byte_perm(q.y, q.w, 0x5410), __byte_perm(q.y, q.w, 0x7632));
}

// 8 columns of a token, zeros for no token or no column.
__device__ __forceinline__ uint4 x8(const bf* x, int64_t N, int d_in, int n, int k) {
  return n < N && k < d_in ? *reinterpret_cast<const uint4*>(x + (int64_t)n * d_in + k)
                           : make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ weights
// Weights of one unit for this lane's two rows (g and g + 8).
//
// 4-bit: a unit is 64 columns.  HALF = false (groups of whole units): the lane holds columns
// [k0 + 16 c, +16) and one scale serves the unit.  HALF = true (groups of 32, 96, ...): columns
// [k0 + 8 c, +8) and [k0 + 32 + 8 c, +8), each half with its own scale.
template <bool HALF>
struct W4Unit {
  static constexpr int kCols = 64;
  uint32_t w[2][2];  // [row][word]
  bf s[2][HALF ? 2 : 1];

  struct Src {
    const uint8_t* row[2];
    const bf* scale[2];
    int d_in, group, ng;
    __device__ Src(const W4Mat& W, int d_out, int d_in_, int group_, int o0, int g)
        : d_in(d_in_), group(group_), ng((d_in_ + group_ - 1) / group_) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t o = min(o0 + g + 8 * r, d_out - 1);  // rows past the last are not stored
        row[r] = W.codes + o * (d_in / 2);
        scale[r] = W.scale + o * ng;
      }
    }
  };
  __device__ static int col(int k0, int c, int j) { return HALF ? k0 + 32 * j + 8 * c : k0 + 16 * c + 8 * j; }
  __device__ void load(const Src& S, int u, int c) {
    const int k0 = u * kCols;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (HALF) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int k = col(k0, c, j);
          w[r][j] = k < S.d_in ? __ldg(reinterpret_cast<const uint32_t*>(S.row[r] + k / 2)) : 0u;
          s[r][j] = k0 + 32 * j < S.d_in ? S.scale[r][(k0 + 32 * j) / S.group] : bf(0.f);
        }
      } else {
        const int k = col(k0, c, 0);
        const uint2 q = k < S.d_in ? __ldg(reinterpret_cast<const uint2*>(S.row[r] + k / 2))
                                   : make_uint2(0u, 0u);
        w[r][0] = q.x;
        w[r][1] = q.y;
        s[r][0] = S.scale[r][k0 / S.group];
      }
    }
  }
  __device__ static uint4 order(const uint4& q) { return w4_order(q); }
  // The codes of the lane's rows as A operands: a[j][2 i + r] = pair i of row r's word j.
  struct A {
    uint32_t a[2][8];
  };
  __device__ A operands() const {
    A o;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) o.a[j][i] = w4_pair(w[i & 1][j], i >> 1);
    return o;
  }
  // acc += this unit's products with 8 tokens, whose ordered columns of word j are xv[j]
  __device__ void mac(float (&acc)[4], const A& o, const uint4 (&xv)[2]) const {
    float t[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t(&a)[8] = o.a[j];
      if (HALF || j == 0)
        mma16816_first(t, a[0], a[1], a[2], a[3], xv[j].x, xv[j].y);
      else
        mma16816(t, a[0], a[1], a[2], a[3], xv[j].x, xv[j].y);
      mma16816(t, a[4], a[5], a[6], a[7], xv[j].z, xv[j].w);
      if (HALF || j == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(to_f32(s[i >> 1][HALF ? j : 0]), t[i], acc[i]);
      }
    }
  }
};

// bf16: a unit is 64 columns, as two halves of 8 columns per lane.
struct W16Unit {
  static constexpr int kCols = 64;
  uint4 w[2][2];  // [row][half]

  struct Src {
    const bf* row[2];
    int d_in;
    __device__ Src(const bf* W, int d_out, int d_in_, int, int o0, int g) : d_in(d_in_) {
#pragma unroll
      for (int r = 0; r < 2; ++r) row[r] = W + (int64_t)min(o0 + g + 8 * r, d_out - 1) * d_in;
    }
  };
  __device__ static int col(int k0, int c, int j) { return k0 + 32 * j + 8 * c; }
  __device__ void load(const Src& S, int u, int c) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = col(u * kCols, c, j);
        w[r][j] = k < S.d_in ? __ldcs(reinterpret_cast<const uint4*>(S.row[r] + k))
                             : make_uint4(0, 0, 0, 0);
      }
  }
  __device__ static uint4 order(const uint4& q) { return q; }
  struct A {};
  __device__ A operands() const { return A{}; }
  __device__ void mac(float (&acc)[4], const A&, const uint4 (&xv)[2]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mma16816(acc, w[0][j].x, w[1][j].x, w[0][j].y, w[1][j].y, xv[j].x, xv[j].y);
      mma16816(acc, w[0][j].z, w[1][j].z, w[0][j].w, w[1][j].w, xv[j].z, xv[j].w);
    }
  }
};

// ------------------------------------------------------------------ kernel
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ float peer_load(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

enum class Few { kF32, kBf16, kGate };  // y fp32, y bf16, or h = act(first) * second in bf16

// NT: tokens in blocks of 8.  GATE uses both matrices, the others the first.
template <class Unit, class Mat, int NT, Few OUT, int ACT>
__global__ void __launch_bounds__(kTpb) few_kernel(int N, int d_in, int d_out, int group, int ks,
                                                   const bf* __restrict__ x, Mat W0, Mat W1,
                                                   void* __restrict__ out, bool first) {
  constexpr int M = OUT == Few::kGate ? 2 : 1;
  constexpr int T = NT * 8;
  // a slot per warp, or per two warps where 8 would pass the static limit of 48 KiB
  constexpr int kSlots = M * NT <= 8 ? kWarps : kWarps / 2;
  __shared__ float part[M][kSlots][T][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rank = ks > 1 ? (int)blockIdx.x % ks : 0;
  const int o0 = (int)blockIdx.x / ks * kRows;
  const int units = (d_in + Unit::kCols - 1) / Unit::kCols;
  const int per = (units + kWarps * ks - 1) / (kWarps * ks);
  const int u0 = (rank * kWarps + warp) * per, u1 = min(units, u0 + per);

  const typename Unit::Src s0(W0, d_out, d_in, group, o0, g), s1(M == 2 ? W1 : W0, d_out, d_in, group, o0, g);
  float acc[M][NT][4];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.f;

  Unit w[M][kBatch];
  const auto fetch = [&](int u) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (u + b < u1) {
        w[0][b].load(s0, u + b, c);
        if (M == 2) w[M - 1][b].load(s1, u + b, c);
      }
  };
  // weights do not depend on the kernel before, x of the second product does
  if (u0 < u1) fetch(u0);
  if (first)
    allow_dependent_launch();
  else
    grid_dependency_wait();
  for (int u = u0; u < u1; u += kBatch) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (u + b >= u1) break;
      const int k0 = (u + b) * Unit::kCols;
      typename Unit::A a[M];
#pragma unroll
      for (int m = 0; m < M; ++m) a[m] = w[m][b].operands();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 xv[2] = {Unit::order(x8(x, N, d_in, t * 8 + g, Unit::col(k0, c, 0))),
                             Unit::order(x8(x, N, d_in, t * 8 + g, Unit::col(k0, c, 1)))};
#pragma unroll
        for (int m = 0; m < M; ++m) w[m][b].mac(acc[m][t], a[m], xv);
      }
    }
    if (u + kBatch < u1) fetch(u + kBatch);
  }

  // rows g, g + 8 and tokens 2c, 2c + 1 of each block of 8
  const auto leave = [&](bool add) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* p = &part[m][warp % kSlots][t * 8 + 2 * c + (i & 1)][g + 8 * (i >> 1)];
          *p = add ? *p + acc[m][t][i] : acc[m][t][i];
        }
  };
  if (warp < kSlots) leave(false);
  __syncthreads();
  if (kSlots < kWarps) {
    if (warp >= kSlots) leave(true);
    __syncthreads();
  }
  for (int e = threadIdx.x; e < M * T * kRows; e += kTpb) {
    const int m = e / (T * kRows), n = e / kRows % T, r = e % kRows;
    float s = part[m][0][n][r];
#pragma unroll
    for (int q = 1; q < kSlots; ++q) s += part[m][q][n][r];
    part[m][0][n][r] = s;
  }
  if (ks > 1) {
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  // each CTA of a cluster finishes its share of the elements
  for (int e = threadIdx.x + rank * kTpb; e < N * kRows; e += kTpb * ks) {
    const int n = e / kRows, r = e % kRows;
    float s[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      s[m] = part[m][0][n][r];
      if (ks > 1) {
        const uint32_t a = smem_addr(&part[m][0][n][r]);
        s[m] = peer_load(a, 0);
        for (int q = 1; q < ks; ++q) s[m] += peer_load(a, q);
      }
    }
    if (o0 + r >= d_out) continue;
    const int64_t at = (int64_t)n * d_out + o0 + r;
    if (OUT == Few::kF32) static_cast<float*>(out)[at] = s[0];
    if (OUT == Few::kBf16) static_cast<bf*>(out)[at] = __float2bfloat16_rn(s[0]);
    if (OUT == Few::kGate)
      static_cast<bf*>(out)[at] = __float2bfloat16_rn(act_fn<ACT>(s[0]) * s[M - 1]);
  }
  if (ks > 1) {  // a CTA's shared memory outlives its peers' reads
    __syncwarp();
    cluster_sync();
  }
}

// ------------------------------------------------------------------ many rows
// More than 16 tokens and many output rows: what bounds few_kernel there is not the weights but
// every 16 rows reading all of x again.  Here a CTA per SM keeps x (or a chunk of its columns)
// in shared memory, in operand order, and each of its warps takes 32 rows through all of k, so
// a read of x serves 32 rows.  The number of warps is chosen so that the rows fill whole
// rounds of the SMs.  Bound by issuing mma.sync with their operands.
constexpr int kWideRows = 32, kWideWarps = 12, kWideBatch = 2;
constexpr int kWideSmem = 225 * 1024;

template <bool HALF, int NT>
__global__ void __launch_bounds__(32 * kWideWarps, 1)
    wide_kernel(int N, int d_in, int d_out, int group, int chunk, const bf* __restrict__ x, W4Mat W,
                float* __restrict__ y) {
  using Unit = W4Unit<HALF>;
  constexpr int T = NT * 8;
  extern __shared__ __align__(16) unsigned char xs[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // rows of x are apart by an odd number of 16-byte columns (HALF: of 64-byte ones), so the 8
  // lanes that read 16 bytes at a time meet no bank twice
  const int pitch = chunk * 2 + (HALF ? 64 : 16);
  const int tiles = (d_out + kWideRows - 1) / kWideRows;
  const int chunks = (d_in + chunk - 1) / chunk;
  for (int first = 0; first < tiles; first += gridDim.x * warps) {  // a round, same for all CTAs
    const int tile = first + warp * gridDim.x + blockIdx.x;
    const bool mine = tile < tiles;
    const typename Unit::Src s0(W, d_out, d_in, group, tile * kWideRows, g);
    const typename Unit::Src s1(W, d_out, d_in, group, tile * kWideRows + 16, g);
    float acc[2][NT][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][t][i] = 0.f;
    for (int ch = 0; ch < chunks; ++ch) {
      const int k0 = ch * chunk, cols = min(chunk, d_in - k0);
      const int u0 = k0 / 64, u1 = u0 + (cols + 63) / 64;
      Unit cur[2][kWideBatch], nxt[2][kWideBatch];
      const auto fetch = [&](Unit (&w)[2][kWideBatch], int u) {
#pragma unroll
        for (int b = 0; b < kWideBatch; ++b)
          if (u + b < u1) {
            w[0][b].load(s0, u + b, c);
            w[1][b].load(s1, u + b, c);
          }
      };
      if (mine) fetch(cur, u0);
      if (first == 0 || chunks > 1) {
        if (ch > 0 || first > 0) __syncthreads();  // the chunk before has been read
        const int blocks = (cols + 63) / 64 * 8;   // 8-column blocks, whole units
        for (int e = threadIdx.x; e < T * blocks; e += blockDim.x) {
          const int n = e / blocks, b = e % blocks;
          *reinterpret_cast<uint4*>(xs + n * pitch + b * 16) =
              w4_order(x8(x, N, d_in, n, k0 + b * 8));
        }
        __syncthreads();
      }
      if (!mine) continue;
      for (int u = u0; u < u1; u += kWideBatch) {
        if (u + kWideBatch < u1) fetch(nxt, u + kWideBatch);
#pragma unroll
        for (int b = 0; b < kWideBatch; ++b) {
          if (u + b >= u1) break;
          const typename Unit::A a0 = cur[0][b].operands(), a1 = cur[1][b].operands();
          const unsigned char* xb = xs + g * pitch;
          const int o0 = Unit::col((u + b - u0) * 64, c, 0) * 2;
          const int o1 = Unit::col((u + b - u0) * 64, c, 1) * 2;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 xv[2] = {*reinterpret_cast<const uint4*>(xb + t * 8 * pitch + o0),
                                 *reinterpret_cast<const uint4*>(xb + t * 8 * pitch + o1)};
            cur[0][b].mac(acc[0][t], a0, xv);
            cur[1][b].mac(acc[1][t], a1, xv);
          }
        }
#pragma unroll
        for (int b = 0; b < kWideBatch; ++b) {
          cur[0][b] = nxt[0][b];
          cur[1][b] = nxt[1][b];
        }
      }
    }
    if (!mine) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = t * 8 + 2 * c + (i & 1), o = tile * kWideRows + r * 16 + g + 8 * (i >> 1);
          if (n < N && o < d_out) y[(int64_t)n * d_out + o] = acc[r][t][i];
        }
  }
}

template <bool HALF, int NT>
cudaError_t launch_wide(int N, int d_in, int d_out, int group, const bf* x, const W4Mat& W,
                        float* y, int sm_count, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(wide_kernel<HALF, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kWideSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  }
  const int pad = HALF ? 64 : 16;
  const int most = (kWideSmem / (NT * 8) - pad) / 2 / 64 * 64;
  const int chunk = std::min((d_in + 63) / 64 * 64, most);
  const int tiles = (d_out + kWideRows - 1) / kWideRows;
  const int per_sm = (tiles + sm_count - 1) / sm_count;
  const int rounds = (per_sm + kWideWarps - 1) / kWideWarps;
  const int warps = (per_sm + rounds - 1) / rounds;
  wide_kernel<HALF, NT><<<std::min(tiles, sm_count), 32 * warps, (size_t)NT * 8 * (chunk * 2 + pad), st>>>(
      N, d_in, d_out, group, chunk, x, W, y);
  PKM_COUNT(1);
  return cudaGetLastError();
}

// Rows enough that every SM has several warps of 32.
bool wide_form(int64_t N, int d_out, int sm_count) {
  return N > 16 && d_out >= 4 * kWideRows * sm_count;
}

// CTAs of a cluster along k: more while the grid leaves SMs empty and every warp still has
// two units.
int split_of(int d_out, int d_in, int sm_count) {
  const int tiles = (d_out + kRows - 1) / kRows, units = (d_in + 63) / 64;
  int ks = 1;
  while (ks < 4 && tiles * ks < 2 * sm_count && units >= 2 * kWarps * 2 * ks) ks *= 2;
  return ks;
}

template <class Unit, class Mat, int NT, Few OUT, int ACT>
cudaError_t launch(int N, int d_in, int d_out, int group, const bf* x, const Mat& W0,
                   const Mat& W1, void* out, bool first, int sm_count, cudaStream_t st) {
  const int ks = split_of(d_out, d_in, sm_count);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((d_out + kRows - 1) / kRows * ks));
  cfg.blockDim = dim3(kTpb);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 1 : 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, few_kernel<Unit, Mat, NT, OUT, ACT>, N, d_in,
                                           d_out, group, ks, x, W0, W1, out, first);
  PKM_COUNT(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class Unit, class Mat, Few OUT, int ACT, int MAXT>
cudaError_t by_tokens(int N, int d_in, int d_out, int group, const bf* x, const Mat& W0,
                      const Mat& W1, void* out, bool first, int sm_count, cudaStream_t st) {
  if (N <= 8)
    return launch<Unit, Mat, 1, OUT, ACT>(N, d_in, d_out, group, x, W0, W1, out, first, sm_count, st);
  if (N <= 16)
    return launch<Unit, Mat, 2, OUT, ACT>(N, d_in, d_out, group, x, W0, W1, out, first, sm_count, st);
  if constexpr (MAXT > 16) {
    if (N <= 32)
      return launch<Unit, Mat, 4, OUT, ACT>(N, d_in, d_out, group, x, W0, W1, out, first, sm_count, st);
    return launch<Unit, Mat, 8, OUT, ACT>(N, d_in, d_out, group, x, W0, W1, out, first, sm_count, st);
  }
  return cudaErrorInvalidValue;
}

template <Few OUT, int ACT>
cudaError_t w4(int N, int d_in, int d_out, int group, const bf* x, const W4Mat& W0,
               const W4Mat& W1, void* out, bool first, int sm_count, cudaStream_t st) {
  return group % 64 ? by_tokens<W4Unit<true>, W4Mat, OUT, ACT, 64>(N, d_in, d_out, group, x, W0, W1,
                                                                   out, first, sm_count, st)
                    : by_tokens<W4Unit<false>, W4Mat, OUT, ACT, 64>(N, d_in, d_out, group, x, W0,
                                                                    W1, out, first, sm_count, st);
}

}  // namespace

cudaError_t launch_w4_matvec(int64_t N, int d_in, int d_out, int group, const void* x,
                             const W4Mat& W, float* y, int sm_count, cudaStream_t st) {
  const bf* xb = static_cast<const bf*>(x);
  const int n = (int)N;
  if (wide_form(N, d_out, sm_count)) {
    if (group % 64)
      return N <= 32 ? launch_wide<true, 4>(n, d_in, d_out, group, xb, W, y, sm_count, st)
                     : launch_wide<true, 8>(n, d_in, d_out, group, xb, W, y, sm_count, st);
    return N <= 32 ? launch_wide<false, 4>(n, d_in, d_out, group, xb, W, y, sm_count, st)
                   : launch_wide<false, 8>(n, d_in, d_out, group, xb, W, y, sm_count, st);
  }
  return w4<Few::kF32, 0>(n, d_in, d_out, group, xb, W, W, y, true, sm_count, st);
}

cudaError_t launch_w4_ffn(const FfnPlan& p, int group, const void* x, const W4Mat& Wg,
                          const W4Mat& Wu, const W4Mat& Wd, void* y, void* ws, cudaStream_t st) {
  const bf* xb = static_cast<const bf*>(x);
  const cudaError_t e =
      p.act == PKM_ACT_GELU
          ? w4<Few::kGate, PKM_ACT_GELU>((int)p.N, p.d_in, p.d_ff, group, xb, Wg, Wu, ws, true, p.sm_count, st)
          : w4<Few::kGate, PKM_ACT_SILU>((int)p.N, p.d_in, p.d_ff, group, xb, Wg, Wu, ws, true, p.sm_count, st);
  if (e != cudaSuccess) return e;
  return w4<Few::kBf16, 0>((int)p.N, p.d_ff, p.d_out, group, static_cast<const bf*>(ws), Wd, Wd, y,
                           false, p.sm_count, st);
}

cudaError_t launch_ffn_few(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                           const void* Wd, void* y, void* ws, cudaStream_t st) {
  const bf* xb = static_cast<const bf*>(x);
  const bf *g = static_cast<const bf*>(Wg), *u = static_cast<const bf*>(Wu),
           *o = static_cast<const bf*>(Wd);
  constexpr int kMost = (int)kFfnFewTokens;
  const cudaError_t e =
      p.act == PKM_ACT_GELU
          ? by_tokens<W16Unit, const bf*, Few::kGate, PKM_ACT_GELU, kMost>(
                (int)p.N, p.d_in, p.d_ff, 0, xb, g, u, ws, true, p.sm_count, st)
          : by_tokens<W16Unit, const bf*, Few::kGate, PKM_ACT_SILU, kMost>(
                (int)p.N, p.d_in, p.d_ff, 0, xb, g, u, ws, true, p.sm_count, st);
  if (e != cudaSuccess) return e;
  return by_tokens<W16Unit, const bf*, Few::kBf16, 0, kMost>(
      (int)p.N, p.d_ff, p.d_out, 0, static_cast<const bf*>(ws), o, o, y, false, p.sm_count, st);
}

}  // namespace pkm
