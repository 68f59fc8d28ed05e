// The gated feed-forward block on CUDA cores, for fp32 storage and PKM_F_SIMT.  Everything
// between the products stays fp32.  Two forms:
//   large   the products by the strided fp32 GEMM (128 x 128 tiles), the activation and its
//           backward as elementwise kernels between them
//   small   32 x 32 tiles whose eight groups of 64 threads split k, with the gate or its
//           gradient as epilogue and independent products in one launch: two launches
//           forward, two backward
#include <algorithm>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

using bf = __nv_bfloat16;

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf* p, float v) { *p = __float2bfloat16_rn(v); }

// One value of a run of 32 columns (one lane each; lanes past the row hold 0) into an 8-bit
// checkpoint.
__device__ __forceinline__ void keep8(float v, int64_t run_idx, int lane, int8_t* codes,
                                      float* scale) {
  const CkptScale s = ckpt_scale<false>(__reduce_max_sync(0xffffffffu, mag_bits(v)));
  codes[run_idx * kCkptRun + lane] = (int8_t)ckpt_code_exact(v, s.top);
  if (lane == 0) scale[run_idx] = s.scale;
}

// g, u [N][f] fp32 -> h over g, and what the backward needs.  One warp per run of 32 columns.
template <int ACT, typename T>
__global__ void gate_kernel(int64_t N, int f, int64_t runs, float* g, const float* u, T* keep_g,
                            T* keep_u, int8_t* cg, int8_t* cu, float* sg, float* su) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < N * runs;
       w += warps) {
    const int64_t row = w / runs, run = w % runs;
    const int64_t col = run * kCkptRun + lane, o = row * f + col;
    const bool in = col < f;
    const float gv = in ? g[o] : 0.f, uv = in ? u[o] : 0.f;
    if (cg) {
      keep8(gv, w, lane, cg, sg);
      keep8(uv, w, lane, cu, su);
    }
    if (!in) continue;
    if (keep_g) {
      put(keep_g + o, gv);
      put(keep_u + o, uv);
    }
    g[o] = act_fn<ACT>(gv) * uv;
  }
}

// dh -> dg (over dh), du, h, from the kept projections.
template <int ACT, typename T>
__global__ void gate_grad_kernel(int64_t N, int f, int64_t runs, float* dh, float* du, float* h,
                                 const T* keep_g, const T* keep_u, const int8_t* cg,
                                 const int8_t* cu, const float* sg, const float* su) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < N * runs;
       w += warps) {
    const int64_t row = w / runs, run = w % runs;
    const int64_t col = run * kCkptRun + lane, o = row * f + col;
    if (col >= f) continue;
    float gv, uv;
    if (cg) {
      gv = (float)cg[w * kCkptRun + lane] * sg[w];
      uv = (float)cu[w * kCkptRun + lane] * su[w];
    } else {
      gv = to_f32(keep_g[o]);
      uv = to_f32(keep_u[o]);
    }
    float a, slope;
    act_and_slope<ACT>(gv, &a, &slope);
    const float d = dh[o];
    dh[o] = d * uv * slope;
    du[o] = d * a;
    h[o] = a * uv;
  }
}

__global__ void to_bf16_kernel(int64_t n, const float* src, bf* dst) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    dst[i] = __float2bfloat16_rn(src[i]);
}

int blocks_for(int64_t threads, int sm_count) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((threads + 255) / 256, sm_count * 8));
}

cudaError_t to_bf16(int64_t n, const float* src, void* dst, int sm_count, cudaStream_t st) {
  to_bf16_kernel<<<blocks_for(n, sm_count), 256, 0, st>>>(n, src, static_cast<bf*>(dst));
  PKM_COUNT(1);
  return cudaGetLastError();
}

#define FFN_TRY(expr)                        \
  do {                                       \
    const cudaError_t _e = (expr);           \
    if (_e != cudaSuccess) return _e;        \
  } while (0)

// ------------------------------------------------------------------ small form
// A tile's time is the depth of its k loop: a step is one round trip to L2 for 64 columns of
// k, with the loads of two steps in flight.
constexpr int kTile = 32, kGroups = 8, kSmallTpb = 64 * kGroups, kStep = 8 * kGroups, kPitch = 36;

struct Operand {  // element (row, k) at p[row * sr + k * sk]
  const void* p;
  int64_t sr, sk;
  bool b16;
  __device__ float at(int64_t i) const {
    return b16 ? to_f32(static_cast<const bf*>(p)[i]) : static_cast<const float*>(p)[i];
  }
};

// A thread's 4 elements of a kTile x kStep block of an operand: neighbours in memory are
// neighbouring threads.
struct Piece {
  float v[4];
  __device__ static int row(const Operand& o, int i) {
    return o.sk == 1 ? (threadIdx.x / kStep) + (kSmallTpb / kStep) * i : threadIdx.x % kTile;
  }
  __device__ static int k(const Operand& o, int i) {
    return o.sk == 1 ? threadIdx.x % kStep : (threadIdx.x / kTile) + (kSmallTpb / kTile) * i;
  }
  __device__ void load(const Operand& o, int64_t rows, int64_t K, int64_t r0, int64_t k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = r0 + row(o, i), kk = k0 + k(o, i);
      v[i] = r < rows && kk < K ? o.at(r * o.sr + kk * o.sk) : 0.f;
    }
  }
  __device__ void store(const Operand& o, float (*S)[kPitch]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) S[k(o, i)][row(o, i)] = v[i];
  }
};

// Products of one 32 x 32 tile with NB right operands (rows m0 .., n0 ..): thread t < 256 ends
// with row t / 8 and columns 4 (t % 8) .. + 3 of each.  `parts` pairs (a[i], b[i]) of k-length K
// follow one another in the sum (NB == 1).
template <int NB>
union TileShared {
  struct {
    float a[kStep][kPitch];
    float b[NB][kStep][kPitch];
  } in;
  float sum[kGroups][kTile][kTile + 4];
};
template <int NB>
__device__ __forceinline__ void tile_product(TileShared<NB>& S, const Operand* a, const Operand* b,
                                             int64_t M, int64_t Nn, int64_t K, int parts,
                                             int64_t m0, int64_t n0, float (&out)[NB][4]) {
  const int t = threadIdx.x, q = t >> 6, ty = (t & 63) >> 3, tx = t & 7;
  float acc[NB][4][4];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][i][j] = 0.f;
  const int64_t steps = (K + kStep - 1) / kStep, total = steps * parts;
  Piece pa[2], pb[2][NB];
  const auto fetch = [&](int64_t s, int slot) {
    if (s >= total) return;
    const int part = s >= steps;
    const int64_t k0 = (s - part * steps) * kStep;
    pa[slot].load(a[part], M, K, m0, k0);
#pragma unroll
    for (int n = 0; n < NB; ++n) pb[slot][n].load(b[part + n], Nn, K, n0, k0);
  };
  const auto step = [&](int64_t s, int slot) {
    const int part = s >= steps;
    pa[slot].store(a[part], S.in.a);
#pragma unroll
    for (int n = 0; n < NB; ++n) pb[slot][n].store(b[part + n], S.in.b[n]);
    __syncthreads();
    fetch(s + 2, slot);
#pragma unroll
    for (int k = q * 8; k < q * 8 + 8; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(&S.in.a[k][ty * 4]);
      const float xa[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float4 y = *reinterpret_cast<const float4*>(&S.in.b[n][k][tx * 4]);
        const float yb[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][i][j] = fmaf(xa[i], yb[j], acc[n][i][j]);
      }
    }
    __syncthreads();
  };
  fetch(0, 0);
  fetch(1, 1);
  for (int64_t s = 0; s < total; s += 2) {
    step(s, 0);
    if (s + 1 < total) step(s + 1, 1);
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(&S.sum[q][ty * 4 + i][tx * 4]) =
          make_float4(acc[n][i][0], acc[n][i][1], acc[n][i][2], acc[n][i][3]);
    __syncthreads();
    if (t < 256) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = t >> 3, c = (t & 7) * 4 + j;
        float v = S.sum[0][r][c];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) v += S.sum[g][r][c];
        out[n][j] = v;
      }
    }
    __syncthreads();
  }
}

// Four columns of a run (eight neighbouring threads) into an 8-bit checkpoint.
__device__ __forceinline__ void keep8_of4(const float (&v)[4], bool in, int64_t run_idx, int c,
                                          int8_t* codes, float* scale) {
  uint32_t top = max(max(mag_bits(v[0]), mag_bits(v[1])), max(mag_bits(v[2]), mag_bits(v[3])));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const CkptScale s = ckpt_scale<false>(top);
  uint32_t w[1];
  ckpt_codes<false>(v, s, w);
  if (!in) return;
  *reinterpret_cast<uint32_t*>(codes + run_idx * kCkptRun + c) = w[0];
  if (c == 0) scale[run_idx] = s.scale;
}

// h = act(x Wg^T) * (x Wu^T) [N][f] fp32, and what the backward needs.
template <int ACT, typename T>
__global__ void __launch_bounds__(kSmallTpb) small_gate_kernel(int64_t N, int f, int d_in, int64_t runs,
                                                         Operand x, Operand wg, Operand wu,
                                                         float* h, T* keep_g, T* keep_u, int8_t* cg,
                                                         int8_t* cu, float* sg, float* su) {
  __shared__ TileShared<2> S;
  const int64_t m0 = (int64_t)blockIdx.x * kTile, n0 = (int64_t)blockIdx.y * kTile;
  const Operand a[1] = {x}, b[2] = {wg, wu};
  float v[2][4];
  tile_product<2>(S, a, b, N, f, d_in, 1, m0, n0, v);
  allow_dependent_launch();
  if (threadIdx.x >= 256) return;
  const int c = (threadIdx.x & 7) * 4;
  const int64_t row = m0 + (threadIdx.x >> 3), col = n0 + c, o = row * f + col;
  if (cg) {
    keep8_of4(v[0], row < N, row * runs + blockIdx.y, c, cg, sg);
    keep8_of4(v[1], row < N, row * runs + blockIdx.y, c, cu, su);
  }
  if (row >= N) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + j >= f) break;
    if (keep_g) {
      put(keep_g + o + j, v[0][j]);
      put(keep_u + o + j, v[1][j]);
    }
    h[o + j] = act_fn<ACT>(v[0][j]) * v[1][j];
  }
}

// dh = dy Wd, and from it dg, du and h [N][f] fp32.
template <int ACT, typename T>
__global__ void __launch_bounds__(kSmallTpb)
    small_gate_grad_kernel(int64_t N, int f, int d_out, int64_t runs, Operand dy, Operand wd,
                           float* dg, float* du, float* h, const T* keep_g, const T* keep_u,
                           const int8_t* cg, const int8_t* cu, const float* sg, const float* su) {
  __shared__ TileShared<1> S;
  const int64_t m0 = (int64_t)blockIdx.x * kTile, n0 = (int64_t)blockIdx.y * kTile;
  float v[1][4];
  tile_product<1>(S, &dy, &wd, N, f, d_out, 1, m0, n0, v);
  allow_dependent_launch();
  if (threadIdx.x >= 256) return;
  const int c = (threadIdx.x & 7) * 4;
  const int64_t row = m0 + (threadIdx.x >> 3), col = n0 + c, o = row * f + col;
  if (row >= N) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + j >= f) break;
    float gv, uv;
    if (cg) {
      const int64_t run = row * runs + blockIdx.y;
      gv = (float)cg[run * kCkptRun + c + j] * sg[run];
      uv = (float)cu[run * kCkptRun + c + j] * su[run];
    } else {
      gv = to_f32(keep_g[o + j]);
      uv = to_f32(keep_u[o + j]);
    }
    float a, slope;
    act_and_slope<ACT>(gv, &a, &slope);
    dg[o + j] = v[0][j] * uv * slope;
    du[o + j] = v[0][j] * a;
    h[o + j] = a * uv;
  }
}

// Independent products, each tile of one of them: out = sum over parts of a[i] b[i]^T.
enum class JobOut { kF32, kAddF32, kBf16 };
struct Job {
  Operand a[2], b[2];
  int64_t M, Nn, K;
  int parts, tiles_n;
  unsigned end;  // tiles of the jobs up to and including this one
  JobOut mode;
  void* out;
};
struct Jobs {
  Job job[4];
  int n;
  unsigned tiles;
  void add(Job j) {
    j.tiles_n = (int)((j.Nn + kTile - 1) / kTile);
    tiles += (unsigned)(j.tiles_n * ((j.M + kTile - 1) / kTile));
    j.end = tiles;
    job[n++] = j;
  }
};
__global__ void __launch_bounds__(kSmallTpb) small_jobs_kernel(const __grid_constant__ Jobs jobs) {
  __shared__ TileShared<1> S;
  int i = 0;
  while (i + 1 < jobs.n && blockIdx.x >= jobs.job[i].end) ++i;
  const Job& j = jobs.job[i];
  const unsigned tile = blockIdx.x - (i ? jobs.job[i - 1].end : 0u);
  const int64_t m0 = (int64_t)(tile / j.tiles_n) * kTile, n0 = (int64_t)(tile % j.tiles_n) * kTile;
  grid_dependency_wait();
  float v[1][4];
  tile_product<1>(S, j.a, j.b, j.M, j.Nn, j.K, j.parts, m0, n0, v);
  const int64_t row = m0 + (threadIdx.x >> 3), col = n0 + (threadIdx.x & 7) * 4;
  if (threadIdx.x >= 256 || row >= j.M) return;
  const int64_t o = row * j.Nn + col;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (col + k >= j.Nn) break;
    if (j.mode == JobOut::kBf16) {
      static_cast<bf*>(j.out)[o + k] = __float2bfloat16_rn(v[0][k]);
    } else {
      float* p = static_cast<float*>(j.out) + o + k;
      *p = j.mode == JobOut::kAddF32 ? *p + v[0][k] : v[0][k];
    }
  }
}
cudaError_t launch_jobs(const Jobs& jobs, cudaStream_t st) {
  if (jobs.n == 0) return cudaSuccess;
  const cudaError_t e = launch_dependent(small_jobs_kernel, dim3(jobs.tiles), dim3(kSmallTpb), 0, st, jobs);
  PKM_COUNT(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Small while the multiplications of one product are few: there launches and the depth of a
// tile's k loop set the time, beyond it the wider tiles' reuse of operands.  fp32 forward and
// backward, small against large: 64 x 64 x 256 20 + 23 us against 64 + 135; 1024 x 256 x 1024
// 140 + 302 against 220 + 754; 1024 x 512 x 1024 266 + 582 against 285 + 788; 1024 x 512 x 2048
// 522 + 1140 against 424 + 1067.
constexpr double kSmallProducts = 536870912.0;  // 2^29
bool small_form(const FfnPlan& p) {
  return (double)p.N * p.d_ff * std::max(p.d_in, p.d_out) <= kSmallProducts;
}

cudaError_t small_forward(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                          const void* Wd, void* y, const pkm_ffn_saved* s, float* h,
                          cudaStream_t st) {
  const bool b = !p.fp32, c8 = s && p.ckpt8, kept = s && !p.ckpt8;
  const dim3 grid((unsigned)((p.N + kTile - 1) / kTile), (unsigned)p.runs);
  const Operand ox{x, p.d_in, 1, b}, og{Wg, p.d_in, 1, b}, ou{Wu, p.d_in, 1, b};
#define FFN_GATE(ACT, T)                                                                          \
  small_gate_kernel<ACT, T><<<grid, kSmallTpb, 0, st>>>(                                                \
      p.N, p.d_ff, p.d_in, p.runs, ox, og, ou, h, kept ? static_cast<T*>(s->g) : nullptr,         \
      kept ? static_cast<T*>(s->u) : nullptr, c8 ? static_cast<int8_t*>(s->g) : nullptr,          \
      c8 ? static_cast<int8_t*>(s->u) : nullptr, c8 ? s->g_scale : nullptr, c8 ? s->u_scale : nullptr)
  if (p.act == PKM_ACT_GELU) {
    if (b) FFN_GATE(PKM_ACT_GELU, bf); else FFN_GATE(PKM_ACT_GELU, float);
  } else {
    if (b) FFN_GATE(PKM_ACT_SILU, bf); else FFN_GATE(PKM_ACT_SILU, float);
  }
#undef FFN_GATE
  PKM_COUNT(1);
  FFN_TRY(cudaGetLastError());
  Jobs jobs{};
  Job j{};
  j.a[0] = Operand{h, p.d_ff, 1, false};
  j.b[0] = Operand{Wd, p.d_ff, 1, b};
  j.M = p.N; j.Nn = p.d_out; j.K = p.d_ff; j.parts = 1;
  j.mode = b ? JobOut::kBf16 : JobOut::kF32;
  j.out = y;
  jobs.add(j);
  return launch_jobs(jobs, st);
}

cudaError_t small_backward(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                           const void* Wd, const pkm_ffn_saved& s, const void* dy, void* dx,
                           void* dWg, void* dWu, void* dWd, float* dg, float* du, float* h,
                           cudaStream_t st) {
  const bool b = !p.fp32, c8 = p.ckpt8;
  const dim3 grid((unsigned)((p.N + kTile - 1) / kTile), (unsigned)p.runs);
  const Operand ody{dy, p.d_out, 1, b}, owd{Wd, 1, p.d_ff, b};
#define FFN_GRAD(ACT, T)                                                                          \
  small_gate_grad_kernel<ACT, T><<<grid, kSmallTpb, 0, st>>>(                                           \
      p.N, p.d_ff, p.d_out, p.runs, ody, owd, dg, du, h,                                          \
      c8 ? nullptr : static_cast<const T*>(s.g), c8 ? nullptr : static_cast<const T*>(s.u),       \
      c8 ? static_cast<const int8_t*>(s.g) : nullptr,                                             \
      c8 ? static_cast<const int8_t*>(s.u) : nullptr, s.g_scale, s.u_scale)
  if (p.act == PKM_ACT_GELU) {
    if (b) FFN_GRAD(PKM_ACT_GELU, bf); else FFN_GRAD(PKM_ACT_GELU, float);
  } else {
    if (b) FFN_GRAD(PKM_ACT_SILU, bf); else FFN_GRAD(PKM_ACT_SILU, float);
  }
#undef FFN_GRAD
  PKM_COUNT(1);
  FFN_TRY(cudaGetLastError());
  Jobs jobs{};
  if (dx) {  // the longest k first
    Job j{};
    j.a[0] = Operand{dg, p.d_ff, 1, false};
    j.a[1] = Operand{du, p.d_ff, 1, false};
    j.b[0] = Operand{Wg, 1, p.d_in, b};
    j.b[1] = Operand{Wu, 1, p.d_in, b};
    j.M = p.N; j.Nn = p.d_in; j.K = p.d_ff; j.parts = 2;
    j.mode = b ? JobOut::kBf16 : JobOut::kF32;
    j.out = dx;
    jobs.add(j);
  }
  const auto weight = [&](const void* a, bool a16, int rows, const void* c, bool c16, int cols,
                          void* out) {
    if (!out) return;
    Job j{};
    j.a[0] = Operand{a, 1, rows, a16};
    j.b[0] = Operand{c, 1, cols, c16};
    j.M = rows; j.Nn = cols; j.K = p.N; j.parts = 1;
    j.mode = p.grad_bf16 ? JobOut::kBf16 : JobOut::kAddF32;
    j.out = out;
    jobs.add(j);
  };
  weight(dg, false, p.d_ff, x, b, p.d_in, dWg);
  weight(du, false, p.d_ff, x, b, p.d_in, dWu);
  weight(dy, b, p.d_out, h, false, p.d_ff, dWd);
  return launch_jobs(jobs, st);
}

}  // namespace

// Forward: g (then h) and u [N][f], and y [N][d_out] when it is stored in bf16.
// Backward: dh (then dg), du and h [N][f], and one bf16 result's fp32 form at a time.
size_t ffn_simt_workspace(const FfnPlan& p, bool backward) {
  const int64_t nf = p.N * p.d_ff;
  int64_t n = (backward ? 3 : 2) * nf;
  if (!p.fp32) {
    int64_t t = p.N * (backward ? p.d_in : p.d_out);
    if (backward && p.grad_bf16)
      t = std::max(t, (int64_t)p.d_ff * std::max(p.d_in, p.d_out));
    n += t;
  }
  return (size_t)n * sizeof(float);
}

cudaError_t launch_ffn_fwd_simt(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                                const void* Wd, void* y, const pkm_ffn_saved* s, void* ws,
                                cudaStream_t st) {
  const bool b = !p.fp32;
  const int64_t nf = p.N * p.d_ff;
  float* g = static_cast<float*>(ws);
  float* u = g + nf;
  if (small_form(p)) return small_forward(p, x, Wg, Wu, Wd, y, s, g, st);
  float* y32 = b ? u + nf : static_cast<float*>(y);
  FFN_TRY(gemm_simt_f32(p.N, p.d_ff, p.d_in, x, b, p.d_in, 1, Wg, b, p.d_in, 1, g, p.d_ff,
                        GemmOut::Store, st));
  FFN_TRY(gemm_simt_f32(p.N, p.d_ff, p.d_in, x, b, p.d_in, 1, Wu, b, p.d_in, 1, u, p.d_ff,
                        GemmOut::Store, st));
  const bool c8 = s && p.ckpt8;
  void* kg = s && !c8 ? s->g : nullptr;
  void* ku = s && !c8 ? s->u : nullptr;
  int8_t* cg = c8 ? static_cast<int8_t*>(s->g) : nullptr;
  int8_t* cu = c8 ? static_cast<int8_t*>(s->u) : nullptr;
  float* sg = c8 ? s->g_scale : nullptr;
  float* su = c8 ? s->u_scale : nullptr;
  const int grid = blocks_for(p.N * p.runs * 32, p.sm_count);
#define FFN_GATE(ACT, T)                                                                       \
  gate_kernel<ACT, T><<<grid, 256, 0, st>>>(p.N, p.d_ff, p.runs, g, u, static_cast<T*>(kg),    \
                                            static_cast<T*>(ku), cg, cu, sg, su)
  if (p.act == PKM_ACT_GELU) {
    if (b) FFN_GATE(PKM_ACT_GELU, bf); else FFN_GATE(PKM_ACT_GELU, float);
  } else {
    if (b) FFN_GATE(PKM_ACT_SILU, bf); else FFN_GATE(PKM_ACT_SILU, float);
  }
#undef FFN_GATE
  PKM_COUNT(1);
  FFN_TRY(cudaGetLastError());
  FFN_TRY(gemm_simt_f32(p.N, p.d_out, p.d_ff, g, false, p.d_ff, 1, Wd, b, p.d_ff, 1, y32, p.d_out,
                        GemmOut::Store, st));
  return b ? to_bf16(p.N * p.d_out, y32, y, p.sm_count, st) : cudaSuccess;
}

cudaError_t launch_ffn_bwd_simt(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                                const void* Wd, const pkm_ffn_saved& s, const void* dy, void* dx,
                                void* dWg, void* dWu, void* dWd, void* ws, cudaStream_t st) {
  const bool b = !p.fp32;
  const int64_t nf = p.N * p.d_ff;
  float* dg = static_cast<float*>(ws);
  float* du = dg + nf;
  float* h = du + nf;
  float* tmp = h + nf;
  if (small_form(p))
    return small_backward(p, x, Wg, Wu, Wd, s, dy, dx, dWg, dWu, dWd, dg, du, h, st);
  // dh[t][j] = sum_o dy[t][o] Wd[o][j]
  FFN_TRY(gemm_simt_f32(p.N, p.d_ff, p.d_out, dy, b, p.d_out, 1, Wd, b, 1, p.d_ff, dg, p.d_ff,
                        GemmOut::Store, st));
  const int grid = blocks_for(p.N * p.runs * 32, p.sm_count);
  const bool c8 = p.ckpt8;
#define FFN_GRAD(ACT, T)                                                                       \
  gate_grad_kernel<ACT, T><<<grid, 256, 0, st>>>(                                              \
      p.N, p.d_ff, p.runs, dg, du, h, c8 ? nullptr : static_cast<const T*>(s.g),               \
      c8 ? nullptr : static_cast<const T*>(s.u), c8 ? static_cast<const int8_t*>(s.g) : nullptr, \
      c8 ? static_cast<const int8_t*>(s.u) : nullptr, s.g_scale, s.u_scale)
  if (p.act == PKM_ACT_GELU) {
    if (b) FFN_GRAD(PKM_ACT_GELU, bf); else FFN_GRAD(PKM_ACT_GELU, float);
  } else {
    if (b) FFN_GRAD(PKM_ACT_SILU, bf); else FFN_GRAD(PKM_ACT_SILU, float);
  }
#undef FFN_GRAD
  PKM_COUNT(1);
  FFN_TRY(cudaGetLastError());
  if (dx) {
    float* d = b ? tmp : static_cast<float*>(dx);
    FFN_TRY(gemm_simt_f32(p.N, p.d_in, p.d_ff, dg, false, p.d_ff, 1, Wg, b, 1, p.d_in, d, p.d_in,
                          GemmOut::Store, st));
    FFN_TRY(gemm_simt_f32(p.N, p.d_in, p.d_ff, du, false, p.d_ff, 1, Wu, b, 1, p.d_in, d, p.d_in,
                          GemmOut::Accumulate, st));
    if (b) FFN_TRY(to_bf16(p.N * p.d_in, d, dx, p.sm_count, st));
  }
  // weight gradients: out[o][i] = sum_t a[t][o] c[t][i]
  const auto weight = [&](const void* a, bool a16, int rows, const void* c, bool c16, int cols,
                          void* out) -> cudaError_t {
    if (!out) return cudaSuccess;
    float* d = p.grad_bf16 ? tmp : static_cast<float*>(out);
    FFN_TRY(gemm_simt_f32(rows, cols, p.N, a, a16, 1, rows, c, c16, 1, cols, d, cols,
                          p.grad_bf16 ? GemmOut::Store : GemmOut::Accumulate, st));
    return p.grad_bf16 ? to_bf16((int64_t)rows * cols, d, out, p.sm_count, st) : cudaSuccess;
  };
  FFN_TRY(weight(dg, false, p.d_ff, x, b, p.d_in, dWg));
  FFN_TRY(weight(du, false, p.d_ff, x, b, p.d_in, dWu));
  return weight(dy, b, p.d_out, h, false, p.d_ff, dWd);
}

}  // namespace pkm
