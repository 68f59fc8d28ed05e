// The gated feed-forward block on CUDA cores, for fp32 storage and PKM_F_SIMT: the products
// by the strided fp32 GEMM, the activation and its backward as elementwise kernels between
// them.  Everything between the products stays fp32.
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
  const CkptScale s = ckpt_scale(__reduce_max_sync(0xffffffffu, mag_bits(v)));
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
