// Internal declarations of the gated feed-forward block, the 8-bit activation checkpoints and
// the 4-bit weight products.
#pragma once

#include "pkm_internal.cuh"

namespace pkm {

// ---------------------------------------------------------------- activations
constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// act(v), fp32.  SiLU: v / (1 + exp(-v)); where exp(-v) overflows the quotient is -0, its
// limit.  GELU through erfc, whose relative accuracy holds in the negative tail.
template <int ACT>
__device__ __forceinline__ float act_fn(float v) {
  if (ACT == PKM_ACT_GELU) return 0.5f * v * erfcf(-v * kInvSqrt2);
  return v / (1.f + expf(-v));
}
// act(v) and act'(v).
template <int ACT>
__device__ __forceinline__ void act_and_slope(float v, float* a, float* slope) {
  if (ACT == PKM_ACT_GELU) {
    const float c = 0.5f * erfcf(-v * kInvSqrt2);
    *a = v * c;
    *slope = c + v * (kInvSqrt2Pi * expf(-0.5f * v * v));
    return;
  }
  const float s = 1.f / (1.f + expf(-v));
  *a = v * s;
  *slope = s * (1.f + v * (1.f - s));
}

// ---------------------------------------------------------------- 8-bit checkpoints
constexpr int kCkptRun = 32;  // columns per scale
inline __host__ __device__ int64_t ckpt_runs(int64_t cols) {
  return (cols + kCkptRun - 1) / kCkptRun;
}

// The magnitude of a value as ordered bits: finite < infinity < NaN, so that one integer
// maximum finds both the largest magnitude of a run and whether it holds a non-finite value.
__device__ __forceinline__ uint32_t mag_bits(float a) { return __float_as_uint(a) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// The scale of a run whose largest magnitude has the bits `top`, and the factor that takes
// its values to codes (0 for an all-zero or non-finite run).
struct CkptScale {
  float scale, inv, top;
};
__device__ __forceinline__ CkptScale ckpt_scale(uint32_t top_bits) {
  CkptScale s;
  s.top = __uint_as_float(top_bits);
  if (top_bits >= kInfBits) {
    s.scale = __uint_as_float(0x7fc00000u);
    s.inv = 0.f;
    s.top = 0.f;
  } else {
    s.scale = s.top / 127.f;
    s.inv = s.top > 0.f ? 127.f / s.top : 0.f;  // overflows to inf below 2^-121: see ckpt_code
  }
  return s;
}
// 127 a / top rounded to the nearest integer, halves to even.  The fp32 product is off by at
// most 127 * 2^-23 = 1.5e-5, so only within 2e-5 of a half can it round the other way: there
// the quotient is formed in 64 bits (127 a is exact, and a quotient that is not a half is
// farther than 2^-26 from one).
__device__ __forceinline__ int ckpt_code(float a, const CkptScale& s) {
  if (s.top == 0.f) return 0;
  const float q = a * s.inv;
  const float r = rintf(q);
  if (fabsf(fabsf(q - r) - 0.5f) > 2e-5f && s.top > 1e-30f) return (int)r;
  return (int)rint((double)a * 127.0 / (double)s.top);
}

// ---------------------------------------------------------------- plan
struct FfnPlan {
  int64_t N;
  int d_in, d_ff, d_out, act;
  int64_t runs;    // scale runs per row of a checkpoint
  bool fp32;       // fp32 storage
  bool simt;       // CUDA-core kernels
  bool ckpt8;      // projections kept in 8 bits
  bool grad_bf16;  // weight gradients bf16, overwritten
  int dev, sm_count;
  int* status;
};

struct W4Mat {
  const uint8_t* codes;
  const __nv_bfloat16* scale;
};

// CUDA-core path (any storage type).
size_t ffn_simt_workspace(const FfnPlan& p, bool backward);
cudaError_t launch_ffn_fwd_simt(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                                const void* Wd, void* y, const pkm_ffn_saved* s, void* ws,
                                cudaStream_t st);
cudaError_t launch_ffn_bwd_simt(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                                const void* Wd, const pkm_ffn_saved& s, const void* dy, void* dx,
                                void* dWg, void* dWu, void* dWd, void* ws, cudaStream_t st);

// Tensor-core path (bf16 storage).
size_t ffn_tc_workspace(const FfnPlan& p, bool backward);
cudaError_t launch_ffn_fwd_tc(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                              const void* Wd, void* y, const pkm_ffn_saved* s, void* ws,
                              cudaStream_t st);
cudaError_t launch_ffn_bwd_tc(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                              const void* Wd, const pkm_ffn_saved& s, const void* dy, void* dx,
                              void* dWg, void* dWu, void* dWd, void* ws, cudaStream_t st);

cudaError_t launch_ckpt8_pack(int64_t rows, int cols, bool fp32, const void* src, int8_t* codes,
                              float* scale, int sm_count, cudaStream_t st);
cudaError_t launch_ckpt8_unpack(int64_t rows, int cols, bool fp32, const int8_t* codes,
                                const float* scale, void* dst, int sm_count, cudaStream_t st);

cudaError_t launch_w4_pack(int d_out, int d_in, int group, const void* W, uint8_t* codes,
                           void* scale, cudaStream_t st);
cudaError_t launch_w4_unpack(int d_out, int d_in, int group, const W4Mat& W, void* out,
                             cudaStream_t st);
cudaError_t launch_w4_matvec(int64_t N, int d_in, int d_out, int group, const void* x,
                             const W4Mat& W, float* y, int sm_count, cudaStream_t st);
cudaError_t launch_w4_ffn(const FfnPlan& p, int group, const void* x, const W4Mat& Wg,
                          const W4Mat& Wu, const W4Mat& Wd, void* y, void* ws, cudaStream_t st);

}  // namespace pkm
