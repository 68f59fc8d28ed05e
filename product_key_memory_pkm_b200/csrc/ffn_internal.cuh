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
// its values to codes.  top: that magnitude, or -1 for a run with a non-finite value.  The
// quotient top / 127 comes from the rounded 1 / 127 and one exact remainder, which gives the
// correctly rounded result for every fp32 mantissa (all 2^23 tried).  inv is correctly rounded or,
// for values exact in bf16 (BF16), whose codes tolerate it, off by up to 3 of its last places.
// Runs outside 1e-30 .. 2e36, where one of the steps could leave the normal numbers (127 a among
// them), divide.
struct CkptScale {
  float scale, inv, top;
  __device__ bool plain() const { return top >= 1e-30f && top <= 2e36f; }
};
template <bool BF16>
__device__ __forceinline__ CkptScale ckpt_scale(uint32_t top_bits) {
  CkptScale s;
  s.top = __uint_as_float(top_bits);
  constexpr float k = 1.f / 127.f;
  const float q = s.top * k;
  s.scale = fmaf(fmaf(-127.f, q, s.top), k, q);
  if (BF16) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s.top));
    s.inv = 127.f * r;
  } else {
    s.inv = 127.f / s.top;
  }
  if (!s.plain()) {
    s.scale = s.top / 127.f;
    s.inv = 0.f;
    if (top_bits >= kInfBits) {
      s.scale = __uint_as_float(0x7fc00000u);
      s.top = -1.f;
    }
  }
  return s;
}
// Code of one value, formed in 64 bits: 127 a is exact there, and a quotient that is not a
// half is farther than 2^-26 from one, so its rounding decides nothing.
__device__ __noinline__ inline int ckpt_code_exact(float a, float top) {
  return top <= 0.f ? 0 : (int)rint((double)a * 127.0 / (double)top);
}
// Codes of N values, four to a word: 127 a / top rounded to the nearest integer, halves to
// even.  Adding 1.5 * 2^23 leaves the rounded number in the low bits.  The product a * inv is not
// exact, so a quotient that is a half, or nearly, needs care:
//   BF16 (values exact in bf16): a quotient 127 a / top that is not a half is at least 2^-16
//     of it away (254 A 2^z against M (2r + 1) with 8-bit integers A and M), so rounding the
//     product to 20 significant bits first turns the halves into exact halves and moves no
//     other across one.  Such halves are frequent there, and this has no branch.
//   else: the fused product is off by 2^-24 of itself, 7.6e-6 at most; within 1e-5 of a half the
//     exact remainder decides.  With 127 a = hi + lo (both fp32) and r the candidate, e = hi - r
//     top is exact (a multiple of top's last place, below top), so is 2|e| - top, and the sum
//     with 2 lo has the sign of the exact remainder less a half.
// Runs that are not plain() are formed in 64 bits.
template <bool BF16, int N>
__device__ __forceinline__ void ckpt_codes(const float (&a)[N], const CkptScale& s,
                                           uint32_t (&w)[N / 4]) {
  constexpr float kMagic = 12582912.f;
  float far = 0.f;
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = a[4 * j + i];
      if (BF16) {
        const float q = v * s.inv, c = q * 17.f;
        b[i] = __float_as_uint(__fadd_rn(__fsub_rn(c, __fsub_rn(c, q)), kMagic));
      } else {
        const float t = fmaf(v, s.inv, kMagic);
        far = fmaxf(far, fabsf(fmaf(v, s.inv, kMagic - t)));
        b[i] = __float_as_uint(t);
      }
    }
    w[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  if (!BF16 && far > 0.5f - 1e-5f) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = a[4 * j + i];
        float r = __fsub_rn(fmaf(v, s.inv, kMagic), kMagic);
        const float hi = __fmul_rn(v, 127.f), lo = fmaf(v, 127.f, -hi);
        const float e = fmaf(-r, s.top, hi), up = e < 0.f ? -1.f : 1.f;
        const float over = __fadd_rn(fmaf(2.f, fabsf(e), -s.top), 2.f * lo * up);
        if (over > 0.f || (over == 0.f && ((int)r & 1))) r += up;
        w[j] |= ((uint32_t)(int)r & 0xffu) << (8 * i);
      }
    }
  }
  if (!s.plain() && s.top != 0.f) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[j] |= ((uint32_t)ckpt_code_exact(a[4 * j + i], s.top) & 0xffu) << (8 * i);
    }
  }
}
// The four codes of a word as floats (exact): byte c ^ 0x80 as the low mantissa byte of 2^23
// stands for 2^23 + 128 + c.
__device__ __forceinline__ void ckpt_floats4(uint32_t w, float (&v)[4]) {
  const uint32_t x = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440 | i)) - 8388736.f;
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
// Scales of a row.  In 64 bits: any positive multiple of 32 is a group, and d_in + group passes
// 2^31 for the largest (which then are one group a row).
inline int w4_groups(int d_in, int group) { return (int)(((int64_t)d_in + group - 1) / group); }

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
                              float* scale, cudaStream_t st);
cudaError_t launch_ckpt8_unpack(int64_t rows, int cols, bool fp32, const int8_t* codes,
                                const float* scale, void* dst, cudaStream_t st);

cudaError_t launch_w4_pack(int d_out, int d_in, int group, const void* W, uint8_t* codes,
                           void* scale, cudaStream_t st);
cudaError_t launch_w4_unpack(int d_out, int d_in, int group, const W4Mat& W, void* out,
                             cudaStream_t st);
cudaError_t launch_w4_matvec(int64_t N, int d_in, int d_out, int group, const void* x,
                             const W4Mat& W, float* y, int sm_count, cudaStream_t st);
cudaError_t launch_w4_ffn(const FfnPlan& p, int group, const void* x, const W4Mat& Wg,
                          const W4Mat& Wu, const W4Mat& Wd, void* y, void* ws, cudaStream_t st);
// The forward of a few tokens with nothing kept (bf16 weights).  ws: h [N][d_ff] bf16.  Up to 16:
// on the device, this against the CTA-pair engine, us, 1600 x 6400 x 1600: 8 tokens 12.6 / 33.3,
// 16 tokens 18.1 / 29.3, 17 tokens 31.6 / 33.8, 32 tokens 31.8 / 29.7, 64 tokens 69.9 / 30.3.
// (Narrower blocks cross later: 1024 x 2728 x 1024 at 32 tokens 13.4 / 24.8, at 64 29.4 / 25.0.)
constexpr int64_t kFfnFewTokens = 16;
cudaError_t launch_ffn_few(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                           const void* Wd, void* y, void* ws, cudaStream_t st);

}  // namespace pkm
