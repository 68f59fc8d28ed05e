// Products with 4-bit weights for few tokens: W[o][i] = (code - 8) * scale[o][i / group].
// Bound by reading the codes (half a byte per weight) and the scales once.
#include <algorithm>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

using bf = __nv_bfloat16;

// One warp per (row, group).
__global__ void w4_pack_kernel(int64_t d_out, int d_in, int group, int ng, const bf* W,
                               uint8_t* codes, bf* scale) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < d_out * ng;
       w += warps) {
    const int64_t row = w / ng;
    const int k0 = (int)(w % ng) * group, k1 = min(d_in - k0, group) + k0;
    const bf* r = W + row * d_in;
    uint32_t top = 0;
    for (int k = k0 + lane; k < k1; k += 32) top = max(top, mag_bits(to_f32(r[k])));
    top = __reduce_max_sync(0xffffffffu, top);
    bf s = __float2bfloat16_rn(__uint_as_float(top) / 7.f);
    if (top >= kInfBits) s = __ushort_as_bfloat16((unsigned short)0x7fc0);
    const float sf = to_f32(s);
    const bool plain = sf > 0.f;  // false for an all-zero group and for a NaN scale
    for (int k = k0 + 2 * lane; k < k1; k += 64) {
      int c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        c[j] = plain ? (int)fminf(fmaxf(rintf(to_f32(r[k + j]) / sf), -8.f), 7.f) + 8 : 8;
      codes[(row * d_in + k) >> 1] = (uint8_t)(c[0] | (c[1] << 4));
    }
    if (lane == 0) scale[w] = s;
  }
}

__global__ void w4_unpack_kernel(int64_t d_out, int d_in, int group, int ng, const uint8_t* codes,
                                 const bf* scale, bf* out) {
  const int64_t n = d_out * (d_in / 2);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / (d_in / 2);
    const int k = 2 * (int)(i % (d_in / 2));
    const float s = to_f32(scale[row * ng + k / group]);
    const int c = codes[i];
    out[2 * i] = __float2bfloat16_rn((float)((c & 15) - 8) * s);
    out[2 * i + 1] = __float2bfloat16_rn((float)((c >> 4) - 8) * s);
  }
}

// One warp per (output, token).  y = sum over groups of scale * (sum of code * x).
__device__ __forceinline__ float w4_dot(const bf* x, const W4Mat& W, int64_t row, int d_in,
                                        int group, int ng, int lane) {
  float acc = 0.f;
  for (int k = 8 * lane; k < d_in; k += 256) {  // 8 columns: within one group
    const uint32_t c = *reinterpret_cast<const uint32_t*>(W.codes + ((row * d_in + k) >> 1));
    float xv[8], part = 0.f;
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(x + k), xv);
#pragma unroll
    for (int j = 0; j < 8; ++j) part = fmaf((float)((int)((c >> (4 * j)) & 15u) - 8), xv[j], part);
    acc = fmaf(to_f32(W.scale[row * ng + k / group]), part, acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}

__global__ void w4_matvec_kernel(int64_t N, int d_in, int64_t d_out, int group, int ng,
                                 const bf* x, W4Mat W, float* y, bf* y16) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < N * d_out;
       w += warps) {
    const int64_t o = w / N, n = w % N;
    const float v = w4_dot(x + n * d_in, W, o, d_in, group, ng, lane);
    if (lane == 0) {
      if (y) y[n * d_out + o] = v; else y16[n * d_out + o] = __float2bfloat16_rn(v);
    }
  }
}

template <int ACT>
__global__ void w4_gate_kernel(int64_t N, int d_in, int64_t f, int group, int ng, const bf* x,
                               W4Mat Wg, W4Mat Wu, bf* h) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < N * f;
       w += warps) {
    const int64_t o = w / N, n = w % N;
    const float g = w4_dot(x + n * d_in, Wg, o, d_in, group, ng, lane);
    const float u = w4_dot(x + n * d_in, Wu, o, d_in, group, ng, lane);
    if (lane == 0) h[n * f + o] = __float2bfloat16_rn(act_fn<ACT>(g) * u);
  }
}

int grid_for(int64_t warps, int sm_count) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8, sm_count * 8));
}

}  // namespace

cudaError_t launch_w4_pack(int d_out, int d_in, int group, const void* W, uint8_t* codes,
                           void* scale, cudaStream_t st) {
  const int ng = (d_in + group - 1) / group;
  w4_pack_kernel<<<grid_for((int64_t)d_out * ng, 148), 256, 0, st>>>(
      d_out, d_in, group, ng, static_cast<const bf*>(W), codes, static_cast<bf*>(scale));
  PKM_COUNT(1);
  return cudaGetLastError();
}

cudaError_t launch_w4_unpack(int d_out, int d_in, int group, const W4Mat& W, void* out,
                             cudaStream_t st) {
  const int ng = (d_in + group - 1) / group;
  w4_unpack_kernel<<<grid_for((int64_t)d_out * d_in / 64 + 1, 148), 256, 0, st>>>(
      d_out, d_in, group, ng, W.codes, W.scale, static_cast<bf*>(out));
  PKM_COUNT(1);
  return cudaGetLastError();
}

cudaError_t launch_w4_matvec(int64_t N, int d_in, int d_out, int group, const void* x,
                             const W4Mat& W, float* y, int sm_count, cudaStream_t st) {
  const int ng = (d_in + group - 1) / group;
  w4_matvec_kernel<<<grid_for(N * d_out, sm_count), 256, 0, st>>>(
      N, d_in, d_out, group, ng, static_cast<const bf*>(x), W, y, nullptr);
  PKM_COUNT(1);
  return cudaGetLastError();
}

cudaError_t launch_w4_ffn(const FfnPlan& p, int group, const void* x, const W4Mat& Wg,
                          const W4Mat& Wu, const W4Mat& Wd, void* y, void* ws, cudaStream_t st) {
  const int ng = (p.d_in + group - 1) / group, nf = (p.d_ff + group - 1) / group;
  bf* h = static_cast<bf*>(ws);
  const int grid = grid_for(p.N * p.d_ff, p.sm_count);
  if (p.act == PKM_ACT_GELU)
    w4_gate_kernel<PKM_ACT_GELU><<<grid, 256, 0, st>>>(p.N, p.d_in, p.d_ff, group, ng,
                                                       static_cast<const bf*>(x), Wg, Wu, h);
  else
    w4_gate_kernel<PKM_ACT_SILU><<<grid, 256, 0, st>>>(p.N, p.d_in, p.d_ff, group, ng,
                                                       static_cast<const bf*>(x), Wg, Wu, h);
  PKM_COUNT(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  w4_matvec_kernel<<<grid_for(p.N * p.d_out, p.sm_count), 256, 0, st>>>(
      p.N, p.d_ff, p.d_out, group, nf, h, Wd, nullptr, static_cast<bf*>(y));
  PKM_COUNT(1);
  return cudaGetLastError();
}

}  // namespace pkm
