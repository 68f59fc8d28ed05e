// 8-bit activation checkpoints: a run of 32 columns of a row shares one fp32 scale.
//
// Pack reads 2 or 4 bytes per value and writes 1.125; unpack the other way round.  Both are
// bound by HBM.
#include <algorithm>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

using bf = __nv_bfloat16;

template <typename T>
__global__ void pack_kernel(int64_t rows, int cols, int64_t runs, const T* src, int8_t* codes,
                            float* scale) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < rows * runs;
       w += warps) {
    const int64_t row = w / runs, col = (w % runs) * kCkptRun + lane;
    const float v = col < cols ? to_f32(src[row * cols + col]) : 0.f;
    const CkptScale s = ckpt_scale(__reduce_max_sync(0xffffffffu, mag_bits(v)));
    codes[w * kCkptRun + lane] = (int8_t)ckpt_code(v, s);
    if (lane == 0) scale[w] = s.scale;
  }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void unpack_kernel(int64_t rows, int cols, int64_t runs, const int8_t* codes,
                              const float* scale, T* dst) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < rows * runs;
       w += warps) {
    const int64_t row = w / runs, col = (w % runs) * kCkptRun + lane;
    if (col < cols) put(dst + row * cols + col, (float)codes[w * kCkptRun + lane] * scale[w]);
  }
}

int grid_for(int64_t warps, int sm_count) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8, sm_count * 8));
}

}  // namespace

cudaError_t launch_ckpt8_pack(int64_t rows, int cols, bool fp32, const void* src, int8_t* codes,
                              float* scale, int sm_count, cudaStream_t st) {
  const int64_t runs = ckpt_runs(cols);
  const int grid = grid_for(rows * runs, sm_count);
  if (fp32)
    pack_kernel<<<grid, 256, 0, st>>>(rows, cols, runs, static_cast<const float*>(src), codes,
                                      scale);
  else
    pack_kernel<<<grid, 256, 0, st>>>(rows, cols, runs, static_cast<const bf*>(src), codes, scale);
  PKM_COUNT(1);
  return cudaGetLastError();
}

cudaError_t launch_ckpt8_unpack(int64_t rows, int cols, bool fp32, const int8_t* codes,
                                const float* scale, void* dst, int sm_count, cudaStream_t st) {
  const int64_t runs = ckpt_runs(cols);
  const int grid = grid_for(rows * runs, sm_count);
  if (fp32)
    unpack_kernel<<<grid, 256, 0, st>>>(rows, cols, runs, codes, scale, static_cast<float*>(dst));
  else
    unpack_kernel<<<grid, 256, 0, st>>>(rows, cols, runs, codes, scale, static_cast<bf*>(dst));
  PKM_COUNT(1);
  return cudaGetLastError();
}

}  // namespace pkm
