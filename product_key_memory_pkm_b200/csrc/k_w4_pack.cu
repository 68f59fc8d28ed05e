// 4-bit weights: packing a bf16 matrix (once per matrix) and unpacking it (once per prompt of more
// tokens than the products take).  Bound by instructions, not by HBM: 50264 x 1600 takes 285 us to
// pack and 143 to unpack where the bytes would take 31; they issue in 71 and 63 % of the cycles, on
// a division per value and a 64-bit division per byte, with 2-byte accesses.
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

int grid_for(int64_t warps, int sm_count) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8, sm_count * 8));
}

}  // namespace

cudaError_t launch_w4_pack(int d_out, int d_in, int group, const void* W, uint8_t* codes,
                           void* scale, cudaStream_t st) {
  const int ng = w4_groups(d_in, group);
  w4_pack_kernel<<<grid_for((int64_t)d_out * ng, 148), 256, 0, st>>>(
      d_out, d_in, group, ng, static_cast<const bf*>(W), codes, static_cast<bf*>(scale));
  PKM_COUNT(1);
  return cudaGetLastError();
}

cudaError_t launch_w4_unpack(int d_out, int d_in, int group, const W4Mat& W, void* out,
                             cudaStream_t st) {
  const int ng = w4_groups(d_in, group);
  w4_unpack_kernel<<<grid_for((int64_t)d_out * d_in / 64 + 1, 148), 256, 0, st>>>(
      d_out, d_in, group, ng, W.codes, W.scale, static_cast<bf*>(out));
  PKM_COUNT(1);
  return cudaGetLastError();
}

}  // namespace pkm
