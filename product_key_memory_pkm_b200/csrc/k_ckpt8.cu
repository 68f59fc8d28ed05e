// 8-bit activation checkpoints: a run of 32 columns of a row shares one fp32 scale.
//
// Bound by HBM: pack reads 2 or 4 bytes per value and writes 1.125, unpack the other way
// round.  A thread takes 8 neighbouring columns (one or two 16-byte accesses on the wide side, 8
// bytes of codes), four threads share a run and find its largest magnitude with two shuffles,
// and a thread has kUnroll such chunks in flight.  16384 x 6400: bf16 unpack 51 us (6.4 TB/s),
// pack 62 to 64 us (5.2 TB/s; it issues instructions in 77 % of the cycles, 118 per chunk, of
// which the exact halves cost 3 per value); fp32 pack 80 us (6.7 TB/s), unpack 127 us (4.2 TB/s).
#include <type_traits>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

using bf = __nv_bfloat16;
constexpr int kTpb = 256, kUnroll = 4;

template <typename T>
struct Chunk;  // 8 values of the wide side
template <>
struct Chunk<bf> {
  uint4 q;
  __device__ void load(const bf* p) { q = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ void floats(float (&v)[8]) const { bf16x8_to_f32(q, v); }
  __device__ uint32_t top() const {  // two 16-bit magnitudes at a time
    constexpr uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(q.x & m, q.y & m), __vmaxu2(q.z & m, q.w & m));
    return max(t << 16, t & 0xffff0000u);
  }
  __device__ static void store(bf* p, const float (&v)[8]) {
    uint4 o;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = o;
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void floats(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ uint32_t top() const {
    return max(max(max(mag_bits(a.x), mag_bits(a.y)), max(mag_bits(a.z), mag_bits(a.w))),
               max(max(mag_bits(b.x), mag_bits(b.y)), max(mag_bits(b.z), mag_bits(b.w))));
  }
  __device__ static void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Offset on the wide side of chunk c (8 columns of a padded row of per_row chunks), or -1
// behind the row's last column.  FLAT: rows are whole runs, so both sides are one sequence.
template <bool FLAT>
__device__ __forceinline__ int64_t wide_offset(int64_t c, int per_row, int cols) {
  if (FLAT) return c * 8;
  const int64_t row = c / per_row;
  const int col = (int)(c - row * per_row) * 8;
  return col < cols ? row * cols + col : -1;
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kTpb) pack_kernel(int64_t chunks, int per_row, int cols,
                                                    const T* src, int8_t* codes, float* scale) {
  // chunks is a multiple of 4, so the four threads of a run are in or out together
  const int64_t base = (int64_t)blockIdx.x * (kTpb * kUnroll) + threadIdx.x;
  Chunk<T> in[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t c = base + i * kTpb;
    const int64_t o = c < chunks ? wide_offset<FLAT>(c, per_row, cols) : -1;
    in[i].zero();
    if (o >= 0) in[i].load(src + o);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t c = base + i * kTpb;
    float v[8];
    in[i].floats(v);
    uint32_t top = in[i].top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const CkptScale s = ckpt_scale<std::is_same<T, bf>::value>(top);
    uint32_t w[2];
    ckpt_codes<std::is_same<T, bf>::value>(v, s, w);
    if (c < chunks) {
      *reinterpret_cast<uint2*>(codes + c * 8) = make_uint2(w[0], w[1]);
      if ((threadIdx.x & 3) == 0) scale[c >> 2] = s.scale;
    }
  }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kTpb) unpack_kernel(int64_t chunks, int per_row, int cols,
                                                      const int8_t* codes, const float* scale,
                                                      T* dst) {
  const int64_t base = (int64_t)blockIdx.x * (kTpb * kUnroll) + threadIdx.x;
  uint2 q[kUnroll];
  float s[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t c = base + i * kTpb;
    q[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (c < chunks) {
      q[i] = __ldcs(reinterpret_cast<const uint2*>(codes + c * 8));
      s[i] = __ldg(scale + (c >> 2));
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t c = base + i * kTpb;
    const int64_t o = c < chunks ? wide_offset<FLAT>(c, per_row, cols) : -1;
    float a[4], b[4], v[8];
    ckpt_floats4(q[i].x, a);
    ckpt_floats4(q[i].y, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j] * s[i];
      v[4 + j] = b[j] * s[i];
    }
    if (o >= 0) Chunk<T>::store(dst + o, v);
  }
}

unsigned blocks_of(int64_t chunks) {
  return (unsigned)((chunks + kTpb * kUnroll - 1) / (kTpb * kUnroll));
}

template <typename T>
cudaError_t pack(int64_t rows, int cols, const void* src, int8_t* codes, float* scale,
                 cudaStream_t st) {
  const int per_row = 4 * (int)ckpt_runs(cols);
  const int64_t chunks = rows * per_row;
  const T* s = static_cast<const T*>(src);
  if (cols % kCkptRun == 0)
    pack_kernel<T, true><<<blocks_of(chunks), kTpb, 0, st>>>(chunks, per_row, cols, s, codes, scale);
  else
    pack_kernel<T, false><<<blocks_of(chunks), kTpb, 0, st>>>(chunks, per_row, cols, s, codes, scale);
  PKM_COUNT(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t unpack(int64_t rows, int cols, const int8_t* codes, const float* scale, void* dst,
                   cudaStream_t st) {
  const int per_row = 4 * (int)ckpt_runs(cols);
  const int64_t chunks = rows * per_row;
  T* d = static_cast<T*>(dst);
  if (cols % kCkptRun == 0)
    unpack_kernel<T, true><<<blocks_of(chunks), kTpb, 0, st>>>(chunks, per_row, cols, codes, scale, d);
  else
    unpack_kernel<T, false><<<blocks_of(chunks), kTpb, 0, st>>>(chunks, per_row, cols, codes, scale, d);
  PKM_COUNT(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt8_pack(int64_t rows, int cols, bool fp32, const void* src, int8_t* codes,
                              float* scale, cudaStream_t st) {
  return fp32 ? pack<float>(rows, cols, src, codes, scale, st)
              : pack<bf>(rows, cols, src, codes, scale, st);
}

cudaError_t launch_ckpt8_unpack(int64_t rows, int cols, bool fp32, const int8_t* codes,
                                const float* scale, void* dst, cudaStream_t st) {
  return fp32 ? unpack<float>(rows, cols, codes, scale, dst, st)
              : unpack<bf>(rows, cols, codes, scale, dst, st);
}

}  // namespace pkm
