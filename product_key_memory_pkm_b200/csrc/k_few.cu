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
//   4-bit   a word is 8 neighbouring codes of one row; spread over 16-bit halves, 0x4300 | code
//           is the bf16 number 128 + code, from which 136 is taken (exact).  Products of codes
//           with bf16 x are exact; the products of a word's 32 columns (four lanes) are summed
//           in fp32 and then scaled by their group's scale in fp32.
//   bf16    a lane's 16 bytes are 8 columns of one row.
//
// A CTA's 8 warps split k for 16 output rows and add up through shared memory; where the rows
// are too few to fill the SMs, 2 or 4 CTAs of a cluster split k further and add up through
// distributed shared memory.  Every sum has a fixed order.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

using bf = __nv_bfloat16;

constexpr int kWarps = 8, kTpb = 32 * kWarps;
constexpr int kRows = 16;   // output rows of a CTA

// (Not volatile: the compiler may interleave independent products.)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The codes of a word as pairs (0,1) (2,3) (4,5) (6,7) of bf16 numbers code - 8.
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t odd = w >> 4;
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = (__byte_perm(w, odd, i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12)) &
                        0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), off);
    p[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// The products of a word start from zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// ------------------------------------------------------------------ weights
// Weights of one unit for this lane's two rows (g and g + 8 of a tile of 16).
//
// 4-bit: a unit is 32 * WORDS columns of one group: 128 where groups are whole multiples of
// that, else 64, else 32, so that one scale serves it.  The lane holds the 8 * WORDS neighbouring
// columns from 8 * WORDS * c, as one load.
struct W4Shape {
  int d_in, d_out, ng;
  uint32_t magic;  // for the quotient by a group's length in units: see group_of
  static int words(int group) { return group % 128 == 0 ? 4 : group % 64 == 0 ? 2 : 1; }
  static W4Shape of(int d_in, int d_out, int group) {
    const uint32_t per = (uint32_t)(group / (32 * words(group)));
    return W4Shape{d_in, d_out, w4_groups(d_in, group),
                   per == 1 ? 0u : (uint32_t)(((uint64_t)1 << 32) / per + 1)};
  }
  // i / per for i < 2^15: magic is above 2^32 / per by 1 at most, which adds i / 2^32 < 2^-17 to
  // the quotient, and that is 1 / per >= 2^-15 below the next integer, or i / per <= 1 - 2^-15.
  __device__ int group_of(int i) const { return magic ? (int)__umulhi((uint32_t)i, magic) : i; }
};
template <int WORDS>
struct W4Unit {
  static constexpr int kCols = 32 * WORDS, kWords = WORDS;
  uint32_t w[2][WORDS];
  uint32_t s[2];  // the scales' bits, not packed: packing would wait for the loads

  struct Src {
    const uint8_t* codes;
    const unsigned short* scale;
    int next_c, next_s;  // from row g to row g + 8, in bytes and in scales
    __device__ Src(const W4Mat& W, const W4Shape& sh, int o0, int g, int c) {
      // rows past the last are read as the last and not stored
      const int64_t o = min(o0 + g, sh.d_out - 1);
      const int to = min(o0 + g + 8, sh.d_out - 1) - (int)o;
      codes = W.codes + o * (sh.d_in / 2) + 4 * WORDS * c;
      scale = reinterpret_cast<const unsigned short*>(W.scale) + o * sh.ng;
      next_c = to * (sh.d_in / 2);
      next_s = to * sh.ng;
    }
  };
  // Lanes 2 and 3 take four words in the order 1, 0, 3, 2, so that the four lanes' columns of x lie
  // in different banks of shared memory (which columns meet in one instruction is of no
  // consequence).  The choice is made where a word is used: at the load it would wait for it.
  __device__ static bool swapped(int c) { return WORDS == 4 && (c & 2); }
  __device__ static int col(int u, int c, int j) {
    return u * kCols + 8 * WORDS * c + 8 * (swapped(c) ? j ^ 1 : j);
  }
  __device__ void load(const Src& S, const W4Shape& sh, int u, int c) {
    // a lane past the row's end reads within the row: its x is zero, and no code is NaN
    const int at = u * (kCols / 2);
    const uint8_t* p = S.codes + (u * kCols + 8 * WORDS * c < sh.d_in ? at : -4 * WORDS * c);
    const unsigned short* q = S.scale + sh.group_of(u);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (WORDS == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[r][0] = v.x; w[r][1] = v.y; w[r][2] = v.z; w[r][3] = v.w;
      } else if constexpr (WORDS == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[r][0] = v.x; w[r][1] = v.y;
      } else {
        w[r][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
      s[r] = __ldg(q);
      p += S.next_c;
      q += S.next_s;
    }
  }
  // The A operands of word j.
  struct A {
    uint32_t g[4], h[4];
  };
  __device__ A operands(int c, int j) const {
    constexpr int x = WORDS == 4 ? 1 : 0;
    A o;
    w4_pairs(swapped(c) ? w[0][j ^ x] : w[0][j], o.g);
    w4_pairs(swapped(c) ? w[1][j ^ x] : w[1][j], o.h);
    return o;
  }
  // t = a word's products with 8 tokens, x their columns; then acc += scale * t
  __device__ static void mac(float (&t)[4], const A& o, const uint4& x) {
    mma16816_first(t, o.g[0], o.h[0], o.g[1], o.h[1], x.x, x.y);
    mma16816(t, o.g[2], o.h[2], o.g[3], o.h[3], x.z, x.w);
  }
  __device__ void close(float (&acc)[4], const float (&t)[4]) const {
    const float sg = __uint_as_float(s[0] << 16), sh = __uint_as_float(s[1] << 16);
    acc[0] = fmaf(sg, t[0], acc[0]);
    acc[1] = fmaf(sg, t[1], acc[1]);
    acc[2] = fmaf(sh, t[2], acc[2]);
    acc[3] = fmaf(sh, t[3], acc[3]);
  }
};

// bf16: a unit is 64 columns, as two halves of 8 columns per lane.
struct W16Shape {
  int d_in, d_out;
  static W16Shape of(int d_in, int d_out, int) { return W16Shape{d_in, d_out}; }
};
struct W16Unit {
  static constexpr int kCols = 64, kWords = 2;
  uint4 w[2][2];  // [row][half]

  struct Src {
    const bf* row;
    int64_t next;
    __device__ Src(const bf* W, const W16Shape& sh, int o0, int g, int c) {
      const int64_t o = min(o0 + g, sh.d_out - 1), p = min(o0 + g + 8, sh.d_out - 1);
      row = W + o * sh.d_in + 8 * c;
      next = (p - o) * sh.d_in;
    }
  };
  __device__ static int col(int u, int c, int j) { return u * kCols + 32 * j + 8 * c; }
  __device__ void load(const Src& S, const W16Shape& sh, int u, int c) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[r][j] = col(u, c, j) < sh.d_in
                      ? __ldcs(reinterpret_cast<const uint4*>(S.row + (r ? S.next : 0) + u * kCols + 32 * j))
                      : make_uint4(0, 0, 0, 0);
  }
  struct A {
    uint4 g, h;
  };
  __device__ A operands(int, int j) const { return A{w[0][j], w[1][j]}; }
  __device__ static void mac(float (&t)[4], const A& o, const uint4& x) {
    mma16816_first(t, o.g.x, o.h.x, o.g.y, o.h.y, x.x, x.y);
    mma16816(t, o.g.z, o.h.z, o.g.w, o.h.w, x.z, x.w);
  }
  __device__ void close(float (&acc)[4], const float (&t)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += t[i];
  }
};
struct W4Of {
  using Mat = W4Mat;
  using Shape = W4Shape;
};
struct W16Of {
  using Mat = const bf*;
  using Shape = W16Shape;
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
// M: blocks of 16 rows of a CTA's tile: one, two (a matrix of many rows: x is read once for
// both), or for the gate one of each matrix.
// Units a warp has in flight, and the CTAs an SM holds: few units and several CTAs, so that
// the CTAs of one grid are resident together and none waits for another's last loads (one
// token, 1600 x 6400 x 1600 in bf16, whole calls: 18 us, on the device 14.4; whole calls with two
// units and 2 CTAs 24, with four units and 1 CTA 32).
template <class Unit, int M, int NT>
struct Depth {  // 4-bit: 8 words per row and matrix in flight, 4 for the two of a gate
  static constexpr int wide = 8 / M / Unit::kWords;
  static constexpr int batch = M * NT > 4 || wide < 1 ? 1 : wide;
  static constexpr int ctas = M * NT <= 2 ? 3 : NT <= 4 ? 2 : 1;
};
template <int M, int NT>
struct Depth<W16Unit, M, NT> {
  static constexpr int batch = M == 2 ? 1 : 2, ctas = M * NT > 2 ? 2 : 3;
};

template <class Unit, class Mat, class Shape, int M, int NT, Few OUT, int ACT>
__global__ void __launch_bounds__(kTpb, Depth<Unit, M, NT>::ctas)
    few_kernel(int N, Shape sh, int ks, const bf* x, Mat W0, Mat W1, void* out, bool first) {
  const int d_in = sh.d_in, d_out = sh.d_out;
  constexpr int kTileRows = OUT == Few::kGate ? kRows : M * kRows;
  constexpr int kNext = OUT == Few::kGate ? 0 : kRows;  // rows from the first block to the second
  constexpr int T = NT * 8, kBatch = Depth<Unit, M, NT>::batch;
  // a slot per warp, or per two warps where 8 would pass the static limit of 48 KiB
  constexpr int kSlots = M * NT <= 8 ? kWarps : kWarps / 2;
  __shared__ float part[M][kSlots][T][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rank = ks > 1 ? (int)blockIdx.x % ks : 0;
  const int tiles = (d_out + kTileRows - 1) / kTileRows, stride = (int)gridDim.x / ks;
  const int units = (d_in + Unit::kCols - 1) / Unit::kCols;
  const int step = kWarps * ks, u0 = rank * kWarps + warp;  // units u0, u0 + step, ...
  int tile = (int)blockIdx.x / ks;

  typename Unit::Src s0(W0, sh, tile * kTileRows, g, c), s1(W1, sh, tile * kTileRows + kNext, g, c);
  Unit w[M][kBatch];
  const auto fetch = [&](int u) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (u + b * step < units) {
        w[0][b].load(s0, sh, u + b * step, c);
        if (M == 2) w[M - 1][b].load(s1, sh, u + b * step, c);
      }
  };
  // Blocks past the last token repeat it: a column of the products that is not stored may hold
  // anything, since columns do not mix.
  const bf* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xp[n] = x + (int64_t)min(n * 8 + g, N - 1) * d_in;

  // Weights do not depend on the kernel before, x of the second product does: that kernel may still
  // be writing it while this one runs up to the wait.  So x is not __restrict__: loads of such a
  // pointer to const may take the read-only path, whose data may not change while a kernel runs,
  // and may be moved ahead of the wait.
  fetch(u0);
  if (first)
    allow_dependent_launch();
  else
    grid_dependency_wait();
  for (; tile < tiles; tile += stride) {
    const int o0 = tile * kTileRows;
    float acc[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.f;
    for (int u = u0; u < units; u += kBatch * step) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (u + b * step >= units) break;
        const int v = u + b * step;
        const auto products = [&](auto edge) {  // edge: the row ends within the unit
#pragma unroll
          for (int j = 0; j < Unit::kWords; ++j) {
            typename Unit::A a[M];
#pragma unroll
            for (int m = 0; m < M; ++m) a[m] = w[m][b].operands(c, j);
            const int k = Unit::col(v, c, j);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint4 xv = make_uint4(0, 0, 0, 0);
              if (!decltype(edge)::value || k < d_in) xv = *reinterpret_cast<const uint4*>(xp[n] + k);
#pragma unroll
              for (int m = 0; m < M; ++m) {
                float p[4];  // scaled word by word: the words' chains are independent
                Unit::mac(p, a[m], xv);
                w[m][b].close(acc[m][n], p);
              }
            }
          }
        };
        if ((v + 1) * Unit::kCols > d_in) products(std::true_type{}); else products(std::false_type{});
      }
      fetch(u + kBatch * step);
    }
    if (tile + stride < tiles) {  // the next tile's first weights travel beside this one's sums
      s0 = typename Unit::Src(W0, sh, o0 + stride * kTileRows, g, c);
      s1 = typename Unit::Src(W1, sh, o0 + stride * kTileRows + kNext, g, c);
      fetch(u0);
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
    const auto own_sum = [&](int m, int n, int r) {
      float s = part[m][0][n][r];
#pragma unroll
      for (int q = 1; q < kSlots; ++q) s += part[m][q][n][r];
      return s;
    };
    if (ks > 1) {
      for (int e = threadIdx.x; e < M * N * kRows; e += kTpb) {
        const int m = e / (N * kRows), n = e / kRows % N, r = e % kRows;
        part[m][0][n][r] = own_sum(m, n, r);
      }
      __syncwarp();
      cluster_sync();
    }
    // each CTA of a cluster finishes its share of the elements
    for (int e = threadIdx.x + rank * kTpb; e < N * kRows; e += kTpb * ks) {
      const int n = e / kRows, r = e % kRows;
      float s[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if (ks > 1) {
          const uint32_t a = smem_addr(&part[m][0][n][r]);
          s[m] = peer_load(a, 0);
          for (int q = 1; q < ks; ++q) s[m] += peer_load(a, q);
        } else {
          s[m] = own_sum(m, n, r);
        }
      }
      if (OUT == Few::kGate) s[0] = act_fn<ACT>(s[0]) * s[M - 1];
#pragma unroll
      for (int m = 0; m < (OUT == Few::kGate ? 1 : M); ++m) {
        const int o = o0 + m * kRows + r;
        const int64_t at = (int64_t)n * d_out + o;
        if (o >= d_out) continue;
        if (OUT == Few::kF32)
          static_cast<float*>(out)[at] = s[m];
        else
          static_cast<bf*>(out)[at] = __float2bfloat16_rn(s[m]);
      }
    }
    // the sums are read before they are written again, or before a CTA of the cluster leaves
    if (ks > 1) {
      __syncwarp();
      cluster_sync();
    } else if (tile + stride < tiles) {
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ many rows
// Many output rows: what bounds few_kernel there is not the weights but every 16 rows reading all
// of x again, and their sums over warps.  Here a CTA per SM keeps x (or a chunk of its columns) in
// shared memory and each of its warps takes 16 rows through all of k.  Rows are dealt so that they
// fill whole rounds of the SMs with as many warps as fit, up to 24: a warp's products depend on
// one another, and other warps and kWideIlp products at a time fill the gaps.  Against 50264 x
// 1600, whole calls: 24 us for 16 tokens (few_kernel 39), 33 for 32 (89), 55 for 64 (140; on the
// device 48 with the weights in L2, 53 from HBM); for 8 tokens both take 20 to 24, so those stay
// there.  The weights alone would take 6.6 us.  At 64 tokens instructions issue in 51 % of the
// cycles, the tensor pipe works in 38 %, and every 16 rows' reading of x keeps the shared-memory
// port busy for 41 %; the rest is the latency of a warp's chain.
constexpr int kWideRows = 16, kWideWarps = 24, kWideIlp = 2;
constexpr int kWideSmem = 225 * 1024;

// 16 bytes global -> shared without registers; zeros when !has.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool has) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(has ? 16 : 0)
               : "memory");
}

__host__ __device__ constexpr int wide_pad(int words) { return words == 1 ? 64 : words == 2 ? 16 : 32; }

template <int WORDS, int NT>
__global__ void __launch_bounds__(32 * kWideWarps, 1)
    wide_kernel(int N, W4Shape sh, int chunk, const bf* __restrict__ x, W4Mat W,
                float* __restrict__ y) {
  using Unit = W4Unit<WORDS>;
  constexpr int T = NT * 8, kIlp = kWideIlp;
  constexpr int kAhead = NT == 8 ? 1 : 2;  // units requested before their use, as registers allow
  extern __shared__ __align__(16) unsigned char xs[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // The 8 lanes that read 16 bytes at a time are two rows' four columns 16 * WORDS bytes apart (4
  // words: two pairs of neighbours, see Unit::col): a pitch of 64, 16, 32 bytes past a multiple of
  // 128 keeps them on different banks for 1, 2, 4 words.
  const int pitch = chunk * 2 + wide_pad(WORDS);
  const int tiles = (sh.d_out + kWideRows - 1) / kWideRows;
  const int chunks = (sh.d_in + chunk - 1) / chunk;
  for (int first = 0; first < tiles; first += gridDim.x * warps) {  // a round, same for all CTAs
    const int tile = first + warp * gridDim.x + blockIdx.x;
    const bool mine = tile < tiles;
    const typename Unit::Src src(W, sh, tile * kWideRows, g, c);
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
    for (int ch = 0; ch < chunks; ++ch) {
      const int k0 = ch * chunk, cols = min(chunk, sh.d_in - k0);
      const int u0 = k0 / Unit::kCols, u1 = u0 + (cols + Unit::kCols - 1) / Unit::kCols;
      Unit w[kAhead];  // units u0 .., kAhead ahead of their use
      const auto fetch = [&](int slot, int u) {
        if (u < u1) w[slot].load(src, sh, u, c);
      };
      if (mine) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i, u0 + i);
      }
      if (first == 0 || chunks > 1) {
        if (ch > 0 || first > 0) __syncthreads();  // the chunk before has been read
        const int blocks = (u1 - u0) * (Unit::kCols / 8);  // 8-column blocks, whole units
        for (int n = warp; n < T; n += warps) {
          const uint32_t dst = smem_addr(xs + n * pitch);
          const bf* src = x + (int64_t)min(n, N - 1) * sh.d_in + k0;
          for (int b = lane; b < blocks; b += 32)
            copy16(dst + b * 16, src + (b * 8 < cols ? b * 8 : 0), n < N && b * 8 < cols);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
      }
      if (!mine) continue;
      const unsigned char* xb = xs + g * pitch;
      for (int u = u0; u < u1; u += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (u + i >= u1) break;
#pragma unroll
          for (int j = 0; j < WORDS; ++j) {
            const typename Unit::A a = w[i].operands(c, j);
            const unsigned char* xj = xb + Unit::col(u + i - u0, c, j) * 2;
            // scaled word by word: no registers for the sums of a whole unit; kIlp products at a
            // time, since each waits for the one before it
#pragma unroll
            for (int t = 0; t < NT; t += kIlp) {
              float p[kIlp][4];
              uint4 xv[kIlp];
#pragma unroll
              for (int e = 0; e < kIlp; ++e)
                xv[e] = *reinterpret_cast<const uint4*>(xj + (t + e) * 8 * pitch);
#pragma unroll
              for (int e = 0; e < kIlp; ++e)
                mma16816_first(p[e], a.g[0], a.h[0], a.g[1], a.h[1], xv[e].x, xv[e].y);
#pragma unroll
              for (int e = 0; e < kIlp; ++e)
                mma16816(p[e], a.g[2], a.h[2], a.g[3], a.h[3], xv[e].z, xv[e].w);
#pragma unroll
              for (int e = 0; e < kIlp; ++e) w[i].close(acc[t + e], p[e]);
            }
          }
          fetch(i, u + i + kAhead);
        }
      }
    }
    if (!mine) continue;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = t * 8 + 2 * c + (i & 1), o = tile * kWideRows + g + 8 * (i >> 1);
        if (n < N && o < sh.d_out) y[(int64_t)n * sh.d_out + o] = acc[t][i];
      }
  }
}

template <int WORDS, int NT>
cudaError_t launch_wide(int N, const W4Shape& sh, const bf* x, const W4Mat& W, float* y,
                        int sm_count, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(wide_kernel<WORDS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kWideSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  }
  const int pad = wide_pad(WORDS);
  const int most = (kWideSmem / (NT * 8) - pad) / 2 / 128 * 128;
  const int chunk = std::min((sh.d_in + 127) / 128 * 128, most);
  const int tiles = (sh.d_out + kWideRows - 1) / kWideRows;
  const int per_sm = (tiles + sm_count - 1) / sm_count;
  const int rounds = (per_sm + kWideWarps - 1) / kWideWarps;
  const int warps = (per_sm + rounds - 1) / rounds;
  wide_kernel<WORDS, NT><<<std::min(tiles, sm_count), 32 * warps,
                          (size_t)NT * 8 * (chunk * 2 + pad), st>>>(N, sh, chunk, x, W, y);
  PKM_COUNT(1);
  return cudaGetLastError();
}

// Rows enough that every SM has several warps.  1600 columns, few_kernel against this, us on the
// device:                  9 tokens     16 tokens    32 tokens    64 tokens
//    7104 rows         5.5   9.3    5.7   9.7   10.6  15.2   18.3  30.3
//    9472 (the limit)  8.1   8.9    8.4   9.3   11.0  14.5   23.9  29.3
//   12000              9.2  10.6    9.4  11.1   15.0  16.4   34.8  31.2
//   18944             13.0  10.6   13.2  10.9   19.8  16.2   45.9  31.8
//   33333             20.5  15.1   20.9  15.6   35.7  22.0   84.4  38.3
// They cross between 9472 and 18944 rows, so near the limit this is up to a third slower.
bool wide_form(int64_t N, int d_out, int sm_count) {
  return N > 8 && d_out >= 4 * kWideRows * sm_count;
}

// CTAs of a cluster along k: more while the grid leaves SMs empty and every warp still has
// two units.
int split_of(int tiles, int d_in, int unit, int sm_count) {
  const int units = (d_in + unit - 1) / unit;
  int ks = 1;
  while (ks < 4 && tiles * ks < 2 * sm_count && units >= 2 * kWarps * 2 * ks) ks *= 2;
  return ks;
}

template <class Unit, class Of, int M, int NT, Few OUT, int ACT>
cudaError_t launch_m(int N, const typename Of::Shape& sh, const bf* x, const typename Of::Mat& W0,
                   const typename Of::Mat& W1, void* out, bool first, int sm_count,
                   cudaStream_t st) {
  const auto kernel = few_kernel<Unit, typename Of::Mat, typename Of::Shape, M, NT, OUT, ACT>;
  constexpr int kTileRows = OUT == Few::kGate ? kRows : M * kRows;
  const int tiles = (sh.d_out + kTileRows - 1) / kTileRows;
  const int ks = split_of(tiles, sh.d_in, Unit::kCols, sm_count);
  cudaLaunchConfig_t cfg = {};
  constexpr int kCtas = Depth<Unit, M, NT>::ctas;
  cfg.gridDim = dim3((unsigned)(std::min(tiles, std::max(1, kCtas * sm_count / ks)) * ks));
  cfg.blockDim = dim3(kTpb);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (ks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = ks;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (!first) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, N, sh, ks, x, W0, W1, out, first);
  PKM_COUNT(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Two blocks of rows per tile where even so every SM gets several tiles.  (For fp32 results of
// more than 8 tokens that is where wide_form holds.)
template <class Unit, class Of, int NT, Few OUT, int ACT>
cudaError_t launch(int N, const typename Of::Shape& sh, const bf* x, const typename Of::Mat& W0,
                   const typename Of::Mat& W1, void* out, bool first, int sm_count,
                   cudaStream_t st) {
  if constexpr (OUT == Few::kGate) {
    return launch_m<Unit, Of, 2, NT, OUT, ACT>(N, sh, x, W0, W1, out, first, sm_count, st);
  } else {
    if constexpr (NT == 1 || (NT == 2 && OUT == Few::kBf16)) {
      if (sh.d_out >= 2 * kRows * 4 * sm_count)
        return launch_m<Unit, Of, 2, NT, OUT, ACT>(N, sh, x, W0, W1, out, first, sm_count, st);
    }
    return launch_m<Unit, Of, 1, NT, OUT, ACT>(N, sh, x, W0, W1, out, first, sm_count, st);
  }
}

template <class Unit, class Of, Few OUT, int ACT, int MAXT>
cudaError_t by_tokens(int64_t N, const typename Of::Shape& sh, const bf* x,
                      const typename Of::Mat& W0, const typename Of::Mat& W1, void* out,
                      bool first, int sm_count, cudaStream_t st) {
  const int n = (int)N;
  if (N <= 8) return launch<Unit, Of, 1, OUT, ACT>(n, sh, x, W0, W1, out, first, sm_count, st);
  if (N <= 16) return launch<Unit, Of, 2, OUT, ACT>(n, sh, x, W0, W1, out, first, sm_count, st);
  if constexpr (MAXT > 16) {
    if (N <= 32) return launch<Unit, Of, 4, OUT, ACT>(n, sh, x, W0, W1, out, first, sm_count, st);
    return launch<Unit, Of, 8, OUT, ACT>(n, sh, x, W0, W1, out, first, sm_count, st);
  }
  return cudaErrorInvalidValue;
}

template <Few OUT, int ACT>
cudaError_t w4(int64_t N, int d_in, int d_out, int group, const bf* x, const W4Mat& W0,
               const W4Mat& W1, void* out, bool first, int sm_count, cudaStream_t st) {
  const W4Shape sh = W4Shape::of(d_in, d_out, group);
  switch (W4Shape::words(group)) {
    case 4: return by_tokens<W4Unit<4>, W4Of, OUT, ACT, 64>(N, sh, x, W0, W1, out, first, sm_count, st);
    case 2: return by_tokens<W4Unit<2>, W4Of, OUT, ACT, 64>(N, sh, x, W0, W1, out, first, sm_count, st);
    default: return by_tokens<W4Unit<1>, W4Of, OUT, ACT, 64>(N, sh, x, W0, W1, out, first, sm_count, st);
  }
}

template <int WORDS>
cudaError_t wide(int N, const W4Shape& sh, const bf* x, const W4Mat& W, float* y, int sm_count,
                 cudaStream_t st) {
  if (N <= 16) return launch_wide<WORDS, 2>(N, sh, x, W, y, sm_count, st);
  return N <= 32 ? launch_wide<WORDS, 4>(N, sh, x, W, y, sm_count, st)
                 : launch_wide<WORDS, 8>(N, sh, x, W, y, sm_count, st);
}

}  // namespace

cudaError_t launch_w4_matvec(int64_t N, int d_in, int d_out, int group, const void* x,
                             const W4Mat& W, float* y, int sm_count, cudaStream_t st) {
  const bf* xb = static_cast<const bf*>(x);
  if (!wide_form(N, d_out, sm_count))
    return w4<Few::kF32, 0>(N, d_in, d_out, group, xb, W, W, y, true, sm_count, st);
  const W4Shape sh = W4Shape::of(d_in, d_out, group);
  switch (W4Shape::words(group)) {
    case 4: return wide<4>((int)N, sh, xb, W, y, sm_count, st);
    case 2: return wide<2>((int)N, sh, xb, W, y, sm_count, st);
    default: return wide<1>((int)N, sh, xb, W, y, sm_count, st);
  }
}

cudaError_t launch_w4_ffn(const FfnPlan& p, int group, const void* x, const W4Mat& Wg,
                          const W4Mat& Wu, const W4Mat& Wd, void* y, void* ws, cudaStream_t st) {
  const bf* xb = static_cast<const bf*>(x);
  const cudaError_t e =
      p.act == PKM_ACT_GELU
          ? w4<Few::kGate, PKM_ACT_GELU>(p.N, p.d_in, p.d_ff, group, xb, Wg, Wu, ws, true, p.sm_count, st)
          : w4<Few::kGate, PKM_ACT_SILU>(p.N, p.d_in, p.d_ff, group, xb, Wg, Wu, ws, true, p.sm_count, st);
  if (e != cudaSuccess) return e;
  return w4<Few::kBf16, 0>(p.N, p.d_ff, p.d_out, group, static_cast<const bf*>(ws), Wd, Wd, y,
                           false, p.sm_count, st);
}

cudaError_t launch_ffn_few(const FfnPlan& p, const void* x, const void* Wg, const void* Wu,
                           const void* Wd, void* y, void* ws, cudaStream_t st) {
  const bf *xb = static_cast<const bf*>(x), *g = static_cast<const bf*>(Wg),
           *u = static_cast<const bf*>(Wu), *o = static_cast<const bf*>(Wd);
  constexpr int kMost = (int)kFfnFewTokens;
  const W16Shape in = W16Shape::of(p.d_in, p.d_ff, 0), back = W16Shape::of(p.d_ff, p.d_out, 0);
  const cudaError_t e =
      p.act == PKM_ACT_GELU
          ? by_tokens<W16Unit, W16Of, Few::kGate, PKM_ACT_GELU, kMost>(p.N, in, xb, g, u, ws, true, p.sm_count, st)
          : by_tokens<W16Unit, W16Of, Few::kGate, PKM_ACT_SILU, kMost>(p.N, in, xb, g, u, ws, true, p.sm_count, st);
  if (e != cudaSuccess) return e;
  return by_tokens<W16Unit, W16Of, Few::kBf16, 0, kMost>(p.N, back, static_cast<const bf*>(ws), o, o,
                                                         y, false, p.sm_count, st);
}

}  // namespace pkm
