// C ABI entry points of the gated feed-forward block, the 8-bit activation checkpoints and the
// 4-bit weight products: host-side validation, plan, launch sequencing.
#include <algorithm>

#include "ffn_internal.cuh"

namespace pkm {
namespace {

// Widths and token counts the kernels' 32-bit coordinates and grids are laid out for.  A weight
// gradient's tile sums over all tokens, 64 to a k-block of about 700 cycles, while its epilogue
// waits: 2^26 tokens keep that wait under half of its bound of 2e9 cycles.
constexpr int kMaxWidth = 1 << 20;
constexpr int64_t kMaxTokens = (int64_t)1 << 26;
constexpr int64_t kMaxTokensSimt = (int64_t)1 << 22;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define PKM_TRY(expr)                  \
  do {                                 \
    pkm_status _s = (expr);            \
    if (_s != PKM_OK) return _s;       \
  } while (0)

#define PKM_NEED(ptr)                                                   \
  do {                                                                  \
    if (!(ptr) || !aligned16(ptr)) return PKM_ERR_INVALID_ARG;          \
  } while (0)

#define PKM_OPT(ptr)                                                    \
  do {                                                                  \
    if ((ptr) && !aligned16(ptr)) return PKM_ERR_INVALID_ARG;           \
  } while (0)

pkm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA; }

// Sizes and flags (the 4-bit block leaves d_out free, so the multiple-of-8 rule of the
// other calls is apart).
pkm_status validate_sizes(const pkm_ffn_dims* d) {
  if (!d) return PKM_ERR_INVALID_ARG;
  if (d->N < 0 || d->d_in <= 0 || d->d_ff <= 0 || d->d_out <= 0) return PKM_ERR_INVALID_ARG;
  if (d->act != PKM_ACT_SILU && d->act != PKM_ACT_GELU) return PKM_ERR_INVALID_ARG;
  if (d->flags & ~(PKM_F_FP32 | PKM_F_SIMT | PKM_FFN_CKPT8 | PKM_FFN_GRAD_BF16))
    return PKM_ERR_INVALID_ARG;
  if ((d->flags & PKM_F_FP32) && (d->flags & PKM_FFN_GRAD_BF16)) return PKM_ERR_INVALID_ARG;
  if (d->d_in > kMaxWidth || d->d_ff > kMaxWidth || d->d_out > kMaxWidth || d->N > kMaxTokens)
    return PKM_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits
  if (d->N * (int64_t)std::max(d->d_in, std::max(d->d_ff, d->d_out)) > (int64_t)1 << 44)
    return PKM_ERR_UNSUPPORTED;
  if ((d->flags & (PKM_F_FP32 | PKM_F_SIMT)) && d->N > kMaxTokensSimt) return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

pkm_status validate(const pkm_ffn_dims* d) {
  PKM_TRY(validate_sizes(d));
  if (d->d_in % 8 || d->d_ff % 8 || d->d_out % 8) return PKM_ERR_INVALID_ARG;
  return PKM_OK;
}

FfnPlan shape_plan(const pkm_ffn_dims* d) {
  FfnPlan p{};
  p.N = d->N;
  p.d_in = d->d_in;
  p.d_ff = d->d_ff;
  p.d_out = d->d_out;
  p.act = d->act;
  p.runs = ckpt_runs(d->d_ff);
  p.fp32 = d->flags & PKM_F_FP32;
  p.simt = d->flags & (PKM_F_FP32 | PKM_F_SIMT);
  p.ckpt8 = d->flags & PKM_FFN_CKPT8;
  p.grad_bf16 = d->flags & PKM_FFN_GRAD_BF16;
  return p;
}

pkm_status make_plan(const pkm_ffn_dims* d, FfnPlan* p) {
  DeviceInfo info;
  if (!current_device(&info)) return PKM_ERR_CUDA;
  *p = shape_plan(d);
  p->dev = info.dev;
  p->sm_count = info.sm_count;
  p->status = info.status;
  return PKM_OK;
}

size_t workspace_bytes_of(const FfnPlan& p, bool backward) {
  return p.simt ? ffn_simt_workspace(p, backward) : ffn_tc_workspace(p, backward);
}

pkm_status check_workspace(size_t need, const void* ws, size_t bytes) {
  if (need == 0) return PKM_OK;
  if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return PKM_ERR_WORKSPACE;
  return PKM_OK;
}

// A buffer of a call.  The kernels of one call read and write in no promised order, so its outputs
// (the first `outs` buffers; the workspace is one) may share no bytes with each other or with what
// it reads.
struct Span {
  const void* p;
  size_t n;
};
template <int COUNT>
pkm_status check_apart(const Span (&s)[COUNT], int outs) {
  for (int i = 0; i < outs; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p);
    for (int j = i + 1; j < COUNT; ++j) {
      const uintptr_t b = reinterpret_cast<uintptr_t>(s[j].p);
      if (a && b && (a <= b ? b - a < s[i].n : a - b < s[j].n)) return PKM_ERR_INVALID_ARG;
    }
  }
  return PKM_OK;
}
size_t w4_codes_bytes(int32_t d_out, int32_t d_in) { return (size_t)d_out * (d_in / 2); }
size_t w4_scale_bytes(int32_t d_out, int32_t d_in, int32_t group) {
  return (size_t)d_out * w4_groups(d_in, group) * 2;
}

pkm_status check_saved(const FfnPlan& p, const pkm_ffn_saved* s) {
  if (!s) return PKM_ERR_INVALID_ARG;
  PKM_NEED(s->g);
  PKM_NEED(s->u);
  if (p.ckpt8) {
    PKM_NEED(s->g_scale);
    PKM_NEED(s->u_scale);
  }
  return PKM_OK;
}

pkm_status validate_ckpt8(int64_t rows, int32_t cols, uint32_t flags) {
  if (rows < 0 || cols <= 0 || cols % 8 || (flags & ~PKM_F_FP32)) return PKM_ERR_INVALID_ARG;
  if (rows > ((int64_t)1 << 38)) return PKM_ERR_UNSUPPORTED;
  // grids of up to 2^31 - 1 blocks of 8192 values
  if (cols > kMaxWidth || rows * ckpt_runs(cols) > ((int64_t)1 << 38)) return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

pkm_status validate_w4(int32_t d_out, int32_t d_in, int32_t group) {
  if (d_out <= 0 || d_in <= 0 || d_in % 32 || group <= 0 || group % 32) return PKM_ERR_INVALID_ARG;
  if (d_out > kMaxWidth || d_in > kMaxWidth) return PKM_ERR_UNSUPPORTED;
  return PKM_OK;
}

pkm_status check_w4(const pkm_w4* W, W4Mat* m) {
  if (!W) return PKM_ERR_INVALID_ARG;
  PKM_NEED(W->codes);
  PKM_NEED(W->scale);
  *m = W4Mat{W->codes, static_cast<const __nv_bfloat16*>(W->scale)};
  return PKM_OK;
}

}  // namespace
}  // namespace pkm

using namespace pkm;

extern "C" {

size_t pkm_ffn_saved_bytes(const pkm_ffn_dims* d, int field) {
  if (validate(d) != PKM_OK) return 0;
  const FfnPlan p = shape_plan(d);
  switch (field) {
    case PKM_FFN_SAVED_G:
    case PKM_FFN_SAVED_U:
      return (size_t)(p.ckpt8 ? p.N * p.runs * kCkptRun : p.N * p.d_ff * (p.fp32 ? 4 : 2));
    case PKM_FFN_SAVED_G_SCALE:
    case PKM_FFN_SAVED_U_SCALE:
      return (size_t)(p.ckpt8 ? p.N * p.runs * 4 : 0);
    default: return 0;
  }
}

size_t pkm_ffn_workspace_bytes(const pkm_ffn_dims* d, int which) {
  if (validate_sizes(d) != PKM_OK || d->N == 0 || (which != PKM_FWD && which != PKM_BWD)) return 0;
  return workspace_bytes_of(shape_plan(d), which == PKM_BWD);
}

pkm_status pkm_ffn_forward(const pkm_ffn_dims* d, const void* x, const void* Wg, const void* Wu,
                           const void* Wd, void* y, const pkm_ffn_saved* saved, void* workspace,
                           size_t workspace_bytes, void* stream) {
  PKM_TRY(validate(d));
  if (d->N == 0) return PKM_OK;
  PKM_NEED(x); PKM_NEED(Wg); PKM_NEED(Wu); PKM_NEED(Wd); PKM_NEED(y);
  if (saved) PKM_TRY(check_saved(shape_plan(d), saved));
  const size_t need = pkm_ffn_workspace_bytes(d, PKM_FWD);
  PKM_TRY(check_workspace(need, workspace, workspace_bytes));
  const size_t e = d->flags & PKM_F_FP32 ? 4 : 2, in = (size_t)d->d_ff * d->d_in * e;
  const size_t kept = saved ? pkm_ffn_saved_bytes(d, PKM_FFN_SAVED_G) : 0;
  const size_t scales = saved ? pkm_ffn_saved_bytes(d, PKM_FFN_SAVED_G_SCALE) : 0;
  PKM_TRY(check_apart<10>({{y, (size_t)d->N * d->d_out * e},
                           {workspace, need},
                           {saved ? saved->g : nullptr, kept},
                           {saved ? saved->u : nullptr, kept},
                           {scales ? saved->g_scale : nullptr, scales},
                           {scales ? saved->u_scale : nullptr, scales},
                           {x, (size_t)d->N * d->d_in * e},
                           {Wg, in},
                           {Wu, in},
                           {Wd, (size_t)d->d_out * d->d_ff * e}}, 6));
  FfnPlan p;
  PKM_TRY(make_plan(d, &p));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!p.simt && !saved && p.N <= kFfnFewTokens)
    return cuda_status(launch_ffn_few(p, x, Wg, Wu, Wd, y, workspace, st));
  return cuda_status(p.simt
                         ? launch_ffn_fwd_simt(p, x, Wg, Wu, Wd, y, saved, workspace, st)
                         : launch_ffn_fwd_tc(p, x, Wg, Wu, Wd, y, saved, workspace, st));
}

pkm_status pkm_ffn_backward(const pkm_ffn_dims* d, const void* x, const void* Wg, const void* Wu,
                            const void* Wd, const pkm_ffn_saved* saved, const void* dy, void* dx,
                            void* dWg, void* dWu, void* dWd, void* workspace,
                            size_t workspace_bytes, void* stream) {
  PKM_TRY(validate(d));
  if (d->N == 0) return PKM_OK;
  PKM_NEED(x); PKM_NEED(Wg); PKM_NEED(Wu); PKM_NEED(Wd); PKM_NEED(dy);
  PKM_TRY(check_saved(shape_plan(d), saved));
  PKM_OPT(dx); PKM_OPT(dWg); PKM_OPT(dWu); PKM_OPT(dWd);
  const size_t need = pkm_ffn_workspace_bytes(d, PKM_BWD);
  PKM_TRY(check_workspace(need, workspace, workspace_bytes));
  const size_t e = d->flags & PKM_F_FP32 ? 4 : 2, ge = d->flags & PKM_FFN_GRAD_BF16 ? 2 : 4;
  const size_t xs = (size_t)d->N * d->d_in, in = (size_t)d->d_ff * d->d_in,
               out = (size_t)d->d_out * d->d_ff;
  const size_t kept = pkm_ffn_saved_bytes(d, PKM_FFN_SAVED_G);
  const size_t scales = pkm_ffn_saved_bytes(d, PKM_FFN_SAVED_G_SCALE);
  PKM_TRY(check_apart<14>({{dx, xs * e},
                           {dWg, in * ge},
                           {dWu, in * ge},
                           {dWd, out * ge},
                           {workspace, need},
                           {x, xs * e},
                           {Wg, in * e},
                           {Wu, in * e},
                           {Wd, out * e},
                           {saved->g, kept},
                           {saved->u, kept},
                           {scales ? saved->g_scale : nullptr, scales},
                           {scales ? saved->u_scale : nullptr, scales},
                           {dy, (size_t)d->N * d->d_out * e}}, 5));
  FfnPlan p;
  PKM_TRY(make_plan(d, &p));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto run = p.simt ? launch_ffn_bwd_simt : launch_ffn_bwd_tc;
  return cuda_status(run(p, x, Wg, Wu, Wd, *saved, dy, dx, dWg, dWu, dWd, workspace, st));
}

pkm_status pkm_ckpt8_pack(int64_t rows, int32_t cols, uint32_t flags, const void* src,
                          int8_t* codes, float* scale, void* stream) {
  PKM_TRY(validate_ckpt8(rows, cols, flags));
  if (rows == 0) return PKM_OK;
  PKM_NEED(src); PKM_NEED(codes); PKM_NEED(scale);
  const size_t runs = (size_t)rows * ckpt_runs(cols);
  PKM_TRY(check_apart<3>({{codes, runs * kCkptRun},
                          {scale, runs * 4},
                          {src, (size_t)rows * cols * (flags & PKM_F_FP32 ? 4 : 2)}}, 2));
  DeviceInfo info;
  if (!current_device(&info)) return PKM_ERR_CUDA;
  return cuda_status(launch_ckpt8_pack(rows, cols, flags & PKM_F_FP32, src, codes, scale,
                                       static_cast<cudaStream_t>(stream)));
}

pkm_status pkm_ckpt8_unpack(int64_t rows, int32_t cols, uint32_t flags, const int8_t* codes,
                            const float* scale, void* dst, void* stream) {
  PKM_TRY(validate_ckpt8(rows, cols, flags));
  if (rows == 0) return PKM_OK;
  PKM_NEED(codes); PKM_NEED(scale); PKM_NEED(dst);
  const size_t runs = (size_t)rows * ckpt_runs(cols);
  PKM_TRY(check_apart<3>({{dst, (size_t)rows * cols * (flags & PKM_F_FP32 ? 4 : 2)},
                          {codes, runs * kCkptRun},
                          {scale, runs * 4}}, 1));
  DeviceInfo info;
  if (!current_device(&info)) return PKM_ERR_CUDA;
  return cuda_status(launch_ckpt8_unpack(rows, cols, flags & PKM_F_FP32, codes, scale, dst,
                                         static_cast<cudaStream_t>(stream)));
}

pkm_status pkm_w4_pack(int32_t d_out, int32_t d_in, int32_t group, const void* W, uint8_t* codes,
                       void* scale, void* stream) {
  PKM_TRY(validate_w4(d_out, d_in, group));
  PKM_NEED(W); PKM_NEED(codes); PKM_NEED(scale);
  PKM_TRY(check_apart<3>({{codes, w4_codes_bytes(d_out, d_in)},
                          {scale, w4_scale_bytes(d_out, d_in, group)},
                          {W, (size_t)d_out * d_in * 2}}, 2));
  DeviceInfo info;
  if (!current_device(&info)) return PKM_ERR_CUDA;
  return cuda_status(
      launch_w4_pack(d_out, d_in, group, W, codes, scale, static_cast<cudaStream_t>(stream)));
}

pkm_status pkm_w4_unpack(int32_t d_out, int32_t d_in, int32_t group, const pkm_w4* W, void* out,
                         void* stream) {
  PKM_TRY(validate_w4(d_out, d_in, group));
  W4Mat m;
  PKM_TRY(check_w4(W, &m));
  PKM_NEED(out);
  PKM_TRY(check_apart<3>({{out, (size_t)d_out * d_in * 2},
                          {W->codes, w4_codes_bytes(d_out, d_in)},
                          {W->scale, w4_scale_bytes(d_out, d_in, group)}}, 1));
  DeviceInfo info;
  if (!current_device(&info)) return PKM_ERR_CUDA;
  return cuda_status(
      launch_w4_unpack(d_out, d_in, group, m, out, static_cast<cudaStream_t>(stream)));
}

pkm_status pkm_w4_matvec(int64_t N, int32_t d_in, int32_t d_out, int32_t group, const void* x,
                         const pkm_w4* W, float* y, void* stream) {
  if (N < 0) return PKM_ERR_INVALID_ARG;
  PKM_TRY(validate_w4(d_out, d_in, group));
  if (N > PKM_W4_MAX_TOKENS) return PKM_ERR_UNSUPPORTED;
  if (N == 0) return PKM_OK;
  PKM_NEED(x); PKM_NEED(y);
  W4Mat m;
  PKM_TRY(check_w4(W, &m));
  PKM_TRY(check_apart<4>({{y, (size_t)N * d_out * 4},
                          {x, (size_t)N * d_in * 2},
                          {W->codes, w4_codes_bytes(d_out, d_in)},
                          {W->scale, w4_scale_bytes(d_out, d_in, group)}}, 1));
  DeviceInfo info;
  if (!current_device(&info)) return PKM_ERR_CUDA;
  return cuda_status(launch_w4_matvec(N, d_in, d_out, group, x, m, y, info.sm_count,
                                      static_cast<cudaStream_t>(stream)));
}

pkm_status pkm_w4_ffn(const pkm_ffn_dims* d, int32_t group, const void* x, const pkm_w4* Wg,
                      const pkm_w4* Wu, const pkm_w4* Wd, void* y, void* workspace,
                      size_t workspace_bytes, void* stream) {
  PKM_TRY(validate_sizes(d));
  if (d->flags) return PKM_ERR_INVALID_ARG;
  PKM_TRY(validate_w4(d->d_ff, d->d_in, group));
  PKM_TRY(validate_w4(d->d_out, d->d_ff, group));
  if (d->N > PKM_W4_MAX_TOKENS) return PKM_ERR_UNSUPPORTED;
  if (d->N == 0) return PKM_OK;
  PKM_NEED(x); PKM_NEED(y);
  W4Mat g, u, o;
  PKM_TRY(check_w4(Wg, &g));
  PKM_TRY(check_w4(Wu, &u));
  PKM_TRY(check_w4(Wd, &o));
  const size_t need = pkm_ffn_workspace_bytes(d, PKM_FWD);
  PKM_TRY(check_workspace(need, workspace, workspace_bytes));
  const size_t cin = w4_codes_bytes(d->d_ff, d->d_in), cout = w4_codes_bytes(d->d_out, d->d_ff);
  const size_t sin = w4_scale_bytes(d->d_ff, d->d_in, group);
  const size_t sout = w4_scale_bytes(d->d_out, d->d_ff, group);
  PKM_TRY(check_apart<9>({{y, (size_t)d->N * d->d_out * 2},
                          {workspace, need},
                          {x, (size_t)d->N * d->d_in * 2},
                          {Wg->codes, cin},
                          {Wg->scale, sin},
                          {Wu->codes, cin},
                          {Wu->scale, sin},
                          {Wd->codes, cout},
                          {Wd->scale, sout}}, 2));
  FfnPlan p;
  PKM_TRY(make_plan(d, &p));
  return cuda_status(
      launch_w4_ffn(p, group, x, g, u, o, y, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
