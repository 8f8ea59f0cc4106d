// pi_norm.cu -- C ABI of the row-wise operators around a block: the norms with
// gate, residual scale and residual add, their gradients, the 8-bit
// quantiser.  Host validation, workspace layout and kernel dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pi_ffn.h"
#include "pi_host.cuh"
#include "pi_norm.cuh"

namespace {

using namespace pi::host;
namespace NM = pi::norm;

constexpr int kMaxNormD = 16384;
constexpr int kMaxI8K = 131056;

// ---------------------------------------------------------------- norms
// Launch shape of the row kernels: up to 512 threads with ch chunks of 4
// elements each; rows over 8192 elements by clusters of two blocks; a ring of
// `rows` rows in shared memory (one row, refilled once it is in registers,
// where two do not fit); `per_sm` blocks per SM.
struct RowShape {
  int threads, ch, rows, per_sm;
  bool cluster;
  size_t smem;
};
constexpr int kRowBlocks = 8;               // blocks per SM of the backward kernel, at most
constexpr size_t kRowSmem = 200 * 1024;     // of the 227 KB per block; the rest is L1 for the column factors
RowShape row_shape(int d, int bytes_per_element, bool backward) {
  RowShape r{};
  r.cluster = d > 8192;
  const int chunks = (r.cluster ? d / 2 : d) / 4;
  // short rows: one warp each, without block barriers (16384 x 448 forward 17.1 us against 23.1)
  r.ch = chunks <= 128 ? cdiv(chunks, 32) : cdiv(chunks, 512);
  r.threads = cdiv(cdiv(chunks, r.ch), 32) * 32;
  const size_t row = (size_t)r.threads * r.ch * 4 * bytes_per_element;
  r.rows = 2 * row <= kRowSmem ? 2 : 1;
  r.smem = r.rows * row;
  r.per_sm = (int)(kRowSmem / (r.smem + 1024));
  // threads that the registers hold: forward up to 38, 64, 64, 115 a thread for
  // ch = 1, 2, 3, 4; backward 98, 102, 126, 128
  const int fits = r.ch > 3 ? 512 : backward ? (r.ch == 1 ? 640 : r.ch == 2 ? 608 : 512) : r.ch == 1 ? 1536 : 1024;
  const int by_threads = fits / r.threads;
  if (r.per_sm > by_threads) r.per_sm = by_threads;
  if (r.per_sm < 1) r.per_sm = 1;
  if (r.per_sm > (backward ? kRowBlocks : 16)) r.per_sm = backward ? kRowBlocks : 16;
  return r;
}
// Row groups (blocks, or clusters of two) that the machine holds.
int row_groups(const RowShape &r, int sms) { return sms * r.per_sm / (r.cluster ? 2 : 1); }
pi_status check_norm(const pi_block_norm_desc *D) {
  if (!D || D->d_model <= 0 || !is_type(D->y_dtype) || !is_type(D->u_dtype)) return PI_ERR_INVALID_ARG;
  if (!(D->eps > 0.f) || !std::isfinite(D->eps) || !std::isfinite(D->residual_scale) || !std::isfinite(D->branch_scale))
    return PI_ERR_INVALID_ARG;
  if (D->w_post && !D->post_norm) return PI_ERR_INVALID_ARG;
  if (D->gate && D->tokens_per_gate <= 0) return PI_ERR_INVALID_ARG;
  if (D->d_model % 8 || D->d_model > kMaxNormD) return PI_ERR_UNSUPPORTED;
  if ((D->w_post && !aligned16(D->w_post)) || (D->w_pre && !aligned16(D->w_pre)) || (D->gate && !aligned16(D->gate)))
    return PI_ERR_MISALIGNED;
  return PI_OK;
}
// Row groups of the backward kernel: enough to fill the machine, but four rows
// each where the tokens allow, since a group leaves a row of partials behind.
// `most` is at most kRowBlocks per SM whatever the types, so that a workspace
// sized for more tokens serves fewer.
int norm_bwd_groups(int most, int tokens, int sms) {
  int g = cdiv(tokens, 4);
  if (g < sms) g = sms;
  if (g > most) g = most;
  return tokens < g ? tokens : g;
}
template <int CH, int R, bool CL>
pi_status fwd_launch(const NM::FwdArgs &a, int groups, const RowShape &r, cudaStream_t st) {
  static void (*const kern[9])(NM::FwdArgs) = {  // 3 * y type + u type
      NM::norm_fwd_kernel<CH, R, CL, 0, 0>, NM::norm_fwd_kernel<CH, R, CL, 0, 1>, NM::norm_fwd_kernel<CH, R, CL, 0, 2>,
      NM::norm_fwd_kernel<CH, R, CL, 1, 0>, NM::norm_fwd_kernel<CH, R, CL, 1, 1>, NM::norm_fwd_kernel<CH, R, CL, 1, 2>,
      NM::norm_fwd_kernel<CH, R, CL, 2, 0>, NM::norm_fwd_kernel<CH, R, CL, 2, 1>, NM::norm_fwd_kernel<CH, R, CL, 2, 2>};
  static DeviceOnce once[9];
  const int k = 3 * a.y_type + a.u_type;
  PI_CUDA(launch1(kern[k], dim3(groups * (CL ? 2 : 1)), r.threads, r.smem, CL ? 2 : 0, &once[k], st, a));
  return PI_OK;
}
template <int CH, int R, bool CL>
pi_status bwd_launch(const NM::BwdArgs &a, int groups, const RowShape &r, cudaStream_t st) {
  static void (*const kern[9])(NM::BwdArgs) = {
      NM::norm_bwd_kernel<CH, R, CL, 0, 0>, NM::norm_bwd_kernel<CH, R, CL, 0, 1>, NM::norm_bwd_kernel<CH, R, CL, 0, 2>,
      NM::norm_bwd_kernel<CH, R, CL, 1, 0>, NM::norm_bwd_kernel<CH, R, CL, 1, 1>, NM::norm_bwd_kernel<CH, R, CL, 1, 2>,
      NM::norm_bwd_kernel<CH, R, CL, 2, 0>, NM::norm_bwd_kernel<CH, R, CL, 2, 1>, NM::norm_bwd_kernel<CH, R, CL, 2, 2>};
  static DeviceOnce once[9];
  const int k = 3 * a.y_type + a.u_type;
  PI_CUDA(launch1(kern[k], dim3(groups * (CL ? 2 : 1)), r.threads, r.smem, CL ? 2 : 0, &once[k], st, a));
  return PI_OK;
}
// Clusters have ch 3 or 4; only the backward kernel's rows of ch = 4 can exceed a ring of two.
pi_status fwd_dispatch(const NM::FwdArgs &a, int groups, const RowShape &r, cudaStream_t st) {
  if (r.cluster) return r.ch == 3 ? fwd_launch<3, 2, true>(a, groups, r, st) : fwd_launch<4, 2, true>(a, groups, r, st);
  switch (r.ch) {
  case 1:
    return fwd_launch<1, 2, false>(a, groups, r, st);
  case 2:
    return fwd_launch<2, 2, false>(a, groups, r, st);
  case 3:
    return fwd_launch<3, 2, false>(a, groups, r, st);
  default:
    return fwd_launch<4, 2, false>(a, groups, r, st);
  }
}
pi_status bwd_dispatch(const NM::BwdArgs &a, int groups, const RowShape &r, cudaStream_t st) {
  if (r.cluster)
    return r.ch == 3     ? bwd_launch<3, 2, true>(a, groups, r, st)
           : r.rows == 2 ? bwd_launch<4, 2, true>(a, groups, r, st)
                         : bwd_launch<4, 1, true>(a, groups, r, st);
  switch (r.ch) {
  case 1:
    return bwd_launch<1, 2, false>(a, groups, r, st);
  case 2:
    return bwd_launch<2, 2, false>(a, groups, r, st);
  case 3:
    return bwd_launch<3, 2, false>(a, groups, r, st);
  default:
    return r.rows == 2 ? bwd_launch<4, 2, false>(a, groups, r, st) : bwd_launch<4, 1, false>(a, groups, r, st);
  }
}
size_t gate_bytes(const pi_block_norm_desc *D, int tokens) {
  if (!D->gate || tokens <= 0) return 0;
  return (size_t)((tokens - 1) / D->tokens_per_gate + 1) * D->d_model * 4;
}
size_t norm_ws_bytes(int d, int G) { return kHeader + (size_t)G * d * 4 * 4; }  // dw_post, dw_pre, 2 gate rows

}  // namespace

extern "C" {

// ====================================================================== norms around a block
pi_status pi_block_norm_forward(const pi_block_norm_desc *desc, const float *x, const void *y, int tokens,
                                float *x_out, void *u, float *rstd_post, float *rstd_pre, pi_stream_t stream) {
  const pi_status s = check_norm(desc);
  if (s != PI_OK) return s;
  if (tokens < 0 || tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  if (tokens == 0) return PI_OK;
  if (!x || (!x_out && !u)) return PI_ERR_INVALID_ARG;
  if ((rstd_post && !(y && desc->post_norm)) || (rstd_pre && !u)) return PI_ERR_INVALID_ARG;
  const void *ptrs[] = {x, y, x_out, u, rstd_post, rstd_pre};
  for (const void *p : ptrs)
    if (p && !aligned16(p)) return PI_ERR_MISALIGNED;
  const size_t n = (size_t)tokens * desc->d_model, t4 = (size_t)tokens * 4, d4 = (size_t)desc->d_model * 4;
  const Range mem[] = {{x_out, n * 4}, {u, n * type_size(desc->u_dtype)}, {rstd_post, t4}, {rstd_pre, t4},
                       {x_out == x ? nullptr : x, n * 4}, {y, n * type_size(desc->y_dtype)}, {desc->w_post, d4},
                       {desc->w_pre, d4}, {desc->gate, gate_bytes(desc, tokens)}};
  if (overlapping(mem, 4, 9)) return PI_ERR_INVALID_ARG;
  NM::FwdArgs a{};
  a.x = x, a.y = y;
  a.w_pre = desc->w_pre;
  if (y) a.w_post = desc->w_post, a.gate = desc->gate;  // without a branch nothing of it enters r
  a.x_out = x_out, a.u = u, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre;
  a.tokens = tokens, a.d = desc->d_model;
  a.tokens_per_gate = desc->tokens_per_gate < tokens ? desc->tokens_per_gate : tokens;
  a.y_type = desc->y_dtype, a.u_type = desc->u_dtype, a.post_norm = y && desc->post_norm ? 1 : 0;
  a.eps = desc->eps, a.alpha = desc->residual_scale, a.beta = desc->branch_scale;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  const RowShape r = row_shape(a.d, 4 + (int)type_size(desc->y_dtype), false);
  const int most = row_groups(r, sms), groups = tokens < most ? tokens : most;
  return fwd_dispatch(a, groups, r, (cudaStream_t)stream);
}

pi_status pi_block_norm_workspace_size(const pi_block_norm_desc *desc, int max_tokens, size_t *bytes) {
  const pi_status s = check_norm(desc);
  if (s != PI_OK) return s;
  if (!bytes) return PI_ERR_INVALID_ARG;
  if (max_tokens < 0 || max_tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  *bytes = norm_ws_bytes(desc->d_model, norm_bwd_groups(sms * kRowBlocks, max_tokens, sms));
  return PI_OK;
}

pi_status pi_block_norm_backward(const pi_block_norm_desc *desc, const float *x_out, const void *y,
                                 const float *rstd_post, const float *rstd_pre, const void *du, const float *dx_out,
                                 int tokens, float *dx, void *dy, float *dw_post, float *dw_pre, float *dgate,
                                 unsigned flags, void *ws, size_t ws_bytes, pi_stream_t stream) {
  pi_status s = check_norm(desc);
  if (s != PI_OK) return s;
  if (flags & ~(unsigned)PI_GRAD_ACCUMULATE) return PI_ERR_INVALID_ARG;
  if ((dw_post && !desc->post_norm) || (dgate && !desc->gate)) return PI_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  if (tokens) {
    if (!du && !dx_out) return PI_ERR_INVALID_ARG;
    if (du ? (!x_out || !rstd_pre) : dw_pre != nullptr) return PI_ERR_INVALID_ARG;
    if (y ? (desc->post_norm && !rstd_post) : (dy || dw_post || dgate)) return PI_ERR_INVALID_ARG;
  }
  const void *ptrs[] = {x_out, y, rstd_post, rstd_pre, du, dx_out, dx, dy, dw_post, dw_pre, dgate};
  for (const void *p : ptrs)
    if (p && !aligned16(p)) return PI_ERR_MISALIGNED;
  const int d = desc->d_model;
  const size_t n = (size_t)tokens * d, nx = n * 4, ny = n * type_size(desc->y_dtype), nu = n * type_size(desc->u_dtype);
  const size_t t4 = (size_t)tokens * 4, d4 = (size_t)d * 4, ng = gate_bytes(desc, tokens);
  Range mem[] = {{dx, nx}, {dy, ny}, {dw_post, d4}, {dw_pre, d4}, {dgate, ng}, {nullptr, 0}, {x_out, nx},
                 {dy == y ? nullptr : y, ny}, {rstd_post, t4}, {rstd_pre, t4}, {du, nu},
                 {dx == dx_out ? nullptr : dx_out, nx}, {desc->w_post, d4}, {desc->w_pre, d4}, {desc->gate, ng}};
  if (overlapping(mem, 6, 15)) return PI_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const int acc = (flags & PI_GRAD_ACCUMULATE) ? 1 : 0;
  if (tokens == 0) {  // no tokens: the sums over them are zero (and there is no gate row)
    if (!acc && dw_post) PI_CUDA(cudaMemsetAsync(dw_post, 0, (size_t)d * 4, st));
    if (!acc && dw_pre) PI_CUDA(cudaMemsetAsync(dw_pre, 0, (size_t)d * 4, st));
    return PI_OK;
  }
  if (!ws) return PI_ERR_WORKSPACE;
  if (!aligned16(ws)) return PI_ERR_MISALIGNED;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  const RowShape r = row_shape(d, 8 + (int)type_size(desc->u_dtype) + (int)type_size(desc->y_dtype), true);
  const int G = norm_bwd_groups(row_groups(r, sms), tokens, sms);
  if (ws_bytes < norm_ws_bytes(d, G)) return PI_ERR_WORKSPACE;
  mem[5] = Range{ws, norm_ws_bytes(d, G)};
  if (overlapping(mem, 6, 15)) return PI_ERR_INVALID_ARG;
  float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + kHeader);
  NM::BwdArgs a{};
  a.x_out = x_out, a.y = y, a.du = du, a.rstd_post = rstd_post, a.rstd_pre = rstd_pre, a.dx_out = dx_out;
  a.w_post = desc->w_post, a.w_pre = desc->w_pre, a.gate = desc->gate;
  a.dx = dx, a.dy = dy, a.dgate = dgate;
  a.part_post = dw_post ? part : nullptr;
  a.part_pre = dw_pre ? part + (size_t)G * d : nullptr;
  a.part_gate = part + (size_t)2 * G * d;
  a.tokens = tokens, a.d = d;
  a.tokens_per_gate = desc->tokens_per_gate < tokens ? desc->tokens_per_gate : tokens;
  a.y_type = desc->y_dtype, a.u_type = desc->u_dtype, a.post_norm = desc->post_norm ? 1 : 0;
  a.accumulate = acc;
  a.alpha = desc->residual_scale, a.beta = desc->branch_scale;
  s = bwd_dispatch(a, G, r, st);
  if (s != PI_OK) return s;
  if (dw_post || dw_pre || dgate) {
    NM::JoinArgs j{};
    j.part_post = a.part_post, j.part_pre = a.part_pre, j.part_gate = a.part_gate;
    j.dw_post = dw_post, j.dw_pre = dw_pre, j.dgate = dgate;
    j.G = G, j.tokens = tokens, j.d = d, j.tokens_per_gate = a.tokens_per_gate, j.accumulate = acc;
    if (dgate) {
      const int rows = cdiv(tokens, a.tokens_per_gate);
      j.long_rows = (long long)a.tokens_per_gate * G > 8ll * tokens;  // fewer than G / 8 rows
      j.gate_jobs = j.long_rows ? rows : rows < NM::kGateJobs ? rows : NM::kGateJobs;
    }
    const dim3 g(cdiv(d, 32), 2 + j.gate_jobs);
    // many partial rows: more warps, so that their loads go out together
    PI_CUDA(G > 256 ? launch1(NM::norm_join_kernel<32>, g, 1024, 0, 0, nullptr, st, j)
                    : launch1(NM::norm_join_kernel<8>, g, 256, 0, 0, nullptr, st, j));
  }
  return PI_OK;
}

// ====================================================================== 8-bit quantiser
pi_status pi_quantize_i8(const void *x, int x_dtype, int rows, int k, int8_t *q, float *scales, pi_stream_t stream) {
  if (k <= 0 || !is_type(x_dtype)) return PI_ERR_INVALID_ARG;
  if (k % 16 || rows < 0 || rows > kMaxTokens || k > kMaxI8K) return PI_ERR_UNSUPPORTED;
  if (rows == 0) return PI_OK;
  if (!x || !q || !scales) return PI_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales)) return PI_ERR_MISALIGNED;
  const Range r[] = {{q, (size_t)rows * k}, {scales, (size_t)rows * 4}, {x, (size_t)rows * k * type_size(x_dtype)}};
  if (overlapping(r, 2, 3)) return PI_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  // a thread keeps up to 4 chunks of 8 elements; more threads for longer rows and for few rows
  const int chunks = cdiv(k, 8);
  const int most = rows < sms ? 1024 : 256;
  int ch = cdiv(chunks, most);
  ch = ch <= 1 ? 1 : ch <= 2 ? 2 : 4;
  int threads = cdiv(cdiv(chunks, ch), 32) * 32;
  if (threads > 1024) threads = 1024;
  const NM::QuantArgs a{x, q, scales, rows, k};
  cudaStream_t st = (cudaStream_t)stream;
  static void (*const kern[3][3])(NM::QuantArgs) = {
      {NM::quantize_i8_kernel<0, 1>, NM::quantize_i8_kernel<0, 2>, NM::quantize_i8_kernel<0, 4>},
      {NM::quantize_i8_kernel<1, 1>, NM::quantize_i8_kernel<1, 2>, NM::quantize_i8_kernel<1, 4>},
      {NM::quantize_i8_kernel<2, 1>, NM::quantize_i8_kernel<2, 2>, NM::quantize_i8_kernel<2, 4>}};
  PI_CUDA(launch1(kern[x_dtype][ch >> 1], dim3(rows < 65535 ? rows : 65535), threads, 0, 0, nullptr, st, a));
  return PI_OK;
}

}  // extern "C"
