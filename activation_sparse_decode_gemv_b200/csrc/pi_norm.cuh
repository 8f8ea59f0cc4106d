// pi_norm.cuh -- the row-wise kernels around a block: the fused norms with
// gate, residual scale and residual add, their gradients, and the quantiser
// of the 8-bit product.  All are bound by HBM: each reads its inputs once and
// writes its outputs once, with every sum and statistic in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pi_device.cuh"

namespace pi {
namespace norm {

enum Type { T_F32 = 0, T_F16 = 1, T_BF16 = 2 };

// ---------------------------------------------------------------- four elements at a time
PI_DEV float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
PI_DEV float4 ld4(const void *p, size_t i, int type) {
  if (type == T_F32) return *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
  const uint2 w = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + i);
  if (type == T_F16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
PI_DEV void st4(void *p, size_t i, int type, float4 v) {
  if (type == T_F32) {
    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i) = v;
    return;
  }
  uint2 w;
  if (type == T_F16) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
  *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p) + i) = w;
}
PI_DEV float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }
PI_DEV float4 scale4(float s, float4 a) { return make_float4(s * a.x, s * a.y, s * a.z, s * a.w); }
PI_DEV float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
PI_DEV float dot4(float4 a, float4 b) { return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x))); }
PI_DEV float4 one4() { return make_float4(1.f, 1.f, 1.f, 1.f); }
PI_DEV float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// Block-wide sums of N values; buf: 32 N floats of shared memory not in use
// since the last barrier but one (callers alternate two buffers).
template <int N>
PI_DEV void block_sum(float (&v)[N], float *buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if (nw == 1) return;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) buf[k * 32 + warp] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < nw ? buf[k * 32 + lane] : 0.f);
}

// ---------------------------------------------------------------- forward
//   m = y rsqrt(mean y^2 + eps) (post_norm; else m = y),  b = m w_post
//   r = alpha x + beta gate b,   u = r rsqrt(mean r^2 + eps) w_pre
struct FwdArgs {
  const float *x;
  const void *y;  // null: no branch
  const float *w_post, *w_pre, *gate;  // null: ones
  float *x_out;   // null: not stored
  void *u;        // null: no pre-norm
  float *rstd_post, *rstd_pre;  // optional
  int tokens, d, tokens_per_gate;
  int y_type, u_type, post_norm;
  float eps, alpha, beta;
};

// One block per row (grid-stride), CH chunks of 4 elements a thread, kept in
// registers from the load to the store; two block sums a row.
template <int CH>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const FwdArgs a) {
  __shared__ float buf[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const float inv_d = 1.f / (float)a.d;
  for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const size_t row = (size_t)t * a.d;
    float4 r[CH], y[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + c * blockDim.x) * 4;
      r[c] = y[c] = zero4();
      if (i < a.d) {
        r[c] = scale4(a.alpha, ld4(a.x + row + i));
        if (a.y) y[c] = ld4(a.y, row + i, a.y_type);
      }
    }
    if (a.y) {
      float k = a.beta;
      if (a.post_norm) {
        float s[1] = {0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) s[0] += dot4(y[c], y[c]);
        block_sum(s, buf[0]);
        const float rp = rsqrtf(s[0] * inv_d + a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rp;
#pragma unroll
        for (int c = 0; c < CH; ++c) y[c] = scale4(rp, y[c]);
      }
      const float *g = a.gate ? a.gate + (size_t)(t / a.tokens_per_gate) * a.d : nullptr;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (threadIdx.x + c * blockDim.x) * 4;
        if (i < a.d) {
          float4 b = y[c];
          if (a.w_post) b = mul4(b, ld4(a.w_post + i));
          if (g) b = mul4(b, ld4(g + i));
          r[c] = add4(r[c], scale4(k, b));
        }
      }
    }
    if (a.x_out)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (threadIdx.x + c * blockDim.x) * 4;
        if (i < a.d) *reinterpret_cast<float4 *>(a.x_out + row + i) = r[c];
      }
    if (a.u) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c) s[0] += dot4(r[c], r[c]);
      block_sum(s, buf[1]);
      const float rr = rsqrtf(s[0] * inv_d + a.eps);
      if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = rr;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (threadIdx.x + c * blockDim.x) * 4;
        if (i < a.d) {
          float4 o = scale4(rr, r[c]);
          if (a.w_pre) o = mul4(o, ld4(a.w_pre + i));
          st4(a.u, row + i, a.u_type, o);
        }
      }
    }
    if (!(a.y && a.post_norm && a.u)) __syncthreads();  // one buffer in use: keep rows apart
  }
}

// ---------------------------------------------------------------- backward
// With n = r rstd_pre, m = y rstd_post (or y), q = beta gate w_post m:
//   dr = dx_out + rstd_pre (du w_pre - n c/d),      c = sum du w_pre n
//   dx = alpha dr,  dgate += beta w_post m dr,  dw_pre += du n,
//   dw_post += beta gate m dr
//   dy = rstd_post (v - m e/d),  v = beta gate w_post dr,
//   e = sum v m = sum q dx_out + rstd_pre (sum q du w_pre - c/d sum q n)
// so one block sum of three values (c and two of e's parts) serves a row.
struct BwdArgs {
  const float *x_out;  // r
  const void *y, *du;  // y null: no branch; du null: no pre-norm
  const float *rstd_post, *rstd_pre, *dx_out;
  const float *w_post, *w_pre, *gate;
  float *dx;
  void *dy;
  float *dgate;
  float *part_post, *part_pre;  // [G x d] column sums of a block's rows
  float *part_gate;             // [G x 2 x d] of its first and last gate rows, where shared with other blocks
  int tokens, d, tokens_per_gate;
  int y_type, u_type, post_norm, accumulate;
  float alpha, beta;
};

PI_DEV int first_token(int tokens, int G, int c) { return (int)((long long)tokens * c / G); }

// One block per contiguous run of rows; column sums stay in registers and are
// written once per block (per gate row for dgate), so their order is fixed.
template <int CH>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const BwdArgs a) {
  __shared__ float buf[2][96];
  pdl_wait();
  pdl_launch_dependents();
  const int G = gridDim.x, cta = blockIdx.x;
  const int t0 = first_token(a.tokens, G, cta), t1 = first_token(a.tokens, G, cta + 1);
  const float inv_d = 1.f / (float)a.d;
  const bool want_gate = a.dgate != nullptr;
  float4 s_pre[CH], s_post[CH], s_gate[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) s_pre[c] = s_post[c] = s_gate[c] = zero4();
  int group = a.gate ? t0 / a.tokens_per_gate : 0;
  const int group0 = group;

  auto flush_gate = [&]() {
    // a gate row used by this block alone is finished here; a shared one goes to the joining kernel
    const long long g0 = (long long)group * a.tokens_per_gate;
    const long long g1 = min((long long)a.tokens, g0 + a.tokens_per_gate);
    const bool whole = g0 >= t0 && g1 <= t1;
    float *dst = whole ? a.dgate + (size_t)group * a.d : a.part_gate + ((size_t)cta * 2 + (group != group0)) * a.d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + c * blockDim.x) * 4;
      if (i < a.d) {
        float4 v = s_gate[c];
        if (whole && a.accumulate) v = add4(v, ld4(dst + i));
        *reinterpret_cast<float4 *>(dst + i) = v;
      }
      s_gate[c] = zero4();
    }
  };

  for (int t = t0; t < t1; ++t) {
    const size_t row = (size_t)t * a.d;
    if (a.gate) {
      const int gi = t / a.tokens_per_gate;
      if (gi != group) {
        if (want_gate) flush_gate();
        group = gi;
      }
    }
    const float *g = a.gate ? a.gate + (size_t)group * a.d : nullptr;
    const float rr = a.du ? a.rstd_pre[t] : 0.f;
    const float rp = a.y && a.post_norm ? a.rstd_post[t] : 1.f;
    float4 n[CH], v[CH], m[CH], dr[CH];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + c * blockDim.x) * 4;
      n[c] = v[c] = m[c] = dr[c] = zero4();
      if (i < a.d) {
        if (a.dx_out) dr[c] = ld4(a.dx_out + row + i);
        if (a.du) {
          n[c] = scale4(rr, ld4(a.x_out + row + i));
          v[c] = ld4(a.du, row + i, a.u_type);
        }
        if (a.y) m[c] = scale4(rp, ld4(a.y, row + i, a.y_type));
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + c * blockDim.x) * 4;
      if (i < a.d) {
        if (a.du) {
          s_pre[c] = add4(s_pre[c], mul4(v[c], n[c]));
          if (a.w_pre) v[c] = mul4(v[c], ld4(a.w_pre + i));
          s[0] += dot4(v[c], n[c]);
          // dr without the term of c
          dr[c] = add4(dr[c], scale4(rr, v[c]));
        }
        if (a.y && a.post_norm) {
          float4 q = scale4(a.beta, m[c]);
          if (g) q = mul4(q, ld4(g + i));
          if (a.w_post) q = mul4(q, ld4(a.w_post + i));
          s[1] += dot4(q, dr[c]);
          s[2] += dot4(q, n[c]);
        }
      }
    }
    block_sum(s, buf[t & 1]);
    const float cd = rr * s[0] * inv_d;           // dr -= cd n
    const float ed = (s[1] - cd * s[2]) * inv_d;  // dy = rp (v - m ed)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (threadIdx.x + c * blockDim.x) * 4;
      if (i < a.d) {
        const float4 d4 = add4(dr[c], scale4(-cd, n[c]));
        if (a.dx) *reinterpret_cast<float4 *>(a.dx + row + i) = scale4(a.alpha, d4);
        if (a.y) {
          float4 b = scale4(a.beta, d4);  // gradient of gate * w_post * m
          const float4 w = a.w_post ? ld4(a.w_post + i) : one4();
          if (want_gate) s_gate[c] = add4(s_gate[c], mul4(b, mul4(w, m[c])));
          if (g) b = mul4(b, ld4(g + i));
          if (a.post_norm) {
            s_post[c] = add4(s_post[c], mul4(b, m[c]));
            b = scale4(rp, add4(mul4(b, w), scale4(-ed, m[c])));
          } else {
            b = mul4(b, w);
          }
          if (a.dy) st4(a.dy, row + i, a.y_type, b);
        }
      }
    }
  }
  if (want_gate && t1 > t0) flush_gate();
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (threadIdx.x + c * blockDim.x) * 4;
    if (i < a.d) {
      if (a.part_post) *reinterpret_cast<float4 *>(a.part_post + (size_t)cta * a.d + i) = s_post[c];
      if (a.part_pre) *reinterpret_cast<float4 *>(a.part_pre + (size_t)cta * a.d + i) = s_pre[c];
    }
  }
}

// Joins the blocks' column sums in block order.  blockIdx.y: 0 dw_post, 1
// dw_pre, 2 + b: the gate row that crosses from block b's rows into block
// b + 1's, taken once, by the first boundary inside it.  A block sums 32
// columns, 8 partial rows at a time.
struct JoinArgs {
  const float *part_post, *part_pre, *part_gate;
  float *dw_post, *dw_pre, *dgate;
  int G, tokens, d, tokens_per_gate, accumulate;
};
__global__ void __launch_bounds__(256) norm_join_kernel(const JoinArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float buf[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  const int job = blockIdx.y;
  int c0 = 0, c1 = a.G;  // blocks whose partials are summed
  float *out = job == 0 ? a.dw_post : a.dw_pre;
  const float *part = job == 0 ? a.part_post : a.part_pre;
  long long g0 = 0;
  if (job >= 2) {
    const int b = job - 2;
    const int cut = first_token(a.tokens, a.G, b + 1);
    const int group = cut / a.tokens_per_gate;
    g0 = (long long)group * a.tokens_per_gate;
    if (g0 == cut || first_token(a.tokens, a.G, b) > g0) return;  // no crossing, or an earlier boundary has it
    const long long g1 = min((long long)a.tokens, g0 + a.tokens_per_gate);
    c0 = b;
    for (c1 = b + 1; c1 < a.G && first_token(a.tokens, a.G, c1) < g1;) ++c1;
    out = a.dgate ? a.dgate + (size_t)group * a.d : nullptr;
    part = a.part_gate;
  }
  if (!out) return;
  float s = 0.f;
  if (i < a.d)
    for (int c = c0 + w; c < c1; c += 8) {
      size_t row = c;
      if (job >= 2)  // the block's first gate row is in its slot 0, another in slot 1
        row = (size_t)c * 2 + (first_token(a.tokens, a.G, c) < g0 ? 1 : 0);
      s += part[row * a.d + i];
    }
  buf[w][lane] = s;
  __syncthreads();
  if (w == 0 && i < a.d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += buf[k][lane];
    out[i] = a.accumulate ? out[i] + s : s;
  }
}

// ---------------------------------------------------------------- 8-bit quantiser
// Row r: scale = amax / 127, q = rint(x / scale) (fp32 quotient, ties to
// even).  A row of zeros has scale 0 and codes 0; a row that holds an
// infinity or a NaN has scale NaN and codes 0, so its products are NaN.
PI_DEV void ld8(const void *p, size_t i, int type, float (&v)[8]) {
  const float4 a = ld4(p, i, type), b = ld4(p, i + 4, type);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
PI_DEV uint32_t code4(const float *v, float scale) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int q = (int)fminf(127.f, fmaxf(-127.f, rintf(__fdiv_rn(v[j], scale))));
    w |= (uint32_t)(q & 255) << (8 * j);
  }
  return w;
}
__global__ void __launch_bounds__(1024) quantize_i8_kernel(const void *__restrict__ x, int type, int rows, int k,
                                                          int8_t *__restrict__ q, float *__restrict__ scales) {
  __shared__ unsigned buf[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int r = blockIdx.x, it = 0; r < rows; r += gridDim.x, ++it) {
    const size_t row = (size_t)r * k;
    unsigned amax = 0;  // bits of |x|: they order like the values, and a NaN above all
    float v0[8];
    for (int i = threadIdx.x * 8; i < k; i += blockDim.x * 8) {
      float v[8];
      ld8(x, row + i, type, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
      if (i == (int)threadIdx.x * 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) v0[j] = v[j];
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0) buf[it & 1][warp] = amax;
    __syncthreads();
    amax = __reduce_max_sync(0xffffffffu, lane < nw ? buf[it & 1][lane] : 0u);
    const bool bad = amax >= 0x7f800000u;
    const float scale = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(__uint_as_float(amax), 127.f);
    if (threadIdx.x == 0) scales[r] = scale;
    const bool zero = bad || scale == 0.f;
    for (int i = threadIdx.x * 8; i < k; i += blockDim.x * 8) {
      uint2 w = make_uint2(0u, 0u);
      if (!zero) {
        if (i != (int)threadIdx.x * 8) ld8(x, row + i, type, v0);
        w = make_uint2(code4(v0, scale), code4(v0 + 4, scale));
      }
      *reinterpret_cast<uint2 *>(q + row + i) = w;
    }
  }
}

}  // namespace norm
}  // namespace pi
