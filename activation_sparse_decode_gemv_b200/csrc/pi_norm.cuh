// pi_norm.cuh -- the row-wise kernels around a block: the fused norms with
// gate, residual scale and residual add, their gradients, and the quantiser
// of the 8-bit product.  All are bound by HBM: each reads its inputs once and
// writes its outputs once, with every sum and statistic in fp32.  Measured
// (bf16 y and u): forward of 8192 x 5120 90.9 us, 5.5 TB/s; gradients of 4096 x
// 7168 109 us, 4.8 TB/s, of which about 96 the row kernel and 13 the joining one
// (alone, with cold caches, 100 and 14); one token of 8192 3.6 us (a launch).
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
PI_DEV float4 one4() { return make_float4(1.f, 1.f, 1.f, 1.f); }
PI_DEV float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// A row is summed by one block, or by a cluster of two blocks with half of its
// columns each (CL; rows over 8192 elements, whose values and column sums do
// not fit one block's registers).  The blocks of a cluster exchange their
// warps' sums through each other's shared memory.
template <bool CL>
PI_DEV int cluster_half() {
  if constexpr (!CL) return 0;
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
template <bool CL>
PI_DEV void row_sync() {
  if constexpr (CL) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
// The blocks of a cluster are launched together, which does not say that the
// other one has begun: its shared memory may be written only after a barrier
// that it has passed too.  Arrival at the kernel's start, the wait before the
// first row's sums, so that the first rows' loads hide it.
template <bool CL>
PI_DEV void peer_started_arrive() {
  if constexpr (CL) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
template <bool CL>
PI_DEV void peer_started_wait() {
  if constexpr (CL) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Row-wide sums of N values; buf: 32 N floats of shared memory that no warp
// has read since the last but one barrier (callers alternate two buffers).
template <int N, bool CL>
PI_DEV void row_sum(float (&v)[N], float *buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if constexpr (CL) {
    const int half = cluster_half<CL>();
    if (lane == 0) {
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(buf + half * 16 + warp);
      uint32_t peer;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(half ^ 1));
#pragma unroll
      for (int k = 0; k < N; ++k) {
        buf[k * 32 + half * 16 + warp] = v[k];
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer + k * 128), "f"(v[k]) : "memory");
      }
    }
    row_sync<CL>();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum((lane & 15) < nw ? buf[k * 32 + lane] : 0.f);
    return;
  }
  if (nw == 1) return;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) buf[k * 32 + warp] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < nw ? buf[k * 32 + lane] : 0.f);
}

// ---------------------------------------------------------------- four values as two packed pairs
// fma.rn.f32x2 and its kin do two fp32 operations an instruction, each rounded
// like the scalar one; the row kernels are short of issue slots, not of
// arithmetic.
struct P4 {
  unsigned long long a, b;
};
PI_DEV unsigned long long pk(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
PI_DEV unsigned long long fma2(unsigned long long x, unsigned long long y, unsigned long long z) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
PI_DEV unsigned long long mul2(unsigned long long x, unsigned long long y) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
PI_DEV P4 fma(P4 x, P4 y, P4 z) { return P4{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
PI_DEV P4 fma(unsigned long long s, P4 y, P4 z) { return P4{fma2(s, y.a, z.a), fma2(s, y.b, z.b)}; }
PI_DEV P4 mul(P4 x, P4 y) { return P4{mul2(x.a, y.a), mul2(x.b, y.b)}; }
PI_DEV P4 mul(unsigned long long s, P4 y) { return P4{mul2(s, y.a), mul2(s, y.b)}; }
PI_DEV unsigned long long dot(P4 x, P4 y, unsigned long long z) { return fma2(x.b, y.b, fma2(x.a, y.a, z)); }
PI_DEV float4 f4(P4 v) {
  float4 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v.a));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.z), "=f"(r.w) : "l"(v.b));
  return r;
}
PI_DEV P4 p4(float4 v) { return P4{pk(v.x, v.y), pk(v.z, v.w)}; }
PI_DEV float sum2(unsigned long long v) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
  return x + y;
}

// ---------------------------------------------------------------- row ring
// A thread owns the same 4-element chunks of every row (chunk tid + c *
// blockDim of CH) and fetches them itself, by cp.async into slots of its own,
// R rows ahead of their use.  No thread reads another's slot, so the ring
// needs no barrier: cp.async.wait_group orders a thread's own copies.
PI_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
PI_DEV void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr __host__ __device__ int chunk_bytes(int type) { return type == T_F32 ? 16 : 8; }

// This thread's chunks of one row of a tensor: `step` = blockDim chunks apart.
template <int CH, int TYPE>
struct Part {
  static constexpr int B = chunk_bytes(TYPE);
  // row0: the tensor's row; valid: bit c set where chunk c lies inside it
  static PI_DEV void fetch(uint32_t slot, const void *row0, int step, unsigned valid) {
    const char *p = static_cast<const char *>(row0) + threadIdx.x * B;
    slot += threadIdx.x * B;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (valid >> c & 1u) {
        if constexpr (TYPE == T_F32)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + c * step * B), "l"(p + c * step * B)
                       : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot + c * step * B), "l"(p + c * step * B)
                       : "memory");
      }
  }
  static PI_DEV P4 load(const unsigned char *slot, int c, int step) {
    const unsigned char *p = slot + (threadIdx.x + c * step) * B;
    if constexpr (TYPE == T_F32) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
      return P4{v.x, v.y};
    } else {
      return p4(ld4(p, 0, TYPE));
    }
  }
  static PI_DEV void store(void *row0, int c, int step, P4 v) {
    char *p = static_cast<char *>(row0) + (threadIdx.x + c * step) * B;
    if constexpr (TYPE == T_F32) *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v.a, v.b);
    else st4(p, 0, TYPE, f4(v));
  }
  // slots that no copy fills read as zero
  static PI_DEV void clear(unsigned char *slot, int step, unsigned valid) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (!(valid >> c & 1u)) {
        unsigned char *p = slot + (threadIdx.x + c * step) * B;
        *reinterpret_cast<unsigned long long *>(p) = 0;
        if (TYPE == T_F32) *reinterpret_cast<unsigned long long *>(p + 8) = 0;
      }
  }
};
template <int CH>
PI_DEV unsigned valid_chunks(int d) {
  unsigned v = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) v |= (unsigned)((int)(threadIdx.x + c * blockDim.x) * 4 < d) << c;
  return v;
}
// element col of row t
PI_DEV const void *row_at(const void *p, int t, int d, int col, int type) {
  return static_cast<const char *>(p) + ((size_t)t * d + col) * (type == T_F32 ? 4 : 2);
}
PI_DEV void *row_at(void *p, int t, int d, int col, int type) {
  return static_cast<char *>(p) + ((size_t)t * d + col) * (type == T_F32 ? 4 : 2);
}

// First of the rows that block c of G takes: contiguous runs of equal length.
PI_DEV int first_token(int tokens, int G, int c) { return (int)((long long)tokens * c / G); }

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

// beta gate w_post of a chunk's columns
PI_DEV float4 branch_factor(const float *gate_row, const float *w_post, float beta, int i) {
  float4 f = make_float4(beta, beta, beta, beta);
  if (w_post) f = mul4(f, ld4(w_post + i));
  if (gate_row) f = mul4(f, ld4(gate_row + i));
  return f;
}

// One block per run of rows; a row stays in registers between its two block
// sums.  Bound by HBM: 4 + |y| bytes read and 4 + |u| written per element.
// The column factors stay in registers too.
template <int CH, int R, bool CL, int YT, int UT>
__global__ void __launch_bounds__(512, CH <= 3 ? 2 : 1) norm_fwd_kernel(const FwdArgs a) {
  using X = Part<CH, T_F32>;
  using Y = Part<CH, YT>;
  using U = Part<CH, UT>;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float buf[2][32];
  peer_started_arrive<CL>();
  const int d = a.d, step = blockDim.x, half = cluster_half<CL>();
  const int dh = CL ? d / 2 : d, col0 = half * dh;  // this block's columns
  const int G = gridDim.x / (CL ? 2 : 1), blk = blockIdx.x / (CL ? 2 : 1);
  const int t0 = first_token(a.tokens, G, blk), t1 = first_token(a.tokens, G, blk + 1);
  const float inv_d = 1.f / (float)d;
  const unsigned valid = valid_chunks<CH>(dh);
  const int xb = CH * step * 16, slot_b = xb + CH * step * Y::B;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    X::clear(ring + k * slot_b, step, valid);
    Y::clear(ring + k * slot_b + xb, step, a.y ? valid : 0u);
  }
  auto fetch = [&](int t, int k) {  // row t into slot k
    if (t < t1) {
      X::fetch(ring_s + k * slot_b, row_at(a.x, t, d, col0, T_F32), step, valid);
      if (a.y) Y::fetch(ring_s + k * slot_b + xb, row_at(a.y, t, d, col0, YT), step, valid);
    }
    cp_commit();
  };
  pdl_wait();
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < R; ++k) fetch(t0 + k, k);
  auto col = [&](int c) { return col0 + (int)(threadIdx.x + c * step) * 4; };
  auto factor = [&](const float *gate_row, int c) {
    return valid >> c & 1u ? p4(branch_factor(gate_row, a.w_post, a.beta, col(c))) : p4(zero4());
  };
  int group = -1;
  P4 bf[CH], wp[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    wp[c] = a.w_pre && (valid >> c & 1u) ? p4(ld4(a.w_pre + col(c))) : p4(one4());
    if (!a.gate) bf[c] = factor(nullptr, c);
  }
  const unsigned long long alpha = pk(a.alpha, a.alpha);
  peer_started_wait<CL>();
  int slot_i = 0;
  for (int t = t0; t < t1; ++t) {
    if (a.gate && t / a.tokens_per_gate != group) {
      group = t / a.tokens_per_gate;
#pragma unroll
      for (int c = 0; c < CH; ++c) bf[c] = factor(a.gate + (size_t)group * d, c);
    }
    cp_wait<R - 1>();
    const unsigned char *slot = ring + slot_i * slot_b;
    P4 r[CH], y[CH];
    unsigned long long q = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      r[c] = mul(alpha, X::load(slot, c, step));
      y[c] = Y::load(slot + xb, c, step);
      q = dot(y[c], y[c], q);
    }
    fetch(t + R, slot_i);
    if (++slot_i == R) slot_i = 0;
    float rp = 1.f;
    if (a.post_norm) {
      float s[1] = {sum2(q)};
      row_sum<1, CL>(s, buf[0]);
      rp = rsqrtf(s[0] * inv_d + a.eps);
      if (a.rstd_post && threadIdx.x == 0 && half == 0) a.rstd_post[t] = rp;
    }
    const unsigned long long rp2 = pk(rp, rp);
    q = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      r[c] = fma(mul(rp2, y[c]), bf[c], r[c]);
      q = dot(r[c], r[c], q);
    }
    if (a.x_out) {
      void *o = row_at(a.x_out, t, d, col0, T_F32);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (valid >> c & 1u) X::store(o, c, step, r[c]);
    }
    if (a.u) {
      float s[1] = {sum2(q)};
      row_sum<1, CL>(s, buf[1]);
      const float rr = rsqrtf(s[0] * inv_d + a.eps);
      if (a.rstd_pre && threadIdx.x == 0 && half == 0) a.rstd_pre[t] = rr;
      const unsigned long long rr2 = pk(rr, rr);
      void *o = row_at(a.u, t, d, col0, UT);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (valid >> c & 1u) U::store(o, c, step, mul(mul(rr2, r[c]), wp[c]));
      }
    }
    if (!(a.post_norm && a.u)) row_sync<CL>();  // one buffer in use: keep rows apart
  }
  if constexpr (CL) row_sync<CL>();  // the other block has written its last sums
}

// ---------------------------------------------------------------- backward
// With n = r rstd_pre, m = y rstd_post (or y), f = beta gate w_post:
//   dr = dx_out + rstd_pre (du w_pre - n c/d),   c = sum du w_pre n
//   dx = alpha dr,   dw_pre += du n
//   dy = rstd_post (f dr - m e/d) (post_norm; else f dr),   e = sum f m dr
//      = sum f m dx_out + rstd_pre (sum f m du w_pre - c/d sum f m n)
// so one block sum of three values (c and e's two parts) serves a row.  The
// gate's and w_post's gradients share S = sum of m dr over the tokens of a gate
// row: dgate = beta w_post S, and dw_post += beta gate S once per gate row.
struct BwdArgs {
  const float *x_out;  // r
  const void *y, *du;  // y null: no branch; du null: no pre-norm
  const float *rstd_post, *rstd_pre, *dx_out;
  const float *w_post, *w_pre, *gate;
  float *dx;
  void *dy;
  float *dgate;
  float *part_post, *part_pre;  // [G x d] column sums of a block's rows (null: not wanted)
  float *part_gate;             // [G x 2 x d] of its first and last gate rows, where shared with other blocks
  int tokens, d, tokens_per_gate;
  int y_type, u_type, post_norm, accumulate;
  float alpha, beta;
};

// At the end of the tokens of gate row `group` (or of the block's rows): adds
// beta gate S to the block's dw_post sums and stores the gate's gradient, for
// the 4 columns at i.  post0: nothing is in part_post yet.
PI_DEV void flush_gate(const BwdArgs &a, int blk, int group, int group0, int t0, int t1, int i, float4 S, bool post0) {
  const float *grow = a.gate ? a.gate + (size_t)group * a.d : nullptr;
  if (a.part_post) {
    float4 v = scale4(a.beta, S);
    if (grow) v = mul4(v, ld4(grow + i));
    float *dst = a.part_post + (size_t)blk * a.d + i;
    if (!post0) v = add4(v, ld4(dst));
    *reinterpret_cast<float4 *>(dst) = v;
  }
  if (a.dgate) {
    // a gate row used by this block alone is finished here; a shared one goes to the joining kernel
    const long long g0 = (long long)group * a.tokens_per_gate;
    const long long g1 = min((long long)a.tokens, g0 + a.tokens_per_gate);
    const bool whole = g0 >= t0 && g1 <= t1;
    float4 v = scale4(a.beta, S);
    if (a.w_post) v = mul4(v, ld4(a.w_post + i));
    float *dst = (whole ? a.dgate + (size_t)group * a.d
                        : a.part_gate + ((size_t)blk * 2 + (group != group0)) * a.d) + i;
    if (whole && a.accumulate) v = add4(v, ld4(dst));
    *reinterpret_cast<float4 *>(dst) = v;
  }
}

// One block per run of rows (CH <= 4 chunks a thread).  Column sums stay in
// registers, dw_post's in the block's own row of partials, so every order is
// fixed.  A tensor that is not given has zeros in its part of the ring.
template <int CH, int R, bool CL, int YT, int UT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const BwdArgs a) {
  using X = Part<CH, T_F32>;
  using Y = Part<CH, YT>;
  using U = Part<CH, UT>;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float buf[2][96];
  peer_started_arrive<CL>();
  const int d = a.d, step = blockDim.x, half = cluster_half<CL>();
  const int dh = CL ? d / 2 : d, col0 = half * dh;  // this block's columns
  const int G = gridDim.x / (CL ? 2 : 1), blk = blockIdx.x / (CL ? 2 : 1);
  const int t0 = first_token(a.tokens, G, blk), t1 = first_token(a.tokens, G, blk + 1);
  const float inv_d = 1.f / (float)d;
  const unsigned valid = valid_chunks<CH>(dh);
  const int o_g = CH * step * 16, o_u = 2 * o_g, o_y = o_u + CH * step * U::B, slot_b = o_y + CH * step * Y::B;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    unsigned char *slot = ring + k * slot_b;
    X::clear(slot, step, a.du ? valid : 0u);
    X::clear(slot + o_g, step, a.dx_out ? valid : 0u);
    U::clear(slot + o_u, step, a.du ? valid : 0u);
    Y::clear(slot + o_y, step, a.y ? valid : 0u);
  }
  auto fetch = [&](int t, int k) {  // row t into slot k
    if (t < t1) {
      const uint32_t slot = ring_s + k * slot_b;
      if (a.du) {
        X::fetch(slot, row_at(a.x_out, t, d, col0, T_F32), step, valid);
        U::fetch(slot + o_u, row_at(a.du, t, d, col0, UT), step, valid);
      }
      if (a.dx_out) X::fetch(slot + o_g, row_at(a.dx_out, t, d, col0, T_F32), step, valid);
      if (a.y) Y::fetch(slot + o_y, row_at(a.y, t, d, col0, YT), step, valid);
    }
    cp_commit();
  };
  pdl_wait();
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < R; ++k) fetch(t0 + k, k);
  const bool post = a.y && a.post_norm;
  auto rr_of = [&](int t) { return a.du ? a.rstd_pre[t] : 0.f; };
  auto rp_of = [&](int t) { return post ? a.rstd_post[t] : 1.f; };
  auto col = [&](int c) { return col0 + (int)(threadIdx.x + c * step) * 4; };
  auto factor = [&](const float *gate_row, int c) {
    return valid >> c & 1u ? p4(branch_factor(gate_row, a.w_post, a.beta, col(c))) : p4(zero4());
  };
  P4 s_pre[CH], S[CH], bf[CH];
  int group = a.gate ? t0 / a.tokens_per_gate : 0;
  const int group0 = group;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    s_pre[c] = S[c] = p4(zero4());
    bf[c] = factor(a.gate ? a.gate + (size_t)group * d : nullptr, c);
  }
  bool post0 = true;  // part_post is empty
  auto flush = [&]() {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (valid >> c & 1u) flush_gate(a, blk, group, group0, t0, t1, col(c), f4(S[c]), post0);
      S[c] = p4(zero4());
    }
    post0 = false;
  };
  const unsigned long long alpha = pk(a.alpha, a.alpha);
  float rr_next = rr_of(t0), rp_next = rp_of(t0);
  peer_started_wait<CL>();
  int slot_i = 0;
  for (int t = t0; t < t1; ++t) {
    if (a.gate) {
      const int gi = t / a.tokens_per_gate;
      if (gi != group) {
        flush();
        group = gi;
#pragma unroll
        for (int c = 0; c < CH; ++c) bf[c] = factor(a.gate + (size_t)group * d, c);
      }
    }
    const float rr = rr_next, rp = rp_next;
    if (t + 1 < t1) rr_next = rr_of(t + 1), rp_next = rp_of(t + 1);
    const unsigned long long rr2 = pk(rr, rr), rp2 = pk(rp, rp);
    cp_wait<R - 1>();
    const unsigned char *slot = ring + slot_i * slot_b;
    P4 n[CH], m[CH], dr[CH];
    unsigned long long q0 = 0, q1 = 0, q2 = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      n[c] = mul(rr2, X::load(slot, c, step));
      m[c] = mul(rp2, Y::load(slot + o_y, c, step));
      P4 v = U::load(slot + o_u, c, step);
      s_pre[c] = fma(v, n[c], s_pre[c]);
      if (a.w_pre && (valid >> c & 1u)) v = mul(v, p4(ld4(a.w_pre + col(c))));
      q0 = dot(v, n[c], q0);
      dr[c] = fma(rr2, v, X::load(slot + o_g, c, step));  // dr without the term of c
      const P4 q = mul(bf[c], m[c]);
      q1 = dot(q, dr[c], q1);
      q2 = dot(q, n[c], q2);
    }
    fetch(t + R, slot_i);
    if (++slot_i == R) slot_i = 0;
    float s[3] = {sum2(q0), sum2(q1), sum2(q2)};
    row_sum<3, CL>(s, buf[t & 1]);
    const float cd = rr * s[0] * inv_d;                         // dr -= cd n
    const float ed = post ? (s[1] - cd * s[2]) * inv_d : 0.f;   // dy = rp (f dr - ed m)
    const unsigned long long cd2 = pk(-cd, -cd), ed2 = pk(-ed, -ed);
    void *dx = a.dx ? row_at(a.dx, t, d, col0, T_F32) : nullptr, *dy = a.dy ? row_at(a.dy, t, d, col0, YT) : nullptr;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const P4 d4 = fma(cd2, n[c], dr[c]);
      S[c] = fma(m[c], d4, S[c]);
      const P4 b = mul(rp2, fma(ed2, m[c], mul(bf[c], d4)));
      if (valid >> c & 1u) {
        if (dx) X::store(dx, c, step, mul(alpha, d4));
        if (dy) Y::store(dy, c, step, b);
      }
    }
  }
  if (a.y && (a.part_post || a.dgate)) flush();
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (a.part_pre && (valid >> c & 1u))
      *reinterpret_cast<float4 *>(a.part_pre + (size_t)blk * d + col(c)) = f4(s_pre[c]);
  if constexpr (CL) row_sync<CL>();  // the other block has written its last sums
}

// Joins the blocks' column sums in block order, 32 columns a block, in jobs
// along y: dw_post, dw_pre, and the gate rows that cross from one block's rows
// into the next's.  A gate row shared by many blocks (tokens_per_gate over 8
// blocks' rows) has a job of its own, summed by all warps; short ones, at most
// one per boundary between blocks, are dealt to the warps of kGateJobs jobs.
constexpr int kGateJobs = 16;
struct JoinArgs {
  const float *part_post, *part_pre, *part_gate;
  float *dw_post, *dw_pre, *dgate;
  int G, tokens, d, tokens_per_gate, accumulate;
  int long_rows;  // gate rows are long: job 2 + row has row
  int gate_jobs;
};
template <int NW>
__global__ void __launch_bounds__(NW * 32) norm_join_kernel(const JoinArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float buf[NW][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  const bool in = i < a.d;
  const int job = blockIdx.y;
  auto put = [&](float *out, float s) { *out = a.accumulate ? *out + s : s; };
  // blocks that hold tokens of gate row `row`: [b0, b1)
  auto blocks_of = [&](int row, int &b0, int &b1) {
    const long long g0 = (long long)row * a.tokens_per_gate, g1 = min((long long)a.tokens, g0 + a.tokens_per_gate);
    b1 = min(a.G, (int)((g1 * a.G + a.tokens - 1) / a.tokens));                       // blocks that begin before g1
    b0 = max(0, min(a.G, (int)(((g0 + 1) * a.G + a.tokens - 1) / a.tokens)) - 1);     // the last that begins by g0
  };
  // a block's first gate row is in its slot 0, another in slot 1: only the
  // first block of a row can have begun before the row
  auto row_part = [&](int c, int b0, int row) {
    const int slot = c == b0 && first_token(a.tokens, a.G, b0) < (long long)row * a.tokens_per_gate;
    return a.part_gate + ((size_t)c * 2 + slot) * a.d;
  };
  if (job < 2 || a.long_rows) {
    float *out = job == 0 ? a.dw_post : job == 1 ? a.dw_pre : a.dgate + (size_t)(job - 2) * a.d;
    const float *part = job == 0 ? a.part_post : job == 1 ? a.part_pre : a.part_gate;
    if (job < 2 && !out) return;
    int b0 = 0, b1 = a.G, stride = 1;
    if (job >= 2) {
      blocks_of(job - 2, b0, b1);
      if (b1 - b0 < 2) return;  // one block's alone: it is stored already
      stride = 2;
    }
    float s = 0.f;
    if (in) {
#pragma unroll 8
      for (int c = b0 + w; c < b1; c += NW)
        s += (c == b0 && job >= 2 ? row_part(c, b0, job - 2) : part + (size_t)c * stride * a.d)[i];
    }
    buf[w][lane] = s;
    __syncthreads();
    if (w == 0 && in) {
#pragma unroll
      for (int k = 1; k < NW; ++k) s += buf[k][lane];
      put(out + i, s);
    }
    return;
  }
  // the row at boundary b (between blocks b and b + 1), if the boundary is the first inside it
  for (int b = (job - 2) + a.gate_jobs * w; b < a.G - 1; b += a.gate_jobs * NW) {
    const int cut = first_token(a.tokens, a.G, b + 1), row = cut / a.tokens_per_gate;
    if (row * a.tokens_per_gate == cut) continue;
    int b0, b1;
    blocks_of(row, b0, b1);
    if (b0 != b || !in) continue;
    float s = 0.f;
    for (int c = b0; c < b1; ++c) s += row_part(c, b0, row)[i];
    put(a.dgate + (size_t)row * a.d + i, s);
  }
}

// ---------------------------------------------------------------- 8-bit quantiser
// Row r: scale = amax / 127, q = rint(x / scale) (fp32 quotient, ties to
// even).  A row of zeros has scale 0 and codes 0; a row that holds an
// infinity or a NaN has scale NaN and codes 0, so its products are NaN.
struct QuantArgs {
  const void *x;
  int8_t *q;
  float *scales;
  int rows, k;
};
// 8 elements as loaded: 16-bit types stay packed
template <int TYPE>
struct Eight {
  uint4 w[TYPE == T_F32 ? 2 : 1];
  PI_DEV void load(const void *p, size_t i) {
    const char *b = static_cast<const char *>(p) + i * (TYPE == T_F32 ? 4 : 2);
    w[0] = *reinterpret_cast<const uint4 *>(b);
    if constexpr (TYPE == T_F32) w[1] = *reinterpret_cast<const uint4 *>(b + 16);
  }
  PI_DEV void clear() {
#pragma unroll
    for (auto &x : w) x = make_uint4(0u, 0u, 0u, 0u);
  }
  // the larger of m and the largest bits of |x|: they order like the values,
  // and a NaN above all.  16-bit types: two halves of a word side by side.
  PI_DEV unsigned amax(unsigned m) const {
#pragma unroll
    for (const auto &x : w) {
      const unsigned v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = TYPE == T_F32 ? max(m, v[j] & 0x7fffffffu) : __vmaxu2(m, v[j] & 0x7fff7fffu);
    }
    return m;
  }
  PI_DEV void values(float (&v)[8]) const {
    if constexpr (TYPE == T_F32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[4 * h] = __uint_as_float(w[h].x), v[4 * h + 1] = __uint_as_float(w[h].y);
        v[4 * h + 2] = __uint_as_float(w[h].z), v[4 * h + 3] = __uint_as_float(w[h].w);
      }
    } else {
      const uint2 h[2] = {make_uint2(w[0].x, w[0].y), make_uint2(w[0].z, w[0].w)};
      const float4 a = ld4(h, 0, TYPE), b = ld4(h, 4, TYPE);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  }
};
// the value whose |.| has these bits (one half of a packed word for 16-bit types)
template <int TYPE>
PI_DEV unsigned f32_bits(unsigned bits) {
  if constexpr (TYPE == T_F32) return bits;
  else if constexpr (TYPE == T_BF16) return bits << 16;
  else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)bits)));
}
PI_DEV uint32_t low_bytes(const float *v) {
  const uint32_t a = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040);
  return __byte_perm(a, b, 0x5410);
}
// Codes of 8 elements.  By definition a code is the nearest integer to the
// fp32 quotient, ties to even.  x inv (inv = 1 / scale) is within 3e-5 of that
// quotient (127 x 2^-22), so where it is further than 1e-4 from a tie it
// rounds alike; adding 1.5 * 2^23 rounds it and leaves the code in the low byte.
// Elements nearer to a tie, and rows whose scale is too small for its inverse,
// divide.
PI_DEV uint2 codes8(const float (&v)[8], float scale, float inv) {
  constexpr float kRound = 12582912.f;
  float t[8], off = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = v[j] * inv;
    t[j] = x + kRound;
    off = fmaxf(off, fabsf(x - (t[j] - kRound)));
  }
  if (off > 0.4999f || inv == 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      t[j] = fminf(127.f, fmaxf(-127.f, rintf(__fdiv_rn(v[j], scale)))) + kRound;
  }
  return make_uint2(low_bytes(t), low_bytes(t + 4));
}

// One block per row; CH chunks of 8 elements a thread, all loads in flight
// together and kept as loaded until they are coded.  Rows longer than CH
// chunks a block (k > 32768) are read again from L2.
template <int TYPE, int CH>
__global__ void __launch_bounds__(1024) quantize_i8_kernel(const QuantArgs a) {
  __shared__ unsigned buf[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int step = blockDim.x * 8;
  for (int r = blockIdx.x, it = 0; r < a.rows; r += gridDim.x, ++it) {
    const size_t row = (size_t)r * a.k;
    Eight<TYPE> e[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x * 8 + c * step;
      if (i < a.k) e[c].load(a.x, row + i);
      else e[c].clear();
    }
    unsigned m = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) m = e[c].amax(m);
    for (int i = threadIdx.x * 8 + CH * step; i < a.k; i += step) {
      Eight<TYPE> t;
      t.load(a.x, row + i);
      m = t.amax(m);
    }
    if constexpr (TYPE != T_F32) m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    if (nw > 1) {
      if (lane == 0) buf[it & 1][warp] = m;
      __syncthreads();
      m = __reduce_max_sync(0xffffffffu, lane < nw ? buf[it & 1][lane] : 0u);
    }
    const unsigned amax = f32_bits<TYPE>(m);
    const bool bad = amax >= 0x7f800000u;
    const float scale = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(__uint_as_float(amax), 127.f);
    if (threadIdx.x == 0) a.scales[r] = scale;
    const bool zero = bad || scale == 0.f;
    const float inv = scale > 1e-30f ? __frcp_rn(scale) : 0.f;
    auto put = [&](int i, const Eight<TYPE> &t) {
      float v[8];
      t.values(v);
      *reinterpret_cast<uint2 *>(a.q + row + i) = zero ? make_uint2(0u, 0u) : codes8(v, scale, inv);
    };
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x * 8 + c * step;
      if (i < a.k) put(i, e[c]);
    }
    for (int i = threadIdx.x * 8 + CH * step; i < a.k; i += step) {
      Eight<TYPE> t;
      t.load(a.x, row + i);
      put(i, t);
    }
  }
}

}  // namespace norm
}  // namespace pi
