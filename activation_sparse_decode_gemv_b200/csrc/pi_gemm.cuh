// pi_gemm.cuh -- tcgen05 matrix-product kernels of the dense operators (the
// gated feed-forward block, its gradients, the 8-bit integer product).
//
// Every product is computed as D[m, n] = sum_k A[m, k] B[n, k] with the
// FEATURE axis (neurons, channels, columns of a weight) on m, the lanes of
// tensor memory, and the TOKEN axis on n, its columns.  Results are row-major
// in tokens, so a warp's 32 lanes store 32 consecutive features of one token:
// the epilogues write from registers, with no transposition.  One orientation
// also serves every token count: n is the small MMA extent when there are few
// tokens, and the weights always fill the 128 or 256 rows.
//
// Operands are 128-byte wide K blocks (64 16-bit or 128 8-bit elements),
// brought by TMA with the 128-byte swizzle and read in place by the MMA:
//   K-major  (row = one m or n, k contiguous):  box 64 k x R rows
//   MN-major (row = one k, m or n contiguous):  boxes 64 m x 64 k
// Elements outside a matrix read as zero, so ragged edges add exact zeros.
//
// Two kernels:
//   pair_gemm_kernel   many tiles: CTA pairs (cta_group::2), tiles of one or
//                      two 256-row blocks x NT columns, persistent; the
//                      epilogue of a tile runs under the next tile's MMAs
//                      (two accumulator buffers), or half of it does (one).
//                      In isolation the tensor pipe is 79% active (gate | up
//                      product of 4096 x 5120 x 13824, 16 bits; 84% in the
//                      weights' gradients, 89 and 93% in y and du; 78% in the
//                      8-bit product of 2011 tokens); back to back
//                      the 1000 W power cap bounds it: 1.31 PFLOP/s for 2048 x
//                      8192 x 28672 against 1.28 for three library products,
//                      where the L2 traffic of a block that each B tile
//                      serves twice counts for energy as much as for time.
//   split_gemm_kernel  few tokens: 128 x NT tiles, K split over a cluster's
//                      CTAs, partial sums joined through distributed shared
//                      memory in rank order (no workspace, no atomics).
//                      Bound by HBM: 5.9 TB/s of weights at one token, 5.3 at
//                      45 (5120 x 13824, 4096 x 16384); a small product is
//                      about 6 us, of which 0.7 set-up, 0.7 first load, 1 each
//                      cluster barrier, 1 to 3 the join.
// Every mbarrier wait is bounded; a wait that gives up records
// PI_ERR_TIMEOUT and the kernel ends.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pi_umma.cuh"

namespace pi {
namespace gemm {

using namespace tc;

enum Epi {
  E_STORE = 0,  // out[n, m] = D  (16-bit or fp32; optionally added to what is there)
  E_GLU = 1,    // rows are gate | up neurons: a = phi(g) p, and optionally g and p themselves
  E_DGLU = 2,   // D = da: dg = da p phi'(g), dp = da phi(g), a = phi(g) p
  E_I8 = 3      // int32 D: out[n, m] = D s_n s_m + bias_m
};
enum GateAct { G_SILU = 0, G_RELU = 1, G_GELU = 2 };
enum OutType { O_F32 = 0, O_F16 = 1, O_BF16 = 2 };

constexpr int kMaxMaps = 3;

struct Args {
  CUtensorMap ma[kMaxMaps], mb[kMaxMaps];  // operand maps, by problem or by K segment (E_DGLU: ma[1], ma[2] of g, p)
  int m, n;          // extents (E_GLU: m = neurons)
  int kb, kb_seg;    // K blocks per tile; per segment (kb = kb_seg x segments)
  int nprob;         // independent products of the same shape (1 segment each)
  int mt, nt;        // tiles along m and n
  int gm;            // m tiles walked together (CTA-pair kernel)
  uint32_t idesc;    // MMA instruction descriptor
  void *out[kMaxMaps];
  long long ldo;     // elements between consecutive n of out, gate_*, up_*
  int out_type;      // OutType
  int accumulate;    // E_STORE: add to out
  int act;           // GateAct
  const void *gate_in, *up_in;  // E_DGLU
  void *gate_out, *up_out;      // E_GLU: g, p (or null); E_DGLU: dg, dp
  const float *s_n, *s_m, *bias;  // E_I8
  int early_a;       // split kernel: A was written before the previous kernel; load it before that one ends
  int *status;
  unsigned long long wait_ns;  // bound of every mbarrier wait
  int withhold;      // test support: finished accumulators are not announced, so that the waits for them run out
};

// ---------------------------------------------------------------- PTX: clusters and CTA pairs
PI_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
PI_DEV uint32_t mapa(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// all threads of the cluster; orders shared memory accesses across it
PI_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
PI_DEV float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
PI_DEV void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
PI_DEV bool mbar_try_cluster(uint64_t *b, unsigned parity, unsigned hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}
// Bounded waits, by a.wait_ns: on a barrier that the other CTA of the pair may
// complete (CLUSTER), or this CTA's own.  A wait that gives up records a
// timeout and makes the CTA's other roles give up too.
template <bool CLUSTER>
__device__ __noinline__ bool wait_slow(uint64_t *b, unsigned parity, volatile int *abort_flag, const Args *a) {
  const unsigned long long t0 = now_ns();
  for (;;) {
    if (CLUSTER ? mbar_try_cluster(b, parity, 20000u) : mbar_try(b, parity, 20000u)) return true;
    if (*abort_flag) return false;
    if (now_ns() - t0 > a->wait_ns) {
      set_status(a->status, kStatusTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}
PI_DEV bool wait_cluster(uint64_t *b, unsigned parity, volatile int *abort_flag, const Args &a) {
  return mbar_try_cluster(b, parity, 0u) || wait_slow<true>(b, parity, abort_flag, &a);
}
PI_DEV bool wait_own(uint64_t *b, unsigned parity, volatile int *abort_flag, const Args &a) {
  return mbar_test(b, parity) || wait_slow<false>(b, parity, abort_flag, &a);
}

// TMA load into this CTA's shared memory that completes on a barrier of
// either CTA of the pair (bar: shared::cluster address)
PI_DEV void tma_load_2d_pair(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// the box at (x, y) into L2 (no shared memory, no completion)
PI_DEV void prefetch_l2_2d(const CUtensorMap *tm, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(tm)),
               "r"(x), "r"(y)
               : "memory");
}

template <int GROUP, bool I8>
PI_DEV void mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (GROUP == 2) {
    if constexpr (I8)
      asm volatile(
          "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
          " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
          "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
          : "memory");
    else
      asm volatile(
          "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
          " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
          "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
          : "memory");
  } else {
    if constexpr (I8)
      asm volatile(
          "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
          " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
          "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
          : "memory");
    else
      mma_ss(d, adesc, bdesc, idesc, accumulate);
  }
}
// arrive on the same barrier of both CTAs of the pair when all MMAs issued so far are done
PI_DEV void mma_commit_pair(uint64_t *b) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          su32(b)),
      "h"((uint16_t)3)
      : "memory");
}
PI_DEV void tmem_alloc_pair(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
PI_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// 16 columns of tensor memory into registers, as a load to be waited for: an
// epilogue starts the next columns' load before it works on the present ones.
PI_DEV void tmem_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// the loads started so far are done; r's values may be used after this only
PI_DEV void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
PI_DEV void as_floats(const uint32_t (&r)[16], float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}

// operand descriptor of K step j (32 bytes of k per row, or 16 k) in a stage
template <int MN>
PI_DEV uint64_t operand_desc(uint32_t base, int j) {
  // K-major: 8-row groups 1 KB apart.  MN-major: 64-element blocks 8 KB
  // apart, 8-k groups 1 KB apart.
  return MN ? sdesc(base + j * 2048, 8192, 1024, kSw128) : sdesc(base + j * 32, 16, 1024, kSw128);
}

// ---------------------------------------------------------------- element types
template <typename T> struct Elem;
template <> struct Elem<__half> {
  static PI_DEV __half from(float v) { return __float2half_rn(v); }
  static PI_DEV float to(__half v) { return __half2float(v); }
};
template <> struct Elem<__nv_bfloat16> {
  static PI_DEV __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
  static PI_DEV float to(__nv_bfloat16 v) { return __bfloat162float(v); }
};

// ---------------------------------------------------------------- gate activations
// phi and phi' in fp32; the caller rounds once.  e^-g = 2^(-g log2 e) and the
// reciprocal are the hardware's approximations (about 2^-22 relative, more by
// |g| 2^-24 from the exponent's rounding), far below that rounding.
PI_DEV float sigmoid(float g) {
  float t, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + t));
  return s;
}
// The normal distribution's tail Phi(-|g|) = erfc(x) / 2 = e^(-x^2) erfcx(x) / 2
// at x = |g| / sqrt 2; e = e^(-x^2) = e^(-g^2/2) is the density's factor too.
// With t = 1 / (1 + p x), erfcx(x) / t is smooth in t from x = 0 to infinity (1
// to p / sqrt pi), and a polynomial of degree 6 in t, fitted here with equal
// ripples of the relative error for p = 0.3725 and x up to 9.5 (beyond, e is
// flushed to zero), is within 6e-7 of it, 1e-6 in fp32.  It is the relative
// error that counts: at g = -4 the tail is 3e-5, and a formula for erf that is
// within 1.5e-7 leaves the tail off by a rounding of fp16, at g = -8 by 1%.
// What is left, up to 1e-5 at |g| = 12, is the rounding of e's exponent.
PI_DEV float normal_tail(float g, float &e) {
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * g * -0.72134752f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3725f * 0.70710678f, fabsf(g), 1.f)));
  float y = fmaf(t, -0.139686595f, 0.414458213f);
  y = fmaf(t, y, -0.16150991f);
  y = fmaf(t, y, 0.302709049f);
  y = fmaf(t, y, 0.158710572f);
  y = fmaf(t, y, 0.215473616f);
  y = fmaf(t, y, 0.209844972f);
  return 0.5f * t * y * e;
}
template <int ACT>
PI_DEV float gate_phi(float g) {
  if constexpr (ACT == G_SILU) return g * sigmoid(g);
  if constexpr (ACT == G_RELU) return g < 0.f ? 0.f : g;  // NaN stays NaN
  float e;
  const float t = normal_tail(g, e);
  return g * (g > 0.f ? 1.f - t : t);
}
template <int ACT>
PI_DEV void gate_phi_grad(float g, float &phi, float &slope) {
  if constexpr (ACT == G_SILU) {
    const float s = sigmoid(g);
    phi = g * s;
    slope = s * (1.f + g * (1.f - s));
  } else if constexpr (ACT == G_RELU) {
    phi = g < 0.f ? 0.f : g;
    slope = g > 0.f ? 1.f : 0.f;
  } else {
    float e;
    const float t = normal_tail(g, e), c = g > 0.f ? 1.f - t : t;
    phi = g * c;
    slope = fmaf(g * 0.39894228f, e, c);
  }
}

// ---------------------------------------------------------------- element epilogues
// NC consecutive columns n0.. of feature m (the lane's row); E_I8 sums are
// int32 bits.  16-bit matrices move as 4-byte words of two features: a lane
// pair swaps halves, so that the even lane holds both features of an even
// column and the odd lane those of the next column.  That costs 3 instructions
// an element where a guarded scalar form costs about 24.  Matrices of an odd
// row length (the 8-bit product's y only) take the scalar form.
template <typename T>
PI_DEV uint32_t pack2(float lo, float hi) {
  if constexpr (sizeof(T) == 2 && __is_same(T, __half)) {
    const __half2 w = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&w);
  } else {
    const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&w);
  }
}
template <typename T>
PI_DEV void unpack2(uint32_t w, float &lo, float &hi) {
  if constexpr (__is_same(T, __half)) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x, hi = f.y;
  } else {
    lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  }
}
// (column j, column j + 1) of one feature <-> (even feature, odd feature) of column j + (lane & 1)
PI_DEV uint32_t pair_swap(uint32_t w) {
  const uint32_t r = __shfl_xor_sync(0xffffffffu, w, 1);
  return __byte_perm(w, r, (threadIdx.x & 1) ? 0x3276 : 0x5410);
}
template <int NC, typename T>
PI_DEV void put_t(const Args &a, void *out, int m, int n0, const float (&v)[NC]) {
  if ((a.ldo & 1) == 0) {  // the number of features is even too
    const int n = n0 + (threadIdx.x & 1);
    char *p = reinterpret_cast<char *>(reinterpret_cast<T *>(out) + (size_t)n * a.ldo + (m & ~1));
    const long long step = 4 * a.ldo;
    const bool in = m < a.m;
    if (n0 + NC <= a.n) {
#pragma unroll
      for (int j = 0; j < NC; j += 2, p += step) {
        const uint32_t w = pair_swap(pack2<T>(v[j], v[j + 1]));
        if (in) *reinterpret_cast<uint32_t *>(p) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NC; j += 2, p += step) {
        const uint32_t w = pair_swap(pack2<T>(v[j], v[j + 1]));
        if (in && n + j < a.n) *reinterpret_cast<uint32_t *>(p) = w;
      }
    }
    return;
  }
  if (m >= a.m) return;
  T *p = reinterpret_cast<T *>(out) + (size_t)n0 * a.ldo + m;
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (n0 + j < a.n) p[(size_t)j * a.ldo] = Elem<T>::from(v[j]);
}
template <int NC>
PI_DEV void put_f32(const Args &a, void *out, int m, int n0, const float (&v)[NC]) {
  if (m >= a.m) return;
  float *p = reinterpret_cast<float *>(out) + (size_t)n0 * a.ldo + m;
  if (n0 + NC <= a.n) {
#pragma unroll
    for (int j = 0; j < NC; ++j, p += a.ldo) *p = v[j];
    return;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (n0 + j < a.n) p[(size_t)j * a.ldo] = v[j];
}
template <int NC, typename T>
PI_DEV void add_t(const Args &a, const void *out, int m, int n0, float (&v)[NC]) {
  const T *p = reinterpret_cast<const T *>(out) + (size_t)n0 * a.ldo + m;
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (m < a.m && n0 + j < a.n) {
      if constexpr (__is_same(T, float)) v[j] += p[(size_t)j * a.ldo];
      else v[j] += Elem<T>::to(p[(size_t)j * a.ldo]);
    }
}
// out: fp32 or T; acc: what is there is added first, and the sum is rounded once
template <int NC, typename T>
PI_DEV void put_cols(const Args &a, void *out, int m, int n0, float (&v)[NC], int type, int acc) {
  if (type == O_F32) {
    if (acc) add_t<NC, float>(a, out, m, n0, v);
    put_f32<NC>(a, out, m, n0, v);
  } else {
    if (acc) add_t<NC, T>(a, out, m, n0, v);
    put_t<NC, T>(a, out, m, n0, v);
  }
}

// features m .. m + 3 (m a multiple of 4) of token n
template <typename T>
PI_DEV void put_row4(const Args &a, void *out, int m, int n, const float (&v)[4]) {
  if (m >= a.m) return;
  T *p = reinterpret_cast<T *>(out) + (size_t)n * a.ldo + m;
  if ((a.ldo & 3) == 0) {  // the number of features is a multiple of 4 too
    if constexpr (__is_same(T, float)) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (m + j < a.m) {
      if constexpr (__is_same(T, float)) p[j] = v[j];
      else p[j] = Elem<T>::from(v[j]);
    }
}

template <int NC>
PI_DEV void epi_i8(const Args &a, int m, int n0, const float (&v)[NC]) {
  // scales may come from the kernel before this one, under which this one starts: no non-coherent loads
  const float sm = m < a.m ? a.s_m[m] : 0.f;
  const float b = m < a.m && a.bias ? a.bias[m] : 0.f;
  float o[NC], sn[NC];
  if (NC % 4 == 0 && n0 + NC <= a.n) {
#pragma unroll
    for (int j = 0; j + 3 < NC; j += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(a.s_n + n0 + j);
      sn[j] = f.x, sn[j + 1] = f.y, sn[j + 2] = f.z, sn[j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j) sn[j] = a.s_n[min(n0 + j, a.n - 1)];
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) o[j] = fmaf((float)__float_as_int(v[j]) * sn[j], sm, b);
  if (a.out_type == O_F32) put_f32<NC>(a, a.out[0], m, n0, o);
  else if (a.out_type == O_F16) put_t<NC, __half>(a, a.out[0], m, n0, o);
  else put_t<NC, __nv_bfloat16>(a, a.out[0], m, n0, o);
}

template <int NC, int ACT>
PI_DEV void dglu_act(const float (&da)[NC], const float (&g)[NC], const float (&p)[NC], float (&dg)[NC],
                     float (&dp)[NC], float (&av)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float phi, slope;
    gate_phi_grad<ACT>(g[j], phi, slope);
    dp[j] = da[j] * phi;
    dg[j] = da[j] * slope * p[j];  // da p alone may pass fp32 (bf16 inputs) where phi' is small or zero
    av[j] = phi * p[j];
  }
}
template <int NC>
PI_DEV void dglu(int act, const float (&da)[NC], const float (&g)[NC], const float (&p)[NC], float (&dg)[NC],
                 float (&dp)[NC], float (&av)[NC]) {
  if (act == G_SILU) dglu_act<NC, G_SILU>(da, g, p, dg, dp, av);
  else if (act == G_RELU) dglu_act<NC, G_RELU>(da, g, p, dg, dp, av);
  else dglu_act<NC, G_GELU>(da, g, p, dg, dp, av);
}
// NC columns of a 16-bit matrix of an even row length, as loaded: the lane
// pair's two features of column n0 + j + (lane & 1); zero outside.  pair_swap
// makes them two columns of the lane's feature.
template <int NC>
PI_DEV void load_words(const Args &a, const void *in, int m, int n0, uint32_t (&w)[NC / 2]) {
  const int n = n0 + (threadIdx.x & 1);
  const char *p = reinterpret_cast<const char *>(reinterpret_cast<const uint16_t *>(in) + (size_t)n * a.ldo + (m & ~1));
  const long long step = 4 * a.ldo;
#pragma unroll
  for (int j = 0; j < NC; j += 2, p += step)
    w[j / 2] = m < a.m && n + j < a.n ? *reinterpret_cast<const uint32_t *>(p) : 0u;
}

template <int NC>
PI_DEV void glu(int act, const float (&g)[NC], const float (&p)[NC], float (&o)[NC]) {
  if (act == G_SILU) {
#pragma unroll
    for (int j = 0; j < NC; ++j) o[j] = gate_phi<G_SILU>(g[j]) * p[j];
  } else if (act == G_RELU) {
#pragma unroll
    for (int j = 0; j < NC; ++j) o[j] = gate_phi<G_RELU>(g[j]) * p[j];
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j) o[j] = gate_phi<G_GELU>(g[j]) * p[j];
  }
}

// K block kb of a tile -> map index (segment) and element offset along K
PI_DEV void k_at(const Args &a, int prob, int kb, int &map, int &blk) {
  const int seg = kb / a.kb_seg;
  map = prob + seg;
  blk = kb - seg * a.kb_seg;
}

// Loads this CTA's 128 A rows of K block blk (row0: first feature; E_GLU: 64
// gate rows from ma[0], then 64 up rows from ma[1]).
template <int EPI, int AMN, typename Load>
PI_DEV void load_a(const Args &a, int map, int blk, int row0, uint32_t dst, Load load) {
  constexpr int KE = EPI == E_I8 ? 128 : 64;  // elements of a K block
  if constexpr (EPI == E_GLU) {
    load(dst, &a.ma[0], blk * KE, row0);
    load(dst + 8192, &a.ma[1], blk * KE, row0);
  } else if constexpr (AMN) {
    load(dst, &a.ma[map], row0, blk * 64);
    load(dst + 8192, &a.ma[map], row0 + 64, blk * 64);
  } else {
    load(dst, &a.ma[map], blk * KE, row0);
  }
}

// ================================================================ CTA-pair kernel
constexpr int kPairThreads = 320;  // producer, MMA issuer, 8 epilogue warps
constexpr int kPairEpi = 8;
constexpr int kLead = 2;           // one buffer of two blocks: K blocks that block 0 runs ahead of block 1

// A pair's tile is MB accumulator blocks of 256 rows (128 per CTA) x NT
// columns: MB x 256 features, or for E_GLU (MB = 2) the gate rows and the up
// rows of the same 256 neurons, so that a lane holds both of a neuron.  Two
// blocks halve the B reads per product: 48 KB a K block instead of 64 for the
// same MMAs (weight gradients of 4096 x 5120 x 13824 1313 us against 1399 to
// 1488).  Tensor memory holds BUFS tiles: the accumulators of two tiles
// alternate where they fit.
template <int EPI, int MB, int NT>
struct PairShape {
  static constexpr int NB = NT / 2;            // B rows that one CTA of the pair loads
  static constexpr int ABYTES = MB * 16384;    // MB x 128 rows x 128 bytes
  static constexpr int STAGE = ABYTES + NB * 128;
  static constexpr int FIT = (227 * 1024 - 1536) / STAGE;
  static constexpr int NS = FIT > 8 ? 8 : FIT;
  static constexpr int CTRL_OFF = NS * STAGE;
  static constexpr int SMEM = CTRL_OFF + 512 + 1024;  // + alignment slack
  static constexpr int BUFS = 2 * MB * NT <= 512 ? 2 : 1;
  static constexpr uint32_t TMEM_COLS = BUFS * MB * NT <= 256 ? 256 : 512;
  static_assert(NS >= 2 * kLead || BUFS == 2, "ring too shallow");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int NS>
struct Ctrl {
  uint64_t full[NS], empty[NS], accfull[4], accfree[4];  // acc*: by accumulator block
  uint32_t tmem;
  int abort_flag;
};

struct TileAt {
  int prob, m, n;  // tile indices
};
// Groups of gm m tiles walked together over all n tiles: the tiles in flight
// on the machine form a block of about gm x 74/gm, so each operand row is read
// from HBM once or twice and from L2 otherwise.
PI_DEV TileAt tile_at(const Args &a, int t) {
  const int GM = a.gm;
  const int per = a.mt * a.nt;
  TileAt r;
  r.prob = t / per;
  const int rem = t - r.prob * per;
  const int gsize = GM * a.nt;
  const int g = rem / gsize, in = rem - g * gsize;
  const int gm = min(GM, a.mt - g * GM);
  r.n = in / gm;
  r.m = g * GM + in - r.n * gm;
  return r;
}

template <int EPI, int AMN, int BMN, int MB, int NT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ Args a) {
  using S = PairShape<EPI, MB, NT>;
  constexpr bool I8 = EPI == E_I8;
  constexpr int BLKS = S::BUFS * MB;             // accumulator blocks in tensor memory
  static_assert(EPI != E_GLU || MB == 2, "gate block and up block");
  extern __shared__ unsigned char smem_raw[];
  // the same offset in both CTAs of the pair (the dynamic shared window starts at the same place)
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  using C_t = Ctrl<S::NS>;
  static_assert(sizeof(C_t) <= 512, "control block");
  C_t &C = *reinterpret_cast<C_t *>(smem + S::CTRL_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int tiles = a.nprob * a.mt * a.nt;

  if (tid == 0) {
    for (int s = 0; s < S::NS; ++s) {
      mbar_init(&C.full[s], 1);   // the leader's expect_tx; both CTAs' copies complete the bytes
      mbar_init(&C.empty[s], 1);  // the leader's commit
    }
    for (int b = 0; b < BLKS; ++b) {
      mbar_init(&C.accfull[b], 1);
      mbar_init(&C.accfree[b], 2 * kPairEpi);  // the epilogue warps of both CTAs
    }
    C.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_pair(&C.tmem, S::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = C.tmem;
  volatile int *abort_flag = &C.abort_flag;
  // accumulator block b of this CTA's tc-th tile, and the parity of that block's use
  auto buf_of = [](int tc, int b) { return S::BUFS == 2 ? (tc & 1) * MB + b : b; };
  auto par_of = [](int tc) { return (unsigned)(S::BUFS == 2 ? (tc >> 1) & 1 : tc & 1); };
  // first row of this CTA's half of block b of tile m
  auto row_of = [&](int m, int b) { return ((EPI == E_GLU ? m : m * MB + b) * 2 + rank) * 128; };

  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer (one lane)
    if (lane == 0) {
      int it = 0, s = 0;
      unsigned ph = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += npairs) {
        const TileAt at = tile_at(a, t);
        const int col0 = at.n * NT + rank * S::NB;
        if constexpr (EPI == E_DGLU) {
          // the tile's g and p into L2, one main loop ahead of the epilogue
          // that reads them (from HBM those reads left 783 TFLOP/s, from L2 1150)
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            const int row0 = row_of(at.m, b);
            if (row0 >= a.m) continue;
            prefetch_l2_2d(&a.ma[1], row0, at.n * NT);
            prefetch_l2_2d(&a.ma[2], row0, at.n * NT);
          }
        }
        for (int kb = 0; kb < a.kb; ++kb) {
          if (it >= S::NS && !wait_cluster(&C.empty[s], ph ^ 1u, abort_flag, a)) {
            ok = false;
            break;
          }
          const uint32_t dst = su32(smem + s * S::STAGE);
          const uint32_t bar = mapa(su32(&C.full[s]), 0);
          if (rank == 0) mbar_expect_tx(&C.full[s], 2 * S::STAGE);
          int map, blk;
          k_at(a, at.prob, kb, map, blk);
          auto load = [&](uint32_t d, const CUtensorMap *tm, int x, int y) { tma_load_2d_pair(d, tm, x, y, bar); };
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            if constexpr (EPI == E_GLU) load(dst + b * 16384, &a.ma[b], blk * 64, row_of(at.m, b));
            else load_a<EPI, AMN>(a, map, blk, row_of(at.m, b), dst + b * 16384, load);
          }
          const CUtensorMap *tb = &a.mb[map];
          if constexpr (BMN) {
#pragma unroll
            for (int h = 0; h < S::NB / 64; ++h) load(dst + S::ABYTES + h * 8192, tb, col0 + h * 64, blk * 64);
          } else {
            load(dst + S::ABYTES, tb, blk * (I8 ? 128 : 64), col0);
          }
          it = it < S::NS ? it + 1 : it;
          if (++s == S::NS) s = 0, ph ^= 1u;
        }
      }
      // the MMAs that read the last stages have finished before this CTA may go
      for (int j = 0; j < it && ok; ++j) {
        if (--s < 0) s = S::NS - 1, ph ^= 1u;
        ok = wait_cluster(&C.empty[s], ph, abort_flag, a);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (one lane of the leader CTA)
    if (rank == 0 && lane == 0) {
      int tc = 0, s = 0;
      unsigned ph = 0;
      bool ok = true;
      auto wait_full = [&](int st, unsigned p) { return wait_cluster(&C.full[st], p, abort_flag, a); };
      auto wait_free = [&](int b) {
        const bool r = tc < S::BUFS ||
                       wait_cluster(&C.accfree[buf_of(tc, b)], par_of(tc) ^ 1u, abort_flag, a);
        tc_fence_after();
        return r;
      };
      auto issue = [&](int b, int st, bool first) {
        const uint32_t base = su32(smem + st * S::STAGE);
        const uint32_t acc = tmem + (uint32_t)(buf_of(tc, b) * NT);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma<2, I8>(acc, operand_desc<AMN>(base + b * 16384, j), operand_desc<BMN>(base + S::ABYTES, j), a.idesc,
                     (first && j == 0) ? 0u : 1u);
      };
      for (int t = pair; t < tiles && ok; t += npairs, ++tc) {
        if constexpr (S::BUFS == 2) {
          for (int b = 0; b < MB && ok; ++b) ok = wait_free(b);
          if (!ok) break;
          for (int kb = 0; kb < a.kb; ++kb) {
            if (!(ok = wait_full(s, ph))) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < MB; ++b) issue(b, s, kb == 0);
            mma_commit_pair(&C.empty[s]);
            if (++s == S::NS) s = 0, ph ^= 1u;
          }
          if (ok && !a.withhold)
#pragma unroll
            for (int b = 0; b < MB; ++b) mma_commit_pair(&C.accfull[buf_of(tc, b)]);
        } else {
          // Block 0 runs kLead K blocks ahead of block 1 at both ends of the
          // tile: its epilogue starts while block 1's last MMAs run, and
          // block 1's epilogue ends under block 0's first MMAs of the next
          // tile.
          const int head = min(kLead, a.kb), tail = min(kLead, a.kb - head);
          int kb = 0;
          auto both = [&](int n, bool first, bool last) {  // n K blocks: all of block 0, then all of block 1
            int s0 = s;
            unsigned p0 = ph;
            for (int i = 0; i < n && ok; ++i) {
              if (!(ok = wait_full(s0, p0))) return;
              tc_fence_after();
              issue(0, s0, first && i == 0);
              if (++s0 == S::NS) s0 = 0, p0 ^= 1u;
            }
            if (last && !a.withhold) mma_commit_pair(&C.accfull[0]);
            if (first && !(ok = wait_free(1))) return;
            for (int i = 0; i < n; ++i) {
              issue(1, s, first && i == 0);
              mma_commit_pair(&C.empty[s]);
              if (++s == S::NS) s = 0, ph ^= 1u;
            }
            kb += n;
          };
          if (!(ok = wait_free(0))) break;
          both(head, true, tail == 0);
          while (ok && kb < a.kb - tail) both(1, false, false);
          if (ok && tail) both(tail, false, true);
          if (ok && !a.withhold) mma_commit_pair(&C.accfull[1]);
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue: lane quarter q, column half h
    const int q = warp & 3, h = (warp - 2) >> 2;
    int tc = 0;
    bool go = true;
    auto wait_acc = [&](int b) {
      const bool r = __all_sync(0xffffffffu, wait_cluster(&C.accfull[b], par_of(tc), abort_flag, a));
      tc_fence_after();
      return r;
    };
    auto free_acc = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa(su32(&C.accfree[b]), 0));
    };
    for (int t = pair; t < tiles && go; t += npairs, ++tc) {
      const TileAt at = tile_at(a, t);
      const int n0 = at.n * NT + h * (NT / 2);
      auto tmem_of = [&](int b) { return tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * NT + h * (NT / 2)); };
      // 16-column chunks of this warp inside the matrix; none where its rows are outside
      auto chunks_of = [&](int m) {
        return (m & ~31) < a.m ? min(NT / 32, max(0, (a.n - n0 + 15) / 16)) : 0;
      };
      if constexpr (EPI == E_GLU) {
        const int bg = buf_of(tc, 0), bu = buf_of(tc, 1);
        if (!(go = wait_acc(bg)) || !(go = wait_acc(bu))) break;
        const int m = row_of(at.m, 0) + q * 32 + lane, nchunks = chunks_of(m);
        const uint32_t tg = tmem_of(bg), tu = tmem_of(bu);
        uint32_t rg[16], ru[16];
        if (nchunks) {
          tmem_ld16_start(tg, rg);
          tmem_ld16_start(tu, ru);
        }
#pragma unroll 1
        for (int c = 0; c < nchunks; ++c) {
          const int nc = n0 + c * 16;
          float g[16], p[16], o[16];
          tmem_ld16_wait(rg);
          tmem_ld16_wait(ru);
          as_floats(rg, g);
          as_floats(ru, p);
          if (c + 1 < nchunks) {
            tmem_ld16_start(tg + (c + 1) * 16, rg);
            tmem_ld16_start(tu + (c + 1) * 16, ru);
          }
          if (a.gate_out) put_t<16, T>(a, a.gate_out, m, nc, g);
          if (a.up_out) put_t<16, T>(a, a.up_out, m, nc, p);
          glu<16>(a.act, g, p, o);
          put_t<16, T>(a, a.out[0], m, nc, o);
        }
        free_acc(bg);
        free_acc(bu);
      } else {
#pragma unroll 1
        for (int blk = 0; blk < MB; ++blk) {
          const int b = buf_of(tc, blk);
          const int m = row_of(at.m, blk) + q * 32 + lane, nchunks = chunks_of(m);
          const uint32_t tb = tmem_of(b);
          uint32_t gw[8], pw[8];
          if constexpr (EPI == E_DGLU) {
            if (nchunks) {
              load_words<16>(a, a.gate_in, m, n0, gw);
              load_words<16>(a, a.up_in, m, n0, pw);
            }
          }
          if (!(go = wait_acc(b))) break;
          uint32_t r[16];
          if (nchunks) tmem_ld16_start(tb, r);
#pragma unroll 1
          for (int c = 0; c < nchunks; ++c) {
            const int nc = n0 + c * 16;
            float v[16];
            tmem_ld16_wait(r);
            as_floats(r, v);
            if (c + 1 < nchunks) tmem_ld16_start(tb + (c + 1) * 16, r);
            if constexpr (EPI == E_DGLU) {
              float g[16], p[16], dg[16], dp[16], av[16];
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                unpack2<T>(pair_swap(gw[j / 2]), g[j], g[j + 1]);
                unpack2<T>(pair_swap(pw[j / 2]), p[j], p[j + 1]);
              }
              if (c + 1 < nchunks) {
                load_words<16>(a, a.gate_in, m, nc + 16, gw);
                load_words<16>(a, a.up_in, m, nc + 16, pw);
              }
              dglu<16>(a.act, v, g, p, dg, dp, av);
              put_t<16, T>(a, a.gate_out, m, nc, dg);
              put_t<16, T>(a, a.up_out, m, nc, dp);
              put_t<16, T>(a, a.out[0], m, nc, av);
            } else if constexpr (EPI == E_I8) {
              epi_i8<16>(a, m, nc, v);
            } else {
              put_cols<16, T>(a, a.out[at.prob], m, nc, v, a.out_type, a.accumulate);
            }
          }
          free_acc(b);
        }
      }
    }
  }
  if (*abort_flag) __nanosleep(1000000);  // copies in flight land before the CTA goes
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, S::TMEM_COLS);
}

// ================================================================ split-K kernel
constexpr int kSplitThreads = 192;  // producer, MMA issuer, 4 epilogue warps

// ring depth with two CTAs per SM
__host__ __device__ constexpr int split_stages(int nt) { return nt <= 16 ? 6 : nt <= 48 ? 5 : nt <= 64 ? 4 : 3; }
template <int NT>
struct SplitShape {
  static constexpr int ABYTES = 16384;
  static constexpr int STAGE = ABYTES + NT * 128;
  static constexpr int NS = split_stages(NT);
  static constexpr int CTRL_OFF = NS * STAGE;
  static constexpr int SMEM = CTRL_OFF + 512 + 1024;
  static constexpr uint32_t TMEM_COLS = NT <= 32 ? 32 : NT <= 64 ? 64 : 128;
  static_assert(NT * 512 <= NS * STAGE, "the partial tile fits the ring");
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int EPI, int AMN, int NT, typename T>
__global__ void __launch_bounds__(kSplitThreads, 2) split_gemm_kernel(const __grid_constant__ Args a) {
  using S = SplitShape<NT>;
  constexpr bool I8 = EPI == E_I8;
  constexpr int MROWS = EPI == E_GLU ? 64 : 128;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  using C_t = Ctrl<S::NS>;
  C_t &C = *reinterpret_cast<C_t *>(smem + S::CTRL_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int split = (int)csize;
  const int tile = blockIdx.x / split;
  const int mtile = tile % a.mt, ntile = tile / a.mt;
  const int row0 = mtile * MROWS, col0 = ntile * NT;
  const int k0 = (int)((long long)a.kb * rank / split), k1 = (int)((long long)a.kb * (rank + 1) / split);

  volatile int *abort_flag = &C.abort_flag;
  auto start_a = [&](int kb, int st) {
    int map, blk;
    k_at(a, 0, kb, map, blk);
    mbar_expect_tx(&C.full[st], S::STAGE);
    load_a<EPI, AMN>(a, map, blk, row0, su32(smem + st * S::STAGE),
                     [&](uint32_t d, const CUtensorMap *tm, int x, int y) { tma_load_2d(d, tm, x, y, &C.full[st]); });
  };
  auto start_b = [&](int kb, int st) {
    int map, blk;
    k_at(a, 0, kb, map, blk);
    tma_load_2d(su32(smem + st * S::STAGE + S::ABYTES), &a.mb[map], blk * (I8 ? 128 : 64), col0, &C.full[st]);
  };
  const int first = min(S::NS, k1 - k0);  // K blocks that fill the ring
  if (tid == 0) {
    for (int s = 0; s < S::NS; ++s) {
      mbar_init(&C.full[s], 1);
      mbar_init(&C.empty[s], 1);
    }
    mbar_init(&C.accfull[0], 1);
    C.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    proxy_fence_async();
    // The producer is this thread: it fills the ring while the others set up.
    // Weights that the previous kernel of the same call does not write are
    // loaded before that one ends.
    if (a.early_a)
      for (int i = 0; i < first; ++i) start_a(k0 + i, i);
    pdl_wait();
    pdl_launch_dependents();  // after the wait: the next kernel may rely on everything before this one
    for (int i = 0; i < first; ++i) {
      if (!a.early_a) start_a(k0 + i, i);
      start_b(k0 + i, i);
    }
  }
  if (warp == 1) tmem_alloc(&C.tmem, S::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;
  bool fine = true;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (one lane)
    if (lane == 0) {
      for (int kb = k0 + first; kb < k1; ++kb) {
        const int i = kb - k0, s = i % S::NS;
        const unsigned ph = (unsigned)((i / S::NS) & 1);
        if (!wait_own(&C.empty[s], ph ^ 1u, abort_flag, a)) break;
        start_a(kb, s);
        start_b(kb, s);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (one lane)
    if (lane == 0) {
      bool ok = true;
      for (int kb = k0; kb < k1; ++kb) {
        const int i = kb - k0, s = i % S::NS;
        if (!wait_own(&C.full[s], (unsigned)((i / S::NS) & 1), abort_flag, a)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = su32(smem + s * S::STAGE);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma<1, I8>(tmem, operand_desc<AMN>(st, j), operand_desc<0>(st + S::ABYTES, j), a.idesc, (i | j) ? 1u : 0u);
        mma_commit(&C.empty[s]);
      }
      if (ok && !a.withhold) mma_commit(&C.accfull[0]);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ partial tile to shared memory
    const int q = warp & 3;
    float *red = reinterpret_cast<float *>(smem);
    fine = __all_sync(0xffffffffu, wait_own(&C.accfull[0], 0u, abort_flag, a));
    if (fine) {
      tc_fence_after();
      const int nv = min(NT, a.n - col0);
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        if (c * 16 < nv) {  // the same for the whole warp
          float v[16];
          tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c * 16, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) red[(c * 16 + j) * 128 + q * 32 + lane] = v[j];
        }
      }
    }
  }
  if (*abort_flag) __nanosleep(1000000);  // copies in flight land before the CTA goes
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA's partial tile is in its shared memory
  {
    // ------------------------------------------------------------ join: this CTA's slice of the tile, summed in rank order
    // (four features of a token at a time, two such items in flight a thread)
    constexpr int Q = MROWS / 4;
    const int nv = min(NT, a.n - col0);
    const int E = nv * Q;
    const int per = ((E + split * 32 - 1) / (split * 32)) * 32;
    const int e0 = rank * per, e1 = min(E, e0 + per);
    const uint32_t red = su32(smem);
    auto sum = [&](int e, float (&v)[4], float (&w)[4]) {
      const uint32_t off = red + (uint32_t)((e / Q) * 128 + (e % Q) * 4) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = w[j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < split; ++c) {
        const float4 f = ld_cluster_f32x4(mapa(off, c));
        if constexpr (I8) {
          v[0] = __int_as_float(__float_as_int(v[0]) + __float_as_int(f.x));
          v[1] = __int_as_float(__float_as_int(v[1]) + __float_as_int(f.y));
          v[2] = __int_as_float(__float_as_int(v[2]) + __float_as_int(f.z));
          v[3] = __int_as_float(__float_as_int(v[3]) + __float_as_int(f.w));
        } else {
          v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
          if constexpr (EPI == E_GLU) {
            const float4 g = ld_cluster_f32x4(mapa(off + 256, c));
            w[0] += g.x, w[1] += g.y, w[2] += g.z, w[3] += g.w;
          }
        }
      }
    };
    // E_DGLU: g and p of an item (rows of a multiple of 8 features)
    auto load_gp = [&](int e, uint4 &gp) {
      const int n = col0 + e / Q, m = row0 + (e % Q) * 4;
      if (m >= a.m) return;
      const size_t at = (size_t)n * a.ldo + m;
      const uint2 g = *reinterpret_cast<const uint2 *>(reinterpret_cast<const T *>(a.gate_in) + at);
      const uint2 p = *reinterpret_cast<const uint2 *>(reinterpret_cast<const T *>(a.up_in) + at);
      gp = make_uint4(g.x, g.y, p.x, p.y);
    };
    auto finish = [&](int e, float (&v)[4], float (&w)[4], const uint4 &gp) {
      const int n = col0 + e / Q, m = row0 + (e % Q) * 4;
      if (m >= a.m) return;
      if constexpr (EPI == E_GLU) {
        float o[4];
        glu<4>(a.act, v, w, o);
        if (a.gate_out) put_row4<T>(a, a.gate_out, m, n, v);
        if (a.up_out) put_row4<T>(a, a.up_out, m, n, w);
        put_row4<T>(a, a.out[0], m, n, o);
      } else if constexpr (EPI == E_I8) {
        const float sn = a.s_n[n];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int mj = min(m + j, a.m - 1);
          v[j] = fmaf((float)__float_as_int(v[j]) * sn, a.s_m[mj], a.bias ? a.bias[mj] : 0.f);
        }
        if (a.out_type == O_F32) put_row4<float>(a, a.out[0], m, n, v);
        else if (a.out_type == O_F16) put_row4<__half>(a, a.out[0], m, n, v);
        else put_row4<__nv_bfloat16>(a, a.out[0], m, n, v);
      } else if constexpr (EPI == E_DGLU) {
        float g[4], p[4], dg[4], dp[4], av[4];
        unpack2<T>(gp.x, g[0], g[1]);
        unpack2<T>(gp.y, g[2], g[3]);
        unpack2<T>(gp.z, p[0], p[1]);
        unpack2<T>(gp.w, p[2], p[3]);
        dglu<4>(a.act, v, g, p, dg, dp, av);
        put_row4<T>(a, a.gate_out, m, n, dg);
        put_row4<T>(a, a.up_out, m, n, dp);
        put_row4<T>(a, a.out[0], m, n, av);
      } else {
        // 16-bit results only: parameter gradients, which may be fp32 or accumulated, take the pair kernel
        put_row4<T>(a, a.out[0], m, n, v);
      }
    };
    for (int e = e0 + tid; e < e1; e += 2 * kSplitThreads) {
      float v0[4], w0[4], v1[4], w1[4];
      uint4 g0, g1;
      const bool two = e + kSplitThreads < e1;
      if constexpr (EPI == E_DGLU) {
        load_gp(e, g0);
        if (two) load_gp(e + kSplitThreads, g1);
      }
      sum(e, v0, w0);
      if (two) sum(e + kSplitThreads, v1, w1);
      finish(e, v0, w0, g0);
      if (two) finish(e + kSplitThreads, v1, w1, g1);
    }
  }
  tc_fence_before();
  cluster_sync();  // the others have read this CTA's partial tile
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::TMEM_COLS);
}

}  // namespace gemm
}  // namespace pi
