// pi_dense.cu -- C ABI of the dense products: the gated feed-forward block and
// its gradients, the 8-bit product.  Host validation, workspace layout and kernel dispatch; the declarations and
// argument contracts live in include/pi_ffn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <new>

#include "pi_ffn.h"
#include "pi_gemm.cuh"
#include "pi_host.cuh"

struct pi_gated_ffn {
  pi_gated_ffn_desc d;
  // weight maps (valid when maps_ok): 64-row boxes of each matrix, which serve
  // as K-major rows of 64 neurons and as MN-major 64 x 64 blocks, and boxes of
  // 128 neurons
  bool maps_ok;
  CUtensorMap gate64, up64, gate128, up128, down64, down128;
};

namespace {

using namespace pi::host;
namespace GM = pi::gemm;

constexpr int kMaxI8K = 131056;        // 128 * 128 * K stays below 2^31
constexpr int kMaxDim = 1 << 20;
constexpr int kMaxSplit = 8;  // CTAs of a cluster

template <int EPI, int AMN, int BMN, int MB, int NT, typename T>
cudaError_t pair_launch(const GM::Args &a, int sms, cudaStream_t st) {
  static DeviceOnce once;
  GM::Args b = a;
  // The side with fewer tiles is swept for each step along the other, so that
  // the larger operand is read once and the smaller stays in L2: forward of
  // 2048 x 8192 x 28672 2160 us with m sweeps of 1, 2185 of 4, 2215 of 8, 2470 of
  // 16; backward of 4096 x 5120 x 13824 2710, 2658, 2624 (its dW: 10 x 54 tiles).
  // Sweeps of more than 24 tiles would not stay in L2.
  b.gm = (a.mt <= a.nt ? a.mt : a.nt) > 24 ? 8 : a.mt <= a.nt ? a.mt : 1;
  const long long tiles = (long long)a.nprob * a.mt * a.nt;
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  return launch1(GM::pair_gemm_kernel<EPI, AMN, BMN, MB, NT, T>, dim3(2 * pairs), GM::kPairThreads,
                 GM::PairShape<EPI, MB, NT>::SMEM, 0, &once, st, b, GM::PairShape<EPI, MB, NT>::SMEM);
}
// Clusters of `split` CTAs with the split kernel's shape that the device holds
// at once (cached per device).  Asked for an empty kernel: for one that
// allocates tensor memory the occupancy calculator answers with one CTA per
// SM, whatever it allocates, but the hardware runs two.
__global__ void __launch_bounds__(GM::kSplitThreads) shape_kernel() {}
// The largest of the widths' shapes, so that what the device holds of it, it
// holds of each.
constexpr int kSplitSmem = GM::SplitShape<48>::SMEM;
struct ClusterCaps {
  int n[kMaxSplit + 1];  // by split; 0: does not run
};
const ClusterCaps *cluster_caps() {
  static std::mutex mu;
  static std::atomic<const ClusterCaps *> ready[64];
  static ClusterCaps caps[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  if (const ClusterCaps *c = ready[dev].load(std::memory_order_acquire)) return c;
  std::lock_guard<std::mutex> lock(mu);
  if (const ClusterCaps *c = ready[dev].load(std::memory_order_acquire)) return c;  // another thread was first
  if (cudaFuncSetAttribute(shape_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
      cudaFuncSetAttribute(shape_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess)
    return nullptr;
  for (int split = 1; split <= kMaxSplit; ++split) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(GM::kSplitThreads);
    cfg.dynamicSmemBytes = kSplitSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, shape_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    caps[dev].n[split] = n;
  }
  ready[dev].store(&caps[dev], std::memory_order_release);
  return &caps[dev];
}
template <int EPI, int AMN, int NT, typename T>
cudaError_t split_launch(const GM::Args &a, int split, cudaStream_t st) {
  static DeviceOnce once;
  using Sh = GM::SplitShape<NT>;
  static_assert(Sh::SMEM <= kSplitSmem, "the capacities are asked for a smaller block");
  const auto kern = GM::split_gemm_kernel<EPI, AMN, NT, T>;
  cudaError_t e = once.ensure([&] {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    return r != cudaSuccess ? r
                            : cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                   cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  return launch1(kern, dim3((unsigned)(a.mt * a.nt * split)), GM::kSplitThreads, Sh::SMEM, split, nullptr, st, a);
}

// The products of this file, each with tilings of its own.
enum Product { P_GLU, P_STORE, P_DGLU, P_WEIGHT, P_I8, kProducts };

// How a product runs.  nt: token columns of a tile; mb: 256-row blocks of a
// CTA-pair tile; split: 0 = CTA-pair kernel, else the split-K kernel with
// clusters of that many CTAs.  nt = 0: none (the device could not be asked).
struct Plan {
  int nt, mb, split;
  int b_rows() const { return split ? nt : nt / 2; }  // rows of the B box
};

// Tilings of the CTA-pair kernel that are built for a product, and the cycles
// of its epilogue for a block of 256 columns.
struct Tilings {
  int n;
  struct {
    int mb, nt;
  } t[8];
  double epilogue;
};
// 160 to 224 columns waste fewer of the last tile's where tokens are not a
// multiple of 256: with them 619 tokens of 8128 x 28176 take 741 to 773 us (bf16
// normal values), without 856
constexpr Tilings kGluTilings{5, {{2, 256}, {2, 224}, {2, 192}, {2, 160}, {2, 128}}, 9000};
constexpr Tilings kDgluTilings{5, {{1, 256}, {1, 224}, {1, 192}, {1, 160}, {1, 128}}, 10000};
constexpr Tilings kStoreTilings{
    8, {{2, 256}, {2, 224}, {2, 192}, {2, 160}, {1, 256}, {1, 192}, {1, 160}, {1, 128}}, 6000};
constexpr Tilings kWeightTilings{2, {{2, 256}, {1, 256}}, 6000};
// {2, 256} measured 10% slower (4096 x 5120 x 13824: 245 us, 224); 430 tokens of
// 4096 x 11008: 28.3 us with 160 to 224 columns, 31.4 without
constexpr Tilings kI8Tilings{5, {{1, 256}, {1, 224}, {1, 192}, {1, 160}, {1, 128}}, 7000};

const Tilings &tilings_of(int product) {
  static const Tilings *const all[kProducts] = {&kGluTilings, &kStoreTilings, &kDgluTilings, &kWeightTilings,
                                                &kI8Tilings};
  return *all[product];
}
// Token columns of the split kernel's tiles, and its cluster sizes: those of 3
// and 7 leave SMs with one CTA where others have two (333 tokens, 1032 x 2760,
// 66 tiles: 15.5 us split by 3, 13.2 by 4; 40 tiles of K 13824: 83.8 us by 7,
// 70.5 by 6).
constexpr int kSplitColumns[] = {16, 32, 48, 64, 128};
constexpr int kSplits[] = {1, 2, 4, 5, 6, 8};

// Test support (pi_debug_dense_plan): the tiling that a product's calls use; nt = 0: the rule's.
Plan g_forced[kProducts];

// Estimated SM cycles of the two kernels, to rank tilings by.  Their constants,
// and the epilogues' cycles above, are fitted, so that the rule takes the fastest
// tiling or one within 10% of it in forced sweeps of 18 products (16 to 4096
// tokens, 16 and 8 bits); they are no measured rates (at 300 tokens of 4096 x
// 11008 an SM draws 37 to 40 B a cycle).  A tiling's K blocks cost the slower
// of the MMAs (2 cycles a column and block), the arrival of its bytes at the
// SMs' share of the L2 (about 6 KB a cycle in all, 60 B at most for one SM) and,
// for the split kernel, the latency of a load over the ring's depth.
double pair_cost(long long tiles, int pairs, int kb, int mb, int nt, double epilogue, bool glu) {
  const long long rounds = (tiles + pairs - 1) / pairs;
  const double active = 2.0 * (tiles < pairs ? tiles : pairs);
  const double rate = 6200.0 / active < 60.0 ? 6200.0 / active : 60.0;
  const double mma = 2.0 * mb * nt, load = (mb * 16384 + nt * 64) / rate;
  const double main = kb * (mma > load ? mma : load);
  const double epi = epilogue * nt / 256.0 * (glu ? 1 : mb);
  // two accumulator buffers: the epilogue of a tile runs under the next one's MMAs; one: about half of it does
  const double body = mb * nt > 256 ? rounds * (main + 0.5 * epi) + 0.5 * epi
                                    : rounds * (main > epi ? main : epi) + (main > epi ? epi : main);
  return body + 5000.0;
}
// ntn: tiles along n, which share the weights that come from HBM (3450 B a
// cycle in all, 19 B for one CTA: one token, 5120 x 13824, 108 tiles: 36 us
// unsplit, 25.5 split by 2, 30.7 by 4, whose clusters take two rounds).
double split_cost(long long tiles, int ntn, int kb, int nt, int split, int cap) {
  const int ns = GM::split_stages(nt);
  const long long rounds = (tiles + cap - 1) / cap;
  const double active = (double)(tiles < cap ? tiles : cap) * split, stage = 16384.0 + nt * 128.0;
  const double hbm = 16384.0 / ntn / (3450.0 / active < 19.0 ? 3450.0 / active : 19.0);
  const double load = stage * active / 6200.0, lat = 2200.0 / ns;
  double per = load > lat ? load : lat;
  if (hbm > per) per = hbm;
  const double join = nt * 32.0 / split / GM::kSplitThreads * 180.0 + (split > 1 ? 800.0 : 0.0);
  return rounds * ((double)((kb + split - 1) / split) * per + 2200.0 + join) + 3000.0;
}

// m_rows: features of a 128-row block (64 for the gate | up product).
Plan choose(Product product, int m, int m_rows, int n, int kb, int sms) {
  if (const Plan &p = g_forced[product]; p.nt) return p.split > 1 && p.split * 2 > kb ? Plan{} : p;
  const Tilings &tilings = tilings_of(product);
  Plan best{};
  double cost = 0;
  const ClusterCaps *caps = cluster_caps();
  if (!caps) return best;
  const bool glu = m_rows == 64;
  if (n > 128)
    for (int i = 0; i < tilings.n; ++i) {
      const auto &t = tilings.t[i];
      const double c = pair_cost((long long)cdiv(m, 2 * t.mb * m_rows) * cdiv(n, t.nt), sms / 2, kb, t.mb, t.nt,
                                 tilings.epilogue, glu);
      if (cost == 0 || c < cost) cost = c, best = Plan{t.nt, t.mb, 0};
    }
  for (const int nt : kSplitColumns) {
    const long long tiles = (long long)cdiv(m, m_rows) * cdiv(n, nt);
    if (tiles > 65536) continue;
    for (const int split : kSplits) {
      if (split > 1 && split * 2 > kb) break;
      const int cap = caps->n[split];
      if (cap <= 0) continue;
      const double c = split_cost(tiles, cdiv(n, nt), kb, nt, split, cap);
      if (cost == 0 || c < cost) cost = c, best = Plan{nt, 1, split};
    }
    if (nt >= n) break;
  }
  return best;
}

uint32_t idesc(int dtype, bool i8, int M, int N, int a_mn, int b_mn) {
  const uint32_t fmt = i8 ? 1u : dtype == PI_DT_BF16 ? 1u : 0u;
  return (i8 ? 2u : 1u) << 4 | fmt << 7 | fmt << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 |
         (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// the tilings of the tables above
template <int EPI, int AMN, int MB, typename T>
cudaError_t pair_dispatch(const GM::Args &a, int nt, int sms, cudaStream_t st) {
  if constexpr (EPI == GM::E_GLU || !(EPI == GM::E_STORE && MB == 2))
    if (nt == 128) return pair_launch<EPI, AMN, 0, MB, 128, T>(a, sms, st);
  if constexpr (!(EPI == GM::E_STORE && MB == 1))
    if (nt == 224) return pair_launch<EPI, AMN, 0, MB, 224, T>(a, sms, st);
  switch (nt) {
  case 160:
    return pair_launch<EPI, AMN, 0, MB, 160, T>(a, sms, st);
  case 192:
    return pair_launch<EPI, AMN, 0, MB, 192, T>(a, sms, st);
  default:
    return pair_launch<EPI, AMN, 0, MB, 256, T>(a, sms, st);
  }
}

void set_waits(GM::Args &a) {
  a.wait_ns = g_wait_fault.limit_ns ? g_wait_fault.limit_ns : pi::tc::kWaitNs;
  a.withhold = g_wait_fault.withhold >= 0;
}

template <int EPI, int AMN, typename T>
cudaError_t run_plan(GM::Args &a, const Plan &p, int dtype, int m_rows, int sms, cudaStream_t st) {
  if (!p.nt) return cudaErrorUnknown;
  set_waits(a);
  a.mt = cdiv(a.m, p.split ? m_rows : 2 * p.mb * m_rows);
  a.nt = cdiv(a.n, p.nt);
  a.idesc = idesc(dtype, EPI == GM::E_I8, p.split ? 128 : 256, p.nt, AMN, 0);
  if (!p.split) {
    if constexpr (EPI == GM::E_GLU) return pair_dispatch<EPI, AMN, 2, T>(a, p.nt, sms, st);
    if constexpr (EPI == GM::E_STORE)
      if (p.mb == 2) return pair_dispatch<EPI, AMN, 2, T>(a, p.nt, sms, st);
    if constexpr (EPI != GM::E_GLU) return pair_dispatch<EPI, AMN, 1, T>(a, p.nt, sms, st);
  }
  switch (p.nt) {
  case 16:
    return split_launch<EPI, AMN, 16, T>(a, p.split, st);
  case 32:
    return split_launch<EPI, AMN, 32, T>(a, p.split, st);
  case 48:
    return split_launch<EPI, AMN, 48, T>(a, p.split, st);
  case 64:
    return split_launch<EPI, AMN, 64, T>(a, p.split, st);
  default:
    return split_launch<EPI, AMN, 128, T>(a, p.split, st);
  }
}

// ---------------------------------------------------------------- gated feed-forward block
struct FfnWs {
  int *status;
  char *a, *dg, *dp;
};
size_t act_bytes(const pi_gated_ffn *h, int tokens) { return align_up((size_t)tokens * h->d.d_ffn * 2, 256); }
size_t ffn_ws_bytes(const pi_gated_ffn *h, int tokens, bool backward) {
  return kHeader + act_bytes(h, tokens) * (backward ? 3 : 1);
}
pi_status ffn_ws(const pi_gated_ffn *h, int tokens, bool backward, void *ws, size_t ws_bytes, FfnWs *w) {
  if (!ws) return PI_ERR_WORKSPACE;
  if (!aligned16(ws)) return PI_ERR_MISALIGNED;
  if (ws_bytes < ffn_ws_bytes(h, tokens, backward)) return PI_ERR_WORKSPACE;
  char *b = static_cast<char *>(ws);
  const size_t n = act_bytes(h, tokens);
  *w = FfnWs{reinterpret_cast<int *>(b), b + kHeader, b + kHeader + n, b + kHeader + 2 * n};
  return PI_OK;
}

// a row-major [rows x cols] matrix of 16-bit elements as K-major token rows or as MN-major blocks
bool map16(CUtensorMap *m, const void *p, int rows, int cols, int box_rows) {
  return map_2d(m, p, true, (uint64_t)cols, (uint64_t)rows, 64, (uint32_t)box_rows, true);
}

template <typename T>
pi_status ffn_forward(const pi_gated_ffn *h, const void *u, int tokens, void *y, void *gate, void *up, const FfnWs &w,
                      cudaStream_t st) {
  const int d = h->d.d_model, f = h->d.d_ffn, dt = h->d.dtype;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  {
    GM::Args a{};
    a.m = f, a.n = tokens, a.nprob = 1;
    a.kb = a.kb_seg = cdiv(d, 64);
    const Plan p = choose(P_GLU, f, 64, tokens, a.kb, sms);
    a.ma[0] = p.split ? h->gate64 : h->gate128, a.ma[1] = p.split ? h->up64 : h->up128;
    if (!map16(&a.mb[0], u, tokens, d, p.b_rows())) return PI_ERR_CUDA;
    a.out[0] = w.a;
    a.ldo = f;
    a.act = h->d.act;
    a.gate_out = gate, a.up_out = up;
    a.status = w.status;
    PI_CUDA((run_plan<GM::E_GLU, 0, T>(a, p, dt, 64, sms, st)));
  }
  GM::Args a{};
  a.m = d, a.n = tokens, a.nprob = 1;
  a.kb = a.kb_seg = cdiv(f, 64);
  const Plan p = choose(P_STORE, d, 128, tokens, a.kb, sms);
  a.ma[0] = h->down64;
  if (!map16(&a.mb[0], w.a, tokens, f, p.b_rows())) return PI_ERR_CUDA;
  a.out[0] = y;
  a.ldo = d;
  a.out_type = dt;
  a.early_a = 1;  // the product above does not write the weights
  a.status = w.status;
  PI_CUDA((run_plan<GM::E_STORE, 1, T>(a, p, dt, 128, sms, st)));
  return PI_OK;
}

template <typename T>
pi_status ffn_backward(const pi_gated_ffn *h, const void *u, const void *gate, const void *up, const void *dy,
                       int tokens, void *du, void *dw_gate, void *dw_up, void *dw_down_t, int grad_dtype, int acc,
                       const FfnWs &w, cudaStream_t st) {
  const int d = h->d.d_model, f = h->d.d_ffn, dt = h->d.dtype;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  {
    // da = dy W2T^T, turned into dg, dp and a in the epilogue
    GM::Args a{};
    a.m = f, a.n = tokens, a.nprob = 1;
    a.kb = a.kb_seg = cdiv(d, 64);
    const Plan p = choose(P_DGLU, f, 128, tokens, a.kb, sms);
    a.ma[0] = h->down128;
    if (!map16(&a.mb[0], dy, tokens, d, p.b_rows())) return PI_ERR_CUDA;
    if (!p.split && (!map_2d(&a.ma[1], gate, true, (uint64_t)f, (uint64_t)tokens, 128, (uint32_t)p.nt, false) ||
                     !map_2d(&a.ma[2], up, true, (uint64_t)f, (uint64_t)tokens, 128, (uint32_t)p.nt, false)))
      return PI_ERR_CUDA;
    a.out[0] = w.a;
    a.ldo = f;
    a.act = h->d.act;
    a.gate_in = gate, a.up_in = up;
    a.gate_out = w.dg, a.up_out = w.dp;
    a.status = w.status;
    PI_CUDA((run_plan<GM::E_DGLU, 0, T>(a, p, dt, 128, sms, st)));
  }
  {
    // the matrices' gradients, [f x d] each: lanes along d, columns along f, K = tokens
    GM::Args a{};
    a.m = d, a.n = f;
    a.kb = a.kb_seg = cdiv(tokens, 64);
    CUtensorMap mu{}, mdy{};
    if (!map16(&mu, u, tokens, d, 64) || !map16(&mdy, dy, tokens, d, 64)) return PI_ERR_CUDA;
    const struct {
      void *out;
      const void *b;
      const CUtensorMap *a;
    } job[3] = {{dw_gate, w.dg, &mu}, {dw_up, w.dp, &mu}, {dw_down_t, w.a, &mdy}};
    for (const auto &j : job) {
      if (!j.out) continue;
      a.ma[a.nprob] = *j.a;
      if (!map16(&a.mb[a.nprob], j.b, tokens, f, 64)) return PI_ERR_CUDA;
      a.out[a.nprob++] = j.out;
    }
    if (a.nprob) {
      a.ldo = d;
      a.out_type = grad_dtype;
      a.accumulate = acc;
      a.status = w.status;
      double best = 0;
      int mb = 1;
      for (int i = 0; i < kWeightTilings.n; ++i) {
        const auto &t = kWeightTilings.t[i];
        const double c = pair_cost((long long)a.nprob * cdiv(d, 256 * t.mb) * cdiv(f, t.nt), sms / 2, a.kb, t.mb, t.nt,
                                   kWeightTilings.epilogue, false);
        if (i == 0 || c < best) best = c, mb = t.mb;
      }
      if (g_forced[P_WEIGHT].nt) mb = g_forced[P_WEIGHT].mb;
      set_waits(a);
      a.mt = cdiv(d, 256 * mb);
      a.nt = cdiv(f, 256);
      a.idesc = idesc(dt, false, 256, 256, 1, 1);
      PI_CUDA((mb == 2 ? pair_launch<GM::E_STORE, 1, 1, 2, 256, T>(a, sms, st)
                      : pair_launch<GM::E_STORE, 1, 1, 1, 256, T>(a, sms, st)));
    }
  }
  if (du) {
    // du = dg Wg + dp Wu: one product with K = [gate neurons, up neurons]
    GM::Args a{};
    a.m = d, a.n = tokens, a.nprob = 1;
    a.kb_seg = cdiv(f, 64);
    a.kb = 2 * a.kb_seg;
    const Plan p = choose(P_STORE, d, 128, tokens, a.kb, sms);
    a.ma[0] = h->gate64, a.ma[1] = h->up64;
    if (!map16(&a.mb[0], w.dg, tokens, f, p.b_rows()) || !map16(&a.mb[1], w.dp, tokens, f, p.b_rows()))
      return PI_ERR_CUDA;
    a.out[0] = du;
    a.ldo = d;
    a.out_type = dt;
    a.early_a = 1;  // the products above do not write the weights
    a.status = w.status;
    PI_CUDA((run_plan<GM::E_STORE, 1, T>(a, p, dt, 128, sms, st)));
  }
  return PI_OK;
}

}  // namespace

extern "C" {

// ====================================================================== gated feed-forward block
pi_status pi_gated_ffn_create(const pi_gated_ffn_desc *desc, pi_gated_ffn_t *out) {
  if (!desc || !out) return PI_ERR_INVALID_ARG;
  const pi_gated_ffn_desc &D = *desc;
  if (D.d_model <= 0 || D.d_ffn <= 0) return PI_ERR_INVALID_ARG;
  if (D.act != PI_GATE_SILU && D.act != PI_GATE_RELU && D.act != PI_GATE_GELU) return PI_ERR_INVALID_ARG;
  if (!is_type(D.dtype)) return PI_ERR_INVALID_ARG;
  if (!D.w_gate || !D.w_up || !D.w_down_t) return PI_ERR_INVALID_ARG;
  if (!is_half(D.dtype) || D.d_model % 8 || D.d_ffn % 8 || D.d_model > kMaxDim || D.d_ffn > kMaxDim)
    return PI_ERR_UNSUPPORTED;
  if (!aligned16(D.w_gate) || !aligned16(D.w_up) || !aligned16(D.w_down_t)) return PI_ERR_MISALIGNED;
  pi_gated_ffn *h = new (std::nothrow) pi_gated_ffn{};
  if (!h) return PI_ERR_INVALID_ARG;
  h->d = D;
  const int d = D.d_model, f = D.d_ffn;
  h->maps_ok = map16(&h->gate64, D.w_gate, f, d, 64) && map16(&h->up64, D.w_up, f, d, 64) &&
               map16(&h->gate128, D.w_gate, f, d, 128) && map16(&h->up128, D.w_up, f, d, 128) &&
               map16(&h->down64, D.w_down_t, f, d, 64) && map16(&h->down128, D.w_down_t, f, d, 128);
  *out = h;
  return PI_OK;
}

void pi_gated_ffn_destroy(pi_gated_ffn_t h) { delete h; }

pi_status pi_gated_ffn_workspace_size(pi_gated_ffn_t h, int max_tokens, int backward, size_t *bytes) {
  if (!h || !bytes) return PI_ERR_INVALID_ARG;
  if (max_tokens < 0 || max_tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  *bytes = ffn_ws_bytes(h, max_tokens, backward != 0);
  return PI_OK;
}

pi_status pi_gated_ffn_forward(pi_gated_ffn_t h, const void *u, int tokens, void *y, void *gate, void *up, void *ws,
                               size_t ws_bytes, pi_stream_t stream) {
  if (!h) return PI_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  if (tokens == 0) return PI_OK;
  if (!u || !y) return PI_ERR_INVALID_ARG;
  if (!aligned16(u) || !aligned16(y) || (gate && !aligned16(gate)) || (up && !aligned16(up))) return PI_ERR_MISALIGNED;
  FfnWs w;
  const pi_status s = ffn_ws(h, tokens, false, ws, ws_bytes, &w);
  if (s != PI_OK) return s;
  const size_t td = (size_t)tokens * h->d.d_model * 2, tf = (size_t)tokens * h->d.d_ffn * 2;
  const size_t wb = (size_t)h->d.d_ffn * h->d.d_model * 2;
  const Range r[] = {{y, td}, {gate, tf},        {up, tf},        {ws, ffn_ws_bytes(h, tokens, false)},
                     {u, td}, {h->d.w_gate, wb}, {h->d.w_up, wb}, {h->d.w_down_t, wb}};
  if (overlapping(r, 4, 8)) return PI_ERR_INVALID_ARG;
  if (!h->maps_ok) return PI_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  return h->d.dtype == PI_DT_F16 ? ffn_forward<__half>(h, u, tokens, y, gate, up, w, st)
                                 : ffn_forward<__nv_bfloat16>(h, u, tokens, y, gate, up, w, st);
}

pi_status pi_gated_ffn_backward(pi_gated_ffn_t h, const void *u, const void *gate, const void *up, const void *dy,
                                int tokens, void *du, void *dw_gate, void *dw_up, void *dw_down_t, int grad_dtype,
                                unsigned flags, void *ws, size_t ws_bytes, pi_stream_t stream) {
  if (!h) return PI_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  if (tokens && (!u || !gate || !up || !dy)) return PI_ERR_INVALID_ARG;
  if (!is_type(grad_dtype) || (flags & ~(unsigned)PI_GRAD_ACCUMULATE)) return PI_ERR_INVALID_ARG;
  if (grad_dtype != PI_DT_F32 && grad_dtype != h->d.dtype) return PI_ERR_UNSUPPORTED;
  const void *ptrs[] = {u, gate, up, dy, du, dw_gate, dw_up, dw_down_t};
  for (const void *p : ptrs)
    if (p && !aligned16(p)) return PI_ERR_MISALIGNED;
  cudaStream_t st = (cudaStream_t)stream;
  const int acc = (flags & PI_GRAD_ACCUMULATE) ? 1 : 0;
  if (tokens == 0) {  // no tokens: the sums over them are zero
    const size_t n = (size_t)h->d.d_ffn * h->d.d_model * type_size(grad_dtype);
    void *const dw[] = {dw_gate, dw_up, dw_down_t};
    if (!acc)
      for (void *p : dw)
        if (p) PI_CUDA(cudaMemsetAsync(p, 0, n, st));
    return PI_OK;
  }
  FfnWs w;
  const pi_status s = ffn_ws(h, tokens, true, ws, ws_bytes, &w);
  if (s != PI_OK) return s;
  const size_t td = (size_t)tokens * h->d.d_model * 2, tf = (size_t)tokens * h->d.d_ffn * 2;
  const size_t fd = (size_t)h->d.d_ffn * h->d.d_model * type_size(grad_dtype);
  const size_t wb = (size_t)h->d.d_ffn * h->d.d_model * 2;
  const Range r[] = {{du, td},  {dw_gate, fd}, {dw_up, fd},       {dw_down_t, fd}, {ws, ffn_ws_bytes(h, tokens, true)},
                     {u, td},   {gate, tf},    {up, tf},          {dy, td},        {h->d.w_gate, wb},
                     {h->d.w_up, wb},          {h->d.w_down_t, wb}};
  if (overlapping(r, 5, 12)) return PI_ERR_INVALID_ARG;
  if (!h->maps_ok) return PI_ERR_CUDA;
  return h->d.dtype == PI_DT_F16
             ? ffn_backward<__half>(h, u, gate, up, dy, tokens, du, dw_gate, dw_up, dw_down_t, grad_dtype, acc, w, st)
             : ffn_backward<__nv_bfloat16>(h, u, gate, up, dy, tokens, du, dw_gate, dw_up, dw_down_t, grad_dtype, acc,
                                           w, st);
}

// ====================================================================== test support
pi_status pi_debug_dense_plan(int product, int mb, int nt, int split) {
  if (product == -1 && !mb && !nt && !split) {
    for (Plan &p : g_forced) p = Plan{};
    return PI_OK;
  }
  if (product < 0 || product >= kProducts) return PI_ERR_INVALID_ARG;
  bool built = false;
  if (split == 0) {
    const Tilings &t = tilings_of(product);
    for (int i = 0; i < t.n; ++i) built |= t.t[i].mb == mb && t.t[i].nt == nt;
  } else if (product != P_WEIGHT && mb == 1) {
    bool columns = false, size = false;
    for (const int c : kSplitColumns) columns |= c == nt;
    for (const int c : kSplits) size |= c == split;
    built = columns && size;
  }
  if (!built) return PI_ERR_INVALID_ARG;
  g_forced[product] = Plan{nt, mb, split};
  return PI_OK;
}

// ====================================================================== 8-bit product
pi_status pi_matmul_i8_workspace_size(int tokens, int n, int k, size_t *bytes) {
  if (!bytes || n <= 0 || k <= 0) return PI_ERR_INVALID_ARG;
  if (k % 16 || k > kMaxI8K || n > kMaxDim || tokens < 0 || tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  *bytes = kHeader;
  return PI_OK;
}

pi_status pi_matmul_i8(const int8_t *xq, const float *x_scales, const int8_t *wq, const float *w_scales,
                       const float *bias, int tokens, int n, int k, void *y, int y_dtype, void *ws, size_t ws_bytes,
                       pi_stream_t stream) {
  if (n <= 0 || k <= 0 || !is_type(y_dtype)) return PI_ERR_INVALID_ARG;
  if (k % 16 || k > kMaxI8K || n > kMaxDim || tokens < 0 || tokens > kMaxTokens) return PI_ERR_UNSUPPORTED;
  if (tokens == 0) return PI_OK;
  if (!xq || !x_scales || !wq || !w_scales || !y) return PI_ERR_INVALID_ARG;
  const void *ptrs[] = {xq, x_scales, wq, w_scales, bias, y};
  for (const void *p : ptrs)
    if (p && !aligned16(p)) return PI_ERR_MISALIGNED;
  if (!ws) return PI_ERR_WORKSPACE;
  if (!aligned16(ws)) return PI_ERR_MISALIGNED;
  if (ws_bytes < kHeader) return PI_ERR_WORKSPACE;
  const size_t t4 = (size_t)tokens * 4, n4 = (size_t)n * 4;
  const Range r[] = {{y, (size_t)tokens * n * type_size(y_dtype)}, {ws, kHeader}, {xq, (size_t)tokens * k},
                     {x_scales, t4}, {wq, (size_t)n * k}, {w_scales, n4}, {bias, n4}};
  if (overlapping(r, 2, 7)) return PI_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return PI_ERR_CUDA;
  GM::Args a{};
  a.m = n, a.n = tokens, a.nprob = 1;
  a.kb = a.kb_seg = cdiv(k, 128);
  const Plan p = choose(P_I8, n, 128, tokens, a.kb, sms);
  if (!map_2d(&a.ma[0], wq, false, (uint64_t)k, (uint64_t)n, 128, 128, true) ||
      !map_2d(&a.mb[0], xq, false, (uint64_t)k, (uint64_t)tokens, 128, (uint32_t)p.b_rows(), true))
    return PI_ERR_CUDA;
  a.out[0] = y;
  a.ldo = n;
  a.out_type = y_dtype;
  a.s_n = x_scales, a.s_m = w_scales, a.bias = bias;
  a.status = static_cast<int *>(ws);
  PI_CUDA((run_plan<GM::E_I8, 0, __half>(a, p, 0, 128, sms, (cudaStream_t)stream)));
  return PI_OK;
}

}  // extern "C"
