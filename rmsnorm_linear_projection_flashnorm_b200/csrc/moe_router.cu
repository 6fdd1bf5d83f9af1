// Router of fn_moe_swiglu: 1/rms of each row, the experts' logits, the choice
// of experts and their weights, sm_100a.
//
//   l_e = r sum_k x_k g_k R[e, k],  r = 1 / sqrt(mean x^2 + eps)
//   score softmax or sigmoid of l; top k by l, or by score + bias; ties to the
//   lower index, NaN below every number
//
// Which experts are chosen is a comparison of values that may lie close, so
// the logits are fp64 sums of exact fp32 products x R (16 significant bits);
// the result then does not depend on the order of the sum in any case a 32-bit
// reference could tell apart.
//
// Bound by latency: 2 E d bytes of router weight from L2 or HBM (0.5 MB at 128
// experts x 2048) and M E d multiply-adds.  One cluster of 8 CTAs takes 1, 2 or
// 4 rows (few enough that the clusters of 64 rows still fill the SMs), each
// CTA an eighth of the experts, a warp one expert at a time; the logits meet
// in distributed shared memory, and one warp per row selects.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace fn {
namespace router {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int RANKS = 8;
constexpr int PER_RANK = kMoeMaxExperts / RANKS;     // experts of one CTA, at most
constexpr int PER_LANE = kMoeMaxExperts / 32;

struct Smem {
  double dot[4][PER_RANK];     // [row][expert / RANKS]
  double part[WARPS];
  double r;
};

struct Params {
  const __nv_bfloat16* x;
  const float* g;
  const __nv_bfloat16* router;
  const float* bias;
  int M, d, E, k, sigmoid, renorm;
  float scale, eps;
  int* ids;            // workspace [M][k]
  float* weight;       // workspace [E][kMoeMaxRows]
  float* rinv;         // workspace [M]
  int* ids_out;        // the caller's, or null
  float* w_out;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int ROWS>
__global__ void __cluster_dims__(RANKS, 1, 1) __launch_bounds__(THREADS) router_kernel(const Params p) {
  __shared__ Smem sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int m0 = static_cast<int>(blockIdx.x / RANKS) * ROWS;
  grid_dependency_wait();
  grid_launch_dependents();
  const int nvec = p.d / 8;
  const uint4* xr[ROWS];
#pragma unroll
  for (int t = 0; t < ROWS; ++t)     // rows past M repeat the last one; nothing is stored for them
    xr[t] = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(min(m0 + t, p.M - 1)) * p.d);

  for (int e = rank + RANKS * warp; e < p.E; e += RANKS * WARPS) {
    const uint4* wr = reinterpret_cast<const uint4*>(p.router + static_cast<int64_t>(e) * p.d);
    double acc[ROWS];
#pragma unroll
    for (int t = 0; t < ROWS; ++t) acc[t] = 0.0;
#pragma unroll 4
    for (int i = lane; i < nvec; i += 32) {
      const uint4 wv = __ldg(wr + i);
      float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (p.g) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.g) + 2 * i);
        const float4 b = __ldg(reinterpret_cast<const float4*>(p.g) + 2 * i + 1);
        g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
      }
      const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int t = 0; t < ROWS; ++t) {
        const uint4 xv = __ldcg(xr[t] + i);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[t] = fma(static_cast<double>(bf16lo_to_f32(xw[j]) * bf16lo_to_f32(w[j])), static_cast<double>(g[2 * j]),
                       acc[t]);
          acc[t] = fma(static_cast<double>(bf16hi_to_f32(xw[j]) * bf16hi_to_f32(w[j])),
                       static_cast<double>(g[2 * j + 1]), acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
      const double s = warp_sum(acc[t]);
      if (lane == 0) sm.dot[t][e / RANKS] = s;
    }
  }
  const int m = m0 + rank;                  // the row this CTA selects for
  const bool mine = rank < ROWS && m < p.M;
  if (mine) {
    double ss = 0.0;
    const uint4* x = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(m) * p.d);
    for (int i = threadIdx.x; i < nvec; i += THREADS) {
      const uint4 v = __ldcg(x + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = bf16lo_to_f32(w[j]), b = bf16hi_to_f32(w[j]);
        ss += static_cast<double>(a * a) + static_cast<double>(b * b);
      }
    }
    ss = warp_sum(ss);
    if (lane == 0) sm.part[warp] = ss;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int w = 0; w < WARPS; ++w) s += sm.part[w];
      sm.r = 1.0 / sqrt(s / p.d + static_cast<double>(p.eps));
    }
  }
  cluster_sync_all();                       // every rank's logits (and this CTA's r) are in shared memory

  if (mine && warp == 0) {
    const double r = sm.r;
    auto logit = [&](int e) {
      return r * __longlong_as_double(static_cast<long long>(dsmem_ld_u64(dsmem_addr(&sm.dot[rank][e / RANKS], e % RANKS))));
    };
    double key[PER_LANE];
    double top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const int e = lane + 32 * j;
      key[j] = e < p.E ? logit(e) : -INFINITY;
      nan |= key[j] != key[j];
      top = fmax(top, key[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (__any_sync(0xffffffffu, nan)) top = NAN;
    // softmax: the sum over all experts where a weight or a key needs it
    double sum = 1.0;
    if (!p.sigmoid && (!p.renorm || p.bias)) {
      sum = 0.0;
      for (int j = 0; j * 32 < p.E; ++j)
        if (lane + 32 * j < p.E) sum += exp(logit(lane + 32 * j) - top);
      sum = warp_sum(sum);
    }
    auto score = [&](double l) { return p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / sum; };
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const int e = lane + 32 * j;
      if (p.bias && e < p.E) key[j] = score(key[j]) + static_cast<double>(__ldg(p.bias + e));
      if (key[j] != key[j]) key[j] = -INFINITY;
    }
    uint32_t taken = 0;
    int my_e = 0;
    for (int c = 0; c < p.k; ++c) {
      double best = -INFINITY;
      int be = kMoeMaxExperts;              // above every index: nothing left on this lane
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j) {
        const int e = lane + 32 * j;
        if (e < p.E && !((taken >> j) & 1u) && (be == kMoeMaxExperts || key[j] > best)) {
          best = key[j];
          be = e;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double ob = __shfl_xor_sync(0xffffffffu, best, o);
        const int oe = __shfl_xor_sync(0xffffffffu, be, o);
        if (oe != kMoeMaxExperts && (be == kMoeMaxExperts || ob > best || (ob == best && oe < be))) {
          best = ob;
          be = oe;
        }
      }
      if ((be & 31) == lane) taken |= 1u << (be >> 5);
      if (lane == c) my_e = be;
    }
    double w = lane < p.k ? score(logit(my_e)) : 0.0;
    if (p.renorm) w /= warp_sum(w);
    const float wf = static_cast<float>(w * static_cast<double>(p.scale));
    for (int e = lane; e < p.E; e += 32) p.weight[static_cast<int64_t>(e) * kMoeMaxRows + m] = 0.f;
    __syncwarp();
    if (lane < p.k) {
      p.weight[static_cast<int64_t>(my_e) * kMoeMaxRows + m] = wf;
      p.ids[m * p.k + lane] = my_e;
      if (p.ids_out) p.ids_out[m * p.k + lane] = my_e;
      if (p.w_out) p.w_out[m * p.k + lane] = wf;
    }
    if (lane == 0) p.rinv[m] = static_cast<float>(r);
  }
  cluster_sync_all();                       // peers stay until their logits have been read
}

template <int ROWS>
cudaError_t launch(const Params& p, cudaStream_t stream) {
  const int clusters = (p.M + ROWS - 1) / ROWS;
  return launch_pdl(router_kernel<ROWS>, static_cast<unsigned>(clusters * RANKS), THREADS, 0, stream, p);
}

}  // namespace router

cudaError_t launch_moe_router(const MoeArgs& a, int* ids, float* weight, float* rinv) {
  router::Params p;
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.g = a.g;
  p.router = static_cast<const __nv_bfloat16*>(a.router);
  p.bias = a.select_bias;
  p.M = static_cast<int>(a.M);
  p.d = static_cast<int>(a.d);
  p.E = static_cast<int>(a.E);
  p.k = a.top_k;
  p.sigmoid = a.sigmoid;
  p.renorm = a.renorm;
  p.scale = a.route_scale;
  p.eps = a.eps;
  p.ids = ids;
  p.weight = weight;
  p.rinv = rinv;
  p.ids_out = a.ids;
  p.w_out = a.weights;
  // rows per cluster: the clusters of 8 CTAs fill the SMs once
  const int64_t fit = a.num_sms / router::RANKS;
  if (a.M <= fit) return router::launch<1>(p, a.stream);
  if (a.M <= 2 * fit) return router::launch<2>(p, a.stream);
  return router::launch<4>(p, a.stream);
}

}  // namespace fn
