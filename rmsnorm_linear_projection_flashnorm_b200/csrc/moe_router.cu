// Router of fn_moe_swiglu: 1/rms of each row, the experts' logits, the choice
// of experts and their weights, sm_100a.
//
//   l_e = r sum_k x_k g_k R[e, k],  r = 1 / sqrt(mean x^2 + eps)
//   score softmax or sigmoid of l; top k by l, or by score + bias; ties to the
//   lower index, NaN as minus infinity
//
// Which experts are chosen is a comparison of values that may lie close, so
// the logits are fp64 sums of the products x g R (8 + 24 + 8 significant bits,
// exact in fp64), and the squares of the norm are fp64 too; the result then does
// not depend on the order of the sum in any case a 32-bit reference could tell
// apart.
//
// Bound by latency: 2 E d bytes of router weight from L2 or HBM (0.5 MB at 128
// experts x 2048) and M E d multiply-adds.  One cluster of 8 CTAs takes 1, 2 or
// 4 rows (few enough that the clusters of 64 rows still fill the SMs), each
// CTA an eighth of the experts.  All warps of a CTA share one expert's k range,
// so a thread has a vector of every expert of a group in flight at once, and
// x g is converted to 64 bits once per group.  The weight is widened by moving
// its bits: the 8-bit exponent in the 11-bit field makes the value times
// 2^-896, which the sum takes back, at two integer operations instead of a
// conversion at a quarter of their rate.
//
// The logits meet in distributed shared memory; the choice has no serial
// rounds: an expert's place is the number of experts that come before it, which
// every thread counts for its own experts.  One row, 64 experts x 2048, 8 chosen:
// 5.9 us; warps with an expert each, conversions and k rounds of a warp-wide
// maximum took 11.4.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dsmem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fn {
namespace router {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int RANKS = 8;
constexpr int PER_RANK = kMoeMaxExperts / RANKS;     // experts of one CTA, at most
constexpr int PER_THREAD = kMoeMaxExperts / THREADS; // experts a thread chooses among
// x g carries 2^600, so no product of finite values, down to subnormal ones,
// leaves the range of normal doubles: |x g w| 2^(600 - 896).
constexpr double SCALE = 0x1p600, UNSCALE = 0x1p296;

struct Smem {
  union {
    double part[WARPS][4][PER_RANK];   // [warp][row][expert / RANKS]
    double key[kMoeMaxExperts];        // later: what the choice goes by
  };
  double ssq[WARPS][4];
  double dot[4][PER_RANK];             // [row][expert / RANKS], read by the other ranks
  double chosen[kMoeMaxTopK];          // scores, best first
  double red[WARPS];
  double r;
};
// The gate/up kernel's CTAs start beside this kernel's: at most 20 KB of shared
// memory and 128 registers a thread leave room for them.  (16 experts in flight
// took 171 registers, and 16 rows of 4544, 4 of 5 experts 48 us instead of 37.)
static_assert(sizeof(Smem) <= 20 * 1024, "beside a gate/up CTA");

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

// Largest value or sum over the block, the same in every thread; NaN wins.
template <bool MAX>
__device__ __forceinline__ double block_reduce(Smem& sm, double v) {
  auto op = [](double a, double b) { return MAX ? (a != a ? a : b != b ? b : fmax(a, b)) : a + b; };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.red[threadIdx.x >> 5] = v;
  __syncthreads();
  double r = sm.red[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) r = op(r, sm.red[w]);
  return r;
}

// A bf16 in the upper half of a word, times 2^-896 (finite values).
__device__ __forceinline__ double widen(uint32_t b) {
  return __hiloint2double(static_cast<int>((b & 0x80000000u) | ((b & 0x7FFF0000u) >> 3)), 0);
}

template <int ROWS>
__global__ void __cluster_dims__(RANKS, 1, 1) __launch_bounds__(THREADS, 2) router_kernel(const Params p) {
  constexpr int GROUP = 8 / ROWS < 4 ? 4 : 8 / ROWS;      // experts in flight
  constexpr int NV = ROWS * GROUP;
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

  // experts rank, rank + 8, ...: `mine` of them
  const int mine = p.E > rank ? (p.E - rank + RANKS - 1) / RANKS : 0;
  double ssq[ROWS];
#pragma unroll
  for (int t = 0; t < ROWS; ++t) ssq[t] = 0.0;
  for (int e0 = 0; e0 < mine || e0 == 0; e0 += GROUP) {
    double acc[NV];
    uint32_t top[GROUP];             // largest exponent field met: 0x7F80 means infinity or NaN
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.0;
#pragma unroll
    for (int q = 0; q < GROUP; ++q) top[q] = 0;
    for (int i = static_cast<int>(threadIdx.x); i < nvec; i += THREADS) {
      uint4 wv[GROUP], xv[ROWS];
#pragma unroll
      for (int t = 0; t < ROWS; ++t) xv[t] = __ldcg(xr[t] + i);
#pragma unroll
      for (int q = 0; q < GROUP; ++q) {
        wv[q] = make_uint4(0, 0, 0, 0);
        if (e0 + q < mine)
          wv[q] = __ldg(reinterpret_cast<const uint4*>(p.router + static_cast<int64_t>(rank + RANKS * (e0 + q)) * p.d) + i);
      }
      float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (p.g) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.g) + 2 * i);
        const float4 b = __ldg(reinterpret_cast<const float4*>(p.g) + 2 * i + 1);
        g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double g0 = static_cast<double>(g[2 * j]) * SCALE, g1 = static_cast<double>(g[2 * j + 1]) * SCALE;
        double x0[ROWS], x1[ROWS];
#pragma unroll
        for (int t = 0; t < ROWS; ++t) {
          const uint32_t xw = j == 0 ? xv[t].x : j == 1 ? xv[t].y : j == 2 ? xv[t].z : xv[t].w;
          const float a = bf16lo_to_f32(xw), b = bf16hi_to_f32(xw);
          x0[t] = static_cast<double>(a) * g0;
          x1[t] = static_cast<double>(b) * g1;
          // squared in 64 bits: in 32 a square leaves the range from 1.8e19 and below 1e-19
          if (e0 == 0) {
            const double a64 = a, b64 = b;
            ssq[t] = fma(a64, a64, fma(b64, b64, ssq[t]));
          }
        }
#pragma unroll
        for (int q = 0; q < GROUP; ++q) {
          const uint32_t w = j == 0 ? wv[q].x : j == 1 ? wv[q].y : j == 2 ? wv[q].z : wv[q].w;
          top[q] = max(top[q], max(w & 0x7F80u, (w >> 16) & 0x7F80u));
          const double w0 = widen(w << 16), w1 = widen(w);
#pragma unroll
          for (int t = 0; t < ROWS; ++t) acc[t * GROUP + q] = fma(x1[t], w1, fma(x0[t], w0, acc[t * GROUP + q]));
        }
      }
    }
#pragma unroll
    for (int q = 0; q < GROUP; ++q)
      if (top[q] == 0x7F80u)
#pragma unroll
        for (int t = 0; t < ROWS; ++t) acc[t * GROUP + q] = NAN;
    // Sums over the warp: halve the values a lane holds with every exchange,
    // then add over the lanes that hold the same one.
    int o = 16, which = 0;
#pragma unroll
    for (int n = NV; n > 1; n >>= 1) {
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const double give = upper ? acc[i] : acc[i + n / 2];
        const double keep = upper ? acc[i + n / 2] : acc[i];
        acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
      which = which * 2 + (upper ? 1 : 0);
      o >>= 1;
    }
#pragma unroll
    for (int h = 16 / NV; h > 0; h >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], h);
    if ((lane & (32 / NV - 1)) == 0 && e0 + which % GROUP < mine) sm.part[warp][which / GROUP][e0 + which % GROUP] = acc[0];
  }
#pragma unroll
  for (int t = 0; t < ROWS; ++t) {
    const double s = warp_sum(ssq[t]);
    if (lane == 0) sm.ssq[warp][t] = s;
  }
  __syncthreads();
  for (int i = static_cast<int>(threadIdx.x); i < ROWS * mine; i += THREADS) {
    const int t = i / mine, e = i - t * mine;
    double s = sm.part[0][t][e];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) s += sm.part[w][t][e];
    sm.dot[t][e] = s * UNSCALE;
  }
  cluster_sync_all();                       // every rank's logits are in shared memory

  const int m = m0 + rank;                  // the row this CTA selects for
  const bool selects = rank < ROWS && m < p.M;
  if (selects) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sm.ssq[w][rank];
    const double r = 1.0 / sqrt(s / p.d + static_cast<double>(p.eps));
    double l[PER_THREAD];
    double top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER_THREAD; ++j) {
      const int e = static_cast<int>(threadIdx.x) + j * THREADS;
      l[j] = -INFINITY;
      if (e < p.E) {
        l[j] = r * __longlong_as_double(static_cast<long long>(
                       dsmem_ld_u64(dsmem_addr(&sm.dot[rank][e / RANKS], e % RANKS))));
        top = l[j] != l[j] || top != top ? NAN : fmax(top, l[j]);
      }
    }
    // softmax: e^(l - top) / sum, the sum over all experts only where a weight or a key needs it
    double sum = 1.0;
    if (!p.sigmoid) {
      top = block_reduce<true>(sm, top);
      if (!p.renorm || p.bias) {
        double v = 0.0;
#pragma unroll
        for (int j = 0; j < PER_THREAD; ++j)
          if (static_cast<int>(threadIdx.x) + j * THREADS < p.E) v += exp(l[j] - top);
        sum = block_reduce<false>(sm, v);
      }
    }
    double score[PER_THREAD];
#pragma unroll
    for (int j = 0; j < PER_THREAD; ++j) {
      const int e = static_cast<int>(threadIdx.x) + j * THREADS;
      if (e < p.E) {
        score[j] = p.sigmoid ? 1.0 / (1.0 + exp(-l[j])) : exp(l[j] - top) / sum;
        double key = p.bias ? score[j] + static_cast<double>(__ldg(p.bias + e)) : l[j];
        sm.key[e] = key != key ? -INFINITY : key;      // NaN ranks with the lowest
      }
    }
    __syncthreads();
    int place[PER_THREAD];
#pragma unroll
    for (int j = 0; j < PER_THREAD; ++j) {
      const int e = static_cast<int>(threadIdx.x) + j * THREADS;
      place[j] = p.E;
      if (e < p.E) {
        const double key = sm.key[e];
        int before = 0;
#pragma unroll 8
        for (int i = 0; i < p.E; ++i) before += (sm.key[i] > key || (sm.key[i] == key && i < e)) ? 1 : 0;
        place[j] = before;
        if (before < p.k) sm.chosen[before] = score[j];
      }
    }
    __syncthreads();
    double norm = 1.0;
    if (p.renorm) {
      norm = 0.0;
      for (int c = 0; c < p.k; ++c) norm += sm.chosen[c];
    }
#pragma unroll
    for (int j = 0; j < PER_THREAD; ++j) {
      const int e = static_cast<int>(threadIdx.x) + j * THREADS;
      if (e < p.E) {
        const bool on = place[j] < p.k;
        const float wf = on ? static_cast<float>(score[j] / norm * static_cast<double>(p.scale)) : 0.f;
        p.weight[static_cast<int64_t>(e) * kMoeMaxRows + m] = wf;
        if (on) {
          p.ids[m * p.k + place[j]] = e;
          if (p.ids_out) p.ids_out[m * p.k + place[j]] = e;
          if (p.w_out) p.w_out[m * p.k + place[j]] = wf;
        }
      }
    }
    if (threadIdx.x == 0) p.rinv[m] = static_cast<float>(r);
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
