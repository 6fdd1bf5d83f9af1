// Fix-up of fn_proj and of fn_moe_swiglu's down projection: adds the fp32
// partials of the tiles whose k range several CTAs shared, in ascending k order,
// and runs the epilogue, sm_100a.
//
// One thread per (tile, 8 rows, column): all SMs take part, so its cost is a
// launch and one round through L2 (about 4 us).  The CTA that happens to be
// last doing it alone took 10 to 30 us above 16 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fn {
namespace fix {

constexpr int THREADS = 256;     // 128 columns x 2 groups of 8 rows
constexpr int IN_FLIGHT = 4;     // contributors' loads in flight

__device__ __forceinline__ long long div64(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__global__ void __launch_bounds__(THREADS) proj_fixup_kernel(const FixupArgs p) {
  const int groups = (p.rows + 15) / 16;               // blocks of 16 rows to a tile and rank
  int b = static_cast<int>(blockIdx.x);
  const int g = (b % groups) * 4 + static_cast<int>(threadIdx.x >> 7) * 2;   // first of two groups of 4 rows
  b /= groups;
  const int rank = b % p.ranks;
  const int t = b / p.ranks;                           // tile, from tile0 on
  const int n = static_cast<int>(threadIdx.x & 127);
  int kblocks = p.kblocks, sharers = p.sharers;
  long long total = p.total;
  if (p.routed) {
    // The experts are counted as the down kernel counted them; the router's ids
    // were complete before that kernel could launch.
    __shared__ uint32_t chosen[kMoeMaxExperts / 32];
    for (int i = threadIdx.x; i < kMoeMaxExperts / 32; i += THREADS) chosen[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.routed; i += THREADS) {
      const int e = __ldcg(p.route.ids + i);
      atomicOr(&chosen[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    int n = 0;
    for (int i = 0; i < kMoeMaxExperts / 32; ++i) n += __popc(chosen[i]);
    kblocks *= n;
    total = static_cast<long long>(p.tiles) * kblocks;
    sharers = static_cast<int>(share_count(p.tiles, kblocks, static_cast<unsigned>(p.sharers)));
  }
  const long long t0 = static_cast<long long>(t) * kblocks;
  const int first = static_cast<int>(div64((t0 + 1) * sharers - 1, total));
  const int last = static_cast<int>(div64((t0 + kblocks) * sharers - 1, total));
  const int tile = p.tile0 + t;
  const int per_group = p.group_m * p.num_n;
  const int first_m = tile / per_group * p.group_m;
  const int gm = min(p.num_m - first_m, p.group_m);
  const int r = tile % per_group;
  const int64_t col = (static_cast<int64_t>(r / gm) * p.ranks + rank) * 128 + n;
  const int64_t row = static_cast<int64_t>(first_m + r % gm) * p.rows + 4 * g;
  const int rows = static_cast<int>(min(p.M - row, static_cast<int64_t>(min(p.rows - 4 * g, 8))));
  grid_dependency_wait();
  grid_launch_dependents();
  if (first == last || rows <= 0 || col >= p.N) return;   // whole tiles are finished already
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int second = rows > 4 ? 128 : 0;               // only what the tile holds is read
  for (int c0 = first; c0 <= last; c0 += IN_FLIGHT) {
    float4 q[IN_FLIGHT][2];
#pragma unroll
    for (int j = 0; j < IN_FLIGHT; ++j) {
      const int c = min(c0 + j, last);
      const int64_t slot = (static_cast<int64_t>(c) * p.ranks + rank) * 2 + (div64(c * total, sharers) >= t0 ? 0 : 1);
      const float4* src = reinterpret_cast<const float4*>(p.part + slot * p.slot_floats) + g * 128 + n;
      q[j][0] = __ldcg(src);
      q[j][1] = __ldcg(src + second);
    }
#pragma unroll
    for (int j = 0; j < IN_FLIGHT; ++j) {
      if (c0 + j <= last) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[4 * h] += q[j][h].x;
          v[4 * h + 1] += q[j][h].y;
          v[4 * h + 2] += q[j][h].z;
          v[4 * h + 3] += q[j][h].w;
        }
      }
    }
  }
  epi_finish<8>(p.epi, row, rows, col, v);
}

}  // namespace fix

cudaError_t launch_proj_fixup(const FixupArgs& a) {
  const unsigned grid = static_cast<unsigned>(a.tiles) * a.ranks * ((a.rows + 15) / 16);
  return launch_pdl(fix::proj_fixup_kernel, grid, fix::THREADS, 0, a.stream, a);
}

}  // namespace fn
