// fn_proj for more rows, or many columns: y = act(x W + b) + residual on pairs of
// SMs, sm_100a.
//
// Each 2-CTA cluster computes 256 weight columns x H * NB rows with
// tcgen05.mma.cta_group::2 (swap-AB: the weight columns on the MMA's M side,
// 128 in each CTA, the rows of x on its N side).  N may be any multiple of 32
// up to 256, so a batch is cut into equal row blocks padded by less than 32
// rows each: 300 rows run as 2 x 160, not as 2 x 256.  Both operands are
// staged by TMA with 128-byte swizzle: the CTA's 128 weight columns (16 KB per
// 64-deep k step, N-major) and its half of the rows (NB / 2, K-major).
// Above 256 rows a tile may take two MMAs per K step (H = 2, up to 512 rows in
// one accumulator of 512 columns): a staged weight byte then feeds twice the
// rows, but the epilogue does not overlap the next tile.  make_plan estimates
// both.
// Ragged K and N read zeros past the edge (TMA fill), the epilogue stores
// what exists.
//
// Bound by the tensor cores (under the power cap) at large M and K, by the
// operands' way from L2 into the SMs at a few hundred rows.  Tiles run whole, one after another per pair, in as many
// rounds as fill every pair; the k ranges of the tiles that are left over
// (fewer than pairs) are cut into equal shares over all pairs where that
// saves more than the exchange costs.  Sharing CTAs write fp32 partials to
// the workspace, and a fix-up kernel adds them in ascending k order and
// finishes the tile (no CTA waits for another, no floating-point atomics,
// bit-identical repeats).
//
// Measured (device time a call) at 1965 MHz, and in a long run under the power
// cap: 4096 x 14336 x 4096 with bias and residual 360 us (1335 TFLOP/s), 419 at
// 1305 MHz; 1024 x 8192 x 4096 53 us, 63 at 1537 MHz; 300 x 14336 x 4096 43 us, 50
// at 1650 MHz; 498 x 416 x 277 6 us.
//
// Layout per CTA: 10 warps.
//   warp 0      TMA producer (own weight columns, own rows)
//   warp 1      TMEM owner; in CTA 0 the pair-MMA issuer
//   warps 2-9   epilogue, two warps per TMEM lane quarter, alternating
//               32-row chunks; two accumulator buffers, so a tile's epilogue
//               overlaps the next tile's MMAs
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fn {
namespace ptile {

constexpr int BK = 64;
constexpr int BN = 256;                        // weight columns per pair
constexpr int MAX_NB = 256;                    // rows per MMA
constexpr int W_BOX_BYTES = 64 * BK * 2;       // 64 columns x 64 k rows
constexpr int W_BYTES = 2 * W_BOX_BYTES;       // a CTA's 128 columns
constexpr int NUM_THREADS = 320;
constexpr int EPI_THREADS = 256;
constexpr int MAX_STAGES = 11;
constexpr int RING_BYTES = 6 * 32 * 1024;      // 6 stages at 256 rows
constexpr int SCRATCH_BYTES = 8 * SCRATCH_FLOATS * 4;   // of the epilogue warps
constexpr int TMEM_COLS = 512;

enum : unsigned { kSiteProdEmpty = 1, kSiteMmaAccEmpty, kSiteMmaFull, kSiteEpiAccFull };

struct Params {
  int M, N;
  int nb;                          // rows per MMA
  int rows;                        // rows per tile: H nb
  int num_m, num_n, kblocks;
  int group_m;                     // tile raster: bands of group_m row blocks
  int full;                        // tiles that run whole
  int rest;                        // tiles whose k blocks are shared between pairs
  int sharers;                     // pairs that take a share of them (each at least one k block)
  int share_q, share_r;            // rest * kblocks by sharers: quotient, remainder
  int stages;
  Epilogue epi;
  int vec;                         // the epilogue's vector form applies
  unsigned int* status;            // workspace header: status word
  float* part;                     // [grid][2][rows x 128]
  unsigned long long budget_ns;
  int withhold;
  const uint8_t* w;                // weight base and row bytes (L2 prefetch addresses)
  int64_t w_row_bytes;
  int wrows;
  int prefetch_iters;
};

struct alignas(8) Bars {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;                  // the last pair MMA completed (both CTAs)
  uint64_t exit_bar;               // the partner is done with this CTA's memory
  uint32_t tmem_base;
  int abort_flag;
  int epi_ok[2];
};
constexpr size_t SMEM = 1024 + RING_BYTES + SCRATCH_BYTES + sizeof(Bars);
static_assert(SMEM <= 232448, "shared memory budget");

// First of the shared tiles' k blocks that pair c takes.
// (c rest kblocks / sharers, with rest kblocks = share_q sharers + share_r: 32
// bits, as 64-bit divisions would stand before the first load.)
__device__ __forceinline__ int share_begin(const Params& p, int c) {
  return c * p.share_q + static_cast<int>(static_cast<unsigned>(c * p.share_r) / static_cast<unsigned>(p.sharers));
}

// Segment i of a pair: a whole tile, or its part of the shared tiles.
struct Seg {
  int tile, kb0, kb1;
  bool shared;
};
struct SegIter {
  int npairs, full, kblocks, next_tile;
  int it, end;
  __device__ SegIter(const Params& p, int pair, int npairs_)
      : npairs(npairs_), full(p.full), kblocks(p.kblocks), next_tile(pair), it(0), end(0) {
    if (pair < p.sharers) {
      it = share_begin(p, pair);
      end = share_begin(p, pair + 1);
    }
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (next_tile < full) {
      s.tile = next_tile;
      s.kb0 = 0;
      s.kb1 = kblocks;
      s.shared = false;
      next_tile += npairs;
      return true;
    }
    if (it >= end) return false;
    const int r = it / kblocks;
    s.tile = full + r;
    s.kb0 = it - r * kblocks;
    s.kb1 = min(kblocks, s.kb0 + (end - it));
    s.shared = s.kb0 != 0 || s.kb1 != kblocks;
    it += s.kb1 - s.kb0;
    return true;
  }
};

__device__ __forceinline__ void tile_coords(int t, const Params& p, int& mb, int& nb) {
  const int per_group = p.group_m * p.num_n;
  const int group = t / per_group;
  const int first_m = group * p.group_m;
  const int gm = min(p.num_m - first_m, p.group_m);
  const int r = t - group * per_group;
  mb = first_m + r % gm;
  nb = r / gm;
}

// Bounded wait that polls without suspending (the pair's critical path).
__device__ __forceinline__ bool mbar_wait_spin(uint64_t* bar, uint32_t parity, const WaitCtl& c, unsigned site) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*c.abort_flag) return false;
    if (globaltimer_ns() - t0 > c.budget_ns) {
      raise_timeout(c, site);
      return false;
    }
  }
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long budget) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (globaltimer_ns() - t0 > budget) return;
  }
}

template <bool F32, int H>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    proj_tile_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                     const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + RING_BYTES + SCRATCH_BYTES);
  constexpr int NBUF = H == 1 ? 2 : 1;               // accumulators
  const int x_bytes = p.nb * (BK * 2 / 2);           // this CTA's nb / 2 rows of an MMA
  const int stage_bytes = W_BYTES + H * x_bytes;
  const int stages = p.stages;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();           // 0: MMA issuer of the pair
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.acc_full[b], 1);
      mbar_init(&bars.acc_empty[b], EPI_THREADS + 1);   // CTA 0's epilogue threads + CTA 1's epilogue
    }
    mbar_init(&bars.drain, 1);
    mbar_init(&bars.exit_bar, 1);
    bars.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars.tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  {
    // This overlaps the previous kernel in the stream: an L2 prefetch of the
    // first k blocks cannot return stale data, whoever wrote the weight.  One
    // 128-byte line per thread and step.
    SegIter segs(p, pair, npairs);
    Seg g;
    if (segs.next(g)) {
      int mb, nb;
      tile_coords(g.tile, p, mb, nb);
      const int n_it = min(p.prefetch_iters, g.kb1 - g.kb0);
      for (int i = threadIdx.x; i < n_it * BK * 2; i += NUM_THREADS) {
        const int64_t k = static_cast<int64_t>(g.kb0 + i / (BK * 2)) * BK + (i >> 1) % BK;
        const int64_t col = static_cast<int64_t>(nb) * BN + rank * 128 + (i & 1) * 64;
        if (k < p.wrows && col < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w + k * p.w_row_bytes + col * 2));
      }
    }
  }
  tc_fence_before();
  cluster_sync_all();                                 // both CTAs' barriers are initialised
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem_base = bars.tmem_base;
  WaitCtl ctl{&bars.abort_flag, p.status, p.budget_ns};
  ctl.peer_abort = dsmem_addr(&bars.abort_flag, rank ^ 1u);

  if (warp == 0) {
    // ------------------------------------------------------------ producer (own halves)
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0, last_ph = 0;
      bool ok = true;
      const uint32_t full0 = dsmem_addr(&bars.full[0], 0);   // CTA 0's barriers count both CTAs' bytes
      SegIter segs(p, pair, npairs);
      Seg g;
      while (ok && segs.next(g)) {
        int mb, nb;
        tile_coords(g.tile, p, mb, nb);
        const int row0 = mb * p.rows + static_cast<int>(rank) * (p.nb / 2);
        const int col0 = nb * BN + static_cast<int>(rank) * 128;
        for (int kb = g.kb0; kb < g.kb1; ++kb) {
          if (!mbar_wait_spin(&bars.empty[s], ph ^ 1, ctl, kSiteProdEmpty)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], 2 * stage_bytes);
          const uint32_t fb = full0 + s * 8;
          uint8_t* st = smem + s * stage_bytes;
          tma_load_2d_pair(st, &tmap_w, fb, col0, kb * BK);
          tma_load_2d_pair(st + W_BOX_BYTES, &tmap_w, fb, col0 + 64, kb * BK);
#pragma unroll
          for (int h = 0; h < H; ++h)
            tma_load_2d_pair(st + W_BYTES + h * x_bytes, &tmap_x, fb, kb * BK, row0 + h * p.nb);
          issued |= 1u << s;
          last_ph = (last_ph & ~(1u << s)) | (ph << s);
          if (++s == stages) { s = 0; ph ^= 1; }
        }
      }
      // No copy may still be landing in shared memory when a CTA exits.  CTA
      // 0's stage barriers count both CTAs' copies, and CTA 1 leaves after
      // CTA 0 (exit_bar below).  After an abort the partner may not have
      // announced a stage's bytes, so the barriers cannot tell: leave the
      // copies a millisecond.
      if (ok) {
        if (rank == 0)
          for (int i = 0; i < stages; ++i)
            if (issued & (1u << i)) drain_wait(&bars.full[i], (last_ph >> i) & 1u, p.budget_ns);
      } else {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      if (rank == 0) {
        // -------------------------------------------------------- pair-MMA issuer
        const uint32_t idesc = idesc_bf16_f32(2 * 128, p.nb, /*a MN-major*/ true, /*b MN-major*/ false);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        int i = 0;
        SegIter segs(p, pair, npairs);
        Seg g;
        for (; ok && segs.next(g); ++i) {
          const int b = NBUF == 2 ? i & 1 : 0;
          const uint32_t aph = NBUF == 2 ? (i >> 1) & 1 : i & 1;
          if (!mbar_wait_spin(&bars.acc_empty[b], aph ^ 1, ctl, kSiteMmaAccEmpty)) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + b * MAX_NB;
          for (int kb = g.kb0; kb < g.kb1; ++kb) {
            if (!mbar_wait_spin(&bars.full[s], ph, ctl, kSiteMmaFull)) { ok = false; break; }
            tc_fence_after();
            const uint32_t w0 = smem_u32(smem + s * stage_bytes);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              // A: 128 weight columns of each CTA, N-major; B: nb / 2 rows of x of each CTA, K-major
              const uint64_t adesc = sdesc_sw128(w0 + kk * 2048, W_BOX_BYTES, 1024);
#pragma unroll
              for (int h = 0; h < H; ++h) {
                const uint64_t bdesc = sdesc_sw128(w0 + W_BYTES + h * x_bytes + kk * 32, 16, 1024);
                umma_bf16_pair(d_tmem + h * p.nb, adesc, bdesc, idesc, (kb != g.kb0 || kk != 0) ? 1u : 0u);
              }
            }
            umma_commit_pair(&bars.empty[s], 0x3);
            if (++s == stages) { s = 0; ph ^= 1; }
          }
          if (!ok) break;
          if (!(p.withhold && i == 0)) umma_commit_pair(&bars.acc_full[b], 0x3);
        }
        umma_commit_pair(&bars.drain, 0x3);
        drain_wait(&bars.drain, 0, p.budget_ns);
      } else {
        drain_wait(&bars.drain, 0, p.budget_ns);   // the pair's last MMA no longer reads this CTA
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (own columns)
    const int q = warp & 3;                        // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;              // which of the quarter's two warps
    const int et = threadIdx.x - 64;               // 0..255
    const uint32_t acc_empty0 = dsmem_addr(&bars.acc_empty[0], 0);
    const int chunks = p.rows / 32;
    int i = 0;
    SegIter segs(p, pair, npairs);
    Seg g;
    for (; segs.next(g); ++i) {
      int mb, nb;
      tile_coords(g.tile, p, mb, nb);
      const int b = NBUF == 2 ? i & 1 : 0;
      const uint32_t aph = NBUF == 2 ? (i >> 1) & 1 : i & 1;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * MAX_NB;
      const int n = q * 32 + lane;                 // column within this CTA's 128
      const int64_t col0 = static_cast<int64_t>(nb) * BN + rank * 128 + q * 32;   // of this warp's 32 columns
      float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.epi.bias) {
        const int64_t last = p.N - 1, c = col0 + lane % 8 * 4;
        bias = make_float4(__ldg(p.epi.bias + min(c, last)), __ldg(p.epi.bias + min(c + 1, last)),
                           __ldg(p.epi.bias + min(c + 2, last)), __ldg(p.epi.bias + min(c + 3, last)));
      }
      const int row0 = mb * p.rows;
      // this warp's chunks of 16 rows: half, half + 2, ...; their residual DEPTH ahead
      constexpr int DEPTH = F32 ? 2 : 3;
      const bool ahead = !g.shared && p.vec && p.epi.residual;
      typename Quad<F32>::Raw raw[DEPTH][4];
      if (ahead)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
          epi_fetch<F32>(p.epi, lane, row0 + 16 * (half + 2 * d), min(p.M - row0 - 16 * (half + 2 * d), 16), col0, p.N, raw[d]);
      // One thread waits and the whole epilogue follows its decision, so the
      // group never splits at the named barriers or the .sync.aligned loads.
      if (et == 0) bars.epi_ok[i & 1] = mbar_wait_spin(&bars.acc_full[b], aph, ctl, kSiteEpiAccFull) ? 1 : 0;
      named_bar_sync(1, EPI_THREADS);
      if (!bars.epi_ok[i & 1]) break;
      tc_fence_after();
      auto release = [&]() {
        // this CTA's epilogue has read TMEM buffer b
        tc_fence_before();
        if (rank == 0) {
          mbar_arrive(&bars.acc_empty[b]);
        } else {
          named_bar_sync(1, EPI_THREADS);
          if (et == 0) mbar_arrive_remote(acc_empty0 + b * 8);
        }
      };
      if (!g.shared) {
        float* scratch = reinterpret_cast<float*>(smem + RING_BYTES) + (warp - 2) * SCRATCH_FLOATS;
        // One copy of the code for every chunk: unrolled by four it took 6 us per
        // tile of 256 rows to fetch and run.
        if (p.vec) {
#pragma unroll 1
          for (int c = half; c < 2 * chunks; c += 2) {
            const int r0 = row0 + 16 * c, rn = r0 + 32 * DEPTH;
            if (r0 >= p.M) break;
            uint32_t v[16];
            float z[16];
            tmem_ld16(taddr + c * 16, v);
            tmem_ld_wait();
            epi_transpose_act(p.epi, scratch, lane, bias, v, z);
            epi_store_vec<F32>(p.epi, raw[0], lane, r0, min(p.M - r0, 16), col0, p.N, z);
#pragma unroll
            for (int d = 0; d + 1 < DEPTH; ++d)
#pragma unroll
              for (int g = 0; g < 4; ++g) raw[d][g] = raw[d + 1][g];
            if (ahead && c + 2 * DEPTH < 2 * chunks)
              epi_fetch<F32>(p.epi, lane, rn, min(p.M - rn, 16), col0, p.N, raw[DEPTH - 1]);
          }
        } else {
#pragma unroll 1
          for (int c = half; c < 2 * chunks; c += 2) {
            const int r0 = row0 + 16 * c;
            if (r0 >= p.M) break;
            float v[16];
            dec::tmem_ld_cols<16>(taddr + c * 16, v);
            if (col0 + lane < p.N) epi_finish<16>(p.epi, r0, min(p.M - r0, 16), col0 + lane, v);
          }
        }
        release();
        continue;
      }
      // Shared tile: publish the partial (float4 groups [row / 4][column]); the
      // fix-up kernel adds them and finishes.
      const int t0 = (g.tile - p.full) * p.kblocks;
      const int slot = static_cast<int>(blockIdx.x) * 2 + (share_begin(p, pair) >= t0 ? 0 : 1);
      float4* mine = reinterpret_cast<float4*>(p.part + static_cast<int64_t>(slot) * (p.rows * 128));
#pragma unroll 1
      for (int c = half; c < chunks; c += 2) {
        float v[32];
        dec::tmem_ld_cols<32>(taddr + c * 32, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row0 + 32 * c + 4 * j < p.M)
            __stcg(mine + (c * 8 + j) * 128 + n, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
      release();
    }
  }

  // Teardown: every role of this CTA is done; wait (bounded) until the partner
  // is done with this CTA's memory too, then release TMEM in both CTAs.
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_arrive_remote(dsmem_addr(&bars.exit_bar, rank ^ 1u));
    drain_wait(&bars.exit_bar, 0, p.budget_ns);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// How a call is cut into tiles and shares.
struct Plan {
  int h, nb, num_m, num_n, kblocks, pairs, full, rest, sharers;
  double us;                       // estimate
  int rows() const { return h * nb; }
};

// One way to cut: tiles of h MMAs of at most most_rows rows; the tiles of the last, partial round whole
// (per_tile 0), shared evenly by per_tile pairs each, or by all pairs (-1).
//
// The estimate, from measurements of this kernel: a k step is bound by the
// tensor cores, 0.30 us per 256 rows while few pairs work and 0.44 when all 74
// do (power), or by the operand bytes that L2 delivers to all SMs (11.1 MB per
// us: 160 rows take 0.36 instead of 0.27 us, the reason for two MMAs per step);
// the last epilogue, and every one of the wide form, takes 4 us per 256 rows;
// sharing costs a second kernel (6 us) and the partials' way through L2
// (3.5 MB per us).  Estimate and measurement (us): 300 x 14336 x 4096 wide 46 : 46,
// narrow 48 : 50; 1024 x 8192 x 4096 whole 56 : 59, shared 69 : 75;
// 4096 x 4096 x 4096 whole 110 : 121, wide 125 : 138.
Plan make_plan(int h, int most_rows, int per_tile, int64_t M, int64_t K, int64_t N, int num_sms) {
  Plan q;
  q.h = h;
  const int64_t blocks = (M + h * most_rows - 1) / (h * most_rows);
  q.num_m = static_cast<int>(blocks);
  q.nb = static_cast<int>(((M + h * blocks - 1) / (h * blocks) + 31) / 32 * 32);
  q.num_n = static_cast<int>((N + BN - 1) / BN);
  q.kblocks = static_cast<int>((K + BK - 1) / BK);
  const int64_t tiles = static_cast<int64_t>(q.num_m) * q.num_n;
  const int64_t pairs = num_sms / 2;
  const int64_t rest = per_tile ? tiles % pairs : 0;
  // at most 8 pairs to a tile, at least 4 k blocks to a share
  int64_t sharers = per_tile > 0 ? rest * per_tile : pairs < rest * 8 ? pairs : rest * 8;
  if (sharers > rest * q.kblocks / 4) sharers = rest * q.kblocks / 4;
  if (sharers > pairs || sharers <= rest) sharers = 0;
  q.full = static_cast<int>(sharers ? tiles - rest : tiles);
  q.rest = static_cast<int>(sharers ? rest : 0);
  q.sharers = static_cast<int>(sharers);
  q.pairs = static_cast<int>(tiles >= pairs ? pairs : sharers ? sharers : tiles);
  const double rows = q.rows();
  auto step = [&](double active) {       // us per k step while so many pairs work
    const double load = active / 74.0;
    return std::max(rows / 256 * (0.30 + 0.137 * load * load), (W_BYTES + rows * BK) * 2 * active / 11.1e6);
  };
  const double epilogue = rows * 4.0 / 256;
  const int64_t rounds = q.full / pairs, last = q.full % pairs;
  q.us = q.kblocks * (rounds * step(static_cast<double>(pairs)) + (last ? step(static_cast<double>(last)) : 0));
  q.us += epilogue * (h == 2 ? static_cast<double>(rounds + (last ? 1 : 0)) : q.full > 0 ? 1 : 0);
  if (sharers)
    q.us += static_cast<double>(rest) * q.kblocks / sharers * step(static_cast<double>(sharers)) + epilogue + 6 +
            static_cast<double>(sharers % rest ? sharers + rest : sharers) * rows * BN * 4 / 3.5e6;
  return q;
}

Plan best_plan(int64_t M, int64_t K, int64_t N, int num_sms) {
  Plan best = make_plan(1, MAX_NB, 0, M, K, N, num_sms);
  auto consider = [&](const Plan& q) {
    if (q.us < best.us) best = q;
  };
  for (int h = 1; h <= (M > MAX_NB ? 2 : 1); ++h)
    for (int per_tile = -1; per_tile <= 8; ++per_tile) consider(make_plan(h, MAX_NB, per_tile, M, K, N, num_sms));
  // fewer rows to a tile, while that makes work for idle pairs (with a short K
  // the epilogue is most of a tile)
  for (int rows = MAX_NB / 2; rows >= 32 && best.num_m * best.num_n < num_sms / 2; rows /= 2)
    consider(make_plan(1, rows, 0, M, K, N, num_sms));
  return best;
}

template <bool F32, int H>
cudaError_t launch_kernel(const Params& p, const Plan& q, cudaStream_t stream, const CUtensorMap& tx,
                          const CUtensorMap& tw) {
  const cudaError_t e = ensure_smem_limit<proj_tile_kernel<F32, H>>(static_cast<int>(SMEM));
  if (e != cudaSuccess) return e;
  return launch_pdl(proj_tile_kernel<F32, H>, static_cast<unsigned>(2 * q.pairs), NUM_THREADS, SMEM, stream, tx, tw, p);
}

}  // namespace ptile

size_t proj_tile_workspace_bytes(int64_t M, int64_t K, int64_t N, int num_sms) {
  const ptile::Plan q = ptile::best_plan(M, K, N, num_sms);
  if (q.rest == 0) return kWsHeaderBytes;
  return kWsHeaderBytes + static_cast<size_t>(q.pairs) * 2 * 2 * q.rows() * 128 * 4;
}

int64_t proj_tile_count(int64_t M, int64_t N) {
  return ((M + ptile::MAX_NB - 1) / ptile::MAX_NB) * ((N + ptile::BN - 1) / ptile::BN);
}

cudaError_t launch_proj_tile(const ProjArgs& a) {
  using namespace ptile;
  const Plan q = best_plan(a.M, a.K, a.N, a.num_sms);
  CUtensorMap tx, tw;
  if (!make_tmap_2d_ld(&tx, a.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.M, a.K, a.ldx, q.nb / 2, BK))
    return cudaErrorInvalidValue;
  if (!make_tmap_2d_ld(&tw, a.W, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.K, a.N, a.ldw, BK, 64))
    return cudaErrorInvalidValue;
  Params p = {};
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.nb = q.nb;
  p.rows = q.rows();
  p.num_m = q.num_m;
  p.num_n = q.num_n;
  p.kblocks = q.kblocks;
  // Raster band: as many row blocks as keep the band's x within about 40 MB
  // of L2 (at most 16), so the weight is fetched once per band.
  const int64_t band_rows = (40ll << 20) / (a.K * 2);
  const int64_t most = 16 * MAX_NB / p.rows;
  p.group_m = static_cast<int>(std::max<int64_t>(1, std::min(band_rows / p.rows, most)));
  p.full = q.full;
  p.rest = q.rest;
  p.sharers = q.sharers;
  if (q.sharers) {
    p.share_q = q.rest * q.kblocks / q.sharers;
    p.share_r = q.rest * q.kblocks % q.sharers;
  }
  const int stage_bytes = W_BYTES + p.rows * BK;
  p.stages = RING_BYTES / stage_bytes;
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  p.epi = a.epi;
  p.vec = epi_vector_ok(a.epi, a.N);
  p.w = static_cast<const uint8_t*>(a.W);
  p.w_row_bytes = a.ldw * 2;
  p.wrows = static_cast<int>(a.K);
  p.prefetch_iters = a.prefetch_iters;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.part = reinterpret_cast<float*>(ws + kWsHeaderBytes);
  p.budget_ns = a.budget_ns;
  p.withhold = a.withhold;
  const cudaError_t l = q.h == 2 ? (a.epi.out_fp32 ? launch_kernel<true, 2>(p, q, a.stream, tx, tw)
                                                   : launch_kernel<false, 2>(p, q, a.stream, tx, tw))
                                 : (a.epi.out_fp32 ? launch_kernel<true, 1>(p, q, a.stream, tx, tw)
                                                   : launch_kernel<false, 1>(p, q, a.stream, tx, tw));
  if (l != cudaSuccess || q.rest == 0) return l;
  FixupArgs f = {};
  f.part = p.part;
  f.slot_floats = p.rows * 128;
  f.total = static_cast<int64_t>(q.rest) * q.kblocks;
  f.kblocks = q.kblocks;
  f.sharers = q.sharers;
  f.ranks = 2;
  f.tile0 = q.full;
  f.tiles = q.rest;
  f.group_m = p.group_m;
  f.num_m = q.num_m;
  f.num_n = q.num_n;
  f.rows = p.rows;
  f.M = a.M;
  f.N = a.N;
  f.epi = a.epi;
  f.stream = a.stream;
  return launch_proj_fixup(f);
}

}  // namespace fn
