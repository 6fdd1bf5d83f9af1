// Projections of few rows (at most 128) whose cost is the weight stream, sm_100a:
//   kProj  y = act(x W + b) + residual (fn_proj)
//   kUp    the chosen experts' SwiGLU, act = w silu(r x G') (r x U') (fn_moe_swiglu)
//   kDown  y = residual + sum over the chosen experts of act D  (fn_moe_swiglu)
//
// Swap-AB as in the norm-fused decode kernel: D[n, m] += W^T[n, k] x^T[k, m],
// 128 weight columns on the MMA's M side, the rows padded to 16, 32, 64 or 128 on
// its N side (tcgen05.mma kind::f16, fp32 accumulators in TMEM), both operands
// staged by TMA with 128-byte swizzle.  Bound by HBM: every weight byte is
// read once, the MMAs hide under the stream.
//
// All three run on one (column tile, 64-deep k block) iteration space that is
// cut into equal contiguous shares, one per SM.  For the experts the space is
// only known on the device (how many experts were chosen), so each CTA derives
// it from the router's list:
//   kUp    tile -> (expert slot, 128 intermediate columns); k runs over d
//   kDown  k block -> (expert slot, 64 intermediate values): the sum over
//          experts is one long contraction accumulated in TMEM
// Every row goes through every chosen expert's MMA: the weights are the cost,
// the flops are not (64 rows x all weights is under a tenth of the tensor
// rate at the HBM rate).  kUp stores zeros for the rows that did not choose an
// expert, scaled by the routing weight for those that did, so kDown needs no
// masks.  Their one rounding to bf16, behind the routing weight, makes them the
// next MMA's operand.
//
// Measured (device time a call): 4096 x 4096, one row, 10.8 us, of which the
// stream takes 4.7 (7.1 TB/s), the first load 0.8, the exchange 3 and the
// kernel boundary 1.2; 8 experts of 2048 x 1024 and one row 35 us with the
// router's 5.9; 64 rows and 8 experts of 4096 x 14336 460 us (6.1 TB/s) at 1965
// MHz, 487 in a long run under the power cap at 1500 MHz.
//
// A tile whose k range falls to one CTA is finished by it.  The CTAs that
// share a tile write fp32 partials to the workspace.  With few rows, and for
// the experts, they count themselves, and the one that counts last adds all
// partials in ascending k order (a fixed order, so repeats are bit-identical)
// and finishes; above 16 rows a fix-up kernel does (kUp: where few experts' tiles
// are all shared).  No CTA waits for another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fn {
namespace strm {

constexpr int BK = 64;
constexpr int NUM_THREADS = 192;           // producer, MMA issuer, 4 epilogue warps
constexpr int W_BOX_BYTES = 64 * BK * 2;   // 64 columns x 64 k rows
constexpr int RC = 8;                      // rows of an epilogue chunk
constexpr int FIXUP_ROWS = 16;             // shared tiles of more rows are left to a fix-up kernel

// kProjRows: kProj where CTAs finish whole tiles of more than RC rows.
enum Mode : int { kProj = 0, kUp = 1, kDown = 2, kProjRows = 3 };
template <int MODE>
constexpr bool is_proj = MODE == kProj || MODE == kProjRows;
enum : unsigned { kSiteProdEmpty = 1, kSiteMmaAccEmpty, kSiteMmaFull, kSiteEpiAccFull };

struct Params {
  int M, ncols;                  // rows; output columns (kProj: N, kUp: I, kDown: d)
  int tiles, kblocks;            // kProj: the whole space; kUp: tiles per expert, k blocks of d;
                                 // kDown: tiles of d, k blocks per expert
  int wrows;                     // weight rows per expert (kUp: d, kDown: I)
  unsigned int* status;          // workspace header: status word and counters
  float* part;                   // [grid][2][slot floats]
  unsigned long long budget_ns;
  int withhold;
  const uint8_t* w;              // weight base and row bytes (L2 prefetch addresses, kProj)
  int64_t w_row_bytes;
  int prefetch_iters;
  int fixup;                     // shared tiles are left to a fix-up kernel
  Epilogue epi;                  // kProj, kDown
  int vec;                       // kProj: the epilogue's vector form applies
  MoeRoute route;                // kUp, kDown
  __nv_bfloat16* act;            // kUp writes [slot][MPAD][I]
};

template <int MPAD, int HALVES, int MODE>
struct Cfg {
  // The expert kernels up to 32 rows leave room for a second CTA on the SM: the
  // next kernel's, which starts on its weights while this one drains.
  static constexpr int SMEM_BUDGET = (is_proj<MODE> || MPAD > 32 ? 200 : MODE == kUp ? 104 : 112) * 1024;
  static constexpr int W_BYTES = HALVES * 2 * W_BOX_BYTES;
  static constexpr int X_BYTES = MPAD * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int STAGES_RAW = SMEM_BUDGET / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 10 ? 10 : STAGES_RAW;
  static constexpr int ACC_COLS = HALVES * MPAD;
  static constexpr int TMEM_COLS = 2 * ACC_COLS;                    // two buffers: 32..256
  static constexpr int SLOT_FLOATS = HALVES * MPAD * 128;
};

template <int STAGES, bool SWAP, bool ROWS>
struct alignas(16) Bars {
  float scratch[ROWS ? 4 : 1][ROWS ? SCRATCH_FLOATS : 4];   // kProjRows: of the epilogue warps
  uint64_t full[STAGES], empty[STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  float swap[SWAP ? 2 : 1][2][SWAP ? RC / 2 * 64 : 1];   // kUp: rows passed between the gate and the up threads
  float weight[2][kMoeMaxRows], rinv[kMoeMaxRows];   // kUp: of the segment's expert; of the rows
  int epi_ok[2];
  int last;                        // the count of the tile's contributors is complete
  int n_active;
  uint32_t active[kMoeMaxExperts / 32];
  int experts[kMoeMaxExperts];     // chosen experts in ascending order
};

template <int MPAD, int HALVES, int MODE>
constexpr size_t smem_bytes() {
  using C = Cfg<MPAD, HALVES, MODE>;
  return 1024 + C::STAGES * C::STAGE_BYTES + sizeof(Bars<C::STAGES, MODE == kUp && HALVES == 1, MODE == kProjRows>);
}
static_assert(smem_bytes<16, 1, kProjRows>() <= 232448 && smem_bytes<32, 1, kProjRows>() <= 232448 &&
                  smem_bytes<64, 1, kProjRows>() <= 232448 && smem_bytes<128, 1, kProjRows>() <= 232448 &&
                  smem_bytes<64, 2, kUp>() <= 232448,
              "shared memory budget");
static_assert(smem_bytes<64, 2, kUp>() + 20 * 1024 + 2048 <= 233472, "the router's CTA beside gate/up's");
static_assert(smem_bytes<32, 2, kUp>() + smem_bytes<32, 1, kDown>() + 2048 <= 233472 &&
                  smem_bytes<16, 2, kUp>() + smem_bytes<16, 1, kDown>() + 2048 <= 233472 &&
                  smem_bytes<16, 1, kUp>() + smem_bytes<16, 1, kDown>() + 2048 <= 233472,
              "two CTAs to an SM");

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long budget) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > budget) return;
  }
}

// kProj: all rows of this warp's 32 columns, from its TMEM lanes.
template <bool F32>
__device__ __forceinline__ void finish_rows(const Params& p, uint32_t taddr, float* scratch, int lane, int64_t col0) {
  if (!p.vec) {
#pragma unroll 1
    for (int m0 = 0; m0 < p.M; m0 += 16) {
      float v[16];
      dec::tmem_ld_cols<16>(taddr + m0, v);
      if (col0 + lane < p.ncols) epi_finish<16>(p.epi, m0, min(p.M - m0, 16), col0 + lane, v);
    }
    return;
  }
  float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.epi.bias) {
    const int64_t last = p.ncols - 1, c = col0 + lane % 8 * 4;
    bias = make_float4(__ldg(p.epi.bias + min(c, last)), __ldg(p.epi.bias + min(c + 1, last)),
                       __ldg(p.epi.bias + min(c + 2, last)), __ldg(p.epi.bias + min(c + 3, last)));
  }
  typename Quad<F32>::Raw raw[2][4];
  if (p.epi.residual) epi_fetch<F32>(p.epi, lane, 0, min(p.M, 16), col0, p.ncols, raw[0]);
#pragma unroll 1
  for (int m0 = 0; m0 < p.M; m0 += 16) {
    uint32_t v[16];
    float z[16];
    tmem_ld16(taddr + m0, v);
    if (p.epi.residual) epi_fetch<F32>(p.epi, lane, m0 + 16, min(p.M - m0 - 16, 16), col0, p.ncols, raw[1]);
    tmem_ld_wait();
    epi_transpose_act(p.epi, scratch, lane, bias, v, z);
    epi_store_vec<F32>(p.epi, raw[0], lane, m0, min(p.M - m0, 16), col0, p.ncols, z);
#pragma unroll
    for (int g = 0; g < 4; ++g) raw[0][g] = raw[1][g];
  }
}

template <int MPAD, int HALVES, int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                  const Params p) {
  using C = Cfg<MPAD, HALVES, MODE>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using Shared = Bars<STAGES, MODE == kUp && HALVES == 1, MODE == kProjRows>;
  Shared& bars = *reinterpret_cast<Shared*>(smem + STAGES * C::STAGE_BYTES);
  auto stage_w = [&](int s) { return smem + s * C::STAGE_BYTES; };
  auto stage_x = [&](int s) { return smem + s * C::STAGE_BYTES + C::W_BYTES; };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const unsigned cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.acc_full[b], 1);
      mbar_init(&bars.acc_empty[b], 128);
    }
    mbar_init(&bars.drain, 1);
    bars.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (!is_proj<MODE>)
    for (int i = threadIdx.x; i < kMoeMaxExperts / 32; i += NUM_THREADS) bars.active[i] = 0;

  // The iteration space: tiles x kblocks, cut into one contiguous share per CTA.
  int tiles = p.tiles, kblocks = p.kblocks;
  unsigned total, grid, it0, it1;
  auto cut = [&]() {
    total = static_cast<unsigned>(tiles) * kblocks;
    grid = share_count(tiles, kblocks, gridDim.x);
    it0 = cta < grid ? cta * total / grid : 0;
    it1 = cta < grid ? (cta + 1) * total / grid : 0;
  };
  if (is_proj<MODE>) {
    cut();
    // This overlaps the previous kernel in the stream: an L2 prefetch of the
    // share's first k blocks cannot return stale data, whoever wrote the
    // weight.  One 128-byte line per thread and step.
    const int n_it = static_cast<int>(min(static_cast<unsigned>(p.prefetch_iters), it1 - it0));
    for (int i = threadIdx.x; i < n_it * BK * 2; i += NUM_THREADS) {
      const unsigned it = it0 + i / (BK * 2);
      const unsigned tile = it / kblocks;
      const int64_t k = static_cast<int64_t>(it - tile * kblocks) * BK + (i >> 1) % BK;
      const int64_t col = static_cast<int64_t>(tile) * 128 + (i & 1) * 64;
      if (k < p.wrows && col < p.ncols)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w + k * p.w_row_bytes + col * 2));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The router has completed before kUp allows kDown to launch (kUp waits for
  // it first), so kDown may read the experts' list and the weights, which no
  // kernel of this call writes, while kUp still runs; its other operand and
  // the workspace only behind the wait.
  if (MODE != kDown) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  if (!is_proj<MODE>) {
    // the chosen experts in ascending order, from the router's ids
    for (int i = threadIdx.x; i < p.M * p.route.k; i += NUM_THREADS) {
      const int e = __ldcg(p.route.ids + i);
      atomicOr(&bars.active[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.route.E; e += NUM_THREADS) {
      int slot = 0;
      for (int w = 0; w < (e >> 5); ++w) slot += __popc(bars.active[w]);
      slot += __popc(bars.active[e >> 5] & ((1u << (e & 31)) - 1u));
      const bool on = (bars.active[e >> 5] >> (e & 31)) & 1u;
      if (on) bars.experts[slot] = e;
      if (e == p.route.E - 1) bars.n_active = slot + (on ? 1 : 0);
    }
    __syncthreads();
    const int n = bars.n_active;
    if (MODE == kUp) tiles *= n;
    else kblocks *= n;
    cut();
  }
  // the CTA whose share holds iteration `it`
  auto owner_of = [&](unsigned it) { return ((it + 1) * grid - 1) / total; };
  // a share: its first tile and k block, then whole tiles
  const int first_tile = static_cast<int>(it0 / kblocks);
  const int first_kb = static_cast<int>(it0) - first_tile * kblocks;
  const int share = static_cast<int>(it1 - it0);

  const uint32_t tmem_base = bars.tmem_base;
  const WaitCtl ctl{&bars.abort_flag, p.status, p.budget_ns};

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t w_policy = l2_policy_evict_first();   // the weight is streamed once
      int s = 0;
      uint32_t ph = 0, issued = 0, last_ph = 0;
      int tile = first_tile, kb = first_kb;
      // what iteration (tile, kb) reads
      int wcol, wcol1, wrow, xrow, kk;      // first and second 64 columns
      auto locate = [&]() {
        wcol = tile * 128;                                  // kProj, kDown: this tile's columns
        wrow = xrow = 0;
        kk = kb;
        wcol1 = wcol + 64;
        if (MODE == kUp) {
          const int t = tile % p.tiles;
          wrow = bars.experts[tile / p.tiles] * p.wrows;
          if (HALVES == 2) {
            wcol = t * 256;                                 // gate | up, 128 columns each
            wcol1 = wcol + 64;
          } else {
            wcol = t / 2 * 256 + t % 2 * 64;                // 64 gate and 64 up columns
            wcol1 = wcol + 128;
          }
        }
        if (MODE == kDown) {
          const int slot = kb / p.kblocks;
          kk = kb - slot * p.kblocks;
          xrow = slot * MPAD;
          wrow = bars.experts[slot] * p.wrows;
        }
      };
      auto step = [&](bool more) {
        ++kk;
        if (++kb == kblocks) {
          kb = 0;
          ++tile;
          if (more) locate();
        } else if (MODE == kDown && kk == p.kblocks) {
          if (more) locate();
        }
      };
      auto load_w = [&](int st) {
#pragma unroll
        for (int bx = 0; bx < 2 * HALVES; ++bx)
          tma_load_2d_hint(stage_w(st) + bx * W_BOX_BYTES, &tmap_w, &bars.full[st],
                           (bx & 1 ? wcol1 : wcol) + (bx & 2) * 64, wrow + kk * BK, w_policy);
      };
      int early = 0;                       // kDown: stages whose weights are on their way
      if (MODE == kDown) {
        early = min(share, STAGES);
        if (share) locate();
        for (int i = 0; i < early; ++i) {
          mbar_arrive_expect_tx(&bars.full[i], C::X_BYTES + C::W_BYTES);
          load_w(i);
          step(i + 1 < early);
        }
        tile = first_tile;
        kb = first_kb;
        grid_dependency_wait();
      }
      if (share) locate();
      for (int i = 0; i < share; ++i) {
        if (i >= early) {
          if (!mbar_wait(&bars.empty[s], ph ^ 1, ctl, kSiteProdEmpty)) break;
          mbar_arrive_expect_tx(&bars.full[s], C::X_BYTES + C::W_BYTES);
        }
        tma_load_2d(stage_x(s), &tmap_x, &bars.full[s], kk * BK, xrow);
        if (i >= early) load_w(s);
        issued |= 1u << s;
        last_ph = (last_ph & ~(1u << s)) | (ph << s);
        if (++s == STAGES) { s = 0; ph ^= 1; }
        step(i + 1 < share);
      }
      for (int i = 0; i < STAGES; ++i)
        if (issued & (1u << i)) drain_wait(&bars.full[i], (last_ph >> i) & 1u, p.budget_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_bf16_f32(128, MPAD, /*a MN-major*/ true, /*b MN-major*/ false);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int kb0 = first_kb, left = share;
      for (int seg = 0; left > 0 && ok; ++seg) {
        const int kb1 = min(kblocks, kb0 + left);
        const int b = seg & 1;
        const uint32_t aph = (seg >> 1) & 1;
        if (!mbar_wait(&bars.acc_empty[b], aph ^ 1, ctl, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&bars.full[s], ph, ctl, kSiteMmaFull)) { ok = false; break; }
          tc_fence_after();
          const uint32_t w0 = smem_u32(stage_w(s));
          const uint32_t x0 = smem_u32(stage_x(s));
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const uint32_t d_tmem = tmem_base + (b * HALVES + h) * MPAD;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              // A = W^T: 128 weight columns, N-major, two 64-column boxes; B = x^T: K-major rows
              const uint64_t adesc = sdesc_sw128(w0 + h * 2 * W_BOX_BYTES + kk * 2048, W_BOX_BYTES, 1024);
              const uint64_t bdesc = sdesc_sw128(x0 + kk * 32, 16, 1024);
              umma_bf16(d_tmem, adesc, bdesc, IDESC, (kb != kb0 || kk != 0) ? 1u : 0u);
            }
          }
          umma_commit(&bars.empty[s]);
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
        if (!ok) break;
        if (!(p.withhold && seg == 0)) umma_commit(&bars.acc_full[b]);
        left -= kb1 - kb0;
        kb0 = 0;
      }
      umma_commit(&bars.drain);
      drain_wait(&bars.drain, 0, p.budget_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                       // TMEM lane quarter this warp may access
    const int n = q * 32 + lane;                  // column within the tile
    const int et = threadIdx.x - 64;              // 0..127
    if (MODE == kDown) {                          // also before this kernel's stores: partials, y
      grid_dependency_wait();
      grid_launch_dependents();
    }
    if (MODE == kUp && et < MPAD) bars.rinv[et] = et < p.M ? __ldcg(p.route.rinv + et) : 0.f;
    int next_tile = first_tile, next_kb = first_kb, left = share;
    for (int seg = 0; left > 0; ++seg) {
      const int tile = next_tile, kb0 = next_kb;
      const int kb1 = min(kblocks, kb0 + left);
      left -= kb1 - kb0;
      ++next_tile;
      next_kb = 0;
      const int b = seg & 1;
      const uint32_t aph = (seg >> 1) & 1;
      if (MODE == kUp && et < MPAD)               // what the tile's expert weighs in each row
        bars.weight[seg & 1][et] =
            et < p.M ? __ldcg(p.route.weight + bars.experts[tile / p.tiles] * kMoeMaxRows + et) : 0.f;
      // One thread waits and the whole group follows its decision, so the
      // group never splits at the named barriers or the .sync.aligned loads.
      if (et == 0) bars.epi_ok[b] = mbar_wait(&bars.acc_full[b], aph, ctl, kSiteEpiAccFull) ? 1 : 0;
      named_bar_sync(1, 128);
      if (!bars.epi_ok[b]) break;
      tc_fence_after();
      // Chunks of RC rows: the code of one chunk serves them all.
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * HALVES * MPAD;
      float w[RC], r[RC];                         // kUp: routing weight and 1 / rms of the chunk's rows
      auto route = [&](int m0) {
        if constexpr (MODE == kUp) {
#pragma unroll
          for (int j = 0; j < RC; ++j) {
            w[j] = bars.weight[seg & 1][m0 + j];
            r[j] = bars.rinv[m0 + j];
          }
        }
      };
      auto finish = [&](int m0, float(&acc)[HALVES][RC]) {
        if constexpr (MODE == kUp && HALVES == 1) {
          // Lanes 0..63 hold the gate of 64 columns, lanes 64..127 their up.
          // The gate threads finish the first half of the rows, the up threads
          // the second, each with what the other passes through shared memory
          // (two buffers, so one barrier per chunk).
          constexpr int H = RC / 2;
          const bool up = n >= 64;
          const int c = n & 63;
          float* give = bars.swap[m0 / RC & 1][up ? 1 : 0];
          const float* take = bars.swap[m0 / RC & 1][up ? 0 : 1];
#pragma unroll
          for (int j = 0; j < H; ++j) give[j * 64 + c] = up ? acc[0][j] : acc[0][H + j];
          named_bar_sync(2, 128);
          __nv_bfloat16* dst = p.act + (static_cast<int64_t>(tile / p.tiles) * MPAD + m0) * p.ncols +
                               tile % p.tiles * 64 + c;
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const float own = up ? acc[0][H + j] : acc[0][j], other = take[j * 64 + c];
            const float wj = up ? w[H + j] : w[j], rj = up ? r[H + j] : r[j];
            const float v = wj * (silu_f32((up ? other : own) * rj) * ((up ? own : other) * rj));
            const int m = up ? H + j : j;
            if (m0 + m < p.M) dst[static_cast<int64_t>(m) * p.ncols] = __float2bfloat16_rn(wj != 0.f ? v : 0.f);
          }
        } else if constexpr (MODE == kUp) {
          // act = w silu(r gate) (r up), one round to bf16; 0 for rows that did not choose the expert
          __nv_bfloat16* dst =
              p.act + (static_cast<int64_t>(tile / p.tiles) * MPAD + m0) * p.ncols + tile % p.tiles * 128 + n;
#pragma unroll
          for (int j = 0; j < RC; ++j) {
            const float v = w[j] * (silu_f32(acc[0][j] * r[j]) * (acc[HALVES - 1][j] * r[j]));
            if (m0 + j < p.M) dst[static_cast<int64_t>(j) * p.ncols] = __float2bfloat16_rn(w[j] != 0.f ? v : 0.f);
          }
        } else {
          const int64_t col = static_cast<int64_t>(tile) * 128 + n;
          if (col < p.ncols) epi_finish<RC>(p.epi, m0, min(p.M - m0, RC), col, acc[0]);
        }
      };
      auto load = [&](int m0, float(&acc)[HALVES][RC]) {
        uint32_t raw[HALVES][RC];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) tmem_ld8(taddr + h * MPAD + m0, raw[h]);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int j = 0; j < RC; ++j) acc[h][j] = __uint_as_float(raw[h][j]);
      };
      if (MODE == kProjRows && kb0 == 0 && kb1 == kblocks) {
        // A whole tile of more rows: through shared memory, as in the tile kernel
        // (one column per thread took 27 us for 48 x 256 x 65536, this 14).
        const int64_t col0 = static_cast<int64_t>(tile) * 128 + q * 32;
        if (p.epi.out_fp32) finish_rows<true>(p, taddr, bars.scratch[q], lane, col0);
        else finish_rows<false>(p, taddr, bars.scratch[q], lane, col0);
        tc_fence_before();
        mbar_arrive(&bars.acc_empty[b]);
        continue;
      }
      if (kb0 == 0 && kb1 == kblocks) {
#pragma unroll 1
        for (int m0 = 0; m0 < p.M; m0 += RC) {
          float acc[HALVES][RC];
          route(m0);
          load(m0, acc);
          finish(m0, acc);
        }
        tc_fence_before();
        mbar_arrive(&bars.acc_empty[b]);
        continue;
      }
      // Shared tile: publish the partial (float4 groups [half][row / 4][column],
      // rows below M only), count, and go on unless this was the last one.
      {
        const int slot = static_cast<int>(cta) * 2 + (seg == 0 ? 0 : 1);
        float4* mine = reinterpret_cast<float4*>(p.part + static_cast<int64_t>(slot) * C::SLOT_FLOATS);
#pragma unroll 1
        for (int m0 = 0; m0 < p.M; m0 += RC) {
          float acc[HALVES][RC];
          load(m0, acc);
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int g = 0; g < RC / 4; ++g)
              if (m0 + 4 * g < p.M)
                __stcg(mine + (h * (MPAD / 4) + m0 / 4 + g) * 128 + n,
                       make_float4(acc[h][4 * g], acc[h][4 * g + 1], acc[h][4 * g + 2], acc[h][4 * g + 3]));
        }
      }
      tc_fence_before();
      mbar_arrive(&bars.acc_empty[b]);
      if (p.fixup) continue;
      const unsigned t0 = static_cast<unsigned>(tile) * kblocks;
      const int c_first = static_cast<int>(owner_of(t0)), c_last = static_cast<int>(owner_of(t0 + kblocks - 1));
      route(0);
      named_bar_sync(1, 128);
      if (et == 0) bars.last = count_partial(p.status, c_first, c_last - c_first + 1);
      named_bar_sync(1, 128);
      if (!bars.last) continue;
      // every partial of the tile is visible: add them in ascending k order
#pragma unroll 1
      for (int m0 = 0; m0 < p.M; m0 += RC) {
        float acc[HALVES][RC];
        if (m0) route(m0);
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int j = 0; j < RC; ++j) acc[h][j] = 0.f;
        constexpr int GROUPS = HALVES * RC / 4;
        constexpr int CB = 16 / GROUPS;                          // contributors in flight
#pragma unroll 1
        for (int c0 = c_first; c0 <= c_last; c0 += CB) {
          float4 v[CB][GROUPS];
#pragma unroll
          for (int j = 0; j < CB; ++j) {
            const unsigned c = min(c0 + j, c_last);
            // a CTA's first segment is slot 0; this tile is not its first when its share begins before it
            const int sl = static_cast<int>(c) * 2 + (c * total / grid >= t0 ? 0 : 1);
            const float4* src =
                reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(sl) * C::SLOT_FLOATS) + m0 / 4 * 128 + n;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
              v[j][g] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (c0 + j <= c_last && m0 + 4 * (g % (RC / 4)) < p.M)
                v[j][g] = __ldcg(src + (g / (RC / 4) * (MPAD / 4) + g % (RC / 4)) * 128);
            }
          }
#pragma unroll
          for (int j = 0; j < CB; ++j) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
              float* a = &acc[g / (RC / 4)][g % (RC / 4) * 4];
              a[0] += v[j][g].x;
              a[1] += v[j][g].y;
              a[2] += v[j][g].z;
              a[3] += v[j][g].w;
            }
          }
        }
        finish(m0, acc);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int MPAD, int HALVES, int MODE>
cudaError_t launch(Params& p, const CUtensorMap& tx, const CUtensorMap& tw, int num_sms, cudaStream_t stream) {
  constexpr size_t SMEM = smem_bytes<MPAD, HALVES, MODE>();
  const cudaError_t e = ensure_smem_limit<stream_kernel<MPAD, HALVES, MODE>>(static_cast<int>(SMEM));
  if (e != cudaSuccess) return e;
  if (num_sms > kMaxCounters) num_sms = kMaxCounters;
  // the experts' space is known to the kernel only
  const unsigned grid = is_proj<MODE> ? share_count(p.tiles, p.kblocks, num_sms) : static_cast<unsigned>(num_sms);
  return launch_pdl(stream_kernel<MPAD, HALVES, MODE>, grid, NUM_THREADS, SMEM, stream, tx, tw, p);
}

// Fix-up of kUp (128 + 128 columns) above FIXUP_ROWS: adds the partials of the
// shared tiles in ascending k order and stores their activations.  A tile is
// shared where a share begins inside it; the block row of its second sharer
// takes it.  One thread per (4 rows, column), 64 rows in 8 blocks.
constexpr int UP_FIX_THREADS = 256;
__global__ void __launch_bounds__(UP_FIX_THREADS) up_fixup_kernel(const Params p, int mpad, int ctas) {
  __shared__ uint32_t chosen[kMoeMaxExperts / 32];
  grid_launch_dependents();              // the down kernel waits for this one before it reads what either wrote
  // The router's ids: complete before the gate/up kernel could let this one start.
  for (int i = threadIdx.x; i < kMoeMaxExperts / 32; i += UP_FIX_THREADS) chosen[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * p.route.k; i += UP_FIX_THREADS) {
    const int e = __ldcg(p.route.ids + i);
    atomicOr(&chosen[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  int active = 0;
  for (int i = 0; i < kMoeMaxExperts / 32; ++i) active += __popc(chosen[i]);
  const int tiles = p.tiles * active;
  const unsigned total = static_cast<unsigned>(tiles) * p.kblocks;
  const unsigned grid = share_count(tiles, p.kblocks, static_cast<unsigned>(ctas));
  const unsigned c = blockIdx.x;
  const int g = static_cast<int>(blockIdx.y) * 2 + static_cast<int>(threadIdx.x >> 7);   // group of 4 rows
  const int n = static_cast<int>(threadIdx.x & 127);
  auto begin = [&](unsigned i) { return i * total / grid; };
  const unsigned tile = c < grid ? begin(c) / p.kblocks : 0, t0 = tile * p.kblocks;
  const unsigned first = ((t0 + 1) * grid - 1) / total, last = ((t0 + p.kblocks) * grid - 1) / total;
  const bool mine = c > 0 && c < grid && begin(c) != t0 && first + 1 == c;
  grid_dependency_wait();
  if (!mine || 4 * g >= p.M) return;
  float4 sum[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  const int64_t half = static_cast<int64_t>(mpad / 4) * 128;      // float4s of a half
  constexpr unsigned IN_FLIGHT = 4;
  for (unsigned c0 = first; c0 <= last; c0 += IN_FLIGHT) {
    float4 q[IN_FLIGHT][2];
#pragma unroll
    for (unsigned j = 0; j < IN_FLIGHT; ++j) {
      const unsigned o = min(c0 + j, last);
      const float4* src = reinterpret_cast<const float4*>(p.part) +
                          (static_cast<int64_t>(o) * 2 + (begin(o) >= t0 ? 0 : 1)) * 2 * half + g * 128 + n;
      q[j][0] = __ldcg(src);
      q[j][1] = __ldcg(src + half);
    }
#pragma unroll
    for (unsigned j = 0; j < IN_FLIGHT; ++j) {
      if (c0 + j <= last) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sum[h].x += q[j][h].x;
          sum[h].y += q[j][h].y;
          sum[h].z += q[j][h].z;
          sum[h].w += q[j][h].w;
        }
      }
    }
  }
  const int slot = static_cast<int>(tile) / p.tiles;
  int expert = 0;                        // the slot-th chosen one
  for (int left = slot, w = 0; w < kMoeMaxExperts / 32; ++w) {
    const int here = __popc(chosen[w]);
    if (left < here) {
      expert = w * 32 + static_cast<int>(__fns(chosen[w], 0, left + 1));
      break;
    }
    left -= here;
  }
  const float gate[4] = {sum[0].x, sum[0].y, sum[0].z, sum[0].w}, up[4] = {sum[1].x, sum[1].y, sum[1].z, sum[1].w};
  const float* wt = p.route.weight + expert * kMoeMaxRows;
  __nv_bfloat16* dst =
      p.act + (static_cast<int64_t>(slot) * mpad + 4 * g) * p.ncols + static_cast<int>(tile) % p.tiles * 128 + n;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = min(4 * g + j, p.M - 1);
    const float w = __ldcg(wt + m), r = __ldcg(p.route.rinv + m);
    const float v = w * (silu_f32(gate[j] * r) * (up[j] * r));
    if (4 * g + j < p.M) dst[static_cast<int64_t>(j) * p.ncols] = __float2bfloat16_rn(w != 0.f ? v : 0.f);
  }
}

// Partials: two slots per CTA.
inline size_t part_bytes(int mpad, int halves, int num_sms) {
  return static_cast<size_t>(num_sms) * 2 * halves * mpad * 128 * 4;
}

}  // namespace strm

// The stream kernel where its weight stream is the cost; the tile kernel, whose
// epilogue has twice the warps and whose pairs read 256 adjacent columns, where
// whole tiles' epilogues are, or rows off the 128-byte lines.  Measured, stream
// against tile kernel (us): 16 x 4096 x 51200 68 : 71, 16 x 4096 x 50000 87 : 73;
// 64 x 8192 x 32768 90 : 94, 64 x 1024 x 32768 22 : 18, 64 x 2048 x 8192 12 : 15;
// 100 x 4096 x 8192 19 : 23, 100 x 2000 x 12000 19 : 17.
bool proj_takes_stream(int64_t M, int64_t K, int64_t N, int num_sms) {
  const int64_t tiles = (N + 127) / 128;
  const bool lines = N % 64 == 0;
  if (M <= 16) return lines || tiles < 2 * num_sms;
  if (M <= 64) return 2 * tiles < 3 * num_sms || (lines && K >= 6144);
  return M <= 128 && 2 * tiles <= num_sms;
}

namespace {
int proj_mpad(int64_t M) { return M <= 64 ? decode_mpad(M) : 128; }
}  // namespace

size_t proj_stream_workspace_bytes(int64_t M, int num_sms) {
  return kWsHeaderBytes + strm::part_bytes(proj_mpad(M), 1, num_sms);
}

template <int MODE>
static cudaError_t launch_rows(int mp, strm::Params& p, const CUtensorMap& tx, const CUtensorMap& tw, const ProjArgs& a) {
  if (mp == 16) return strm::launch<16, 1, MODE>(p, tx, tw, a.num_sms, a.stream);
  if (mp == 32) return strm::launch<32, 1, MODE>(p, tx, tw, a.num_sms, a.stream);
  if (mp == 64) return strm::launch<64, 1, MODE>(p, tx, tw, a.num_sms, a.stream);
  return strm::launch<128, 1, MODE>(p, tx, tw, a.num_sms, a.stream);
}

cudaError_t launch_proj_stream(const ProjArgs& a) {
  using namespace strm;
  const int mp = proj_mpad(a.M);
  CUtensorMap tx, tw;
  if (!make_tmap_2d_ld(&tx, a.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.M, a.K, a.ldx, mp, BK)) return cudaErrorInvalidValue;
  // A row of a box is 128 bytes; where rows start off 128-byte lines, a fetch
  // widened to 256 bytes brings a neighbour's bytes that L2 drops again before
  // they are used (32 x 4096 x 50000: 110 us, 88 without, 71 with aligned rows).
  const auto promotion = a.ldw % 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!make_tmap_2d_ld(&tw, a.W, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.K, a.N, a.ldw, BK, 64, true, promotion))
    return cudaErrorInvalidValue;
  Params p = {};
  p.M = static_cast<int>(a.M);
  p.ncols = static_cast<int>(a.N);
  p.tiles = static_cast<int>((a.N + 127) / 128);
  p.kblocks = static_cast<int>((a.K + BK - 1) / BK);
  p.wrows = static_cast<int>(a.K);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.part = reinterpret_cast<float*>(ws + kWsHeaderBytes);
  p.budget_ns = a.budget_ns;
  p.withhold = a.withhold;
  p.w = static_cast<const uint8_t*>(a.W);
  p.w_row_bytes = a.ldw * 2;
  p.prefetch_iters = a.prefetch_iters;
  p.epi = a.epi;
  p.vec = epi_vector_ok(a.epi, a.N);
  p.fixup = a.M > FIXUP_ROWS;
  const int ctas = a.num_sms < kMaxCounters ? a.num_sms : kMaxCounters;
  const bool whole = a.M > RC && share_count(p.tiles, p.kblocks, ctas) <= static_cast<unsigned>(p.tiles);
  const cudaError_t e = whole ? launch_rows<kProjRows>(mp, p, tx, tw, a) : launch_rows<kProj>(mp, p, tx, tw, a);
  if (e != cudaSuccess || !p.fixup) return e;
  FixupArgs f = {};
  f.sharers = static_cast<int>(share_count(p.tiles, p.kblocks, ctas));
  if (f.sharers <= p.tiles && p.tiles % f.sharers == 0) return e;       // whole tiles only
  f.part = p.part;
  f.slot_floats = static_cast<int64_t>(mp) * 128;
  f.total = static_cast<int64_t>(p.tiles) * p.kblocks;
  f.kblocks = p.kblocks;
  f.ranks = 1;
  f.tile0 = 0;
  f.tiles = p.tiles;
  f.group_m = f.num_m = 1;
  f.num_n = p.tiles;
  f.rows = static_cast<int>((a.M + 3) / 4 * 4);
  f.M = a.M;
  f.N = a.N;
  f.epi = a.epi;
  f.stream = a.stream;
  return launch_proj_fixup(f);
}

// ---------------------------------------------------------------------------
// fn_moe_swiglu: router, then the two expert kernels
// ---------------------------------------------------------------------------
namespace {
// Workspace: header | 1/rms | weight table | ids | partials | act
struct MoeLayout {
  size_t rinv, weight, ids, part, act, end;
  int64_t slots;       // most experts that can be chosen
};
MoeLayout moe_layout(int64_t M, int64_t I, int64_t E, int top_k, int num_sms) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const int mp = decode_mpad(M);
  MoeLayout l;
  l.slots = E < M * top_k ? E : M * top_k;
  l.rinv = kWsHeaderBytes;
  l.weight = l.rinv + up(kMoeMaxRows * 4);
  l.ids = l.weight + up(static_cast<size_t>(E) * kMoeMaxRows * 4);
  l.part = l.ids + up(static_cast<size_t>(kMoeMaxRows) * kMoeMaxTopK * 4);
  l.act = l.part + up(strm::part_bytes(mp, 2, num_sms));
  l.end = l.act + static_cast<size_t>(l.slots) * mp * I * 2;
  return l;
}
}  // namespace

size_t moe_workspace_bytes(int64_t M, int64_t I, int64_t E, int top_k, int num_sms) {
  return moe_layout(M, I, E, top_k, num_sms).end;
}

template <int MPAD, int UP_HALVES>
static cudaError_t launch_experts(strm::Params& p, const MoeArgs& a, const CUtensorMap (&maps)[4]) {
  using namespace strm;
  p.ncols = static_cast<int>(a.I);
  p.tiles = static_cast<int>(a.I / (64 * UP_HALVES));
  p.kblocks = static_cast<int>(a.d / BK);
  p.wrows = static_cast<int>(a.d);
  // Gate/up: only where no CTA finishes whole tiles (55 rows, 5 experts of 4544 x
  // 384: layer 50 -> 38 us); among whole ones the last sharer's work hides (40 rows,
  // 256 experts of 4096 x 256: 238 us, 244 with the fix-up kernel).
  const int64_t slots = a.E < a.M * a.top_k ? a.E : a.M * a.top_k;
  p.fixup = a.M > FIXUP_ROWS && slots * p.tiles < a.num_sms;
  const int ctas = a.num_sms < kMaxCounters ? a.num_sms : kMaxCounters;
  cudaError_t e = strm::launch<MPAD, UP_HALVES, kUp>(p, maps[0], maps[1], a.num_sms, a.stream);
  if (e != cudaSuccess) return e;
  if (p.fixup) {
    static_assert(UP_HALVES == 2 || MPAD <= FIXUP_ROWS, "the fix-up adds gate and up");
    e = launch_pdl_grid(up_fixup_kernel, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((a.M + 7) / 8)),
                        UP_FIX_THREADS, 0, a.stream, p, MPAD, ctas);
    if (e != cudaSuccess) return e;
  }
  p.ncols = static_cast<int>(a.d);
  p.tiles = static_cast<int>((a.d + 127) / 128);
  p.kblocks = static_cast<int>(a.I / BK);
  p.wrows = static_cast<int>(a.I);
  p.fixup = a.M > FIXUP_ROWS;
  e = strm::launch<MPAD, 1, kDown>(p, maps[2], maps[3], a.num_sms, a.stream);
  if (e != cudaSuccess || !p.fixup) return e;
  FixupArgs f = {};
  f.part = p.part;
  f.slot_floats = MPAD * 128;
  f.kblocks = p.kblocks;                 // per expert: the kernel counts the experts
  f.route = p.route;
  f.routed = static_cast<int>(a.M) * a.top_k;
  f.sharers = ctas;
  f.ranks = 1;
  f.tiles = p.tiles;
  f.group_m = f.num_m = 1;
  f.num_n = p.tiles;
  f.rows = static_cast<int>((a.M + 3) / 4 * 4);
  f.M = a.M;
  f.N = a.d;
  f.epi = p.epi;
  f.stream = a.stream;
  return launch_proj_fixup(f);
}

cudaError_t launch_moe(const MoeArgs& a) {
  using namespace strm;
  const int mp = decode_mpad(a.M);
  const MoeLayout l = moe_layout(a.M, a.I, a.E, a.top_k, a.num_sms);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  constexpr CUtensorMapDataType BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap maps[4];   // x, gate/up weight; act, down weight
  if (!make_tmap_2d(&maps[0], a.x, BF16, 2, a.M, a.d, mp, BK) ||
      !make_tmap_2d(&maps[1], a.Wgu, BF16, 2, a.E * a.d, 2 * a.I, BK, 64) ||
      !make_tmap_2d(&maps[2], ws + l.act, BF16, 2, l.slots * mp, a.I, mp, BK) ||
      !make_tmap_2d(&maps[3], a.Wd, BF16, 2, a.E * a.I, a.d, BK, 64))
    return cudaErrorInvalidValue;
  Params p = {};
  p.M = static_cast<int>(a.M);
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.part = reinterpret_cast<float*>(ws + l.part);
  p.budget_ns = a.budget_ns;
  p.withhold = a.withhold;
  p.route.ids = reinterpret_cast<const int*>(ws + l.ids);
  p.route.weight = reinterpret_cast<const float*>(ws + l.weight);
  p.route.rinv = reinterpret_cast<const float*>(ws + l.rinv);
  p.route.E = static_cast<int>(a.E);
  p.route.k = a.top_k;
  p.act = reinterpret_cast<__nv_bfloat16*>(ws + l.act);
  p.epi.residual = a.residual;
  p.epi.ldr = a.d;
  p.epi.y = a.y;
  p.epi.ldy = a.d;
  const cudaError_t e = launch_moe_router(a, reinterpret_cast<int*>(ws + l.ids), reinterpret_cast<float*>(ws + l.weight),
                                          reinterpret_cast<float*>(ws + l.rinv));
  if (e != cudaSuccess) return e;
  // Gate/up tiles of 64 + 64 columns when one token's experts then fill the SMs
  // with whole tiles, which need no exchange (2048 x 1024, 8 experts: layer
  // 38.4 -> 36.5 us); otherwise 128 + 128, which read 512 bytes of a weight row at
  // a time (13 rows, 8 of 128 experts of 2048 x 768: layer 83 us, 103 us with 64).
  const int tiles64 = static_cast<int>(a.I / 64) * a.top_k;
  const bool split = a.M == 1 && tiles64 <= a.num_sms &&
                     share_count(tiles64, static_cast<int>(a.d / BK), a.num_sms) == static_cast<unsigned>(tiles64);
  if (mp == 16) return split ? launch_experts<16, 1>(p, a, maps) : launch_experts<16, 2>(p, a, maps);
  if (mp == 32) return launch_experts<32, 2>(p, a, maps);
  return launch_experts<64, 2>(p, a, maps);
}

}  // namespace fn
