// Bias, activation and residual of a projection's epilogue, shared by the
// kernels of fn_proj (stream.cu, proj_tile.cu).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fn {

// Counters of the CTAs that have written their partial of a shared tile: one
// byte each in the workspace header behind the status word (bytes 16..255), so
// whatever other calls leave in the workspace body, they are zero between
// calls.  A shared tile counts in the byte of the first CTA (or pair and rank)
// that shares it; no other shared tile starts there.
constexpr int kCounterOffset = 16;
constexpr int kMaxCounters = static_cast<int>(kWsHeaderBytes) - kCounterOffset;

// CTAs that take a share of tiles x kblocks iterations: all of them, but no
// more than s to a tile (s rounds of partials to add, kblocks / s iterations to
// stream: the sum is least near the root of kblocks); or a whole number per
// tile where that costs at most ALIGN_SLACK iterations more, since a share that
// ends with its tile has one exchange instead of two, and none if it is whole.
constexpr unsigned ALIGN_SLACK = 3, WHOLE_SLACK = 8;
__host__ __device__ __forceinline__ unsigned share_count(int tiles, int kblocks, unsigned ctas) {
  const unsigned total = static_cast<unsigned>(tiles) * kblocks;
  unsigned most = total < ctas ? total : ctas;
  unsigned per_tile = 16;
  while (per_tile < 64 && per_tile * per_tile < 2u * kblocks) per_tile += 16;
  if (most > tiles * per_tile) most = tiles * per_tile;
  const unsigned s = most / tiles;
  if (s == 0) return most;
  const unsigned slack = s == 1 ? WHOLE_SLACK : ALIGN_SLACK;
  return (kblocks + s - 1) / s <= (total + most - 1) / most + slack ? s * tiles : most;
}

// Count this CTA's partial; true for the last of `n` (which resets the byte).
// One thread calls it behind a barrier that follows all of the CTA's stores,
// and a barrier follows before the others' partials are read: the acquire and
// release of the atomic carry what the barriers have ordered.
__device__ __forceinline__ bool count_partial(unsigned int* header, int index, int n) {
  unsigned int* word = header + (kCounterOffset + index) / 4;
  const int shift = (index & 3) * 8;
  unsigned int old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
               : "=r"(old) : "l"(word), "r"(1u << shift) : "memory");
  const bool last = ((old >> shift) & 0xFFu) == static_cast<unsigned int>(n - 1);
  if (last) atomicSub(word, static_cast<unsigned int>(n) << shift);
  return last;
}

// The epilogue of N rows of one column: act(v + bias) + residual, rounded once.
// The activation, the types and the residual are the same for the whole call,
// so each is one branch around a straight loop: a branch per element makes the
// instruction stream jump through code that a small call fetches for the first
// time (45 rows x 4099 columns took 36 us that way).
template <int N>
__device__ __forceinline__ void epi_act(int act, float (&z)[N]) {
  switch (act) {
    case 1:                                                          // relu (NaN stays)
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = z[j] < 0.f ? 0.f : z[j];
      break;
    case 2:                                                          // gelu: z Phi(z), no cancellation for z < 0
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = 0.5f * z[j] * erfcf(z[j] * -0.70710678118654752f);
      break;
    case 3:                                                          // gelu, tanh form
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // (1 + tanh u) / 2 = 1 / (1 + e^{-2u})
        const float u2 = 1.5957691216057308f * (z[j] + 0.044715f * z[j] * z[j] * z[j]);
        z[j] = z[j] / (1.f + __expf(-u2));
      }
      break;
    case 4:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = silu_f32(z[j]);
      break;
  }
}

// Rows past the end repeat the last one: without a condition on each, all loads
// are in flight before the first value is used (with one, the conversion sat
// behind every load, and a residual doubled the time of 4096 x 2048 x 4096).
template <int N, typename T>
__device__ __forceinline__ void epi_load(const T* src, int64_t ld, int rows, T (&r)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) r[j] = src[min(j, rows - 1) * ld];
}

// Rows row0 .. row0 + rows - 1 (1 to N of them) of column col.
template <int N>
__device__ __forceinline__ void epi_finish(const Epilogue& e, int64_t row0, int rows, int64_t col, float (&v)[N]) {
  float res[N];
  if (!e.residual) {
#pragma unroll
    for (int j = 0; j < N; ++j) res[j] = 0.f;
  } else if (e.out_fp32) {
    epi_load<N>(static_cast<const float*>(e.residual) + row0 * e.ldr + col, e.ldr, rows, res);
  } else {
    __nv_bfloat16 h[N];
    epi_load<N>(static_cast<const __nv_bfloat16*>(e.residual) + row0 * e.ldr + col, e.ldr, rows, h);
#pragma unroll
    for (int j = 0; j < N; ++j) res[j] = __bfloat162float(h[j]);
  }
  const float bias = e.bias ? __ldg(e.bias + col) : 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] += bias;
  epi_act<N>(e.act, v);
  const int64_t at = row0 * e.ldy + col;
  if (e.out_fp32) {
    float* dst = static_cast<float*>(e.y) + at;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < rows) dst[j * e.ldy] = v[j] + res[j];
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(e.y) + at;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < rows) dst[j * e.ldy] = __float2bfloat16_rn(v[j] + res[j]);
  }
}

// The same for a warp that holds 16 rows of 32 columns, one column per lane:
// the values pass through shared memory (16 rows of SCRATCH_LD floats of this
// warp's own), so that a lane has 4 columns of 4 rows and reads the residual and
// writes the output 8 or 16 bytes at a time.  One column per lane takes 2-byte
// stores, and four times as many of them.
constexpr int SCRATCH_LD = 36;
constexpr int SCRATCH_FLOATS = 16 * SCRATCH_LD;

// Whether every row's groups of 4 columns lie on whole vectors; where not,
// lanes store one column each (a group of 4 as single elements leaves gaps
// between the lanes; with it, and 256 rows to a tile whatever the number of
// tiles, 498 x 416 x 277 took 23 us instead of 8).
inline __host__ bool epi_vector_ok(const Epilogue& e, int64_t N) {
  const uintptr_t bytes = e.out_fp32 ? 16 : 8;
  return N % 4 == 0 && e.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(e.y) % bytes == 0 &&
         (!e.residual || (e.ldr % 4 == 0 && reinterpret_cast<uintptr_t>(e.residual) % bytes == 0));
}

template <bool F32>
struct Quad;             // 4 values of the output's type
template <>
struct Quad<true> {
  using Raw = float4;
  static __device__ __forceinline__ void get(const Raw& r, float* f) { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
  static __device__ __forceinline__ Raw put(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Quad<false> {
  using Raw = uint2;
  static __device__ __forceinline__ void get(const Raw& r, float* f) {
    f[0] = bf16lo_to_f32(r.x), f[1] = bf16hi_to_f32(r.x), f[2] = bf16lo_to_f32(r.y), f[3] = bf16hi_to_f32(r.y);
  }
  static __device__ __forceinline__ Raw put(const float* f) {
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
};

// The residual of 16 rows of 32 columns ahead of its use, in the vector form:
// a dependent load in the epilogue waits 1 us while the operand stream fills L2.
template <bool F32>
__device__ __forceinline__ void epi_fetch(const Epilogue& e, int lane, int64_t row0, int rows, int64_t col0, int64_t N,
                                          typename Quad<F32>::Raw (&r)[4]) {
  using T = typename Quad<F32>::Raw;
  const int64_t col = col0 + lane % 8 * 4;
  if (rows <= 0 || col >= N) return;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int64_t at = (row0 + min(g * 4 + lane / 8, rows - 1)) * e.ldr + col;
    r[g] = F32 ? *reinterpret_cast<const T*>(static_cast<const float*>(e.residual) + at)
               : *reinterpret_cast<const T*>(static_cast<const __nv_bfloat16*>(e.residual) + at);
  }
}

// Transpose to 4 rows of 4 columns, add the bias, apply the activation.
__device__ __forceinline__ void epi_transpose_act(const Epilogue& e, float* scratch, int lane, const float4& bias,
                                                  const uint32_t (&v)[16], float (&z)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) scratch[j * SCRATCH_LD + lane] = __uint_as_float(v[j]);
  __syncwarp();
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float4 f = *reinterpret_cast<const float4*>(scratch + (g * 4 + lane / 8) * SCRATCH_LD + lane % 8 * 4);
    z[4 * g] = f.x + bias.x, z[4 * g + 1] = f.y + bias.y, z[4 * g + 2] = f.z + bias.z, z[4 * g + 3] = f.w + bias.w;
  }
  __syncwarp();
  epi_act<16>(e.act, z);
}

template <bool F32>
__device__ __forceinline__ void epi_store_vec(const Epilogue& e, const typename Quad<F32>::Raw (&raw)[4], int lane,
                                              int64_t row0, int rows, int64_t col0, int64_t N, float (&z)[16]) {
  using Q = Quad<F32>;
  using T = typename Q::Raw;
  const int64_t col = col0 + lane % 8 * 4;
  if (e.residual) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[4];
      Q::get(raw[g], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[4 * g + j] += f[j];
    }
  }
  const int64_t at = (row0 + lane / 8) * e.ldy + col;
  T* dst = F32 ? reinterpret_cast<T*>(static_cast<float*>(e.y) + at)
               : reinterpret_cast<T*>(static_cast<__nv_bfloat16*>(e.y) + at);
#pragma unroll
  for (int g = 0; g < 4; ++g)
    if (g * 4 + lane / 8 < rows && col < N) dst[g * e.ldy] = Q::put(z + 4 * g);   // 4 rows are ldy groups of 4
}

}  // namespace fn
