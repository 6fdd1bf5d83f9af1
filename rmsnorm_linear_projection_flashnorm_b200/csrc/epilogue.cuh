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

template <int N, typename T>
__device__ __forceinline__ void epi_load(const T* src, int64_t ld, int rows, float (&r)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) r[j] = j < rows ? static_cast<float>(src[j * ld]) : 0.f;
}

// Rows row0 .. row0 + rows - 1 (at most N) of column col.
template <int N>
__device__ __forceinline__ void epi_finish(const Epilogue& e, int64_t row0, int rows, int64_t col, float (&v)[N]) {
  float res[N];
#pragma unroll
  for (int j = 0; j < N; ++j) res[j] = 0.f;
  if (e.residual) {
    const int64_t at = row0 * e.ldr + col;
    if (e.out_fp32) epi_load<N>(static_cast<const float*>(e.residual) + at, e.ldr, rows, res);
    else epi_load<N>(static_cast<const __nv_bfloat16*>(e.residual) + at, e.ldr, rows, res);
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

}  // namespace fn
