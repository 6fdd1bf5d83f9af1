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
// Thread-level: the caller orders the partial's stores before and the others'
// loads after (__threadfence on both sides).
__device__ __forceinline__ bool count_partial(unsigned int* header, int index, int n) {
  unsigned int* word = header + (kCounterOffset + index) / 4;
  const int shift = (index & 3) * 8;
  const bool last = ((atomicAdd(word, 1u << shift) >> shift) & 0xFFu) == static_cast<unsigned int>(n - 1);
  if (last) atomicSub(word, static_cast<unsigned int>(n) << shift);
  return last;
}

// fp32 in, fp32 out; the result is rounded once, after the residual.
__device__ __forceinline__ float epi_act(int act, float z) {
  switch (act) {
    case 1: return z < 0.f ? 0.f : z;                               // relu (NaN stays)
    case 2: return 0.5f * z * erfcf(z * -0.70710678118654752f);        // gelu: z Phi(z), no cancellation for z < 0
    case 3: {                                                       // gelu, tanh form
      // (1 + tanh u) / 2 = 1 / (1 + e^{-2u})
      const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
      return z / (1.f + __expf(-u2));
    }
    case 4: return silu_f32(z);
  }
  return z;
}

__device__ __forceinline__ float epi_residual(const Epilogue& e, int64_t m, int64_t n) {
  if (!e.residual) return 0.f;
  if (e.out_fp32) return static_cast<const float*>(e.residual)[m * e.ldr + n];
  return __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[m * e.ldr + n]);
}

__device__ __forceinline__ void epi_store(const Epilogue& e, int64_t m, int64_t n, float v) {
  if (e.out_fp32) static_cast<float*>(e.y)[m * e.ldy + n] = v;
  else static_cast<__nv_bfloat16*>(e.y)[m * e.ldy + n] = __float2bfloat16_rn(v);
}

}  // namespace fn
