// Log probabilities of given tokens, entropies and top alternatives from the
// logits of a head projection, and their gradient, sm_100a.
//
// With z = scale * logits, m = max z, d_v = z_v - m, over a row of V logits:
//   s = sum_v e^{d_v},  t = sum_v d_v e^{d_v}
//   lse = m + ln s,  logprob = d_target - ln s,  entropy = ln s - t / s
// all from ONE pass over the logits with running (m, s, t): when the maximum
// grows by D the sums become s' = s e^{-D}, t' = e^{-D} (t - s D).  The
// products run in the base-2 exponent domain, c = scale log2 e, 32-bit floats:
// d = fma(x, c, -mu) with mu = m c rounded, one instruction for a pair, and the
// rounding of mu (known exactly, fma(m, c, -mu)) taken out behind the loop.  Where
// that rounding is not small, d = (x - m) scale log2 e.
//
// The pass is bound by HBM (2 or 4 bytes per logit, read once) without
// alternatives, by issue slots with them: a pair of 16-bit logits takes 15
// instructions, two of them ex2, and 20 with 8 alternatives.
// Every thread copies the vectors that it will read itself to shared memory
// two tiles ahead (cp.async), so loads are in flight while it computes and the
// main loop has no barrier.
//
// Top alternatives in the same pass: a logit becomes a 64-bit key, its ordered
// bit pattern above the complement of its index, so keys are unique, ties go
// to the lower index and the order of arrival does not matter.  Each warp
// keeps its 32 largest keys, sorted, one per lane.  A threshold key, never
// above the true k-th largest, filters the stream: one comparison per tile of a
// thread (32 logits, 16 in fp32).  It is the largest of
//   the k-th largest of all threads' maxima, taken after 1, 4, 16, ... tiles
//     (about k logits of a tile lie above it, however many there were before);
//   the warps' own k-th keys;
//   where many lanes of a warp hold survivors (rows that grow steadily), the
//     k-th largest of their maxima.
// What a warp does per survivor decides the speed (at 8 alternatives of 131072
// logits, 130 instructions for each survivor of the warps' own thresholds
// doubled the kernel's time), so a thread that holds one only queues the place
// of its vectors; 32 of them at a time are read again and give up their keys.
// A warp whose buffer fills sorts it into a list of its 32 largest; most rows
// end before that.  At the end a key's place is the number of keys above it,
// which a thread counts for each.  Logits of -inf never survive; where fewer
// than k others are left, the row's first ones fill the places.
//
// Work split: one thread-block cluster per row; C = 1, 2, 4 or 8 CTAs, more
// when there are few rows, so one decoded token still uses 8 SMs.  The CTAs'
// (m, s, t) and top lists meet in distributed shared memory in rank order:
// one launch, no workspace, no atomics on results, bit-identical repeats.
//
// Measured at 1965 MHz (and in a long run under the power cap, at 1.6 to 1.7
// GHz): 4096 x 131072 bf16 with 8 alternatives 208 us (240), 5.2 TB/s; without
// 162 us (195), 6.6 TB/s; 2048 x 131072 fp32 with 8 alternatives 183 us (191);
// one row with 20 alternatives 10 us.  A thread that has met nothing but a mask's
// fill of -2^24 / c and below takes the exact differences: with such a fill in the
// first three quarters of each row 2048 x 131072 bf16 takes 116 us instead of 94.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cfloat>

#include "dsmem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fn {
namespace lp {

constexpr int MAX_THREADS = 256;
constexpr int VECS = 4;                       // 16-byte vectors per thread and tile
constexpr int MAX_K = kMaxTopAlternatives;    // 32: one key per lane
constexpr int STAGES = 2;                     // tiles in flight
constexpr int CROWD = 12;                     // lanes with survivors from which the threshold is raised first
constexpr float FAR = -200.f;                 // 2^FAR is 0 in fp32: nothing below it counts
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
static_assert(MAX_K == 32, "one list entry per lane");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Element types: 16-byte vectors as packed words, the NaN-propagating maximum
// of a vector, and the unpacked fp32 values.
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo_to_f32(w[i]);
      f[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
  }
  static __device__ __forceinline__ uint32_t wmax(uint32_t a, uint32_t b) {   // NaN if either is
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return a;
  }
  static __device__ __forceinline__ float wvalue(uint32_t a) { return max_nan(bf16lo_to_f32(a), bf16hi_to_f32(a)); }
  // Largest pair of values not above f, and both halves of a word kept from below it.
  static __device__ __forceinline__ bool floor_word(float f, uint32_t& w) {
    const __nv_bfloat16 h = __float2bfloat16_rd(f);
    const uint32_t u = __bfloat16_as_ushort(h);
    w = u | u << 16;
    return isfinite(__bfloat162float(h));
  }
  static __device__ __forceinline__ uint32_t clamp(uint32_t v, uint32_t w) {
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(w));
    return v;
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ __nv_bfloat16 from(float f) { return __float2bfloat16_rn(f); }
};
template <>
struct Elem<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint32_t wmax(uint32_t a, uint32_t b) {
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return a;
  }
  static __device__ __forceinline__ float wvalue(uint32_t a) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
    return max_nan(f.x, f.y);
  }
  static __device__ __forceinline__ bool floor_word(float f, uint32_t& w) {
    const __half h = __float2half_rd(f);
    const uint32_t u = __half_as_ushort(h);
    w = u | u << 16;
    return isfinite(__half2float(h));
  }
  static __device__ __forceinline__ uint32_t clamp(uint32_t v, uint32_t w) {
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(w));
    return v;
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ __half from(float f) { return __float2half_rn(f); }
};
template <>
struct Elem<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint32_t wmax(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float wvalue(uint32_t a) { return __uint_as_float(a); }
  static __device__ __forceinline__ bool floor_word(float f, uint32_t& w) {
    w = __float_as_uint(f);
    return isfinite(f);
  }
  static __device__ __forceinline__ uint32_t clamp(uint32_t v, uint32_t w) {
    return __float_as_uint(max_nan(__uint_as_float(v), __uint_as_float(w)));
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ float from(float f) { return f; }
};

// Maximum of a vector as a packed word; NaN if any value is.
template <typename T>
__device__ __forceinline__ uint32_t vmax(const uint4& v) {
  using E = Elem<T>;
  return E::wmax(E::wmax(v.x, v.y), E::wmax(v.z, v.w));
}

// ---------------------------------------------------------------------------
// keys: (ordered value, complement of the index); 0 is below every real key
// ---------------------------------------------------------------------------
using Key = unsigned long long;

__device__ __forceinline__ uint32_t ordered(float v) {
  v += 0.0f;                                        // -0 ties with +0
  const uint32_t u = __float_as_uint(v);
  if (v != v) return 0xFFFFFFFFu;                   // NaN ranks first
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ Key make_key(float v, uint32_t idx) {
  return (static_cast<Key>(ordered(v)) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(Key k) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}

// The largest key of -inf; those above it have values.
constexpr Key NOTHING = 0x007FFFFFFFFFFFFFull;

// One step of a bitonic network over the lanes: keep the larger key where
// `keep_max`, else the smaller.
template <typename K>
__device__ __forceinline__ K cmp_xchg(K k, int mask, bool keep_max) {
  const K o = __shfl_xor_sync(0xffffffffu, k, mask);
  return (k > o) == keep_max ? k : o;
}
// Sort 32 keys over the lanes, largest in lane 0.
template <typename K>
__device__ __forceinline__ K warp_sort(K k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) {
      const bool down = (lane & size) == 0;          // this run is sorted downwards
      k = cmp_xchg(k, j, ((lane & j) == 0) == down);
    }
  }
  return k;
}
// The 32 largest of two sorted runs, sorted: the larger of a[i] and b[31 - i]
// is a bitonic run that holds them.
template <typename K>
__device__ __forceinline__ K warp_merge(K a, K b, int lane) {
  const K r = __shfl_sync(0xffffffffu, b, 31 - lane);
  K k = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) k = cmp_xchg(k, j, (lane & j) == 0);
  return k;
}

struct Stat {
  float m, s, t;   // maximum (raw logits), sum of 2^d, sum of d 2^d
};
// The reference of d for maximum m: d = fma(x, c, -mu) where mu = m c is of
// ordinary size, else d = (x - m) scale log2 e (a mask's finite fill, a large scale, a
// maximum near the type's lowest value, or infinite).  Ordinary ends at 2^24:
// mu is then off by at most 1/2, so the largest term of the sum, 2^delta with
// delta = m c - mu, lies within a factor of 2^(1/2) of 1.  (Half a step of mu
// passes 127 at 2^31; from there 2^delta may be infinite or 0.)
constexpr float ORDINARY = 0x1p24f;
// (x - m) scale, as (x h - m h) (scale / h) with h = 1/2 at scales below 1, where
// halves are exact as far as they count: the difference of two finite logits may
// be infinite when its product is not.
struct Scale {
  float half, rest;   // h, scale / h
};
__device__ __forceinline__ float difference(float x, float m, const Scale& k) {
  return fmaf(x, k.half, -(m * k.half)) * k.rest;
}
__device__ __forceinline__ float exact_distance(float x, float m, const Scale& k) {
  return difference(x, m, k) * LOG2E;    // not by c: it is infinite at scales above 2.3e38, and 0 times it NaN
}
__device__ __forceinline__ float reference_delta(float m, float c) {
  const float mu = __fmul_rn(m, c);
  return fabsf(mu) < ORDINARY ? fmaf(m, c, -mu) : 0.f;
}
// Two results whose reference is the maximum itself.
__device__ __forceinline__ Stat merge_stat(const Stat& a, const Stat& b, const Scale& k) {
  const bool first = a.m >= b.m;
  const float lo = first ? b.m : a.m, hi = first ? a.m : b.m;
  const float ls = first ? b.s : a.s, lt = first ? b.t : a.t;
  const float D = lo == hi ? 0.f : max_nan(exact_distance(lo, hi, k), FAR);
  const float f = ex2(D);
  Stat r;
  r.m = max_nan(a.m, b.m);
  r.s = fmaf(f, ls, first ? a.s : b.s);
  r.t = fmaf(f, fmaf(ls, D, lt), first ? a.t : b.t);
  return r;
}

template <int THREADS>
struct Smem {
  static constexpr int WARPS = THREADS / 32, TILE = THREADS * VECS;   // of 16-byte vectors
  union {
    uint4 stage[STAGES][TILE];
    Key pool[WARPS * 64];        // at the end: what the warps kept, then what the ranks kept
  };
  Key buf[WARPS][64];            // survivors
  int queue[WARPS][64];          // first vectors of threads with survivors
  Key top[32];                   // this CTA's result, read by rank 0 of the cluster
  Key thr;                       // largest of the warps' k-th keys
  int pooled;                    // keys in the pool
  uint32_t vals[WARPS][32];      // sorted maxima of the lanes, merged in vals[0]
  Stat wstat[WARPS];
  Stat stat;            // this CTA's (m, s, t), read by rank 0
};

__device__ __forceinline__ void copy_async(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The k largest of the n unique keys in sm.pool, largest first, to sm.top.  All
// threads call, behind a barrier; ends with one.
template <int THREADS>
__device__ __forceinline__ void select_top(Smem<THREADS>& sm, int n, int k) {
  for (int i = static_cast<int>(threadIdx.x); i < n; i += THREADS) {
    const Key key = sm.pool[i];
    int above = 0;
#pragma unroll 8
    for (int o = 0; o < n; ++o) above += sm.pool[o] > key ? 1 : 0;
    if (above < k) sm.top[above] = key;
  }
  __syncthreads();
}

struct Params {
  const void* logits;
  int64_t ld;
  int V, C, k;
  const int* targets;
  float scale;
  Scale by;
  float *logprob, *entropy, *lse, *top_logprobs;
  int* top_ids;
};

template <typename T, bool TOPK, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const Params p) {
  using E = Elem<T>;
  constexpr int N = E::N;
  constexpr int WARPS = THREADS / 32, TILE = THREADS * VECS;
  __shared__ Smem<THREADS> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % p.C);
  const int64_t row = blockIdx.x / p.C;
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  const float c = p.scale * LOG2E;
  if (TOPK && threadIdx.x == 0) {
    sm.thr = 0;
    sm.pooled = 0;
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // Scalars up to the first 16-byte boundary, whole vectors, scalars behind
  // them.  Each rank takes a contiguous share of the vectors, rank 0 the (at
  // most 2 N - 2) scalars too.
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int head = min(mis ? N - mis : 0, p.V);
  const int nv = (p.V - head) / N;
  const int tail0 = head + nv * N;
  const int v0 = static_cast<int>(static_cast<int64_t>(nv) * rank / p.C);
  const int v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / p.C);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);

  auto fetch = [&](int base, int s) {         // this thread's vectors of a tile
    const uint4* src = xv + base + threadIdx.x;
    uint4* dst = &sm.stage[s][threadIdx.x];
    if (base + TILE <= v1) {
#pragma unroll
      for (int j = 0; j < VECS; ++j) copy_async(dst + j * THREADS, src + j * THREADS);
    } else {
#pragma unroll
      for (int j = 0; j < VECS; ++j)
        if (base + j * THREADS + static_cast<int>(threadIdx.x) < v1) copy_async(dst + j * THREADS, src + j * THREADS);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(v0 + s * TILE, s);
  if (TOPK) __syncthreads();                  // sm.thr is set

  Stat st{-INFINITY, 0.f, 0.f};
  // top alternatives of this warp
  Key best = 0, bound = 0;                    // bound: from all threads' maxima
  Key thr = NOTHING;                          // keys above it survive: values above thr_v,
  float thr_v = -FLT_MAX;                     // or equal to it with an index up to thr_i
  uint32_t thr_i = 0xFFFFFFFFu;
  int pending = 0, queued = 0, tile = 0, refresh = 1;
  auto raise = [&](Key t) {
    if (t > thr) {
      thr = t;
      thr_v = key_value(t + 1);
      thr_i = 0xFFFFFFFFu - static_cast<uint32_t>(t + 1);
    }
  };
  auto flush = [&]() {                        // the first 32 survivors into the list
    __syncwarp();
    best = warp_merge(best, warp_sort(lane < pending ? sm.buf[warp][lane] : 0, lane), lane);
    const Key rest = sm.buf[warp][32 + lane];
    __syncwarp();
    pending = max(pending - 32, 0);
    if (lane < pending) sm.buf[warp][lane] = rest;
    const Key kth = __shfl_sync(0xffffffffu, best, p.k - 1);
    if (lane == 0 && kth > thr) atomicMax(&sm.thr, kth);
    raise(kth);
  };
  auto append = [&](bool on, Key k) {
    const uint32_t b = __ballot_sync(0xffffffffu, on);
    if (on) sm.buf[warp][pending + __popc(b & ((1u << lane) - 1u))] = k;
    pending += __popc(b);
    if (pending >= 32) flush();
  };
  auto process = [&]() {                      // the first 32 of the queue
    __syncwarp();
    uint32_t mask = 0;                        // candidates of this lane's VECS vectors
    int v = 0;
    Key seen;
    auto filter = [&](uint32_t among) {
      seen = thr;
      mask = 0;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        if ((among >> (j * N) & ((1u << N) - 1u)) && v + j * THREADS < v1) {
          float f[N];
          E::unpack(__ldg(xv + v + j * THREADS), f);
          const uint32_t i0 = static_cast<uint32_t>(head + (v + j * THREADS) * N);
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (!(f[e] < thr_v) && !(f[e] == thr_v && i0 + e > thr_i)) mask |= 1u << (j * N + e);
        }
      }
      mask &= among;
    };
    if (lane < queued) {
      v = sm.queue[warp][lane];
      filter(0xFFFFFFFFu);
    }
    while (__any_sync(0xffffffffu, mask != 0)) {
      Key k = 0;                              // the lane's next candidate
      if (mask) {
        const int b = __ffs(static_cast<int>(mask)) - 1;
        const int i = head + (v + b / N * THREADS) * N + b % N;
        k = make_key(E::load(x + i), static_cast<uint32_t>(i));
        mask &= mask - 1;
      }
      seen = thr;
      append(k > thr, k);
      if (thr != seen && mask) filter(mask);  // a flush has raised the threshold (long ties)
    }
    const int rest = sm.queue[warp][32 + lane];
    __syncwarp();
    sm.queue[warp][lane] = rest;
    queued = max(queued - 32, 0);
    __syncwarp();
  };

  if (rank == 0 && warp == 0) {
    const int nscal = head + p.V - tail0;
    const int idx = lane < head ? lane : tail0 + lane - head;
    const bool on = lane < nscal;
    float v = 0.f;
    if (on) {
      v = E::load(x + idx);
      st.m = v;
      st.s = v == -INFINITY ? 0.f : (isinf(v) ? NAN : v - v + 1.f);   // NaN for NaN and +inf
      const float mu = __fmul_rn(v, c);
      if (fabsf(mu) < ORDINARY) {                                    // d = fma(v, c, -mu): mu's rounding
        const float d = fmaf(v, c, -mu);
        st.s = ex2(d);
        st.t = d * st.s;
      }
    }
    if (TOPK) append(on && v != -INFINITY, make_key(v, idx));
  }

  for (int base = v0, s = 0; base < v1; base += TILE, s ^= 1) {
    uint4 q[VECS];
    int have = VECS;                          // of this thread's vectors, the first so many
    float bm = -INFINITY;
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    const uint4* own = &sm.stage[s][threadIdx.x];
    if (base + TILE <= v1) {
#pragma unroll
      for (int j = 0; j < VECS; ++j) q[j] = own[j * THREADS];
      uint32_t w = vmax<T>(q[0]);
#pragma unroll
      for (int j = 1; j < VECS; ++j) w = E::wmax(w, vmax<T>(q[j]));
      bm = E::wvalue(w);
    } else {
      have = 0;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        if (base + j * THREADS + static_cast<int>(threadIdx.x) < v1) {
          q[j] = own[j * THREADS];
          bm = max_nan(bm, E::wvalue(vmax<T>(q[j])));
          have = j + 1;
        }
      }
    }
    fetch(base + STAGES * TILE, s);           // the slot's vectors are in registers
    // running softmax statistics
    if (!(bm <= st.m)) {                      // grows, or NaN
      if (st.s > 0.f) {
        // from the old reference to the new one (bm > st.m here, or NaN)
        const float D = max_nan(exact_distance(st.m, bm, p.by) + (reference_delta(bm, c) - reference_delta(st.m, c)), FAR);
        const float f = ex2(D);
        st.t = f * fmaf(st.s, D, st.t);
        st.s *= f;
      }
      st.m = max_nan(st.m, bm);               // NaN stays
    }
    const float mu = __fmul_rn(st.m, c);
    // Nothing below `low` counts: masked logits are finite from here on.  Rounded
    // down, so it stays below the maximum however coarse the steps there are.
    uint32_t low;
    if (E::floor_word(__fadd_rd(st.m, FAR / c), low) && fabsf(mu) < ORDINARY) {
      const uint64_t nm2 = f2_pack(-mu, -mu), c2 = f2_pack(c, c);
      uint64_t s2 = f2_pack(st.s, 0.f), t2 = f2_pack(st.t, 0.f);
      auto add = [&](const uint4& v) {
        float f[N];
        E::unpack(make_uint4(E::clamp(v.x, low), E::clamp(v.y, low), E::clamp(v.z, low), E::clamp(v.w, low)), f);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const uint64_t d2 = f2_fma(f2_pack(f[e], f[e + 1]), c2, nm2);
          const uint64_t e2 = f2_pack(ex2(f2_lo(d2)), ex2(f2_hi(d2)));
          s2 = f2_add(s2, e2);
          t2 = f2_fma(d2, e2, t2);
        }
      };
      if (have == VECS) {
#pragma unroll
        for (int j = 0; j < VECS; ++j) add(q[j]);
      } else {
#pragma unroll 1
        for (int j = 0; j < have; ++j) add(j == 0 ? q[0] : j == 1 ? q[1] : q[2]);
      }
      st.s = f2_lo(s2) + f2_hi(s2);
      st.t = f2_lo(t2) + f2_hi(t2);
    } else if (st.m != -INFINITY) {
      // a maximum out of the ordinary (or infinite, or NaN): exact differences
#pragma unroll 1
      for (int j = 0; j < have; ++j) {
        const uint4 v = j == 0 ? q[0] : j == 1 ? q[1] : j == 2 ? q[2] : q[3];
        float f[N];
        E::unpack(v, f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float d =
              max_nan(fabsf(mu) < ORDINARY ? fmaf(f[e], c, -mu) : exact_distance(f[e], st.m, p.by), FAR);
          const float w = ex2(d);
          st.s += w;
          st.t = fmaf(d, w, st.t);
        }
      }
    }

    if constexpr (TOPK) {
      if (++tile == refresh) {
        refresh *= 4;
        uint32_t o = warp_sort(ordered(st.m), lane);
        sm.vals[warp][lane] = o;
#pragma unroll
        for (int w = WARPS / 2; w > 0; w >>= 1) {
          __syncthreads();
          if (warp < w) {
            o = warp_merge(o, sm.vals[warp + w][lane], lane);
            sm.vals[warp][lane] = o;
          }
        }
        __syncthreads();
        bound = (static_cast<Key>(sm.vals[0][p.k - 1]) << 32) - 1;
        raise(bound);
        __syncthreads();
      }
      const int v = base + static_cast<int>(threadIdx.x);
      auto holds = [&]() {
        return have && !(bm < thr_v) && !(bm == thr_v && static_cast<uint32_t>(head + v * N) > thr_i);
      };
      uint32_t hit = __ballot_sync(0xffffffffu, holds());
      if (__popc(hit) > CROWD) {
        raise(*static_cast<volatile Key*>(&sm.thr));      // any earlier value is a bound too
        const uint32_t kth = __shfl_sync(0xffffffffu, warp_sort(have ? ordered(bm) : 0u, lane), p.k - 1);
        if (kth) raise((static_cast<Key>(kth) << 32) - 1);
        hit = __ballot_sync(0xffffffffu, holds());
      }
      if (hit) {
        if (hit >> lane & 1u) sm.queue[warp][queued + __popc(hit & ((1u << lane) - 1u))] = v;
        queued += __popc(hit);
        if (queued >= 32) process();
      }
    }
  }
  if (TOPK && queued > 0) process();

  // this CTA's statistics, fixed order; from here on the reference is the maximum itself
  const float delta = reference_delta(st.m, c), back = ex2(-delta);
  st.t = back * fmaf(st.s, -delta, st.t);
  st.s *= back;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat b;
    b.m = __shfl_down_sync(0xffffffffu, st.m, o);
    b.s = __shfl_down_sync(0xffffffffu, st.s, o);
    b.t = __shfl_down_sync(0xffffffffu, st.t, o);
    st = merge_stat(st, b, p.by);
  }
  if (lane == 0) sm.wstat[warp] = st;
  __syncthreads();                            // every thread is done with its vectors
  if constexpr (TOPK) {
    // the pool: this warp's buffer and list, as far as all warps' bounds leave them
    const Key cut = max(sm.thr, bound + 1);
    const Key kept = lane < pending ? sm.buf[warp][lane] : 0;
    const uint32_t buf = __ballot_sync(0xffffffffu, kept >= cut && kept != 0);
    const uint32_t list = __ballot_sync(0xffffffffu, best >= cut && best != 0);
    int at = 0;
    if (lane == 0) at = atomicAdd(&sm.pooled, __popc(buf) + __popc(list));
    at = __shfl_sync(0xffffffffu, at, 0);
    const uint32_t before = (1u << lane) - 1u;
    if (buf >> lane & 1u) sm.pool[at + __popc(buf & before)] = kept;
    if (list >> lane & 1u) sm.pool[at + __popc(buf) + __popc(list & before)] = best;
    if (threadIdx.x < 32) sm.top[threadIdx.x] = 0;
    __syncthreads();
    select_top(sm, sm.pooled, p.k);
  }
  if (threadIdx.x == 0) {
    Stat a = sm.wstat[0];
    for (int w = 1; w < WARPS; ++w) a = merge_stat(a, sm.wstat[w], p.by);
    sm.stat = a;
  }
  if (THREADS == MAX_THREADS && p.C > 1) {    // warp w serves rank w
    cluster_sync_all();
    if (rank == 0) {
      // warp w fetches rank w's results
      if (warp > 0 && warp < p.C && lane == 0) {
        const uint32_t sa = dsmem_addr(&sm.stat, warp);
        sm.wstat[warp].m = dsmem_ld_f32(sa);
        sm.wstat[warp].s = dsmem_ld_f32(sa + 4);
        sm.wstat[warp].t = dsmem_ld_f32(sa + 8);
      }
      if (TOPK && warp < p.C && lane < p.k)
        sm.pool[warp * p.k + lane] = dsmem_ld_u64(dsmem_addr(&sm.top[lane], warp));
      __syncthreads();
      if constexpr (TOPK) select_top(sm, p.C * p.k, p.k);
      if (threadIdx.x == 0) {
        Stat a = sm.stat;
        for (int r = 1; r < p.C; ++r) a = merge_stat(a, sm.wstat[r], p.by);
        sm.stat = a;
      }
    }
    cluster_sync_all();          // peers stay until rank 0 has read them
  } else {
    __syncthreads();
  }
  if (rank != 0 || warp != 0) return;

  if constexpr (TOPK) {
    int found = __popc(__ballot_sync(0xffffffffu, lane < p.k && sm.top[lane] != 0));
    for (int i0 = 0; found < p.k && i0 < p.V; i0 += 32) {
      const int i = i0 + lane;
      const bool on = i < p.V && E::load(x + i) == -INFINITY;
      const uint32_t b = __ballot_sync(0xffffffffu, on);
      const int at = found + __popc(b & ((1u << lane) - 1u));
      if (on && at < p.k) sm.top[at] = make_key(-INFINITY, static_cast<uint32_t>(i));
      found += __popc(b);
    }
    __syncwarp();
  }
  const Stat a = sm.stat;
  const float zmax = a.m * p.scale;
  const bool empty = zmax == -INFINITY;      // the mask leaves nothing
  const float ls = logf(a.s);
  if (TOPK && lane < p.k) {
    const Key k = sm.top[lane];
    p.top_ids[row * p.k + lane] = key_index(k);
    p.top_logprobs[row * p.k + lane] = empty ? -INFINITY : difference(key_value(k), a.m, p.by) - ls;
  }
  if (lane == 0) {
    if (p.lse) p.lse[row] = empty ? -INFINITY : zmax + ls;
    if (p.entropy) {
      const float h = ls - a.t / a.s * LN2;
      p.entropy[row] = empty || h < 0.f ? 0.f : h;
    }
    if (p.logprob) {
      const int t = p.targets[row];
      float v = 0.f;                         // no token
      if (t >= p.V) v = NAN;                 // nothing is read out of range
      else if (t >= 0) v = empty ? -INFINITY : difference(E::load(x + t), a.m, p.by) - ls;
      p.logprob[row] = v;
    }
  }
}

template <typename T>
cudaError_t launch_fwd(const LogprobArgs& a) {
  Params p;
  p.logits = a.logits;
  p.ld = a.ld;
  p.V = static_cast<int>(a.V);
  p.k = a.top_k;
  p.targets = a.targets;
  p.scale = a.scale;
  p.by.half = a.scale < 1.f ? 0.5f : 1.f;
  p.by.rest = a.scale / p.by.half;
  p.logprob = a.logprob;
  p.entropy = a.entropy;
  p.lse = a.lse;
  p.top_ids = a.top_ids;
  p.top_logprobs = a.top_logprobs;
  // CTAs per row: as many as keep every CTA at least one full tile and the
  // grid within two waves of the 4 CTAs an SM holds
  constexpr int64_t LOGITS = static_cast<int64_t>(MAX_THREADS) * VECS * Elem<T>::N;
  int C = 1;
  while (C < 8 && a.M * C * 2 <= 8LL * a.num_sms && a.V >= LOGITS * C * 2) C *= 2;
  p.C = C;
  const unsigned grid = static_cast<unsigned>(a.M * C);
  // CTAs of 4 warps where the rows alone fill the SMs: what a warp does per row
  // apart from its logits (thresholds, survivors, sums) is then done half as often
  if (C == 1 && a.M * 2 > 8LL * a.num_sms)
    return a.top_k > 0 ? launch_pdl(logprobs_kernel<T, true, 128>, grid, 128, 0, a.stream, p)
                       : launch_pdl(logprobs_kernel<T, false, 128>, grid, 128, 0, a.stream, p);
  if (a.top_k > 0) {
    return C > 1 ? launch_pdl_cluster(logprobs_kernel<T, true, MAX_THREADS>, grid, C, MAX_THREADS, 0, a.stream, p)
                 : launch_pdl(logprobs_kernel<T, true, MAX_THREADS>, grid, MAX_THREADS, 0, a.stream, p);
  }
  return C > 1 ? launch_pdl_cluster(logprobs_kernel<T, false, MAX_THREADS>, grid, C, MAX_THREADS, 0, a.stream, p)
               : launch_pdl(logprobs_kernel<T, false, MAX_THREADS>, grid, MAX_THREADS, 0, a.stream, p);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// dlogits_v = scale * (gl (1[v = target] - p_v) - gh p_v (log p_v + H)) with
// p_v = e^{z_v - lse}: one read and one write of the row, bound by HBM.  A
// thread reads and writes the same elements, so the gradient may overwrite
// the logits.
// 8 vectors a thread and blocks of 128: 2048 x 131072 bf16 in 172 us (6.2 TB/s)
// at 1965 MHz, 183 in a long run under the power cap; 4, 12 and 16 vectors took
// 187, 186 and 200 us with blocks of 256.
//
// lse comes rounded to fp32, so log p is off by half a step of lse, and p by a
// relative |lse| 2^-24.  Where |lse| is in the millions no digit of p is left (a
// row filled throughout with -1e9 would get p = 1 for each logit, the most that a
// mask can do wrong).  So from |lse| = FAR_LSE on the row's first block takes the
// maximum and the sum again and does the whole row alone, since the gradient may
// overwrite the logits: 0.27 ms where one row of 2048 is such a row, 0.92 where all
// are.
constexpr int THREADS = 128;
constexpr int BWD_VECS = 8;

constexpr float FAR_LSE = 1024.f;            // p off by 2^-14 at most below it

struct BwdParams {
  const void* logits;
  void* dlogits;
  int64_t ld, ldd;
  int V, chunks;
  const int* targets;
  const float *lse, *entropy, *gl, *gh;
  float scale;
};

template <bool FAST>
__device__ __forceinline__ float grad_of(float x, float scale, float lse, float gl, float gh, float H) {
  const float lp = fmaf(x, scale, -lse);
  const float pv = FAST ? ex2(lp * LOG2E) : expf(lp);
  // masked: p = 0 and log p = -inf, no gradient
  return pv == 0.f ? 0.f : -scale * pv * fmaf(gh, lp + H, gl);
}

// A whole row by one block, from its own maximum and sum.
template <typename T>
__device__ __noinline__ void far_row(const T* x, T* dx, int V, int t, float scale, float gl, float gh, float H) {
  using E = Elem<T>;
  __shared__ float ms[THREADS / 32][2];
  // running maximum and sum of e^(z - max z); masked logits add nothing
  float m = -INFINITY, s = 0.f;
  auto merge = [&](float om, float os) {
    const float hi = fmaxf(m, om);
    if (hi == -INFINITY) return;
    s = s * expf((m - hi) * scale) + os * expf((om - hi) * scale);
    m = hi;
  };
  constexpr int BATCH = 8;                    // loads in flight
  for (int64_t i0 = threadIdx.x; i0 < V; i0 += THREADS * BATCH) {
    float v[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) v[j] = i0 + j * THREADS < V ? E::load(x + i0 + j * THREADS) : -INFINITY;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) merge(v[j], 1.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_down_sync(0xffffffffu, m, o), os = __shfl_down_sync(0xffffffffu, s, o);
    merge(om, os);
  }
  if ((threadIdx.x & 31) == 0) {
    ms[threadIdx.x >> 5][0] = m;
    ms[threadIdx.x >> 5][1] = s;
  }
  __syncthreads();                            // also: the row has been read before it is written
  m = ms[0][0];
  s = ms[0][1];
  for (int w = 1; w < THREADS / 32; ++w) merge(ms[w][0], ms[w][1]);
  const float ls = logf(s), hot = gl * scale;
  for (int64_t i0 = threadIdx.x; i0 < V; i0 += THREADS * BATCH) {
    float v[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) v[j] = i0 + j * THREADS < V ? E::load(x + i0 + j * THREADS) : -INFINITY;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int64_t i = i0 + j * THREADS;
      const float lp = (v[j] - m) * scale - ls;
      const float pv = expf(lp);
      float g = pv == 0.f ? 0.f : -scale * pv * fmaf(gh, lp + H, gl);
      if (i == t) g += hot;
      if (i < V) dx[i] = E::from(g);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) logprobs_bwd_kernel(const BwdParams p) {
  using E = Elem<T>;
  constexpr int N = E::N;
  constexpr bool FAST = sizeof(T) == 2;      // the result is rounded to 8 or 11 bits anyway
  const int64_t row = blockIdx.x / p.chunks;
  const int chunk = static_cast<int>(blockIdx.x % p.chunks);
  grid_dependency_wait();
  grid_launch_dependents();
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  T* dx = static_cast<T*>(p.dlogits) + row * p.ldd;
  const int t = p.gl ? __ldg(p.targets + row) : -1;
  const float gl = t < 0 ? 0.f : t >= p.V ? NAN : __ldg(p.gl + row);
  const float gh = p.gh ? __ldg(p.gh + row) : 0.f;
  const float H = p.gh ? __ldg(p.entropy + row) : 0.f;
  const float lse = __ldg(p.lse + row);
  const float hot = gl * p.scale;
  const bool empty = lse == -INFINITY;
  const bool far = !empty && fabsf(lse) >= FAR_LSE;      // then nothing is stored before far_row
  const int lo = static_cast<int>(static_cast<int64_t>(p.V) * chunk / p.chunks);
  const int hi = static_cast<int>(static_cast<int64_t>(p.V) * (chunk + 1) / p.chunks);
  auto one = [&](int i) {
    float g = empty ? 0.f : grad_of<FAST>(E::load(x + i), p.scale, lse, gl, gh, H);
    if (i == t && !empty) g += hot;
    dx[i] = E::from(g);
  };
  // N gradients from a vector whose first logit is i
  auto vec = [&](const uint4& q, int i) {
    float f[N];
    E::unpack(q, f);
    const int rel = t - i;                     // the target's place in this vector
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float g = grad_of<FAST>(f[e], p.scale, lse, gl, gh, H);
      if (rel == e) g += hot;
      f[e] = empty ? 0.f : g;
    }
    return E::pack(f);
  };
  const uintptr_t ax = reinterpret_cast<uintptr_t>(x + lo), ad = reinterpret_cast<uintptr_t>(dx + lo);
  if (((ax ^ ad) & 15u) != 0) {
    if (far) {
      if (chunk == 0) far_row<T>(x, dx, p.V, t, p.scale, gl, gh, H);
      return;
    }
    // The rows lie differently to 16-byte boundaries: whole vectors of the
    // gradient, each from the two vectors of logits that it straddles (the
    // second comes from L1), as far as both lie within this block's logits.
    const int misd = static_cast<int>((ad & 15u) / sizeof(T));
    int b = lo + (misd ? N - misd : 0);                                   // dx + b is aligned
    const int m = static_cast<int>((reinterpret_cast<uintptr_t>(x + b) & 15u) / sizeof(T));
    if (b - m < lo) b += N;                                               // x + b - m is aligned
    const int nv = b - m + 2 * N <= hi ? (hi - (b - m)) / N - 1 : 0;
    for (int i = lo + static_cast<int>(threadIdx.x); i < min(b, hi); i += THREADS) one(i);
    for (int i = b + nv * N + static_cast<int>(threadIdx.x); i < hi; i += THREADS) one(i);
    const uint4* xv = reinterpret_cast<const uint4*>(x + b - m);
    uint4* dv = reinterpret_cast<uint4*>(dx + b);
    const int words = m * static_cast<int>(sizeof(T)) / 4;                // 0..3, and half a word
    const bool half = (m * sizeof(T)) % 4 != 0;
    constexpr int BATCH = 4;
    for (int base = static_cast<int>(threadIdx.x); base < nv; base += THREADS * BATCH) {
      uint4 q[BATCH][2];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int k = min(base + j * THREADS, nv - 1);
        q[j][0] = __ldg(xv + k);
        q[j][1] = __ldg(xv + k + 1);
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int k = base + j * THREADS;
        if (k < nv) {
          uint32_t w[8] = {q[j][0].x, q[j][0].y, q[j][0].z, q[j][0].w, q[j][1].x, q[j][1].y, q[j][1].z, q[j][1].w};
          if (words & 2)
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
          if (words & 1)
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
          if (half)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
          __stcs(dv + k, vec(make_uint4(w[0], w[1], w[2], w[3]), b + k * N));
        }
      }
    }
    return;
  }
  const int mis = static_cast<int>((ax & 15u) / sizeof(T));
  const int b = min(lo + (mis ? N - mis : 0), hi);
  const int nv = (hi - b) / N;
  const int e0 = b + nv * N;
  const uint4* xv = reinterpret_cast<const uint4*>(x + b);
  uint4* dv = reinterpret_cast<uint4*>(dx + b);
  for (int base = 0; base == 0 || base < nv; base += THREADS * BWD_VECS) {
    uint4 q[BWD_VECS];
#pragma unroll
    for (int j = 0; j < BWD_VECS; ++j) {
      const int i = base + j * THREADS + static_cast<int>(threadIdx.x);
      if (i < nv) q[j] = __ldcs(xv + i);
    }
    if (base == 0) {                           // behind the loads, which then do not wait for lse
      if (far) {
        if (chunk == 0) far_row<T>(x, dx, p.V, t, p.scale, gl, gh, H);
        return;
      }
      if (lo + static_cast<int>(threadIdx.x) < b) one(lo + static_cast<int>(threadIdx.x));
      if (e0 + static_cast<int>(threadIdx.x) < hi) one(e0 + static_cast<int>(threadIdx.x));
    }
#pragma unroll
    for (int j = 0; j < BWD_VECS; ++j) {
      const int i = base + j * THREADS + static_cast<int>(threadIdx.x);
      if (i < nv) __stcs(dv + i, vec(q[j], b + i * N));
    }
  }
}

template <typename T>
cudaError_t launch_bwd(const LogprobBwdArgs& a) {
  BwdParams p;
  p.logits = a.logits;
  p.dlogits = a.dlogits;
  p.ld = a.ld;
  p.ldd = a.ldd;
  p.V = static_cast<int>(a.V);
  constexpr int64_t CHUNK = static_cast<int64_t>(THREADS) * BWD_VECS * Elem<T>::N;
  p.chunks = static_cast<int>((a.V + CHUNK - 1) / CHUNK);
  p.targets = a.targets;
  p.lse = a.lse;
  p.entropy = a.entropy;
  p.gl = a.grad_logprob;
  p.gh = a.grad_entropy;
  p.scale = a.scale;
  return launch_pdl(logprobs_bwd_kernel<T>, static_cast<unsigned>(a.M * p.chunks), THREADS, 0, a.stream, p);
}

}  // namespace lp

int64_t logprobs_bwd_blocks(int64_t M, int64_t V, int elem_bytes) {
  const int64_t tile = static_cast<int64_t>(lp::THREADS) * lp::BWD_VECS * (16 / elem_bytes);
  return M * ((V + tile - 1) / tile);
}

cudaError_t launch_logprobs(const LogprobArgs& a) {
  if (a.type == 0) return lp::launch_fwd<__nv_bfloat16>(a);
  if (a.type == 1) return lp::launch_fwd<__half>(a);
  return lp::launch_fwd<float>(a);
}

cudaError_t launch_logprobs_bwd(const LogprobBwdArgs& a) {
  if (a.type == 0) return lp::launch_bwd<__nv_bfloat16>(a);
  if (a.type == 1) return lp::launch_bwd<__half>(a);
  return lp::launch_bwd<float>(a);
}

}  // namespace fn
