// Device helpers shared by the attention kernels.
#pragma once

#include "fp8_util.h"

namespace wq {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

typedef float float16v_t __attribute__((ext_vector_type(16)));

// Division of numbers below 2^31 by one that the host knows: n / d is
// (n + n * mul / 2^32) >> shift with 2^shift >= d the smallest such power.
struct Divisor {
  uint32_t d, mul, shift;
  static Divisor of(uint32_t d) {
    uint32_t s = 0;
    while ((1u << s) < d) ++s;
    return Divisor{d, (uint32_t)((((uint64_t)1 << 32) * ((1u << s) - d)) / d + 1), s};
  }
  __device__ __forceinline__ int quotient(int n) const {
    return (int)(((uint32_t)n + __umulhi((uint32_t)n, mul)) >> shift);
  }
};

// What a row at `pos` sees of its sequence: the tokens [0, first) and [from, pos],
// `n` in all; visible token i is token i for i < first, else i - first + from.
struct Visible {
  int first, from, n;
};
__device__ __forceinline__ Visible visible_of(int pos, int window, int sinks) {
  Visible v;
  v.from = pos >= window ? pos - window + 1 : 0;
  v.first = min(sinks, v.from);
  v.n = pos < 0 ? 0 : pos + 1 - v.from + v.first;
  return v;
}

// tokens of a sequence: its entry of lens within what its row of the page table holds
__device__ __forceinline__ int tokens_of(const AttentionCall& a, int len) {
  const int64_t room = a.max_pages << a.cache.lg_page;
  return (int)min((int64_t)max(len, 0), room);
}

// p[i] with an i that is the same in every lane, as a scalar load: a vector load would
// wait behind all loads in flight
__device__ __forceinline__ int scalar_at(const int32_t* p, int i) {
  using C = const __attribute__((address_space(4))) int32_t*;
  return ((C)(uintptr_t)p)[__builtin_amdgcn_readfirstlane(i)];
}

__device__ __forceinline__ int page_of(const AttentionCall& a, const int32_t* table, int token) {
  return min(max(table[token >> a.cache.lg_page], 0), a.cache.pages - 1);
}

// The kernel's arguments of type A, read where they are used: those that only a piece's
// start or end needs would otherwise take scalar registers all along, more than there are.
template <typename A>
using ArgsAt = const __attribute__((address_space(4))) A*;
template <typename A>
__device__ __forceinline__ ArgsAt<A> args_here() {
  auto p = (ArgsAt<A>)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// two weights rounded to nearest even into one word (low half first)
template <int T>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  const float2v_t v = {lo, hi};
  if constexpr (T == WQ_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2v_t));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2_t));
}

template <int T>
__device__ __forceinline__ float4_t mfma16(uint4_t a, uint4_t b, float4_t c) {
  if constexpr (T == WQ_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// four E4M3 codes -> four 16-bit values (exact)
template <int T>
__device__ __forceinline__ uint2_t widen4(uint32_t w) {
  uint2_t r;
  if constexpr (T == WQ_BF16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
  }
  return r;
}

// a value of this lane and of the lanes 16, 32 and 48 away
__device__ __forceinline__ float max_quarters(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_quarters(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The reference of exponents: the running maximum, or 0 where nothing counted yet
// (all z so far are -inf, and exp2 of them stays 0).
__device__ __forceinline__ float exp_ref(float m) { return m == -INFINITY ? 0.0f : m; }

// Counts of the sequences 0 .. m-1, each known to `count(i)`, in a line.  Up to 64
// sequences every wave scans them by itself, one in a lane; more go through LDS
// (kLineWords), a block of consecutive ones per thread.  The workgroup has NT threads.
struct Line {
  int total;                           // of all sequences
  int mine;                            // before this lane's sequence (up to 64)
};

__device__ __forceinline__ int scan64(int v) {           // inclusive, over the wave
  const int lane = (int)__lane_id();
#pragma unroll
  for (int w = 1; w < 64; w *= 2) {
    const int up = __shfl_up(v, w);
    if (lane >= w) v += up;
  }
  return v;
}

template <int NT, typename F>
__device__ __forceinline__ Line line_up(int m, int* part, F count) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (m <= 64) {
    const int own = lane < m ? count(min(lane, m - 1)) : 0;
    const int sum = scan64(own);
    return Line{__builtin_amdgcn_readlane(sum, m - 1), sum - own};
  }
  const int per = (m + NT - 1) / NT, i0 = tid * per, i1 = min(i0 + per, m);
  int own = 0;
  for (int i = i0; i < i1; ++i) own += count(i);
  const int sum = scan64(own);
  if (lane == 63) part[NT + wave] = sum;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    if (w < wave) base += part[NT + w];
    total += part[NT + w];
  }
  part[tid] = base + sum - own;
  __syncthreads();
  return Line{total, 0};
}

// the sequence that holds place `want` (below the total), and the places before it
template <int NT, typename F>
__device__ __forceinline__ int line_find(int m, const Line& line, const int* part, int want,
                                         int& before, F count) {
  if (m == 1) {
    before = 0;
    return 0;
  }
  if (m <= 64) {
    // the last one that starts at or before it: empty ones share their start with the
    // next, and those past the end start at the total
    const int lane = (int)__lane_id();
    const int seq = 63 - __builtin_clzll(__ballot(lane < m && line.mine <= want));
    before = __builtin_amdgcn_readlane(line.mine, seq);
    return seq;
  }
  int t = 0;                           // the same among the blocks
#pragma unroll
  for (int w = NT / 2; w > 0; w /= 2)
    if (part[t + w] <= want) t += w;
  const int per = (m + NT - 1) / NT;
  int seq = t * per;
  before = part[t];
  if (per == 1) return seq;            // without its count, one load less in the chain
  for (;;) {
    const int n = count(seq);
    if (before + n > want || seq + 1 >= m) return seq;
    before += n;
    ++seq;
  }
}
template <int NT>
constexpr int kLineWords = NT + NT / 64;

}  // namespace wq
