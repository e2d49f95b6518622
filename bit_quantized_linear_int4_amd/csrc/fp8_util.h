// Device helpers shared by the FP8 and mixture-of-experts kernels: 16-bit
// vector access, E4M3 scales and conversions, reductions inside a wave.
#pragma once

#include <atomic>

#include "internal.h"

namespace wq {

constexpr int kF8Block = 128;      // elements that share an FP8 scale
constexpr float kF8Max = 448.0f;   // largest finite E4M3 value

typedef float float2v_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v_t __attribute__((ext_vector_type(2)));
typedef unsigned int uint2_t __attribute__((ext_vector_type(2)));
typedef int int8v_t __attribute__((ext_vector_type(8)));

// the two 16-bit values of a word (low half first) as fp32
template <int DT>
__device__ __forceinline__ void unpack2(uint32_t u, float& lo, float& hi) {
  if constexpr (DT == WQ_BF16) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xFFFF0000u);
  } else {
    half2_t h;
    __builtin_memcpy(&h, &u, 4);
    lo = (float)h.x;
    hi = (float)h.y;
  }
}
template <int DT>
__device__ __forceinline__ void unpack8(uint4_t raw, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2<DT>(raw[i], v[2 * i], v[2 * i + 1]);
}

// two fp32 values rounded to nearest even into one word (low half = lo);
// unlike the integer rounding of f32_to_bf16_bits a NaN stays a NaN
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const float2v_t v = {as_f32(lo), as_f32(hi)};
  uint32_t u;
  if constexpr (DT == WQ_BF16) {
    const bf16x2v_t b = __builtin_convertvector(v, bf16x2v_t);
    __builtin_memcpy(&u, &b, 4);
  } else {
    const half2_t h = __builtin_convertvector(v, half2_t);
    __builtin_memcpy(&u, &h, 4);
  }
  return u;
}
template <int DT>
__device__ __forceinline__ uint4_t pack8(const float (&v)[8]) {
  uint4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
  return o;
}

// four fp32 values -> four E4M3 bytes (nearest even)
__device__ __forceinline__ uint32_t pack4_fp8(float a, float b, float c, float d) {
  int o = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, o, true);
}

// The scale of a block whose largest magnitude has the fp32 bits `bits`
// (sign cleared): amax / 448, 1 for a block of zeros, and never below the
// smallest normal fp32 value, so that 1 / s stays finite and |v| / s at most
// 448 (and a rounding).  The bits of an infinity or a NaN compare above every
// finite magnitude, so a block that holds one gets that as its scale, and what is
// read back from it is not finite either.
// The quotient is that of an fp32 division: a product with 1 / 448 and its
// residual; a / 448 is never within a fourteenth of a step of a midpoint.
__device__ __forceinline__ float fp8_scale(uint32_t bits) {
  const float a = __uint_as_float(bits);
  constexpr float kInv = 1.0f / kF8Max, kTiny = 0x1p-126f;
  const float q = a * kInv;
  const float s = bits < 0x7F800000u ? fmaf(fmaf(-q, kF8Max, a), kInv, q) : a;
  if (s < kTiny) return a == 0.0f ? 1.0f : kTiny;
  return s;
}

// Codes of v / s, rounded as an fp32 division rounds it, with one reciprocal for a
// whole block: q = v * (1 / s) gains its residual v - q * s times 1 / s, which
// leaves at most 2^-21 of an fp32 step.  A code could then change only next to one
// of its midpoints, for scales within 13 steps of a 4-bit value, and for those the
// reciprocal's own residual is enough (q alone changes one code in about a
// million).  A small scale and its values are scaled up together, so that no
// residual is subnormal; the residual's sign is taken such that a zero keeps its
// own.  An infinite scale gives 0 for finite values, a NaN one NaN.
// Against q alone: norm of 8192 rows of 8192 85.1 us either way, 1 row of 4096
// 2.49 and 2.44, gated rows 2048 of 14336 28.9 either way.
__device__ __forceinline__ uint2_t fp8_codes(float s, const float (&v)[8]) {
  float a[8], q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = v[i];
  if (s < 0x1p-64f) {
    s *= 0x1p64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= 0x1p64f;
  }
  const float d = __float_as_uint(s) == 0x7F800000u ? 0.0f : s;
  float inv = __builtin_amdgcn_rcpf(s);                  // within one step
  inv = fmaf(fmaf(-d, inv, 1.0f), inv, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = a[i] * inv;
    q[i] = fmaf(-fmaf(q[i], d, -a[i]), inv, q[i]);
  }
  return uint2_t{pack4_fp8(q[0], q[1], q[2], q[3]), pack4_fp8(q[4], q[5], q[6], q[7])};
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// *(T*)(base + off) with a base that is the same in every lane.  The empty asm
// holds the base in scalar registers and the offset in one 32-bit register
// until here, so the load takes the form with a scalar base and a lane offset;
// left to itself the compiler keeps a 64-bit address per lane and load in
// vector registers across a loop.
template <typename T>
__device__ __forceinline__ T load_at(const void* base, uint32_t off) {
  uint64_t b = reinterpret_cast<uint64_t>(base);
  asm("" : "+s"(b), "+v"(off));
  using G = const __attribute__((address_space(1))) char*;
  return *(const __attribute__((address_space(1))) T*)((G)b + off);
}

// MFMA operands want lane 16 kq + nl to hold piece kq of row nl, but a load
// whose adjacent lanes are on different lines takes 64 cycles to address
// instead of 16 (a 16-byte load, four adjacent lanes on 64 contiguous bytes).
// So rows are loaded with a row's four pieces in adjacent lanes, 4 nl + kq, and
// this moves them: what lane 4 nl + kq holds, to lane 16 kq + nl.
__device__ __forceinline__ uint4_t operand_order(uint4_t v) {
  const int lane = (int)__lane_id(), from = ((lane & 15) * 4 + (lane >> 4)) * 4;
  uint4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[i]);
  return r;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// largest value over each 16 lanes of a wave, in all of them (lane xor 1, xor
// 2, then mirrored halves and rows)
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  v = max(v, dpp<0x140>(v));
  return v;
}
// sum over each 16 lanes of a wave, in all of them
__device__ __forceinline__ float sum16(float v) {
  v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x140>(__float_as_uint(v)));
  return v;
}
// sum over the wave, in every lane (uniform)
__device__ __forceinline__ float sum64(float v) {
  const int s = __float_as_int(sum16(v));
  return (__int_as_float(__builtin_amdgcn_readlane(s, 0)) +
          __int_as_float(__builtin_amdgcn_readlane(s, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(s, 32)) +
          __int_as_float(__builtin_amdgcn_readlane(s, 48)));
}

// Lets `kern` take `bytes` of dynamic LDS on the current device, once per device
// and kernel (`done`: a bit per device).
inline hipError_t allow_lds(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if ((done.load(std::memory_order_acquire) & bit) != 0) return hipSuccess;
  e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// v / (1 + exp(-v)) with the hardware exponential and reciprocal; exp overflow
// gives the limit 0.  The exponent v * log2(e) is rounded to fp32, which costs up to
// |v| * 2^-24 of the value where v is negative: 1e-6 at -16 (57 * 2^-24 at most down
// to -80), where an E4M3 or a 16-bit rounding of the result, 2^-4 to 2^-12 of it,
// follows in every use.  With the exponent's rest added, good to 10 * 2^-24, the
// gated packer, which the vector units bound as much as HBM does, takes 29.9 us
// instead of 28.1 for 2048 rows of 14336 and 6.3 instead of 5.7 for 300.
__device__ __forceinline__ float silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

}  // namespace wq
