// Mixture-of-experts layer for a few tokens (at most 64):
//   l = x Wr^T, p = softmax(l), the top_k largest (ties to the lowest index),
//   y = sum_j p_j W_down[e_j] (silu(W_gate[e_j] x) * (W_up[e_j] x))
// with INT4 (scale and zero point per group of 128, 64 or 32) or FP8 (scale
// per 128 x 128 block) experts and 16-bit activations.
//
// Bound by HBM: every touched expert's codes are read once, and each launch is
// laid out around that stream.
//   1. router     one wave per expert and four tokens.
//   2. gate/up    every workgroup first finds the top_k of all tokens itself
//                 (a few hundred logits: cheaper than one more launch), then
//                 walks units of 16 gate rows and the same 16 up rows of one
//                 expert; its waves split k.  It stores
//                 a = round16(p * silu(g) * u) for every token of the expert.
//                 The first workgroup also leaves the table of active experts.
//   3. down       a workgroup owns 16 rows of y over all active experts, whose
//                 columns form one long k that its waves split; nothing leaves
//                 the workgroup but y, and the order of the sum is fixed.
//
// The multiply runs on v_mfma_f32_16x16x32 with up to 16 tokens as the A
// operand and 16 weight rows as the B operand.  INT4 codes are not rounded to
// 16-bit weights: OR-ing a code into the top mantissa bits of 16.0 gives
// exactly 16 + q in fp16 and in bf16, the MFMA sums x * (16 + q) over a
// group, and s * (that - (16 + z) * sum x) is added in fp32, sum x being an
// MFMA against ones.  FP8 codes are exact in either 16-bit type.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8_util.h"

namespace wq {
namespace {

constexpr int kMaxE = kMoeMaxExperts, kMaxT = kMoeMaxTokens, kMaxK = kMoeMaxTopK;

// an expert some token is routed to
struct Active {
  uint64_t tokens;    // bit t: token t
  int32_t expert;
  int32_t slot;       // its first row of the intermediate, one row per token
};

struct MoeArgs {
  const uint16_t* x;         // [t][h]
  const uint16_t* router;    // [e][h]
  float* logits;             // [t][e]
  const void *gate, *gate_s, *up, *up_s, *down, *down_s;
  const uint8_t *gate_z, *up_z, *down_z;
  Active* table;             // [min(e, t * top_k)], after the int32 count
  int32_t* count;
  uint16_t* mid;             // [t * top_k][i]
  void* y;                   // [t][h]
  int32_t* ids;              // [t][top_k] or nullptr
  float* probs;              // [t][top_k] or nullptr
  int t, e, top_k, h, i, renorm, ydt;
};

template <int XDT>
__device__ __forceinline__ float4_t mfma16(uint4_t a, uint4_t b, float4_t c) {
  if constexpr (XDT == WQ_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// ------------------------------------------------------------------ router
constexpr int kRouterTok = 4;

template <int XDT>
__global__ __launch_bounds__(256) void moe_router_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63;
  const int e = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int t0 = (int)blockIdx.y * kRouterTok;
  if (e >= a.e) return;
  float acc[kRouterTok] = {};
  const uint16_t* const wr = a.router + (int64_t)e * a.h;
#pragma unroll 4
  for (int c = lane * 8; c < a.h; c += 512) {
    float w[8];
    unpack8<XDT>(*reinterpret_cast<const uint4_t*>(wr + c), w);
#pragma unroll
    for (int j = 0; j < kRouterTok; ++j) {
      const int t = min(t0 + j, a.t - 1);
      float v[8];
      unpack8<XDT>(*reinterpret_cast<const uint4_t*>(a.x + (int64_t)t * a.h + c), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j] = fmaf(w[i], v[i], acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRouterTok; ++j) {
    const float s = sum64(acc[j]);
    if (lane == 0 && t0 + j < a.t) a.logits[(int64_t)(t0 + j) * a.e + e] = s;
  }
}

// ----------------------------------------------------------------- routing
__device__ __forceinline__ uint32_t max64(uint32_t v) {
  const int s = (int)max16(v);
  return max(max((uint32_t)__builtin_amdgcn_readlane(s, 0), (uint32_t)__builtin_amdgcn_readlane(s, 16)),
             max((uint32_t)__builtin_amdgcn_readlane(s, 32), (uint32_t)__builtin_amdgcn_readlane(s, 48)));
}

// fp32 -> uint32 in the same order; NaN above everything, never 0, and -0
// equal to 0
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

struct Routing {
  uint32_t mask[kMaxE][2];            // tokens of an expert
  int32_t ids[kMaxT * kMaxK];
  float probs[kMaxT * kMaxK];
  float slot_prob[kMaxT * kMaxK];     // by row of the intermediate
  uint8_t slot_tok[kMaxT * kMaxK];
  int32_t slot_of[kMaxE];
  Active act[kMaxE];
  int32_t count;
};

// The top_k of one token by one wave: lane j < top_k gets choice j.  A masked
// expert (logit -inf) has probability 0 and comes last; with every expert
// masked all probabilities are 0.  A NaN or +inf logit makes the token's
// probabilities NaN; the ids stay valid.
template <int R>
__device__ __forceinline__ void top_k_of(const float* l, int e, int top_k, int renorm, int lane,
                                         int& id, float& prob) {
  uint32_t key[R];
  uint32_t best = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = lane + 64 * r;
    key[r] = j < e ? order_key(l[j]) : 0u;
    best = max(best, key[r]);
  }
  best = max64(best);
  const float top = best == 0xFFFFFFFFu ? __builtin_nanf("") : order_value(best);
  float sum = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (key[r] != 0) sum += __expf(order_value(key[r]) - top);
  sum = sum64(sum);
  id = 0;
  prob = 0.0f;
  for (int k = 0; k < top_k; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) m = max(m, key[r]);
    m = max64(m);
    // lowest index among the largest: the largest of 0xFFFF - index
    uint32_t at = 0;
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
      if (key[r] == m) at = 0xFFFFu - (uint32_t)(lane + 64 * r);
    const int j = 0xFFFF - (int)max64(at);
    if (lane == k) {
      id = j;
      prob = __expf(order_value(m) - top);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (j == lane + 64 * r) key[r] = 0;
  }
  const float total = renorm ? sum64(lane < top_k ? prob : 0.0f) : sum;
  // top is -inf only when every expert is masked
  prob = __float_as_uint(top) == 0xFF800000u ? 0.0f : __fdiv_rn(prob, total);
}

// Fills `r` for all tokens; every thread of the workgroup calls it.
template <int NW>
__device__ void route(const MoeArgs& a, Routing& r) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < a.e; i += NW * 64) r.mask[i][0] = r.mask[i][1] = 0;
  for (int t = wave; t < a.t; t += NW) {
    int id;
    float p;
    const float* l = a.logits + (int64_t)t * a.e;
    if (a.e <= 64) top_k_of<1>(l, a.e, a.top_k, a.renorm, lane, id, p);
    else if (a.e <= 256) top_k_of<4>(l, a.e, a.top_k, a.renorm, lane, id, p);
    else top_k_of<kMaxE / 64>(l, a.e, a.top_k, a.renorm, lane, id, p);
    if (lane < a.top_k) {
      r.ids[t * a.top_k + lane] = id;
      r.probs[t * a.top_k + lane] = p;
    }
  }
  __syncthreads();
  const int picks = a.t * a.top_k;
  for (int i = tid; i < picks; i += NW * 64) {
    const int t = i / a.top_k;
    // a probability of 0 adds nothing to y: such a choice is not computed
    if (r.probs[i] != 0.0f) atomicOr(&r.mask[r.ids[i]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  if (wave == 0) {
    int na = 0, slot = 0;
    for (int e0 = 0; e0 < a.e; e0 += 64) {
      const int e = e0 + lane;
      const uint64_t m = e < a.e ? ((uint64_t)r.mask[e][1] << 32) | r.mask[e][0] : 0;
      const int cnt = __popcll(m);
      int run = cnt;                      // inclusive sum over the lanes
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(run, o);
        if (lane >= o) run += v;
      }
      const uint64_t on = __ballot(m != 0);
      if (m != 0) {
        const int at = na + __popcll(on & ((1ull << lane) - 1));
        r.act[at] = Active{m, e, slot + run - cnt};
        r.slot_of[e] = slot + run - cnt;
      }
      na += __popcll(on);
      slot += __shfl(run, 63);
    }
    if (lane == 0) r.count = na;
  }
  __syncthreads();
  for (int i = tid; i < picks; i += NW * 64) {
    const int t = i / a.top_k, e = r.ids[i];
    if (r.probs[i] != 0.0f) {
      const uint64_t m = ((uint64_t)r.mask[e][1] << 32) | r.mask[e][0];
      const int s = r.slot_of[e] + __popcll(m & ((1ull << t) - 1));
      r.slot_prob[s] = r.probs[i];
      r.slot_tok[s] = (uint8_t)t;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------ weight units
// One unit: 16 rows x 128 values of k of one matrix, in the lane layout of
// the B operand: lane (row nl, quarter kq).
//   INT4 (S groups per unit): 16 bytes = codes [32 kq, 32 kq + 32) of the row.
//   FP8: bytes [16 kq, +16) and [64 + 16 kq, +16).
template <int FMT>
struct Unit {
  uint4_t c[FMT == WQ_FMT_FP8_BLOCK ? 2 : 1];
  uint32_t s[2];       // INT4: S fp16 scales; FP8: s[0] = the fp32 scale
  uint32_t z;          // INT4: S zero points, 4 bits each
};

template <int FMT, int S>
__device__ __forceinline__ Unit<FMT> load_unit(const void* codes, const void* scales,
                                               const uint8_t* zeros, int64_t row, int k, int u,
                                               int kq) {
  Unit<FMT> w;
  const int ku = k >> 7;
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) {
    const uint8_t* p = static_cast<const uint8_t*>(codes) + row * k + u * 128 + kq * 16;
    w.c[0] = *reinterpret_cast<const uint4_t*>(p);
    w.c[1] = *reinterpret_cast<const uint4_t*>(p + 64);
    w.s[0] = static_cast<const uint32_t*>(scales)[(row >> 7) * ku + u];
    w.s[1] = 0;
    w.z = 0;
  } else {
    w.c[0] = *reinterpret_cast<const uint4_t*>(static_cast<const uint8_t*>(codes) +
                                               row * (k >> 1) + u * 64 + kq * 16);
    const uint16_t* sp = static_cast<const uint16_t*>(scales) + row * (ku * S) + u * S;
    const uint8_t* zp = zeros + row * ((ku * S + 1) >> 1) + ((u * S) >> 1);
    w.s[1] = 0;
    if constexpr (S == 1) {
      w.s[0] = *sp;
      w.z = (u & 1) ? (uint32_t)*zp >> 4 : (uint32_t)*zp & 15u;
    } else if constexpr (S == 2) {
      w.s[0] = *reinterpret_cast<const uint32_t*>(sp);
      w.z = *zp;
    } else {
      w.s[0] = reinterpret_cast<const uint32_t*>(sp)[0];
      w.s[1] = reinterpret_cast<const uint32_t*>(sp)[1];
      w.z = (uint32_t)zp[0] | ((uint32_t)zp[1] << 8);
    }
  }
  return w;
}

// first value of k (within the unit) that operand f of lane quarter kq holds
template <int FMT, int S>
__device__ __forceinline__ int unit_k(int f, int kq) {
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) return 64 * (f >> 1) + 16 * kq + 8 * (f & 1);
  else if constexpr (S == 1) return 32 * kq + 8 * f;
  else return 32 * f + 8 * kq;       // operand f covers 32 consecutive values
}

// (x0..x7) -> (x0,x4),(x1,x5),(x2,x6),(x3,x7), the order the code unpack gives
__device__ __forceinline__ uint4_t pair_order(uint4_t d) {
  uint4_t r;
  r[0] = __builtin_amdgcn_perm(d[2], d[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(d[2], d[0], 0x07060302u);
  r[2] = __builtin_amdgcn_perm(d[3], d[1], 0x05040100u);
  r[3] = __builtin_amdgcn_perm(d[3], d[1], 0x07060302u);
  return r;
}

// 8 codes -> 16 + q in pairs (q0,q4),(q1,q5),(q2,q6),(q3,q7): the code lands
// in the top four mantissa bits of 16.0 (fp16: bits 6-9, bf16: bits 3-6)
template <int XDT>
__device__ __forceinline__ uint4_t unpack_codes(uint32_t w) {
  uint4_t r;
  if constexpr (XDT == WQ_BF16) {
    constexpr uint32_t kM = 0x00780078u, kB = 0x41804180u;
    r[0] = ((w << 3) & kM) | kB;
    r[1] = ((w >> 1) & kM) | kB;
    r[2] = ((w >> 5) & kM) | kB;
    r[3] = ((w >> 9) & kM) | kB;
  } else {
    constexpr uint32_t kM = 0x03C003C0u, kB = 0x4C004C00u;
    r[0] = ((w << 6) & kM) | kB;
    r[1] = ((w << 2) & kM) | kB;
    r[2] = ((w >> 2) & kM) | kB;
    r[3] = ((w >> 6) & kM) | kB;
  }
  return r;
}

// 8 E4M3 bytes -> 8 values of the activation type
template <int XDT>
__device__ __forceinline__ uint4_t unpack_fp8(uint32_t lo, uint32_t hi) {
  uint4_t r;
  const uint32_t w[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (XDT == WQ_BF16) {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[i], 1.0f, false);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[i], 1.0f, true);
      r[2 * i] = __builtin_bit_cast(uint32_t, a);
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, b);
    } else {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i], 1.0f, false);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i], 1.0f, true);
      r[2 * i] = __builtin_bit_cast(uint32_t, a);
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, b);
    }
  }
  return r;
}

// 4 x 4 transpose of 32-bit words over the four lane quarters: word j of
// quarter q becomes word q of quarter j
__device__ __forceinline__ uint4_t quarter_transpose(uint4_t v) {
  // quarters 0,1 <-> 2,3 for words (0,2) and (1,3), then 0 <-> 1 and 2 <-> 3
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return uint4_t{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
}

// The activations of one unit as A operands, and (INT4) their sums per group
template <int FMT, int S>
struct Acts {
  uint4_t f[4];
  float4_t sum[FMT == WQ_FMT_FP8_BLOCK ? 1 : S];
};

template <int XDT, int FMT, int S>
__device__ __forceinline__ void prepare_acts(Acts<FMT, S>& x) {
  if constexpr (FMT != WQ_FMT_FP8_BLOCK) {
    constexpr uint32_t kOne = XDT == WQ_BF16 ? 0x3F803F80u : 0x3C003C00u;
    const uint4_t ones = {kOne, kOne, kOne, kOne};
#pragma unroll
    for (int g = 0; g < S; ++g) {
      x.sum[g] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int f = g * 4 / S; f < (g + 1) * 4 / S; ++f) {
        x.f[f] = pair_order(x.f[f]);
        x.sum[g] = mfma16<XDT>(x.f[f], ones, x.sum[g]);
      }
    }
  }
}

// acc += x . w^T over one unit
template <int XDT, int FMT, int S>
__device__ __forceinline__ void unit_mac(const Unit<FMT>& w, const Acts<FMT, S>& x, float4_t& acc) {
  const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) {
    float4_t c = zero;
#pragma unroll
    for (int f = 0; f < 4; ++f)
      c = mfma16<XDT>(x.f[f], unpack_fp8<XDT>(w.c[f >> 1][2 * (f & 1)], w.c[f >> 1][2 * (f & 1) + 1]), c);
    const float s = __uint_as_float(w.s[0]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(c[e], s, acc[e]);
  } else {
    const uint4_t q = S == 1 ? w.c[0] : quarter_transpose(w.c[0]);
#pragma unroll
    for (int g = 0; g < S; ++g) {
      float4_t c = zero;
#pragma unroll
      for (int f = g * 4 / S; f < (g + 1) * 4 / S; ++f)
        c = mfma16<XDT>(x.f[f], unpack_codes<XDT>(q[f]), c);
      const float s = f16_bits_to_f32((uint16_t)(w.s[g >> 1] >> (16 * (g & 1))));
      const float z = 16.0f + (float)((w.z >> (4 * g)) & 15u);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(s, fmaf(-z, x.sum[g][e], c[e]), acc[e]);
    }
  }
}

// ----------------------------------------------------------------- gate/up
template <int XDT, int FMT, int S, int NW>
__global__ __launch_bounds__(NW * 64) void moe_gate_up_kernel(MoeArgs a) {
  __shared__ Routing r;
  __shared__ float4_t red[2][NW][64];
  route<NW>(a, r);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int nact = __builtin_amdgcn_readfirstlane(r.count);
  if (blockIdx.x == 0) {
    for (int i = tid; i < nact; i += NW * 64) a.table[i] = r.act[i];
    if (tid == 0) *a.count = nact;
    for (int i = tid; i < a.t * a.top_k; i += NW * 64) {
      if (a.ids != nullptr) a.ids[i] = r.ids[i];
      if (a.probs != nullptr) a.probs[i] = r.probs[i];
    }
  }
  const int tiles = a.i >> 4, units = nact * tiles, ku = a.h >> 7;
  const int per = (units + (int)gridDim.x - 1) / (int)gridDim.x;
  const int u0 = (int)blockIdx.x * per, u1 = min(u0 + per, units);
  for (int un = u0; un < u1; ++un) {
    const int ai = un / tiles, tile = un - ai * tiles;
    const int expert = __builtin_amdgcn_readfirstlane(r.act[ai].expert);
    const int slot = __builtin_amdgcn_readfirstlane(r.act[ai].slot);
    const int cnt = __builtin_amdgcn_readfirstlane(__popcll(r.act[ai].tokens));
    const int64_t row = (int64_t)expert * a.i + tile * 16 + nl;
    for (int c0 = 0; c0 < cnt; c0 += 16) {
      const bool on = c0 + nl < cnt;
      const uint16_t* const xr =
          a.x + (int64_t)(on ? r.slot_tok[slot + c0 + nl] : 0) * a.h;
      float4_t ga = {0, 0, 0, 0}, ua = {0, 0, 0, 0};
      for (int u = wave; u < ku; u += NW) {
        const Unit<FMT> gw = load_unit<FMT, S>(a.gate, a.gate_s, a.gate_z, row, a.h, u, kq);
        const Unit<FMT> uw = load_unit<FMT, S>(a.up, a.up_s, a.up_z, row, a.h, u, kq);
        Acts<FMT, S> x;
#pragma unroll
        for (int f = 0; f < 4; ++f)
          x.f[f] = on ? *reinterpret_cast<const uint4_t*>(xr + u * 128 + unit_k<FMT, S>(f, kq))
                      : uint4_t{0, 0, 0, 0};
        prepare_acts<XDT, FMT, S>(x);
        unit_mac<XDT, FMT, S>(gw, x, ga);
        unit_mac<XDT, FMT, S>(uw, x, ua);
      }
      red[0][wave][lane] = ga;
      red[1][wave][lane] = ua;
      __syncthreads();
      // value (token j, row n) of the tile sits in lane 16 (j / 4) + n, element j % 4
      if (tid < 256) {
        const int j = tid >> 4, n = tid & 15, l = (j >> 2) * 16 + n, e = j & 3;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          g += red[0][w][l][e];
          u += red[1][w][l][e];
        }
        if (c0 + j < cnt) {
          const int s = slot + c0 + j;
          a.mid[(int64_t)s * a.i + tile * 16 + n] =
              (uint16_t)pack2<XDT>(silu(g) * u * r.slot_prob[s], 0.0f);
        }
      }
      __syncthreads();
    }
  }
}

// -------------------------------------------------------------------- down
template <int XDT, int FMT, int S, int NW, int TC>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(MoeArgs a) {
  extern __shared__ uint4_t dsm[];
  Active* const act = reinterpret_cast<Active*>(dsm);                    // [kMaxE]
  float4_t* const red = reinterpret_cast<float4_t*>(act + kMaxE);        // [NW][TC][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int nact = *a.count;
  for (int i = tid; i < nact; i += NW * 64) act[i] = a.table[i];
  __syncthreads();
  const int ku = a.i >> 7, steps = nact * ku, n0 = (int)blockIdx.x * 16;
  float4_t acc[TC];
#pragma unroll
  for (int c = 0; c < TC; ++c) acc[c] = float4_t{0, 0, 0, 0};
  for (int st = wave; st < steps; st += NW) {
    const int ai = st / ku, u = st - ai * ku;
    const Active ac = act[ai];
    const int64_t row = (int64_t)ac.expert * a.h + n0 + nl;
    const Unit<FMT> w = load_unit<FMT, S>(a.down, a.down_s, a.down_z, row, a.i, u, kq);
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      if (((ac.tokens >> (16 * c)) & 0xFFFFu) == 0) continue;
      const int t = 16 * c + nl;
      const bool on = (ac.tokens >> t) & 1;
      const int s = ac.slot + __popcll(ac.tokens & ((1ull << t) - 1));
      Acts<FMT, S> x;
#pragma unroll
      for (int f = 0; f < 4; ++f)
        x.f[f] = on ? *reinterpret_cast<const uint4_t*>(a.mid + (int64_t)s * a.i + u * 128 +
                                                        unit_k<FMT, S>(f, kq))
                    : uint4_t{0, 0, 0, 0};
      prepare_acts<XDT, FMT, S>(x);
      unit_mac<XDT, FMT, S>(w, x, acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < TC; ++c) red[(wave * TC + c) * 64 + lane] = acc[c];
  __syncthreads();
  for (int i = tid; i < TC * 256; i += NW * 64) {
    const int c = i >> 8, j = (i >> 4) & 15, n = i & 15, l = (j >> 2) * 16 + n, e = j & 3;
    const int t = 16 * c + j;
    if (t >= a.t) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[(w * TC + c) * 64 + l][e];
    const int64_t o = (int64_t)t * a.h + n0 + n;
    if (a.ydt == WQ_F32) static_cast<float*>(a.y)[o] = v;
    else if (a.ydt == WQ_BF16) static_cast<uint16_t*>(a.y)[o] = (uint16_t)pack2<WQ_BF16>(v, 0.0f);
    else static_cast<uint16_t*>(a.y)[o] = (uint16_t)pack2<WQ_F16>(v, 0.0f);
  }
}

// ------------------------------------------------------------------ launch
template <int XDT, int FMT, int S, int TC>
hipError_t down_tc(const MoeArgs& a, hipStream_t s) {
  constexpr int NW = 8;
  constexpr int bytes = kMaxE * (int)sizeof(Active) + NW * TC * 1024;
  moe_down_kernel<XDT, FMT, S, NW, TC><<<dim3((unsigned)(a.h / 16)), NW * 64, bytes, s>>>(a);
  return hipGetLastError();
}

template <int XDT, int FMT, int S>
hipError_t moe_fmt(const MoeArgs& a, hipStream_t s) {
  constexpr int NW = 8;
  if (a.router != nullptr) {
    const dim3 grid((unsigned)((a.e + 3) / 4), (unsigned)((a.t + kRouterTok - 1) / kRouterTok));
    moe_router_kernel<XDT><<<grid, 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t units = (int64_t)std::min(a.e, a.t * a.top_k) * (a.i / 16);
  const unsigned grid = (unsigned)std::min<int64_t>(units, 512);
  moe_gate_up_kernel<XDT, FMT, S, NW><<<dim3(grid), NW * 64, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.t <= 16) return down_tc<XDT, FMT, S, 1>(a, s);
  if (a.t <= 32) return down_tc<XDT, FMT, S, 2>(a, s);
  return down_tc<XDT, FMT, S, 4>(a, s);
}

template <int XDT>
hipError_t moe_xdt(const MoeArgs& a, int fmt, int group, hipStream_t s) {
  if (fmt == WQ_FMT_FP8_BLOCK) return moe_fmt<XDT, WQ_FMT_FP8_BLOCK, 1>(a, s);
  if (group == 128) return moe_fmt<XDT, WQ_FMT_INT4_ASYM, 1>(a, s);
  if (group == 64) return moe_fmt<XDT, WQ_FMT_INT4_ASYM, 2>(a, s);
  return moe_fmt<XDT, WQ_FMT_INT4_ASYM, 4>(a, s);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

// workspace: logits fp32 [t][e] | count | table | intermediate [t * top_k][i]
size_t moe_ws_bytes(int64_t t, int64_t e, int64_t top_k, int64_t i) {
  return up256((size_t)(t * e) * 4) + 256 + up256(kMaxE * sizeof(Active)) +
         up256((size_t)(t * top_k * i) * 2);
}

hipError_t launch_moe(const MoeCall& c, hipStream_t s) {
  MoeArgs a{};
  a.x = c.x;
  a.router = c.router;
  a.gate = c.gate->codes; a.gate_s = c.gate->scales; a.gate_z = c.gate->zeros;
  a.up = c.up->codes; a.up_s = c.up->scales; a.up_z = c.up->zeros;
  a.down = c.down->codes; a.down_s = c.down->scales; a.down_z = c.down->zeros;
  char* p = static_cast<char*>(c.workspace);
  a.logits = c.router != nullptr ? reinterpret_cast<float*>(p) : const_cast<float*>(c.logits);
  p += up256((size_t)(c.t * c.e) * 4);
  a.count = reinterpret_cast<int32_t*>(p);
  p += 256;
  a.table = reinterpret_cast<Active*>(p);
  p += up256(kMaxE * sizeof(Active));
  a.mid = reinterpret_cast<uint16_t*>(p);
  a.y = c.y;
  a.ids = c.ids;
  a.probs = c.probs;
  a.t = (int)c.t; a.e = (int)c.e; a.top_k = c.top_k; a.h = (int)c.h; a.i = (int)c.i;
  a.renorm = c.renorm; a.ydt = c.ydt;
  return c.xdt == WQ_BF16 ? moe_xdt<WQ_BF16>(a, c.gate->fmt, c.gate->group, s)
                          : moe_xdt<WQ_F16>(a, c.gate->fmt, c.gate->group, s);
}

}  // namespace wq
