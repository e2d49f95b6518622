// Mixture-of-experts layer for a few tokens (at most 64):
//   l = x Wr^T, p = softmax(l), the top_k largest (ties to the lowest index),
//   y = sum_j p_j W_down[e_j] (silu(W_gate[e_j] x) * (W_up[e_j] x))
// with INT4 (scale and zero point per group of 128, 64 or 32) or FP8 (scale
// per 128 x 128 block) experts and 16-bit activations.
//
// Bound by HBM: every touched expert's codes are read once, and each launch is
// laid out around that stream.
//   1. router     16 experts x 16 tokens per workgroup.
//   2. gate/up    every workgroup first finds the top_k of all tokens itself
//                 (a few hundred logits: cheaper than one more launch), then
//                 walks units of 16 gate rows and the same 16 up rows of one
//                 expert; its waves split k.  It stores
//                 a = round16(silu(g) * u) for every token of the expert.
//   3. down       a workgroup owns 16 or 32 rows of y over all active experts,
//                 whose columns form one long k that its waves, and with more
//                 than a few choices several workgroups, split; the order of
//                 the sum is fixed.  Parts of k are added by a fourth launch.
// The first workgroup of 2 leaves the routing (experts, rows, tokens, their p)
// for 3, which multiplies an expert's sums by p in fp32: a share of one in
// several hundred experts, multiplied in before the rounding to fp16, would
// push a among the subnormals and cost most of its bits.
//
// One MI355X, us: one token, 8 of 64 INT4 experts of 2048 x 1024 18.5 (25 MB, 5
// at the rate of a copy; three dependent launches); 24 tokens, 6 of 64 FP8 82
// (365 MB, 70); 64 tokens, 2 of 8 INT4 of 4096 x 14336 243 to 249 (735 MB, 142).
// The last: an expert with more than 16 tokens is read and unpacked twice.  In 2.
// its codes come from L2 the second time (495 MB fetched for 488), and a step (a
// tile, 16 tokens) takes the 3 us that its loads, one step ahead, need.  In 3. the
// two chunks of an expert are far apart in k, and both come from HBM (379 MB
// fetched for 244).  Groups of 128, 64 and 32: one token 18.5, 19.3, 21.9; 24
// tokens, 6 of 64 61.9, 63.7, 71.0; 64 tokens, 2 of 8 245, 259, 296.
//
// a is kept in the activations' type, which the matrix instructions of 3. take:
// with y in the same type the error of y is the square root of two times that of
// y's rounding alone (bf16 2.3e-3 against 1.7e-3); in two parts a would double 3.'s
// products.
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
  int32_t expert;
  int32_t slot;       // its first row of the intermediate, one row per token
  int32_t cnt;        // its tokens
  int32_t chunk;      // pieces of 16 tokens of the experts before it
};
constexpr int kMaxChunks = kMaxE + kMaxT * kMaxK / 16;
// at most 16 tokens of one expert
struct Chunk {
  int32_t expert, slot, cnt;
};

struct MoeArgs {
  const uint16_t* x;         // [t][h]
  const uint16_t* router;    // [e][h]
  float* logits;             // [t][e]
  const void *gate, *gate_s, *up, *up_s, *down, *down_s;
  const uint8_t *gate_z, *up_z, *down_z;
  int32_t* count;            // of chunks
  Chunk* table;
  uint8_t* slot_tok;         // [t * top_k] token of a row of the intermediate
  float* slot_prob;          // [t * top_k] and its p
  uint16_t* mid;             // [t * top_k][i]
  float* part;               // [parts][t][h]
  void* y;                   // [t][h]
  int32_t* ids;              // [t][top_k] or nullptr
  float* probs;              // [t][top_k] or nullptr
  int t, e, top_k, h, i, renorm, ydt;
};

__device__ __forceinline__ void store_as(void* y, int dt, int64_t i, float v) {
  if (dt == WQ_F32) static_cast<float*>(y)[i] = v;
  else if (dt == WQ_BF16) static_cast<uint16_t*>(y)[i] = (uint16_t)pack2<WQ_BF16>(v, 0.0f);
  else static_cast<uint16_t*>(y)[i] = (uint16_t)pack2<WQ_F16>(v, 0.0f);
}

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
// logits of 16 experts x 16 tokens per workgroup, k split over 16 waves (exact
// products, fp32 sums).  Bound by latency: every load of a wave is issued
// before its first use for h up to 4096 (one memory round trip), with one wave
// per expert and four tokens it was a chain of them (24 tokens, 64 experts,
// h = 2048: 9.9 against 4.6 us; one token 5.4 against 3.8).
template <int XDT>
__global__ __launch_bounds__(1024) void moe_router_kernel(MoeArgs a) {
  constexpr int NW = 16;
  __shared__ float4_t red[NW][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int e0 = (int)blockIdx.x * 16, t0 = (int)blockIdx.y * 16;
  // four adjacent lanes load 64 bytes of a row; see operand_order()
  const int row = lane >> 2, piece = (lane & 3) * 8;
  const uint16_t* const wr = a.router + (int64_t)min(e0 + row, a.e - 1) * a.h + piece;
  const uint16_t* const xr = a.x + (int64_t)min(t0 + row, a.t - 1) * a.h + piece;
  float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int u = wave; u < a.h >> 7; u += 2 * NW) {
    const int v = min(u + NW, (a.h >> 7) - 1);
    uint4_t w[2][4], x[2][4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      w[0][f] = *reinterpret_cast<const uint4_t*>(wr + u * 128 + f * 32);
      x[0][f] = *reinterpret_cast<const uint4_t*>(xr + u * 128 + f * 32);
      w[1][f] = *reinterpret_cast<const uint4_t*>(wr + v * 128 + f * 32);
      x[1][f] = *reinterpret_cast<const uint4_t*>(xr + v * 128 + f * 32);
    }
#pragma unroll
    for (int f = 0; f < 4; ++f)
      acc = mfma16<XDT>(operand_order(x[0][f]), operand_order(w[0][f]), acc);
    if (u + NW < a.h >> 7) {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        acc = mfma16<XDT>(operand_order(x[1][f]), operand_order(w[1][f]), acc);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    // value (token j, expert n) sits in lane 16 (j / 4) + n, element j % 4
    const int j = threadIdx.x >> 4, n = threadIdx.x & 15, l = (j >> 2) * 16 + n;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][l][j & 3];
    if (t0 + j < a.t && e0 + n < a.e) a.logits[(int64_t)(t0 + j) * a.e + e0 + n] = v;
  }
}

// ----------------------------------------------------------------- routing
__device__ __forceinline__ uint32_t max64(uint32_t v) {
  const int s = (int)max16(v);
  return max(max((uint32_t)__builtin_amdgcn_readlane(s, 0),
                 (uint32_t)__builtin_amdgcn_readlane(s, 16)),
             max((uint32_t)__builtin_amdgcn_readlane(s, 32),
                 (uint32_t)__builtin_amdgcn_readlane(s, 48)));
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
  uint16_t act_of[kMaxChunks];        // the active expert of a chunk
  int32_t count, chunks;
};

// The top_k of one token by one wave: lane j < top_k gets choice j.  A masked
// expert (logit -inf) has probability 0 and comes last; with every expert
// masked all probabilities are 0.  A NaN or +inf logit makes the token's
// probabilities NaN; the ids stay valid.
// Lane l holds logits l, l + 64, ...
template <int R>
__device__ __forceinline__ void top_k_of(const float (&l)[R], int e, int top_k, int renorm,
                                         int lane, int& id, float& prob) {
  uint32_t key[R];
  uint32_t best = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    key[r] = lane + 64 * r < e ? order_key(l[r]) : 0u;
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
  uint32_t mine = 0;                   // the key of this lane's choice
  for (int k = 0; k < top_k; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) m = max(m, key[r]);
    m = max64(m);
    int j = 0;                         // the lowest index among the largest
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const uint64_t on = __ballot(key[r] == m);
      if (on != 0) j = 64 * r + __builtin_ctzll(on);
    }
    if (lane == k) {
      id = j;
      mine = m;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (j == lane + 64 * r) key[r] = 0;
  }
  prob = lane < top_k ? __expf(order_value(mine) - top) : 0.0f;
  const float total = renorm ? sum64(prob) : sum;
  // top is -inf only when every expert is masked
  prob = __float_as_uint(top) == 0xFF800000u ? 0.0f : __fdiv_rn(prob, total);
}

// The top_k of tokens wave, wave + NW, ... into `r`, the next one's logits loaded
// while one is sorted; lane j gets choice j of the last.
template <int NW, int R>
__device__ __forceinline__ void top_k_all(const MoeArgs& a, Routing& r, int wave, int lane,
                                          int& id, float& p) {
  auto load = [&](int t, float (&l)[R]) {
    const float* const row = a.logits + (int64_t)min(t, a.t - 1) * a.e;
#pragma unroll
    for (int i = 0; i < R; ++i) l[i] = row[min(lane + 64 * i, a.e - 1)];
  };
  float l[R];
  load(wave, l);
  for (int t = wave; t < a.t; t += NW) {
    float next[R];
    load(t + NW, next);
    top_k_of<R>(l, a.e, a.top_k, a.renorm, lane, id, p);
    if (lane < a.top_k) {
      r.ids[t * a.top_k + lane] = id;
      r.probs[t * a.top_k + lane] = p;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) l[i] = next[i];
  }
}
template <int NW>
__device__ __forceinline__ void top_k_any(const MoeArgs& a, Routing& r, int wave, int lane,
                                          int& id, float& p) {
  if (a.e <= 64) top_k_all<NW, 1>(a, r, wave, lane, id, p);
  else if (a.e <= 256) top_k_all<NW, 4>(a, r, wave, lane, id, p);
  else top_k_all<NW, kMaxE / 64>(a, r, wave, lane, id, p);
}

// Fills `r` for all tokens; every thread of the workgroup calls it.
template <int NW>
__device__ void route(const MoeArgs& a, Routing& r) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (a.t == 1) {
    // one token: each choice is an expert with that token, nothing to sort
    // (one token, 8 of 64 experts: this and the sums cost 3.2 us by the way below)
    if (wave == 0) {
      int id = 0;
      float p = 0.0f;
      top_k_any<NW>(a, r, 0, lane, id, p);
      const bool on = lane < a.top_k && p != 0.0f;
      const uint64_t live = __ballot(on);
      const int at = __popcll(live & ((1ull << lane) - 1));
      if (on) {
        r.act[at] = Active{id, at, 1, at};
        r.act_of[at] = (uint16_t)at;
        r.slot_prob[at] = p;
        r.slot_tok[at] = 0;
      }
      if (lane == 0) r.count = r.chunks = __popcll(live);
    }
    __syncthreads();
    return;
  }
  for (int i = tid; i < a.e; i += NW * 64) r.mask[i][0] = r.mask[i][1] = 0;
  int id;
  float p;
  top_k_any<NW>(a, r, wave, lane, id, p);
  __syncthreads();
  const int picks = a.t * a.top_k;
  for (int i = tid; i < picks; i += NW * 64) {
    const int t = i / a.top_k;
    // a probability of 0 adds nothing to y: such a choice is not computed
    if (r.probs[i] != 0.0f) atomicOr(&r.mask[r.ids[i]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  if (wave == 0) {
    int na = 0, slot = 0, chunk = 0;
    for (int e0 = 0; e0 < a.e; e0 += 64) {
      const int e = e0 + lane;
      const uint64_t m = e < a.e ? ((uint64_t)r.mask[e][1] << 32) | r.mask[e][0] : 0;
      const int cnt = __popcll(m);
      // inclusive sums over the lanes: tokens, and pieces of 16 above bit 16
      const int own = cnt | ((cnt + 15) >> 4) << 16;
      int run = own;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(run, o);
        if (lane >= o) run += v;
      }
      const int before = run - own, all = __shfl(run, 63);
      const uint64_t on = __ballot(m != 0);
      if (m != 0) {
        const int at = na + __popcll(on & ((1ull << lane) - 1));
        r.act[at] = Active{e, slot + (before & 0xFFFF), cnt, chunk + (before >> 16)};
        for (int c = 0; 16 * c < cnt; ++c) r.act_of[chunk + (before >> 16) + c] = (uint16_t)at;
        r.slot_of[e] = slot + (before & 0xFFFF);
      }
      na += __popcll(on);
      slot += all & 0xFFFF;
      chunk += all >> 16;
    }
    if (lane == 0) {
      r.count = na;
      r.chunks = chunk;
    }
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
// One unit: 16 rows x 128 values of k of one matrix.  The B operand wants it
// in lane (row nl, quarter kq):
//   INT4 (S groups per unit): 16 bytes = codes [32 kq, 32 kq + 32) of the row.
//   FP8: bytes [16 kq, +16) and [64 + 16 kq, +16).
// It is loaded with a row's four pieces in adjacent lanes (lane 4 nl + kq), and
// operand_order() moves the pieces to their lanes when they are used; until
// then they are kept as loaded, since arithmetic on a value right after its
// load would make the wave wait for it there.
template <int FMT>
struct Unit {
  uint4_t c[FMT == WQ_FMT_FP8_BLOCK ? 2 : 1];
  uint32_t s;          // FP8: the fp32 scale
};

// One matrix of an expert from a row tile on (uniform).  Every code load is a
// uniform base plus a 32-bit lane offset that never changes.
struct Tile {
  const uint8_t *codes, *scales, *zeros;
};
template <int FMT>
__device__ __forceinline__ uint32_t code_off(int k, int lane) {
  return (uint32_t)((lane >> 2) * (FMT == WQ_FMT_FP8_BLOCK ? k : k >> 1) + (lane & 3) * 16);
}
template <int FMT, int S>
__device__ __forceinline__ Tile tile_at(const void* codes, const void* scales,
                                        const uint8_t* zeros, int64_t row, int k) {
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  const uint8_t* s = static_cast<const uint8_t*>(scales);
  const int64_t g = (k >> 7) * S;
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) return {c + row * k, s + (row >> 7) * g * 4, nullptr};
  else return {c + row * (k >> 1), s + row * g * 2, zeros + row * ((g + 1) >> 1)};
}

template <int FMT>
__device__ __forceinline__ void load_unit(Unit<FMT>& w, const Tile& t, uint32_t off, int u) {
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) {
    w.c[0] = load_at<uint4_t>(t.codes + u * 128, off);
    w.c[1] = load_at<uint4_t>(t.codes + u * 128, off + 64);
    w.s = reinterpret_cast<const uint32_t*>(t.scales)[u];
  } else {
    w.c[0] = load_at<uint4_t>(t.codes + u * 64, off);
  }
}

// INT4: the scale and zero point of one group in one word
__device__ __forceinline__ uint32_t meta_word(uint32_t scale16, uint32_t zero4) {
  return scale16 | zero4 << 16;
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
  // the constants in vector registers, opaque to the compiler: one and-or
  // instruction cannot take two scalar or literal operands
  uint32_t m = XDT == WQ_BF16 ? 0x00780078u : 0x03C003C0u;
  uint32_t b = XDT == WQ_BF16 ? 0x41804180u : 0x4C004C00u;
  asm("" : "+v"(m), "+v"(b));
  uint4_t r;
  if constexpr (XDT == WQ_BF16) {
    r[0] = ((w << 3) & m) | b;
    r[1] = ((w >> 1) & m) | b;
    r[2] = ((w >> 5) & m) | b;
    r[3] = ((w >> 9) & m) | b;
  } else {
    r[0] = ((w << 6) & m) | b;
    r[1] = ((w << 2) & m) | b;
    r[2] = ((w >> 2) & m) | b;
    r[3] = ((w >> 6) & m) | b;
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

// The intermediate is laid out as the down product reads it: the rows of one
// chunk (cnt <= 16 tokens of one expert) together, within them [unit of k]
// [operand f][quarter kq][row][8 values], the 8 values in pair order for INT4.
// One operand load of a wave is then cnt * 64 contiguous bytes, adjacent lanes
// 16 bytes apart (with adjacent lanes on different lines a load takes four
// times as long to address), and needs no reordering.  Element offset of value
// k of row j from the chunk's begin:
template <int FMT, int S>
__device__ __forceinline__ int64_t mid_offset(int k, int j, int cnt) {
  const int q = k & 127, e = k & 7;
  int f, kq;
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) {
    f = 2 * (q >> 6) + ((q >> 3) & 1);
    kq = (q >> 4) & 3;
  } else if constexpr (S == 1) {
    f = (q >> 3) & 3;
    kq = q >> 5;
  } else {
    f = q >> 5;
    kq = (q >> 3) & 3;
  }
  const int at = FMT == WQ_FMT_FP8_BLOCK ? e : (e < 4 ? 2 * e : 2 * e - 7);
  return ((int64_t)((k >> 7) * 16 + f * 4 + kq) * cnt + j) * 8 + at;
}

// The activations of one unit as A operands
struct Acts {
  uint4_t f[4];
};

// acc[i] += x . w[i]^T over one unit of N matrices.  INT4: x in pair order,
// meta[i][g] the word of group g of matrix i.
template <int XDT, int FMT, int S, int N>
__device__ __forceinline__ void unit_mac(const Unit<FMT> (&w)[N], const uint32_t (&meta)[N][S],
                                         const Acts& x, float4_t (&acc)[N]) {
  const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (FMT == WQ_FMT_FP8_BLOCK) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4_t q[2] = {operand_order(w[i].c[0]), operand_order(w[i].c[1])};
      float4_t c = zero;
#pragma unroll
      for (int f = 0; f < 4; ++f)
        c = mfma16<XDT>(x.f[f], unpack_fp8<XDT>(q[f >> 1][2 * (f & 1)],
                                                q[f >> 1][2 * (f & 1) + 1]), c);
      const float s = __uint_as_float(w[i].s);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(c[e], s, acc[i][e]);
    }
  } else {
    constexpr uint32_t kOne = XDT == WQ_BF16 ? 0x3F803F80u : 0x3C003C00u;
    const uint4_t ones = {kOne, kOne, kOne, kOne};
    uint4_t q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[i] = operand_order(w[i].c[0]);
      if constexpr (S > 1) q[i] = quarter_transpose(q[i]);
    }
#pragma unroll
    for (int g = 0; g < S; ++g) {
      float4_t sum = zero, c[N];
#pragma unroll
      for (int i = 0; i < N; ++i) c[i] = zero;
#pragma unroll
      for (int f = g * 4 / S; f < (g + 1) * 4 / S; ++f) {
        sum = mfma16<XDT>(x.f[f], ones, sum);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma16<XDT>(x.f[f], unpack_codes<XDT>(q[i][f]), c[i]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float s = f16_bits_to_f32((uint16_t)meta[i][g]);
        const float z = 16.0f + (float)(meta[i][g] >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(s, fmaf(-z, sum[e], c[i][e]), acc[i][e]);
      }
    }
  }
}

// ----------------------------------------------------------------- gate/up
// The loads of the streams below are never under a branch: after one the
// compiler no longer knows how many loads are in flight and waits for all of
// them.  Positions past the end load the last valid data again, and lanes
// without a token the row of the last one (their results are not used).
//
// `off`: byte offset of the lane's token row from base.
template <int FMT, int S>
__device__ __forceinline__ void load_acts(Acts& x, const uint16_t* base, uint32_t off, int u,
                                          int kq) {
  const char* const p = reinterpret_cast<const char*>(base) + u * 256;
  const uint32_t lo = off + 2 * unit_k<FMT, S>(0, kq);
#pragma unroll
  for (int f = 0; f < 4; ++f)
    x.f[f] = load_at<uint4_t>(p, lo + 2 * (unit_k<FMT, S>(f, 0) - unit_k<FMT, S>(0, 0)));
}

// A workgroup walks tiles of 16 gate rows and the same up rows of one expert
// after the other; its waves split k, two units each (`passes` rounds of that
// where k is longer).  With one pass a wave meets the same values of k in
// every tile, so it keeps the activations of the expert's tokens (up to 16 at a
// time), in pair order, in registers, and the loop streams nothing but codes
// and scales, one tile ahead and also across experts.
//
// The INT4 scales and zero points of a tile come in one load of each per
// thread and group of a unit, and reach the lanes through LDS (two buffers).
// Loaded by every wave for its own two units, two bytes and one byte from each
// of 16 rows, they cost more than the codes: 444 against 300 us with them
// left out, 64 tokens through 2 of 8 experts of 4096 x 14336.
template <int XDT, int FMT, int S, int NW>
__global__ __launch_bounds__(NW * 64, 4) void moe_gate_up_kernel(MoeArgs a, int passes) {
  constexpr bool kInt4 = FMT == WQ_FMT_INT4_ASYM;
  constexpr int GP = NW * 2 * S;       // groups of k per row and pass
  __shared__ Routing r;
  __shared__ float4_t red[2][2][NW][64];
  __shared__ uint32_t meta[kInt4 ? 2 : 1][kInt4 ? 2 * GP * 16 : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4, ku = a.h >> 7;
  Acts x0, x1;                         // of the wave's two units
  auto keep_acts = [&](int u) {        // units past the end of k add nothing
    vm_wait<0>();
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (u >= ku) x0.f[f] = uint4_t{0, 0, 0, 0};
      if (u + 1 >= ku) x1.f[f] = uint4_t{0, 0, 0, 0};
      if constexpr (kInt4) {
        x0.f[f] = pair_order(x0.f[f]);
        x1.f[f] = pair_order(x1.f[f]);
      }
    }
  };
  // one token's activations do not depend on its choices
  const bool one = a.t == 1 && passes == 1;
  if (one) {
    load_acts<FMT, S>(x0, a.x, 0, min(wave * 2, ku - 1), kq);
    load_acts<FMT, S>(x1, a.x, 0, min(wave * 2 + 1, ku - 1), kq);
  }
  route<NW>(a, r);
  if (one) keep_acts(wave * 2);
  const int nact = __builtin_amdgcn_readfirstlane(r.count);
  if (blockIdx.x == 0) {
    for (int i = tid; i < nact; i += NW * 64) {
      const Active ac = r.act[i];
      for (int c = 0; c < ac.cnt; c += 16)
        a.table[ac.chunk + (c >> 4)] = Chunk{ac.expert, ac.slot + c, min(16, ac.cnt - c)};
    }
    if (tid == 0) *a.count = r.chunks;
    for (int i = tid; i < a.t * a.top_k; i += NW * 64) {
      a.slot_tok[i] = r.slot_tok[i];
      a.slot_prob[i] = r.slot_prob[i];
      if (a.ids != nullptr) a.ids[i] = r.ids[i];
      if (a.probs != nullptr) a.probs[i] = r.probs[i];
    }
  }
  // Every workgroup takes as many steps: tiles times chunks (16 tokens of an
  // expert).  The order is expert, block of `per` tiles, chunk, tile, and
  // neighbours in it run on the same XCD: the chunks of one block are about
  // one workgroup each, next to each other, so the codes of a block come from
  // HBM for the first and from that XCD's L2 for the others.
  const int tiles = a.i >> 4, groups = ku * S;
  const int steps = tiles * __builtin_amdgcn_readfirstlane(r.chunks), G = (int)gridDim.x;
  const int per = (steps + G - 1) / G;
  const int xcd = (int)blockIdx.x & 7;
  const int wg = xcd * (G >> 3) + min(xcd, G & 7) + ((int)blockIdx.x >> 3);
  const int st0 = wg * per, st1 = min(st0 + per, steps);
  if (st0 >= st1) return;
  const uint32_t off = code_off<FMT>(a.h, lane);

  struct Pos {
    int64_t row;                       // first gate row of the expert
    int st;                            // step
    int ai, cnt, slot;                 // expert, its tokens and their first row
    int lo, hi, tile, ch;              // block [lo, hi), tile and chunk in it
    int pass;
    int fresh;                         // other activations than the step before
  };
  auto enter = [&](Pos& p) {           // expert p.ai
    const Active ac = r.act[p.ai];
    p.slot = __builtin_amdgcn_readfirstlane(ac.slot);
    p.cnt = __builtin_amdgcn_readfirstlane(ac.cnt);
    p.row = (int64_t)__builtin_amdgcn_readfirstlane(ac.expert) * a.i;
  };
  auto advance = [&](Pos& p) {
    p.fresh = passes > 1;
    if (++p.pass < passes) return;
    p.pass = 0;
    if (++p.st >= st1) {               // stays on the last tile
      --p.tile;
    } else if (p.tile + 1 == p.hi) {
      p.fresh = !one;
      if (16 * ++p.ch >= p.cnt) {
        p.ch = 0;
        p.lo = p.hi;
        if (p.lo == tiles) {
          p.lo = 0;
          ++p.ai;
          enter(p);
        }
        p.hi = min(p.lo + per, tiles);
      }
      p.tile = p.lo - 1;
    }
    ++p.tile;
  };
  auto start = [&]() {                 // at step st0
    Pos p{};
    p.st = st0;
    p.ai = __builtin_amdgcn_readfirstlane((int)r.act_of[st0 / tiles]);
    enter(p);
    const int nch = (p.cnt + 15) >> 4;
    const int in = st0 - __builtin_amdgcn_readfirstlane(r.act[p.ai].chunk) * tiles;
    p.lo = in / (per * nch) * per;
    p.hi = min(p.lo + per, tiles);
    p.ch = (in - p.lo * nch) / (p.hi - p.lo);
    p.tile = p.lo + (in - p.lo * nch) % (p.hi - p.lo);
    p.fresh = !one;
    return p;
  };
  auto unit_of = [&](const Pos& p) { return (p.pass * NW + wave) * 2; };
  auto row_of = [&](const Pos& p) { return p.row + (int64_t)p.tile * 16; };
  // unit u + j of both matrices at position p
  auto load = [&](const Pos& p, int j, Unit<FMT> (&w)[2]) {
    const int u = min(unit_of(p) + j, ku - 1);
    const int64_t row = row_of(p);
    load_unit<FMT>(w[0], tile_at<FMT, S>(a.gate, a.gate_s, a.gate_z, row, a.h), off, u);
    load_unit<FMT>(w[1], tile_at<FMT, S>(a.up, a.up_s, a.up_z, row, a.h), off, u);
  };
  // this thread's share of a tile's 2 x 16 x GP metadata words: words tid +
  // NW * 64 * i in the order [matrix][row][group]
  uint32_t ms[S], mz[S];
  auto load_meta = [&](const Pos& p) {
    const int64_t row = row_of(p);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = tid + NW * 64 * i, mat = e / (16 * GP), rw = (e / GP) & 15;
      const int g = min(p.pass * GP + e % GP, groups - 1);
      const Tile t = mat ? tile_at<FMT, S>(a.up, a.up_s, a.up_z, row, a.h)
                         : tile_at<FMT, S>(a.gate, a.gate_s, a.gate_z, row, a.h);
      ms[i] = *reinterpret_cast<const uint16_t*>(t.scales + (rw * groups + g) * 2);
      mz[i] = t.zeros[rw * ((groups + 1) >> 1) + (g >> 1)];
    }
  };
  auto keep_meta = [&](const Pos& p, int buf) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = tid + NW * 64 * i, mat = e / (16 * GP), rw = (e / GP) & 15;
      const int g = min(p.pass * GP + e % GP, groups - 1);
      meta[buf][(mat * GP + e % GP) * 16 + rw] = meta_word(ms[i], (mz[i] >> (4 * (g & 1))) & 15u);
    }
  };

  float4_t acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  int flip = 0, rflip = 0;
  Pos cur = start();
  // a unit's registers take the next tile's as soon as it is multiplied
  Unit<FMT> w0[2], w1[2];
  if constexpr (kInt4) load_meta(cur);
  // in this order, as the loop waits for them
  load(cur, 0, w0);
  __builtin_amdgcn_sched_barrier(0);
  load(cur, 1, w1);
  if constexpr (kInt4) {
    keep_meta(cur, 0);
    lgkm_wait0();
    wg_barrier();
  }
  auto step = [&](auto more) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value;         // another step follows
    const int u = unit_of(cur);
    Pos nxt = cur;
    if constexpr (MORE) advance(nxt);
    if (cur.fresh) {
      const uint32_t tok = r.slot_tok[cur.slot + min(16 * cur.ch + nl, cur.cnt - 1)];
      const uint32_t xo = tok * (uint32_t)(a.h * 2);
      load_acts<FMT, S>(x0, a.x, xo, min(u, ku - 1), kq);
      load_acts<FMT, S>(x1, a.x, xo, min(u + 1, ku - 1), kq);
      keep_acts(u);
    }
    // the words of unit j of both matrices
    auto read_meta = [&](int j, uint32_t (&m)[2][S]) {
      if constexpr (kInt4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int g = 0; g < S; ++g)
            m[i][g] = meta[flip][(i * GP + (2 * wave + j) * S + g) * 16 + nl];
      }
    };
    if constexpr (kInt4 && MORE) load_meta(nxt);
    uint32_t m[2][S];
    read_meta(0, m);
    // the barriers keep the compiler from unpacking everything at once, which
    // would not fit the registers
    __builtin_amdgcn_sched_barrier(0);
    unit_mac<XDT, FMT, S, 2>(w0, m, x0, acc);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MORE) load(nxt, 0, w0);
    read_meta(1, m);
    __builtin_amdgcn_sched_barrier(0);
    unit_mac<XDT, FMT, S, 2>(w1, m, x1, acc);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MORE) {
      load(nxt, 1, w1);
      if constexpr (kInt4) keep_meta(nxt, flip ^ 1);
    }
    const bool last = cur.pass + 1 == passes;
    // the buffers of the step before are free: every wave has passed the
    // barrier after its last read of them
    if (last) {
      red[rflip][0][wave][lane] = acc[0];
      red[rflip][1][wave][lane] = acc[1];
      acc[0] = acc[1] = float4_t{0, 0, 0, 0};
    }
    if (kInt4 || last) {
      lgkm_wait0();
      wg_barrier();                    // the loads stay in flight
    }
    if (last) {
      // value (token j, row n) of the tile sits in lane 16 (j / 4) + n, element j % 4
      if (tid < 256) {
        const int j = tid >> 4, n = tid & 15, l = (j >> 2) * 16 + n, e = j & 3;
        float g = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          g += red[rflip][0][w][l][e];
          v += red[rflip][1][w][l][e];
        }
        const int c0 = 16 * cur.ch;
        if (c0 + j < cur.cnt) {
          const int sl = cur.slot + c0;
          a.mid[(int64_t)sl * a.i +
                mid_offset<FMT, S>(cur.tile * 16 + n, j, min(16, cur.cnt - c0))] =
              (uint16_t)pack2<XDT>(silu(g) * v, 0.0f);
        }
      }
      rflip ^= 1;
    }
    flip ^= 1;
    cur = nxt;
  };
  // The last step loads nothing ahead and so waits for nothing (one token, 8 of
  // 64 experts of 2048 x 1024: 1 us of 22); four groups per unit leave no
  // registers for a second copy of the step.
  if constexpr (S == 4) {
    while (cur.st < st1) step(std::true_type{});
  } else {
    while (cur.st + 1 < st1 || cur.pass + 1 < passes) step(std::true_type{});
    step(std::false_type{});
  }
}

// -------------------------------------------------------------------- down
// A workgroup owns RT tiles of 16 rows of y.  The columns of all chunks (up to
// 16 tokens of one expert) form one k of chunks * i values, in groups of R
// units; its gridDim.y parts go to as many workgroups, and of a part each wave
// takes a contiguous piece.  A wave's sums over one chunk (a row of the MFMA
// result per token), times the token's p, go into the wave's own rows of y in
// LDS when the chunk ends, so no two waves touch the same value and the order is fixed.  R units
// per wave are in flight, and 16 waves share the CU.
//
// INT4: one load of scales and one of zero points serves the R x RT units of a
// group (four), R adjacent lanes fetching those of one row; a permute brings
// them to the lanes of that row.
template <int XDT, int FMT, int S, int NW, int RT>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(MoeArgs a) {
  constexpr bool kInt4 = FMT == WQ_FMT_INT4_ASYM;
  constexpr int R = (kInt4 ? 4 : 2) / RT;
  extern __shared__ uint4_t dsm[];
  Chunk* const chunk = reinterpret_cast<Chunk*>(dsm);                  // [kMaxChunks]
  uint8_t* const tok = reinterpret_cast<uint8_t*>(chunk + kMaxChunks); // [kMaxT * kMaxK]
  float* const prob = reinterpret_cast<float*>(tok + kMaxT * kMaxK);   // [kMaxT * kMaxK]
  float* const ys = prob + kMaxT * kMaxK;                              // [NW][t][16 RT]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  // the table before its length is known (the rest of it is never used): the
  // count and the table are one memory round trip, not two
  const int most = min(a.e, a.t * a.top_k) + a.t * a.top_k / 16;
  for (int i = tid; i < most; i += NW * 64) chunk[i] = a.table[i];
  const int chunks = *a.count;
  for (int i = tid; i < a.t * a.top_k; i += NW * 64) {
    tok[i] = a.slot_tok[i];
    prob[i] = a.slot_prob[i];
  }
  for (int i = tid; i < NW * a.t * 16 * RT; i += NW * 64) ys[i] = 0.0f;
  __syncthreads();
  const int ku = a.i >> 7, kg = (ku + R - 1) / R, n0 = (int)blockIdx.x * 16 * RT;
  const int steps = chunks * kg, pieces = (int)gridDim.y * NW;
  const int per = (steps + pieces - 1) / pieces;
  const int s0 = min(((int)blockIdx.y * NW + wave) * per, steps), s1 = min(s0 + per, steps);
  float* const yw = ys + wave * a.t * 16 * RT;
  const uint32_t off = code_off<FMT>(a.i, lane);

  if (s0 < s1) {
    // a group of units: its chunk, and the first of its units
    struct Pos {
      int64_t row;
      int ci, g, slot, cnt;
    };
    auto enter = [&](Pos& p) {
      const Chunk c = chunk[p.ci];
      p.slot = __builtin_amdgcn_readfirstlane(c.slot);
      p.cnt = __builtin_amdgcn_readfirstlane(c.cnt);
      p.row = (int64_t)__builtin_amdgcn_readfirstlane(c.expert) * a.h + n0;
    };
    auto tile_of = [&](const Pos& p, int r) {
      return tile_at<FMT, S>(a.down, a.down_s, a.down_z, p.row + 16 * r, a.i);
    };
    auto load = [&](const Pos& p, int j, Unit<FMT> (&w)[RT], Acts& x) {
      const int u = min(p.g * R + j, ku - 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) load_unit<FMT>(w[r], tile_of(p, r), off, u);
      const uint16_t* const m = a.mid + (int64_t)p.slot * a.i + u * 128 * p.cnt;
      const uint32_t xo = (uint32_t)(kq * p.cnt + min(nl, p.cnt - 1)) * 16;
#pragma unroll
      for (int f = 0; f < 4; ++f) x.f[f] = load_at<uint4_t>(m + f * 32 * p.cnt, xo);
    };
    // scales and zero points of unit lane % R of the group, row lane / R
    uint32_t ms[2], mz;
    auto load_meta = [&](const Pos& p) {
      const int u = min(p.g * R + (lane & (R - 1)), ku - 1), g = ku * S, rw = lane / R;
      const uint32_t so = (uint32_t)((rw * g + u * S) * 2);
      const uint32_t zo = (uint32_t)(rw * ((g + 1) >> 1) + ((u * S) >> 1));
      const Tile t = tile_of(p, 0);
      if constexpr (S == 1) {
        ms[0] = load_at<uint16_t>(t.scales, so);
        mz = load_at<uint8_t>(t.zeros, zo);
      } else if constexpr (S == 2) {
        ms[0] = load_at<uint32_t>(t.scales, so);
        mz = load_at<uint8_t>(t.zeros, zo);
      } else {
        const uint2_t v = load_at<uint2_t>(t.scales, so);
        ms[0] = v[0];
        ms[1] = v[1];
        mz = load_at<uint16_t>(t.zeros, zo);
      }
    };
    // as one word per group of k
    auto words = [&](const Pos& p, uint32_t (&m)[S]) {
      const int u = min(p.g * R + (lane & (R - 1)), ku - 1);
#pragma unroll
      for (int g = 0; g < S; ++g)
        m[g] = meta_word((ms[g >> 1] >> (16 * (g & 1))) & 0xFFFFu,
                         (mz >> (4 * (S == 1 ? u & 1 : g))) & 15u);
    };

    Pos cur{0, s0 / kg, 0, 0, 0};
    cur.g = s0 - cur.ci * kg;
    enter(cur);
    float4_t acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = float4_t{0, 0, 0, 0};
    auto flush = [&](const Pos& p) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 4 * kq + e;
        if (j < p.cnt) {
          float* const o = yw + tok[p.slot + j] * RT * 16 + nl;
          const float pr = prob[p.slot + j];
#pragma unroll
          for (int r = 0; r < RT; ++r) o[r * 16] = fmaf(acc[r][e], pr, o[r * 16]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = float4_t{0, 0, 0, 0};
    };
    Unit<FMT> w[R][RT];
    Acts x[R];
    if constexpr (kInt4) load_meta(cur);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      load(cur, j, w[j], x[j]);
      // in this order, as the loop waits for them
      __builtin_amdgcn_sched_barrier(0);
    }
    auto step = [&](auto more) __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value;       // another group follows
      Pos nxt = cur;
      if (MORE && ++nxt.g == kg) {
        nxt.g = 0;
        ++nxt.ci;
        enter(nxt);
      }
      uint32_t m[S];
      if constexpr (kInt4) {
        words(cur, m);
        if constexpr (MORE) load_meta(nxt);
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        uint32_t mj[RT][S];
        if constexpr (kInt4) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int g = 0; g < S; ++g)
              mj[r][g] = (uint32_t)__builtin_amdgcn_ds_bpermute(((16 * r + nl) * R + j) * 4,
                                                                (int)m[g]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (cur.g * R + j < ku) unit_mac<XDT, FMT, S, RT>(w[j], mj, x[j], acc);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MORE) load(nxt, j, w[j], x[j]);
      }
      if (!MORE || nxt.ci != cur.ci) flush(cur);
      cur = nxt;
    };
    for (int st = s0; st + 1 < s1; ++st) step(std::true_type{});
    step(std::false_type{});
  }
  __syncthreads();
  constexpr int BR = 16 * RT;
  for (int i = tid; i < a.t * BR; i += NW * 64) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += ys[w * a.t * BR + i];
    const int64_t o = (int64_t)(i / BR) * a.h + n0 + i % BR;
    if (gridDim.y > 1) a.part[(int64_t)blockIdx.y * a.t * a.h + o] = v;
    else store_as(a.y, a.ydt, o, v);
  }
}

// y = the sum of the parts, in their order; four are loaded before the first is
// added, so their latencies do not add up
__global__ __launch_bounds__(256) void moe_join_kernel(const float* __restrict__ part, int parts,
                                                       int count, void* y, int ydt) {
  const int i = (int)blockIdx.x * 256 + (int)threadIdx.x;
  if (i >= count) return;
  float v = 0.0f;
  int p = 0;
  for (; p + 4 <= parts; p += 4) {
    float t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = part[(int64_t)(p + j) * count + i];
#pragma unroll
    for (int j = 0; j < 4; ++j) v += t[j];
  }
  for (; p < parts; ++p) v += part[(int64_t)p * count + i];
  store_as(y, ydt, i, v);
}

// ------------------------------------------------------------------ launch
constexpr int kDownTables = kMaxChunks * (int)sizeof(Chunk) + kMaxT * kMaxK * 5;

// Parts of k in the down product with two row tiles per workgroup, as many as
// fill the 256 CUs once, or 0: one row tile, all of k, no join.  Two tiles read
// the intermediate once for both, which the L2 carries at several times the
// codes' size: 64 tokens, 2 of 8 experts of 4096 x 14336 INT4 take 247 us (two
// tiles, 2 parts), 262 (one tile), 322 (two tiles, one part); 24 tokens, 6 of
// 64 FP8 experts of 2048 x 1024 83 us (two tiles, 4 parts) against 98; 4 tokens, 8
// of 64 INT4 34.2 against 39.6.  For a few choices the join costs more than that
// gives: one token, 8 of 64 18.5 us with one tile, 19.5 with two in 4 parts.
int down_parts(int64_t t, int64_t top_k, int64_t h) {
  return t * top_k <= 8 ? 0 : (int)std::max<int64_t>(1, 256 * 32 / h);
}

template <int XDT, int FMT, int S, int RT>
hipError_t down_launch(const MoeArgs& a, int parts, hipStream_t s) {
  constexpr int NW = 16;
  constexpr int most = kDownTables + NW * kMaxT * 64 * RT;
  auto* kern = &moe_down_kernel<XDT, FMT, S, NW, RT>;
  static std::atomic<uint64_t> done{0};
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), most, done);
  if (e != hipSuccess) return e;
  const int bytes = kDownTables + NW * a.t * 64 * RT;
  kern<<<dim3((unsigned)(a.h / (16 * RT)), (unsigned)parts), NW * 64, bytes, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  const int count = a.t * a.h;
  moe_join_kernel<<<dim3((unsigned)((count + 255) / 256)), 256, 0, s>>>(a.part, parts, count, a.y,
                                                                       a.ydt);
  return hipGetLastError();
}

template <int XDT, int FMT, int S>
hipError_t moe_fmt(const MoeArgs& a, hipStream_t s) {
  if (a.router != nullptr) {
    const dim3 grid((unsigned)((a.e + 15) / 16), (unsigned)((a.t + 15) / 16));
    moe_router_kernel<XDT><<<grid, 1024, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // 8 waves and two workgroups per CU, which are seldom at the same point of a
  // step, where they cover k in one pass; else 16 waves and one: 16 tokens, 8 of
  // 64 INT4 experts, h = 2048, 61.0 us with 8 waves, 73.8 with 16; 64 tokens, 2
  // of 8, h = 4096, 363 with 8 (two passes), 247 with 16
  const int64_t units = (int64_t)std::min(a.e, a.t * a.top_k) * (a.i / 16);
  if (a.h <= 8 * 256) {
    const unsigned grid = (unsigned)std::min<int64_t>(units, 512);
    moe_gate_up_kernel<XDT, FMT, S, 8><<<dim3(grid), 8 * 64, 0, s>>>(a, 1);
  } else {
    const unsigned grid = (unsigned)std::min<int64_t>(units, 256);
    moe_gate_up_kernel<XDT, FMT, S, 16>
        <<<dim3(grid), 16 * 64, 0, s>>>(a, (a.h + 16 * 256 - 1) / (16 * 256));
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int parts = down_parts(a.t, a.top_k, a.h);
  if (parts == 0) return down_launch<XDT, FMT, S, 1>(a, 1, s);
  return down_launch<XDT, FMT, S, 2>(a, parts, s);
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

// workspace: logits fp32 [t][e] | count | table | token of each row | its p |
// intermediate [t * top_k][i] | parts of y fp32 [parts][t][h]
size_t moe_ws_bytes(int64_t t, int64_t e, int64_t top_k, int64_t h, int64_t i) {
  return up256((size_t)(t * e) * 4) + 256 + up256(kMaxChunks * sizeof(Chunk)) + kMaxT * kMaxK * 5 +
         up256((size_t)(t * top_k * i) * 2) + (size_t)down_parts(t, top_k, h) * t * h * 4;
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
  a.table = reinterpret_cast<Chunk*>(p);
  p += up256(kMaxChunks * sizeof(Chunk));
  a.slot_tok = reinterpret_cast<uint8_t*>(p);
  p += kMaxT * kMaxK;
  a.slot_prob = reinterpret_cast<float*>(p);
  p += kMaxT * kMaxK * 4;
  a.mid = reinterpret_cast<uint16_t*>(p);
  p += up256((size_t)(c.t * c.top_k * c.i) * 2);
  a.part = reinterpret_cast<float*>(p);
  a.y = c.y;
  a.ids = c.ids;
  a.probs = c.probs;
  a.t = (int)c.t; a.e = (int)c.e; a.top_k = c.top_k; a.h = (int)c.h; a.i = (int)c.i;
  a.renorm = c.renorm; a.ydt = c.ydt;
  return c.xdt == WQ_BF16 ? moe_xdt<WQ_BF16>(a, c.gate->fmt, c.gate->group, s)
                          : moe_xdt<WQ_F16>(a, c.gate->fmt, c.gate->group, s);
}

}  // namespace wq
