// FP8 linear: y[i][j] = sum_b sx[b][i] * sw[j/128][b] * sum_{c in block b} xq[i][c] * wq[j][c],
// E4M3 activations with a scale per token and 128 values of k, E4M3 weights
// with a scale per 128 x 128 block.
//
// The sum over one block of 128 is exactly one v_mfma_f32_16x16x128_f8f6f4,
// so every matrix instruction starts from zero and its four results per lane
// are added to the fp32 totals with one fused multiply-add each.
//
// The FP8 matrix instructions (all of them: 16x16x32, 16x16x128 and 32x32x64
// give the same bits) cut every product towards zero at 2^-17 of the largest power
// of two among a sum's products: measured on N(0, 100) codes 1.5e-5 of the sum's
// size, 4.6e-5 with one outlier per block, and at worst 2^-10 of the largest
// product (256 * 256 beside 127 products alike: 0.43 * 2^-16 of it each).  On
// activations that is far below the rounding of a 16-bit y (up to 2^-8 or 2^-11 of
// the value), and the worst is no larger than it, so those outputs use them.  An
// fp32 y takes the exact products instead: the codes converted to bf16 (exact) and
// four v_mfma_f32_16x16x32_bf16 per block, 1e-8 on the same codes, at half the
// matrix rate.
//
// Operands: the weights are the A operand (16 output features), the activations
// the B operand (16 tokens): a lane then holds four consecutive features of ONE
// token, whose scale product sx * sw is one value per lane and instruction
// group, and which store as one piece of a row of y.
//
// Which bytes of a block a lane feeds into the K positions of the instruction
// is free as long as both operands agree: lane group g = lane / 16 takes the
// 16-byte chunks g and g + 4.
//
// Four schedules, chosen in plan_fp8; all bring both operands into LDS by direct
// loads, 128 bytes of k at a time:
//  * decode, up to 64 tokens: bound by HBM (one token 14336 x 4000 5.5 TB/s).  A
//    workgroup owns 16 features over all of k; its waves take the blocks of k in
//    turn and add their totals in LDS in a fixed order.
//  * tiles of 64 or 128 tokens x 128 features (fp8_gemm_kernel): bound by
//    latency, the chain of a block's loads, operand reads and products (512
//    tokens 4096 x 4096 19 us, of which the products are 4).  Where the tiles
//    are too few to fill the GPU, k is split over workgroups whose fp32 totals
//    a second kernel adds.
//  * tiles of 256 x 256 (fp8_halves_kernel): bound by the matrix cores and by
//    what their operands cost (4096 tokens 14336 x 4096 214 to 222 us over boxes,
//    2170 to 2250 TFLOP/s; a library product without block scales 205 us).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8_util.h"

namespace wq {
namespace {

struct Fp8Args {
  const uint8_t* x;          // [m][k]
  const float* sx;           // [kb][m]
  const uint8_t* w;          // [n][k]
  const float* sw;           // [ceil(n/128)][kb]
  void* y;                   // [m][n]
  float* part;               // split totals [splits][m][n], or nullptr
  int m, n, k, kb, splits;
  int ld;                    // features of y
};

__device__ const uint4_t kZero16 = {0, 0, 0, 0};   // what chunks past k read

__device__ __forceinline__ float4_t mfma_fp8(int8v_t a, int8v_t b) {
  const float4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// 4 E4M3 bytes -> 4 bf16 values (exact)
__device__ __forceinline__ void fp8_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, true);
  lo = __builtin_bit_cast(uint32_t, a);
  hi = __builtin_bit_cast(uint32_t, b);
}

// A lane's 32 bytes of one block as an operand: as they are, or (EXACT)
// converted to bf16, 8 values for each of four instructions
template <bool EXACT>
struct Operand;
template <>
struct Operand<false> {
  int8v_t v;
  __device__ __forceinline__ void set(uint4_t a, uint4_t b) {
    const uint4_t t[2] = {a, b};
    __builtin_memcpy(&v, t, 32);
  }
};
template <>
struct Operand<true> {
  uint4_t v[4];
  __device__ __forceinline__ void piece(int f, uint4_t a, uint4_t b) {
    const uint32_t c[2] = {f < 2 ? a[2 * f] : b[2 * f - 4], f < 2 ? a[2 * f + 1] : b[2 * f - 3]};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t lo, hi;
      fp8_to_bf16(c[i], lo, hi);
      v[f][2 * i] = lo;
      v[f][2 * i + 1] = hi;
    }
  }
  __device__ __forceinline__ void set(uint4_t a, uint4_t b) {
#pragma unroll
    for (int f = 0; f < 4; ++f) piece(f, a, b);
  }
};

// the sum over one block of k, from zero
__device__ __forceinline__ float4_t block_sum(const Operand<false>& a, const Operand<false>& b) {
  return mfma_fp8(a.v, b.v);
}
__device__ __forceinline__ float4_t block_sum(const Operand<true>& a, const Operand<true>& b) {
  float4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v[i]),
                                                __builtin_bit_cast(bf16x8_t, b.v[i]), c, 0, 0, 0);
  return c;
}

template <int YDT>
__device__ __forceinline__ void store1(void* y, int64_t i, float v) {
  if constexpr (YDT == WQ_F32) static_cast<float*>(y)[i] = v;
  else static_cast<uint16_t*>(y)[i] = (uint16_t)pack2<YDT>(v, 0.0f);
}
// four consecutive values; `wide` when the address allows one store
template <int YDT>
__device__ __forceinline__ void store4(void* y, int64_t i, float4_t v, bool wide, int count) {
  if (wide) {
    if constexpr (YDT == WQ_F32) {
      *reinterpret_cast<float4_t*>(static_cast<float*>(y) + i) = v;
    } else {
      *reinterpret_cast<uint2_t*>(static_cast<uint16_t*>(y) + i) =
          uint2_t{pack2<YDT>(v[0], v[1]), pack2<YDT>(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < count) store1<YDT>(y, i + e, v[e]);
  }
}

// ------------------------------------------------------------------ decode
// s_waitcnt for all but the loads of the n newest blocks, `per` loads each
template <int PER, int MAX>
__device__ __forceinline__ void wait_blocks(int n) {
  if constexpr (MAX == 0) {
    vm_wait<0>();
  } else {
    if (n >= MAX) vm_wait<MAX * PER>();
    else wait_blocks<PER, MAX - 1>(n);
  }
}

// Up to 64 tokens.  A workgroup owns 16 features over all of k, a wave every
// NW-th block of it.  Weights, activations (MT tiles of 16 tokens) and their
// scales reach a ring of R blocks per wave in LDS by direct loads, so R blocks
// per wave are in flight and a load's adjacent lanes take adjacent bytes, eight
// lanes to a 128-byte row (loaded as the matrix instruction wants them,
// adjacent lanes on different rows, each load takes four times as long to
// address: 12.9 against 10.0 us for 16 x 4096 x 11008, 5.7 against 4.7 for one
// token and 4096 x 4096).  MT = 0: a single token, whose 128 bytes come in one
// 4-byte load per lane and whose scale is a scalar load.
template <int MT>
constexpr int decode_slot_bytes() {
  return 16 * kF8Block + (MT == 0 ? 256 : MT * 16 * kF8Block + 256);
}

template <int YDT, int NW, int R, int MT>
__global__ __launch_bounds__(NW * 64) void fp8_decode_kernel(Fp8Args a) {
  constexpr bool ONE = MT == 0;
  constexpr int T = ONE ? 1 : MT, TB = 16 * kF8Block;      // token tiles, bytes of a tile
  constexpr int SLOT = decode_slot_bytes<MT>(), LPB = ONE ? 3 : 2 * MT + 3, SO = TB * (1 + T);
  extern __shared__ uint4_t dsm[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int n0 = (int)blockIdx.x * 16;
  char* const ring = reinterpret_cast<char*>(dsm) + wave * R * SLOT;
  using cfloat = const __attribute__((address_space(4))) float;
  cfloat* const swr = (cfloat*)(a.sw + (int64_t)(n0 / kF8Block) * a.kb);
  const int nb = a.kb > wave ? (a.kb - wave + NW - 1) / NW : 0;    // blocks of this wave

  // chunk (l & 7) ^ (row & 7) of row l / 8 goes to slot l & 7 of that row
  const int lr = lane >> 3, lc = ((lane & 7) ^ lr) * 16;
  const uint8_t* const w0 = a.w + (int64_t)min(n0 + lr, a.n - 1) * a.k;
  const uint8_t* const w1 = a.w + (int64_t)min(n0 + 8 + lr, a.n - 1) * a.k;
  auto issue = [&](int i) {
    const int b = wave + i * NW, c = b * kF8Block + lc;
    char* const l = ring + (i % R) * SLOT;
    const bool in = c < a.k;                 // chunks past k are zeros
    lds_dma16(in ? w0 + c : (const void*)&kZero16, (lds_void_t*)l);
    lds_dma16(in ? w1 + c : (const void*)&kZero16, (lds_void_t*)(l + 1024));
    if constexpr (ONE) {
      const int d = b * kF8Block + (lane & 31) * 4;
      lds_dma4(d < a.k ? a.x + d : (const void*)&kZero16, (lds_void_t*)(l + TB));
    } else {
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        const uint8_t* const xr = a.x + (int64_t)min(8 * t + lr, a.m - 1) * a.k;
        lds_dma16(in ? xr + c : (const void*)&kZero16, (lds_void_t*)(l + TB + t * 1024));
      }
      lds_dma4(a.sx + (int64_t)b * a.m + min(lane, a.m - 1), (lds_void_t*)(l + SO));
    }
  };
  for (int i = 0; i < min(R, nb); ++i) issue(i);
  const int s0 = nl * kF8Block + (kq ^ (nl & 7)) * 16;
  const int s1 = nl * kF8Block + ((kq + 4) ^ (nl & 7)) * 16;
  float4_t acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < nb; ++i) {
    const char* const l = ring + (i % R) * SLOT;
    const int b = wave + i * NW;
    float s = swr[b];
    if constexpr (ONE) s *= ((cfloat*)a.sx)[b];
    wait_blocks<LPB, R - 1>(nb - 1 - i);
    asm volatile("" ::: "memory");
    Operand<YDT == WQ_F32> wa;
    wa.set(*reinterpret_cast<const uint4_t*>(l + s0), *reinterpret_cast<const uint4_t*>(l + s1));
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const char* const xl = l + TB * (1 + t);
      Operand<YDT == WQ_F32> xb;
      float st = s;
      if constexpr (ONE) {
        xb.set(*reinterpret_cast<const uint4_t*>(xl + kq * 16),
               *reinterpret_cast<const uint4_t*>(xl + 64 + kq * 16));
      } else {
        xb.set(*reinterpret_cast<const uint4_t*>(xl + s0),
               *reinterpret_cast<const uint4_t*>(xl + s1));
        st *= *reinterpret_cast<const float*>(l + SO + (t * 16 + nl) * 4);
      }
      const float4_t c = block_sum(wa, xb);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(c[e], st, acc[t][e]);
    }
    // the operands are in registers: the slot is free
    if (i + R < nb) {
      lgkm_wait0();
      issue(i + R);
    }
  }
  // the waves' totals, over the rings
  __syncthreads();
  float4_t* const red = reinterpret_cast<float4_t*>(dsm);
#pragma unroll
  for (int t = 0; t < T; ++t) red[(wave * T + t) * 64 + lane] = acc[t];
  __syncthreads();
  if (wave < T) {
    float4_t v = red[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[(w * T + wave) * 64 + lane];
    const int n = n0 + kq * 4, m = wave * 16 + nl;
    if (m < a.m && n < a.n)
      store4<YDT>(a.y, (int64_t)m * a.n + n, v, (a.n & 3) == 0, a.n - n);
  }
}

template <int YDT, int NW, int R, int MT>
hipError_t decode_launch(const Fp8Args& a, hipStream_t s) {
  constexpr int bytes = NW * R * decode_slot_bytes<MT>();
  static_assert(bytes >= NW * (MT == 0 ? 1 : MT) * 1024 && NW >= MT, "room for the totals");
  auto* kern = &fp8_decode_kernel<YDT, NW, R, MT>;
  static std::atomic<uint64_t> done{0};
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), bytes, done);
  if (e != hipSuccess) return e;
  kern<<<dim3((unsigned)((a.n + 15) / 16)), NW * 64, bytes, s>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------------------- tiles
// direct global -> LDS load with a uniform base, a 32-bit lane offset and a
// uniform address in LDS
__device__ __forceinline__ void lds_dma16_s(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds)
               : "memory");
}

// tile t of T in an order in which each XCD (workgroups reach the 8 XCDs in
// turn) runs a contiguous range, walked GM token tiles at a time
__device__ __forceinline__ void tile_of_block(int bid, int T, int tm, int tn, int& im, int& in) {
  constexpr int GM = 4;
  const int q = T >> 3, r = T & 7, xcd = bid & 7;
  const int t = xcd * q + min(xcd, r) + (bid >> 3);
  const int per = GM * tn, g = t / per, w = t - g * per;
  const int gm = min(GM, tm - g * GM);
  im = g * GM + w % gm;
  in = w / gm;
}

// 2 x 2 waves, each 64 features x TM tiles of 16 tokens.  A wave holds a whole
// block's operands in registers and reads each one's successor from LDS right
// after its last product, so one barrier per block, early in it, frees the
// block's buffer for the loads of NB blocks later and finds the next block
// arrived.  The scaled additions of a result wait until three more matrix
// instructions are issued.
//
// Nothing between two blocks may make the compiler wait for all loads: a load of
// scales under a branch without its own wait did, in every block, and cost more
// than the products (512 tokens 4096 x 4096 24 us as split tiles, then 19).
// Blocks in flight: 64 x 128 tiles take NB = 6 (150 KB, one workgroup per CU),
// 128 x 128 tiles two with two workgroups per CU (1000 tokens 4096 x 4096 28.3
// us, NB = 4 with one workgroup 27.8; the exact products, which need the second
// wave to convert operands under the products, 41.8 and 44.2).
constexpr int kTileN = 128;
template <int TM>
constexpr int fp8_buf_bytes() { return (kTileN + TM * 32) * kF8Block + TM * 32 * 4; }

template <int YDT, int TM, int NB>
__global__ __launch_bounds__(256, 2) void fp8_gemm_kernel(Fp8Args a, int tm, int tn) {
  constexpr bool EXACT = YDT == WQ_F32;
  constexpr int NW = 4, TN = 4, T = TN * TM, BN = kTileN, BM = TM * 32;
  constexpr int BUF = fp8_buf_bytes<TM>();
  constexpr int WI = BN / 8 / NW, XI = BM / 8 / NW;      // direct loads per wave and block,
  constexpr int SL = BM / NW;                            // and tokens whose scales it brings
  constexpr int L = 1 + WI + XI;
  static_assert(TM % 2 == 0 && TM <= 4 && (NB - 1) * L <= 63, "counted loads");
  extern __shared__ uint4_t dsm[];
  char* const lds = reinterpret_cast<char*>(dsm);
  const uint32_t l0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int nl = lane & 15, kq = lane >> 4;
  int im, in;
  tile_of_block((int)blockIdx.x, tm * tn, tm, tn, im, in);
  const int n0 = in * BN, m0 = im * BM;
  // this workgroup's blocks of k
  const int per = (a.kb + a.splits - 1) / a.splits;
  const int b0 = (int)blockIdx.y * per, b1 = min(b0 + per, a.kb);

  // Lane l of a load brings chunk (l & 7) ^ f of row l / 8 into slot l & 7 of
  // that row, with f different for the 8 rows that an operand read takes at
  // once, so that they hold the same chunk in 8 different slots.  Rows past the
  // end read the last row; their results are not stored.
  const int lr = lane >> 3, lcx = ((lane & 7) ^ lr) * 16;
  const int lcw = EXACT ? lcx : ((lane & 7) ^ ((lr & 3) | (wave & 1) << 2)) * 16;
  const uint8_t* const wbase = a.w + (int64_t)n0 * a.k;
  const uint8_t* const xbase = a.x + (int64_t)m0 * a.k;
  uint32_t woff[WI], xoff[XI];
#pragma unroll
  for (int i = 0; i < WI; ++i)
    woff[i] = (uint32_t)min((i * NW + wave) * 8 + lr, a.n - 1 - n0) * (uint32_t)a.k;
#pragma unroll
  for (int i = 0; i < XI; ++i)
    xoff[i] = (uint32_t)min((i * NW + wave) * 8 + lr, a.m - 1 - m0) * (uint32_t)a.k;
  const int ms = min(m0 + wave * SL + lane, a.m - 1);
  // Load i of the L of block b into the buffer at `buf`.  A chunk past k is its
  // row's first instead: the weight operands are cleared there, and a NaN code
  // in a row of x has made its whole row of y NaN in any case.
  auto chunk = [&](int b, int lc) {
    const int c = b * kF8Block + lc;
    return (uint32_t)(c < a.k ? c : 0);
  };
  auto load = [&](int b, uint32_t buf, int i) __attribute__((always_inline)) {
    if (i < WI) {
      lds_dma16_s(wbase, woff[i] + chunk(b, lcw), l0 + buf + (i * NW + wave) * 1024);
    } else if (i < WI + XI) {
      lds_dma16_s(xbase, xoff[i - WI] + chunk(b, lcx),
                  l0 + buf + BN * kF8Block + ((i - WI) * NW + wave) * 1024);
    } else if (lane < SL) {
      lds_dma4(a.sx + (int64_t)b * a.m + ms,
               (lds_void_t*)(lds + buf + (BN + BM) * kF8Block + wave * SL * 4));
    }
  };

  // the weight scales of 64 blocks at a time, one per lane
  const int nbw = min((n0 + wn * TN * 16) / kF8Block, (a.n - 1) / kF8Block);
  const float* const swr = a.sw + (int64_t)nbw * a.kb;
  float swl = swr[min(b0 + lane, a.kb - 1)];
  asm volatile("" : "+v"(swl));            // waited for before the direct loads

  float4_t acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // Slots of this lane's two chunks in its operand rows.  Row nl of weight
  // operand i is feature 32 (i / 2) + 8 (nl / 4) + 4 (i % 2) + nl % 4 of the
  // wave's 64 (16-bit y): a lane's results of two operands are then eight
  // consecutive features, one 16-byte store.  fp32 y: 16 i + nl.
  const int s0 = (kq ^ (nl & 7)) * 16, s1 = ((kq + 4) ^ (nl & 7)) * 16;
  const int wo = (wn * TN * 16 + (EXACT ? nl : (nl >> 2) * 8 + (nl & 3))) * kF8Block;
  auto wrow = [](int i) { return EXACT ? i * 16 : (i >> 1) * 32 + (i & 1) * 4; };
  const int xo = (BN + wm * TM * 16 + nl) * kF8Block;
  const int so = (BN + BM) * kF8Block + (wm * TM * 16 + nl) * 4;
  uint4_t wr[TN][2], xr[TM][2];
  float xs[TM];
  auto read_w = [&](int b, uint32_t buf, int i, bool tail) __attribute__((always_inline)) {
    const char* const l = lds + buf + wo + wrow(i) * kF8Block;
    wr[i][0] = *reinterpret_cast<const uint4_t*>(l + s0);
    wr[i][1] = *reinterpret_cast<const uint4_t*>(l + s1);
    if (tail) {
      if (b * kF8Block + kq * 16 >= a.k) wr[i][0] = uint4_t{0, 0, 0, 0};
      if (b * kF8Block + kq * 16 + 64 >= a.k) wr[i][1] = uint4_t{0, 0, 0, 0};
    }
  };
  auto read_x = [&](uint32_t buf, int j) __attribute__((always_inline)) {
    const char* const l = lds + buf;
    xr[j][0] = *reinterpret_cast<const uint4_t*>(l + xo + j * 16 * kF8Block + s0);
    xr[j][1] = *reinterpret_cast<const uint4_t*>(l + xo + j * 16 * kF8Block + s1);
    xs[j] = *reinterpret_cast<const float*>(l + so + j * 64);
  };

  float4_t ring[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
  float sr[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](int t) __attribute__((always_inline)) {  // result t of a block to its total
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[t % TN][t / TN][e] = fmaf(ring[t & 3][e], sr[t & 3], acc[t % TN][t / TN][e]);
    // the total is formed here: put off, the results would not fit
    asm volatile("" : "+v"(acc[t % TN][t / TN]));
  };
  uint32_t cb = 0;                         // buffer of the block
  Operand<EXACT> w[TN], x[2];
  auto step = [&](int b, auto inner) __attribute__((always_inline)) {
    constexpr bool IN = decltype(inner)::value;          // NB more blocks follow
    const float sw =
        __int_as_float(__builtin_amdgcn_readlane(__float_as_int(swl), (b - b0) & 63));
    const uint32_t nb = cb + BUF == NB * BUF ? 0 : cb + BUF;
    float s;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int i = t % TN, j = t / TN;
      if (t == TN) {
        // every operand of this block is in registers, and the next has arrived
        if constexpr (IN) vm_wait<(NB - 2) * L>();
        else wait_blocks<L, NB - 2>(min(max(b1 - 2 - b, 0), NB - 2));
        lgkm_wait0();
        __builtin_amdgcn_sched_barrier(0);
        wg_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i == 0) s = xs[j] * sw;
      if constexpr (EXACT) {
        // the conversions of the next operands run under the products
        ring[t & 3] = block_sum(w[i], x[j & 1]);
        x[(j + 1) & 1].piece(i, xr[(j + 1) % TM][0], xr[(j + 1) % TM][1]);
        if (j == 0 && i + 1 < TN) w[i + 1].set(wr[i + 1][0], wr[i + 1][1]);
        if (t == T - 1) w[0].set(wr[0][0], wr[0][1]);
      } else {
        if (i == 0) x[0].set(xr[j][0], xr[j][1]);
        if (j == 0) w[i].set(wr[i][0], wr[i][1]);
        ring[t & 3] = block_sum(w[i], x[0]);
        __builtin_amdgcn_sched_barrier(0);
      }
      sr[t & 3] = s;
      add((t + T - 3) % T);
      // an operand's registers take the next block's after its last product
      if (i == 0 && j > 0) read_x(nb, j - 1);
      if (j == TM - 1) read_w(b + 1, nb, i, !IN && (b + 2) * kF8Block > a.k);
      if (t == T - 1) read_x(nb, j);
      if (IN && t >= TN) {
#pragma unroll
        for (int l = t - TN; l < L; l += T - TN) load(b + NB, cb, l);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    cb = nb;
  };
#pragma unroll
  for (int d = 0; d < NB; ++d)
    if (b0 + d < b1) {
#pragma unroll
      for (int i = 0; i < L; ++i) load(b0 + d, d * BUF, i);
    }
  wait_blocks<L, NB - 1>(min(b1 - 1 - b0, NB - 1));
  wg_barrier();
#pragma unroll
  for (int j = 0; j < TM; ++j) read_x(0, j);
#pragma unroll
  for (int i = 0; i < TN; ++i) read_w(b0, 0, i, (b0 + 1) * kF8Block > a.k);
  if constexpr (EXACT) {
    x[0].set(xr[0][0], xr[0][1]);
    w[0].set(wr[0][0], wr[0][1]);
  }
  auto scales = [&](int b) {
    if (((b - b0) & 63) == 0 && b > b0) {
      swl = swr[min(b + lane, a.kb - 1)];
      asm volatile("" : "+v"(swl));        // waited for here, not in every block
    }
  };
  int b = b0;
  for (; b + NB < b1; ++b) {
    scales(b);
    step(b, std::true_type{});
  }
  for (; b < b1; ++b) {
    scales(b);
    step(b, std::false_type{});
  }
  add(T - 3);
  add(T - 2);
  add(T - 1);

  const int ns = n0 + wn * TN * 16 + kq * (EXACT ? 4 : 8), mst = m0 + wm * TM * 16 + nl;
  const bool wide = (a.n & (EXACT ? 3 : 7)) == 0;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int m = mst + j * 16;
    if (m >= a.m) continue;
    if (a.part != nullptr) {
      float* const out = a.part + ((int64_t)blockIdx.y * a.m + m) * a.n;
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int n = ns + wrow(i);
        if (n < a.n) store4<WQ_F32>(out, n, acc[i][j], (a.n & 3) == 0, a.n - n);
      }
    } else if (!EXACT && wide) {
#pragma unroll
      for (int i = 0; i < TN; i += 2)
        if (ns + i * 16 < a.n)
          *reinterpret_cast<uint4_t*>(static_cast<uint16_t*>(a.y) + (int64_t)m * a.n + ns +
                                      i * 16) =
              uint4_t{pack2<YDT>(acc[i][j][0], acc[i][j][1]),
                      pack2<YDT>(acc[i][j][2], acc[i][j][3]),
                      pack2<YDT>(acc[i + 1][j][0], acc[i + 1][j][1]),
                      pack2<YDT>(acc[i + 1][j][2], acc[i + 1][j][3])};
    } else {
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int n = ns + wrow(i);
        if (n < a.n)
          store4<YDT>(a.y, (int64_t)m * a.n + n, acc[i][j], (a.n & 3) == 0, a.n - n);
      }
    }
  }
}

// ------------------------------------------------------ tiles in two halves
// 256 features x 32 TM tokens, 8 waves of 64 features x 16 TM tokens.  Waves 0-3
// and 4-7 (one of each per SIMD) are half a step apart: while one half reads its
// operands from LDS the other multiplies, and a barrier swaps them.  A step takes
// a block of k in two parts: all weights and the first half of the tokens, then
// the second half.  So the matrix cores always have a wave with all its operands
// in registers, LDS reads and their latency hide under its products, and a wave
// needs registers for half the tokens' operands only.
//
// LDS holds two blocks.  The weights, scales and first tokens of a block are read
// in its first part, so their space takes the block after next from the second
// part on; the other tokens' space follows in the next block's first part.  Every
// load thus has about three parts to arrive, counted exactly (vm_wait), and
// half of them are issued between products, where the load unit is idle.
//
// Workgroups are persistent (one per CU) and start the next tile's loads before
// they store a tile, which goes past the caches: y would push the operands out of
// L2.  The last round, if at most half the tiles are left, is made of tiles of
// half the tokens.
//
// 4096 tokens 14336 x 4096, us: both halves in step, one barrier per block 294;
// halves alternating 246; loads between products 228; wide stores 222; one
// launch with persistent workgroups 217; stores past the caches 214.  Marginal
// cost of a block per CU 1.37 us, 64 instructions per SIMD: 1.1 us at the 35
// cycles that one takes with its additions.
constexpr int kHalvesN = 256;
constexpr int kCus = 256;
template <int TM>
constexpr int halves_buf_bytes() { return (kHalvesN + TM * 32) * kF8Block + TM * 32 * 4; }

template <int YDT, int TM>
__device__ __forceinline__ void halves_tiles(const Fp8Args& a, char* lds) {
  constexpr int TN = 4, BN = kHalvesN, BM = TM * 32, NW = 8, H = TM / 2, T = TN * H;
  constexpr int BUF = halves_buf_bytes<TM>();
  constexpr int WI = BN / 8 / NW, XI = BM / 16 / NW;     // direct loads per wave; XI per half
  static_assert(BM % (16 * NW) == 0 && T % 4 == 0, "whole loads, the ring goes on");
  const int tm = (a.m + BM - 1) / BM, tn = (a.n + BN - 1) / BN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wn = wave & 3, wm = wave >> 2;
  const int nl = lane & 15, kq = lane >> 4;
  // as in fp8_gemm_kernel, with the weights' rows in the order below
  int n0, m0;
  const uint8_t *wbase, *xbase;
  constexpr int SL = BM / NW;              // tokens whose scales a wave brings
  const float* swr;
  auto place = [&](int tile) __attribute__((always_inline)) {
    int im, in;
    tile_of_block(tile, tm * tn, tm, tn, im, in);
    n0 = in * BN;
    m0 = im * BM;
    wbase = a.w + (int64_t)n0 * a.k;
    xbase = a.x + (int64_t)m0 * a.k;
    swr = a.sw + (int64_t)min((n0 + wn * TN * 16) / kF8Block, (a.n - 1) / kF8Block) * a.kb;
  };
  // Direct loads of 8 rows.  Their offsets are formed each time (rows of a tile
  // are below 256: 24-bit products): kept, they would not fit the registers.
  // A chunk past k is its row's first instead: the weight operands are cleared
  // there, and a NaN code in a row of x has made its row of y NaN in any case.
  const int lr = lane >> 3, lcx = ((lane & 7) ^ lr) * 16;
  const int lcw = ((lane & 7) ^ ((lr & 3) | (wave & 1) << 2)) * 16;
  auto offset = [&](int b, int row, int rows, int lc) {
    int r = lr;
    asm volatile("" : "+v"(r));
    const int c = b * kF8Block + lc;
    return __umul24(min(row + r, rows - 1), a.k) + (uint32_t)(c < a.k ? c : 0);
  };
  const uint32_t l0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)lds);
  auto load_w = [&](int b, int i) {
    int row = wave * 8;
    asm volatile("" : "+s"(row));
    row += i * NW * 8;
    lds_dma16_s(wbase, offset(b, row, a.n - n0, lcw), l0 + (b & 1) * BUF + row * kF8Block);
  };
  const int xw = (wave / TM) * TM * 16 + (wave % TM) * 8;  // its 8 rows of a half's first
  auto load_x = [&](int b, int h, int i) {
    int row = xw;
    asm volatile("" : "+s"(row));
    row += i * NW * 16 + h * TM * 8;
    lds_dma16_s(xbase, offset(b, row, a.m - m0, lcx),
                l0 + (b & 1) * BUF + (BN + row) * kF8Block);
  };
  auto load_s = [&](int b) {
    int l = lane;
    asm volatile("" : "+v"(l));
    if (l < SL)
      lds_dma4(a.sx + (int64_t)b * a.m + min(m0 + wave * SL + l, a.m - 1),
               (lds_void_t*)(lds + (b & 1) * BUF + (BN + BM) * kF8Block + wave * SL * 4));
  };
  auto load_lo = [&](int b) {
    load_s(b);
#pragma unroll
    for (int i = 0; i < XI; ++i) load_x(b, 0, i);
  };

  using cfloat = const __attribute__((address_space(4))) float;
  float4_t acc[TN][TM];
  const int s0 = (kq ^ (nl & 7)) * 16, s1 = ((kq + 4) ^ (nl & 7)) * 16;
  // Row nl of weight operand i is feature 32 (i / 2) + 8 (nl / 4) + 4 (i % 2) +
  // nl % 4 of the wave's 64: a lane's results of two operands are then eight
  // consecutive features, one 16-byte store.
  const int wo = (wn * TN * 16 + ((nl >> 2) * 8 + (nl & 3))) * kF8Block;
  auto wrow = [](int i) { return ((i >> 1) * 32 + (i & 1) * 4) * kF8Block; };
  const int xo = (BN + wm * TM * 16 + nl) * kF8Block;
  const int so = (BN + BM) * kF8Block + (wm * TM * 16 + nl) * 4;

  float4_t ring[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
  float sr[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](int h, int t) {           // result t of half h to its total
    const int i = t % TN, j = h * H + t / TN;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(ring[t & 3][e], sr[t & 3], acc[i][j][e]);
    asm volatile("" : "+v"(acc[i][j]));
  };
  auto step = [&](int b, auto inner) {
    constexpr bool IN = decltype(inner)::value;          // two more blocks follow
    const char* const buf = lds + (b & 1) * BUF;
    Operand<false> w[TN];
    float s[TM];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // ---- operands
      Operand<false> x[H];
      float sw;
      if (IN && h == 1) load_lo(b + 2);
      if (h == 0) {
        sw = ((cfloat*)swr)[b];
#pragma unroll
        for (int j = 0; j < TM; ++j) s[j] = *reinterpret_cast<const float*>(buf + so + j * 64);
        const bool p0 = b * kF8Block + kq * 16 >= a.k, p1 = b * kF8Block + kq * 16 + 64 >= a.k;
        const bool tail = !IN && (b + 1) * kF8Block > a.k;
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          uint4_t c0 = *reinterpret_cast<const uint4_t*>(buf + wo + wrow(i) + s0);
          uint4_t c1 = *reinterpret_cast<const uint4_t*>(buf + wo + wrow(i) + s1);
          if (tail) {
            if (p0) c0 = uint4_t{0, 0, 0, 0};
            if (p1) c1 = uint4_t{0, 0, 0, 0};
          }
          w[i].set(c0, c1);
        }
      }
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const int jj = h * H + j;
        x[j].set(*reinterpret_cast<const uint4_t*>(buf + xo + jj * 16 * kF8Block + s0),
                 *reinterpret_cast<const uint4_t*>(buf + xo + jj * 16 * kF8Block + s1));
      }
      if (h == 0) {
        if constexpr (IN) vm_wait<1 + XI + WI>();
        else vm_wait<0>();
      } else {
        if constexpr (IN) {
          vm_wait<1 + 2 * XI>();
        } else {
          vm_wait<0>();
        }
      }
      if (h == 0) {
#pragma unroll
        for (int j = 0; j < TM; ++j) s[j] *= sw;
      }
      lgkm_wait0();
      __builtin_amdgcn_sched_barrier(0);
      wg_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // ---- products
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        ring[t & 3] = block_sum(w[t % TN], x[t / TN]);
        sr[t & 3] = s[h * H + t / TN];
        __builtin_amdgcn_sched_barrier(0);
        add(t >= 3 ? h : h ^ 1, (t + T - 3) % T);
        if (h == 0) {
          if (t % 4 == 1 && t / 4 < XI && (IN || b + 1 < a.kb)) load_x(b + 1, 1, t / 4);
        } else {
          if (IN && t % (T / WI) == 1) load_w(b + 2, t / (T / WI));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      wg_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the first block and the first parts of the second
  auto begin = [&]() __attribute__((always_inline)) {
    load_lo(0);
#pragma unroll
    for (int i = 0; i < WI; ++i) load_w(0, i);
#pragma unroll
    for (int i = 0; i < XI; ++i) load_x(0, 1, i);
    if (a.kb > 1) {
      load_lo(1);
#pragma unroll
      for (int i = 0; i < WI; ++i) load_w(1, i);
    }
  };
  const int tiles = tm * tn;
  if ((int)blockIdx.x >= tiles) return;
  place((int)blockIdx.x);
  begin();
  if (a.kb > 1) vm_wait<1 + XI + WI>();
  else vm_wait<0>();
  for (int tile = (int)blockIdx.x;;) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    wg_barrier();
    if (wm == 1) wg_barrier();
    int b = 0;
    for (; b + 2 < a.kb; ++b) step(b, std::true_type{});
    for (; b < a.kb; ++b) step(b, std::false_type{});
    if (wm == 0) wg_barrier();
    add(1, T - 3);
    add(1, T - 2);
    add(1, T - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ring[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      sr[i] = 0.0f;
    }

    // the next tile's first loads fly while this one's results are stored
    const int ns = n0 + wn * TN * 16 + kq * 8, mst = m0 + wm * TM * 16 + nl;
    const bool whole = m0 + BM <= a.m && n0 + BN <= a.n && (a.ld & 7) == 0;
    tile += (int)gridDim.x;
    const bool more = tile < tiles;
    if (more) {
      place(tile);
      begin();
    }
    constexpr int NS = TN * TM / 2;      // stores of a whole tile
    if (whole) {
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        uint16_t* const o = static_cast<uint16_t*>(a.y) + (int64_t)(mst + j * 16) * a.ld + ns;
#pragma unroll
        for (int i = 0; i < TN; i += 2) {
          const uint4_t v = {pack2<YDT>(acc[i][j][0], acc[i][j][1]),
                             pack2<YDT>(acc[i][j][2], acc[i][j][3]),
                             pack2<YDT>(acc[i + 1][j][0], acc[i + 1][j][1]),
                             pack2<YDT>(acc[i + 1][j][2], acc[i + 1][j][3])};
          __builtin_nontemporal_store(v, reinterpret_cast<uint4_t*>(o + i * 16));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TM; ++j) {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          const int m = mst + j * 16, n = ns + (i >> 1) * 32 + (i & 1) * 4;
          if (m < a.m && n < a.n)
            store4<YDT>(a.y, (int64_t)m * a.ld + n, acc[i][j], (a.ld & 3) == 0, a.n - n);
        }
      }
    }
    if (!more) break;
    // NS stores, one instruction each, are newer than the loads
    asm volatile("" ::: "memory");
    if (whole && a.kb > 1) vm_wait<1 + XI + WI + NS>();
    else vm_wait<0>();
  }
}

// the first f columns of 256 features as 256 x 256 tiles, the others as tiles of
// 128 tokens
template <int YDT>
__global__ __launch_bounds__(512, 2) void fp8_halves_kernel(Fp8Args a, int f) {
  extern __shared__ uint4_t dsm[];
  char* const lds = reinterpret_cast<char*>(dsm);
  Fp8Args p = a;
  p.n = min(a.n, f * kHalvesN);
  if (p.n > 0) halves_tiles<YDT, 8>(p, lds);
  if (p.n < a.n) {
    Fp8Args r = a;
    r.n = a.n - p.n;
    r.w += (int64_t)p.n * a.k;
    r.sw += (int64_t)(p.n / kF8Block) * a.kb;
    r.y = static_cast<uint16_t*>(a.y) + p.n;
    halves_tiles<YDT, 4>(r, lds);
  }
}

template <int YDT>
hipError_t halves_launch(const Fp8Args& a, int f, hipStream_t s) {
  constexpr int bytes = 2 * halves_buf_bytes<8>();
  auto* kern = &fp8_halves_kernel<YDT>;
  static std::atomic<uint64_t> done{0};
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), bytes, done);
  if (e != hipSuccess) return e;
  kern<<<kCus, 512, bytes, s>>>(a, f);
  return hipGetLastError();
}

// y = the sum of the splits' totals, in their order; four are loaded before the
// first is added, so their latencies do not add up
template <int YDT>
__global__ __launch_bounds__(256) void fp8_join_kernel(const float* __restrict__ part, int splits,
                                                       int64_t count, void* y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  if (i + 4 <= count && (count & 3) == 0) {
    float4_t t = {0.0f, 0.0f, 0.0f, 0.0f};
    int s = 0;
    for (; s + 4 <= splits; s += 4) {
      float4_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const float4_t*>(part + (s + j) * count + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) t += v[j];
    }
    for (; s < splits; ++s) t += *reinterpret_cast<const float4_t*>(part + s * count + i);
    store4<YDT>(y, i, t, true, 4);
  } else {
    for (int64_t e = i; e < min(i + 4, count); ++e) {
      float t = part[e];
      for (int s = 1; s < splits; ++s) t += part[s * count + e];
      store1<YDT>(y, e, t);
    }
  }
}

template <int YDT, int TM, int NB>
hipError_t gemm_launch(const Fp8Args& a, hipStream_t s) {
  constexpr int bytes = NB * fp8_buf_bytes<TM>();
  auto* kern = &fp8_gemm_kernel<YDT, TM, NB>;
  static std::atomic<uint64_t> done{0};
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), bytes, done);
  if (e != hipSuccess) return e;
  const int tm = (a.m + TM * 32 - 1) / (TM * 32), tn = (a.n + kTileN - 1) / kTileN;
  kern<<<dim3((unsigned)(tm * tn), (unsigned)a.splits), 256, bytes, s>>>(a, tm, tn);
  return hipGetLastError();
}

template <int YDT>
hipError_t fp8_ydt(Fp8Args a, const Fp8Plan& p, hipStream_t s) {
  if (p.tile == 0) {
    // 16 features per workgroup.  Up to 256 of them (n <= 4096) a CU holds one,
    // which then needs all the waves it can have; with more, several should fit
    // a CU, whose LDS their rings share: one token 4096 x 4096 4.7 us with 16
    // waves, 5.1 with 8 (14336 rows: 10.5 and 10.3); 8 tokens 5.0 and 5.8; 16
    // tokens 11008 x 4096 11.8 and 10.2; 64 tokens 4096 x 4096 8.0 with 8, 8.7
    // with 5 waves, 5000 x 4096 12.2 and 11.0.  The exact products convert every
    // operand and want more waves: fp32 y 14336 x 4096 22.5 with 7, 26.8 with 5.
    // 40 tokens as three tiles of 16 14336 x 4096 16.8, as four 17.7.
    const bool few = a.n <= 4096;
    if (a.m == 1) return decode_launch<YDT, 16, 2, 0>(a, s);
    if (a.m <= 16)
      return few ? decode_launch<YDT, 16, 2, 1>(a, s) : decode_launch<YDT, 8, 2, 1>(a, s);
    if (a.m <= 32) return decode_launch<YDT, 8, 1, 2>(a, s);
    if (a.m <= 48) return decode_launch<YDT, 8, 1, 3>(a, s);
    return few ? decode_launch<YDT, 8, 1, 4>(a, s)
               : decode_launch<YDT, YDT == WQ_F32 ? 7 : 5, 1, 4>(a, s);
  }
  hipError_t e;
  if constexpr (YDT == WQ_F32) {
    e = gemm_launch<YDT, 4, 2>(a, s);
  } else {
    if (p.tile == 3) return halves_launch<YDT>(a, p.full, s);
    e = p.tile == 1 ? gemm_launch<YDT, 2, 6>(a, s) : gemm_launch<YDT, 4, 2>(a, s);
  }
  if (e != hipSuccess || a.part == nullptr) return e;
  const int64_t count = (int64_t)a.m * a.n;
  fp8_join_kernel<YDT><<<dim3((unsigned)((count + 1023) / 1024)), 256, 0, s>>>(a.part, a.splits,
                                                                              count, a.y);
  return hipGetLastError();
}

}  // namespace

Fp8Plan plan_fp8(int64_t m, int64_t n, int64_t k, int ydt) {
  Fp8Plan p{};
  p.splits = 1;
  const int64_t kb = (k + kF8Block - 1) / kF8Block;
  const bool exact = ydt == WQ_F32;
  // Few tokens: the weights stream past them (tile 0).  From 33 tokens on and
  // with many features tiles take less, except where they convert operands: 40
  // tokens 11008 x 4096 13.7 us against 14.6 in tiles, 14336 x 4096 16.8 and
  // 16.3; 64 tokens 8192 x 4096 12.6 and 14.6, 14336 x 4096 20.0 and 17.8; fp32
  // y 22.5 and 26.0.
  if (m <= 32 || (m <= 64 && (exact || n <= (m <= 48 ? 12288 : 8192)))) return p;
  const int64_t tn = (n + 127) / 128, t64 = (m + 63) / 64 * tn, t128 = (m + 127) / 128 * tn;
  // One round of tiles if 256 workgroups hold them, the smaller the better:
  // 512 tokens 4096 x 4096 20.0 us in 64 x 128 (tokens x features), 23.7 in
  // 128 x 128 tiles; 1000 tokens 35.3 and 27.8 us.  Past that the large tiles
  // (1536 tokens, 384 tiles of 128 x 128: 36 and 38 us).  The exact products
  // are bound by converting the operands, which small tiles share less.
  p.tile = !exact && t64 <= kCus ? 1 : exact || t128 <= kCus ? 2 : 3;
  if (p.tile < 3) {
    // few tiles: k in parts of at least four blocks
    const int64_t tiles = p.tile == 1 ? t64 : t128;
    int64_t s = std::max<int64_t>(1, kCus / tiles);
    s = std::min<int64_t>(s, std::max<int64_t>(1, kb / 4));
    while (s > 1 && s * m * n * 4 > ((int64_t)64 << 20)) --s;
    // no empty split
    const int64_t per = (kb + s - 1) / s;
    p.splits = (int)((kb + per - 1) / per);
    p.ws_bytes = p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0;
  } else {
    // whole rounds of 256 x 256 tiles, then half tiles if they fill one round
    const int64_t tm = (m + 255) / 256, tc = (n + 255) / 256;
    p.full = (int)(tm * tc / kCus * kCus / tm);
    if ((tc - p.full) * ((m + 127) / 128) > kCus) p.full = (int)tc;
  }
  return p;
}

hipError_t launch_linear_fp8(const uint8_t* x, const float* sx, int64_t m, const wq_weight* w,
                             void* y, int ydt, const Fp8Plan& plan, float* part, hipStream_t s) {
  const Fp8Args a{x, sx, static_cast<const uint8_t*>(w->codes),
                  static_cast<const float*>(w->scales), y, plan.splits > 1 ? part : nullptr,
                  (int)m, (int)w->n, (int)w->k, (int)((w->k + kF8Block - 1) / kF8Block),
                  plan.splits, (int)w->n};
  if (ydt == WQ_F32) return fp8_ydt<WQ_F32>(a, plan, s);
  if (ydt == WQ_BF16) return fp8_ydt<WQ_BF16>(a, plan, s);
  return fp8_ydt<WQ_F16>(a, plan, s);
}

}  // namespace wq
