// Causal attention of several tokens per sequence over a paged cache (formulas in wq.h).
//
// Bound by the matrix cores for long prompts, by HBM for a few rows behind a long
// context.  A workgroup takes rows of one sequence and kv head, a row being a token and
// one of the query heads that share the kv head, tokens outermost: all of them read the
// same keys and values, also where a chunk has few tokens.  Tiles of 64 visible tokens go
// through LDS, the next two on their way while one is computed; a wave has 32 rows.  With
// KS = 1 a workgroup is 256 rows, 128 for heads of 64, of which three fit into a CU.  With
// KS = 2 it is 128 rows, whose tiles two halves of its waves take in turn and whose sums
// they join at the end, without a way through HBM: so the longest row of a shorter prompt
// takes half as long.  Where that leaves CUs idle, parts of the tokens go to workgroups of
// their own (`splits`), and a second kernel joins them.
//
// S^T = K Q^T and O^T = V^T P^T on 32x32x16 matrix instructions: the sums of S^T leave a
// lane with one row and 16 tokens of each 32, so the softmax needs one exchange between
// two lanes, and the weights are the operand of P^T as they are, with the tokens of its
// k in the order in which the sums hold them.  V^T takes its tokens in the same order
// through the transposing LDS reads.
//
// LDS rows are whole heads; their 16-byte pieces are swapped by row (the loads into LDS
// fetch them in that order), so that no read meets more than its share of a bank.
//
// Measured, 32 heads on 8: 8192 tokens, heads of 128 520 us (1050 TFLOP/s at 2.0 GHz; the
// matrix cores are busy for half of the cycles and the vector units, a third of whose time
// is the exponentials, for the other: two waves of a SIMD are mostly in the same phase), from
// an E4M3 cache 610 (matrix cores 37% of the cycles, vector units 49), heads of 64 332 (half
// the products for the same weights: 39 and 67%); 64 tokens 9.3; 7 behind 30000 33 (3.7
// TB/s).  A wave with 64 rows, 512 registers and the scores of
// the next 32 tokens between the weights of the last ones reads LDS half as often, but has
// nobody beside it at barriers and loads: 585.  The same with 32 rows 572.
#include <algorithm>

#include "attention.h"

namespace wq {
namespace {

constexpr int kTile = 64;              // tokens of a tile
// In the place of a part's sum of weights: the workspace has no sums of it, as y is written
// (in the first part) or the part has no tiles.  What a part with tiles holds never decides
// whether it counts: NaN scores leave the maximum at -inf and reach y through the sums alone.
constexpr float kNoSums = -1.0f;
// Parts of `steps` steps of KS tiles, at most `splits`: as many as make the time of a part
// and of the parts' way through HBM least (about 2 us a step, and for 1e6 components of all
// rows; there are `million` times as many).  7 tokens behind 240, 370, 500 and 1000, 32 heads
// of 128: 10.5, 10.6, 10.5 and 11.4 us with parts of one step, 10.0, 11.8, 13.8 and 16.1 with
// at least three; 300 behind 1000, 8 heads of 64, twice: 23 with parts of one step, 17 so.
__host__ __device__ __forceinline__ int parts_of(int steps, int splits, float million) {
  return min(min(splits, steps), (int)sqrtf((float)steps / million));
}

struct PromptArgs {
  AttentionCall a;
  Divisor group;                       // query heads per kv head
  Divisor kv_heads;
  Divisor splits;                      // parts of the visible tokens, each a workgroup's
  float million;                       // components of all rows
  int longest_first;                   // the order of the workgroups; up to 64 sequences
  int tokens;                          // of a workgroup's rows, at least 1
  Divisor by_tokens;
  uint32_t page16, token16;            // strides in 16 bytes; a cache spans less than 2^31
};

// rows of sequence i: where they start in q, and how many
struct Rows {
  int start, n;
};
__device__ __forceinline__ Rows rows_of(const AttentionCall& a, int i) {
  const int m = (int)a.m;
  const int s = min(max(a.starts[i], 0), m), e = min(max(a.starts[i + 1], 0), m);
  return Rows{s, max(e - s, 0)};
}

// the same for an `i` that is the same in every lane
__device__ __forceinline__ Rows uniform_rows(const AttentionCall& a, int i) {
  const int m = (int)a.m;
  const int s = min(max(scalar_at(a.starts, i), 0), m);
  const int e = min(max(scalar_at(a.starts, i + 1), 0), m);
  return Rows{s, max(e - s, 0)};
}

// sum and largest over the wave, in every lane
__device__ __forceinline__ int sum_wave(int v) {
  uint32_t s = (uint32_t)v;
  s += dpp<0xB1>(s);
  s += dpp<0x4E>(s);
  s += dpp<0x141>(s);
  s += dpp<0x140>(s);
  return (__builtin_amdgcn_readlane((int)s, 0) + __builtin_amdgcn_readlane((int)s, 16)) +
         (__builtin_amdgcn_readlane((int)s, 32) + __builtin_amdgcn_readlane((int)s, 48));
}
__device__ __forceinline__ int max_wave(int v) {         // of values from 0 on
  const int s = (int)max16((uint32_t)v);
  return max(max(__builtin_amdgcn_readlane(s, 0), __builtin_amdgcn_readlane(s, 16)),
             max(__builtin_amdgcn_readlane(s, 32), __builtin_amdgcn_readlane(s, 48)));
}

template <int T>
__device__ __forceinline__ float16v_t mfma32(uint4_t a, uint4_t b, float16v_t c) {
  if constexpr (T == WQ_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// 16-byte piece of a row of LDS that holds piece 0: keys are read a piece of 16 rows at a
// time, values four pieces of 8 rows
template <int D>
__device__ __forceinline__ int key_swap(int row) {
  return D == 128 ? row & 15 : (row >> 1) & 7;
}
template <int D>
__device__ __forceinline__ int value_swap(int row) {
  return D == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

// four tokens of 16 components, transposed: lane i of 16 gets component i of each; and the
// four that are `more` bytes behind them
__device__ __forceinline__ uint4_t read_transposed(uint32_t at, uint32_t more) {
  typedef short short4v_t __attribute__((ext_vector_type(4)));
  using L = __attribute__((address_space(3))) short4v_t*;
  const short4v_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)at);
  const short4v_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(at + more));
  return __builtin_bit_cast(uint4_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// LDS by address: plain pointers into it take a check and an addition at each use
template <typename T>
__device__ __forceinline__ T lds_at(uint32_t at) {
  return *(const __attribute__((address_space(3))) T*)at;
}
template <typename T>
__device__ __forceinline__ void lds_put(uint32_t at, T v) {
  *(__attribute__((address_space(3))) T*)at = v;
}

// exponent bits of a 16-bit type: all set in infinities and NaN
template <int T>
constexpr uint32_t kExponent = T == WQ_BF16 ? 0x7F80u : 0x7C00u;

__device__ __forceinline__ float max_halves(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Row waves of a workgroup, 32 rows each.  For heads of 64 workgroups of four leave each
// other the matrix cores at their starts and ends (10001 tokens, window 1024, 16 heads: 78
// us, 101 with eight waves; 7 x 900 behind 500 28 and 38; 8192 tokens 342 and 343); heads of
// 128 have registers for eight waves a CU, which load a tile once (8192 tokens 516 us, 547
// with two workgroups of four).
template <int D, int KS>
constexpr int kRowWaves = D == 128 && KS == 1 ? 8 : 4;
// waves of a SIMD that registers are left for
template <int DT, int CT, int D, int KS>
constexpr int kWaves = D == 64 && KS == 1 && !(DT == WQ_F16 && CT == WQ_E4M3) ? 3 : 2;

template <int DT, int CT, int D, int KS>
__global__ __launch_bounds__(64 * KS * (kRowWaves<D, KS>), (kWaves<DT, CT, D, KS>))
void prompt_kernel(PromptArgs args) {
  constexpr bool F8 = CT == WQ_E4M3;
  constexpr int VT = F8 ? WQ_BF16 : DT;                  // type of the values' products
  constexpr bool TWO = F8 && DT == WQ_F16;               // weights in two parts of bf16
  // exponents as in the decode kernel: from a reference that lags the maximum by up to
  // 2^8 (8192 tokens 521 us, 544 without the lag); weights of f16 2^7 larger
  constexpr float kLag = 8.0f, kShift = VT == WQ_F16 ? 7.0f : 0.0f;
  constexpr int NW = kRowWaves<D, KS>, BM = NW * 32;     // row waves, rows
  constexpr int HT = 64 * NW, NT = HT * KS;              // threads that load a tile; all
  constexpr int RB = D * 2;                              // bytes of a row in LDS
  constexpr int KB = kTile * RB;                         // and of a tile
  constexpr int PC = D / 8;                              // 16-byte pieces of a row
  constexpr int NL = KB / 1024 / NW;                     // loads of 1 KB per wave and tile
  // tiles on their way while one is computed (two halves of D = 128 fill LDS with one; 8192
  // tokens 551 us with two tiles and the places of eight tiles' rows found at once, 641 with
  // one and a tile's)
  constexpr int AHEAD = KS == 2 && D == 128 ? 1 : 2, BUFS = AHEAD + 1;
  constexpr int NC = D / 16, NB = D / 32;                // k-steps of S^T, blocks of O^T
  const AttentionCall& a = args.a;
  const KvCache& cc = a.cache;
  const int tid = threadIdx.x, lane = tid & 63;
  const int all_wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = KS == 1 ? 0 : all_wave / NW, wave = all_wave - half * NW;
  const int ht = tid - half * HT;
  const int nl = lane & 31, hi = lane >> 5;

  extern __shared__ __align__(1024) char lds[];          // per half keys, values BUFS x KB each
  __shared__ int part[kLineWords<NT>];
  __shared__ __align__(16) float scales[KS][F8 ? BUFS : 1][F8 ? 2 : 1][F8 ? kTile : 1];
  __shared__ uint32_t odd[KS][2][2];

  // this workgroup's kv head, and its tile of rows: later rows of a sequence, which see
  // more, come first
  const int batch = (int)a.batch, group = (int)args.group.d;
  const int of_head = args.kv_heads.quotient(blockIdx.x), kh = blockIdx.x - of_head * cc.kv_heads;
  const int work = args.splits.quotient(of_head), split = of_head - work * (int)args.splits.d;
  auto tiles = [&](int i) { return (rows_of(a, i).n * group + BM - 1) / BM; };
  int seq = 0, nth = work;                               // of the sequence's tiles, last first
  if (KS == 1 && batch > 1 && args.longest_first) {
    // All sequences' tiles by decreasing tokens: those of a lane's sequence have `size`,
    // and BM / group less each.  The least x that at most `work` tiles pass, and of the
    // tiles of just x tokens the one in its turn.
    const int mine = min(lane, batch - 1), step = args.tokens;
    const int have = lane < batch ? tiles(mine) : 0;
    const int size = tokens_of(a, a.lens[mine]);
    auto longer = [&](int x) {
      return min(args.by_tokens.quotient(max(size - x + step - 1, 0)), have);
    };
    int lo = -1, hi = 0;                                   // keys below 0 count as 0: rows
    hi = max_wave(have > 0 ? size : 0);                    // before their sequence
    if (work >= sum_wave(have)) return;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sum_wave(longer(mid)) <= work) hi = mid; else lo = mid;
    }
    // (for x = -1 all that are there)
    const int above = longer(hi), with = lo < 0 ? have : longer(lo);
    int turn = work - sum_wave(above);
    uint64_t lanes = __ballot(with > above);
    if (hi == 0) {
      // several tiles of a sequence may be left, all of few tokens or none: in its order
      const int left = with - above, behind = scan64(left) - left;
      lanes = __ballot(lane < batch && behind <= turn && turn < behind + left);
      seq = __builtin_ctzll(lanes);
      nth = __builtin_amdgcn_readlane(above, seq) + turn - __builtin_amdgcn_readlane(behind, seq);
    } else {
      for (; turn > 0; --turn) lanes &= lanes - 1;
      seq = __builtin_ctzll(lanes);
      nth = __builtin_amdgcn_readlane(above, seq);
    }
  } else if (batch > 1) {
    const Line line = line_up<NT>(batch, part, tiles);
    if (work >= __builtin_amdgcn_readfirstlane(line.total)) return;
    int before;
    seq = __builtin_amdgcn_readfirstlane(line_find<NT>(batch, line, part, work, before, tiles));
    nth = work - __builtin_amdgcn_readfirstlane(before);
  }
  const Rows rows = uniform_rows(a, seq);
  const int count = rows.n * group;                      // of this sequence and kv head
  const int row_tile = (count + BM - 1) / BM - 1 - nth;
  if (row_tile < 0) return;
  const int len = tokens_of(a, scalar_at(a.lens, seq));
  const int before_rows = len - rows.n;                  // position of row 0; may be negative

  // this lane's row, and what the wave's and the workgroup's rows see
  const int r0 = row_tile * BM, rw = r0 + wave * 32, r = rw + nl;
  const bool live = r < count;
  const int token = args.group.quotient(min(r, count - 1));
  const int head = kh * group + min(r, count - 1) - token * group;
  const int pos = before_rows + token;
  // it sees the tokens [see, see + width) and those below `sunk`
  const int see = pos >= a.window ? pos - a.window + 1 : 0;
  const int width = max(pos + 1 - see, 0), sunk = min(a.sinks, max(pos + 1, 0));
  const int wave_lo = before_rows + args.group.quotient(min(rw, count - 1));
  const int wave_hi = before_rows + args.group.quotient(min(rw + 31, count - 1));
  const int wg_lo = max(before_rows + args.group.quotient(r0), 0);
  const int wg_hi = before_rows + args.group.quotient(min(r0 + BM - 1, count - 1));
  // the tokens that some row sees: as one row's, from the first row's window on
  Visible vis;
  vis.from = wg_lo >= a.window ? wg_lo - a.window + 1 : 0;
  vis.first = min(a.sinks, vis.from);
  vis.n = wg_hi < 0 ? 0 : wg_hi + 1 - vis.from + vis.first;
  auto token_at = [&](int i) { return i < vis.first ? i : i - vis.first + vis.from; };
  // Parts past the last one are empty (tiles are below 2^24, splits at most 64).  A single
  // part writes y itself, and kNoSums for the join: the host plans for what the page table
  // has room for (512 tokens in a table for 131072: 22 us, 24 through the workspace).
  const int all_tiles = (vis.n + kTile - 1) / kTile;
  const int parts = max(parts_of((all_tiles + KS - 1) / KS, (int)args.splits.d, args.million), 1);
  if (parts == 1 && split > 0) return;
  const int t_begin = split < parts ? all_tiles * split / parts : 0;
  const int t_end = split < parts ? all_tiles * (split + 1) / parts : 0;

  float16v_t o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[b][e] = 0.0f;
  float m = -INFINITY, l = 0.0f;

  if (t_begin < t_end) {
    // Q^T: lane (row nl, half hi) has 8 components of each k-step
    uint4_t q[NC];
    {
      const uint16_t* qp = a.q + (int64_t)(rows.start + token) * a.ldq + (int64_t)head * D + hi * 8;
#pragma unroll
      for (int c = 0; c < NC; ++c) q[c] = *reinterpret_cast<const uint4_t*>(qp + c * 16);
    }
    const float zscale = a.scale * kLog2e;
    const uint32_t kl = (uint32_t)(uintptr_t)(lds_void_t*)lds + half * 2 * BUFS * KB;
    const uint32_t vl = kl + BUFS * KB;

    // Tiles by what the wave's rows see of them: all of [whole0, whole1) and of those below
    // `sink_tiles`, nothing of [out0, out1) and from past1 on, and of the others each row
    // its own; from out0 on a tile is one stretch of tokens without a sink.  All rows of
    // the workgroup see all of [same0, same1).
    const int shift = vis.from - vis.first;                // token of visible i >= first
    const int sink_tiles = vis.first / kTile, one0 = (vis.first + kTile - 1) / kTile;
    const int whole0 = max(one0, ((wave_hi - a.window - shift) >> 6) + 1);
    const int whole1 = ((wave_lo - (kTile - 1) - shift) >> 6) + 1;
    const int out0 = max(one0, (a.sinks - shift + kTile - 1) >> 6);
    const int out1 = ((wave_lo - a.window - (kTile - 1) - shift) >> 6) + 1;
    const int past1 = rw < count ? ((wave_hi - shift) >> 6) + 1 : 0;
    const int same0 = max(one0, ((wg_hi - a.window - shift) >> 6) + 1);
    const int same1 = ((wg_lo - (kTile - 1) - shift) >> 6) + 2 - KS;

    // LDS addresses of this lane in a tile: of keys for the first k-step (that of step c is
    // this one xor 32 c), of values for the first 32 components (block b's: xor 64 b)
    const int ka = nl * RB + ((hi ^ key_swap<D>(nl)) << 4);
    const int vr = 4 * hi + ((lane & 15) >> 2);            // row within 8
    const int vp = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int va = vr * RB + ((vp ^ value_swap<D>(vr)) << 4) + 8 * (lane & 1);

    // A wave loads RW rows of each of its half's tiles.  Where they are in the cache is
    // found for GROUP tiles at once, a row in a lane, a group ahead of its use.
    constexpr int RW = 64 / NW, GROUP = 64 / RW;
    auto tile_of = [&](int i) { return t_begin + i * KS + half; };
    auto group_token = [&](int i) {                        // tiles i .. i + GROUP - 1
      return token_at(min(tile_of(i + lane / RW) * kTile + wave * RW + lane % RW, vis.n - 1));
    };
    int page = 0;
    uint32_t off = 0, off_scale = 0;                       // in 16 bytes; in scales
    auto look_up = [&](int i) {
      const auto k = args_here<PromptArgs>();
      const int32_t* table = k->a.pages + (int64_t)seq * k->a.ldp;
      page = table[group_token(i) >> k->a.cache.lg_page];
    };
    auto take_group = [&](int i) {                         // its pages are there
      const auto k = args_here<PromptArgs>();
      const int lg_page = k->a.cache.lg_page, place = group_token(i) & ((1 << lg_page) - 1);
      const uint32_t inside = (uint32_t)min(max(page, 0), k->a.cache.pages - 1);
      off = inside * k->page16 + (uint32_t)place * k->token16;
      if constexpr (F8)
        off_scale = ((inside * k->a.cache.kv_heads + kh) << lg_page) + place;
      look_up(i + GROUP);
    };
    // what a lane loads of its rows, 16 bits: one of PC pieces of NL rows, into LDS at once;
    // E4M3: CB codes of one row, which wait in registers until they are widened into LDS
    constexpr int CB = F8 ? D * RW / 64 : 16;
    uint32_t kc[CB / 4], vc[CB / 4];
    float sc = 0.0f;
    auto fetch = [&](const char* p, uint32_t (&c)[CB / 4]) {
      if constexpr (CB >= 16) {
#pragma unroll
        for (int w = 0; w < CB / 4; w += 4) {
          const uint4_t x = *reinterpret_cast<const uint4_t*>(p + 4 * w);
#pragma unroll
          for (int e = 0; e < 4; ++e) c[w + e] = x[e];
        }
      } else {
        const uint2_t x = *reinterpret_cast<const uint2_t*>(p);
        c[0] = x[0];
        c[1] = x[1];
      }
    };
    const char* const kbase = cc.k + kh * cc.head_stride;
    const char* const vbase = cc.v + kh * cc.head_stride;
    const float* const sbase = lane % GROUP == 0 ? cc.ks : cc.vs;
    auto load = [&](int i, int buf) {
      if (i % GROUP == 0) take_group(i);
      const int first = i % GROUP * RW;
      if constexpr (F8) {
        const int from = (first + lane / GROUP) * 4;       // GROUP threads per row
        const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)off) << 4;
        fetch(kbase + at + lane % GROUP * CB, kc);
        fetch(vbase + at + lane % GROUP * CB, vc);
        // the row's first two threads take the scales of its key and value
        sc = sbase[(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)off_scale)];
      } else {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int r = j * (1024 / RB) + lane / PC, row = wave * RW + r;
          const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(
                                  (first + r) * 4, (int)off) << 4;
          const int to = buf * KB + wave * RW * RB + j * 1024;
          lds_dma16(kbase + at + ((lane % PC ^ key_swap<D>(row)) << 4),
                    (lds_void_t*)(uintptr_t)(kl + to));
          lds_dma16(vbase + at + ((lane % PC ^ value_swap<D>(row)) << 4),
                    (lds_void_t*)(uintptr_t)(vl + to));
        }
      }
    };
    auto store = [&](int buf) {                            // E4M3: into LDS
      if constexpr (F8) {
        const int row = wave * RW + lane / GROUP;
#pragma unroll
        for (int w = 0; w < CB / 4; w += 2) {
          const uint2_t k0 = widen4<DT>(kc[w]), k1 = widen4<DT>(kc[w + 1]);
          const uint2_t v0 = widen4<VT>(vc[w]), v1 = widen4<VT>(vc[w + 1]);
          const int piece = lane % GROUP * (CB / 8) + w / 2, at = buf * KB + row * RB;
          lds_put(kl + at + ((piece ^ key_swap<D>(row)) << 4), uint4_t{k0[0], k0[1], k1[0], k1[1]});
          lds_put(vl + at + ((piece ^ value_swap<D>(row)) << 4),
                  uint4_t{v0[0], v0[1], v1[0], v1[1]});
        }
        // those of keys with the scale of z in them
        if (lane % GROUP < 2)
          scales[half][buf][lane % GROUP][row] = lane % GROUP == 0 ? sc * zscale : sc;
      }
    };

    // Values that are not finite would make NaN of the weights 0 of rows that do not see
    // them.  In steps where rows of the workgroup see different tokens, such values
    // become 0 in LDS and their tokens' bits are set in `odd`; the sums of the rows that do
    // see them get them by hand.
    auto clear_odd = [&](int buf, int step) {
#pragma unroll
      for (int i = 0; i < KB / 16 / HT; ++i) {
        const int at = (i * HT + ht) * 16;
        const uint32_t p = vl + buf * KB + at;
        uint4_t x = lds_at<uint4_t>(p);
        typedef unsigned short us2_t __attribute__((ext_vector_type(2)));
        us2_t top = {0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w)
          top = __builtin_elementwise_max(top, __builtin_bit_cast(us2_t, x[w] & 0x7FFF7FFFu));
        constexpr uint32_t kE = kExponent<VT>;
        if (top[0] >= kE || top[1] >= kE) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if ((x[w] & kE) == kE) x[w] &= 0xFFFF0000u;
            if ((x[w] >> 16 & kE) == kE) x[w] &= 0x0000FFFFu;
          }
          lds_put(p, x);
          atomicOr(&odd[half][step & 1][at / RB / 32], 1u << (at / RB % 32));
        }
      }
    };
    auto add_odd = [&](int t, int i) {                     // token i of the tile
      const auto k = args_here<PromptArgs>();
      const int tok = token_at(min(t * kTile + i, vis.n - 1));
      const bool ok = ((uint32_t)(tok - see) < (uint32_t)width) | (tok < sunk);
      const int place = tok & ((1 << k->a.cache.lg_page) - 1);
      const int32_t* row = k->a.pages + (int64_t)seq * k->a.ldp;
      const int at = min(max(scalar_at(row, tok >> k->a.cache.lg_page), 0), k->a.cache.pages - 1);
      const char* p = k->a.cache.v + kh * k->a.cache.head_stride + at * k->a.cache.page_stride +
                      place * k->a.cache.token_stride;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d0 = 32 * b + 8 * j + 4 * hi;
          uint2_t x;
          if constexpr (F8) x = widen4<VT>(*reinterpret_cast<const uint32_t*>(p + d0));
          else x = *reinterpret_cast<const uint2_t*>(p + 2 * d0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo, up;
            unpack2<VT>(x[e / 2], lo, up);
            const float f = e % 2 == 0 ? lo : up;
            if (ok && !(fabsf(f) < INFINITY)) o[b][4 * j + e] += f;
          }
          // the compiler would keep the results of all comparisons in scalar registers
          __builtin_amdgcn_sched_barrier(0);
        }
    };

    auto compute = [&](int t, int buf, int step, bool mixed) {
      if (t >= past1 || (t >= out0 && t < out1)) return;
      const bool whole = (t >= whole0 && t < whole1) || t < sink_tiles;
      float16v_t z[2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) z[b][e] = 0.0f;
      const uint32_t k = kl + buf * KB + ka, v = vl + buf * KB + va;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          z[b] = mfma32<DT>(lds_at<uint4_t>((k ^ (c << 5)) + b * 32 * RB), q[c], z[b]);
      // three k-steps of operands ahead of the products (8192 tokens 521 us, 527 in the
      // compiler's order)
      __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
      for (int c = 0; c < NC - 3; ++c) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
      // a wave of this SIMD that is past its scores goes before one that multiplies (8192
      // tokens 520 us, 527 without)
      __builtin_amdgcn_s_setprio(1);
      // scores in units of ln 2: 16 bits z * zscale; E4M3 z, with the scale of the key
      const float unit = F8 ? 1.0f : zscale;
      if constexpr (F8) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4_t ks =
                *reinterpret_cast<const float4_t*>(&scales[half][buf][0][32 * b + 8 * j + 4 * hi]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[b][4 * j + e] *= ks[e];
          }
      }
      if (!whole) {
        if (t >= out0) {
          const int x = t * kTile + shift + 4 * hi - see;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const bool ok = (uint32_t)(x + 32 * b + 8 * (e / 4) + e % 4) < (uint32_t)width;
              z[b][e] = ok ? z[b][e] : -INFINITY;
            }
        } else {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int tok = token_at(t * kTile + 32 * b + 8 * (e / 4) + 4 * hi + e % 4);
              const bool ok = ((uint32_t)(tok - see) < (uint32_t)width) | (tok < sunk);
              z[b][e] = ok ? z[b][e] : -INFINITY;
            }
        }
      }
      float big = z[0][0];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) big = fmaxf(big, z[b][e]);
      big = max_halves(big) * unit;
      if (__any(big > m + kLag)) {
        // each row by itself, so that it does not depend on the others
        const float mn = big > m + kLag ? big : m;
        const float fade = __builtin_amdgcn_exp2f(m - exp_ref(mn));
        m = mn;
        l *= fade;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[b][e] *= fade;
      }
      const float ref = exp_ref(m) - kShift;
      float sum = 0.0f;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          z[b][e] = __builtin_amdgcn_exp2f(F8 ? z[b][e] - ref : fmaf(z[b][e], unit, -ref));
          sum += z[b][e];
        }
      l += sum;
      if constexpr (F8) {
        // the scales of the values join the weights; where rows see different tokens, a
        // weight of 0 stays 0
        auto scale = [&](auto f) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4_t vs = *reinterpret_cast<const float4_t*>(
                  &scales[half][buf][1][32 * b + 8 * j + 4 * hi]);
#pragma unroll
              for (int e = 0; e < 4; ++e) z[b][4 * j + e] = f(z[b][4 * j + e], vs[e]);
            }
        };
        if (whole)
          scale([](float w, float s) { return w * s; });
        else
          scale([](float w, float s) { return w != 0.0f ? w * s : 0.0f; });
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // 16 tokens: weights of this lane's 8, rounded to the products' type: half a step
          // each, by chance up or down over the tokens, so y is 2.2e-3 of a row's norm off
          // in bf16 where its own rounding is 1.6e-3, and two parts would cost half of the
          // products again (8192 tokens 706 us, 526 with one).  Two parts where bf16 weights
          // meet an f16 y (codes and their scales: 792 us, 618 with one, but bf16's error)
          uint4_t p, rest;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float w0 = z[b][8 * s + 2 * w], w1 = z[b][8 * s + 2 * w + 1];
            p[w] = pack_weights<VT>(w0, w1);
            if constexpr (TWO) {
              float h0, h1;
              unpack2<VT>(p[w], h0, h1);
              rest[w] = pack_weights<VT>(w0 - h0, w1 - h1);
            }
          }
#pragma unroll
          for (int e = 0; e < NB; ++e) {
            const uint4_t x = read_transposed((v ^ (e << 6)) + (32 * b + 16 * s) * RB, 8 * RB);
            o[e] = mfma32<VT>(x, p, o[e]);
            if constexpr (TWO) o[e] = mfma32<VT>(x, rest, o[e]);
          }
        }
      __builtin_amdgcn_s_setprio(0);
      if (mixed) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t bits = __builtin_amdgcn_readfirstlane(odd[half][step & 1][w]);
          for (; bits != 0; bits &= bits - 1) add_odd(t, 32 * w + __builtin_ctz(bits));
        }
      }
    };

    // A step is KS tiles, one for each half; past the last one the half has none, and what
    // is loaded is not used.  16 bits: tile i + AHEAD is loaded in step i, once all waves are
    // done with tile i - 1, whose place it takes.  E4M3: tile i + 2 is fetched into registers
    // and tile i + 1 stored.
    const int steps = (t_end - t_begin + KS - 1) / KS;
    look_up(0);
    load(0, 0);
    if constexpr (F8) {
      store(0);
      load(1, 1);
    } else if constexpr (AHEAD == 2) {
      load(1, 1);
    }
    if (ht < 2) odd[half][0][ht] = 0;
    for (int step = 0, buf = 0; step < steps; ++step) {
      const int t = tile_of(step), next = buf + 1 == BUFS ? 0 : buf + 1;
      // this wave's loads of tile t are done (those of the next may go on); after the
      // barrier all waves'
      vm_wait<F8 ? 63 : (AHEAD - 1) * 2 * NL>();
      lgkm_wait0();
      wg_barrier();
      if constexpr (!F8) load(step + AHEAD, buf == 0 ? BUFS - 1 : buf - 1);
      const int t0 = t - half;
      const bool mixed = !((t0 >= same0 && t0 < same1) || t0 + KS <= sink_tiles);
      if (ht < 2) odd[half][(step + 1) & 1][ht] = 0;
      if (mixed) {
        clear_odd(buf, step);
        lgkm_wait0();
        wg_barrier();
      }
      if (t < t_end) compute(t, buf, step, mixed);
      if constexpr (F8) {
        store(next);
        load(step + 2, 0);
      }
      buf = next;
    }
    vm_wait<0>();                                          // nothing is on its way into LDS
  }

  l = sum_halves(l);
  const int64_t out = (int64_t)(rows.start + token) * args_here<PromptArgs>()->a.heads + head;
  if constexpr (KS == 2) {
    // the second half's sums join the first's, through the tiles' place in LDS: lane's
    // values next to each other over the lanes
    __syncthreads();
    float* x = reinterpret_cast<float*>(lds) + wave * (16 * NB + 2) * 64 + lane;
    if (half == 1) {
      x[0] = m;
      x[64] = l;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[(2 + 16 * b + e) * 64] = o[b][e];
    }
    __syncthreads();
    if (half == 1) return;
    const float om = x[0], mn = fmaxf(m, om), ref = exp_ref(mn);
    const float f = __builtin_amdgcn_exp2f(m - ref), g = __builtin_amdgcn_exp2f(om - ref);
    m = mn;
    l = l * f + x[64] * g;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[b][e] = o[b][e] * f + x[(2 + 16 * b + e) * 64] * g;
  }
  const auto k = args_here<PromptArgs>();
  if (k->splits.d > 1) {
    // m, l and the sums of this part
    const int64_t total = k->a.m * k->a.heads;
    float* ml = k->a.ws + (int64_t)k->splits.d * total * D + (split * total + out) * 2;
    if (live && hi == 0) {
      ml[0] = m;
      ml[1] = parts == 1 || split >= parts ? kNoSums : l;
    }
    if (parts > 1) {
      if (!live || split >= parts) return;
      float* w = k->a.ws + (split * total + out) * D;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4_t*>(w + 32 * b + 8 * j + 4 * hi) =
              float4_t{o[b][4 * j], o[b][4 * j + 1], o[b][4 * j + 2], o[b][4 * j + 3]};
      return;
    }
  }
  const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      // this half's 4 components of two groups of 8; after the swap 8 of one group
      uint32_t w[2][2];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[g][e] = pack2<DT>(o[b][4 * (j + g) + 2 * e] * inv, o[b][4 * (j + g) + 2 * e + 1] * inv);
      auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
      auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
      if (live)
        *reinterpret_cast<uint4_t*>(k->a.y + out * D + 32 * b + 8 * (j + hi)) =
            uint4_t{s0[0], s1[0], s0[1], s1[1]};
    }
  if (k->a.lse != nullptr && live && hi == 0)
    k->a.lse[out] = l == 0.0f ? -INFINITY : (m - kShift + __builtin_amdgcn_logf(l)) * kLn2;
}

// Joins the parts of a row and head: G groups of D / 4 threads take them in turn, four
// loaded together.
template <int DT, int D, int G>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptArgs args, float shift) {
  constexpr int L = D / 4, U = 4;
  constexpr int kPer = 256 / (L * G);                    // rows and heads of a workgroup
  const AttentionCall& a = args.a;
  const int splits = (int)args.splits.d;
  const int who = threadIdx.x / (L * G), g = threadIdx.x / L % G, c = threadIdx.x % L;
  const int64_t total = a.m * a.heads;
  const int64_t out = min((int64_t)blockIdx.x * kPer + who, total - 1), row = out / a.heads;
  const bool live = (int64_t)blockIdx.x * kPer + who < total && row >= a.starts[0] &&
                    row < a.starts[a.batch];
  const float* ml = a.ws + (int64_t)splits * total * D;
  const bool done = ml[2 * out + 1] == kNoSums;
  float m = -INFINITY, l = 0.0f;
  float4_t x = {0, 0, 0, 0};
  for (int s0 = g; s0 < splits; s0 += U * G) {
    float pm[U], pl[U];
    float4_t px[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t at = min(s0 + i * G, splits - 1) * total + out;
      pm[i] = ml[2 * at];
      pl[i] = ml[2 * at + 1];
      px[i] = *reinterpret_cast<const float4_t*>(a.ws + at * D + c * 4);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool some = s0 + i * G < splits && pl[i] != kNoSums;
      const float mn = some ? fmaxf(m, pm[i]) : m, ref = exp_ref(mn);
      const float fade = __builtin_amdgcn_exp2f(m - ref);
      const float f = some ? __builtin_amdgcn_exp2f(pm[i] - ref) : 0.0f;
      l = l * fade + (some ? pl[i] * f : 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = x[e] * fade + (some ? px[i][e] * f : 0.0f);
      m = mn;
    }
  }
  if constexpr (G > 1) {
    __shared__ __align__(16) float sx[kPer][G][D];
    __shared__ float sm[kPer][G], sl[kPer][G];
    *reinterpret_cast<float4_t*>(&sx[who][g][c * 4]) = x;
    if (c == 0) {
      sm[who][g] = m;
      sl[who][g] = l;
    }
    __syncthreads();
    if (g != 0) return;
    float big = m;
#pragma unroll
    for (int i = 1; i < G; ++i) big = fmaxf(big, sm[who][i]);
    x = float4_t{0, 0, 0, 0};
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float f = __builtin_amdgcn_exp2f(sm[who][i] - exp_ref(big));
      l += sl[who][i] * f;
      x += f * *reinterpret_cast<const float4_t*>(&sx[who][i][c * 4]);
    }
    m = big;
  }
  if (!live || done) return;
  const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
  *reinterpret_cast<uint2_t*>(a.y + out * D + c * 4) =
      uint2_t{pack2<DT>(x[0] * inv, x[1] * inv), pack2<DT>(x[2] * inv, x[3] * inv)};
  if (a.lse != nullptr && c == 0)
    a.lse[out] = l == 0.0f ? -INFINITY : (m - shift + __builtin_amdgcn_logf(l)) * kLn2;
}

float millions(int64_t m, int64_t heads, const KvCache& c) {
  return (float)(m * heads * c.d) * 1e-6f;
}

struct PromptPlan {
  int halves, splits;                  // KS, and parts of the tokens
  int64_t tiles;                       // of rows, at most
};
// `most`: tokens that a row can see
PromptPlan plan_prompt(int64_t m, int64_t heads, int64_t batch, const KvCache& c, int64_t most) {
  const int64_t rows = m * (heads / c.kv_heads);
  auto tiles = [&](int64_t bm) {
    return batch == 1 ? (rows + bm - 1) / bm : rows / bm + std::min(batch, m);
  };
  // More than a round of workgroups of all eight waves: KS = 1, which reads each tile for
  // twice the rows (32 heads on 8 of 128, KS = 1 | 2: 2600 tokens 79 | 89 us, 8 x 300 25 | 37,
  // 8 x 200 behind 3000 108 | 126).  One round or less: 128 rows, of which the short ones of
  // a causal prompt run beside the long ones (2048 tokens 65 | 60, 1024 behind 8000 221 |
  // 160; only just one round behind a long context loses, 2048 behind 8000 302 | 328).
  // Heads of 64, workgroups of four waves: from one and a half a CU on (1500 tokens 29 | 23,
  // 30 x 4 behind 2000 38 | 30, 4000 tokens, window 1024, 16 heads, E4M3 47 | 55).
  PromptPlan p{1, 1, tiles(c.d == 128 ? 256 : 128)};
  if (p.tiles * c.kv_heads > (c.d == 128 ? 256 : 384)) return p;
  p = PromptPlan{2, 1, tiles(128)};
  // parts that fill the GPU once, by the tiles that there are in earnest
  const int64_t wgs = std::max((rows + 127) / 128, std::min(batch, m)) * c.kv_heads;
  const int64_t steps = (most + 2 * kTile - 1) / (2 * kTile);
  const float million = millions(m, heads, c);
  const int n = parts_of((int)steps, (int)std::min<int64_t>(64, 256 / wgs), million);
  // where they save more than the join costs (100 behind 500, 32 heads of 128, 19.1 us in two
  // parts and 18.0 in one; 512 behind 2000 42 and 50)
  if (n > 1 && steps - (steps + n - 1) / n > 1.5f + 1.5f * million * n) p.splits = n;
  return p;
}

template <int DT, int CT, int D, int KS>
hipError_t prompt_go(const AttentionCall& a, const PromptPlan& p, hipStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr int kRows = 32 * kRowWaves<D, KS>;
  // tiles as in the kernel, and the place where two halves join
  constexpr int kBufs = KS == 2 && D == 128 ? 2 : 3;
  constexpr int kLds =
      std::max(KS * 2 * kBufs * kTile * D * 2, KS == 2 ? 4 * (D / 2 + 2) * 256 : 0);
  const auto kern = prompt_kernel<DT, CT, D, KS>;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), kLds, done);
  if (e != hipSuccess) return e;
  const int64_t wgs = p.tiles * p.splits * a.cache.kv_heads;
  const uint32_t group = (uint32_t)(a.heads / a.cache.kv_heads);
  const uint32_t tokens = std::max<uint32_t>(kRows / group, 1);
  // Past one round of workgroups the order matters: 11 prompts of 5730 tokens, 4 heads, 519
  // us in the sequences' order and 447 by length; 11 of 2000, 32 heads, 435 and 440, what
  // finding it costs.  Rounds of shorter workgroups gain nothing (16 sequences of 4 rows 59
  // and 62).
  const bool longest_first = KS == 1 && a.batch > 1 && a.batch <= 64;
  const PromptArgs args{a, Divisor::of(group), Divisor::of((uint32_t)a.cache.kv_heads),
                        Divisor::of((uint32_t)p.splits),
                        millions(a.m, a.heads, a.cache), longest_first, (int)tokens,
                        Divisor::of(tokens),
                        (uint32_t)(a.cache.page_stride >> 4),
                        (uint32_t)(a.cache.token_stride >> 4)};
  kern<<<dim3((unsigned)wgs), kRows / 32 * 64 * KS, kLds, s>>>(args);
  e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  constexpr float kShift = CT != WQ_E4M3 && DT == WQ_F16 ? 7.0f : 0.0f;
  // Many parts of few rows: eight groups of a workgroup's threads share them, where one
  // group for each row would leave most CUs idle (2 tokens behind 8000 15 us, 19 with one
  // group a row; 33 behind 700, 56 heads, 19.8 and 18.7).
  const int64_t total = a.m * a.heads;
  if (p.splits > 4 && total * (D / 4) < 256 * 64) {
    const int64_t per = 32 / (D / 4);
    const dim3 grid((unsigned)((total + per - 1) / per));
    prompt_join_kernel<DT, D, 8><<<grid, 256, 0, s>>>(args, kShift);
  } else {
    const int64_t per = 256 / (D / 4);
    const dim3 grid((unsigned)((total + per - 1) / per));
    prompt_join_kernel<DT, D, 1><<<grid, 256, 0, s>>>(args, kShift);
  }
  return hipGetLastError();
}
template <int DT, int CT, int D>
hipError_t prompt_ks(const AttentionCall& a, hipStream_t s) {
  const PromptPlan p = plan_prompt(
      a.m, a.heads, a.batch, a.cache, a.max_pages << a.cache.lg_page);
  return p.halves == 1 ? prompt_go<DT, CT, D, 1>(a, p, s) : prompt_go<DT, CT, D, 2>(a, p, s);
}
template <int DT, int D>
hipError_t prompt_ct(const AttentionCall& a, hipStream_t s) {
  return a.cache.dt == WQ_E4M3 ? prompt_ks<DT, WQ_E4M3, D>(a, s) : prompt_ks<DT, DT, D>(a, s);
}
template <int DT>
hipError_t prompt_d(const AttentionCall& a, hipStream_t s) {
  return a.cache.d == 128 ? prompt_ct<DT, 128>(a, s) : prompt_ct<DT, 64>(a, s);
}

}  // namespace

// What a call of m or fewer rows can need: its parts are at most 64, and with wgs workgroups
// of 128 rows or less, at least m * heads / 128 of them, at most 256 / wgs.
size_t prompt_ws_bytes(int64_t m, int64_t heads, const KvCache& c) {
  const int64_t parts = std::min(64, 256 / c.kv_heads);
  if (parts < 2) return 0;
  return (size_t)std::min<int64_t>(parts * m * heads, 256 * 128) * (c.d + 2) * sizeof(float);
}

int64_t prompt_wgs(int64_t m, int64_t heads, int64_t batch, const KvCache& c) {
  const PromptPlan p = plan_prompt(m, heads, batch, c, int64_t(1) << 30);
  return p.tiles * p.splits * c.kv_heads;
}

hipError_t launch_attention_prompt(const AttentionCall& a, hipStream_t s) {
  return a.dt == WQ_BF16 ? prompt_d<WQ_BF16>(a, s) : prompt_d<WQ_F16>(a, s);
}

}  // namespace wq
