// Attention of one new token per sequence over a paged cache (formulas in wq.h).
//
// The keys and values that are seen are read once, so the kernel is bound by HBM, and
// by the latency of its chain (lens, page table, keys, values, join) for short ones.
//
// Split.  An item is a sequence, a kv head and up to 16 of its query heads; a unit is
// 128 visible tokens of an item.  The units of all items stand in one line, and every
// workgroup takes an equal stretch of it, found from lens on the device: one long
// sequence, many short ones and any mixture load all CUs alike, also where a captured
// call is replayed with other lens.  A stretch that covers a whole item writes y; parts
// of items go to the workspace (at most one that ends and one that goes on per
// workgroup), and a second kernel joins them.
//
// One wave takes 32 tokens a step.  S^T = K Q^T and O^T = V^T P^T on 16x16x32 matrix
// instructions: the sums of S^T leave a lane with one query head and 8 tokens, which is
// the operand P^T wants, so the weights never move between lanes.  Keys are loaded with
// a row's pieces in adjacent lanes and reordered by lane permutes; a lane's values are
// the same D / 16 components of its 8 tokens, transposed in registers.  The loads of
// the next step are in flight while one is computed, its page numbers one step more.
#include <algorithm>

#include "attention.h"

namespace wq {
namespace {

constexpr int kUnit = 128;             // tokens of a unit: 4 waves of 32
constexpr int kRows = 16;              // query heads of an item

struct DecodeArgs {
  AttentionCall a;
  int group, tiles;                    // query heads per kv head; items of 16 of them
};

// where the visible units of the sequences stand in the line
struct Line {
  int64_t total;                       // units of all sequences, per kv head and tile
  int64_t before;                      // units before the sequence found
  int64_t seq;                         // the sequence that holds unit `want`
};

__device__ __forceinline__ Visible decode_visible(const AttentionCall& a, int64_t seq) {
  return visible_of(tokens_of(a, seq) - 1, a.window, a.sinks);
}
__device__ __forceinline__ int units_of(const Visible& v) { return (v.n + kUnit - 1) / kUnit; }

// units per sequence summed over the threads' blocks of sequences; part[t]: the units
// before thread t's block
__device__ __forceinline__ int64_t line_sums(const AttentionCall& a, int64_t* part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t per = (a.m + 255) / 256, i0 = tid * per, i1 = min(i0 + per, a.m);
  int64_t own = 0;
  for (int64_t i = i0; i < i1; ++i) own += units_of(decode_visible(a, i));
  int64_t sum = own;
#pragma unroll
  for (int w = 1; w < 64; w *= 2) {
    const int64_t up = __shfl_up(sum, w);
    if (lane >= w) sum += up;
  }
  if (lane == 63) part[256 + wave] = sum;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) base += part[256 + w];
    total += part[256 + w];
  }
  part[tid] = base + sum - own;
  __syncthreads();
  return total;
}

// the sequence that holds unit `want` (below the total) of the line
__device__ __forceinline__ Line line_find(const AttentionCall& a, const int64_t* part,
                                          int64_t total, int64_t want) {
  int t = 0;                           // the last block that starts at or before it
#pragma unroll
  for (int w = 128; w > 0; w /= 2)
    if (part[t + w] <= want) t += w;
  const int64_t per = (a.m + 255) / 256;
  // blocks past the last sequence start at the total, which is past `want`; blocks of
  // no units share their start with the next, so this one holds it
  int64_t seq = t * per, before = part[t];
  for (;;) {
    const int n = units_of(decode_visible(a, seq));
    if (before + n > want || seq + 1 >= a.m) break;
    before += n;
    ++seq;
  }
  return Line{total, before, seq};
}

template <int CT, int D>
struct Tile {
  static constexpr int E = CT == WQ_E4M3 ? 1 : 2;        // bytes of a component
  static constexpr int KC = D * E / 64;                  // 64-byte pieces of a key
  static constexpr int VW = D * E / 64;                  // words of a lane's part of a value
  uint4_t k[2][KC];
  uint32_t v[8][VW];
  float scale;                                           // lanes 0-31 of keys, 32-63 of values
};

template <int W>
__device__ __forceinline__ void load_words(const char* p, uint32_t (&r)[W]) {
  if constexpr (W == 4) {
    const uint4_t t = *reinterpret_cast<const uint4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = t[i];
  } else if constexpr (W == 2) {
    const uint2_t t = *reinterpret_cast<const uint2_t*>(p);
    r[0] = t[0];
    r[1] = t[1];
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int DT, int CT, int D>
__global__ __launch_bounds__(256, 2) void decode_kernel(DecodeArgs args) {
  constexpr bool F8 = CT == WQ_E4M3;
  constexpr int VT = F8 ? WQ_BF16 : DT;                  // type of the values' products
  // weights of f16 are kept 2^15 larger, away from its subnormal range
  constexpr float kShift = VT == WQ_F16 ? 15.0f : 0.0f;
  constexpr int KC = Tile<CT, D>::KC, VW = Tile<CT, D>::VW;
  constexpr int NI = D / 16;                             // O^T tiles, components of a lane
  constexpr int OS = D + 4;                              // LDS row of O, in floats
  const AttentionCall& a = args.a;
  const KvCache& cc = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nl = lane & 15, kq = lane >> 4;

  __shared__ int64_t part[260];
  __shared__ __align__(16) float so[4 * kRows * OS];
  __shared__ float sm[4][kRows], sl[4][kRows];

  const int64_t per_unit = (int64_t)cc.kv_heads * args.tiles;
  const int64_t total = line_sums(a, part);
  const int64_t line = total * per_unit;

  // rows that see nothing are in no unit
  for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) {
    if (decode_visible(a, i).n > 0) continue;
    for (int64_t e = tid; e < a.heads * (D / 8); e += 256)
      reinterpret_cast<uint4_t*>(a.y)[i * a.heads * (D / 8) + e] = uint4_t{0, 0, 0, 0};
    if (a.lse != nullptr)
      for (int64_t e = tid; e < a.heads; e += 256) a.lse[i * a.heads + e] = -INFINITY;
  }

  const int64_t wgs = min((int64_t)gridDim.x, line);     // none without a unit
  if (blockIdx.x >= wgs) return;
  int64_t u = line * blockIdx.x / wgs;
  const int64_t u_end = line * (blockIdx.x + 1) / wgs;
  const Line at = line_find(a, part, total, u / per_unit);
  int64_t seq = at.seq, item0 = at.before * per_unit;    // the line's unit where seq starts

  while (u < u_end) {
    const Visible vis = decode_visible(a, seq);
    const int units = units_of(vis);
    if (u >= item0 + units * per_unit) {
      item0 += units * per_unit;
      ++seq;
      continue;
    }
    const int sub = (int)((u - item0) / units);          // kv head and tile of query heads
    const int kh = sub / args.tiles, ht = sub - kh * args.tiles;
    const int64_t first = item0 + (int64_t)sub * units;  // the item's first unit
    const int ua = (int)(u - first), ub = (int)min((int64_t)units, u_end - first);
    const int rows = min(kRows, args.group - ht * kRows);
    const int64_t head0 = (int64_t)kh * args.group + ht * kRows;

    // Q^T: lane (row nl, piece kq); rows past the group are zeros
    uint4_t q[D / 32];
    {
      const uint16_t* qp = a.q + seq * a.ldq + (head0 + min(nl, rows - 1)) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const int d0 = F8 ? 64 * (c / 2) + 16 * kq + 8 * (c % 2) : 32 * c + 8 * kq;
        q[c] = *reinterpret_cast<const uint4_t*>(qp + d0);
        if (nl >= rows) q[c] = uint4_t{0, 0, 0, 0};
      }
    }
    const int32_t* table = a.pages + seq * a.ldp;
    const char* kbase = cc.k + kh * cc.head_stride;
    const char* vbase = cc.v + kh * cc.head_stride;
    const float* scales = lane < 32 ? cc.ks : cc.vs;

    const int begin = ua * kUnit + wave * 32, end = min(ub * kUnit, vis.n);
    const int steps = begin < end ? (end - begin + kUnit - 1) / kUnit : 0;

    // token of this lane in a step: lanes 0-31 and 32-63 the 32 tokens
    auto token = [&](int step) {
      const int i = min(begin + step * kUnit + (lane & 31), end - 1);
      return i < vis.first ? i : i - vis.first + vis.from;
    };
    auto load = [&](Tile<CT, D>& t, int step, int page) {
      const int place = token(step) & ((1 << cc.lg_page) - 1);
      // 16-byte units: a cache spans at most 2^34 elements
      const uint32_t off = (uint32_t)((page * cc.page_stride + place * cc.token_stride) >> 4);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * s + (lane >> 2)) * 4,
                                                                  (int)off);
        const char* p = kbase + ((uint64_t)o << 4) + (lane & 3) * 16;
#pragma unroll
        for (int c = 0; c < KC; ++c)
          t.k[s][c] = *reinterpret_cast<const uint4_t*>(p + c * 64);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int from = (i < 4 ? 4 * kq + i : 12 + 4 * kq + i) * 4;
        const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)off);
        load_words<VW>(vbase + ((uint64_t)o << 4) + nl * (VW * 4), t.v[i]);
      }
      if constexpr (F8)
        t.scale = scales[(((int64_t)page * cc.kv_heads + kh) << cc.lg_page) + place];
    };

    float m = -INFINITY, l = 0.0f;
    float4_t o[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) o[i] = float4_t{0, 0, 0, 0};
    const float zscale = a.scale * kLog2e;

    auto compute = [&](Tile<CT, D>& t, int step) {
      float z[8];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float4_t acc = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4_t k = operand_order(t.k[s][c]);
          if constexpr (F8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2_t lo = widen4<DT>(k[2 * h]), hi = widen4<DT>(k[2 * h + 1]);
              acc = mfma16<DT>(uint4_t{lo[0], lo[1], hi[0], hi[1]}, q[2 * c + h], acc);
            }
          } else {
            acc = mfma16<DT>(k, q[c], acc);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) z[4 * s + r] = acc[r] * zscale;
      }
      const int base = begin + step * kUnit + 4 * kq;
      float vs[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = i < 4 ? i : 12 + i;              // from 4 kq on
        if constexpr (F8) {
          const int from = (4 * kq + tok) * 4;
          z[i] *= __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(t.scale)));
          vs[i] = __int_as_float(__builtin_amdgcn_ds_bpermute(from + 128,
                                                              __float_as_int(t.scale)));
        }
        z[i] = base + tok < end ? z[i] : -INFINITY;
      }
      float big = z[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) big = fmaxf(big, z[i]);
      const float mn = fmaxf(m, max_quarters(big)), ref = exp_ref(mn) - kShift;
      const float fade = __builtin_amdgcn_exp2f(m - (ref + kShift));
      m = mn;
      float p[8], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(z[i] - ref);
        sum += p[i];
      }
      l = l * fade + sum;
#pragma unroll
      for (int i = 0; i < NI; ++i) o[i] *= fade;
      if constexpr (F8) {
        // a token past the end repeats the last one, whose scale may not be finite
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = base + (i < 4 ? i : 12 + i) < end ? p[i] * vs[i] : 0.0f;
      }
      // two parts of 8 (bf16) or 11 bits: against one part, whose rounding is as large as
      // that of a 16-bit y, this costs matrix instructions that wait for HBM anyway
      uint4_t hi, lo;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        hi[w] = pack2<VT>(p[2 * w], p[2 * w + 1]);
        float h0, h1;
        unpack2<VT>(hi[w], h0, h1);
        lo[w] = pack2<VT>(p[2 * w] - h0, p[2 * w + 1] - h1);
      }
      // 16-bit values of the 8 tokens, D / 16 components each
      uint32_t vv[8][NI / 2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (F8) {
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const uint2_t x = widen4<VT>(t.v[i][w]);
            vv[i][2 * w] = x[0];
            vv[i][2 * w + 1] = x[1];
          }
        } else {
#pragma unroll
          for (int w = 0; w < VW; ++w) vv[i][w] = t.v[i][w];
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint4_t x;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          x[w] = __builtin_amdgcn_perm(vv[2 * w + 1][i / 2], vv[2 * w][i / 2],
                                       i % 2 == 0 ? 0x05040100u : 0x07060302u);
        o[i] = mfma16<VT>(x, hi, o[i]);
        o[i] = mfma16<VT>(x, lo, o[i]);
      }
    };

    if (steps > 0) {
      Tile<CT, D> t0, t1;
      int page = page_of(a, table, token(0));
      int next = page_of(a, table, token(1));
      load(t0, 0, page);
      for (int s = 0; s < steps; s += 2) {
        page = next;
        next = page_of(a, table, token(s + 2));
        load(t1, s + 1, page);
        compute(t0, s);
        page = next;
        next = page_of(a, table, token(s + 3));
        load(t0, s + 2, page);
        compute(t1, s + 1);                              // past the end: all masked
      }
    }
    l = sum_quarters(l);

    // join the four waves
    if (kq == 0) {
      sm[wave][nl] = m;
      sl[wave][nl] = l;
    }
    __syncthreads();
    float mx = sm[0][nl];
#pragma unroll
    for (int w = 1; w < 4; ++w) mx = fmaxf(mx, sm[w][nl]);
    const float f = __builtin_amdgcn_exp2f(m - exp_ref(mx));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // components (D / 16) (4 kq + r) + i of row nl
      float* p = so + (wave * kRows + nl) * OS + NI * (4 * kq + r);
#pragma unroll
      for (int i = 0; i < NI; i += 4)
        *reinterpret_cast<float4_t*>(p + i) =
            float4_t{o[i][r] * f, o[i + 1][r] * f, o[i + 2][r] * f, o[i + 3][r] * f};
    }
    __syncthreads();
    const bool whole = ua == 0 && ub == units;
    float* slot = a.ws + (2 * (int64_t)blockIdx.x + (ub < units ? 1 : 0)) * (kRows * (D + 2));
    for (int e = tid; e < rows * (D / 8); e += 256) {
      const int row = e / (D / 8), c = e % (D / 8);
      float big = sm[0][row], sum = 0.0f, v[8];
#pragma unroll
      for (int w = 1; w < 4; ++w) big = fmaxf(big, sm[w][row]);
#pragma unroll
      for (int w = 0; w < 4; ++w)
        sum += sl[w][row] * __builtin_amdgcn_exp2f(sm[w][row] - exp_ref(big));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += so[(w * kRows + row) * OS + c * 8 + i];
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        const int64_t out = seq * a.heads + head0 + row;
        *reinterpret_cast<uint4_t*>(a.y + out * D + c * 8) = pack8<DT>(v);
        if (a.lse != nullptr && c == 0)
          a.lse[out] = sum == 0.0f ? -INFINITY
                                   : (big - kShift + __builtin_amdgcn_logf(sum)) * kLn2;
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          *reinterpret_cast<float4_t*>(slot + row * D + c * 8 + i) =
              float4_t{v[i], v[i + 1], v[i + 2], v[i + 3]};
        if (c == 0) {
          slot[kRows * D + row] = big;
          slot[kRows * (D + 1) + row] = sum;
        }
      }
    }
    __syncthreads();
    u = first + ub;
  }
}

// One workgroup per row and query head: the parts of its item, in the line's order.
template <int DT, int D>
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs args, int most, float shift) {
  const AttentionCall& a = args.a;
  const int tid = threadIdx.x;
  __shared__ int64_t part[260];
  __shared__ float weight[kDecodeMaxWgs + 1];
  __shared__ float red[8];
  __shared__ __align__(16) float so[256 / (D / 4)][D];
  const int64_t seq = blockIdx.x;
  const int head = blockIdx.y, kh = head / args.group;
  const int ht = (head - kh * args.group) / kRows, row = (head - kh * args.group) % kRows;
  const int units = units_of(decode_visible(a, seq));
  if (units == 0) return;
  const int64_t total = line_sums(a, part);
  const int64_t per_unit = (int64_t)a.cache.kv_heads * args.tiles, line = total * per_unit;
  const int64_t wgs = min((int64_t)most, line);
  // units before this sequence: its block's, then the sequences of the block
  const int64_t per = (a.m + 255) / 256;
  int64_t before = part[seq / per];
  for (int64_t i = seq / per * per; i < seq; ++i) before += units_of(decode_visible(a, i));
  const int64_t first = before * per_unit + (int64_t)(kh * args.tiles + ht) * units;
  const int64_t last = first + units - 1;
  const int w0 = (int)(((first + 1) * wgs - 1) / line), w1 = (int)(((last + 1) * wgs - 1) / line);
  if (w0 == w1) return;                                  // one workgroup had it whole
  const int n = w1 - w0 + 1;
  auto slot = [&](int i) {
    return a.ws + (2 * (int64_t)(w0 + i) + (i + 1 < n ? 1 : 0)) * (kRows * (D + 2));
  };
  float big = -INFINITY;
  for (int i = tid; i < n; i += 256) {
    const float v = slot(i)[kRows * D + row];
    weight[i] = v;
    big = fmaxf(big, v);
  }
#pragma unroll
  for (int w = 1; w < 64; w *= 2) big = fmaxf(big, __shfl_xor(big, w));
  if ((tid & 63) == 0) red[tid >> 6] = big;
  __syncthreads();
  big = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float sum = 0.0f;
  for (int i = tid; i < n; i += 256) {
    const float f = __builtin_amdgcn_exp2f(weight[i] - exp_ref(big));
    weight[i] = f;
    sum += f * slot(i)[kRows * (D + 1) + row];
  }
  sum = sum64(sum);
  if ((tid & 63) == 0) red[4 + (tid >> 6)] = sum;
  __syncthreads();
  sum = (red[4] + red[5]) + (red[6] + red[7]);
  constexpr int L = D / 4, G = 256 / L;
  const int c = tid % L, g = tid / L;
  float4_t v = {0, 0, 0, 0};
#pragma unroll 4
  for (int i = g; i < n; i += G)
    v += weight[i] * *reinterpret_cast<const float4_t*>(slot(i) + row * D + c * 4);
  *reinterpret_cast<float4_t*>(&so[g][c * 4]) = v;
  __syncthreads();
  if (tid >= D / 8) return;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += so[i][tid * 8 + e];
  const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  const int64_t out = seq * a.heads + head;
  *reinterpret_cast<uint4_t*>(a.y + out * D + tid * 8) = pack8<DT>(x);
  if (a.lse != nullptr && tid == 0)
    a.lse[out] = sum == 0.0f ? -INFINITY : (big - shift + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Workgroups: two per CU (what their registers allow at a time), no more than there
// can be units.
int decode_wgs(int64_t m, int64_t heads, const KvCache& c, int64_t most) {
  const int64_t group = heads / c.kv_heads, tiles = (group + kRows - 1) / kRows;
  const int64_t units = (most + kUnit - 1) / kUnit;
  const int64_t items = m * c.kv_heads * tiles;
  if (units >= kDecodeMaxWgs || items >= kDecodeMaxWgs) return kDecodeMaxWgs;
  return (int)std::max<int64_t>(1, std::min<int64_t>(kDecodeMaxWgs, items * units));
}

template <int DT, int CT, int D>
hipError_t decode_go(const AttentionCall& a, hipStream_t s) {
  const int group = (int)(a.heads / a.cache.kv_heads);
  const DecodeArgs args{a, group, (group + kRows - 1) / kRows};
  int64_t most = std::min<int64_t>(a.max_pages << a.cache.lg_page, INT32_MAX);
  most = std::min<int64_t>(most, (int64_t)a.window + a.sinks);
  const int wgs = decode_wgs(a.m, a.heads, a.cache, most);
  decode_kernel<DT, CT, D><<<dim3((unsigned)wgs), 256, 0, s>>>(args);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || most <= kUnit) return e;        // nothing is in parts
  constexpr float kShift = CT != WQ_E4M3 && DT == WQ_F16 ? 15.0f : 0.0f;
  decode_join_kernel<DT, D>
      <<<dim3((unsigned)a.m, (unsigned)a.heads), 256, 0, s>>>(args, wgs, kShift);
  return hipGetLastError();
}
template <int DT, int D>
hipError_t decode_ct(const AttentionCall& a, hipStream_t s) {
  return a.cache.dt == WQ_E4M3 ? decode_go<DT, WQ_E4M3, D>(a, s) : decode_go<DT, DT, D>(a, s);
}
template <int DT>
hipError_t decode_d(const AttentionCall& a, hipStream_t s) {
  return a.cache.d == 128 ? decode_ct<DT, 128>(a, s) : decode_ct<DT, 64>(a, s);
}

}  // namespace

size_t decode_ws_bytes(int64_t m, int64_t heads, const KvCache& c) {
  return (size_t)decode_wgs(m, heads, c, INT32_MAX) * 2 * kRows * (c.d + 2) * sizeof(float);
}

hipError_t launch_attention_decode(const AttentionCall& a, hipStream_t s) {
  return a.dt == WQ_BF16 ? decode_d<WQ_BF16>(a, s) : decode_d<WQ_F16>(a, s);
}

}  // namespace wq
