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
// the next step are in flight while one is computed, its page numbers one step more; a
// third step in registers gains nothing (64 x 4096 tokens, E4M3 109 us and 109).
//
// Measured with 8 kv heads of 128, two launches where items are split: 1 token 5.3 us, 1000
// 8.2, 131072 in E4M3 for 64 query heads 58 (4.8 TB/s, the join 5 of it); 64 x 4096 bf16
// 185 (5.8 TB/s), E4M3 109 (5.0); 24 of 1 to 8000 tokens, 32 kv heads 88 (4.6).  Heads of
// 64 in E4M3: 64 x 4096 61 (4.7); 129 windows of 1024 for 4 kv heads 23.5, of which HBM asks
// for 11 and a launch for 2: ten steps a workgroup, whose start, joins and page numbers are
// chains of latency.
#include <algorithm>

#include "attention.h"

namespace wq {
namespace {

constexpr int kStep = 128;             // tokens of a workgroup's step: 4 waves of 32
constexpr int kRows = 16;              // query heads of an item

// What the join is to do for an item: its parts are workgroup `wg`'s second slot, the
// next ones' second and the last one's first.  Fewer than two parts: nothing.
struct Joined {
  int wg, seq, head, rows_parts;       // rows << 16 | parts
};

struct DecodeArgs {
  AttentionCall a;
  // behind the parts in the workspace: per item where there are no more items than
  // workgroups, else per workgroup, for the item that starts in its stretch and goes on
  Joined* joined;
  int per_item;
  int group, tiles;                    // query heads per kv head; items of 16 of them
  int lg_unit;                         // log2 of a unit's tokens
  uint32_t page16, token16;            // strides in 16 bytes; a cache spans less than 2^31
};

__device__ __forceinline__ Visible decode_visible(const AttentionCall& a, int seq) {
  return visible_of(tokens_of(a, a.lens[seq]) - 1, a.window, a.sinks);
}
// the same for a `seq` that is the same in every lane
template <typename A>
__device__ __forceinline__ Visible uniform_visible(const A& a, int seq) {
  const int64_t room = a.max_pages << a.cache.lg_page;
  const int len = (int)min((int64_t)max(scalar_at(a.lens, seq), 0), room);
  return visible_of(len - 1, a.window, a.sinks);
}
__device__ __forceinline__ int units_of(const DecodeArgs& args, const Visible& v) {
  return (v.n + (1 << args.lg_unit) - 1) >> args.lg_unit;
}

// `units` of the line over `wgs` workgroups (at most as many): the first `more` take
// one unit above `each`
struct Share {
  int each, more;
  __device__ Share(int units, int wgs) : each(units / wgs), more(units - each * wgs) {}
  __device__ int start(int wg) const { return wg * each + min(wg, more); }
  __device__ int owner(int unit) const {
    const int big = more * (each + 1);
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  }
};

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

// Whose sums a step adds to: kept in two words, for each step on its way.
struct Owner {
  int seq, rest;
  static constexpr int kStarts = 1, kEnds = 2;           // the item's first, last unit is here
  static constexpr int kLast = 4, kFinal = 8;            // last step of the piece, of the workgroup
  __device__ int kh() const { return rest >> 12; }
  __device__ int ht() const { return (rest >> 4) & 255; }
};

// one step of a wave: its owner, how many of its 32 tokens are there, and this lane's
// page and place in it
struct Step {
  Owner owner;
  int count, page, place;
};

template <int DT, int CT, int D>
__global__ __launch_bounds__(256, 2) void decode_kernel(DecodeArgs args) {
  constexpr bool F8 = CT == WQ_E4M3;
  constexpr int VT = F8 ? WQ_BF16 : DT;                  // type of the values' products
  // Exponents are taken from a reference that follows the running maximum only where it
  // is passed by more than 2^8, so that the sums are rarely rescaled (which the prompt
  // kernel needs; HBM hides it here).  Weights of f16 are kept 2^7 larger: at most 2^15, and
  // less of them in its subnormal range, where the second part rounds to multiples of 2^-24:
  // a weight is off by 2^-32 at most, and the row's largest is 1 (the reference's) or more.
  constexpr float kLag = 8.0f, kShift = VT == WQ_F16 ? 7.0f : 0.0f;
  constexpr int KC = Tile<CT, D>::KC, VW = Tile<CT, D>::VW;
  constexpr int NI = D / 16;                             // O^T tiles, components of a lane
  constexpr int OS = D + 4;                              // LDS row of O, in floats
  constexpr int NT = 2;                                  // steps whose tiles are in registers
  const AttentionCall& a = args.a;
  const KvCache& cc = a.cache;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;

  __shared__ int part[kLineWords<256>];
  __shared__ __align__(16) float so[4 * kRows * OS];
  __shared__ float sm[4][kRows], sl[4][kRows];

  const int per_unit = cc.kv_heads * args.tiles, m_rows = (int)a.m;
  auto count = [&](int i) { return units_of(args, decode_visible(a, i)); };
  const Line line = m_rows == 1 ? Line{units_of(args, uniform_visible(a, 0)), 0}
                                : line_up<256>(m_rows, part, count);
  const int all = line.total * per_unit;

  // rows that see nothing are in no unit
  for (int i = blockIdx.x; i < m_rows; i += gridDim.x) {
    if (uniform_visible(a, i).n > 0) continue;
    if (args.per_item)
      for (int e = tid; e < per_unit; e += 256)
        args.joined[i * per_unit + e] = Joined{0, 0, 0, 0};
    for (int64_t e = tid; e < a.heads * (D / 8); e += 256)
      reinterpret_cast<uint4_t*>(a.y)[i * a.heads * (D / 8) + e] = uint4_t{0, 0, 0, 0};
    if (a.lse != nullptr)
      for (int64_t e = tid; e < a.heads; e += 256) a.lse[i * a.heads + e] = -INFINITY;
  }

  if (!args.per_item && tid == 0) args.joined[blockIdx.x] = Joined{0, 0, 0, 0};
  const int wgs = min((int)gridDim.x, all);              // none without a unit
  if ((int)blockIdx.x >= wgs) return;
  const Share share(all, wgs);
  int u = share.start(blockIdx.x);
  const int u_end = share.start(blockIdx.x + 1);
  int item0;                                             // the line's unit where seq starts
  int seq = line_find<256>(m_rows, line, part, u / per_unit, item0, count);
  seq = __builtin_amdgcn_readfirstlane(seq);
  item0 = __builtin_amdgcn_readfirstlane(item0) * per_unit;

  // Two stages ahead of the sums: a step's page numbers, then its keys and values.  Both
  // run on into the next piece (a part of one item) while this one is joined.
  Owner ahead;
  Visible vis;
  int at, end;                                           // visible tokens, from the wave's on
  auto take = [&]() {                                    // the piece that starts at u < u_end
    const auto k = args_here<DecodeArgs>();
    const int lg_unit = k->lg_unit, tiles = k->tiles, per_unit = k->a.cache.kv_heads * tiles;
    const Share share(all, wgs);
    const int u_end = share.start(blockIdx.x + 1);
    auto look = [&]() {
      const int room = (int)(k->a.max_pages << k->a.cache.lg_page);
      const int len = min(max(scalar_at(k->a.lens, seq), 0), room);
      vis = visible_of(len - 1, k->a.window, k->a.sinks);
      return (vis.n + (1 << lg_unit) - 1) >> lg_unit;
    };
    int units = look();
    while (u >= item0 + units * per_unit) {
      item0 += units * per_unit;
      ++seq;
      units = look();
    }
    const int sub = (u - item0) / units;                 // kv head and tile of query heads
    const int kh = sub / tiles, ht = sub - kh * tiles;
    const int first = item0 + sub * units;               // the item's first unit
    const int ua = u - first, ub = min(units, u_end - first);
    ahead.seq = seq;
    ahead.rest = kh << 12 | ht << 4 | (ua == 0 ? Owner::kStarts : 0) |
                 (ub == units ? Owner::kEnds : 0);
    at = ua << lg_unit;
    end = min(ub << lg_unit, vis.n);
    u = first + ub;
    if (ua == 0 && (ub < units || k->per_item) && tid == 0) {
      const int parts = share.owner(first + units - 1) - (int)blockIdx.x + 1;
      const int rows = min(kRows, k->group - ht * kRows);
      k->joined[k->per_item ? seq * per_unit + sub : (int)blockIdx.x] =
          Joined{(int)blockIdx.x, seq, kh * k->group + ht * kRows, rows << 16 | parts};
    }
  };
  take();
  auto look_up = [&]() {
    Step s;
    s.owner = ahead;
    s.count = end - at - wave * 32;
    const int i = min(at + wave * 32 + (lane & 31), end - 1);
    const int token = i < vis.first ? i : i - vis.first + vis.from;
    s.page = page_of(a, a.pages + (int64_t)ahead.seq * a.ldp, token);
    s.place = token & ((1 << cc.lg_page) - 1);
    at += kStep;
    if (at >= end) {
      s.owner.rest |= Owner::kLast;
      if (u < u_end) {
        take();
      } else {
        s.owner.rest |= Owner::kFinal;
        at = end;                                        // what follows is loaded for nothing
      }
    }
    return s;
  };
  auto load = [&](Tile<CT, D>& t, const Step& s) {
    const uint32_t off = (uint32_t)s.page * args.page16 + (uint32_t)s.place * args.token16;
    const int kh = s.owner.kh();
    const char* kbase = cc.k + kh * cc.head_stride;
    const char* vbase = cc.v + kh * cc.head_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * h + (lane >> 2)) * 4,
                                                                (int)off);
      const char* p = kbase + ((uint64_t)o << 4) + (lane & 3) * 16;
#pragma unroll
      for (int c = 0; c < KC; ++c) t.k[h][c] = *reinterpret_cast<const uint4_t*>(p + c * 64);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = (i < 4 ? 4 * kq + i : 12 + 4 * kq + i) * 4;
      const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)off);
      load_words<VW>(vbase + ((uint64_t)o << 4) + nl * (VW * 4), t.v[i]);
    }
    if constexpr (F8) {
      const float* scales = lane < 32 ? cc.ks : cc.vs;
      t.scale = scales[(((int64_t)s.page * cc.kv_heads + kh) << cc.lg_page) + s.place];
    }
  };

  // Q^T: lane (row nl, piece kq); rows past the group are zeros
  uint4_t q[D / 32];
  auto load_q = [&](const Owner& p) {
    const auto k = args_here<DecodeArgs>();
    const int rows = min(kRows, k->group - p.ht() * kRows);
    const int64_t head = (int64_t)p.kh() * k->group + p.ht() * kRows + min(nl, rows - 1);
    const uint16_t* qp = k->a.q + (int64_t)p.seq * k->a.ldq + head * D;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const int d0 = F8 ? 64 * (c / 2) + 16 * kq + 8 * (c % 2) : 32 * c + 8 * kq;
      q[c] = *reinterpret_cast<const uint4_t*>(qp + d0);
      if (nl >= rows) q[c] = uint4_t{0, 0, 0, 0};
    }
  };

  float m = -INFINITY, l = 0.0f;
  float4_t o[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) o[i] = float4_t{0, 0, 0, 0};
  const float zscale = a.scale * kLog2e;

  auto compute = [&](const Tile<CT, D>& t, int count) {
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
      for (int r = 0; r < 4; ++r) z[4 * s + r] = acc[r];
    }
    // scores in units of ln 2: 16 bits z * zscale; E4M3 z, with the scale of the key
    float vs[8];
    if constexpr (F8) {
      const float ts = lane < 32 ? t.scale * zscale : t.scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = 4 * kq + (i < 4 ? i : 12 + i);
        z[i] *= __int_as_float(__builtin_amdgcn_ds_bpermute(tok * 4, __float_as_int(ts)));
        vs[i] = __int_as_float(__builtin_amdgcn_ds_bpermute(tok * 4 + 128, __float_as_int(ts)));
      }
    }
    const float unit = F8 ? 1.0f : zscale;
    if (count < 32) {                                    // tokens past the end repeat the last
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool live = 4 * kq + (i < 4 ? i : 12 + i) < count;
        z[i] = live ? z[i] : -INFINITY;
        if constexpr (F8) vs[i] = live ? vs[i] : 0.0f;   // it may not be finite
      }
    }
    float big = z[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) big = fmaxf(big, z[i]);
    big = max_quarters(big) * unit;
    if (__any(big > m + kLag)) {
      // each row by itself, so that it does not depend on the others
      const float mn = big > m + kLag ? big : m;
      const float fade = __builtin_amdgcn_exp2f(m - exp_ref(mn));
      m = mn;
      l *= fade;
#pragma unroll
      for (int i = 0; i < NI; ++i) o[i] *= fade;
    }
    const float ref = exp_ref(m) - kShift;
    float p[8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(F8 ? z[i] - ref : fmaf(z[i], unit, -ref));
      sum += p[i];
    }
    l += sum;
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] *= vs[i];
    }
    // two parts of 8 (bf16) or 11 bits (f16, down to 2^-24): one part's rounding would be as
    // large as that of a 16-bit y, and saves little (64 x 4096 tokens 186.1 us with two, 185.5
    // with one; 500 tokens 8.2 and 7.9)
    uint4_t hi, lo;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      hi[w] = pack_weights<VT>(p[2 * w], p[2 * w + 1]);
      float h0, h1;
      unpack2<VT>(hi[w], h0, h1);
      lo[w] = pack_weights<VT>(p[2 * w] - h0, p[2 * w + 1] - h1);
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

  // joins the four waves' sums of a piece and starts new ones
  auto finish = [&](const Owner& p) {
    const auto k = args_here<DecodeArgs>();
    const bool starts = p.rest & Owner::kStarts, ends = p.rest & Owner::kEnds;
    l = sum_quarters(l);
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
      float* x = so + (wave * kRows + nl) * OS + NI * (4 * kq + r);
#pragma unroll
      for (int i = 0; i < NI; i += 4)
        *reinterpret_cast<float4_t*>(x + i) =
            float4_t{o[i][r] * f, o[i + 1][r] * f, o[i + 2][r] * f, o[i + 3][r] * f};
    }
    __syncthreads();
    const int rows = min(kRows, k->group - p.ht() * kRows);
    float* slot = k->a.ws + (2 * (int64_t)blockIdx.x + (ends ? 0 : 1)) * (kRows * (D + 2));
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
      if (starts && ends) {
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        const int64_t out =
            (int64_t)p.seq * k->a.heads + (int64_t)p.kh() * k->group + p.ht() * kRows + row;
        *reinterpret_cast<uint4_t*>(k->a.y + out * D + c * 8) = pack8<DT>(v);
        if (k->a.lse != nullptr && c == 0)
          k->a.lse[out] = sum == 0.0f ? -INFINITY
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
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) o[i] = float4_t{0, 0, 0, 0};
  };

  Tile<CT, D> t[NT];
  Step s[NT], next = look_up();
  load_q(next.owner);
#pragma unroll
  for (int j = 0; j + 1 < NT; ++j) {
    s[j] = next;
    next = look_up();
    load(t[j], s[j]);
  }
  for (;;) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      constexpr int kAhead = NT - 1;
      s[(j + kAhead) % NT] = next;
      next = look_up();
      load(t[(j + kAhead) % NT], s[(j + kAhead) % NT]);
      compute(t[j], s[j].count);
      if (s[j].owner.rest & Owner::kLast) {
        finish(s[j].owner);
        if (s[j].owner.rest & Owner::kFinal) return;
        load_q(s[(j + 1) % NT].owner);
      }
    }
  }
}

// A workgroup takes rows of an item.  Its groups of D / 4 threads take parts in turn, each
// with a running reference, four parts loaded together: BY_ROW a group a row and all its
// parts, else all groups the parts of one row, which they then join.
template <int DT, int D, bool BY_ROW>
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs args, float shift) {
  const AttentionCall& a = args.a;
  constexpr int L = D / 4, G = 256 / L, STEP = BY_ROW ? 1 : G;
  const int tid = threadIdx.x, c = tid % L, g = tid / L;
  const Joined item = args.joined[blockIdx.x];
  const int n = item.rows_parts & 0xFFFF, rows = item.rows_parts >> 16;
  const int row = BY_ROW ? (int)blockIdx.y * G + g : blockIdx.y;
  if (n < 2 || row >= rows) return;
  float m = -INFINITY, l = 0.0f;
  float4_t o = {0, 0, 0, 0};
  for (int i0 = BY_ROW ? 0 : g; i0 < n; i0 += 4 * STEP) {
    float pm[4], pl[4];
    float4_t po[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(i0 + j * STEP, n - 1);
      const float* slot =
          a.ws + (2 * (int64_t)(item.wg + i) + (i + 1 < n ? 1 : 0)) * (kRows * (D + 2));
      po[j] = *reinterpret_cast<const float4_t*>(slot + row * D + c * 4);
      pm[j] = slot[kRows * D + row];
      pl[j] = slot[kRows * (D + 1) + row];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool live = i0 + j * STEP < n;
      const float mn = fmaxf(m, live ? pm[j] : -INFINITY), ref = exp_ref(mn);
      const float fade = __builtin_amdgcn_exp2f(m - ref);
      const float f = live ? __builtin_amdgcn_exp2f(pm[j] - ref) : 0.0f;
      l = l * fade + (live ? pl[j] * f : 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o[e] * fade + (live ? po[j][e] * f : 0.0f);
      m = mn;
    }
  }
  if constexpr (!BY_ROW) {
    __shared__ __align__(16) float so[G][D];
    __shared__ float sm[G], sl[G];
    *reinterpret_cast<float4_t*>(&so[g][c * 4]) = o;
    if (c == 0) {
      sm[g] = m;
      sl[g] = l;
    }
    __syncthreads();
    if (g != 0) return;
    m = sm[0];
#pragma unroll
    for (int i = 1; i < G; ++i) m = fmaxf(m, sm[i]);
    l = 0.0f;
    o = float4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float f = __builtin_amdgcn_exp2f(sm[i] - exp_ref(m));
      l += sl[i] * f;
      o += f * *reinterpret_cast<const float4_t*>(&so[i][c * 4]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
  const int64_t out = (int64_t)item.seq * a.heads + item.head + row;
  *reinterpret_cast<uint2_t*>(a.y + out * D + c * 4) =
      uint2_t{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
  if (a.lse != nullptr && c == 0)
    a.lse[out] = l == 0.0f ? -INFINITY : (m - shift + __builtin_amdgcn_logf(l)) * kLn2;
}

// Workgroups: two per CU (what their registers allow at a time; for heads of 64 three fit:
// 129 windows of 1024 a tenth less, but where two a CU come out even more: 64 x 1000 tokens
// 33 us against 29, 64 x 4096 in E4M3 65 against 60), no more than there can be units.
int decode_wgs(int64_t items, int64_t units) {
  if (units >= kDecodeMaxWgs || items >= kDecodeMaxWgs) return kDecodeMaxWgs;
  return (int)std::max<int64_t>(1, std::min<int64_t>(kDecodeMaxWgs, items * units));
}
int64_t decode_tiles(int64_t heads, const KvCache& c) {
  return (heads / c.kv_heads + kRows - 1) / kRows;
}

template <int DT, int CT, int D>
hipError_t decode_go(const AttentionCall& a, hipStream_t s) {
  const int64_t tiles = decode_tiles(a.heads, a.cache), items = a.m * a.cache.kv_heads * tiles;
  // what a row can see at most
  int64_t most = std::min<int64_t>(a.max_pages << a.cache.lg_page, int64_t(1) << 30);
  most = std::min<int64_t>(most, (int64_t)a.window + a.sinks);
  // A unit is one step.  It is four where no item has more, so that none is split and the
  // join not launched (bf16, 8 kv heads of 128: 1 sequence of 250 tokens 6.3 us and 7.9
  // split, of 500 8.2 and 8.2, 64 of 500 27.6 and 29.6; and the call one launch, 3.6 us of
  // the host's time, shorter), and more where the line could pass 32 bits.
  int lg_unit = most <= (kStep << 2) ? 9 : 7;
  while (((most >> lg_unit) + 1) > (int64_t(1) << 30) / items) ++lg_unit;
  const int64_t units = (most + (int64_t(1) << lg_unit) - 1) >> lg_unit;
  const int wgs = decode_wgs(items, units);
  Joined* joined = reinterpret_cast<Joined*>(a.ws + (int64_t)wgs * 2 * kRows * (D + 2));
  const bool per_item = items <= wgs;
  const DecodeArgs args{a, joined, per_item, (int)(a.heads / a.cache.kv_heads), (int)tiles, lg_unit,
                        (uint32_t)(a.cache.page_stride >> 4),
                        (uint32_t)(a.cache.token_stride >> 4)};
  decode_kernel<DT, CT, D><<<dim3((unsigned)wgs), 256, 0, s>>>(args);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || units <= 1) return e;           // nothing is in parts
  constexpr float kShift = CT != WQ_E4M3 && DT == WQ_F16 ? 7.0f : 0.0f;
  const int64_t records = per_item ? items : wgs;
  const int rows = std::min(kRows, args.group);
  // Many items have few parts each (129 windows of 1024, heads of 64 24.1 us by row and 25.6
  // else; 16 x 2048 17.5 and 18.9), few have many (1 x 8000 17.9 and 10.2).  One long
  // sequence among many has at most wgs / kv_heads: all its heads are as long.
  if (4 * items >= wgs && a.cache.kv_heads >= 4) {
    const int groups = 256 / (D / 4);
    const dim3 grid((unsigned)records, (unsigned)((rows + groups - 1) / groups));
    decode_join_kernel<DT, D, true><<<grid, 256, 0, s>>>(args, kShift);
  } else {
    decode_join_kernel<DT, D, false>
        <<<dim3((unsigned)records, (unsigned)rows), 256, 0, s>>>(args, kShift);
  }
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
  const int64_t items = m * c.kv_heads * decode_tiles(heads, c);
  return (size_t)decode_wgs(items, INT32_MAX) *
         (2 * kRows * (c.d + 2) * sizeof(float) + sizeof(Joined));
}

hipError_t launch_attention_decode(const AttentionCall& a, hipStream_t s) {
  return a.dt == WQ_BF16 ? decode_d<WQ_BF16>(a, s) : decode_d<WQ_F16>(a, s);
}

}  // namespace wq
