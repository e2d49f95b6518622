// Rotary rotation of queries and keys, and append of keys and values to a paged
// cache in 16 bits or E4M3 (formulas in wq.h).
//
// Bound by HBM for many rows (8191 rows, 32 query and 32 kv heads of 128, bf16: 79 us,
// 5.1 TB/s) and by latency (slot or position, table, store) for few (1 row 2.5 us, where a
// launch takes 2; 50 rows into E4M3 3.1).  A head is D / 8 lanes of 8 elements; a thread
// takes the same elements of U heads of one row, so the row's cos and sin are loaded once
// and all its loads are in flight together.  The other element of a pair (i, i + rot / 2)
// is in another lane of the same head and comes from it by a lane permute, so q_out may be q.
#include "fp8_util.h"

namespace wq {
namespace {

// largest value over the L = 8 or 16 lanes of a head
template <int L>
__device__ __forceinline__ uint32_t max_head(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  if constexpr (L == 16) v = max(v, dpp<0x140>(v));
  return v;
}

template <int DT, int D, bool F8, int U>
__global__ __launch_bounds__(256) void append_kv_kernel(AppendCall a) {
  constexpr int L = D / 8, HP = 256 / L;              // lanes per head, heads per round
  const KvCache& cc = a.cache;
  const int64_t row = blockIdx.x;
  const int sub = threadIdx.x / L, c = threadIdx.x % L;
  const int heads = (int)a.heads, kvh = cc.kv_heads, units = heads + 2 * kvh;
  const int u0 = (int)blockIdx.y * U * HP + sub;

  uint4_t raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = min(u0 + i * HP, units - 1);        // every lane loads
    const uint16_t* p = u < heads ? a.q + row * a.ldq + (int64_t)u * D
                        : u < heads + kvh ? a.k + row * a.ldk + (int64_t)(u - heads) * D
                                          : a.v + row * a.ldv + (int64_t)(u - heads - kvh) * D;
    raw[i] = *reinterpret_cast<const uint4_t*>(p + c * 8);
  }
  const int slot = a.slots[row];

  // cos and sin of this thread's elements: element e of the chunk takes co[e], si[e]
  // times its partner (the sign in si); past rot they are 1 and 0
  const int half = a.rot / 2;
  const bool turn = c * 8 < a.rot;
  float co[8], si[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) co[e] = 1.0f, si[e] = 0.0f;
  if (turn) {
    const int64_t last = a.max_pos - 1;
    const int64_t pos = min((int64_t)max(a.positions[row], 0), last);
    const float* t = a.cos_sin + pos * a.rot;
    if (a.interleaved) {
      const float4_t cv = *reinterpret_cast<const float4_t*>(t + c * 4);
      const float4_t sv = *reinterpret_cast<const float4_t*>(t + half + c * 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = cv[e / 2];
        si[e] = e % 2 == 0 ? -sv[e / 2] : sv[e / 2];
      }
    } else {
      const bool low = c * 8 < half;
      const int i0 = low ? c * 8 : c * 8 - half;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float4_t cv = *reinterpret_cast<const float4_t*>(t + i0 + 4 * p);
        const float4_t sv = *reinterpret_cast<const float4_t*>(t + half + i0 + 4 * p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          co[4 * p + e] = cv[e];
          si[4 * p + e] = low ? -sv[e] : sv[e];
        }
      }
    }
  }
  // the lane that holds the partners of this chunk
  const int lane = (int)__lane_id();
  const int from = !turn || a.interleaved ? lane : lane + (c * 8 < half ? half / 8 : -half / 8);

  const bool stored = slot >= 0 && (slot >> cc.lg_page) < cc.pages;
  const int64_t page = stored ? slot >> cc.lg_page : 0;
  const int64_t at = slot & ((1 << cc.lg_page) - 1);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = u0 + i * HP;
    float v[8];
    unpack8<DT>(raw[i], v);
    uint4_t other;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      other[w] = (uint32_t)__builtin_amdgcn_ds_bpermute(from * 4, (int)raw[i][w]);
    const bool is_v = u >= heads + kvh;
    bool same = true;                                  // 16-bit outputs are the input's bits
    if (turn && !is_v) {
      float p[8];
      unpack8<DT>(other, p);
      float r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float b = a.interleaved ? v[e ^ 1] : p[e];
        r[e] = fmaf(v[e], co[e], b * si[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = r[e];
      same = false;
    }
    const uint4_t bits = same ? raw[i] : pack8<DT>(v);
    if (u < heads) {
      *reinterpret_cast<uint4_t*>(a.q_out + row * a.ldo + (int64_t)u * D + c * 8) = bits;
    }
    const bool live = u >= heads && u < units && stored;
    const int h = is_v ? u - heads - kvh : u - heads;
    char* base = is_v ? cc.v : cc.k;
    const int64_t off = page * cc.page_stride + h * cc.head_stride + at * cc.token_stride;
    if constexpr (F8) {
      uint32_t big = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) big = max(big, abs_bits(v[e]));
      const float s = fp8_scale(max_head<L>(big));
      if (live) {
        *reinterpret_cast<uint2_t*>(base + off + c * 8) = fp8_codes(s, v);
        float* sc = is_v ? cc.vs : cc.ks;
        if (c == 0) sc[((page * kvh + h) << cc.lg_page) + at] = s;
      }
    } else {
      if (live) *reinterpret_cast<uint4_t*>(base + off + c * 16) = bits;
    }
  }
}

template <int DT, int D, bool F8, int U>
hipError_t append_u(const AppendCall& a, hipStream_t s) {
  constexpr int HP = 256 / (D / 8);
  const int64_t units = a.heads + 2 * a.cache.kv_heads;
  const dim3 grid((unsigned)a.m, (unsigned)((units + U * HP - 1) / (U * HP)));
  append_kv_kernel<DT, D, F8, U><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
// Few rows: more workgroups, each with fewer loads before its first store; many rows: the
// row's cos and sin serve more heads (32 query and 8 kv heads of 128, bf16 | E4M3: 1 row
// 2.5 | 2.6 us with one head a thread and 3.1 | 3.2 with four, 128 rows 3.0 and 3.5, 512
// 4.4 and 4.4, 8192 43.4 | 43.1 and 41.2 | 39.2).
template <int DT, int D, bool F8>
hipError_t append_rows(const AppendCall& a, hipStream_t s) {
  return a.m < 512 ? append_u<DT, D, F8, 1>(a, s) : append_u<DT, D, F8, 4>(a, s);
}
template <int DT, int D>
hipError_t append_f8(const AppendCall& a, hipStream_t s) {
  return a.cache.dt == WQ_E4M3 ? append_rows<DT, D, true>(a, s) : append_rows<DT, D, false>(a, s);
}
template <int DT>
hipError_t append_d(const AppendCall& a, hipStream_t s) {
  return a.cache.d == 128 ? append_f8<DT, 128>(a, s) : append_f8<DT, 64>(a, s);
}

}  // namespace

hipError_t launch_append_kv(const AppendCall& a, hipStream_t s) {
  return a.dt == WQ_BF16 ? append_d<WQ_BF16>(a, s) : append_d<WQ_F16>(a, s);
}

}  // namespace wq
