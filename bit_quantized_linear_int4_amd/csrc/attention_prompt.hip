// Attention over a paged cache of keys and values (formulas in wq.h).
//
// One wave per row and query head.  A head of D components is D / 8 lanes of 8;
// the 512 / D groups of lanes take the visible tokens in turn, each with a running
// maximum and sums of its own, and are joined at the end.
#include "attention.h"

namespace wq {
namespace {

// 8 components from p: 16 bytes of a 16-bit type, or 8 of E4M3
template <int CT>
__device__ __forceinline__ void load8(const char* p, float (&v)[8]) {
  if constexpr (CT == WQ_E4M3) {
    const uint2_t r = *reinterpret_cast<const uint2_t*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2v_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)r[i], false);
      const float2v_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)r[i], true);
      v[4 * i] = lo[0];
      v[4 * i + 1] = lo[1];
      v[4 * i + 2] = hi[0];
      v[4 * i + 3] = hi[1];
    }
  } else {
    unpack8<CT>(*reinterpret_cast<const uint4_t*>(p), v);
  }
}

template <int DT, int CT, int D>
__global__ __launch_bounds__(64) void attention_rows_kernel(AttentionCall a) {
  constexpr int L = D / 8, G = 64 / L;
  const KvCache& cc = a.cache;
  const int64_t row = blockIdx.x;
  const int head = blockIdx.y, lane = threadIdx.x;
  const int c = lane % L, g = lane / L;
  const int kh = head / (int)(a.heads / cc.kv_heads);

  // the row's sequence, and its position in it
  int64_t seq = row, after = 0;                        // rows of the sequence after this one
  if (a.starts != nullptr) {
    int64_t lo = 0, hi = a.batch;                      // the last start at or before row
    if (row < a.starts[0] || row >= a.starts[a.batch]) return;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (a.starts[mid] <= row) lo = mid; else hi = mid;
    }
    seq = lo;
    after = (int64_t)a.starts[seq + 1] - 1 - row;
  }
  const int64_t room = a.max_pages << cc.lg_page;
  const int64_t len = min((int64_t)max(a.lens[seq], 0), room);
  const int64_t pos = len - 1 - after;
  // visible: [0, first) and [from, pos]
  int64_t from = a.window == INT32_MAX ? 0 : max((int64_t)0, pos + 1 - a.window);
  const int64_t first = min((int64_t)a.sinks, from);
  const int64_t seen = pos < 0 ? 0 : first + pos + 1 - from;

  float q[8];
  unpack8<DT>(*reinterpret_cast<const uint4_t*>(a.q + row * a.ldq + (int64_t)head * D + c * 8), q);
  float m = -INFINITY, l = 0.0f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.0f;
  const int32_t* table = a.pages + seq * a.ldp;
  const float scale = a.scale * kLog2e;
  for (int64_t i0 = 0; i0 < seen; i0 += G) {
    const int64_t i = i0 + g;
    const bool live = i < seen;
    const int64_t j = !live ? pos : i < first ? i : i - first + from;
    const int64_t page = min(max(table[j >> cc.lg_page], 0), cc.pages - 1);
    const int64_t at = j & ((1 << cc.lg_page) - 1);
    const int64_t off = page * cc.page_stride + kh * cc.head_stride + at * cc.token_stride;
    const int64_t sat = ((page * cc.kv_heads + kh) << cc.lg_page) + at;
    constexpr int B = CT == WQ_E4M3 ? 8 : 16;
    float k[8], v[8], z = 0.0f, vs = 1.0f;
    load8<CT>(cc.k + off + c * B, k);
    load8<CT>(cc.v + off + c * B, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) z = fmaf(q[e], k[e], z);
#pragma unroll
    for (int w = 1; w < L; w *= 2) z += __shfl_xor(z, w);
    if constexpr (CT == WQ_E4M3) {
      z *= cc.ks[sat];
      vs = cc.vs[sat];
    }
    z = live ? z * scale : -INFINITY;
    if (z == -INFINITY) continue;
    const float mn = fmaxf(m, z);
    const float r = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(z - mn);
    l = l * r + p;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * r + p * (v[e] * vs);
    m = mn;
  }
#pragma unroll
  for (int w = L; w < 64; w *= 2) {
    const float mo = __shfl_xor(m, w), lo = __shfl_xor(l, w), mn = fmaxf(m, mo);
    const float r = m == -INFINITY ? 0.0f : exp2f(m - mn);
    const float ro = mo == -INFINITY ? 0.0f : exp2f(mo - mn);
    l = l * r + lo * ro;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * r + __shfl_xor(o[e], w) * ro;
    m = mn;
  }
  if (g != 0) return;
  const float inv = l > 0.0f || l != l ? __fdiv_rn(1.0f, l) : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= inv;
  *reinterpret_cast<uint4_t*>(a.y + (row * a.heads + head) * D + c * 8) = pack8<DT>(o);
  if (a.lse != nullptr && c == 0)
    a.lse[row * a.heads + head] = l == 0.0f ? -INFINITY : m * kLn2 + __logf(l);
}

template <int DT, int CT, int D>
hipError_t rows_go(const AttentionCall& a, hipStream_t s) {
  attention_rows_kernel<DT, CT, D>
      <<<dim3((unsigned)a.m, (unsigned)a.heads), 64, 0, s>>>(a);
  return hipGetLastError();
}
template <int DT, int D>
hipError_t rows_ct(const AttentionCall& a, hipStream_t s) {
  return a.cache.dt == WQ_E4M3 ? rows_go<DT, WQ_E4M3, D>(a, s) : rows_go<DT, DT, D>(a, s);
}
template <int DT>
hipError_t rows_d(const AttentionCall& a, hipStream_t s) {
  return a.cache.d == 128 ? rows_ct<DT, 128>(a, s) : rows_ct<DT, 64>(a, s);
}

}  // namespace

hipError_t launch_attention_prompt(const AttentionCall& a, hipStream_t s) {
  return a.dt == WQ_BF16 ? rows_d<WQ_BF16>(a, s) : rows_d<WQ_F16>(a, s);
}

}  // namespace wq
