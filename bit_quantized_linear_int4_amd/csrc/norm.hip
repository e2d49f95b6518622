// Residual addition with root-mean-square norm, and the FP8 packers.
//
// add_rmsnorm, per row of k values:
//   h = x + residual                      (fp32; residual_out = round16(h))
//   v = h * rsqrt(sum(h^2) / k + eps) * gain
//   y = round16(v), and per 128 values of v:  s = max|v| / 448, q = E4M3(v / s)
// The norm is taken of the unrounded h; every statistic is fp32.  The row
// stays in registers between the sum and the outputs, so each input is read
// once and each output written once: the kernel is bound by HBM for many rows
// and by the latency of one load, one barrier and one store for few.  bf16 with
// a residual to FP8, 8192 rows of 8192: 85 us, 5520 GB/s (a copy of 1 GiB: 5130
// to 5180); 1 row of 4096: 2.5 us, of 256: 2.0.
// One row per workgroup, and outputs stored past the caches, which keeps them
// for the inputs: with four rows per workgroup 97 us, with ordinary stores 96
// (84 then for one row and these stores).
//
// quantize_rows: the same scale and code for given rows, or for silu(x) * up
// (what stands between the gate/up and the down product of an MLP); bound by
// HBM and, gated, as much by the vector units: 2048 rows of 14336 28 to 29 us,
// 5030 to 5270 GB/s.
//
// quantize_block: weights, one scale per 128 x 128 block; once per weight: 14336
// x 4096 41 us, 4300 GB/s, 28672 x 8192 132 us, 5350 GB/s.
//
// Scales of rows are stored [ceil(k / 128)][m]: the linear reads the scales of
// all its tokens for one block of k at once, so they are contiguous.
#include "fp8_util.h"

namespace wq {
namespace {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;       // or nullptr
  uint16_t* res_out;         // or nullptr
  const uint16_t* gain;
  uint16_t* y;               // or nullptr
  uint8_t* q;                // or nullptr
  float* scales;
  int64_t ldx, ldr;
  int m, k;
  float eps;
};

// 16 or 8 bytes of an output, past the caches: nothing here reads them again
template <typename T>
__device__ __forceinline__ void put(void* p, T v) {
  __builtin_nontemporal_store(v, static_cast<T*>(p));
}

// the inputs of one 16-byte chunk; every lane loads (past the end of the row
// its last chunk), so that no load waits behind a branch
struct NormChunk {
  uint4_t x, r, g;
};
__device__ __forceinline__ NormChunk norm_load(const NormArgs& a, int64_t row, int c) {
  NormChunk t;
  t.x = *reinterpret_cast<const uint4_t*>(a.x + row * a.ldx + c * 8);
  constexpr uint32_t kNone = 0x80008000u;  // -0, -0: x + -0 is x, whatever its sign
  t.r = a.res != nullptr ? *reinterpret_cast<const uint4_t*>(a.res + row * a.ldr + c * 8)
                         : uint4_t{kNone, kNone, kNone, kNone};
  t.g = *reinterpret_cast<const uint4_t*>(a.gain + c * 8);
  return t;
}
// h of the chunk, zeros where the row has ended
template <int DT>
__device__ __forceinline__ void norm_sum(const NormChunk& t, bool live, float (&h)[8]) {
  float r[8];
  unpack8<DT>(t.x, h);
  unpack8<DT>(t.r, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = live ? h[i] + r[i] : 0.0f;
}

// the outputs of one chunk; the 16 lanes of a scale block are consecutive and
// all call this (`live` false past the end of the row)
template <int DT>
__device__ __forceinline__ void norm_store(const NormArgs& a, int64_t row, int c, bool live,
                                           const float (&h)[8], uint4_t graw, float rstd) {
  if (a.res_out != nullptr && live) put(a.res_out + row * a.ldr + c * 8, pack8<DT>(h));
  float g[8], v[8];
  unpack8<DT>(graw, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = h[i] * rstd * g[i];
  if (a.y != nullptr && live) put(a.y + row * a.k + c * 8, pack8<DT>(v));
  if (a.q != nullptr) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, abs_bits(v[i]));
    const float s = fp8_scale(max16(live ? big : 0u));
    if (live) {
      put(a.q + row * a.k + c * 8, fp8_codes(s, v));
      if ((c & 15) == 0) a.scales[(int64_t)(c >> 4) * a.m + row] = s;
    }
  }
}

// sum over the workgroup, in every thread
template <int NT>
__device__ __forceinline__ float wg_sum(float v) {
  v = sum64(v);
  if constexpr (NT == 64) return v;
  __shared__ float part[NT / 64];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) t += part[i];
  return t;
}

// One row per workgroup, V chunks of 8 values per thread; V = 0: rows of any
// length, read twice.
template <int DT, int NT, int V>
__global__ __launch_bounds__(NT) void add_rmsnorm_kernel(NormArgs a) {
  const int tid = threadIdx.x;
  const int nc = a.k / 8;
  const int64_t row = blockIdx.x;
  const float rk = __fdiv_rn(1.0f, (float)a.k);
  float ss = 0.0f;
  if constexpr (V > 0) {
    NormChunk t[V];
    float h[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) t[j] = norm_load(a, row, min(tid + j * NT, nc - 1));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      norm_sum<DT>(t[j], tid + j * NT < nc, h[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
    }
    const float rstd = rsqrtf(wg_sum<NT>(ss) * rk + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + j * NT;
      norm_store<DT>(a, row, c, c < nc, h[j], t[j].g, rstd);
    }
  } else {
    for (int c = tid; c < nc; c += NT) {
      float h[8];
      norm_sum<DT>(norm_load(a, row, c), true, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
    }
    const float rstd = rsqrtf(wg_sum<NT>(ss) * rk + a.eps);
    // every value is read by the thread that writes it, so residual_out may be
    // the residual itself; all lanes take part in each round
    for (int c0 = 0; c0 < nc; c0 += NT) {
      const int c = c0 + tid;
      const NormChunk t = norm_load(a, row, min(c, nc - 1));
      float h[8];
      norm_sum<DT>(t, c < nc, h);
      norm_store<DT>(a, row, c, c < nc, h, t.g, rstd);
    }
  }
}

struct RowsArgs {
  const uint16_t* x;
  const uint16_t* up;        // or nullptr
  uint8_t* q;
  float* scales;
  int m, k, kb, kt;          // kt workgroups along k
};

// 16 lanes per scale block; a workgroup takes RT rows x 16/RT blocks of k in
// each of U rounds, so with RT = 16 the scales it writes are 64 contiguous
// bytes per block of k.  Workgroups next to each other continue along k.  Two
// rounds: 16 rows of 11008 2.7 us, 3.8 with four.
template <int DT, int RT, int U>
__global__ __launch_bounds__(256) void quantize_rows_kernel(RowsArgs a) {
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int rt = (int)blockIdx.x / a.kt;
  const int64_t row = (int64_t)rt * RT + sub % RT;
  const int b0 = ((int)blockIdx.x - rt * a.kt) * U * (16 / RT) + sub / RT;
  const bool rlive = row < a.m;
  float v[U][8];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (b0 + u * (16 / RT)) * kF8Block + l * 8;
    live[u] = rlive && c < a.k;
    if (live[u]) {
      unpack8<DT>(*reinterpret_cast<const uint4_t*>(a.x + row * a.k + c), v[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
    }
  }
  if (a.up != nullptr) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      const int c = (b0 + u * (16 / RT)) * kF8Block + l * 8;
      float w[8];
      unpack8<DT>(*reinterpret_cast<const uint4_t*>(a.up + row * a.k + c), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = silu(v[u][i]) * w[i];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int b = b0 + u * (16 / RT), c = b * kF8Block + l * 8;
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, abs_bits(v[u][i]));
    const float s = fp8_scale(max16(big));
    if (live[u]) {
      put(a.q + row * a.k + c, fp8_codes(s, v[u]));
      if (l == 0) a.scales[(int64_t)b * a.m + row] = s;
    }
  }
}

// one workgroup per 128 x 128 block of a weight; 16 lanes per row, 16 rows a
// round, the block held in registers between the maximum and the codes
template <int DT>
__global__ __launch_bounds__(256) void quantize_block_kernel(const uint16_t* __restrict__ w,
                                                             int64_t n, int64_t k, int kb,
                                                             uint8_t* __restrict__ q,
                                                             float* __restrict__ scales) {
  __shared__ uint32_t wmax[4];
  const int64_t nb = blockIdx.x / kb;
  const int b = blockIdx.x % kb;
  const int sub = threadIdx.x >> 4, c = b * kF8Block + (threadIdx.x & 15) * 8;
  float v[8][8];
  uint32_t big = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = nb * kF8Block + j * 16 + sub;
    if (row < n && c < k) {
      unpack8<DT>(*reinterpret_cast<const uint4_t*>(w + row * k + c), v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, abs_bits(v[j][i]));
  }
  big = max16(big);
  big = max(max((uint32_t)__builtin_amdgcn_readlane((int)big, 0),
                (uint32_t)__builtin_amdgcn_readlane((int)big, 16)),
            max((uint32_t)__builtin_amdgcn_readlane((int)big, 32),
                (uint32_t)__builtin_amdgcn_readlane((int)big, 48)));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = big;
  __syncthreads();
  big = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const float s = fp8_scale(big);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = nb * kF8Block + j * 16 + sub;
    if (row < n && c < k) *reinterpret_cast<uint2_t*>(q + row * k + c) = fp8_codes(s, v[j]);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

template <int DT, int NT, int V>
hipError_t norm_nt(const NormArgs& a, hipStream_t s) {
  add_rmsnorm_kernel<DT, NT, V><<<dim3((unsigned)a.m), NT, 0, s>>>(a);
  return hipGetLastError();
}
template <int DT>
hipError_t norm_dt(const NormArgs& a, hipStream_t s) {
  const int nc = a.k / 8;
  // Up to two rows per CU the time is one chain of latencies (load, sum, store),
  // shortest with one chunk per thread; with more rows several workgroups share
  // a CU, and smaller ones fit better: k = 8192, 1 row 3.0 us with 1024 threads
  // and 3.7 with 256, 256 rows 4.1 and 4.7, 1024 rows 11.7 and 10.6, 2048 rows
  // 21.2 and 19.8.
  const bool few = a.m <= 512;
  if (nc <= 64) return norm_nt<DT, 64, 1>(a, s);
  if (nc <= 128) return norm_nt<DT, 128, 1>(a, s);
  if (nc <= 256) return norm_nt<DT, 256, 1>(a, s);
  if (nc <= 512) return few ? norm_nt<DT, 512, 1>(a, s) : norm_nt<DT, 256, 2>(a, s);
  if (nc <= 1024) return few ? norm_nt<DT, 1024, 1>(a, s) : norm_nt<DT, 256, 4>(a, s);
  if (nc <= 2048) return norm_nt<DT, 256, 8>(a, s);
  return norm_nt<DT, 256, 0>(a, s);
}

template <int DT, int RT>
hipError_t rows_rt(RowsArgs a, hipStream_t s) {
  constexpr int U = 2;
  constexpr int per = 16 / RT * U;
  a.kt = (a.kb + per - 1) / per;
  const dim3 grid((unsigned)((int64_t)a.kt * ((a.m + RT - 1) / RT)));
  quantize_rows_kernel<DT, RT, U><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int DT>
hipError_t rows_dt(const RowsArgs& a, hipStream_t s) {
  if (a.m >= 16) return rows_rt<DT, 16>(a, s);
  if (a.m >= 4) return rows_rt<DT, 4>(a, s);
  return rows_rt<DT, 1>(a, s);
}

}  // namespace

hipError_t launch_add_rmsnorm(const uint16_t* x, int dt, int64_t m, int64_t k, int64_t ldx,
                              const uint16_t* res, uint16_t* res_out, int64_t ldr,
                              const uint16_t* gain, float eps, uint16_t* y, uint8_t* q,
                              float* scales, hipStream_t s) {
  const NormArgs a{x, res, res_out, gain, y, q, scales, ldx, ldr, (int)m, (int)k, eps};
  return dt == WQ_BF16 ? norm_dt<WQ_BF16>(a, s) : norm_dt<WQ_F16>(a, s);
}

hipError_t launch_quantize_fp8_rows(const uint16_t* x, const uint16_t* up, int dt, int64_t m,
                                    int64_t k, uint8_t* q, float* scales, hipStream_t s) {
  const RowsArgs a{x, up, q, scales, (int)m, (int)k, (int)((k + kF8Block - 1) / kF8Block), 0};
  return dt == WQ_BF16 ? rows_dt<WQ_BF16>(a, s) : rows_dt<WQ_F16>(a, s);
}

hipError_t launch_quantize_fp8_block(const uint16_t* w, int dt, int64_t n, int64_t k, uint8_t* q,
                                     float* scales, hipStream_t s) {
  const int64_t kb = (k + kF8Block - 1) / kF8Block, nb = (n + kF8Block - 1) / kF8Block;
  const dim3 grid((unsigned)(kb * nb));
  if (dt == WQ_BF16)
    quantize_block_kernel<WQ_BF16><<<grid, 256, 0, s>>>(w, n, k, (int)kb, q, scales);
  else
    quantize_block_kernel<WQ_F16><<<grid, 256, 0, s>>>(w, n, k, (int)kb, q, scales);
  return hipGetLastError();
}

}  // namespace wq
