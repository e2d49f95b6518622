// Residual addition with root-mean-square norm, and the FP8 packers.
//
// add_rmsnorm, per row of k values:
//   h = x + residual                      (fp32; residual_out = round16(h))
//   v = h * rsqrt(sum(h^2) / k + eps) * gain
//   y = round16(v), and per 128 values of v:  s = max|v| / 448, q = E4M3(v / s)
// The norm is taken of the unrounded h; every statistic is fp32.  The row
// stays in registers between the sum and the outputs, so each input is read
// once and each output written once: the kernel is bound by HBM for many rows
// and by the latency of one load, one barrier and one store for few.
//
// quantize_rows: the same scale and code for given rows, or for silu(x) * up
// (what stands between the gate/up and the down product of an MLP).
//
// quantize_block: weights, one scale per 128 x 128 block.
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

// h of one 16-byte chunk
template <int DT>
__device__ __forceinline__ void norm_load(const NormArgs& a, int64_t row, int c, float (&h)[8]) {
  unpack8<DT>(*reinterpret_cast<const uint4_t*>(a.x + row * a.ldx + c * 8), h);
  if (a.res != nullptr) {
    float r[8];
    unpack8<DT>(*reinterpret_cast<const uint4_t*>(a.res + row * a.ldr + c * 8), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += r[i];
  }
}

// the outputs of one chunk; the 16 lanes of a scale block are consecutive and
// all call this (`live` false past the end of the row)
template <int DT>
__device__ __forceinline__ void norm_store(const NormArgs& a, int64_t row, int c, bool live,
                                           const float (&h)[8], uint4_t graw, float rstd) {
  if (a.res_out != nullptr && live)
    *reinterpret_cast<uint4_t*>(a.res_out + row * a.ldr + c * 8) = pack8<DT>(h);
  float g[8], v[8];
  unpack8<DT>(graw, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = h[i] * rstd * g[i];
  if (a.y != nullptr && live)
    *reinterpret_cast<uint4_t*>(a.y + row * a.k + c * 8) = pack8<DT>(v);
  if (a.q != nullptr) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, abs_bits(v[i]));
    const float s = fp8_scale(max16(live ? big : 0u));
    const float inv = __fdiv_rn(1.0f, s);
    if (live) {
      const uint2_t o = {pack4_fp8(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                         pack4_fp8(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
      *reinterpret_cast<uint2_t*>(a.q + row * a.k + c * 8) = o;
      if ((c & 15) == 0) a.scales[(int64_t)(c >> 4) * a.m + row] = s;
    }
  }
}

// Sum over the workgroup, in every thread.  `part` holds one float per wave;
// two of them alternate from row to row, so one barrier per row is enough.
template <int NT>
__device__ __forceinline__ float wg_sum(float v, float* part) {
  v = sum64(v);
  if constexpr (NT == 64) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) t += part[i];
  return t;
}

// V chunks of 8 values per thread; V = 0: rows of any length, read twice
template <int DT, int NT, int V>
__global__ __launch_bounds__(NT) void add_rmsnorm_kernel(NormArgs a, int rows_per_wg) {
  __shared__ float part[2][NT / 64];
  const int tid = threadIdx.x;
  const int nc = a.k / 8;
  const float rk = __fdiv_rn(1.0f, (float)a.k);
  const int64_t r0 = (int64_t)blockIdx.x * rows_per_wg;
  const int64_t r1 = r0 + rows_per_wg < a.m ? r0 + rows_per_wg : a.m;
  constexpr int VN = V > 0 ? V : 1;
  uint4_t g[VN];
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = tid + j * NT;
      g[j] = c < nc ? *reinterpret_cast<const uint4_t*>(a.gain + c * 8) : uint4_t{0, 0, 0, 0};
    }
  }
  for (int64_t row = r0; row < r1; ++row) {
    float* const p = part[(row - r0) & 1];
    float ss = 0.0f;
    if constexpr (V > 0) {
      float h[VN][8];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = tid + j * NT;
        if (c < nc) {
          norm_load<DT>(a, row, c, h[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
      const float rstd = rsqrtf(wg_sum<NT>(ss, p) * rk + a.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = tid + j * NT;
        norm_store<DT>(a, row, c, c < nc, h[j], g[j], rstd);
      }
    } else {
      for (int c = tid; c < nc; c += NT) {
        float h[8];
        norm_load<DT>(a, row, c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
      }
      const float rstd = rsqrtf(wg_sum<NT>(ss, p) * rk + a.eps);
      // every value is read by the thread that writes it, so residual_out
      // may be the residual itself; all lanes take part in each round
      for (int c0 = 0; c0 < nc; c0 += NT) {
        const int c = c0 + tid;
        const bool live = c < nc;
        float h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        uint4_t gr = {0, 0, 0, 0};
        if (live) {
          norm_load<DT>(a, row, c, h);
          gr = *reinterpret_cast<const uint4_t*>(a.gain + (int64_t)c * 8);
        }
        norm_store<DT>(a, row, c, live, h, gr, rstd);
      }
    }
  }
}

struct RowsArgs {
  const uint16_t* x;
  const uint16_t* up;        // or nullptr
  uint8_t* q;
  float* scales;
  int m, k, kb;
};

// 16 lanes per scale block; a workgroup takes RT rows x 16/RT blocks of k in
// each of U rounds, so with RT = 16 the scales it writes are 64 contiguous
// bytes per block of k
template <int DT, int RT, int U>
__global__ __launch_bounds__(256) void quantize_rows_kernel(RowsArgs a) {
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * RT + sub % RT;
  const int b0 = ((int)blockIdx.y * U) * (16 / RT) + sub / RT;
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
    const float inv = __fdiv_rn(1.0f, s);
    if (live[u]) {
      const uint2_t o = {
          pack4_fp8(v[u][0] * inv, v[u][1] * inv, v[u][2] * inv, v[u][3] * inv),
          pack4_fp8(v[u][4] * inv, v[u][5] * inv, v[u][6] * inv, v[u][7] * inv)};
      *reinterpret_cast<uint2_t*>(a.q + row * a.k + c) = o;
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
  const float inv = __fdiv_rn(1.0f, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = nb * kF8Block + j * 16 + sub;
    if (row < n && c < k) {
      const uint2_t o = {
          pack4_fp8(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv),
          pack4_fp8(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv)};
      *reinterpret_cast<uint2_t*>(q + row * k + c) = o;
    }
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

template <int DT>
hipError_t norm_dt(const NormArgs& a, hipStream_t s) {
  constexpr int NT = 256;
  const int nc = a.k / 8;
  // workgroups of at least one row; many rows run as consecutive ranges
  const int64_t wgs = a.m < 2048 ? a.m : 2048;
  const int per = (int)((a.m + wgs - 1) / wgs);
  const dim3 grid((unsigned)((a.m + per - 1) / per));
  if (nc <= NT) add_rmsnorm_kernel<DT, NT, 1><<<grid, NT, 0, s>>>(a, per);
  else if (nc <= 2 * NT) add_rmsnorm_kernel<DT, NT, 2><<<grid, NT, 0, s>>>(a, per);
  else if (nc <= 4 * NT) add_rmsnorm_kernel<DT, NT, 4><<<grid, NT, 0, s>>>(a, per);
  else if (nc <= 8 * NT) add_rmsnorm_kernel<DT, NT, 8><<<grid, NT, 0, s>>>(a, per);
  else add_rmsnorm_kernel<DT, NT, 0><<<grid, NT, 0, s>>>(a, per);
  return hipGetLastError();
}

template <int DT, int RT>
hipError_t rows_rt(const RowsArgs& a, hipStream_t s) {
  constexpr int U = 4;
  const int per = 16 / RT * U;
  const dim3 grid((unsigned)((a.m + RT - 1) / RT), (unsigned)((a.kb + per - 1) / per));
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
  const RowsArgs a{x, up, q, scales, (int)m, (int)k, (int)((k + kF8Block - 1) / kF8Block)};
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
