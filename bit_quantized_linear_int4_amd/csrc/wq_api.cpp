// C ABI of libwq: argument validation, schedule choice, launch.
//
// Every check runs before the first HIP call, so an error other than
// WQ_ERR_HIP means nothing was enqueued.  No C++ exception crosses the ABI.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "internal.h"

using namespace wq;

namespace {

// Size limits: every dimension below 2^23 and every matrix at most 2^34
// elements, so every launch's grid stays within 32-bit work-item counts.
constexpr int64_t kMaxDim = int64_t(1) << 23;
constexpr int64_t kMaxElems = int64_t(1) << 34;
// LLM.int8: the int32 accumulator holds 127 * 127 * k exactly for k up to
// this bound (k multiples of 128: 133,120 at most).
constexpr int64_t kMaxInt8K = ((int64_t(1) << 31) - 1) / (127 * 127);

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is16(int32_t dt) { return dt == WQ_F16 || dt == WQ_BF16; }
bool is_out(int32_t dt) { return dt == WQ_F16 || dt == WQ_BF16 || dt == WQ_F32; }
uintptr_t dt_bytes(int32_t dt) { return dt == WQ_F32 ? 4 : 2; }

wq_status hip_status(hipError_t e) { return e == hipSuccess ? WQ_OK : WQ_ERR_HIP; }

bool sizes_ok(int64_t n, int64_t k) {
  return n >= 1 && k >= 1 && n < kMaxDim && k < kMaxDim && n <= kMaxElems / k;
}

// Validates a weight descriptor for the given use.  `linear_w4` restricts to
// the formats and group sizes wq_linear_w4a16 runs.
wq_status check_weight(const wq_weight* w, bool linear_w4) {
  if (w == nullptr || w->codes == nullptr || w->scales == nullptr) return WQ_ERR_NULL;
  if (!sizes_ok(w->n, w->k)) return WQ_ERR_SHAPE;
  if (!aligned(w->codes, 16)) return WQ_ERR_ALIGN;
  if (w->perm != nullptr) {
    if (w->fmt != WQ_FMT_INT4_ASYM) return WQ_ERR_UNSUPPORTED;   // act-order is INT4 only
    if (!aligned(w->perm, 4)) return WQ_ERR_ALIGN;
  }
  switch (w->fmt) {
    case WQ_FMT_INT4_ASYM:
      if (w->zeros == nullptr) return WQ_ERR_NULL;
      if (w->group != 32 && w->group != 64 && w->group != 128) return WQ_ERR_UNSUPPORTED;
      if (w->k % w->group != 0 || w->k % 8 != 0) return WQ_ERR_SHAPE;
      if (!aligned(w->scales, 2)) return WQ_ERR_ALIGN;
      return WQ_OK;
    case WQ_FMT_NF4:
    case WQ_FMT_FP4:
      if (w->group != 64) return WQ_ERR_UNSUPPORTED;
      if (w->scales2 != nullptr && w->group2 != 256) return WQ_ERR_UNSUPPORTED;
      if ((w->n * w->k) % 64 != 0 || w->k % 8 != 0) return WQ_ERR_SHAPE;
      if (w->scales2 == nullptr && !aligned(w->scales, 4)) return WQ_ERR_ALIGN;
      if (w->scales2 != nullptr && !aligned(w->scales2, 4)) return WQ_ERR_ALIGN;
      return WQ_OK;
    case WQ_FMT_INT8_SYM_ROW:
      if (linear_w4) return WQ_ERR_UNSUPPORTED;
      if (w->group != w->k || w->k % 16 != 0) return WQ_ERR_SHAPE;
      if (!aligned(w->scales, 4)) return WQ_ERR_ALIGN;
      return WQ_OK;
    case WQ_FMT_FP8_BLOCK:
      if (linear_w4) return WQ_ERR_UNSUPPORTED;
      if (w->group != 128) return WQ_ERR_UNSUPPORTED;
      if (w->k % 16 != 0) return WQ_ERR_SHAPE;
      if (!aligned(w->scales, 4)) return WQ_ERR_ALIGN;
      return WQ_OK;
    default:
      return WQ_ERR_UNSUPPORTED;
  }
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Workspace of wq_linear_w4a16: the activations gathered into the order of
// an act-order weight (m x k 16-bit values); none for any other weight.
size_t linear_ws_bytes(int64_t m, const wq_weight* w) {
  if (w->perm == nullptr) return 0;
  return round256((size_t)m * (size_t)w->k * 2);
}

// FP4 weights run the NF4 kernels with the FP4 level table.
const float* levels_for(const wq_weight* w) {
  return w->fmt == WQ_FMT_FP4 ? fp4_levels() : nf4_levels();
}
wq_weight kernel_view(const wq_weight* w) {
  wq_weight c = *w;
  if (c.fmt == WQ_FMT_FP4) c.fmt = WQ_FMT_NF4;
  return c;
}

}  // namespace

extern "C" {

const char* wq_status_string(int32_t status) {
  switch (status) {
    case WQ_OK: return "WQ_OK";
    case WQ_ERR_NULL: return "WQ_ERR_NULL: a required pointer is NULL";
    case WQ_ERR_SHAPE: return "WQ_ERR_SHAPE: sizes do not fit the format";
    case WQ_ERR_ALIGN: return "WQ_ERR_ALIGN: a pointer misses its alignment";
    case WQ_ERR_UNSUPPORTED: return "WQ_ERR_UNSUPPORTED: combination not implemented";
    case WQ_ERR_WORKSPACE: return "WQ_ERR_WORKSPACE: workspace missing or too small";
    case WQ_ERR_HIP: return "WQ_ERR_HIP: kernel launch failed";
    default: return "unknown wq_status";
  }
}

wq_status wq_fp4_codebook(float* out) {
  if (out == nullptr) return WQ_ERR_NULL;
  const float* l = fp4_levels();
  for (int i = 0; i < 16; ++i) out[i] = l[i];
  return WQ_OK;
}

wq_status wq_nf4_codebook(float* out) {
  if (out == nullptr) return WQ_ERR_NULL;
  const float* l = nf4_levels();
  for (int i = 0; i < 16; ++i) out[i] = l[i];
  return WQ_OK;
}

wq_status wq_quantize_groupwise(const void* w, int32_t wdt, int64_t n, int64_t k, int32_t bits,
                                int32_t group, int32_t symmetric, void* codes, void* scales,
                                uint8_t* zeros, void* stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr) return WQ_ERR_NULL;
  if (!is16(wdt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(n, k) || k % 8 != 0) return WQ_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(codes, 16)) return WQ_ERR_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (bits == 4 && symmetric == 0) {
    if (zeros == nullptr) return WQ_ERR_NULL;
    if (group != 32 && group != 64 && group != 128) return WQ_ERR_UNSUPPORTED;
    if (k % group != 0) return WQ_ERR_SHAPE;
    if (!aligned(scales, 2)) return WQ_ERR_ALIGN;
    return hip_status(launch_quant_int4(w, wdt, n, k, group, static_cast<uint32_t*>(codes),
                                        static_cast<uint16_t*>(scales), zeros, s));
  }
  if (bits == 8 && symmetric == 1) {
    if (group != k) return WQ_ERR_UNSUPPORTED;
    if (zeros != nullptr) return WQ_ERR_UNSUPPORTED;
    if (!aligned(scales, 4)) return WQ_ERR_ALIGN;
    return hip_status(launch_quant_int8_rows(w, wdt, n, k, static_cast<int8_t*>(codes),
                                             static_cast<float*>(scales), s));
  }
  return WQ_ERR_UNSUPPORTED;
}

static wq_status pack_blockwise(const void* w, int32_t wdt, int64_t n, int64_t k, int32_t block,
                                int32_t double_quant, int32_t block2, uint8_t* codes,
                                void* absmax, float* absmax_scale, void* stream, bool fp4) {
  if (w == nullptr || codes == nullptr || absmax == nullptr) return WQ_ERR_NULL;
  if (!is16(wdt)) return WQ_ERR_UNSUPPORTED;
  if (block != 64) return WQ_ERR_UNSUPPORTED;
  if (double_quant) {
    if (absmax_scale == nullptr) return WQ_ERR_NULL;
    if (block2 != 256) return WQ_ERR_UNSUPPORTED;
    if (!aligned(absmax_scale, 4)) return WQ_ERR_ALIGN;
  } else {
    if (absmax_scale != nullptr) return WQ_ERR_UNSUPPORTED;
    if (!aligned(absmax, 4)) return WQ_ERR_ALIGN;
  }
  if (!sizes_ok(n, k) || (n * k) % 64 != 0) return WQ_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(codes, 16)) return WQ_ERR_ALIGN;
  return hip_status(launch_pack_nf4(w, wdt, n * k, double_quant ? 1 : 0,
                                    fp4 ? fp4_thresholds() : nf4_thresholds(), codes, absmax,
                                    absmax_scale, static_cast<hipStream_t>(stream), fp4));
}

wq_status wq_pack_nf4(const void* w, int32_t wdt, int64_t n, int64_t k, int32_t block,
                      int32_t double_quant, int32_t block2, uint8_t* codes, void* absmax,
                      float* absmax_scale, void* stream) {
  return pack_blockwise(w, wdt, n, k, block, double_quant, block2, codes, absmax, absmax_scale,
                        stream, false);
}

wq_status wq_pack_fp4(const void* w, int32_t wdt, int64_t n, int64_t k, int32_t block,
                      int32_t double_quant, int32_t block2, uint8_t* codes, void* absmax,
                      float* absmax_scale, void* stream) {
  return pack_blockwise(w, wdt, n, k, block, double_quant, block2, codes, absmax, absmax_scale,
                        stream, true);
}

size_t wq_linear_w4a16_workspace(int64_t m, const wq_weight* w) {
  if (m < 1 || m >= kMaxDim || check_weight(w, true) != WQ_OK) return 0;
  return linear_ws_bytes(m, w);
}

wq_status wq_linear_w4a16(const void* x, int32_t xdt, int64_t m, const wq_weight* w, void* y,
                          int32_t ydt, void* workspace, size_t ws_bytes, void* stream) {
  if (x == nullptr || y == nullptr) return WQ_ERR_NULL;
  const wq_status ws = check_weight(w, true);
  if (ws != WQ_OK) return ws;
  if (!is16(xdt) || !is_out(ydt)) return WQ_ERR_UNSUPPORTED;
  if (m < 1 || m >= kMaxDim || m > kMaxElems / w->k || m > kMaxElems / w->n)
    return WQ_ERR_SHAPE;
  if (w->k % 128 != 0) return WQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, dt_bytes(ydt))) return WQ_ERR_ALIGN;
  const wq_weight kv = kernel_view(w);
  const W4Plan plan = plan_w4a16(m, &kv);
  const size_t need = linear_ws_bytes(m, w);
  if (need > 0) {
    if (workspace == nullptr || ws_bytes < need) return WQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return WQ_ERR_ALIGN;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (w->perm != nullptr) {
    // act-order: x[:, perm] into the workspace, then the plain linear on it
    void* xp = workspace;
    const hipError_t e = launch_permute_cols(static_cast<const uint16_t*>(x), m, w->k, w->perm,
                                             static_cast<uint16_t*>(xp), s);
    if (e != hipSuccess) return WQ_ERR_HIP;
    x = xp;
  }
  return hip_status(launch_w4a16(x, xdt, m, &kv, levels_for(w), y, ydt, plan, s));
}

wq_status wq_linear_w4a16_gate_up(const void* x, int32_t xdt, int64_t m,
                                  const wq_weight* w_gate, const wq_weight* w_up, int32_t act,
                                  void* y_gate, void* y_up, int32_t ydt, void* stream) {
  if (x == nullptr || y_gate == nullptr) return WQ_ERR_NULL;
  if (act != 0 && act != 1) return WQ_ERR_UNSUPPORTED;
  if (act == 0 && y_up == nullptr) return WQ_ERR_NULL;
  wq_status st = check_weight(w_gate, true);
  if (st != WQ_OK) return st;
  st = check_weight(w_up, true);
  if (st != WQ_OK) return st;
  // both matrices in one format (INT4, NF4 or FP4), NF4/FP4 both with or both
  // without double quantization
  if (w_gate->fmt != w_up->fmt || w_gate->fmt == WQ_FMT_INT8_SYM_ROW) return WQ_ERR_UNSUPPORTED;
  if ((w_gate->scales2 == nullptr) != (w_up->scales2 == nullptr) ||
      (w_gate->scales2 != nullptr && w_gate->group2 != w_up->group2))
    return WQ_ERR_UNSUPPORTED;
  if (w_gate->perm != nullptr || w_up->perm != nullptr) return WQ_ERR_UNSUPPORTED;
  if (!is16(xdt) || !is_out(ydt)) return WQ_ERR_UNSUPPORTED;
  if (w_gate->n != w_up->n || w_gate->k != w_up->k || w_gate->group != w_up->group ||
      w_gate->k % 128 != 0)
    return WQ_ERR_SHAPE;
  if (m < 1 || m >= kMaxDim || m > kMaxElems / w_gate->k || m > kMaxElems / w_gate->n)
    return WQ_ERR_SHAPE;
  // act 1 with m > 16 runs two GEMMs and needs y_up to hold the up projection
  const bool up_out = act == 0 || m > 16;
  if (act == 1 && m > 16 && y_up == nullptr) return WQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y_gate, dt_bytes(ydt)) ||
      (up_out && !aligned(y_up, dt_bytes(ydt))))
    return WQ_ERR_ALIGN;
  const wq_weight kg = kernel_view(w_gate), ku = kernel_view(w_up);
  const W4Plan plan = plan_w4a16_pair(m, &kg, &ku);
  return hip_status(launch_w4a16_pair(x, xdt, m, &kg, &ku, levels_for(w_gate), act, y_gate,
                                      up_out ? y_up : nullptr, ydt, plan,
                                      static_cast<hipStream_t>(stream)));
}

size_t wq_linear_int8_decomp_workspace(int64_t m, int64_t k) {
  if (m < 1 || k < 16 || k % 16 != 0 || !sizes_ok(m, k)) return 0;
  // mask u8[k] | idx i32[k] | count i32 | qx i8[m][k] | sx f32[m], each 256-aligned
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  return up((size_t)k) + up(4 * (size_t)k) + up(4) + up((size_t)m * (size_t)k) + up(4 * (size_t)m);
}

wq_status wq_int8_prepare_activations(const void* x, int64_t m, int64_t k, float threshold,
                                      uint8_t* mask, int32_t* idx, int32_t* count, int8_t* qx,
                                      float* sx, void* stream) {
  if (x == nullptr || mask == nullptr || idx == nullptr || count == nullptr || qx == nullptr ||
      sx == nullptr)
    return WQ_ERR_NULL;
  if (!sizes_ok(m, k) || k % 16 != 0) return WQ_ERR_SHAPE;
  if (!(threshold >= 0.0f)) return WQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(qx, 16) || !aligned(mask, 16) || !aligned(idx, 4) ||
      !aligned(count, 4) || !aligned(sx, 4))
    return WQ_ERR_ALIGN;
  return hip_status(launch_int8_prepare(static_cast<const uint16_t*>(x), m, k, threshold, mask,
                                        idx, count, qx, sx, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Argument checks shared by the two LLM.int8 entry points (everything but
// the workspace).
wq_status check_int8_decomp(const void* x, int64_t m, const wq_weight* w, float threshold,
                            const void* y, int32_t ydt, const int32_t* outlier_count,
                            const int32_t* acc_out) {
  if (x == nullptr || y == nullptr) return WQ_ERR_NULL;
  const wq_status st = check_weight(w, false);
  if (st != WQ_OK) return st;
  if (w->fmt != WQ_FMT_INT8_SYM_ROW) return WQ_ERR_UNSUPPORTED;
  if (!is_out(ydt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(m, w->k) || m > kMaxElems / w->n || w->k % 128 != 0 || w->k > kMaxInt8K)
    return WQ_ERR_SHAPE;
  if (!(threshold >= 0.0f)) return WQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, dt_bytes(ydt))) return WQ_ERR_ALIGN;
  if (outlier_count != nullptr && !aligned(outlier_count, 4)) return WQ_ERR_ALIGN;
  if (acc_out != nullptr && !aligned(acc_out, 4)) return WQ_ERR_ALIGN;
  return WQ_OK;
}

// The two launches of the decomposition with the scratch at `base`
// (256-byte aligned, at least wq_linear_int8_decomp_workspace(m, k) bytes).
// Every scratch byte a kernel reads was written earlier in the same call, so
// the scratch needs no clearing.
wq_status run_int8_decomp(const void* x, int64_t m, const wq_weight* w, float threshold, void* y,
                          int32_t ydt, char* base, int32_t* outlier_count, int32_t* acc_out,
                          hipStream_t s) {
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  const size_t k = (size_t)w->k;
  uint8_t* mask = reinterpret_cast<uint8_t*>(base);
  int32_t* idx = reinterpret_cast<int32_t*>(base + up(k));
  int32_t* count = reinterpret_cast<int32_t*>(base + up(k) + up(4 * k));
  int8_t* qx = reinterpret_cast<int8_t*>(base + up(k) + up(4 * k) + up(4));
  float* sx = reinterpret_cast<float*>(base + up(k) + up(4 * k) + up(4) + up((size_t)m * k));
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  hipError_t e = launch_int8_prepare(xp, m, w->k, threshold, mask, idx, count, qx, sx, s);
  if (e != hipSuccess) return WQ_ERR_HIP;
  e = launch_int8_gemm(xp, m, w, qx, sx, idx, count, y, ydt, acc_out, s);
  if (e != hipSuccess) return WQ_ERR_HIP;
  if (outlier_count != nullptr) {
    e = hipMemcpyAsync(outlier_count, count, sizeof(int32_t), hipMemcpyDeviceToDevice, s);
    if (e != hipSuccess) return WQ_ERR_HIP;
  }
  return WQ_OK;
}

// Scratch of wq_linear_int8_decomp_noalloc: a device array of fixed size,
// one copy per GPU, held until the process ends.  In host code `scratch`
// names a host-side stand-in, not device memory: kernels get the address
// hipGetSymbolAddress returns for the current device, looked up once per
// device and kept in `g_scratch`.
constexpr size_t kNoAllocScratchBytes = WQ_INT8_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 64;
std::atomic<void*> g_scratch[kMaxDevices];
std::mutex g_scratch_mu;

// The current device's scratch address, or nullptr if it cannot be had.
void* device_scratch() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  void* p = g_scratch[dev].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  p = g_scratch[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess) return nullptr;
    g_scratch[dev].store(p, std::memory_order_release);
  }
  return p;
}

constexpr int64_t kMaxHeads = 1024;

// m rows of `row` elements, ld apart
bool rows_ok(int64_t m, int64_t row, int64_t ld) {
  return sizes_ok(m, row) && ld >= row && ld < kMaxDim && ld % 8 == 0;
}

wq_status check_cache(const wq_kv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return WQ_ERR_NULL;
  const bool f8 = c->dt == WQ_E4M3;
  if (!f8 && !is16(c->dt)) return WQ_ERR_UNSUPPORTED;
  if (f8 && (c->k_scales == nullptr || c->v_scales == nullptr)) return WQ_ERR_NULL;
  if (!f8 && (c->k_scales != nullptr || c->v_scales != nullptr)) return WQ_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return WQ_ERR_UNSUPPORTED;
  if (c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->pages < 1) return WQ_ERR_SHAPE;
  if (c->page_size < 1 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0)
    return WQ_ERR_SHAPE;
  if (c->pages > INT32_MAX / c->page_size) return WQ_ERR_SHAPE;
  struct {
    int64_t n, stride;
  } dim[3] = {{c->pages, c->page_stride}, {c->kv_heads, c->head_stride},
              {c->page_size, c->token_stride}};
  const int64_t unit = f8 ? 16 : 8;
  std::sort(dim, dim + 3, [](const auto& a, const auto& b) { return a.stride < b.stride; });
  int64_t span = c->head_dim;                    // elements that the dimensions so far cover
  for (const auto& t : dim) {
    if (t.n == 1) continue;
    if (t.stride < span || t.stride % unit != 0) return WQ_ERR_SHAPE;
    if (t.stride > (kMaxElems - span) / (t.n - 1)) return WQ_ERR_SHAPE;
    span += t.stride * (t.n - 1);
  }
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) ||
      !aligned(c->v_scales, 4))
    return WQ_ERR_ALIGN;
  return WQ_OK;
}

KvCache kernel_cache(const wq_kv_cache* c) {
  const int64_t b = c->dt == WQ_E4M3 ? 1 : 2;
  // the stride of a dimension of one place is never used: any value may stand there
  auto bytes = [b](int64_t n, int64_t stride) { return n == 1 ? 0 : stride * b; };
  return KvCache{static_cast<char*>(c->k), static_cast<char*>(c->v), c->k_scales, c->v_scales,
                 bytes(c->pages, c->page_stride), bytes(c->kv_heads, c->head_stride),
                 bytes(c->page_size, c->token_stride), c->dt, c->kv_heads, c->head_dim,
                 __builtin_ctz((unsigned)c->page_size), (int32_t)c->pages};
}

bool attention_sizes_ok(int64_t m, int64_t heads, const wq_kv_cache* cache) {
  return check_cache(cache) == WQ_OK && heads >= 1 && heads <= kMaxHeads &&
         heads % cache->kv_heads == 0 && sizes_ok(m, heads * cache->head_dim);
}

// the checks that both attention calls share; fills everything but starts and ws
wq_status check_attention(const void* q, int32_t dt, int64_t m, int64_t heads, int64_t ldq,
                          int64_t batch, const wq_kv_cache* cache, const int32_t* pages,
                          int64_t max_pages, int64_t ldp, const int32_t* lens, float scale,
                          int64_t window, int64_t sinks, void* y, float* lse, AttentionCall* c) {
  if (q == nullptr || pages == nullptr || lens == nullptr || y == nullptr) return WQ_ERR_NULL;
  const wq_status st = check_cache(cache);
  if (st != WQ_OK) return st;
  if (!is16(dt) || (cache->dt != WQ_E4M3 && cache->dt != dt)) return WQ_ERR_UNSUPPORTED;
  if (!attention_sizes_ok(m, heads, cache) || !rows_ok(m, heads * cache->head_dim, ldq))
    return WQ_ERR_SHAPE;
  if (batch < 1 || batch >= kMaxDim || !sizes_ok(batch, max_pages) || ldp < max_pages ||
      ldp >= kMaxDim || max_pages > kNoWindow / cache->page_size)
    return WQ_ERR_SHAPE;
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0 || sinks < 0) return WQ_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(pages, 4) || !aligned(lens, 4) || !aligned(y, 16) ||
      !aligned(lse, 4))
    return WQ_ERR_ALIGN;
  auto i32 = [](int64_t v) { return (int32_t)std::min<int64_t>(v, kNoWindow); };
  *c = AttentionCall{static_cast<const uint16_t*>(q), dt, m, heads, ldq, nullptr, batch,
                     kernel_cache(cache), pages, max_pages, ldp, lens, scale,
                     window == 0 ? kNoWindow : i32(window), i32(sinks),
                     static_cast<uint16_t*>(y), lse, nullptr};
  return WQ_OK;
}

wq_status run_attention(AttentionCall* c, void* workspace, size_t ws_bytes, size_t need,
                        void* stream) {
  if (need > 0) {
    if (workspace == nullptr || ws_bytes < need) return WQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return WQ_ERR_ALIGN;
  }
  c->ws = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return hip_status(c->starts == nullptr ? launch_attention_decode(*c, s)
                                         : launch_attention_prompt(*c, s));
}

}  // namespace

extern "C" {

wq_status wq_linear_int8_decomp(const void* x, int64_t m, const wq_weight* w, float threshold,
                                void* y, int32_t ydt, void* workspace, size_t ws_bytes,
                                int32_t* outlier_count, int32_t* acc_out, void* stream) {
  const wq_status st = check_int8_decomp(x, m, w, threshold, y, ydt, outlier_count, acc_out);
  if (st != WQ_OK) return st;
  const size_t need = wq_linear_int8_decomp_workspace(m, w->k);
  if (workspace == nullptr || ws_bytes < need) return WQ_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return WQ_ERR_ALIGN;
  return run_int8_decomp(x, m, w, threshold, y, ydt, static_cast<char*>(workspace),
                         outlier_count, acc_out, static_cast<hipStream_t>(stream));
}

wq_status wq_linear_int8_decomp_noalloc(const void* x, int64_t m, const wq_weight* w,
                                        float threshold, void* y, int32_t ydt,
                                        int32_t* outlier_count, int32_t* acc_out,
                                        void* stream) {
  const wq_status st = check_int8_decomp(x, m, w, threshold, y, ydt, outlier_count, acc_out);
  if (st != WQ_OK) return st;
  if (wq_linear_int8_decomp_workspace(m, w->k) > kNoAllocScratchBytes) return WQ_ERR_WORKSPACE;
  void* base = device_scratch();
  if (base == nullptr) return WQ_ERR_HIP;
  return run_int8_decomp(x, m, w, threshold, y, ydt, static_cast<char*>(base), outlier_count,
                         acc_out, static_cast<hipStream_t>(stream));
}

wq_status wq_permute_columns(const void* src, int32_t dt, int64_t rows, int64_t k,
                             const int32_t* perm, void* dst, void* stream) {
  if (src == nullptr || perm == nullptr || dst == nullptr) return WQ_ERR_NULL;
  if (!is16(dt)) return WQ_ERR_UNSUPPORTED;
  if (src == dst) return WQ_ERR_UNSUPPORTED;                 // not in place
  if (!sizes_ok(rows, k) || k % 8 != 0) return WQ_ERR_SHAPE;
  if (!aligned(src, 2) || !aligned(dst, 16) || !aligned(perm, 4)) return WQ_ERR_ALIGN;
  return hip_status(launch_permute_cols(static_cast<const uint16_t*>(src), rows, k, perm,
                                        static_cast<uint16_t*>(dst),
                                        static_cast<hipStream_t>(stream)));
}

wq_status wq_scale_columns(const void* src, int32_t dt, int64_t rows, int64_t k,
                           const float* scale, void* dst, void* stream) {
  if (src == nullptr || scale == nullptr || dst == nullptr) return WQ_ERR_NULL;
  if (!is16(dt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(rows, k) || k % 8 != 0) return WQ_ERR_SHAPE;
  if (!aligned(src, 16) || !aligned(dst, 16) || !aligned(scale, 4)) return WQ_ERR_ALIGN;
  return hip_status(launch_scale_cols(static_cast<const uint16_t*>(src), dt, rows, k, scale,
                                      static_cast<uint16_t*>(dst),
                                      static_cast<hipStream_t>(stream)));
}

wq_status wq_add_rmsnorm(const void* x, int32_t dt, int64_t m, int64_t k, int64_t ldx,
                         const void* residual, void* residual_out, int64_t ldr,
                         const void* gain, float eps, void* y, void* q, float* scales,
                         void* stream) {
  if (x == nullptr || gain == nullptr || (y == nullptr && q == nullptr)) return WQ_ERR_NULL;
  if ((residual == nullptr) != (residual_out == nullptr)) return WQ_ERR_NULL;
  if ((q == nullptr) != (scales == nullptr)) return WQ_ERR_NULL;
  if (!is16(dt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(m, k) || k % 8 != 0) return WQ_ERR_SHAPE;
  if (ldx < k || ldx >= kMaxDim || ldx % 8 != 0) return WQ_ERR_SHAPE;
  if (residual != nullptr && (ldr < k || ldr >= kMaxDim || ldr % 8 != 0)) return WQ_ERR_SHAPE;
  if (!(eps >= 0.0f)) return WQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(gain, 16) || !aligned(residual, 16) ||
      !aligned(residual_out, 16) || !aligned(y, 16) || !aligned(q, 8) || !aligned(scales, 4))
    return WQ_ERR_ALIGN;
  return hip_status(launch_add_rmsnorm(
      static_cast<const uint16_t*>(x), dt, m, k, ldx, static_cast<const uint16_t*>(residual),
      static_cast<uint16_t*>(residual_out), ldr, static_cast<const uint16_t*>(gain), eps,
      static_cast<uint16_t*>(y), static_cast<uint8_t*>(q), scales,
      static_cast<hipStream_t>(stream)));
}

wq_status wq_quantize_fp8_rows(const void* x, const void* up, int32_t dt, int64_t m, int64_t k,
                               void* q, float* scales, void* stream) {
  if (x == nullptr || q == nullptr || scales == nullptr) return WQ_ERR_NULL;
  if (!is16(dt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(m, k) || k % 8 != 0) return WQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(up, 16) || !aligned(q, 8) || !aligned(scales, 4))
    return WQ_ERR_ALIGN;
  return hip_status(launch_quantize_fp8_rows(
      static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(up), dt, m, k,
      static_cast<uint8_t*>(q), scales, static_cast<hipStream_t>(stream)));
}

wq_status wq_quantize_fp8_block(const void* w, int32_t wdt, int64_t n, int64_t k, void* codes,
                                float* scales, void* stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr) return WQ_ERR_NULL;
  if (!is16(wdt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(n, k) || k % 16 != 0) return WQ_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return WQ_ERR_ALIGN;
  return hip_status(launch_quantize_fp8_block(static_cast<const uint16_t*>(w), wdt, n, k,
                                              static_cast<uint8_t*>(codes), scales,
                                              static_cast<hipStream_t>(stream)));
}

size_t wq_linear_fp8_workspace(int64_t m, const wq_weight* w) {
  if (check_weight(w, false) != WQ_OK || w->fmt != WQ_FMT_FP8_BLOCK) return 0;
  if (!sizes_ok(m, w->k) || m > kMaxElems / w->n) return 0;
  // enough for every type of y
  return std::max(plan_fp8(m, w->n, w->k, WQ_F32).ws_bytes,
                  plan_fp8(m, w->n, w->k, WQ_F16).ws_bytes);
}

wq_status wq_linear_fp8(const void* q, const float* scales, int64_t m, const wq_weight* w,
                        void* y, int32_t ydt, void* workspace, size_t ws_bytes, void* stream) {
  if (q == nullptr || scales == nullptr || y == nullptr) return WQ_ERR_NULL;
  const wq_status st = check_weight(w, false);
  if (st != WQ_OK) return st;
  if (w->fmt != WQ_FMT_FP8_BLOCK || !is_out(ydt)) return WQ_ERR_UNSUPPORTED;
  if (!sizes_ok(m, w->k) || m > kMaxElems / w->n) return WQ_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(y, 16)) return WQ_ERR_ALIGN;
  const Fp8Plan plan = plan_fp8(m, w->n, w->k, ydt);
  if (plan.ws_bytes > 0) {
    if (workspace == nullptr || ws_bytes < plan.ws_bytes) return WQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return WQ_ERR_ALIGN;
  }
  return hip_status(launch_linear_fp8(static_cast<const uint8_t*>(q), scales, m, w, y, ydt, plan,
                                      static_cast<float*>(workspace),
                                      static_cast<hipStream_t>(stream)));
}

size_t wq_moe_workspace(int64_t m, int32_t top_k, const wq_weight* gate, int64_t experts) {
  if (gate == nullptr || m < 1 || m > kMoeMaxTokens || experts < 1 || experts > kMoeMaxExperts ||
      top_k < 1 || top_k > kMoeMaxTopK || top_k > experts)
    return 0;
  if (check_weight(gate, gate->fmt != WQ_FMT_FP8_BLOCK) != WQ_OK || gate->perm != nullptr ||
      (gate->fmt != WQ_FMT_INT4_ASYM && gate->fmt != WQ_FMT_FP8_BLOCK))
    return 0;
  if (gate->k % 128 != 0 || gate->n % (experts * 128) != 0) return 0;
  return moe_ws_bytes(m, experts, top_k, gate->k, gate->n / experts);
}

wq_status wq_moe(const void* x, int32_t xdt, int64_t m, const void* router, const float* logits,
                 int64_t experts, int32_t top_k, int32_t renormalize, const wq_weight* gate,
                 const wq_weight* up, const wq_weight* down, void* y, int32_t ydt, int32_t* ids,
                 float* probs, void* workspace, size_t ws_bytes, void* stream) {
  if (x == nullptr || y == nullptr || (router == nullptr) == (logits == nullptr))
    return WQ_ERR_NULL;
  for (const wq_weight* w : {gate, up, down}) {
    if (w == nullptr) return WQ_ERR_NULL;
    const wq_status st = check_weight(w, w->fmt != WQ_FMT_FP8_BLOCK);
    if (st != WQ_OK) return st;
    if (w->fmt != WQ_FMT_INT4_ASYM && w->fmt != WQ_FMT_FP8_BLOCK) return WQ_ERR_UNSUPPORTED;
    if (w->fmt != gate->fmt || w->perm != nullptr) return WQ_ERR_UNSUPPORTED;
    if (w->fmt == WQ_FMT_INT4_ASYM && (!aligned(w->scales, 8) || !aligned(w->zeros, 2)))
      return WQ_ERR_ALIGN;
  }
  if (!is16(xdt) || !is_out(ydt)) return WQ_ERR_UNSUPPORTED;
  if (m < 1 || experts < 1 || top_k < 1 || top_k > experts) return WQ_ERR_SHAPE;
  if (m > kMoeMaxTokens || experts > kMoeMaxExperts || top_k > kMoeMaxTopK)
    return WQ_ERR_UNSUPPORTED;
  if (gate->group != up->group || gate->group != down->group) return WQ_ERR_SHAPE;
  const int64_t h = gate->k, i = down->k;
  if (h % 128 != 0 || i % 128 != 0 || gate->n != experts * i || up->n != gate->n || up->k != h ||
      down->n != experts * h)
    return WQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(router, 16) || !aligned(logits, 4) ||
      !aligned(y, dt_bytes(ydt)) || !aligned(ids, 4) || !aligned(probs, 4))
    return WQ_ERR_ALIGN;
  if (workspace == nullptr || ws_bytes < moe_ws_bytes(m, experts, top_k, h, i))
    return WQ_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return WQ_ERR_ALIGN;
  const MoeCall c{static_cast<const uint16_t*>(x), xdt, m, h, experts, i, top_k,
                  renormalize ? 1 : 0, static_cast<const uint16_t*>(router), logits, gate, up,
                  down, y, ydt, ids, probs, workspace};
  return hip_status(launch_moe(c, static_cast<hipStream_t>(stream)));
}

wq_status wq_append_kv(const void* q, const void* k, const void* v, int32_t dt, int64_t m,
                       int64_t heads, int64_t ldq, int64_t ldk, int64_t ldv,
                       const int32_t* positions, const float* cos_sin, int64_t max_pos,
                       int64_t rot, int32_t interleaved, void* q_out, int64_t ldo,
                       const int32_t* slots, const wq_kv_cache* cache, void* stream) {
  if (k == nullptr || v == nullptr || slots == nullptr || (q == nullptr) != (q_out == nullptr))
    return WQ_ERR_NULL;
  const wq_status st = check_cache(cache);
  if (st != WQ_OK) return st;
  if (rot != 0 && (positions == nullptr || cos_sin == nullptr)) return WQ_ERR_NULL;
  if (!is16(dt) || (cache->dt != WQ_E4M3 && cache->dt != dt)) return WQ_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return WQ_ERR_UNSUPPORTED;
  const int64_t d = cache->head_dim;
  if (rot < 0 || rot > d || rot % 16 != 0) return WQ_ERR_SHAPE;
  if (rot != 0 && (max_pos < 1 || max_pos > INT32_MAX || max_pos > kMaxElems / rot))
    return WQ_ERR_SHAPE;
  if (!rows_ok(m, cache->kv_heads * d, ldk) || !rows_ok(m, cache->kv_heads * d, ldv))
    return WQ_ERR_SHAPE;
  if (q != nullptr && (heads < 1 || heads > kMaxHeads || !rows_ok(m, heads * d, ldq) ||
                       !rows_ok(m, heads * d, ldo)))
    return WQ_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(positions, 4) || !aligned(cos_sin, 16) || !aligned(slots, 4))
    return WQ_ERR_ALIGN;
  const AppendCall c{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                     static_cast<const uint16_t*>(v), dt, m, q == nullptr ? 0 : heads, ldq, ldk,
                     ldv, ldo, positions, cos_sin, max_pos, (int)rot, interleaved,
                     static_cast<uint16_t*>(q_out), slots, kernel_cache(cache)};
  return hip_status(launch_append_kv(c, static_cast<hipStream_t>(stream)));
}

size_t wq_attention_decode_workspace(int64_t m, int64_t heads, const wq_kv_cache* cache) {
  if (!attention_sizes_ok(m, heads, cache)) return 0;
  return decode_ws_bytes(m, heads, kernel_cache(cache));
}

size_t wq_attention_prompt_workspace(int64_t m, int64_t heads, int64_t batch,
                                     const wq_kv_cache* cache) {
  if (!attention_sizes_ok(m, heads, cache) || batch < 1 || batch >= kMaxDim) return 0;
  if (prompt_wgs(m, heads, batch, kernel_cache(cache)) > kPromptMaxWgs) return 0;
  return prompt_ws_bytes(m, heads, kernel_cache(cache));
}

wq_status wq_attention_decode(const void* q, int32_t dt, int64_t m, int64_t heads, int64_t ldq,
                              const wq_kv_cache* cache, const int32_t* pages, int64_t max_pages,
                              int64_t ldp, const int32_t* lens, float scale, int64_t window,
                              int64_t sinks, void* y, float* lse, void* workspace,
                              size_t ws_bytes, void* stream) {
  AttentionCall c;
  const wq_status st = check_attention(q, dt, m, heads, ldq, m, cache, pages, max_pages, ldp, lens,
                                       scale, window, sinks, y, lse, &c);
  if (st != WQ_OK) return st;
  c.starts = nullptr;
  return run_attention(&c, workspace, ws_bytes, wq_attention_decode_workspace(m, heads, cache),
                       stream);
}

wq_status wq_attention_prompt(const void* q, int32_t dt, int64_t m, int64_t heads, int64_t ldq,
                              const int32_t* starts, int64_t batch, const wq_kv_cache* cache,
                              const int32_t* pages, int64_t max_pages, int64_t ldp,
                              const int32_t* lens, float scale, int64_t window, int64_t sinks,
                              void* y, float* lse, void* workspace, size_t ws_bytes,
                              void* stream) {
  if (starts == nullptr) return WQ_ERR_NULL;
  AttentionCall c;
  const wq_status st = check_attention(q, dt, m, heads, ldq, batch, cache, pages, max_pages, ldp,
                                       lens, scale, window, sinks, y, lse, &c);
  if (st != WQ_OK) return st;
  if (prompt_wgs(m, heads, batch, c.cache) > kPromptMaxWgs) return WQ_ERR_SHAPE;
  if (!aligned(starts, 4)) return WQ_ERR_ALIGN;
  c.starts = starts;
  return run_attention(&c, workspace, ws_bytes,
                       wq_attention_prompt_workspace(m, heads, batch, cache), stream);
}

wq_status wq_dequantize(const wq_weight* w, void* out, int32_t odt, void* stream) {
  if (out == nullptr) return WQ_ERR_NULL;
  const wq_status st = check_weight(w, false);
  if (st != WQ_OK) return st;
  if (!is16(odt)) return WQ_ERR_UNSUPPORTED;
  if (!aligned(out, 16)) return WQ_ERR_ALIGN;
  const wq_weight kv = kernel_view(w);
  return hip_status(
      launch_dequantize(&kv, levels_for(w), out, odt, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
