// Rotary positions and the 8-bit key/value cache: validation, planning and
// launches of rope_apply, kv8_append, kv8_fetch, attn_splitkv_decode_kv8 and
// kv8_evict.  A translation unit of its own (with its own device error word).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include "skv_internal.h"
#include "skv_device.cuh"

#include "rope.cuh"
#include "kv8.cuh"
#include "decode_kv8.cuh"
#include "evict.cuh"

namespace skv {

int read_cache_error(int* code) { return cudaMemcpyFromSymbol(code, g_skv_device_error, sizeof(int)); }

int clear_cache_error() {
  const int zero = 0;
  return cudaMemcpyToSymbol(g_skv_device_error, &zero, sizeof(int));
}

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// non-null and aligned
bool good(const void* p, uintptr_t a) { return p != nullptr && aligned(p, a); }

// whether [p, p + np) and [q, q + nq) share a byte
bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p != nullptr && q != nullptr && a < b + nq && b < a + np;
}

struct Span {
  const void* p;
  size_t n;
};
// Whether anything written shares a byte with anything read or with another output.
template <size_t kIn, size_t kOut>
bool clash(const Span (&in)[kIn], const Span (&to)[kOut]) {
  for (size_t i = 0; i < kOut; ++i) {
    for (const Span& x : in)
      if (overlap(to[i].p, to[i].n, x.p, x.n)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(to[i].p, to[i].n, to[j].p, to[j].n)) return true;
  }
  return false;
}

// Launches `kern` as a programmatic dependent of the kernel before it on the
// stream (every kernel here waits for that one before it touches memory), in
// clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, skv_stream_t stream, unsigned cluster,
           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// Sizes and types every call on the cache shares.
skv_status check_cache(const void* k, const void* v, const float* ks, const float* vs, int B, int Hkv, int capacity,
                       int D, int block, skv_code codes) {
  if (!good(k, 16) || !good(v, 16) || !good(ks, 4) || !good(vs, 4)) return SKV_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || capacity < 1 || D < 1) return SKV_ERR_INVALID_ARG;
  if (codes != SKV_INT8 && codes != SKV_E4M3) return SKV_ERR_INVALID_ARG;
  if (block < 1 || capacity % block != 0) return SKV_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return SKV_ERR_UNSUPPORTED;
  if (block != 16 && block != 32 && block != 64 && block != 128) return SKV_ERR_UNSUPPORTED;
  // 32-bit tile coordinates, also of tiles that reach behind the last token
  if (static_cast<int64_t>(B) * Hkv * capacity > (int64_t(1) << 31) - 4096 || capacity > (1 << 30))
    return SKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * Hkv > 65535) return SKV_ERR_UNSUPPORTED;  // grid.y
  return SKV_OK;
}

skv_status check_half(skv_dtype dt) {
  if (dt != SKV_BF16 && dt != SKV_FP16 && dt != SKV_FP32) return SKV_ERR_INVALID_ARG;
  return dt == SKV_FP32 ? SKV_ERR_UNSUPPORTED : SKV_OK;
}

int log2_of(int block) { return block == 16 ? 4 : (block == 32 ? 5 : (block == 64 ? 6 : 7)); }

template <int D, typename T>
int launch_append(const Kv8AppendArgs& a, skv_code codes, dim3 grid, skv_stream_t st) {
  return codes == SKV_E4M3 ? launch(kv8_append_kernel<D, T, true>, grid, kAppendThreads<D>, 0, st, 1, a)
                           : launch(kv8_append_kernel<D, T, false>, grid, kAppendThreads<D>, 0, st, 1, a);
}

template <typename T>
int launch_append_d(const Kv8AppendArgs& a, int D, skv_code codes, dim3 grid, skv_stream_t st) {
  if (D == 64) return launch_append<64, T>(a, codes, grid, st);
  if (D == 128) return launch_append<128, T>(a, codes, grid, st);
  return launch_append<256, T>(a, codes, grid, st);
}

template <int D, typename T>
int launch_fetch(const Kv8FetchArgs& a, int B, skv_code codes, skv_stream_t st) {
  const dim3 grid(static_cast<unsigned>(ceil_div64(a.n, 256 * kFetchUnroll / (D / 8))),
                  static_cast<unsigned>(B * a.Hkv), 2);
  return codes == SKV_E4M3 ? launch(kv8_fetch_kernel<D, T, true>, grid, 256, 0, st, 1, a)
                           : launch(kv8_fetch_kernel<D, T, false>, grid, 256, 0, st, 1, a);
}

template <typename T>
int launch_fetch_d(const Kv8FetchArgs& a, int B, int D, skv_code codes, skv_stream_t st) {
  if (D == 64) return launch_fetch<64, T>(a, B, codes, st);
  if (D == 128) return launch_fetch<128, T>(a, B, codes, st);
  return launch_fetch<256, T>(a, B, codes, st);
}

template <int D>
int launch_move(const EvictArgs& a, dim3 grid, skv_code codes, skv_stream_t st) {
  return codes == SKV_E4M3 ? launch(evict_move_kernel<D, true>, grid, 256, 0, st, 1, a)
                           : launch(evict_move_kernel<D, false>, grid, 256, 0, st, 1, a);
}

// ---- tile maps: the codes as rows of 128 (D = 64: two tokens; D = 128: one)
// or 256 bytes, boxes 128 bytes wide, 128-byte swizzle
int encode_codes(CUtensorMap* m, const void* base, int64_t tokens, int D) {
  static std::mutex mu;
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (encode == nullptr) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
      if (e != cudaSuccess) return e;
      if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
  }
  const cuuint64_t width = D == 256 ? 256 : 128;
  const cuuint64_t dims[2] = {width, static_cast<cuuint64_t>(tokens) * D / width};
  const cuuint64_t strides[1] = {width};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(D == 64    ? Kv8DecodeCfg<64>::kBoxRows
                                                          : D == 128 ? Kv8DecodeCfg<128>::kBoxRows
                                                                     : Kv8DecodeCfg<256>::kBoxRows)};
  const cuuint32_t one[2] = {1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : static_cast<int>(cudaErrorInvalidValue);
}

template <int D, typename T, bool kE4M3, bool kLogits, int kHalves>
int launch_decode_kv8(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8DecodeArgs& a, dim3 grid,
                      skv_stream_t st) {
  using Cfg = Kv8DecodeCfg<D>;
  auto kern = decode_kv8_kernel<D, T, kE4M3, kLogits, kHalves>;
  static std::atomic<uint64_t> ready{0};  // devices (below 64) the limit is set on
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (ready.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch(kern, grid, kKv8Threads, Cfg::kSmemBytes, st, 1, tk, tv, a);
}

template <int D, typename T, int kHalves>
int launch_decode_kv8_h(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8DecodeArgs& a, skv_code codes,
                        dim3 grid, skv_stream_t st) {
  if (codes == SKV_E4M3)
    return a.logits ? launch_decode_kv8<D, T, true, true, kHalves>(tk, tv, a, grid, st)
                    : launch_decode_kv8<D, T, true, false, kHalves>(tk, tv, a, grid, st);
  return a.logits ? launch_decode_kv8<D, T, false, true, kHalves>(tk, tv, a, grid, st)
                  : launch_decode_kv8<D, T, false, false, kHalves>(tk, tv, a, grid, st);
}

template <int D, typename T>
int launch_decode_kv8_d(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8DecodeArgs& a, skv_code codes,
                        dim3 grid, skv_stream_t st) {
  return a.Hq / a.Hkv * a.Lq <= kKv8Rows / 2 ? launch_decode_kv8_h<D, T, 1>(tk, tv, a, codes, grid, st)
                                             : launch_decode_kv8_h<D, T, 2>(tk, tv, a, codes, grid, st);
}

// keys of a tile of the division among CTAs
int kv8_cta_keys(int D) {
  return D == 64 ? Kv8DecodeCfg<64>::kCtaKeys : (D == 128 ? Kv8DecodeCfg<128>::kCtaKeys : Kv8DecodeCfg<256>::kCtaKeys);
}

int64_t kv8_units(int B, int Hq, int Hkv, int Lq) {
  return static_cast<int64_t>(B) * Hkv * ceil_div64(static_cast<int64_t>(Hq / Hkv) * Lq, kKv8Rows);
}

// [B + 1] table | [slots, 16] LSE | [slots, 16, D] O where a unit can be
// divided (slots: units + CTAs), then with weights [rows] LSE | [rows, capacity] logits
struct Kv8Ws {
  size_t table = 0, part_lse = 0, part_o = 0, lse = 0, logits = 0, total = 0;
  bool divided = false;
};
Kv8Ws kv8_ws_layout(int B, int Hq, int Hkv, int Lq, int capacity, int D, int ctas, int weights) {
  Kv8Ws w;
  auto take = [&](size_t bytes) {
    const size_t at = w.total;
    w.total += align256(bytes);
    return at;
  };
  w.divided = ctas > 1 && capacity > kv8_cta_keys(D);
  if (w.divided) {
    const size_t slots = static_cast<size_t>(kv8_units(B, Hq, Hkv, Lq)) + ctas;
    w.table = take((static_cast<size_t>(B) + 1) * 4);
    w.part_lse = take(slots * kKv8Rows * 4);
    w.part_o = take(slots * kKv8Rows * D * 4);
  }
  if (weights) {
    const size_t rows = static_cast<size_t>(B) * Hq * Lq;
    w.lse = take(rows * 4);
    w.logits = take(rows * static_cast<size_t>(capacity) * 4);
  }
  return w;
}

template <typename T>
int launch_kv8_merge(const Kv8DecodeArgs& a, int D, int ctas, unsigned rows, skv_stream_t st) {
  if (D == 64) return launch(kv8_merge_kernel<64, T>, dim3(rows, D / 64), 256, 0, st, 1, a, ctas);
  if (D == 128) return launch(kv8_merge_kernel<128, T>, dim3(rows, D / 64), 256, 0, st, 1, a, ctas);
  return launch(kv8_merge_kernel<256, T>, dim3(rows, D / 64), 256, 0, st, 1, a, ctas);
}

}  // namespace
}  // namespace skv

using namespace skv;

extern "C" {

// ------------------------------------------------------------------ rope

skv_status rope_inv_freq(int rotary_dim, double base, skv_rope_scaling scaling, double factor, int original_len,
                         double beta_fast, double beta_slow, double* inv_freq, double* attn_factor) {
  if (inv_freq == nullptr || attn_factor == nullptr) return SKV_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim % 2 != 0) return SKV_ERR_INVALID_ARG;
  if (!(std::isfinite(base) && base > 1.0)) return SKV_ERR_INVALID_ARG;
  if (scaling < SKV_ROPE_NONE || scaling > SKV_ROPE_YARN) return SKV_ERR_INVALID_ARG;
  if (scaling != SKV_ROPE_NONE && !(std::isfinite(factor) && factor >= 1.0)) return SKV_ERR_INVALID_ARG;
  if (scaling == SKV_ROPE_NTK && rotary_dim < 4) return SKV_ERR_INVALID_ARG;
  if (scaling == SKV_ROPE_YARN && !(original_len > 0 && std::isfinite(beta_fast) && std::isfinite(beta_slow) &&
                                    beta_slow > 0.0 && beta_fast >= beta_slow))
    return SKV_ERR_INVALID_ARG;
  const int half = rotary_dim / 2;
  if (scaling == SKV_ROPE_NTK) base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  double lo = 0.0, hi = 0.0;
  if (scaling == SKV_ROPE_YARN) {
    // the pair that turns `turns` times over the original length
    auto pair_of = [&](double turns) {
      return rotary_dim * std::log(original_len / (turns * 2.0 * 3.141592653589793)) / (2.0 * std::log(base));
    };
    lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
    // (may lie behind the last pair: all of them then turn more than beta_slow times)
    hi = std::min(std::ceil(pair_of(beta_slow)), rotary_dim - 1.0);
  }
  for (int i = 0; i < half; ++i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == SKV_ROPE_LINEAR) f /= factor;
    if (scaling == SKV_ROPE_YARN) {
      const double g = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1.0 - g) + f / factor * g;
    }
    inv_freq[i] = f;
  }
  *attn_factor = scaling == SKV_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return SKV_OK;
}

skv_status rope_apply(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                      const double* inv_freq, int B, int Hq, int Hkv, int S, int D, int rotary_dim, float factor,
                      skv_dtype dtype, skv_layout layout, int interleaved, int inverse, skv_stream_t stream) {
  if (!good(q, 16) || !good(q_out, 16) || !good(positions, 4) || !good(inv_freq, 8)) return SKV_ERR_INVALID_ARG;
  if ((k == nullptr) != (k_out == nullptr) || !aligned(k, 16) || !aligned(k_out, 16)) return SKV_ERR_INVALID_ARG;
  if (layout != SKV_HND && layout != SKV_NHD && layout != SKV_TND) return SKV_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || S < 0 || D < 1 || (k != nullptr ? Hkv < 1 : Hkv != 0)) return SKV_ERR_INVALID_ARG;
  if (layout == SKV_TND && B != 1) return SKV_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > D) return SKV_ERR_INVALID_ARG;
  if (!std::isfinite(factor)) return SKV_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return SKV_ERR_INVALID_ARG;
  if (skv_status s = check_half(dtype)) return s;
  // a CTA's table holds a token's pairs, and its threads a head's units
  if (D % 16 != 0 || rotary_dim % 16 != 0 || rotary_dim * 4 > kRopeTableBytes || D > 16 * kRopeMaxThreads)
    return SKV_ERR_UNSUPPORTED;
  const size_t row = static_cast<size_t>(B) * S * D * 2;
  const size_t nq = row * Hq, nk = row * Hkv;
  // in place is fine, any other overlap is not
  if ((q_out != q && overlap(q_out, nq, q, nq)) || (k != nullptr && k_out != k && overlap(k_out, nk, k, nk)) ||
      overlap(q_out, nq, k, nk) || overlap(q, nq, k_out, nk) || overlap(q_out, nq, k_out, nk))
    return SKV_ERR_INVALID_ARG;
  // every CTA reads positions and frequencies while others already write
  const Span angles[] = {{positions, static_cast<size_t>(B) * S * 4}, {inv_freq, static_cast<size_t>(rotary_dim) * 4}};
  for (const Span& x : angles)
    if (overlap(q_out, nq, x.p, x.n) || overlap(k_out, nk, x.p, x.n)) return SKV_ERR_INVALID_ARG;
  if (S == 0) return SKV_OK;
  RopeArgs a;
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = q_out;
  a.y[1] = k_out;
  a.heads[0] = Hq;
  a.heads[1] = k != nullptr ? Hkv : 0;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.factor = factor;
  a.inverse = inverse;
  a.S = S;
  a.D = D;
  a.R = rotary_dim;
  a.token_major = layout != SKV_HND;
  const int sms = sm_count();
  if (sms <= 0) return cuda_status(cudaErrorNoDevice);
  const int64_t tokens = static_cast<int64_t>(B) * S;
  if (tokens > (1 << 30)) return SKV_ERR_UNSUPPORTED;
  const int64_t heads = static_cast<int64_t>(a.heads[0]) + a.heads[1];
  // all tokens of a CTA at once where that still gives every SM two CTAs and their
  // table fits, else one; the heads in equal groups of at most 512 threads, or one
  // group more where long calls then fill an SM better by an eighth (48 heads of 128, 7001
  // tokens: 5 CTAs of 192 threads 29.5 us, 2 of 384 31.6; 40 heads: 3 of 320 either way)
  a.tokens = static_cast<int>(tokens);
  a.per_cta = tokens >= static_cast<int64_t>(sms) * 2 * kRopeTokens && rotary_dim * 4 * kRopeTokens <= kRopeTableBytes
                  ? kRopeTokens : 1;
  const int units = D / 16;
  const int64_t gx = ceil_div64(tokens, a.per_cta);
  // heads of a CTA, and its threads, with the heads in n groups
  auto group_of = [&](int64_t n) {
    int64_t g = ceil_div64(heads, n);
    while (g > 1 && g * units > kRopeMaxThreads) --g;
    return static_cast<int>(g);
  };
  // threads of an SM (1024 at 64 registers) with groups of g heads
  auto resident = [&](int g) {
    const int64_t t = ceil_div64(static_cast<int64_t>(g) * units, 32) * 32;
    return 1024 / t * t;
  };
  const int64_t gy = ceil_div64(heads * units, kRopeMaxThreads);
  a.group = group_of(gy);
  if (a.per_cta > 1 && resident(group_of(gy + 1)) * 8 > resident(a.group) * 9) a.group = group_of(gy + 1);
  const int threads = static_cast<int>(ceil_div64(static_cast<int64_t>(a.group) * units, 32) * 32);
  const int64_t groups = ceil_div64(heads, a.group);
  if (groups > 65535) return SKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(groups));
  int e;
  if (dtype == SKV_BF16)
    e = interleaved ? launch(rope_kernel<__nv_bfloat16, true>, grid, threads, 0, stream, 1, a)
                    : launch(rope_kernel<__nv_bfloat16, false>, grid, threads, 0, stream, 1, a);
  else
    e = interleaved ? launch(rope_kernel<__half, true>, grid, threads, 0, stream, 1, a)
                    : launch(rope_kernel<__half, false>, grid, threads, 0, stream, 1, a);
  return cuda_status(e);
}

// ------------------------------------------------------------------ the cache

skv_status kv8_append(const void* k_new, const void* v_new, void* k_codes, void* v_codes, float* k_scale,
                      float* v_scale, const int32_t* start, const int32_t* num_new, const int32_t* cu_seqlens, int B,
                      int Hkv, int S, int T, int capacity, int D, int block, skv_dtype dtype, skv_code codes,
                      skv_layout layout, skv_stream_t stream) {
  if (layout != SKV_HND && layout != SKV_NHD && layout != SKV_TND) return SKV_ERR_INVALID_ARG;
  if (!good(k_new, 16) || !good(v_new, 16) || !good(start, 4) || !aligned(num_new, 4) || !aligned(cu_seqlens, 4))
    return SKV_ERR_INVALID_ARG;
  if (S < 0) return SKV_ERR_INVALID_ARG;
  if (layout == SKV_TND ? (cu_seqlens == nullptr || num_new != nullptr || T < 0 || S > T) : cu_seqlens != nullptr)
    return SKV_ERR_INVALID_ARG;
  if (skv_status s = check_cache(k_codes, v_codes, k_scale, v_scale, B, Hkv, capacity, D, block, codes)) return s;
  if (skv_status s = check_half(dtype)) return s;
  const size_t heads = static_cast<size_t>(B) * Hkv, nb = static_cast<size_t>(B) * 4;
  const size_t fresh = (layout == SKV_TND ? static_cast<size_t>(T) * Hkv : heads * S) * D * 2;
  const Span in[] = {{k_new, fresh}, {v_new, fresh}, {start, nb}, {num_new, nb}, {cu_seqlens, nb + 4}};
  const Span to[] = {{k_codes, heads * capacity * D}, {v_codes, heads * capacity * D},
                     {k_scale, heads * (capacity / block) * 4}, {v_scale, heads * (capacity / block) * 4}};
  if (clash(in, to)) return SKV_ERR_INVALID_ARG;
  if (S == 0) return SKV_OK;
  Kv8AppendArgs a;
  a.x[0] = k_new;
  a.x[1] = v_new;
  a.codes[0] = static_cast<uint8_t*>(k_codes);
  a.codes[1] = static_cast<uint8_t*>(v_codes);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.start = start;
  a.num_new = num_new;
  a.cu = cu_seqlens;
  a.B = B;
  a.Hkv = Hkv;
  a.S = S;
  a.T = T;
  a.capacity = capacity;
  a.block = block;
  a.token_major = layout != SKV_HND;
  // windows that S tokens touch at most, wherever they start
  const int64_t windows = std::min<int64_t>((static_cast<int64_t>(S) + kKv8Window - 2) / kKv8Window + 1,
                                            ceil_div64(capacity, kKv8Window));
  if (windows * Hkv > 0x7fffffff) return SKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(windows * Hkv), static_cast<unsigned>(B), D == 64 ? 2 / kAppendSides<64> : 2);
  return cuda_status(dtype == SKV_BF16 ? launch_append_d<__nv_bfloat16>(a, D, codes, grid, stream)
                                       : launch_append_d<__half>(a, D, codes, grid, stream));
}

skv_status kv8_fetch(const void* k_codes, const void* v_codes, const float* k_scale, const float* v_scale, void* k_out,
                     void* v_out, const int32_t* start, const int32_t* kv_len, int B, int Hkv, int n, int capacity,
                     int D, int block, skv_dtype dtype, skv_code codes, skv_layout layout, skv_stream_t stream) {
  if (layout != SKV_HND && layout != SKV_NHD) return SKV_ERR_INVALID_ARG;
  if (!good(k_out, 16) || !good(v_out, 16) || !aligned(start, 4) || !aligned(kv_len, 4) || n < 0)
    return SKV_ERR_INVALID_ARG;
  if (skv_status s = check_cache(k_codes, v_codes, k_scale, v_scale, B, Hkv, capacity, D, block, codes)) return s;
  if (skv_status s = check_half(dtype)) return s;
  const size_t heads = static_cast<size_t>(B) * Hkv, nb = static_cast<size_t>(B) * 4, window = heads * n * D * 2;
  const Span in[] = {{k_codes, heads * capacity * D}, {v_codes, heads * capacity * D},
                     {k_scale, heads * (capacity / block) * 4}, {v_scale, heads * (capacity / block) * 4},
                     {start, nb}, {kv_len, nb}};
  const Span to[] = {{k_out, window}, {v_out, window}};
  if (clash(in, to)) return SKV_ERR_INVALID_ARG;
  if (n == 0) return SKV_OK;
  Kv8FetchArgs a;
  a.codes[0] = static_cast<const uint8_t*>(k_codes);
  a.codes[1] = static_cast<const uint8_t*>(v_codes);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.start = start;
  a.kv_len = kv_len;
  a.Hkv = Hkv;
  a.capacity = capacity;
  a.block_shift = log2_of(block);
  a.n = n;
  a.token_major = layout == SKV_NHD;
  return cuda_status(dtype == SKV_BF16 ? launch_fetch_d<__nv_bfloat16>(a, B, D, codes, stream)
                                       : launch_fetch_d<__half>(a, B, D, codes, stream));
}

// ------------------------------------------------------------------ decode

skv_status attn_splitkv_kv8_plan(int B, int Hq, int Hkv, int Lq, int capacity, int D, int num_sms,
                                 int requested_ctas, int* num_ctas) {
  if (num_ctas == nullptr || B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || capacity < 1 || D < 1 || Hq % Hkv != 0)
    return SKV_ERR_INVALID_ARG;
  if (requested_ctas < 0 || requested_ctas > kKv8MaxCtas) return SKV_ERR_INVALID_ARG;
  if (requested_ctas == 0 && num_sms < 1) return SKV_ERR_INVALID_ARG;
  const int64_t places = kv8_units(B, Hq, Hkv, Lq) * (ceil_div64(capacity, kv8_cta_keys(D)) + 1);
  const int64_t most = requested_ctas > 0 ? requested_ctas : std::min(2 * num_sms, kKv8MaxCtas);
  *num_ctas = static_cast<int>(std::min(most, places));
  return SKV_OK;
}

size_t attn_splitkv_kv8_workspace(int B, int Hq, int Hkv, int Lq, int capacity, int D, int num_ctas, int weights) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Lq < 1 || capacity < 1 || D < 1 || num_ctas < 1) return 0;
  return kv8_ws_layout(B, Hq, Hkv, Lq, capacity, D, num_ctas, weights).total;
}

skv_status attn_splitkv_decode_kv8(const void* q, const void* k_codes, const void* v_codes, const float* k_scale,
                                   const float* v_scale, void* out, float* lse, float* weights, int B, int Hq, int Hkv,
                                   int Lq, int capacity, int D, int block, float scale, skv_dtype dtype,
                                   skv_code codes, const int32_t* kv_len, int causal, int num_ctas, void* workspace,
                                   size_t workspace_bytes, skv_stream_t stream) {
  if (!good(q, 16) || !good(out, 16) || !aligned(lse, 4) || !aligned(weights, 16) || !aligned(kv_len, 4))
    return SKV_ERR_INVALID_ARG;
  if (Hq < 1 || Lq < 1 || Hkv < 1 || Hq % Hkv != 0) return SKV_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return SKV_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return SKV_ERR_INVALID_ARG;
  if (num_ctas < 0 || num_ctas > kKv8MaxCtas) return SKV_ERR_INVALID_ARG;
  if (skv_status s = check_cache(k_codes, v_codes, k_scale, v_scale, B, Hkv, capacity, D, block, codes)) return s;
  if (skv_status s = check_half(dtype)) return s;
  const int64_t group_rows = static_cast<int64_t>(Hq / Hkv) * Lq;
  const int64_t row_groups = ceil_div64(group_rows, kKv8Rows);
  const int64_t rows = static_cast<int64_t>(B) * Hq * Lq;
  // places of the division fit 32 bits
  if (rows > (1 << 30) || kv8_units(B, Hq, Hkv, Lq) * (ceil_div64(capacity, kv8_cta_keys(D)) + 1) > 0x7fffffff)
    return SKV_ERR_UNSUPPORTED;
  const int sms = num_ctas == 0 ? sm_count() : 1;
  if (sms <= 0) return cuda_status(cudaErrorNoDevice);
  int ctas = 0;
  if (skv_status s = attn_splitkv_kv8_plan(B, Hq, Hkv, Lq, capacity, D, sms, num_ctas, &ctas)) return s;
  const Kv8Ws w = kv8_ws_layout(B, Hq, Hkv, Lq, capacity, D, ctas, weights != nullptr);
  if (workspace_bytes < w.total) return SKV_ERR_WORKSPACE_TOO_SMALL;
  if (w.total > 0 && !good(workspace, 256)) return SKV_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(B) * Hkv;
  const Span in[] = {{q, static_cast<size_t>(rows) * D * 2}, {k_codes, heads * capacity * D},
                     {v_codes, heads * capacity * D}, {k_scale, heads * (capacity / block) * 4},
                     {v_scale, heads * (capacity / block) * 4}, {kv_len, static_cast<size_t>(B) * 4}};
  const Span to[] = {{out, static_cast<size_t>(rows) * D * 2}, {lse, static_cast<size_t>(rows) * 4},
                     {weights, heads * capacity * 4}, {workspace, w.total}};
  if (clash(in, to)) return SKV_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* merged = lse;  // the LSE the weights are taken against
  if (weights != nullptr && lse == nullptr) merged = reinterpret_cast<float*>(ws + w.lse);

  CUtensorMap tk, tv;
  const int64_t tokens = static_cast<int64_t>(B) * Hkv * capacity;
  int e = encode_codes(&tk, k_codes, tokens, D);
  if (e) return cuda_status(e);
  e = encode_codes(&tv, v_codes, tokens, D);
  if (e) return cuda_status(e);
  Kv8DecodeArgs a;
  a.q = q;
  a.out = out;
  a.lse = merged;
  a.table = w.divided && kv_len != nullptr ? reinterpret_cast<uint32_t*>(ws + w.table) : nullptr;
  a.part_o = w.divided ? reinterpret_cast<float*>(ws + w.part_o) : nullptr;
  a.part_lse = w.divided ? reinterpret_cast<float*>(ws + w.part_lse) : nullptr;
  a.logits = weights != nullptr ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.kv_len = kv_len;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.Lq = Lq;
  a.capacity = capacity;
  a.block_shift = log2_of(block);
  a.row_groups = static_cast<int>(row_groups);
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  const dim3 grid(static_cast<unsigned>(ctas));
  if (dtype == SKV_BF16) {
    if (D == 64) e = launch_decode_kv8_d<64, __nv_bfloat16>(tk, tv, a, codes, grid, stream);
    else if (D == 128) e = launch_decode_kv8_d<128, __nv_bfloat16>(tk, tv, a, codes, grid, stream);
    else e = launch_decode_kv8_d<256, __nv_bfloat16>(tk, tv, a, codes, grid, stream);
  } else {
    if (D == 64) e = launch_decode_kv8_d<64, __half>(tk, tv, a, codes, grid, stream);
    else if (D == 128) e = launch_decode_kv8_d<128, __half>(tk, tv, a, codes, grid, stream);
    else e = launch_decode_kv8_d<256, __half>(tk, tv, a, codes, grid, stream);
  }
  if (e) return cuda_status(e);
  if (w.divided) {
    e = dtype == SKV_BF16 ? launch_kv8_merge<__nv_bfloat16>(a, D, ctas, static_cast<unsigned>(rows), stream)
                          : launch_kv8_merge<__half>(a, D, ctas, static_cast<unsigned>(rows), stream);
    if (e) return cuda_status(e);
  }
  if (weights != nullptr) {
    Kv8WeightArgs wa;
    wa.logits = a.logits;
    wa.lse = merged;
    wa.weights = weights;
    wa.kv_len = kv_len;
    wa.Hkv = Hkv;
    wa.rows = static_cast<int>(group_rows);
    wa.capacity = capacity;
    const dim3 wgrid(static_cast<unsigned>(ceil_div64(capacity, 4 * kWeightThreads)), static_cast<unsigned>(B * Hkv));
    e = group_rows <= 2 ? launch(kv8_weights_kernel<2>, wgrid, kWeightThreads, 0, stream, 1, wa)
                        : launch(kv8_weights_kernel<8>, wgrid, kWeightThreads, 0, stream, 1, wa);
  }
  return cuda_status(e);
}

// ------------------------------------------------------------------ eviction

skv_status kv8_evict(const void* k_codes, const void* v_codes, const float* k_scale, const float* v_scale,
                     const float* weights, const int32_t* kv_len, void* to_k_codes, void* to_v_codes,
                     float* to_k_scale, float* to_v_scale, float* to_weights, int32_t* kept, int32_t* new_len, int B,
                     int Hkv, int capacity, int to_capacity, int D, int block, skv_code codes, int budget, int sink,
                     int recent, skv_stream_t stream) {
  if (!good(weights, 4) || !good(to_weights, 4) || !good(kept, 4) || !good(new_len, 4) || !aligned(kv_len, 4))
    return SKV_ERR_INVALID_ARG;
  if (budget < 1 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget) return SKV_ERR_INVALID_ARG;
  if (skv_status s = check_cache(k_codes, v_codes, k_scale, v_scale, B, Hkv, capacity, D, block, codes)) return s;
  if (skv_status s = check_cache(to_k_codes, to_v_codes, to_k_scale, to_v_scale, B, Hkv, to_capacity, D, block, codes))
    return s;
  if (budget > to_capacity) return SKV_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(B) * Hkv;
  const Span in[] = {{k_codes, heads * capacity * D}, {v_codes, heads * capacity * D},
                     {k_scale, heads * (capacity / block) * 4}, {v_scale, heads * (capacity / block) * 4},
                     {weights, heads * capacity * 4}, {kv_len, static_cast<size_t>(B) * 4}};
  const Span to[] = {{to_k_codes, heads * to_capacity * D}, {to_v_codes, heads * to_capacity * D},
                     {to_k_scale, heads * (to_capacity / block) * 4}, {to_v_scale, heads * (to_capacity / block) * 4},
                     {to_weights, heads * to_capacity * 4}, {kept, heads * budget * 4},
                     {new_len, static_cast<size_t>(B) * 4}};
  if (clash(in, to)) return SKV_ERR_INVALID_ARG;
  EvictArgs a;
  a.weights = weights;
  a.kv_len = kv_len;
  a.kept = kept;
  a.new_len = new_len;
  a.codes[0] = static_cast<const uint8_t*>(k_codes);
  a.codes[1] = static_cast<const uint8_t*>(v_codes);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.to_codes[0] = static_cast<uint8_t*>(to_k_codes);
  a.to_codes[1] = static_cast<uint8_t*>(to_v_codes);
  a.to_scale[0] = to_k_scale;
  a.to_scale[1] = to_v_scale;
  a.to_weights = to_weights;
  a.B = B;
  a.Hkv = Hkv;
  a.capacity = capacity;
  a.to_capacity = to_capacity;
  a.block_shift = log2_of(block);
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  // as many tokens a CTA as keep a warp's keys in registers: 4096 (fewer only add
  // rounds through the cluster: 8 heads of 4096 took 9.8 us, 12.1 with 2048 a CTA), or
  // 8192 where CTAs of 4096 would not be resident at once; at most 8 CTAs a cluster
  const int sms = sm_count();
  if (sms <= 0) return cuda_status(cudaErrorNoDevice);
  const int64_t bh = static_cast<int64_t>(B) * Hkv;
  const int64_t each = bh * std::min<int64_t>(8, ceil_div64(capacity, 4096)) > 2 * sms ? 8192 : 4096;
  unsigned cluster = 1;
  while (cluster < 8 && cluster * each < capacity) cluster *= 2;
  const dim3 sgrid(cluster, static_cast<unsigned>(bh));
  int e = ceil_div64(capacity, cluster) > 4096 ? launch(evict_select_kernel<16>, sgrid, kEvictThreads, 0, stream, cluster, a)
                                               : launch(evict_select_kernel<8>, sgrid, kEvictThreads, 0, stream, cluster, a);
  if (e) return cuda_status(e);
  const int64_t most = std::min(budget, capacity);
  const dim3 grid(static_cast<unsigned>(ceil_div64(most, kKv8Window)), static_cast<unsigned>(B * Hkv));
  e = D == 64 ? launch_move<64>(a, grid, codes, stream)
              : (D == 128 ? launch_move<128>(a, grid, codes, stream) : launch_move<256>(a, grid, codes, stream));
  return cuda_status(e);
}

}  // extern "C"
