// The 8-bit key/value cache: codes [B, Hkv, capacity, D] (int8 or e4m3), one
// fp32 scale per (block of tokens, head); a value is code * scale.
//
// Append.  The block's new tokens have the largest magnitude a; with qmax = 127
// (int8) or 448 (e4m3)
//   s = max(a / qmax, s_old)      s_old: the scale of older tokens of the block
//   code = rne(x * (1 / s))       older codes c -> rne((c * s_old) * (1 / s)) if s > s_old
// in fp32: one IEEE quotient and one reciprocal per block, one product per
// value.  A scale below 2^-126 (its reciprocal would overflow) is stored as 0
// with codes 0.  A NaN or infinity makes its block's scale NaN or infinite
// with codes 0, so every value of the block reads back as NaN; codes
// themselves are always finite.
//
// Bound by bytes (16 bits in, 8 out).  One CTA takes 128 tokens of one
// (batch entry, head) of K or of V (of both at D = 64), each of its warps 16 of them (8 at D = 256),
// which it holds in registers between the maximum and the codes: one read, one
// write.  Every block size (16, 32, 64, 128) is then a whole number of warps.
// 4 sequences of 8192 tokens, bf16, 201 MB in and out: 39.6 us at D = 128 with 8 heads
// (5.1 TB/s), 43.6 us at D = 64 with 16 (4.6), 44.5 us at D = 256 with 4 (4.5).  What
// is missing is the chain of a CTA (start, values, maximum, codes) at the CTAs that
// registers allow; fewer instructions (packed products and sums) changed nothing.
// The addresses of the codes are formed behind the loads of the values: ahead of them
// a token each of 32 sequences took 0.5 us longer, long prompts 0.6 less.
#pragma once

#include "skv_device.cuh"

namespace skv {

constexpr int kKv8Window = 128;   // tokens per append CTA
template <int D>
constexpr int kAppendThreads = D == 256 ? 512 : 256;
// K and V of a CTA: both at D = 64, whose rows leave registers for it (43.6 us against
// 50.0 for 4 sequences of 8192 tokens, 16 heads), one of them above.
template <int D>
constexpr int kAppendSides = D == 64 ? 2 : 1;
constexpr float kKv8TinyScale = 1.17549435e-38f;  // 2^-126

template <bool kE4M3>
struct Kv8Code {
  static constexpr float kMax = kE4M3 ? 448.f : 127.f;
  // codes of four values times inv = 1 / scale (|.| <= kMax up to rounding)
  static __device__ __forceinline__ uint32_t encode4(float2 a, float2 b, uint64_t inv) {
    const uint64_t p = fmul2(f2_pack(a.x, a.y), inv), q = fmul2(f2_pack(b.x, b.y), inv);
    if constexpr (kE4M3) {
      const float2 x = f2_unpack(p), y = f2_unpack(q);
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x.y), "f"(x.x));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y.y), "f"(y.x));
      return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    } else {
      // adding 1.5 * 2^23 rounds to a whole number (ties to even) in the low
      // bits; the low byte is the two's complement code
      // (scalar sums: a packed product and a packed sum were contracted into one
      // rounding, which is another code where a product lies next to a tie)
      const float2 x = f2_unpack(p), y = f2_unpack(q);
      const uint32_t i0 = __float_as_uint(__fadd_rn(x.x, 12582912.f)), i1 = __float_as_uint(__fadd_rn(x.y, 12582912.f));
      const uint32_t i2 = __float_as_uint(__fadd_rn(y.x, 12582912.f)), i3 = __float_as_uint(__fadd_rn(y.y, 12582912.f));
      return __byte_perm(__byte_perm(i0, i1, 0x0040), __byte_perm(i2, i3, 0x0040), 0x5410);
    }
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    if constexpr (kE4M3) {
      uint32_t h0, h1;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w & 0xffff)));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
      const float2 f0 = unpack2<__half>(h0), f1 = unpack2<__half>(h1);
      x[0] = f0.x; x[1] = f0.y; x[2] = f1.x; x[3] = f1.y;
    } else {
      // 0x4b000000 | u is 2^23 + u in fp32, with u = code + 128 (the type
      // conversion instruction runs at an eighth of this rate)
      const uint32_t u = w ^ 0x80808080u;
      x[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.f;
      x[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.f;
      x[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - 8388736.f;
      x[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - 8388736.f;
    }
  }
  // codes of (code * from) / to, given 1 / to
  static __device__ __forceinline__ uint32_t recode4(uint32_t w, float from, uint64_t inv) {
    float x[4];
    decode4(w, x);
    return encode4(make_float2(__fmul_rn(x[0], from), __fmul_rn(x[1], from)),
                   make_float2(__fmul_rn(x[2], from), __fmul_rn(x[3], from)), inv);
  }
};

// 1 / s for a block's codes; 0 where the codes are 0 (s == 0, or not finite)
__device__ __forceinline__ float kv8_inverse(float s) {
  return (s > 0.f && s < INFINITY) ? __frcp_rn(s) : 0.f;
}

struct Kv8AppendArgs {
  const void* x[2];         // new k, v
  uint8_t* codes[2];
  float* scale[2];          // [B, Hkv, capacity / block]
  const int32_t* start;     // [B]
  const int32_t* num_new;   // [B] or null (= S)
  const int32_t* cu;        // [B + 1] (packed rows) or null
  int B, Hkv, S, T, capacity, block;
  int token_major;          // 1: rows ordered (b, s, h); 0: (b, h, s)
};

template <int D, typename T, bool kE4M3>
__global__ void __launch_bounds__(kAppendThreads<D>, D == 256 ? 2 : 4)
    kv8_append_kernel(const Kv8AppendArgs a) {
  using Code = Kv8Code<kE4M3>;
  constexpr int kLanes = D / 8;            // lanes of one row, 8 values each
  constexpr int kRows = 32 / kLanes;       // rows a warp takes at once
  constexpr int kWarps = kAppendThreads<D> / 32;
  constexpr int kTokens = kKv8Window / kWarps;  // of a warp
  constexpr int kPasses = kTokens / kRows;
  constexpr int kSides = kAppendSides<D>;  // K and V, or one of them
  // a programmatic dependent of the kernel before it: waits before any load
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // heads beside each other: in token-major rows they share DRAM pages
  const int b = blockIdx.y, h = blockIdx.x % a.Hkv, side0 = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int start = min(max(a.start[b], 0), a.capacity);
  int count = a.S, first_row = 0;
  if (a.cu != nullptr) {
    first_row = min(max(a.cu[b], 0), a.T);
    count = min(max(a.cu[b + 1], first_row), a.T) - first_row;
    count = min(count, a.S);
  } else if (a.num_new != nullptr) {
    count = min(max(a.num_new[b], 0), a.S);
  }
  const int end = start + min(count, a.capacity - start);
  const int base = (start / kKv8Window + static_cast<int>(blockIdx.x) / a.Hkv) * kKv8Window;
  if (base >= end || start >= end) return;  // the whole CTA: nothing new in this window

  const int cl = lane % kLanes, rl = lane / kLanes;
  const int wpos = base + warp * kTokens;  // this warp's first position
  const int pos0 = wpos + rl;              // this lane's rows: pos0 + kRows * p
  const int per = a.block / kTokens;       // warps of one block
  const int group = warp / per;
  const int block_pos = base + group * a.block;
  const bool touched = block_pos < end && block_pos + a.block > start;
  const bool has_old = touched && block_pos < start;  // older tokens, with a scale of their own
  const bool whole = wpos >= start && wpos + kTokens <= end;  // new rows only
  const uint32_t at = (static_cast<uint32_t>(b) * a.Hkv + h) * (a.capacity / a.block) + block_pos / a.block;
  float s_old[kSides];
#pragma unroll
  for (int d = 0; d < kSides; ++d) s_old[d] = has_old ? a.scale[side0 + d][at] : 0.f;
  // rows of token i: row0 + i * step
  const int64_t step = (a.cu != nullptr || a.token_major) ? a.Hkv : 1;
  const int64_t row0 = a.cu != nullptr ? static_cast<int64_t>(first_row) * a.Hkv + h
                       : a.token_major ? static_cast<int64_t>(b) * a.S * a.Hkv + h
                                       : (static_cast<int64_t>(b) * a.Hkv + h) * a.S;
  const int64_t src0 = (row0 + (pos0 - start) * step) * D + cl * 8, src_pass = step * kRows * D;
  // (a cache has less than 2^31 tokens)
  const uint32_t token = (static_cast<uint32_t>(b) * a.Hkv + h) * a.capacity + pos0;
  auto codes_of = [&](int d) { return a.codes[side0 + d] + static_cast<uint64_t>(token) * D + cl * 8; };
  // a lane's rows: new values, or (first block only) the codes of older tokens
  uint4 v[kSides][kPasses];
#pragma unroll
  for (int d = 0; d < kSides; ++d) {
    const T* src = static_cast<const T*>(a.x[side0 + d]) + src0;
    if (whole) {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) v[d][p] = __ldg(reinterpret_cast<const uint4*>(src + p * src_pass));
    } else {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int pos = pos0 + kRows * p;
        v[d][p] = make_uint4(0, 0, 0, 0);
        if (pos >= start && pos < end) {
          v[d][p] = __ldg(reinterpret_cast<const uint4*>(src + p * src_pass));
        } else if (has_old && pos < start) {
          const uint2 w = *reinterpret_cast<const uint2*>(codes_of(d) + kRows * p * D);
          v[d][p].x = w.x;
          v[d][p].y = w.y;
        }
      }
    }
  }
  __shared__ uint32_t warp_top[kSides][kWarps];
#pragma unroll
  for (int d = 0; d < kSides; ++d) {
    uint32_t top = 0;  // largest magnitude bits of the new values, two 16-bit halves
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      // magnitude bits of 16-bit floats order as whole numbers, NaN above infinity
      const uint32_t t = __vmaxu2(__vmaxu2(v[d][p].x & 0x7fff7fffu, v[d][p].y & 0x7fff7fffu),
                                  __vmaxu2(v[d][p].z & 0x7fff7fffu, v[d][p].w & 0x7fff7fffu));
      if (whole || pos0 + kRows * p >= start) top = __vmaxu2(top, t);
    }
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if (lane == 0) warp_top[d][warp] = top;
  }
  __syncthreads();  // also orders every read of the old scale before its new value is written
  if (!touched) return;
#pragma unroll
  for (int d = 0; d < kSides; ++d) {
    uint32_t top = 0;
    for (int w = group * per; w < (group + 1) * per; ++w) top = max(top, warp_top[d][w]);
    const float amax = unpack2<T>(top).x;
    const float fresh = __fdiv_rn(amax, Code::kMax);
    float s = (fresh > s_old[d] || isnan(fresh)) ? fresh : s_old[d];
    if (s < kKv8TinyScale) s = 0.f;
    const bool poisoned = !(s < INFINITY);
    const float inv = kv8_inverse(s);
    if (warp == group * per && lane == 0) a.scale[side0 + d][at] = s;

    uint8_t* codes = codes_of(d);
    const uint64_t inv2 = f2_pack(inv, inv);
    auto encode = [&](const uint4& x) {
      uint2 w;
      w.x = Code::encode4(unpack2<T>(x.x), unpack2<T>(x.y), inv2);
      w.y = Code::encode4(unpack2<T>(x.z), unpack2<T>(x.w), inv2);
      return w;
    };
    if (whole && !poisoned) {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) *reinterpret_cast<uint2*>(codes + kRows * p * D) = encode(v[d][p]);
      continue;
    }
    const bool wider = s > s_old[d] || (poisoned && s_old[d] < INFINITY);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int pos = pos0 + kRows * p;
      if (pos >= end || (pos < start && !wider)) continue;
      uint2 w = make_uint2(0, 0);
      if (!poisoned)
        w = pos >= start ? encode(v[d][p])
                         : make_uint2(Code::recode4(v[d][p].x, s_old[d], inv2), Code::recode4(v[d][p].y, s_old[d], inv2));
      *reinterpret_cast<uint2*>(codes + kRows * p * D) = w;
    }
  }
}

// Fetch.  A window of the cache in 16 bits: out[b, h, i] = code * scale of
// position start[b] + i, zero where that is not in [0, kv_len[b]).  Bound by
// bytes (8 bits in, 16 out): 4 sequences of 8192 tokens, 201 MB in and out, 34.5 us e4m3
// (5.8 TB/s), 36.1 us int8 (5.6), at every D.
struct Kv8FetchArgs {
  const uint8_t* codes[2];
  const float* scale[2];
  void* out[2];
  const int32_t* start;    // [B] or null (= 0)
  const int32_t* kv_len;   // [B] or null (= capacity)
  int Hkv, capacity, block_shift, n;
  int token_major;         // out [B, n, Hkv, D] instead of [B, Hkv, n, D]
};

constexpr int kFetchUnroll = 8;  // pieces of 8 codes a thread has in flight (each a full 16 bytes out)

template <int D, typename T, bool kE4M3>
__global__ void __launch_bounds__(256) kv8_fetch_kernel(const Kv8FetchArgs a) {
  constexpr int kUnits = D / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int bh = blockIdx.y, which = blockIdx.z;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int64_t start = a.start != nullptr ? a.start[b] : 0;
  const int len = a.kv_len != nullptr ? min(a.kv_len[b], a.capacity) : a.capacity;
  const uint8_t* codes = a.codes[which] + static_cast<int64_t>(bh) * a.capacity * D;
  const float* scale = a.scale[which] + static_cast<int64_t>(bh) * (a.capacity >> a.block_shift);
  T* out = static_cast<T*>(a.out[which]);
  constexpr int kRowsCta = 256 * kFetchUnroll / kUnits;
  const int i0 = blockIdx.x * kRowsCta + threadIdx.x / kUnits, u = threadIdx.x % kUnits;
  uint2 w[kFetchUnroll];
  float s[kFetchUnroll];
#pragma unroll
  for (int j = 0; j < kFetchUnroll; ++j) {
    const int i = i0 + j * (256 / kUnits);
    const int64_t pos = start + i;
    w[j] = make_uint2(0, 0);
    s[j] = 0.f;  // a position without a token: zeros
    if (i < a.n && pos >= 0 && pos < len) {
      w[j] = __ldg(reinterpret_cast<const uint2*>(codes + pos * D) + u);
      s[j] = __ldg(scale + (pos >> a.block_shift));
    }
  }
  const int64_t row0 = a.token_major ? static_cast<int64_t>(b) * a.n * a.Hkv + h : static_cast<int64_t>(bh) * a.n;
  const int64_t step = a.token_major ? a.Hkv : 1;
#pragma unroll
  for (int j = 0; j < kFetchUnroll; ++j) {
    const int i = i0 + j * (256 / kUnits);
    if (i >= a.n) break;
    const uint64_t ss = f2_pack(s[j], s[j]);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x[4];
      Kv8Code<kE4M3>::decode4(e ? w[j].y : w[j].x, x);
      const float2 p = f2_unpack(fmul2(f2_pack(x[0], x[1]), ss)), q = f2_unpack(fmul2(f2_pack(x[2], x[3]), ss));
      o[2 * e] = pack2<T>(p.x, p.y);
      o[2 * e + 1] = pack2<T>(q.x, q.y);
    }
    reinterpret_cast<uint4*>(out + (row0 + i * step) * D)[u] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace skv
