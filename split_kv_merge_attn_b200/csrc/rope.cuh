// Rotary positions applied to q and k in one launch, or their transpose (the
// gradient).
//
// Pair i (i < R/2) of every head row at position p turns by t = p * f_i:
//   (x, y) -> factor * (x cos t - y sin t, x sin t + y cos t),
// with t -> -t for the transpose.  Pairs are (i, i + R/2) ("half") or
// (2i, 2i + 1) ("interleaved"); dimensions >= R are copied.
//
// The angle: a position near 2^20 times a frequency near 1, rounded to fp32,
// is off by up to 0.03 rad, so t / (2 pi) is formed in fp64 and its whole turns
// are dropped there; the remaining half turn at most goes to sincospif in fp32
// (off by 2^-25 turns).  The values turn in fp32 and are rounded once.
//
// Bound by bytes: each value is read and written once.  A thread has one unit of
// 8 pairs, two 16-byte pieces half a rotary dimension apart (in either layout of
// pairs: neighbouring threads then fill whole sectors), of one head, and takes it
// through the CTA's tokens; the CTA's sines and cosines are computed once, into
// shared memory, while the values are on their way.  8192 tokens, 32 + 8 heads, D =
// 128, bf16: 29.5 us, 5.7 TB/s (a copy reaches 6.6); 8 tokens: 1.7 us, a launch.
#pragma once

#include "skv_device.cuh"

namespace skv {

constexpr int kRopeMaxThreads = 512;
constexpr int kRopeTokens = 4;         // of a CTA at most, all in flight at once
constexpr int kRopeTableBytes = 16384;

struct RopeArgs {
  const void* x[2];   // q, k
  void* y[2];
  int heads[2];       // Hq, Hkv (0: no k)
  const int32_t* pos;
  const double* inv_freq;
  float factor;
  int inverse;
  int tokens;         // B * S
  int S, D, R;
  int token_major;    // 1: [B, S, H, D] (NHD, TND); 0: [B, H, S, D]
  int per_cta;        // tokens of a CTA: 1 or kRopeTokens
  int group;          // heads of a CTA
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeMaxThreads, 2) rope_kernel(const RopeArgs a) {
  __shared__ float4 table4[kRopeTableBytes / 16];  // (cos, sin) of [token][pair]
  float2* table = reinterpret_cast<float2*>(table4);
  const int half = a.R >> 1, units = a.D >> 4;
  const int t0 = blockIdx.x * a.per_cta;
  const int nt = min(a.per_cta, a.tokens - t0);
  const int hh = threadIdx.x / units, u = threadIdx.x - hh * units;
  const int head = blockIdx.y * a.group + hh;  // q's heads, then k's
  const int which = head >= a.heads[0] ? 1 : 0;
  const int h = head - (which ? a.heads[0] : 0), H = a.heads[which];
  const int turning = a.R >> 4;                // units of pairs; the others are copied
  const bool turns = u < turning;
  const int gap = turns ? half : (a.D - a.R) >> 1;
  const T* src = static_cast<const T*>(a.x[which]);
  T* dst = static_cast<T*>(a.y[which]);
  const bool mine = hh < a.group && head < a.heads[0] + a.heads[1] && (turns || src != dst);

  // element offset of the unit in each token
  int64_t at[kRopeTokens];
  const int d = turns ? u * 8 : a.R + (u - turning) * 8;
  if (a.token_major) {
#pragma unroll
    for (int i = 0; i < kRopeTokens; ++i) at[i] = (static_cast<int64_t>(t0 + i) * H + h) * a.D + d;
  } else {
    int b = t0 / a.S, s = t0 - b * a.S;
#pragma unroll
    for (int i = 0; i < kRopeTokens; ++i) {
      at[i] = ((static_cast<int64_t>(b) * H + h) * a.S + s) * a.D + d;
      if (++s == a.S) {
        s = 0;
        ++b;
      }
    }
  }
  // a programmatic dependent of the kernel before it: waits before any load
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint4 v[kRopeTokens][2];
#pragma unroll
  for (int i = 0; i < kRopeTokens; ++i) {
    if (mine && i < nt) {
      v[i][0] = *reinterpret_cast<const uint4*>(src + at[i]);
      v[i][1] = *reinterpret_cast<const uint4*>(src + at[i] + gap);
    }
  }
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    // entry i is the one of (token, quarter e, unit, lower or upper pair of the
    // quarter): a quarter's entries lie side by side for neighbouring units
    const int tt = i / half, j = i - tt * half;
    const int e = j / (2 * turning), in = j - e * 2 * turning, unit = in >> 1, up = in & 1;
    const int pair = kInterleaved ? (e >> 1) * (half >> 1) + unit * 4 + (e & 1) * 2 + up : unit * 8 + e * 2 + up;
    const double t = static_cast<double>(a.pos[t0 + tt]) * (a.inverse ? -0.15915494309189535 : 0.15915494309189535) *
                     a.inv_freq[pair];  // turns
    float c, s;
    sincospif(static_cast<float>(2.0 * (t - rint(t))), &s, &c);
    table[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
  if (!mine) return;
#pragma unroll
  for (int i = 0; i < kRopeTokens; ++i) {
    if (i >= nt) break;
    uint32_t w0[4] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w};
    uint32_t w1[4] = {v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    if (turns) {
      const float4* cs = reinterpret_cast<const float4*>(table + i * half) + u;  // quarter e: cs[e * turning]
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 t = cs[e * turning];  // (cos, sin) of two pairs
        if constexpr (kInterleaved) {
          // quarters 0 and 1 are words of the first piece, 2 and 3 of the second
          uint32_t& wa = e < 2 ? w0[2 * e] : w1[2 * e - 4];
          uint32_t& wb = e < 2 ? w0[2 * e + 1] : w1[2 * e - 3];
          const float2 fa = unpack2<T>(wa), fb = unpack2<T>(wb);
          wa = pack2<T>(fa.x * t.x - fa.y * t.y, fa.x * t.y + fa.y * t.x);
          wb = pack2<T>(fb.x * t.z - fb.y * t.w, fb.x * t.w + fb.y * t.z);
        } else {
          const float2 f0 = unpack2<T>(w0[e]), f1 = unpack2<T>(w1[e]);
          w0[e] = pack2<T>(f0.x * t.x - f1.x * t.y, f0.y * t.z - f1.y * t.w);
          w1[e] = pack2<T>(f0.x * t.y + f1.x * t.x, f0.y * t.w + f1.y * t.z);
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + at[i]) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
    *reinterpret_cast<uint4*>(dst + at[i] + gap) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
  }
}

}  // namespace skv
