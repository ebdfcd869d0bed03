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
// Bound by bytes: each value is read and written once.  A CTA takes a few tokens
// and many heads: their sines and cosines are computed once into shared memory,
// then its threads walk units of 8 pairs (two 16-byte pieces) in the order of
// memory (heads inside a token, or tokens inside a head).
#pragma once

#include "skv_device.cuh"

namespace skv {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;      // units a thread has in flight
constexpr int kRopeTableBytes = 16384;

struct RopeArgs {
  const void* x[2];   // q, k
  void* y[2];
  int heads[2];       // Hq, Hkv (0: no k)
  const int32_t* pos;
  const double* inv_freq;
  float factor;
  int inverse;
  int B, S, D, R;
  int token_major;    // 1: [B, S, H, D] (NHD, TND); 0: [B, H, S, D]
  int tokens;         // of a CTA: tokens * R / 2 pairs fit the table
  int group;          // heads of a CTA
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  __shared__ float4 table4[kRopeTableBytes / 16];  // (cos, sin) of [token][pair]
  float2* table = reinterpret_cast<float2*>(table4);
  // a programmatic dependent of the kernel before it: waits before any load
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int half = a.R >> 1, units = a.D >> 4;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens), static_cast<int64_t>(a.B) * a.S - t0));
  const int h0 = blockIdx.y * a.group, nh = min(a.group, a.heads[0] + a.heads[1] - h0);
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tt = i / half, pair = i - tt * half;
    const double t = static_cast<double>(a.pos[t0 + tt]) * (a.inverse ? -0.15915494309189535 : 0.15915494309189535) *
                     a.inv_freq[pair];  // turns
    float c, s;
    sincospif(static_cast<float>(2.0 * (t - rint(t))), &s, &c);
    table[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
  const int total = nt * nh * units;
  for (int e0 = threadIdx.x; e0 < total; e0 += kRopeThreads * kRopeUnroll) {
    uint4 v[kRopeUnroll][2];
    T* dst[kRopeUnroll];
    int place[kRopeUnroll];  // first pair of a unit in the table, or -1 where it is copied
    int gap[kRopeUnroll];    // values between its two pieces
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      const int e = e0 + j * kRopeThreads;
      dst[j] = nullptr;
      if (e >= total) continue;
      const int r = e / units, u = e - r * units;
      int tt, hh;
      if (a.token_major) {
        tt = r / nh;
        hh = r - tt * nh;
      } else {
        hh = r / nt;
        tt = r - hh * nt;
      }
      const int which = h0 + hh >= a.heads[0] ? 1 : 0;
      const int h = h0 + hh - (which ? a.heads[0] : 0), H = a.heads[which];
      const int64_t token = t0 + tt;
      int64_t row = token * H + h;
      if (!a.token_major) {
        const int64_t b = token / a.S;
        row = (b * H + h) * a.S + (token - b * a.S);
      }
      const bool turns = u * 16 < a.R;
      const bool split = turns && !kInterleaved;  // pieces half a rotary dimension apart
      const int64_t at = row * a.D + (split ? u * 8 : u * 16);
      gap[j] = split ? half : 8;
      place[j] = turns ? tt * half + u * 8 : -1;
      const T* src = static_cast<const T*>(a.x[which]) + at;
      T* to = static_cast<T*>(a.y[which]) + at;
      if (!turns && src == to) continue;  // copied onto itself
      dst[j] = to;
      v[j][0] = *reinterpret_cast<const uint4*>(src);
      v[j][1] = *reinterpret_cast<const uint4*>(src + gap[j]);
    }
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      if (dst[j] == nullptr) continue;
      uint32_t w0[4] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w};
      uint32_t w1[4] = {v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
      if (place[j] >= 0) {
        const float4* cs = reinterpret_cast<const float4*>(table + place[j]);  // two pairs each
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f0 = unpack2<T>(w0[e]), f1 = unpack2<T>(w1[e]);
          if constexpr (kInterleaved) {
            const float4 ta = cs[e >> 1], tb = cs[2 + (e >> 1)];
            const float ca = e & 1 ? ta.z : ta.x, sa = e & 1 ? ta.w : ta.y;
            const float cb = e & 1 ? tb.z : tb.x, sb = e & 1 ? tb.w : tb.y;
            w0[e] = pack2<T>(f0.x * ca - f0.y * sa, f0.x * sa + f0.y * ca);
            w1[e] = pack2<T>(f1.x * cb - f1.y * sb, f1.x * sb + f1.y * cb);
          } else {
            const float4 t = cs[e];
            w0[e] = pack2<T>(f0.x * t.x - f1.x * t.y, f0.y * t.z - f1.y * t.w);
            w1[e] = pack2<T>(f0.x * t.y + f1.x * t.x, f0.y * t.w + f1.y * t.z);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst[j]) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
      *reinterpret_cast<uint4*>(dst[j] + gap[j]) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
    }
  }
}

}  // namespace skv
