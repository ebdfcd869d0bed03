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
// Bound by bytes: each value is read and written once.  A thread owns 8 pairs
// (two 16-byte pieces) of one token and walks a group of heads with them, so
// the 8 sines and cosines are paid once per group.
#pragma once

#include "skv_device.cuh"

namespace skv {

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
  int group;          // heads a thread walks
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  // a programmatic dependent of the kernel before it: waits before any load
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int units = a.D >> 4;  // 16 values each
  const int64_t tokens = static_cast<int64_t>(a.B) * a.S;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t token = id / units;
  const int u = static_cast<int>(id - token * units);
  if (token >= tokens) return;
  const int b = static_cast<int>(token / a.S);
  const int s = static_cast<int>(token - static_cast<int64_t>(b) * a.S);
  const bool turns = u * 16 < a.R;
  float c[8], sn[8];
  if (turns) {
    const double p = static_cast<double>(a.pos[token]) * (a.inverse ? -0.15915494309189535 : 0.15915494309189535);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double t = p * a.inv_freq[u * 8 + e];  // turns
      sincospif(static_cast<float>(2.0 * (t - rint(t))), &sn[e], &c[e]);
      c[e] *= a.factor;
      sn[e] *= a.factor;
    }
  }
  // the two 16-byte pieces of this unit
  const int d0 = (kInterleaved || !turns) ? u * 16 : u * 8;
  const int d1 = (kInterleaved || !turns) ? u * 16 + 8 : a.R / 2 + u * 8;
  const int heads = a.heads[0] + a.heads[1];
  const int h_begin = blockIdx.y * a.group, h_end = min(heads, h_begin + a.group);
#pragma unroll 4
  for (int hh = h_begin; hh < h_end; ++hh) {
    const int which = hh >= a.heads[0] ? 1 : 0;
    const int h = which ? hh - a.heads[0] : hh;
    const int H = a.heads[which];
    const int64_t row = a.token_major ? token * H + h : (static_cast<int64_t>(b) * H + h) * a.S + s;
    const T* src = static_cast<const T*>(a.x[which]) + row * a.D;
    T* dst = static_cast<T*>(a.y[which]) + row * a.D;
    if (!turns && src == dst) continue;
    uint4 v0 = *reinterpret_cast<const uint4*>(src + d0);
    uint4 v1 = *reinterpret_cast<const uint4*>(src + d1);
    if (turns) {
      uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f0 = unpack2<T>(w0[e]), f1 = unpack2<T>(w1[e]);
        if constexpr (kInterleaved) {
          w0[e] = pack2<T>(f0.x * c[e] - f0.y * sn[e], f0.x * sn[e] + f0.y * c[e]);
          w1[e] = pack2<T>(f1.x * c[e + 4] - f1.y * sn[e + 4], f1.x * sn[e + 4] + f1.y * c[e + 4]);
        } else {
          w0[e] = pack2<T>(f0.x * c[2 * e] - f1.x * sn[2 * e], f0.y * c[2 * e + 1] - f1.y * sn[2 * e + 1]);
          w1[e] = pack2<T>(f0.x * sn[2 * e] + f1.x * c[2 * e], f0.y * sn[2 * e + 1] + f1.y * c[2 * e + 1]);
        }
      }
      v0 = make_uint4(w0[0], w0[1], w0[2], w0[3]);
      v1 = make_uint4(w1[0], w1[1], w1[2], w1[3]);
    }
    *reinterpret_cast<uint4*>(dst + d0) = v0;
    *reinterpret_cast<uint4*>(dst + d1) = v1;
  }
}

}  // namespace skv
