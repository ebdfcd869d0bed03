// Split-KV decode over the 8-bit cache: per (batch entry, kv head, group of 16
// query rows, split) one CTA streams its split's codes from HBM exactly once.
//
// With code blocks of scales ks, vs (one per block of tokens and head):
//   x_j = scale * log2(e) * ks_j * (q . ck_j),  p_j = 2^(x_j - m),  m = max x_j
//   LSE = m + log2 sum p_j,   O = sum p_j vs_j cv_j / sum p_j.
//
// Codes are exact in fp16, so both products run as m16n8k16 fp16 MMAs with
// fp32 sums whatever the type of q: a q row is multiplied by a power of two
// that brings its largest magnitude into [1, 2) (exact but for values 2^-14
// times smaller), and ks, that power and log2(e) scale the fp32 logits.  For
// P V the weights carry the block's scale: p_j vs_j is kept relative to its own
// running maximum M >= x_j + log2 vs_j, apart from the softmax's m, so that the
// fp16 weights use their range however much the scales of V differ.
//
// What bounds it: bytes.  At HBM rate an SM receives about 23 codes per clock;
// turning them into fp16 costs 1.25 (K) and 1.5 (V) lane instructions each,
// about a quarter of the issue slots, and the 16 rows' MMAs about as much
// again, so mma.sync keeps pace (tcgen05 would want 128 rows).
//
// Layout: the fragment orders of the MMAs are free as long as both operands
// agree, so a thread's fragments are contiguous bytes: of a key row, the 32
// codes at 32 (lane & 3) feed 8 steps of Q K^T; of a value row, the 16 codes at
// 16 (lane >> 2) are column n = lane >> 2 of 16 n-tiles.  Both are 16-byte
// shared loads without bank conflicts in the 128-byte swizzle TMA writes, and q
// is loaded into its fragments straight from global memory.
#pragma once

#include "skv_device.cuh"
#include "kv8.cuh"

namespace skv {

constexpr int kKv8Warps = 4;                    // consumer warps, 16 keys of a tile each
constexpr int kKv8Threads = (kKv8Warps + 1) * 32;
constexpr int kKv8Tile = kKv8Warps * 16;        // keys per tile
constexpr int kKv8Rows = 16;

template <int D>
struct Kv8DecodeCfg {
  static constexpr int kTileBytes = kKv8Tile * D;              // one K or V tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBoxes = D == 256 ? 2 : 1;              // 128-byte wide boxes
  static constexpr int kStages = D == 64 ? 8 : (D == 128 ? 6 : 3);
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kCombineBytes = 1024 + kKv8Warps * kKv8Rows * D * 4;
  static_assert(kRingBytes >= kCombineBytes, "the combine area reuses the ring");
  static constexpr int kQBytes = D == 256 ? kKv8Rows * D * 2 : 0;  // D = 256: Q fragments in shared memory
  static constexpr int kSmemBytes = kRingBytes + kQBytes + 2 * kStages * 8 + 16 + 1024;
  static constexpr int kSteps = D / 16;                        // k-steps of Q K^T
  static constexpr int kTilesN = D / 8;                        // n-tiles of P V
};

struct Kv8DecodeArgs {
  const void* q;
  void* out;
  float* lse;
  float* part_o;
  float* part_lse;
  float* logits;           // [B, Hkv, G * Lq, capacity] log2-domain logits, or null
  const float* k_scale;
  const float* v_scale;
  const int* kv_len;
  int B, Hq, Hkv, Lq, capacity, block_shift;
  int num_splits;
  int row_groups;
  int causal;
  float scale_log2;
};

// four int8 codes (a word) -> two fp16 pairs; 0x6400 | u is 1024 + u in fp16
template <bool kE4M3>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& h0, uint32_t& h1) {
  if constexpr (kE4M3) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;  // code + 128
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1024 + 128
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias), hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    h0 = *reinterpret_cast<uint32_t*>(&ha);
    h1 = *reinterpret_cast<uint32_t*>(&hb);
  }
}

template <int D, typename T, bool kE4M3, bool kLogits>
__global__ void __launch_bounds__(kKv8Threads, 2)
    decode_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const Kv8DecodeArgs a) {
  using Cfg = Kv8DecodeCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint4* qfrag = reinterpret_cast<uint4*>(smem + Cfg::kRingBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kRingBytes + Cfg::kQBytes);
  uint64_t* empty = full + Cfg::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + Cfg::kStages);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int split = blockIdx.x;
  const int G = a.Hq / a.Hkv;
  const int rows_total = G * a.Lq;
  const int rg = blockIdx.y % a.row_groups;
  const int hkv = (blockIdx.y / a.row_groups) % a.Hkv;
  const int b = blockIdx.y / (a.row_groups * a.Hkv);

  if (tid == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kKv8Warps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // a programmatic dependent of the kernel before it: waits before it touches memory
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int n = a.capacity;
  if (a.kv_len != nullptr) n = min(max(a.kv_len[b], 0), a.capacity);
  int s0 = 0, s1 = 0;
  if (n > 0) {  // the split rule of the host planner
    const int per = (n + a.num_splits - 1) / a.num_splits;
    const int C = ((per + 63) / 64) * 64;
    const int64_t lo = static_cast<int64_t>(split) * C;
    s0 = static_cast<int>(min(lo, static_cast<int64_t>(n)));
    s1 = static_cast<int>(min(lo + C, static_cast<int64_t>(n)));
  }
  const int ntiles = (s1 - s0 + kKv8Tile - 1) / kKv8Tile;
  const int64_t bh = static_cast<int64_t>(b) * a.Hkv + hkv;

  if (warp == kKv8Warps) {
    // ================= producer warp: TMA ring
    if (lane == 0 && ntiles > 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      int issued = 0;
      for (int t = 0; t < ntiles; ++t) {
        const int st = t % Cfg::kStages;
        if (t >= Cfg::kStages) {
          if (!mbar_wait(&empty[st], ((t / Cfg::kStages) & 1) ^ 1, abort_flag, kErrKv8EmptyWait)) break;
        }
        mbar_arrive_expect_tx(&full[st], Cfg::kStageBytes);
        uint8_t* kt = ring + st * Cfg::kStageBytes;
        uint8_t* vt = kt + Cfg::kTileBytes;
        const int64_t token = bh * a.capacity + s0 + static_cast<int64_t>(t) * kKv8Tile;
        const int row = static_cast<int>(D == 64 ? token >> 1 : token);  // D = 64: two tokens in a 128-byte row
#pragma unroll
        for (int bx = 0; bx < Cfg::kBoxes; ++bx) {
          tma_load_2d(kt + bx * kKv8Tile * 128, &tmK, &full[st], bx * 128, row);
          tma_load_2d(vt + bx * kKv8Tile * 128, &tmV, &full[st], bx * 128, row);
        }
        issued = t + 1;
      }
      if (*abort_flag) {
        // let every load already issued land before the CTA's shared memory goes away
        for (int t = max(0, issued - Cfg::kStages); t < issued; ++t)
          mbar_drain(&full[t % Cfg::kStages], (t / Cfg::kStages) & 1, 20000000ull);
      }
    }
    return;
  }

  // ================= consumer warps
  const int g = lane >> 2, tq = lane & 3;
  // keys of a 16-key group that n-tile nt, column c stands for
  auto key_of = [](int nt, int c) { return D == 64 ? 4 * (c >> 1) + 2 * nt + (c & 1) : nt * 8 + c; };

  // ---- Q fragments: rows g and g + 8, the D / 4 values of this thread's share
  // of every key row (64 bytes of codes per box: 32 tq .. 32 tq + 31)
  constexpr int kShare = D == 64 ? 16 : 32;   // contiguous values per box
  uint32_t qa[D == 256 ? 1 : Cfg::kSteps][4];
  float qscale[2];
  {
    uint32_t raw[2][D / 8];  // D / 4 values of each row, packed pairs
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      const int r = rg * kKv8Rows + g + 8 * hr;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) raw[hr][i] = 0;
      if (r < rows_total) {
        const int h = hkv * G + r / a.Lq;
        const T* src = static_cast<const T*>(a.q) + ((static_cast<int64_t>(b) * a.Hq + h) * a.Lq + r % a.Lq) * D;
#pragma unroll
        for (int bx = 0; bx < Cfg::kBoxes; ++bx)
#pragma unroll
          for (int i = 0; i < kShare / 8; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + bx * 128 + tq * kShare) + i);
            uint32_t* dst = &raw[hr][bx * 16 + i * 4];
            dst[0] = u.x; dst[1] = u.y; dst[2] = u.z; dst[3] = u.w;
          }
      }
    }
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, raw[hr][i] & 0x7fff7fffu);
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^-e and 2^e of the row's largest magnitude in [2^e, 2^(e + 1)); 1 for a
      // row of zeros (or beyond what both powers can hold: such a row is scaled less)
      const float amax = unpack2<T>(top).x;
      int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      e = amax > 0.f ? min(max(e, -126), 126) : 0;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      qscale[hr] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 f = unpack2<T>(raw[hr][i]);
        raw[hr][i] = pack_f16x2(f.x * down, f.y * down);
      }
    }
    // step kk takes this thread's values 4 kk .. 4 kk + 3: two packed pairs
    if constexpr (D == 256) {
      if (warp == 0) {
#pragma unroll
        for (int kk = 0; kk < Cfg::kSteps; ++kk)
          qfrag[kk * 32 + lane] = make_uint4(raw[0][2 * kk], raw[1][2 * kk], raw[0][2 * kk + 1], raw[1][2 * kk + 1]);
      }
      named_barrier_sync(1, kKv8Warps * 32);
    } else {
#pragma unroll
      for (int kk = 0; kk < Cfg::kSteps; ++kk) {
        qa[kk][0] = raw[0][2 * kk];
        qa[kk][1] = raw[1][2 * kk];
        qa[kk][2] = raw[0][2 * kk + 1];
        qa[kk][3] = raw[1][2 * kk + 1];
      }
    }
  }
  const float xs0 = a.scale_log2 * qscale[0], xs1 = a.scale_log2 * qscale[1];

  // keys each of this thread's two rows may see
  int row_end[2] = {s1, s1};
  if (a.causal) {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      const int i = (rg * kKv8Rows + g + 8 * hr) % a.Lq;
      row_end[hr] = min(s1, max(n - a.Lq + 1 + i, 0));
    }
  }
  float* lrow[2] = {nullptr, nullptr};  // this thread's logit rows
  if constexpr (kLogits) {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      const int r = rg * kKv8Rows + g + 8 * hr;
      if (r < rows_total) lrow[hr] = a.logits + (bh * rows_total + r) * a.capacity;
    }
  }

  const float* ksc = a.k_scale + bh * (a.capacity >> a.block_shift);
  const float* vsc = a.v_scale + bh * (a.capacity >> a.block_shift);
  // the 16 keys of a warp lie in one block of every block size: one scale each.
  // Scales are fetched one tile ahead.
  float ks_next = 0.f, vs_next = 0.f;
  {
    const int key0 = s0 + warp * 16;
    if (key0 < s1) {
      ks_next = __ldg(ksc + (key0 >> a.block_shift));
      vs_next = __ldg(vsc + (key0 >> a.block_shift));
    }
  }

  float m[2] = {-INFINITY, -INFINITY};    // running maximum of x
  float mv[2] = {-INFINITY, -INFINITY};   // running maximum of x + log2 vs: O's unit is 2^mv
  float lsum[2] = {0.f, 0.f};
  float o[Cfg::kTilesN][4];
#pragma unroll
  for (int j = 0; j < Cfg::kTilesN; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

  for (int t = 0; t < ntiles; ++t) {
    const int st = t % Cfg::kStages;
    const int key0 = s0 + t * kKv8Tile + warp * 16;
    const int nvalid = s1 - key0;  // may be <= 0 or > 16
    const float ks = ks_next, vs = vs_next;
    if (key0 + kKv8Tile < s1) {
      ks_next = __ldg(ksc + ((key0 + kKv8Tile) >> a.block_shift));
      vs_next = __ldg(vsc + ((key0 + kKv8Tile) >> a.block_shift));
    }
    if (!mbar_wait(&full[st], (t / Cfg::kStages) & 1, abort_flag, kErrKv8FullWait)) break;
    if (nvalid > 0) {
      const uint8_t* kt = ring + st * Cfg::kStageBytes;
      const uint8_t* vt = kt + Cfg::kTileBytes;

      // ---- S = Q K^T for 16 rows x 16 keys (two chains of MMAs per n-tile)
      float sc[2][2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) sc[nt][i][0] = sc[nt][i][1] = sc[nt][i][2] = sc[nt][i][3] = 0.f;
#pragma unroll
      for (int bx = 0; bx < Cfg::kBoxes; ++bx) {
#pragma unroll
        for (int half = 0; half < (D == 64 ? 1 : 2); ++half) {
          uint4 kw[2];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const uint32_t key = warp * 16 + key_of(nt, g);
            uint32_t off;
            if constexpr (D == 64) off = sw128(key >> 1, (key & 1) * 4 + tq);
            else off = bx * kKv8Tile * 128 + sw128(key, 2 * tq + half);
            kw[nt] = *reinterpret_cast<const uint4*>(kt + off);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kk = bx * 8 + half * 4 + i;
            uint32_t aq[4];
            if constexpr (D == 256) {
              const uint4 u = qfrag[kk * 32 + lane];
              aq[0] = u.x; aq[1] = u.y; aq[2] = u.z; aq[3] = u.w;
            } else {
              aq[0] = qa[kk][0]; aq[1] = qa[kk][1]; aq[2] = qa[kk][2]; aq[3] = qa[kk][3];
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const uint32_t w = i == 0 ? kw[nt].x : (i == 1 ? kw[nt].y : (i == 2 ? kw[nt].z : kw[nt].w));
              uint32_t b0, b1;
              codes_to_half<kE4M3>(w, b0, b1);
              mma_16816<__half>(sc[nt][i & 1], aq, b0, b1);
            }
          }
        }
      }

      // ---- online softmax (exp2 domain), rows g and g + 8
      const float f0 = xs0 * ks, f1 = xs1 * ks;
      float x[2][4];
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + key_of(nt, 2 * tq + (e & 1));
          const float val = (sc[nt][0][e] + sc[nt][1][e]) * (e < 2 ? f0 : f1);
          x[nt][e] = key < row_end[e >> 1] ? val : -INFINITY;
        }
        mx0 = fmaxf(mx0, fmaxf(x[nt][0], x[nt][1]));
        mx1 = fmaxf(mx1, fmaxf(x[nt][2], x[nt][3]));
      }
      if constexpr (kLogits) {
        // up to 16-key alignment the slots behind the last key are this warp's too
        // (-inf there); the capacity is a multiple of 16
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          if (lrow[hr] != nullptr) {
            if constexpr (D == 64) {
              *reinterpret_cast<float4*>(lrow[hr] + key0 + 4 * tq) =
                  make_float4(x[0][2 * hr], x[0][2 * hr + 1], x[1][2 * hr], x[1][2 * hr + 1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < 2; ++nt)
                *reinterpret_cast<float2*>(lrow[hr] + key0 + nt * 8 + 2 * tq) =
                    make_float2(x[nt][2 * hr], x[nt][2 * hr + 1]);
            }
          }
        }
      }
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      const float lv = __log2f(vs);  // -inf for a block of zeros
      const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
      const float vn0 = fmaxf(mv[0], mx0 + lv), vn1 = fmaxf(mv[1], mx1 + lv);
      // exponents are taken against 0 while nothing has been seen
      const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
      const float vu0 = vn0 == -INFINITY ? 0.f : vn0, vu1 = vn1 == -INFINITY ? 0.f : vn1;
      lsum[0] *= ex2_approx(m[0] - mu0);
      lsum[1] *= ex2_approx(m[1] - mu1);
      const float al0 = ex2_approx(mv[0] - vu0), al1 = ex2_approx(mv[1] - vu1);
      m[0] = mn0; m[1] = mn1;
      mv[0] = vn0; mv[1] = vn1;
      // p vs / 2^mv = p * 2^(m + log2 vs - mv); a masked key's weight is 0 whatever the scale
      // (kept finite where m lies far above the keys that set mv: their p is 0 then, and 0 * inf is not)
      float w0 = ex2_approx(mu0 + lv - vu0), w1 = ex2_approx(mu1 + lv - vu1);
      w0 = w0 == INFINITY ? 3.0e38f : w0;
      w1 = w1 == INFINITY ? 3.0e38f : w1;
      uint32_t pa[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float pw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = ex2_approx(x[nt][e] - (e < 2 ? mu0 : mu1));
          lsum[e >> 1] += p;
          pw[e] = x[nt][e] == -INFINITY ? 0.f : p * (e < 2 ? w0 : w1);
        }
        pa[2 * nt] = pack_f16x2(pw[0], pw[1]);
        pa[2 * nt + 1] = pack_f16x2(pw[2], pw[3]);
      }
      // the running maximum seldom moves after the first tiles
      if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
        for (int j = 0; j < Cfg::kTilesN; ++j) {
          o[j][0] *= al0; o[j][1] *= al0;
          o[j][2] *= al1; o[j][3] *= al1;
        }
      }

      // ---- O += P V
#pragma unroll
      for (int bx = 0; bx < Cfg::kBoxes; ++bx) {
        // 16 codes (8 for D = 64) of each of this thread's four keys
        constexpr int kWords = D == 64 ? 2 : 4;
        uint32_t r[4][kWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kin = key_of(i >> 1, 2 * tq + (i & 1));
          const uint32_t key = warp * 16 + kin;
          if constexpr (D == 64) {
            const uint2 u = *reinterpret_cast<const uint2*>(vt + sw128(key >> 1, (key & 1) * 4 + (g >> 1)) + (g & 1) * 8);
            r[i][0] = u.x; r[i][1] = u.y;
          } else {
            const uint4 u = *reinterpret_cast<const uint4*>(vt + bx * kKv8Tile * 128 + sw128(key, g));
            r[i][0] = u.x; r[i][1] = u.y; r[i][2] = u.z; r[i][3] = u.w;
          }
          // codes behind the last key may be anything (unfilled cache, e4m3 NaN):
          // their weight is 0 and so must the codes be
          if (kin >= nvalid) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) r[i][w] = 0;
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          // bytes of key pairs side by side: {k0.b0, k1.b0, k0.b1, k1.b1} and so on
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const uint32_t lo = __byte_perm(r[0][w], r[1][w], hb ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(r[2][w], r[3][w], hb ? 0x7362 : 0x5140);
            uint32_t l0, l1, h0, h1;
            codes_to_half<kE4M3>(lo, l0, l1);
            codes_to_half<kE4M3>(hi, h0, h1);
            const int j = bx * 16 + w * 4 + hb * 2;
            mma_16816<__half>(o[j], pa, l0, h0);
            mma_16816<__half>(o[j + 1], pa, l1, h1);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }

  // ---- combine the four warps' states
  named_barrier_sync(1, kKv8Warps * 32);
  if (*abort_flag != 0) return;
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    lsum[hr] += __shfl_xor_sync(0xffffffffu, lsum[hr], 1);
    lsum[hr] += __shfl_xor_sync(0xffffffffu, lsum[hr], 2);
  }
  float* cm = reinterpret_cast<float*>(ring);            // [4][16] running max
  float* cl = cm + kKv8Warps * kKv8Rows;                 // [4][16] sums
  float* cv = cl + kKv8Warps * kKv8Rows;                 // [4][16] O's units
  float4* co4 = reinterpret_cast<float4*>(ring + 1024);  // [4][D / 8][32] fragments
  if (tq == 0) {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      cm[warp * 16 + g + 8 * hr] = m[hr];
      cl[warp * 16 + g + 8 * hr] = lsum[hr];
      cv[warp * 16 + g + 8 * hr] = mv[hr];
    }
  }
#pragma unroll
  for (int j = 0; j < Cfg::kTilesN; ++j)
    co4[(warp * Cfg::kTilesN + j) * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
  named_barrier_sync(1, kKv8Warps * 32);

  // Per row: M = max_w m_w, L = sum_w 2^(m_w - M) l_w; O = sum_w 2^(mv_w - M) O_w / L
  // (2^(mv_w - M) <= the largest vs: finite), LSE = M + log2 L.
  const int rows_here = min(kKv8Rows, rows_total - rg * kKv8Rows);
  const int64_t rows_all = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
  const int64_t orow0 = (static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(hkv) * G) * a.Lq +
                        static_cast<int64_t>(rg) * kKv8Rows;
  if (g >= rows_here) return;
  float wt[2][kKv8Warps];
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    const int r = g + 8 * hr;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) M = fmaxf(M, cm[w * 16 + r]);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) {
      const float mw = cm[w * 16 + r], vw = cv[w * 16 + r];
      // a warp whose maximum is -inf saw no key, or only NaN: its sum then says so
      L += mw == -INFINITY ? cl[w * 16 + r] : ex2_approx(mw - M) * cl[w * 16 + r];
      wt[hr][w] = vw == -INFINITY ? 0.f : ex2_approx(vw - (M == -INFINITY ? 0.f : M));
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) wt[hr][w] *= inv;
    if (warp == 0 && tq == 0 && r < rows_here) {
      float lse = L == 0.f ? -INFINITY : M + __log2f(L);
      if (a.num_splits == 1) {
        if (a.lse != nullptr) a.lse[orow0 + r] = lse;
      } else {
        // a NaN partial is handed on as +inf: the merge's maximum would drop a
        // NaN and take the row for empty, while 2^(inf - inf) keeps it
        a.part_lse[static_cast<int64_t>(split) * rows_all + orow0 + r] = isnan(lse) ? INFINITY : lse;
      }
    }
  }
  const bool hi = g + 8 < rows_here;
  // thread t combines fragment slots j = warp + 4 k of its lane: columns
  // 2 tq and 2 tq + 1 of n-tile j, i.e. values d(2 tq) and d(2 tq + 1)
#pragma unroll
  for (int k = 0; k < Cfg::kTilesN / kKv8Warps; ++k) {
    const int j = warp + kKv8Warps * k;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) {
      const float4 v = co4[(w * Cfg::kTilesN + j) * 32 + lane];
      acc.x = fmaf(wt[0][w], v.x, acc.x);
      acc.y = fmaf(wt[0][w], v.y, acc.y);
      acc.z = fmaf(wt[1][w], v.z, acc.z);
      acc.w = fmaf(wt[1][w], v.w, acc.w);
    }
    constexpr int kSpan = D == 64 ? 8 : 16;  // columns of n stand kSpan values apart
    const int d = (j / 16) * 128 + 2 * tq * kSpan + j % 16;
    if (a.num_splits == 1) {
      T* dst = static_cast<T*>(a.out) + (orow0 + g) * D + d;
      const uint32_t lo = pack2<T>(acc.x, acc.y), up = pack2<T>(acc.z, acc.w);
      *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(lo);
      *reinterpret_cast<uint16_t*>(dst + kSpan) = static_cast<uint16_t>(lo >> 16);
      if (hi) {
        *reinterpret_cast<uint16_t*>(dst + 8 * D) = static_cast<uint16_t>(up);
        *reinterpret_cast<uint16_t*>(dst + 8 * D + kSpan) = static_cast<uint16_t>(up >> 16);
      }
    } else {
      float* dst = a.part_o + (static_cast<int64_t>(split) * rows_all + orow0 + g) * D + d;
      dst[0] = acc.x;
      dst[kSpan] = acc.y;
      if (hi) {
        dst[8 * D] = acc.z;
        dst[8 * D + kSpan] = acc.w;
      }
    }
  }
}

// Attention weights of the keys: weights[b, h, j] += sum over the rows of kv
// head h of 2^(x_j - LSE), from the logits the split kernel left and the merged
// LSE (rows that see no key add nothing).  Bound by bytes: 4 per row and key,
// most of them still in L2, and 8 per key.  A thread takes 4 keys.
struct Kv8WeightArgs {
  const float* logits;   // [B, Hkv, rows, capacity]
  const float* lse;      // [B, Hkv, rows]
  float* weights;        // [B, Hkv, capacity]
  const int* kv_len;
  int Hkv, rows, capacity;
};

__global__ void __launch_bounds__(256) kv8_weights_kernel(const Kv8WeightArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / a.Hkv);
  const int n = a.kv_len != nullptr ? min(max(a.kv_len[b], 0), a.capacity) : a.capacity;
  const int j = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (j >= n) return;
  const float* x = a.logits + bh * a.rows * a.capacity + j;
  const float* lse = a.lse + bh * a.rows;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int r = 0; r < a.rows; ++r) {
    const float4 v = *reinterpret_cast<const float4*>(x + static_cast<int64_t>(r) * a.capacity);
    const float L = lse[r];
    if (L == -INFINITY) continue;  // no visible key
    s[0] += ex2_approx(v.x - L);
    s[1] += ex2_approx(v.y - L);
    s[2] += ex2_approx(v.z - L);
    s[3] += ex2_approx(v.w - L);
  }
  float* w = a.weights + bh * a.capacity + j;
  if (j + 4 <= n) {
    float4 v = *reinterpret_cast<float4*>(w);
    v.x += s[0]; v.y += s[1]; v.z += s[2]; v.w += s[3];
    *reinterpret_cast<float4*>(w) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < n) w[e] += s[e];
  }
}

}  // namespace skv
