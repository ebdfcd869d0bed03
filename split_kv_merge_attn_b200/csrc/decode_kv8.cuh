// Split-KV decode over the 8-bit cache.  The keys of every unit (batch entry, kv
// head, group of 16 query rows) form tiles; all units' tiles in a row are divided
// evenly among the CTAs, two to an SM, whatever the sequences' lengths.  A CTA's
// share is one or more segments of units; it streams each segment's codes from HBM
// exactly once and writes the unit's result where the segment is all of it, else a
// partial (O, LSE) that kv8_merge_kernel joins.  (Equal splits of each sequence
// left SMs idle where lengths differ or units do not divide the SMs: B = 16, 16
// heads, D = 64, lengths 4096 to 16384: 89 us with one split, 74 with the best,
// 65 so, all without the keys' weights.)
//
// With code blocks of scales ks, vs (one per block of tokens and head):
//   x_j = scale * log2(e) * ks_j * (q . ck_j),  p_j = 2^(x_j - m),  m = max x_j
//   LSE = m + log2 sum p_j,   O = sum p_j vs_j cv_j / sum p_j.
//
// Codes are exact in fp16, so both products run as m16n8k16 fp16 MMAs with
// fp32 sums whatever the type of q: a q row is multiplied by a power of two
// that brings its largest magnitude into [1, 2) (exact but for values 2^-14
// times smaller), and ks, that power and log2(e) scale the fp32 logits.  For
// P V the weights carry the block's scale: p_j vs_j is kept relative to a reference
// of its own, 2^d beside the softmax's 2^m with d >= x_j - m + log2 vs_j, so that the
// fp16 weights use their range however much the scales of V differ (and d is small
// whatever the logits: kept as m + d it lost V's scale beside large ones).  Both
// references follow the maxima loosely (within a factor of 2^8), and the weights'
// lies 2^7 below: they end at 2^15, and what is dropped lies 2^-32 below the heaviest.
//
// What bounds it: bytes at D = 64 and e4m3 (6.1 TB/s; a copy reaches 6.6), else the
// latency of each warp's own chain of arrival, conversion, Q K^T, softmax and P V, with
// the two warps a scheduler that registers allow.  At D = 128, int8, 32768 keys nothing
// is saturated: issue 41%, tensor pipe 30%, DRAM 55%; of the 4.8 cycles between two
// instructions of a warp 1.6 are fixed latencies of the instruction before, 0.8 waits
// for loads and barriers, 0.3 for a busy pipe.  (Turning a code costs 1.25 (K) and 1.5
// (V) lane instructions for int8, less for e4m3; tcgen05 would want 128 rows.)  Whole
// calls, bf16 q, one row a head:
//   D = 64,  B = 16, 16 / 16 heads, 16384 keys: e4m3 87.5 us (6.1 TB/s), int8 99.0 (5.4)
//   D = 128, B = 2, 32 / 8 heads, 32768 keys:   e4m3 28.1 us (4.8 TB/s), int8 30.5 (4.4)
//   D = 256, B = 1, 16 / 4 heads, 131072 keys:  e4m3 49.8 us (5.4 TB/s), int8 55.8 (4.8)
//   D = 128, B = 1, 32 / 8 heads, 4096 keys:    e4m3 8.7 us, int8 8.9: latency
// Of these about 5 us are the start, the four warps' combine and the merge launch: at
// 4096 keys the decode over 16-bit keys, of fewer parts, takes 6.8 us (at 32768 keys,
// B = 2, 45.3).
//
// Layout: the order of a product's summands is free as long as both operands
// agree, so of a key row a thread takes the 32 contiguous codes at 32 (lane & 3)
// for 8 steps of Q K^T (16-byte shared loads, no bank conflicts in the 128-byte
// swizzle TMA writes), and q is loaded into its fragments straight from global
// memory.  V comes through ldmatrix.trans as 16-bit units: a register holds
// values 2g, 2g + 1 of two keys, which unpack into fragments of an even and an
// odd n-tile.
//
// Each warp runs alone: it loads its own tiles (16 to 64 keys) into its own ring
// and refills a stage as soon as it has read it, so there is no producer warp,
// no barrier among warps until the end, and eight warps share an SM's registers.
#pragma once

#include <type_traits>

#include "skv_device.cuh"
#include "kv8.cuh"

namespace skv {

constexpr int kKv8Warps = 4;
constexpr int kKv8Threads = kKv8Warps * 32;
constexpr int kKv8Rows = 16;

template <int D>
struct Kv8DecodeCfg {
  static constexpr int kKeys = D == 64 ? 64 : (D == 128 ? 32 : 16);  // keys of a load (4 KB of K, 4 KB of V)
  static constexpr int kLoads = D == 128 ? 2 : 1;              // loads of one softmax tile
  static constexpr int kTileKeys = kKeys * kLoads;             // of a warp
  static constexpr int kCtaKeys = kKv8Warps * kTileKeys;       // a tile of the division among CTAs
  static constexpr int kTileBytes = kKeys * D;                 // one load of K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kBoxes = D == 256 ? 2 : 1;              // 128-byte wide boxes
  static constexpr int kBoxRows = D == 64 ? kKeys / 2 : kKeys;
  static constexpr int kStages = 3;
  static constexpr int kRingBytes = kKv8Warps * kStages * kStageBytes;
  static constexpr int kCombineBytes = 1024 + kKv8Warps * kKv8Rows * D * 4;
  static_assert(kRingBytes >= kCombineBytes, "the combine area reuses the ring");
  static constexpr int kQBytes = D == 256 ? kKv8Rows * D * 2 : 0;  // D = 256: Q fragments in shared memory
  static constexpr int kSmemBytes = kRingBytes + kQBytes + kKv8Warps * 2 * kStages * 8 + 16 + 1024;
  static constexpr int kSteps = D / 16;                        // k-steps of Q K^T
  static constexpr int kTilesN = D / 8;                        // n-tiles of P V
  static constexpr int kGroups = kTileKeys / 16;               // 16-key groups of a tile
};

// 2-D tiled load (no multicast) whose lines leave L2 first: codes are read once,
// the partials and logits again (B = 2, 32768 keys with weights: 48 -> 44 us).
__device__ __forceinline__ void tma_load_2d_once(void* smem_dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], "
      "[%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

struct Kv8DecodeArgs {
  const void* q;
  void* out;
  float* lse;
  uint32_t* table;         // [B + 1] places (of one head and row group) of the sequences before each, for the
                           // merge, where kv_len is given and units can be divided; else null
  float* part_o;           // [slots, 16, D]
  float* part_lse;         // [slots, 16]
  float* logits;           // [B, Hkv, G * Lq, capacity] log2-domain logits, or null
  const float* k_scale;
  const float* v_scale;
  const int* kv_len;
  int B, Hq, Hkv, Lq, capacity, block_shift;
  int row_groups;
  int causal;
  float scale_log2;
};

// How `total` places are divided among `ctas` CTAs (no more than places): the
// first `rest` of them take quota + 1, the others quota.  A unit of T > 0 tiles has
// T + 1 places: one before its first tile, for the time a CTA takes to change
// units (about a tile's), which holds no keys.  Segment (c, unit u) has partial
// slot c + u: along the places either grows by one.
struct Kv8Division {
  uint32_t ctas, quota, rest;
  __device__ __forceinline__ Kv8Division(uint32_t total, uint32_t most) {
    ctas = max(1u, min(most, total));
    quota = total / ctas;
    rest = total - quota * ctas;
  }
  // first place of CTA c's share
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return min(c, ctas) * quota + min(c, rest); }
  // the CTA that has place t
  __device__ __forceinline__ uint32_t owner(uint32_t t) const {
    const uint32_t big = rest * (quota + 1);
    return t < big ? t / (quota + 1) : rest + (t - big) / quota;
  }
};

// A word of codes {a, b, c, d} -> fp16 pairs (a, b) and (c, d).  int8: 0x6400 | u
// is 1024 + u in fp16, with u = code + 128.
template <bool kE4M3>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& h0, uint32_t& h1) {
  if constexpr (kE4M3) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1024 + 128
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias), hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    h0 = *reinterpret_cast<uint32_t*>(&ha);
    h1 = *reinterpret_cast<uint32_t*>(&hb);
  }
}

// The smaller of two values, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The same with the pairs (a, c) and (b, d).
template <bool kE4M3>
__device__ __forceinline__ void codes_to_half_even_odd(uint32_t w, uint32_t& h0, uint32_t& h1) {
  if constexpr (kE4M3) {
    codes_to_half<true>(__byte_perm(w, 0, 0x3120), h0, h1);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias), hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    h0 = *reinterpret_cast<uint32_t*>(&ha);
    h1 = *reinterpret_cast<uint32_t*>(&hb);
  }
}

// The weights of a tile from its scores s (x = s f): p = 2^(x - m), added to the
// sums, and fp16 p vs / 2^d, the A fragments of P V.  kSplit: what that rounding
// leaves, in fp16 too (pl); kLow: the same in rows 8-15, which hold no rows of their
// own (kHalves = 1).  kCareful: some keys are masked (s = -inf), or m is so large that
// x must be rounded as it was for m: fused with the difference, the product's own rounding,
// 2^-24 of it, would be in p's exponent.
template <int kGroups, int kHalves, bool kCareful, bool kSplit, bool kLow>
__device__ __forceinline__ void tile_weights(const float (&s)[2 * kGroups][4], const float (&f)[kHalves][kGroups],
                                             const float (&lv)[kGroups], const float (&m)[kHalves],
                                             const float (&d)[kHalves], float (&lsum)[kHalves], uint32_t (&pa)[kGroups][4],
                                             uint32_t (&pl)[kSplit ? kGroups : 1][4]) {
#pragma unroll
  for (int hr = 0; hr < kHalves; ++hr) {
    uint64_t sum = f2_pack(0.f, 0.f);
    const uint64_t minus_m = f2_pack(-m[hr], -m[hr]);
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
      // p vs / 2^d = p * 2^(log2 vs - d), kept finite where m lies far above the keys
      // that set d: their p is 0 then, and 0 * inf is not
      const float w = min_nan(ex2_approx(lv[gr] - d[hr]), 3.0e38f);
      const uint64_t ww = f2_pack(w, w), ff = f2_pack(f[hr][gr], f[hr][gr]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float sa = s[2 * gr + i][2 * hr], sb = s[2 * gr + i][2 * hr + 1];
        const float2 x = kCareful ? make_float2(__fsub_rn(__fmul_rn(sa, f[hr][gr]), m[hr]),
                                                __fsub_rn(__fmul_rn(sb, f[hr][gr]), m[hr]))
                                  : f2_unpack(ffma2(f2_pack(sa, sb), ff, minus_m));
        float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        if constexpr (kCareful) {  // a masked key's weight is 0 whatever its scales
          p.x = sa == -INFINITY ? 0.f : p.x;
          p.y = sb == -INFINITY ? 0.f : p.y;
        }
        const uint64_t pp = f2_pack(p.x, p.y);
        sum = fadd2(sum, pp);
        float2 pw = f2_unpack(fmul2(pp, ww));
        if constexpr (kCareful) {
          pw.x = sa == -INFINITY ? 0.f : pw.x;
          pw.y = sb == -INFINITY ? 0.f : pw.y;
        }
        pa[gr][2 * i + hr] = pack_f16x2(pw.x, pw.y);
        if constexpr (kSplit || kLow) {
          const float2 kept = unpack2<__half>(pa[gr][2 * i + hr]);
          (kLow ? pa[gr][2 * i + 1] : pl[gr][2 * i + hr]) = pack_f16x2(pw.x - kept.x, pw.y - kept.y);
        } else if constexpr (kHalves == 1) {
          pa[gr][2 * i + 1] = 0u;
        }
      }
    }
    const float2 both = f2_unpack(sum);
    lsum[hr] += both.x + both.y;
  }
}

// kHalves: 1 where a unit has at most 8 query rows (MMA rows 0-7), which leaves out
// half the softmax, else 2 (with one row, bf16: B = 16, 16 heads, D = 64, 16384 keys, e4m3
// 87.5 us against 95.5, int8 99.0 against 103.9; more rows need 2).
template <int D, typename T, bool kE4M3, bool kLogits, int kHalves>
__global__ void __launch_bounds__(kKv8Threads, 2)
    decode_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const Kv8DecodeArgs a) {
  using Cfg = Kv8DecodeCfg<D>;
  constexpr int kKeys = Cfg::kKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint4* qfrag = reinterpret_cast<uint4*>(smem + Cfg::kRingBytes);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  uint8_t* ring = smem + warp * Cfg::kStages * Cfg::kStageBytes;  // this warp's
  // arrival of the K tile, and of the V tile, of each stage
  uint64_t* full_k = reinterpret_cast<uint64_t*>(smem + Cfg::kRingBytes + Cfg::kQBytes) + warp * 2 * Cfg::kStages;
  uint64_t* full_v = full_k + Cfg::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kRingBytes + Cfg::kQBytes +
                                                             kKv8Warps * 2 * Cfg::kStages * 8);
  const int G = a.Hq / a.Hkv;
  const int rows_total = G * a.Lq;
  const int heads = a.Hkv * a.row_groups;  // units of a sequence
  __shared__ uint32_t scan[kKv8Warps];
  __shared__ uint32_t s_base;
  __shared__ int s_b;

  if (lane == 0) {
    for (int s = 0; s < 2 * Cfg::kStages; ++s) mbar_init(&full_k[s], 1);
    fence_mbar_init();
  }
  if (tid == 0) *abort_flag = 0;
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  __syncthreads();
  // a programmatic dependent of the kernel before it: waits before it touches memory
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  constexpr int kTileKeys = Cfg::kTileKeys;
  constexpr int kStride = Cfg::kCtaKeys;
  auto length = [&](int b) { return a.kv_len != nullptr ? min(max(__ldg(a.kv_len + b), 0), a.capacity) : a.capacity; };
  auto tiles = [](int n) { return (n + kStride - 1) / kStride; };
  auto places = [&](int n) { return n > 0 ? static_cast<uint32_t>(tiles(n)) + 1 : 0u; };
  // ---- this CTA's places [w, w1), and the sequence the first lies in: b, whose
  // places begin at `base`
  uint32_t w, w1, base;
  int b;
  if (a.kv_len == nullptr) {
    const uint32_t each = places(a.capacity) * heads;
    const Kv8Division division(each * a.B, gridDim.x);
    w = division.begin(blockIdx.x);
    w1 = division.begin(blockIdx.x + 1);
    b = static_cast<int>(w / each);
    base = b * each;
  } else {
    // thread i sums the places of sequences i * per ...
    const int per = (a.B + kKv8Threads - 1) / kKv8Threads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    uint32_t mine = 0;
    for (int i = b0; i < b1; ++i) mine += places(length(i));
    uint32_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) scan[warp] = before;
    __syncthreads();
    before -= mine;
    uint32_t total = 0;
#pragma unroll
    for (int i = 0; i < kKv8Warps; ++i) {
      if (i < warp) before += scan[i];
      total += scan[i];
    }
    const Kv8Division division(total * heads, gridDim.x);
    w = division.begin(blockIdx.x);
    w1 = division.begin(blockIdx.x + 1);
    if (w >= before * heads && w < (before + mine) * heads) {
      uint32_t at = before;
      int i = b0;
      for (; i < b1; ++i) {
        const uint32_t t = places(length(i));
        if (w < (at + t) * heads) break;
        at += t;
      }
      s_b = i;
      s_base = at * heads;
    }
    if (a.table != nullptr && blockIdx.x == 0) {
      for (int i = b0; i < b1; ++i) {
        a.table[i] = before;
        before += places(length(i));
      }
      if (tid == 0) a.table[a.B] = total;
    }
    __syncthreads();
    b = s_b;       // (not set, and not used, where the share is empty)
    base = s_base;
  }
  // units without keys: O = 0, LSE = -inf
  if (a.kv_len != nullptr) {
    for (int64_t u = blockIdx.x; u < static_cast<int64_t>(a.B) * heads; u += gridDim.x) {
      const int ub = static_cast<int>(u / heads), uh = static_cast<int>(u - static_cast<int64_t>(ub) * heads);
      if (length(ub) > 0) continue;
      const int r0 = uh % a.row_groups * kKv8Rows, rn = min(kKv8Rows, rows_total - r0);
      const int64_t row = (static_cast<int64_t>(ub) * a.Hq + static_cast<int64_t>(uh / a.row_groups) * G) * a.Lq + r0;
      for (int i = tid; i < rn * (D / 8); i += kKv8Threads)
        reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * D)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse != nullptr && tid < rn) a.lse[row + tid] = -INFINITY;
    }
  }

  const int g = lane >> 2, tq = lane & 3;
  int st_k = 0, st_v = 0;            // stages of the next K and V load to be read
  uint32_t phase_k = 0, phase_v = 0;
  int seen = 0;                      // loads of the segments before
  while (w < w1) {
    const int n = length(b);
    const uint32_t unit_places = places(n);
    if (w >= base + unit_places * heads) {  // the next sequence
      base += unit_places * heads;
      ++b;
      continue;
    }
    const int uh = static_cast<int>((w - base) / unit_places);
    const uint32_t p0 = w - base - uh * unit_places, p1 = min(unit_places, p0 + (w1 - w));
    w += p1 - p0;
    const int t_first = max(static_cast<int>(p0), 1) - 1, t_end = static_cast<int>(p1) - 1;
    if (t_end <= t_first) continue;         // only the place without keys
    const bool whole_unit = t_end - t_first == tiles(n);
    const int hkv = uh / a.row_groups, rg = uh - hkv * a.row_groups;
    const int s0 = t_first * kStride, s1 = min(n, t_end * kStride);
    const int64_t bh = static_cast<int64_t>(b) * a.Hkv + hkv;
    // this warp's tiles: keys first + t * kStride; loads u = kLoads * t + i of their
    // kKeys keys, the last ones of which may lie behind the end
    const int first = s0 + warp * kTileKeys;
    const int ntiles = first < s1 ? (s1 - first + kStride - 1) / kStride : 0;
    const int nloads = ntiles * Cfg::kLoads;

    // load u of K (part 0) or V (1) into its stage (lane 0)
    const int64_t token0 = bh * a.capacity + first;
    auto load = [&](int u, int st, const CUtensorMap* map, int part, uint64_t* full) {
      uint8_t* dst = ring + st * Cfg::kStageBytes + part * Cfg::kTileBytes;
      const int64_t token = token0 + u / Cfg::kLoads * kStride + u % Cfg::kLoads * kKeys;
      const int row = static_cast<int>(D == 64 ? token >> 1 : token);  // D = 64: two tokens in a 128-byte row
      mbar_arrive_expect_tx(&full[st], Cfg::kTileBytes);
#pragma unroll
      for (int bx = 0; bx < Cfg::kBoxes; ++bx)
        tma_load_2d_once(dst + bx * kKeys * 128, map, &full[st], bx * 128, row, policy);
    };
    // ---- Q fragments: rows g and g + 8, this thread's share of every key row
    // (32 contiguous values per box at 32 tq; 16 at 16 tq for D = 64)
    constexpr int kShare = D == 64 ? 16 : 32;
    uint32_t qa[D == 256 ? 1 : Cfg::kSteps][4];
    float qscale[kHalves];
    {
      uint32_t raw[kHalves][D / 8];
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr) {
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
      // the first tiles, behind q's loads: behind every CTA's tiles q arrived 3 to 4 us late
      if (lane == 0) {
        int st = st_k;  // = st_v between segments
        for (int u = 0; u < min(nloads, Cfg::kStages); ++u) {
          load(u, st, &tmK, 0, full_k);
          load(u, st, &tmV, 1, full_v);
          if (++st == Cfg::kStages) st = 0;
        }
      }
      __syncwarp();
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, raw[hr][i] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e and 2^e of the row's largest magnitude in [2^e, 2^(e + 1)); 1 for a
        // row of zeros (clamped where one of the powers would not be a normal number)
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
            qfrag[kk * 32 + lane] = make_uint4(raw[0][2 * kk], kHalves == 2 ? raw[kHalves - 1][2 * kk] : 0u,
                                               raw[0][2 * kk + 1], kHalves == 2 ? raw[kHalves - 1][2 * kk + 1] : 0u);
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int kk = 0; kk < Cfg::kSteps; ++kk) {
          qa[kk][0] = raw[0][2 * kk];
          qa[kk][1] = kHalves == 2 ? raw[kHalves - 1][2 * kk] : 0u;
          qa[kk][2] = raw[0][2 * kk + 1];
          qa[kk][3] = kHalves == 2 ? raw[kHalves - 1][2 * kk + 1] : 0u;
        }
      }
    }
    float xs[kHalves];
#pragma unroll
    for (int hr = 0; hr < kHalves; ++hr) xs[hr] = a.scale_log2 * qscale[hr];

    // keys each of this thread's two rows may see; every row sees those below safe_end
    int row_end[kHalves];
#pragma unroll
    for (int hr = 0; hr < kHalves; ++hr) row_end[hr] = s1;
    int safe_end = s1;
    if (a.causal) {
      safe_end = min(s1, n - a.Lq + 1);
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr) {
        const int i = (rg * kKv8Rows + g + 8 * hr) % a.Lq;
        row_end[hr] = min(s1, max(n - a.Lq + 1 + i, 0));
      }
    }
    float* lrow[kHalves] = {};  // this thread's logit rows
    if constexpr (kLogits) {
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr) {
        const int r = rg * kKv8Rows + g + 8 * hr;
        if (r < rows_total) lrow[hr] = a.logits + (bh * rows_total + r) * a.capacity;
      }
    }

    const float* ksc = a.k_scale + bh * (a.capacity >> a.block_shift);
    const float* vsc = a.v_scale + bh * (a.capacity >> a.block_shift);
    // 16 keys lie in one block of every block size, so a tile has one pair of scales
    // for each group of 16.  A lane holds those of one group of the next 32 / kGroups
    // tiles (0 for a group behind the last key), loaded that many tiles ahead: under
    // load a scale takes longer to arrive than a tile to compute (one tile ahead cost
    // 1.2 us of 31 at D = 128, 15 us of 110 at D = 64).
    constexpr int kChunk = 32 / Cfg::kGroups;  // tiles of a chunk
    float ks_chunk = 0.f, lv_chunk = 0.f, ks_ahead = 0.f, vs_ahead = 0.f;
    auto fetch_scales = [&](int key0) {
      const int64_t key = key0 + static_cast<int64_t>(lane / Cfg::kGroups) * kStride + lane % Cfg::kGroups * 16;
      ks_ahead = key < s1 ? __ldg(ksc + (key >> a.block_shift)) : 0.f;
      vs_ahead = key < s1 ? __ldg(vsc + (key >> a.block_shift)) : 0.f;
    };
    fetch_scales(first);
    int chunk_tile = 0;  // the current tile's place in its chunk

    // m and d are references a little behind the running maxima of x and of x - m +
    // log2 vs: they move only when a value lies more than 2^kSlack above, so
    // most tiles need no reduction over a row and no rescaling.  p then reaches
    // 2^kSlack, and the fp16 weights p vs / 2^d, with d kLift below, 2^(kSlack + kLift): within
    // fp16's limit, and as far as can be from its smallest step.  (With d at the maximum
    // a warp lost the keys 2^-25 below its heaviest: of 2^20 keys of one CTA, 2^-26 each
    // beside one of 1, a quarter of their sum.)
    constexpr float kSlack = 8.f, kLift = 7.f;
    constexpr float kNone = -3.0e38f;   // nothing seen yet
    constexpr float kLowest = -1.0e30f; // no value of V but zeros yet
    constexpr float kLarge = 65536.f;   // of m: x is off by less than 2^-8 below it
    bool large = false;                 // some row's m lies above that (the same for the whole warp)
    float m[kHalves], d[kHalves], lsum[kHalves];
#pragma unroll
    for (int hr = 0; hr < kHalves; ++hr) {
      m[hr] = kNone;
      d[hr] = kLowest;
      lsum[hr] = 0.f;
    }
    float o[Cfg::kTilesN][4];
#pragma unroll
    for (int j = 0; j < Cfg::kTilesN; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    // A weight rounded to fp16 once (2^-11 of it at most) turns about one bf16 output in
    // sixteen to the other side of a tie and adds 1.2 to 1.6 times an fp16 output's own
    // rounding.  Of at most 8 rows a weight is two fp16 numbers (2^-22), the second in rows
    // 8-15, at no MMA (whole calls, bf16, in two numbers against one: B = 16, 16 heads, D =
    // 64, 16384 keys, e4m3 87.5 us against 87.0, int8 99.0 against 100.7; D = 256, 131072
    // keys, e4m3 49.7 against 50.7).  Of 16 rows that takes twice the MMAs of P V (B = 2, 32 /
    // 8 heads, Lq = 4, D = 128, 32768 keys, int8: 37.5 us against 31.6): fp16 outputs have
    // it, bf16 ones have one number, off by an eighth of bf16's own 2^-8 at most.
    constexpr bool kLow = kHalves == 1;
    constexpr bool kSplit = std::is_same<T, __half>::value && kHalves == 2;
    constexpr int kNt = kTileKeys / 8;
    // O += P V over one group of 16 keys, nvalid of them before the end
    auto add_values = [&](uint32_t vt, int gr, const uint32_t (&pa)[4], const uint32_t (&pl)[4], int nvalid,
                          auto partial) {
#pragma unroll
      for (int c = 0; c < D / 16; c += 2) {
        // keys 0-7 and 8-15 of values 16 c .. 16 c + 15, then of the next 16
        const uint32_t key = gr * 16 + (lane & 15);
        const int cc = c + (lane >> 4);
        uint32_t addr;
        if constexpr (D == 64) addr = vt + sw128(key >> 1, (key & 1) * 4 + cc);
        else addr = vt + (c / 8) * kKeys * 128 + sw128(key, cc % 8);
        uint32_t v[4];
        ldmatrix_x4_trans(addr, v[0], v[1], v[2], v[3]);
        if constexpr (decltype(partial)::value) {
          // codes behind the last key may be anything (unfilled cache, e4m3 NaN):
          // their weight is 0 and so must the codes be
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k0 = 2 * tq + 8 * (i & 1);  // this register's keys: k0 (low half), k0 + 1
            v[i] &= (k0 < nvalid ? 0xffffu : 0u) | (k0 + 1 < nvalid ? 0xffff0000u : 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t e0, o0, e1, o1;
          codes_to_half_even_odd<kE4M3>(v[2 * i], e0, o0);
          codes_to_half_even_odd<kE4M3>(v[2 * i + 1], e1, o1);
          mma_16816<__half>(o[2 * (c + i)], pa, e0, e1);
          mma_16816<__half>(o[2 * (c + i) + 1], pa, o0, o1);
          if constexpr (kSplit) {
            mma_16816<__half>(o[2 * (c + i)], pl, e0, e1);
            mma_16816<__half>(o[2 * (c + i) + 1], pl, o0, o1);
          }
        }
      }
    };

    // the warp gives up as one: a lane whose limit expires takes the others along
    auto wait = [&](uint64_t* full, uint32_t phase) {
      return __all_sync(0xffffffffu, mbar_wait(full, phase, abort_flag, kErrKv8FullWait)) != 0;
    };
    int uk = 0, uv = 0;  // loads of K and of V read so far
    bool ok = true;
    for (int key0 = first; key0 < s1; key0 += kStride) {
      if (chunk_tile == 0) {
        // (an infinite scale becomes NaN: times a negative sum of codes it would be a
        // logit of -inf, a key without weight)
        ks_chunk = fmaf(ks_ahead, 0.f, ks_ahead);
        lv_chunk = __log2f(vs_ahead);  // -inf for a block of zeros
        fetch_scales(key0 + kChunk * kStride);
      }
      float f[kHalves][Cfg::kGroups], lv[Cfg::kGroups];
#pragma unroll
      for (int gr = 0; gr < Cfg::kGroups; ++gr) {
        const float ks = __shfl_sync(0xffffffffu, ks_chunk, chunk_tile * Cfg::kGroups + gr);
        lv[gr] = __shfl_sync(0xffffffffu, lv_chunk, chunk_tile * Cfg::kGroups + gr);
#pragma unroll
        for (int hr = 0; hr < kHalves; ++hr) f[hr][gr] = xs[hr] * ks;
      }
      chunk_tile = (chunk_tile + 1) % kChunk;

      // ---- S = Q K^T for 16 rows x kTileKeys keys
      float s[kNt][4];
#pragma unroll
      for (int ld = 0; ld < Cfg::kLoads; ++ld) {
        ok = ok && wait(&full_k[st_k], phase_k);
        if (!ok) continue;
        const uint8_t* kt = ring + st_k * Cfg::kStageBytes;
        constexpr int kN = kKeys / 8;              // n-tiles of a load
        constexpr int kChains = kN == 2 ? 2 : 1;   // with two n-tiles only, two chains of MMAs each
        float sc[kN][kChains][4];
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int i = 0; i < kChains; ++i) sc[nt][i][0] = sc[nt][i][1] = sc[nt][i][2] = sc[nt][i][3] = 0.f;
#pragma unroll
        for (int bx = 0; bx < Cfg::kBoxes; ++bx) {
#pragma unroll
          for (int half = 0; half < (D == 64 ? 1 : 2); ++half) {
            uint4 kw[kN];
#pragma unroll
            for (int nt = 0; nt < kN; ++nt) {
              const uint32_t key = nt * 8 + g;
              uint32_t off;
              if constexpr (D == 64) off = sw128(key >> 1, (key & 1) * 4 + tq);
              else off = bx * kKeys * 128 + sw128(key, 2 * tq + half);
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
              for (int nt = 0; nt < kN; ++nt) {
                const uint32_t w = i == 0 ? kw[nt].x : (i == 1 ? kw[nt].y : (i == 2 ? kw[nt].z : kw[nt].w));
                uint32_t b0, b1;
                codes_to_half<kE4M3>(w, b0, b1);
                mma_16816<__half>(sc[nt][i % kChains], aq, b0, b1);
              }
            }
          }
        }
        __syncwarp();  // the whole warp has read this load
        if (lane == 0 && uk + Cfg::kStages < nloads) load(uk + Cfg::kStages, st_k, &tmK, 0, full_k);
        ++uk;
        if (++st_k == Cfg::kStages) {
          st_k = 0;
          phase_k ^= 1u;
        }
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[ld * kN + nt][e] = sc[nt][0][e];
            if constexpr (kChains == 2) s[ld * kN + nt][e] += sc[nt][1][e];
          }
      }
      if (!ok) break;

      // ---- softmax (exp2 domain), rows g and g + 8
      const bool masked = key0 + kTileKeys > safe_end;  // the same for the whole warp
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 2 * kHalves; ++e)
            if (key0 + nt * 8 + 2 * tq + (e & 1) >= row_end[e >> 1]) s[nt][e] = -INFINITY;
      }
      if constexpr (kLogits) {
        // up to 16-key alignment the slots behind the last key are this warp's too
        // (nothing reads them); the capacity is a multiple of 16
#pragma unroll
        for (int hr = 0; hr < kHalves; ++hr) {
          if (lrow[hr] != nullptr) {
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
              if (key0 + nt / 2 * 16 < s1) {
                const float sa = s[nt][2 * hr], sb = s[nt][2 * hr + 1], fx = f[hr][nt / 2];
                *reinterpret_cast<float2*>(lrow[hr] + key0 + nt * 8 + 2 * tq) =
                    make_float2(masked && sa == -INFINITY ? sa : sa * fx, masked && sb == -INFINITY ? sb : sb * fx);
              }
          }
        }
      }
      // a row's largest x in one group of 16 keys, of this lane's (a rounded product of
      // its own, for m and for what is subtracted from it)
      auto top = [&](int hr, int gr) {
        return __fmul_rn(fmaxf(fmax3(s[2 * gr][2 * hr], s[2 * gr][2 * hr + 1], s[2 * gr + 1][2 * hr]), s[2 * gr + 1][2 * hr + 1]),
                         f[hr][gr]);
      };
      bool above = false;
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr) {
        float mx, vx;  // this lane's largest x - m, largest x - m + log2 vs
#pragma unroll
        for (int gr = 0; gr < Cfg::kGroups; ++gr) {
          const float x = top(hr, gr) - m[hr];
          mx = gr == 0 ? x : fmaxf(mx, x);
          vx = gr == 0 ? x + lv[gr] : fmaxf(vx, x + lv[gr]);
        }
        above = above || mx > kSlack || vx > d[hr] + (kSlack + kLift);
      }
      if (__any_sync(0xffffffffu, above)) {
        large = false;
#pragma unroll
        for (int hr = 0; hr < kHalves; ++hr) {
          float mn = m[hr], vn = kLowest;
#pragma unroll
          for (int gr = 0; gr < Cfg::kGroups; ++gr) mn = fmaxf(mn, top(hr, gr));
#pragma unroll
          for (int sh = 1; sh < 4; sh <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, sh));
#pragma unroll
          for (int gr = 0; gr < Cfg::kGroups; ++gr) vn = fmaxf(vn, top(hr, gr) - mn + lv[gr] - kLift);
#pragma unroll
          for (int sh = 1; sh < 4; sh <<= 1) vn = fmaxf(vn, __shfl_xor_sync(0xffffffffu, vn, sh));
          const float down = m[hr] - mn, was = d[hr] + down;
          vn = fmaxf(vn, was);
          lsum[hr] *= ex2_approx(down);
          const float al = ex2_approx(was - vn);
          m[hr] = mn;
          d[hr] = vn;
          large = large || (fabsf(mn) > kLarge && mn != kNone);
#pragma unroll
          for (int j = 0; j < Cfg::kTilesN; ++j) {
            o[j][2 * hr] *= al;
            o[j][2 * hr + 1] *= al;
            if constexpr (kLow) {
              o[j][2] *= al;
              o[j][3] *= al;
            }
          }
        }
        large = __any_sync(0xffffffffu, large);
      }
      uint32_t pa[Cfg::kGroups][4], pl[kSplit ? Cfg::kGroups : 1][4];
      if (masked || large) tile_weights<Cfg::kGroups, kHalves, true, kSplit, kLow>(s, f, lv, m, d, lsum, pa, pl);
      else tile_weights<Cfg::kGroups, kHalves, false, kSplit, kLow>(s, f, lv, m, d, lsum, pa, pl);

      // ---- O += P V
#pragma unroll
      for (int ld = 0; ld < Cfg::kLoads; ++ld) {
        ok = ok && wait(&full_v[st_v], phase_v);
        if (!ok) continue;
        const uint32_t vt = smem_u32(ring + st_v * Cfg::kStageBytes + Cfg::kTileBytes);
        const int key1 = key0 + ld * kKeys;
        if (key1 + kKeys <= s1) {
#pragma unroll
          for (int gr = 0; gr < kKeys / 16; ++gr) {
            const int at = ld * (kKeys / 16) + gr;
            add_values(vt, gr, pa[at], pl[kSplit ? at : 0], 16, std::false_type{});
          }
        } else {
#pragma unroll
          for (int gr = 0; gr < kKeys / 16; ++gr)
            if (key1 + 16 * gr < s1) {
              const int at = ld * (kKeys / 16) + gr;
              add_values(vt, gr, pa[at], pl[kSplit ? at : 0], s1 - key1 - 16 * gr, std::true_type{});
            }
        }
        __syncwarp();  // the whole warp has read this load
        if (lane == 0 && uv + Cfg::kStages < nloads) load(uv + Cfg::kStages, st_v, &tmV, 1, full_v);
        ++uv;
        if (++st_v == Cfg::kStages) {
          st_v = 0;
          phase_v ^= 1u;
        }
      }
      if (!ok) break;
    }
    if (uv < nloads && lane == 0) {
      // a wait gave up: let the loads already issued land before the shared memory goes away
      for (int u = seen + uk; u < seen + min(nloads, uk + Cfg::kStages); ++u)
        mbar_drain(&full_k[u % Cfg::kStages], (u / Cfg::kStages) & 1, 20000000ull);
      for (int u = seen + uv; u < seen + min(nloads, uv + Cfg::kStages); ++u)
        mbar_drain(&full_v[u % Cfg::kStages], (u / Cfg::kStages) & 1, 20000000ull);
    }

    seen += nloads;

    // ---- combine the four warps' states
    __syncthreads();
    if (*abort_flag != 0) return;
#pragma unroll
    for (int hr = 0; hr < kHalves; ++hr) {
      lsum[hr] += __shfl_xor_sync(0xffffffffu, lsum[hr], 1);
      lsum[hr] += __shfl_xor_sync(0xffffffffu, lsum[hr], 2);
    }
    float* cm = reinterpret_cast<float*>(smem);            // [4][16] running max
    float* cl = cm + kKv8Warps * kKv8Rows;                 // [4][16] sums
    float* cv = cl + kKv8Warps * kKv8Rows;                 // [4][16] O's units beside the maximum's
    float4* co4 = reinterpret_cast<float4*>(smem + 1024);  // [4][D / 16][2][32]: values 16 c + 4 tq ..+3 of rows g, g + 8
    if constexpr (kLow) {
#pragma unroll
      for (int j = 0; j < Cfg::kTilesN; ++j) {
        o[j][0] += o[j][2];
        o[j][1] += o[j][3];
      }
    }
    if (tq == 0) {
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr) {
        cm[warp * 16 + g + 8 * hr] = m[hr] == kNone ? -INFINITY : m[hr];
        cl[warp * 16 + g + 8 * hr] = lsum[hr];
        cv[warp * 16 + g + 8 * hr] = d[hr];
      }
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
#pragma unroll
      for (int hr = 0; hr < kHalves; ++hr)
        co4[((warp * (D / 16) + c) * 2 + hr) * 32 + lane] = make_float4(o[2 * c][2 * hr], o[2 * c + 1][2 * hr],
                                                                       o[2 * c][2 * hr + 1], o[2 * c + 1][2 * hr + 1]);
    }
    __syncthreads();

    // Per row: M = max_w m_w, L = sum_w 2^(m_w - M) l_w; O = sum_w 2^(m_w - M + d_w) O_w / L
    // (that power <= the largest vs: finite), LSE = M + log2 L.
    const int rows_here = min(kKv8Rows, rows_total - rg * kKv8Rows);
    const int64_t orow0 = (static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(hkv) * G) * a.Lq +
                          static_cast<int64_t>(rg) * kKv8Rows;
    const int64_t slot = (blockIdx.x + static_cast<int64_t>(b) * heads + uh) * kKv8Rows;
#pragma unroll
    for (int hr = 0; hr < kHalves; ++hr) {
      const int r = g + 8 * hr;
      if (r >= rows_here) break;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKv8Warps; ++w) M = fmaxf(M, cm[w * 16 + r]);
      float L = 0.f, wt[kKv8Warps];
#pragma unroll
      for (int w = 0; w < kKv8Warps; ++w) {
        const float mw = cm[w * 16 + r];
        // a warp whose maximum is -inf saw no key, or only NaN: its sum then says so
        L += mw == -INFINITY ? cl[w * 16 + r] : ex2_approx(mw - M) * cl[w * 16 + r];
        wt[w] = mw == -INFINITY ? 0.f : ex2_approx(mw - M + cv[w * 16 + r]);
      }
      const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
      for (int w = 0; w < kKv8Warps; ++w) wt[w] *= inv;
      if (warp == 0 && tq == 0) {
        const float lse = L == 0.f ? -INFINITY : M + __log2f(L);
        if (whole_unit) {
          if (a.lse != nullptr) a.lse[orow0 + r] = lse;
        } else {
          // a NaN partial is handed on as +inf: the merge's maximum would drop a
          // NaN and take the row for empty, while 2^(inf - inf) keeps it
          a.part_lse[slot + r] = isnan(lse) ? INFINITY : lse;
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16 / kKv8Warps; ++k) {
        const int c = warp + kKv8Warps * k;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kKv8Warps; ++w) {
          const float4 v = co4[((w * (D / 16) + c) * 2 + hr) * 32 + lane];
          acc.x = fmaf(wt[w], v.x, acc.x);
          acc.y = fmaf(wt[w], v.y, acc.y);
          acc.z = fmaf(wt[w], v.z, acc.z);
          acc.w = fmaf(wt[w], v.w, acc.w);
        }
        const int d = 16 * c + 4 * tq;
        if (whole_unit)
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (orow0 + r) * D + d) =
              make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
        else
          *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + d) = acc;
      }
    }
    // the next segment's loads may overwrite what the combine has just read and written
    fence_proxy_async_smem();
    __syncthreads();
  }
}

// Joins the partials of each row whose unit is divided: parts c0 + u .. c1 + u of
// unit u, M = max_p L_p, w_p = 2^(L_p - M), O = sum w_p O_p / sum w_p, LSE = M +
// log2 sum w_p.  One CTA takes 64 values of a row, its threads over columns and
// parts (a whole row of 256 left each thread 18 of 74 parts: 5 us instead of 2).
// Bound by latency: a launch, the LSEs, a few rounds of parts.
constexpr int kKv8MaxCtas = 1024;

template <int D, typename T>
__global__ void __launch_bounds__(256) kv8_merge_kernel(const Kv8DecodeArgs a, int ctas) {
  constexpr int kStride = Kv8DecodeCfg<D>::kCtaKeys;
  constexpr int kCols = 16;             // of four values
  constexpr int kLanes = 256 / kCols;   // threads of a column, each with every kLanes-th part
  constexpr int kFlight = 4;
  __shared__ float weight[kKv8MaxCtas];
  __shared__ float4 sums[256];
  __shared__ float red[16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, G = a.Hq / a.Hkv, heads = a.Hkv * a.row_groups;
  const int row = blockIdx.x;           // (b, h, i)
  const int h = row / a.Lq % a.Hq, b = row / a.Lq / a.Hq;
  const int r = h % G * a.Lq + row % a.Lq;  // of the kv head's rows
  const int uh = h / G * a.row_groups + r / kKv8Rows;
  uint32_t before, unit_places, total;
  if (a.kv_len == nullptr) {
    unit_places = static_cast<uint32_t>((a.capacity + kStride - 1) / kStride) + 1;
    before = b * unit_places;
    total = a.B * unit_places;
  } else {
    before = __ldg(a.table + b);
    unit_places = __ldg(a.table + b + 1) - before;
    total = __ldg(a.table + a.B);
  }
  if (unit_places == 0) return;         // no keys: written by the split kernel
  const Kv8Division division(total * heads, ctas);
  const uint32_t t0 = before * heads + uh * unit_places;
  const uint32_t c0 = division.owner(t0 + 1);
  const int parts = static_cast<int>(division.owner(t0 + unit_places - 1) - c0) + 1;
  if (parts == 1) return;               // whole: written by the split kernel
  const int64_t slot = (c0 + static_cast<int64_t>(b) * heads + uh) * kKv8Rows + r % kKv8Rows;
  const float* L = a.part_lse + slot;
  const int col = tid % kCols, lane = tid / kCols;
  const float4* O = reinterpret_cast<const float4*>(a.part_o + slot * D) + blockIdx.y * kCols + col;
  constexpr int64_t kStep = kKv8Rows * D / 4;  // float4s from one part to the next
  float4 x[kFlight];
#pragma unroll
  for (int i = 0; i < kFlight; ++i) {
    const int p = lane + i * kLanes;
    if (p < parts) x[i] = __ldg(O + p * kStep);
  }
  float top = -INFINITY;
  for (int p = tid; p < parts; p += 256) {
    const float v = __ldg(L + static_cast<int64_t>(p) * kKv8Rows);
    weight[p] = v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, red[i]);
  float sum = 0.f;
  for (int p = tid; p < parts; p += 256) {
    const float v = weight[p] == -INFINITY ? 0.f : ex2_approx(weight[p] - top);
    weight[p] = v;
    sum += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) red[8 + (tid >> 5)] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += red[8 + i];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = lane; p0 < parts; p0 += kFlight * kLanes) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int p = p0 + i * kLanes;
      if (p >= parts) break;
      const float v = weight[p];
      acc.x = fmaf(v, x[i].x, acc.x);
      acc.y = fmaf(v, x[i].y, acc.y);
      acc.z = fmaf(v, x[i].z, acc.z);
      acc.w = fmaf(v, x[i].w, acc.w);
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int p = p0 + (kFlight + i) * kLanes;
      if (p < parts) x[i] = __ldg(O + p * kStep);
    }
  }
  sums[tid] = acc;
  __syncthreads();
  if (tid < kCols) {
#pragma unroll
    for (int i = 1; i < kLanes; ++i) {
      const float4 v = sums[i * kCols + tid];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // every part empty: 0
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + static_cast<int64_t>(row) * D + (blockIdx.y * kCols + tid) * 4) =
        make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
    if (tid == 0 && blockIdx.y == 0 && a.lse != nullptr) a.lse[row] = sum == 0.f ? -INFINITY : top + __log2f(sum);
  }
}

// Attention weights of the keys: weights[b, h, j] += sum over the rows of kv
// head h of 2^(x_j - LSE), from the logits the split kernel left and the merged
// LSE (rows that see no key add nothing).  Bound by bytes: 4 per row and key,
// most of them still in L2, and 8 per key; with the logits' stores it adds 11 us
// to 31 us of decode (B = 2, 8 kv heads, 16 rows each, 32768 keys, int8).  A thread
// takes 4 keys, and kRows rows at a time in flight: 8, or 2 where a head has no
// more (more threads to an SM: one row, 16 heads, B = 16, 10000 keys: 79 us of
// decode against 84; with 16 rows, 8 are 44 against 46).
struct Kv8WeightArgs {
  const float* logits;   // [B, Hkv, rows, capacity]
  const float* lse;      // [B, Hkv, rows]
  float* weights;        // [B, Hkv, capacity]
  const int* kv_len;
  int Hkv, rows, capacity;
};

constexpr int kWeightThreads = 128;

template <int kRows>
__global__ void __launch_bounds__(kWeightThreads) kv8_weights_kernel(const Kv8WeightArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / a.Hkv);
  const int n = a.kv_len != nullptr ? min(max(__ldg(a.kv_len + b), 0), a.capacity) : a.capacity;
  const int j = (blockIdx.x * kWeightThreads + threadIdx.x) * 4;
  if (j >= n) return;
  const float* x = a.logits + bh * a.rows * a.capacity + j;
  const float* lse = a.lse + bh * a.rows;
  float* w = a.weights + bh * a.capacity + j;
  const bool four = j + 4 <= n;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f);  // what is there already, requested first
  if (four) old = *reinterpret_cast<const float4*>(w);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < a.rows; r0 += kRows) {
    float4 v[kRows];
    float L[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      L[i] = -INFINITY;
      if (r0 + i < a.rows) {
        L[i] = __ldg(lse + r0 + i);
        v[i] = *reinterpret_cast<const float4*>(x + static_cast<int64_t>(r0 + i) * a.capacity);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (L[i] == -INFINITY) continue;  // no visible key (or no such row)
      s[0] += ex2_approx(v[i].x - L[i]);
      s[1] += ex2_approx(v[i].y - L[i]);
      s[2] += ex2_approx(v[i].z - L[i]);
      s[3] += ex2_approx(v[i].w - L[i]);
    }
  }
  if (four) {
    *reinterpret_cast<float4*>(w) = make_float4(old.x + s[0], old.y + s[1], old.z + s[2], old.w + s[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < n) w[e] += s[e];
  }
}

}  // namespace skv
