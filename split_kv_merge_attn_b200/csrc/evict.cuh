// Eviction from the 8-bit cache by accumulated attention weight.
//
// Of the first n = kv_len[b] tokens of each head, keep the first `sink`, the
// last `recent` and, of those between, the heaviest budget - sink - recent
// (equal weights: the lowest position); if n <= budget, all.  The kept tokens
// move in order into another cache.  A block of that cache gets the largest of
// its tokens' scales s_j as its scale s, and its codes rne((c * s_j) * (1 / s)):
// a token whose scale is the block's keeps its codes.
//
// Selection: weights map to whole numbers of the same order (NaN below all,
// -0 equal to +0) and the threshold is found 8 bits at a time: a histogram of
// the candidates that share the bits found so far, then the bin in which the
// wanted rank falls.  A head's tokens are divided over the CTAs of a cluster,
// which add up their histograms through distributed shared memory.
#pragma once

#include "skv_device.cuh"
#include "kv8.cuh"

namespace skv {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 256;

struct EvictArgs {
  const float* weights;      // [B, Hkv, capacity]
  const int32_t* kv_len;     // [B] or null (= capacity)
  int32_t* kept;             // [B, Hkv, budget]
  int32_t* new_len;          // [B]
  const uint8_t* codes[2];
  const float* scale[2];
  uint8_t* to_codes[2];
  float* to_scale[2];
  float* to_weights;         // [B, Hkv, to_capacity]
  int B, Hkv, D, capacity, to_capacity, block_shift, budget, sink, recent;
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // >= 0x007fffff for -inf
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a 32-bit word of another CTA of the cluster, at the same shared address as `local`
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* local, uint32_t rank) {
  uint32_t addr, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// One cluster per (batch entry, head).
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const EvictArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t rank = cluster_ctarank(), parts = cluster_nctarank();
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / a.Hkv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.kv_len != nullptr ? min(max(a.kv_len[b], 0), a.capacity) : a.capacity;
  const int total = min(n, a.budget);
  int32_t* kept = a.kept + bh * a.budget;
  if (bh % a.Hkv == 0 && rank == 0 && tid == 0) a.new_len[b] = total;
  for (int i = total + static_cast<int>(rank) * kEvictThreads + tid; i < a.budget; i += kEvictThreads * static_cast<int>(parts))
    kept[i] = -1;
  if (n <= a.budget) {  // the whole cluster: nothing to choose
    for (int i = static_cast<int>(rank) * kEvictThreads + tid; i < n; i += kEvictThreads * static_cast<int>(parts)) kept[i] = i;
    return;
  }
  // candidates lie in [sink, n - recent); n > budget >= sink + recent
  const int lo = a.sink, hi = n - a.recent;
  const int wanted = a.budget - a.sink - a.recent;
  const float* w = a.weights + bh * a.capacity;

  // this CTA's candidates, and this warp's (in order, whole warps of 32)
  const int per_cta = ((hi - lo + static_cast<int>(parts) - 1) / static_cast<int>(parts) + 31) / 32 * 32;
  const int c0 = min(lo + static_cast<int>(rank) * per_cta, hi), c1 = min(c0 + per_cta, hi);
  const int per_warp = ((c1 - c0 + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int w0 = min(c0 + warp * per_warp, c1), w1 = min(w0 + per_warp, c1);

  __shared__ uint32_t hist[kEvictBins];      // read by the whole cluster
  __shared__ uint32_t sums[kEvictBins];      // the cluster's histogram
  __shared__ uint32_t found[2];              // bin, candidates above it
  __shared__ uint32_t counts[2];             // this CTA's kept: above the threshold, equal to it
  __shared__ uint32_t warp_counts[2][kEvictWarps];

  uint32_t prefix = 0;
  uint32_t rest = static_cast<uint32_t>(wanted);  // still to take among those that share the prefix
  if (wanted > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
      for (int j = c0 + tid; j < c1; j += kEvictThreads) {
        const uint32_t k = weight_key(__ldg(w + j));
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      cluster_barrier();
      if (tid < kEvictBins) {
        uint32_t s = 0;
        for (uint32_t r = 0; r < parts; ++r) s += ld_cluster_u32(&hist[tid], r);
        sums[tid] = s;
      }
      cluster_barrier();  // every CTA has read the histograms before they are cleared
      if (warp == 0) {
        // lane l holds bins 255 - 8 l .. 248 - 8 l, from the top
        uint32_t s[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[i] = sums[255 - 8 * lane - i];
          mine += s[i];
        }
        uint32_t before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        before -= mine;  // candidates in higher bins
        if (before < rest && before + mine >= rest) {
          uint32_t above = before;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (above < rest && above + s[i] >= rest) {
              found[0] = static_cast<uint32_t>(255 - 8 * lane - i);
              found[1] = above;
            }
            above += s[i];
          }
        }
      }
      __syncthreads();
      prefix |= found[0] << shift;
      rest -= found[1];
      __syncthreads();
    }
  }
  const uint32_t threshold = prefix;
  // kept candidates: key > threshold, and the first `rest` of those equal to it
  uint32_t above = 0, equal = 0;
  if (wanted > 0) {
    for (int j = w0 + lane; j < w1; j += 32) {
      const uint32_t k = weight_key(__ldg(w + j));
      above += k > threshold;
      equal += k == threshold;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
  }
  if (lane == 0) {
    warp_counts[0][warp] = above;
    warp_counts[1][warp] = equal;
  }
  __syncthreads();
  if (tid < 2) {
    uint32_t s = 0;
    for (int i = 0; i < kEvictWarps; ++i) s += warp_counts[tid][i];
    counts[tid] = s;
  }
  cluster_barrier();
  uint32_t place = 0, seen = 0;  // candidates above / equal before this warp's
  for (uint32_t r = 0; r < rank; ++r) {
    place += ld_cluster_u32(&counts[0], r);
    seen += ld_cluster_u32(&counts[1], r);
  }
  cluster_barrier();  // nobody leaves while its counts may be read
  for (int i = 0; i < warp; ++i) {
    place += warp_counts[0][i];
    seen += warp_counts[1][i];
  }
  if (wanted > 0) {
    // place: candidates kept before this one
    place += min(seen, rest);
    for (int j = w0; j < w1; j += 32) {
      const int jj = j + lane;
      const uint32_t k = jj < w1 ? weight_key(__ldg(w + jj)) : 0u;
      const bool eq = jj < w1 && k == threshold;
      const uint32_t eq_mask = __ballot_sync(0xffffffffu, eq);
      const uint32_t below = (1u << lane) - 1u;
      const bool take = (jj < w1 && k > threshold) || (eq && seen + __popc(eq_mask & below) < rest);
      const uint32_t mask = __ballot_sync(0xffffffffu, take);
      if (take) kept[a.sink + static_cast<int>(place) + __popc(mask & below)] = jj;
      place += __popc(mask);
      seen += __popc(eq_mask);
    }
  }
  for (int i = static_cast<int>(rank) * kEvictThreads + tid; i < a.sink; i += kEvictThreads * static_cast<int>(parts)) kept[i] = i;
  for (int i = static_cast<int>(rank) * kEvictThreads + tid; i < a.recent; i += kEvictThreads * static_cast<int>(parts))
    kept[a.sink + wanted + i] = hi + i;
}

// Compaction: one warp per 16 kept tokens of one (batch entry, head), K and V;
// blocks larger than 16 tokens share their scale through shared memory.
// Bound by bytes: the kept tokens' codes in and out.
template <bool kE4M3>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  using Code = Kv8Code<kE4M3>;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = min(a.kv_len != nullptr ? min(max(a.kv_len[b], 0), a.capacity) : a.capacity, a.budget);
  const int base = blockIdx.x * kKv8Window;
  if (base >= total) return;
  const int32_t* kept = a.kept + bh * a.budget;
  const int pos = base + warp * 16 + (lane & 15);
  const int from = pos < total ? kept[pos] : -1;
  const int which_lane = lane >> 4;  // lanes 0-15: K's scales, 16-31: V's
  const float* scale = a.scale[which_lane] + bh * (a.capacity >> a.block_shift);
  const float s_tok = from >= 0 ? scale[from >> a.block_shift] : 0.f;
  // magnitude bits: scales are >= 0, and NaN must win
  uint32_t top = __float_as_uint(s_tok) & 0x7fffffffu;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  __shared__ uint32_t tops[8][2];
  if ((lane & 15) == 0) tops[warp][which_lane] = top;
  __syncthreads();
  const int per = (1 << a.block_shift) >> 4;
  const int first = warp / per * per;
  for (int i = first; i < first + per; ++i) top = max(top, tops[i][which_lane]);
  float s = __uint_as_float(top);
  if (s < kKv8TinyScale) s = 0.f;
  const int64_t to_blocks = a.to_capacity >> a.block_shift;
  const int block_pos = base + first * 16;
  if (warp == first && (lane & 15) == 0 && block_pos < total)
    a.to_scale[which_lane][bh * to_blocks + (block_pos >> a.block_shift)] = s;
  if (lane < 16 && from >= 0) a.to_weights[bh * a.to_capacity + pos] = a.weights[bh * a.capacity + from];
  const float inv = kv8_inverse(s);
  const int words = a.D >> 4;  // 16-byte pieces of a row
  const int live = min(16, total - (base + warp * 16));
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const float si = __shfl_sync(0xffffffffu, inv, which * 16);
    const float sb = __shfl_sync(0xffffffffu, s, which * 16);
    const uint8_t* src = a.codes[which] + bh * a.capacity * a.D;
    uint8_t* dst = a.to_codes[which] + (bh * a.to_capacity + base + warp * 16) * a.D;
    for (int i0 = 0; i0 < 16 * words; i0 += 32) {  // 16 * words is a multiple of 32: whole warps
      const int i = i0 + lane;
      const int t = i / words, c = i - t * words;
      const int f = __shfl_sync(0xffffffffu, from, t);
      const float st = __shfl_sync(0xffffffffu, s_tok, which * 16 + t);
      if (t >= live) continue;
      uint4 v = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(f) * a.D + c * 16);
      if (st != sb) {
        uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[4];
          Code::decode4(u[e], x);
#pragma unroll
          for (int d = 0; d < 4; ++d) x[d] = __fmul_rn(__fmul_rn(x[d], st), si);
          u[e] = sb < INFINITY ? Code::encode4(x[0], x[1], x[2], x[3]) : 0u;
        }
        v = make_uint4(u[0], u[1], u[2], u[3]);
      }
      *reinterpret_cast<uint4*>(dst + t * a.D + c * 16) = v;
    }
  }
}

}  // namespace skv
