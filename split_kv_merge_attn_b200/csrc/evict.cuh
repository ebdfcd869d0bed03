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
// -0 equal to +0) and the threshold is found 11, 11 and 10 bits at a time: a
// histogram of the candidates that share the bits found so far, then the bin in
// which the wanted rank falls.  (8 bits at a time took four such rounds, and had
// more lanes meet at a bin: weights of a head share few exponents.)  A head's
// tokens are divided over the CTAs of a cluster, which add what their bins hold to
// those of the first through distributed shared memory; that one finds the bin
// and tells the others.  (Every CTA reading all the others' bins instead moved 64 KB
// a round and CTA: 3.5 us a round against 0.9 us for a head of one CTA.)  Bound by
// the rounds' latency: a head's weights are a few bytes per clock.  Both kernels, D =
// 128, int8: 8 heads of 4096 to 1024 tokens 10.8 us (selection about 7); 64 heads of
// 32768 to 8192 68.7 us (selection 20).  Four copies of the first round's bins, so
// that lanes meet less often, changed neither.
#pragma once

#include "skv_device.cuh"
#include "kv8.cuh"

namespace skv {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;

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
  int B, Hkv, capacity, to_capacity, block_shift, budget, sink, recent;
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // >= 0x007fffff (that of -inf)
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
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// words of another CTA of the cluster, at the same shared address as `local`
__device__ __forceinline__ uint32_t cluster_address(const void* local, uint32_t rank) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
  return addr;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_address(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void add_cluster_u32(const uint32_t* local, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_address(local, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(const uint32_t* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_address(local, rank)), "r"(v) : "memory");
}

// One cluster per (batch entry, head); a lane holds up to kChunk keys at a time.
template <int kChunk>
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

  // this CTA's candidates, and this warp's (in order), in chunks of 32 * kChunk to a warp
  const int per_cta = ((hi - lo + static_cast<int>(parts) - 1) / static_cast<int>(parts) + 31) / 32 * 32;
  const int c0 = min(lo + static_cast<int>(rank) * per_cta, hi), c1 = min(c0 + per_cta, hi);
  const int per_warp = ((c1 - c0 + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int w0 = min(c0 + warp * per_warp, c1), w1 = min(w0 + per_warp, c1);
  // keys j, j + 32, ... of a chunk in a lane; 0 (below every weight's) behind the
  // end, where NaN is 1.  A warp of one chunk keeps it in registers.
  uint32_t key[kChunk];
  auto load = [&](int j) {
    float x[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) x[i] = j + 32 * i + lane < w1 ? __ldg(w + j + 32 * i + lane) : 0.f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) key[i] = j + 32 * i + lane < w1 ? weight_key(x[i]) : 0u;
  };
  const bool one_chunk = w1 - w0 <= 32 * kChunk;
  load(w0);

  constexpr int kRounds = 3;
  __shared__ uint4 hist4[kRounds][kEvictBins / 4];  // read by the whole cluster
  __shared__ uint32_t warp_sums[kRounds][kEvictWarps];
  __shared__ uint32_t found[kRounds][2];     // bin, candidates above it
  __shared__ uint32_t counts[2];             // this CTA's kept: above the threshold, equal to it
  __shared__ uint32_t warp_counts[2][kEvictWarps];

  uint32_t prefix = 0;
  uint32_t rest = static_cast<uint32_t>(wanted);  // still to take among those that share the prefix
  if (wanted > 0) {
    static_assert(kEvictBins == 4 * kEvictThreads, "a thread has four bins");
#pragma unroll
    for (int i = 0; i < kRounds; ++i) hist4[i][tid] = make_uint4(0, 0, 0, 0);
    if (parts > 1) cluster_barrier();  // the first CTA's bins are clear before others add to them
    else __syncthreads();
#pragma unroll 1
    for (int round = 0; round < kRounds; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0), bits = round == 2 ? 10 : 11;
      uint32_t* hist = reinterpret_cast<uint32_t*>(hist4[round]);
      for (int j = w0; j < w1; j += 32 * kChunk) {
        if (!one_chunk) load(j);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const uint32_t k = key[i];
          if (k != 0 && (round == 0 || ((k ^ prefix) >> (shift + bits)) == 0))
            atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
        }
      }
      __syncthreads();
      if (parts > 1) {
        if (rank != 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // (lanes beside each other add to neighbouring bins)
            const uint32_t c = hist[tid + i * kEvictThreads];
            if (c != 0) add_cluster_u32(hist + tid + i * kEvictThreads, 0, c);
          }
        }
        cluster_barrier();
      }
      if (rank == 0) {
        // bins from the top: thread t has 2047 - 4 t (t[0]) .. 2044 - 4 t (t[3])
        const uint4 v = hist4[round][kEvictThreads - 1 - tid];
        const uint32_t t[4] = {v.w, v.z, v.y, v.x};
        const uint32_t mine = t[0] + t[1] + t[2] + t[3];
        uint32_t before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        if (lane == 31) warp_sums[round][warp] = before;
        __syncthreads();
        before -= mine;  // candidates in higher bins
#pragma unroll
        for (int i = 0; i < kEvictWarps; ++i) before += i < warp ? warp_sums[round][i] : 0u;
        if (before < rest && before + mine >= rest) {
          uint32_t above = before;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (above < rest && above + t[i] >= rest) {
              const uint32_t bin = static_cast<uint32_t>(kEvictBins - 1 - 4 * tid - i);
              for (uint32_t r = 0; r < parts; ++r) {
                st_cluster_u32(&found[round][0], r, bin);
                st_cluster_u32(&found[round][1], r, above);
              }
            }
            above += t[i];
          }
        }
      }
      if (parts > 1) cluster_barrier();
      else __syncthreads();
      prefix |= found[round][0] << shift;
      rest -= found[round][1];
    }
  }
  const uint32_t threshold = prefix;
  // kept candidates: key > threshold, and the first `rest` of those equal to it
  uint32_t above = 0, equal = 0;
  if (wanted > 0) {
    for (int j = w0; j < w1; j += 32 * kChunk) {
      if (!one_chunk) load(j);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        above += key[i] > threshold;
        equal += key[i] == threshold;
      }
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
    uint32_t t = 0;
    for (int i = 0; i < kEvictWarps; ++i) t += warp_counts[tid][i];
    counts[tid] = t;
  }
  if (parts > 1) cluster_barrier();
  uint32_t place = 0, seen = 0;  // candidates above / equal before this warp's
#pragma unroll
  for (uint32_t r = 0; r < 7; ++r) {
    if (r < rank) {
      place += ld_cluster_u32(&counts[0], r);
      seen += ld_cluster_u32(&counts[1], r);
    }
  }
  if (parts > 1) cluster_barrier();  // nobody leaves while its counts or histograms may be read
  for (int i = 0; i < warp; ++i) {
    place += warp_counts[0][i];
    seen += warp_counts[1][i];
  }
  if (wanted > 0) {
    // place: candidates kept before this one
    place += min(seen, rest);
    const uint32_t below = (1u << lane) - 1u;
    for (int j = w0; j < w1; j += 32 * kChunk) {
      if (!one_chunk) load(j);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const bool eq = key[i] == threshold;
        const uint32_t eq_mask = __ballot_sync(0xffffffffu, eq);
        const bool take = key[i] > threshold || (eq && seen + __popc(eq_mask & below) < rest);
        const uint32_t mask = __ballot_sync(0xffffffffu, take);
        if (take) kept[a.sink + static_cast<int>(place) + __popc(mask & below)] = j + 32 * i + lane;
        place += __popc(mask);
        seen += __popc(eq_mask);
      }
    }
  }
  for (int i = static_cast<int>(rank) * kEvictThreads + tid; i < a.sink; i += kEvictThreads * static_cast<int>(parts)) kept[i] = i;
  for (int i = static_cast<int>(rank) * kEvictThreads + tid; i < a.recent; i += kEvictThreads * static_cast<int>(parts))
    kept[a.sink + wanted + i] = hi + i;
}

// Compaction: one warp per 16 kept tokens of one (batch entry, head), K and V;
// blocks larger than 16 tokens share their scale through shared memory.
// Bound by bytes: the kept tokens' codes in and out.  The codes are requested
// before the scales are known, all of a warp's at once.  64 heads, 8192 tokens
// kept of 32768, D = 128, int8: 49 us for 268 MB (5.5 TB/s; nearly every token is
// rescaled to its new block).
template <int D, bool kE4M3>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  using Code = Kv8Code<kE4M3>;
  constexpr int kUnits = D / 16;              // 16-byte pieces of a row
  constexpr int kIters = 16 * kUnits / 32;    // pieces a lane moves of K, and of V
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
  uint4 v[2][kIters];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int t = (i * 32 + lane) / kUnits, c = (i * 32 + lane) % kUnits;
      const int f = __shfl_sync(0xffffffffu, from, t);
      v[which][i] = make_uint4(0, 0, 0, 0);
      if (f >= 0) v[which][i] = __ldg(reinterpret_cast<const uint4*>(a.codes[which] + (bh * a.capacity + f) * D) + c);
    }
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
  const int live = total - (base + warp * 16);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const float i1 = __shfl_sync(0xffffffffu, inv, which * 16);
    const uint64_t si = f2_pack(i1, i1);
    const float sb = __shfl_sync(0xffffffffu, s, which * 16);
    uint4* dst = reinterpret_cast<uint4*>(a.to_codes[which] + (bh * a.to_capacity + base + warp * 16) * D);
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int t = (i * 32 + lane) / kUnits;
      const float st = __shfl_sync(0xffffffffu, s_tok, which * 16 + t);
      uint4 w = v[which][i];
      if (st != sb) {
        const bool good = sb < INFINITY;
        w.x = good ? Code::recode4(w.x, st, si) : 0u;
        w.y = good ? Code::recode4(w.y, st, si) : 0u;
        w.z = good ? Code::recode4(w.z, st, si) : 0u;
        w.w = good ? Code::recode4(w.w, st, si) : 0u;
      }
      if (t < live) dst[i * 32 + lane] = w;
    }
  }
}

}  // namespace skv
