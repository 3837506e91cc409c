// moe_layout.cuh -- device code of the expert layouts: which row each routed
// slot takes.  Routed row r = t * topk + k goes to expert e[r] (-1: dropped);
// an expert's rows keep their order r.
//
// One cluster does the whole count -> scan -> rank chain: the slots are split
// into one contiguous run per CTA and, inside it, one per warp.  A first walk
// counts each warp's slots per expert (a ballot per bit of the expert finds the
// lanes of one expert; the lowest adds their number to a counter that only its
// warp uses), the warps' counters are scanned in shared memory and the CTAs'
// totals through distributed shared memory, and a second walk hands out the
// rows.  Everything is integer work in a fixed order: ranks are stable.
//
// It is a chain of latencies, not of work: each walk loads up to 8 steps of 32
// slots at once, a warp's first 8 steps stay in registers for the second walk,
// and the scan over the warps reads all its counters before it adds
// (32768 slots, 64 experts: 9 us on cold caches).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fp8gemm.h"
#include "ptx.cuh"

namespace fp8g {
namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopk = 16;
constexpr int kLayoutThreads = 1024;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kMaxCtas = 8;  // of the layout kernel's cluster
constexpr int kAhead = 8;  // steps of 32 slots that a warp loads at once

// Expert of routed row r, or -1 (dropped, or out of range: flagged).
__device__ __forceinline__ int expert_at(const int32_t* e, int G, long r, uint32_t* err) {
  const int g = __ldg(e + r);
  if (g < G && g >= -1) return g;
  if (err) atomicOr(err, FP8G_DEVERR_BAD_EXPERT);
  return -1;
}

// The lanes with the same expert g as this one (of no use to lanes with g < 0),
// from one ballot per bit.  __match_any_sync gives the same, but took 90 cycles
// of the SM for every warp and step: 12.9 us for 32768 slots over 64 experts.
__device__ __forceinline__ uint32_t peers_of(int g, int bits) {
  uint32_t m = __ballot_sync(0xffffffffu, g >= 0);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    if (b >= bits) break;
    const bool one = g >> b & 1;
    const uint32_t with = __ballot_sync(0xffffffffu, one);
    m &= one ? with : ~with;
  }
  return m;
}

// Earlier slots of each of a token's experts e[k], counted by the warps of a CTA
// (a share of the slots before `before` each): s_part[warp][k].  Slots of the
// token itself count by the first warp.  A barrier has to follow.
template <int kCap, int kThreads = 0>
__device__ __forceinline__ void count_earlier(const int32_t* expert, int before, const int (&e)[kCap],
                                              int32_t (*s_part)[kCap]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = kThreads ? kThreads : blockDim.x;
  int n[kCap];
#pragma unroll
  for (int k = 0; k < kCap; ++k) n[k] = 0;
  for (int r0 = 32 * warp; r0 < before; r0 += kAhead * threads) {
    int g[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * threads + lane;
      g[a] = r < before ? __ldg(expert + r) : -1;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (r0 + a * threads >= before) break;  // warp-uniform
#pragma unroll
      for (int k = 0; k < kCap; ++k) n[k] += __popc(__ballot_sync(0xffffffffu, g[a] == e[k]));
    }
  }
#pragma unroll
  for (int k = 0; k < kCap; ++k) {
#pragma unroll
    for (int a = 0; a < k; ++a) n[k] += warp == 0 && e[a] == e[k];  // the same expert twice in a token
    if (lane == k) s_part[warp][k] = n[k];
  }
}

// Slots of every expert, counted by a CTA into s_cnt [kMaxExperts]; flags bad
// experts if err is given.  Starts and ends with a barrier.
template <int kThreads = 0>
__device__ __forceinline__ void count_experts(const int32_t* expert, int R, int G, int32_t* s_cnt, uint32_t* err) {
  const int threads = kThreads ? kThreads : blockDim.x;
  for (int g = threadIdx.x; g < kMaxExperts; g += threads) s_cnt[g] = 0;
  __syncthreads();
  for (int r0 = threadIdx.x; r0 < R; r0 += kAhead * threads) {
    int g[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) g[a] = r0 + a * threads < R ? expert_at(expert, G, r0 + a * threads, err) : -1;
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (g[a] >= 0) atomicAdd(&s_cnt[g[a]], 1);
  }
  __syncthreads();
}

__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// A used block of the contiguous layout as the layout kernel leaves it for the
// kernel that moves the rows: its expert and its filled rows (1 to 128).  That
// kernel's padding CTAs count themselves in the bits above (kBlockArrival) and the
// last one leaves the expert alone.
constexpr int32_t kBlockArrival = 1 << 16;
__device__ __forceinline__ int32_t block_entry(int g, int filled) { return g | filled << 8; }
__device__ __forceinline__ int block_expert(int32_t entry) { return entry & 0xFF; }
__device__ __forceinline__ int block_filled(int32_t entry) { return entry >> 8 & 0xFF; }
__device__ __forceinline__ int block_arrivals(int32_t entry) { return entry >> 16; }

// kMasked: pos[r] = g * Mmax + rank, -1 at and behind Mmax; counts[g] =
// min(rows of g, Mmax).  Otherwise the contiguous layout: pos[r] = first row
// of g's segment + rank, segments padded to 128 rows; counts [blocks] = a
// block_entry, -1 for an unused block.  Launched as one cluster of 1 to 8 CTAs.
template <bool kMasked>
__global__ void __launch_bounds__(kLayoutThreads) moe_layout_kernel(const int32_t* __restrict__ expert, int R, int G,
                                                                    int Mmax, int32_t* __restrict__ pos,
                                                                    int32_t* __restrict__ counts, int blocks,
                                                                    uint32_t* err) {
  __shared__ int32_t s_w[kLayoutWarps][kMaxExperts];  // per warp: slots of each expert, then the warp's next rank
  __shared__ int32_t s_total[kMaxExperts];            // this CTA's slots of each expert (read by the cluster)
  __shared__ int32_t s_first[kMaxExperts];            // first row that this CTA hands out for each expert
  __shared__ int32_t s_end[kMaxExperts];              // contiguous: end of each segment in blocks,
  __shared__ int32_t s_rows[kMaxExperts];             // and its rows
  __shared__ int32_t s_warp[kMaxExperts / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  if (tid == 0) grid_launch_dependents();  // the kernel that moves the rows may take its place; it waits for this one
  for (int g = lane; g < G; g += 32) s_w[w][g] = 0;
  __syncwarp();
  // rows of this warp: whole steps of 32 slots
  const long steps = (static_cast<long>(R) + 32L * kLayoutWarps * ctas - 1) / (32L * kLayoutWarps * ctas);
  const long r0 = (static_cast<long>(rank) * kLayoutWarps + w) * steps * 32 + lane;
  int g[kAhead];
  uint32_t peers[kAhead];
  auto load = [&](long i0, uint32_t* flag) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const long r = r0 + 32 * (i0 + i);
      g[i] = i0 + i < steps && r < R ? expert_at(expert, G, r, flag) : -1;
    }
  };
  const uint32_t below = (1u << lane) - 1u;
  const int bits = G > 1 ? 32 - __clz(G - 1) : 0;  // of an expert's number
  for (long i0 = 0; i0 < steps; i0 += kAhead) {
    load(i0, err);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= steps) break;  // the same for the whole CTA
      peers[i] = peers_of(g[i], bits);
      if (g[i] >= 0 && (peers[i] & below) == 0) s_w[w][g[i]] += __popc(peers[i]);
      __syncwarp();
    }
  }
  __syncthreads();
  if (tid < kMaxExperts) {
    int32_t v[kLayoutWarps], run = 0;
#pragma unroll
    for (int ww = 0; ww < kLayoutWarps; ++ww) v[ww] = tid < G ? s_w[ww][tid] : 0;
#pragma unroll
    for (int ww = 0; ww < kLayoutWarps; ++ww) {
      if (tid < G) s_w[ww][tid] = run;
      run += v[ww];
    }
    s_total[tid] = run;
  }
  if (ctas > 1) cluster_sync_all();
  else __syncthreads();
  int32_t before = 0, total = 0;
  if (tid < kMaxExperts) {
    const uint32_t mine = smem_u32(&s_total[tid]);
    int32_t v[kMaxCtas];
#pragma unroll
    for (int c = 0; c < kMaxCtas; ++c) v[c] = c < ctas ? ld_cluster_s32(mapa(mine, c)) : 0;
#pragma unroll
    for (int c = 0; c < kMaxCtas; ++c) {
      if (c < rank) before += v[c];
      total += v[c];
    }
  }
  // No CTA leaves while another may still read its totals: arrive here, where they
  // have been read and before the stores of pos (which a release would wait for),
  // wait at the end.
  if (ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if constexpr (kMasked) {
    if (tid < kMaxExperts) s_first[tid] = before;
    if (rank == 0 && tid < G) {
      counts[tid] = min(total, Mmax);
      if (total > Mmax) atomicOr(err, FP8G_DEVERR_MASKED_OVER);
    }
    __syncthreads();
  } else {
    // inclusive scan of the segments' blocks over the experts (8 warps)
    const int32_t nblk = (total + 127) / 128;
    int32_t incl = nblk;
    if (tid < kMaxExperts) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (lane == 31) s_warp[w] = incl;
    }
    __syncthreads();
    if (tid < kMaxExperts) {
      for (int i = 0; i < w; ++i) incl += s_warp[i];
      s_end[tid] = incl;
      s_rows[tid] = total;
      s_first[tid] = (incl - nblk) * 128 + before;
    }
    __syncthreads();
    for (int b = rank * kLayoutThreads + tid; b < blocks; b += ctas * kLayoutThreads) {
      // the first expert whose segment ends behind block b
      int lo = 0, hi = G;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_end[mid] > b) hi = mid;
        else lo = mid + 1;
      }
      // only a segment's last block is not full
      counts[b] = lo < G ? block_entry(lo, b + 1 < s_end[lo] ? 128 : (s_rows[lo] - 1) % 128 + 1) : -1;
    }
  }
  for (long i0 = 0; i0 < steps; i0 += kAhead) {
    if (steps > kAhead) load(i0, nullptr);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= steps) break;
      const long r = r0 + 32 * (i0 + i);
      if (steps > kAhead) peers[i] = peers_of(g[i], bits);
      int32_t row = -1;
      if (g[i] >= 0) {
        row = s_first[g[i]] + s_w[w][g[i]] + __popc(peers[i] & below);
        if constexpr (kMasked) row = row < Mmax ? g[i] * Mmax + row : -1;
      }
      __syncwarp();
      if (g[i] >= 0 && (peers[i] & below) == 0) s_w[w][g[i]] += __popc(peers[i]);
      __syncwarp();
      if (r < R) pos[r] = row;
    }
  }
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster of up to 8 CTAs, a CTA for every 4096 slots.
template <bool kMasked>
cudaError_t launch_layout(const int32_t* expert, int R, int G, int Mmax, int32_t* pos, int32_t* counts, int blocks,
                          uint32_t* err, cudaStream_t stream) {
  int ctas = 1;
  while (ctas < kMaxCtas && R > 4096 * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kLayoutThreads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, moe_layout_kernel<kMasked>, expert, R, G, Mmax, pos, counts, blocks, err);
}

}  // namespace moe
}  // namespace fp8g
