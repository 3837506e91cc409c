// moe_grad.cu -- the expert sort of unquantised rows, its gradient, and the
// gradient of the weighted combine, sm_100a.
//
//   permute            xs[pos[r]] = x[r / topk], padding rows zero
//   permute backward   dx[t] = sum_k dxs[pos[t topk + k]]
//   combine backward   of out[t] = sum_k w[r] D[pos[r]]:
//                      dD[pos[r]] = w[r] dout[t], dw[r] = <dout[t], D[pos[r]]>
//
// All three are HBM-bound streams.  A CTA takes a token (several, where rows are
// narrow and tokens many): its row of x or dout is read once for all of its
// slots, and every row of the layout is touched once.  Positions are checked against the layout's rows before any access; a
// position outside is flagged and its slot skipped.
//
// Padding rows.  The rows of a used block (one that holds a routed row) that
// no slot fills are set to zero by CTAs of their own in the same launch, each
// with a share of the rows of a run of blocks.  The sort learns from its layout how
// many rows of each block are filled: until its last padding CTA has seen it, a
// block's entry of m_indices holds that number too.  The combine's gradient
// has only pos: its padding CTAs mark the rows that pos names in a bitmap in
// shared memory.  Reading pos (4 bytes a slot) once per such CTA costs little
// next to rows of some thousand columns, and saves the workspace, the launches
// and the atomics on memory that a map from rows to slots would need.
//
// Times in this file: calls back to back as a program makes them, into outputs of
// their own and for long enough that the power cap acts; "replayed" means the
// same calls in a short CUDA graph at full clock, whose outputs stay in L2 in part.
// Comparisons of two forms are replayed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8gemm.h"
#include "moe_layout.cuh"
#include "quant8.cuh"
#include "rows.cuh"

namespace {

using namespace fp8g::rows;
using fp8g::moe::kMaxExperts;
using fp8g::moe::kMaxTopk;

constexpr int kPadBlocks = 256;  // most blocks of a padding CTA: its bitmap is 4 KB
// CTAs that share a group of blocks, each with every 8th of its rows: one SM
// alone zeroes 370 KB (45 rows of 4096 bf16) in some 15 us
constexpr int kPadSlices = 8;
// Routed slots up to which the sort may be one launch, while its CTAs are few
// enough to run at once (999 slots of 2112 FP32: 7.4 us against 8.0 with the
// layout kernel, and one launch on the host).
constexpr int kDirectSlots = 4096;

// A slot's position if it names a row of the layout, -1 if the slot is dropped;
// anything else is flagged and treated as dropped.
__device__ __forceinline__ int checked_pos(int p, int M, uint32_t* err) {
  if (p >= -1 && p < M) return p;
  atomicOr(err, FP8G_DEVERR_BAD_POS);
  return -1;
}

// Calls zero_row(row) for a share of the rows of blocks [b0, b1) that no slot
// fills, in blocks with at least one filled row: every kPadSlices-th row, from
// `slice` on.  All threads of the CTA call it; a warp takes a row at a time.
template <typename ZeroRow>
__device__ __forceinline__ void pad_blocks(const int32_t* __restrict__ pos, long R, int b0, int b1, int slice,
                                           uint32_t* bits, uint32_t* err, ZeroRow zero_row) {
  const int words = (b1 - b0) * 4;
  for (int i = threadIdx.x; i < words; i += blockDim.x) bits[i] = 0u;
  __syncthreads();
  const int lo = b0 * 128, n = (b1 - b0) * 128;
  auto mark = [&](int p) {
    const uint32_t i = static_cast<uint32_t>(p - lo);
    if (i < static_cast<uint32_t>(n) && (atomicOr(&bits[i >> 5], 1u << (i & 31)) >> (i & 31) & 1u))
      atomicOr(err, FP8G_DEVERR_BAD_POS);  // two slots in one row
  };
  // scalar loads up to the first 16-byte boundary, then four slots a load
  const long head = min(R, static_cast<long>((16 - (reinterpret_cast<uintptr_t>(pos) & 15)) & 15) / 4);
  if (threadIdx.x < head) mark(__ldg(pos + threadIdx.x));
  const int4* p4 = reinterpret_cast<const int4*>(pos + head);
  const long quads = (R - head) / 4;
  for (long i0 = threadIdx.x; i0 < quads; i0 += 4L * blockDim.x) {
    int4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long at = i0 + static_cast<long>(i) * blockDim.x;
      v[i] = at < quads ? __ldg(p4 + at) : make_int4(-1, -1, -1, -1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) mark(v[i].x), mark(v[i].y), mark(v[i].z), mark(v[i].w);
  }
  const long tail = head + 4 * quads + threadIdx.x;
  if (tail < R) mark(__ldg(pos + tail));
  __syncthreads();
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  for (int i = slice + kPadSlices * w; i < n; i += kPadSlices * nw) {
    const uint32_t* blk = bits + (i >> 7) * 4;
    if (!(blk[0] | blk[1] | blk[2] | blk[3])) continue;  // an unused block
    if (bits[i >> 5] >> (i & 31) & 1u) continue;
    zero_row(static_cast<long>(lo + i));
  }
}

// Blocks of padding CTA `cta` of `pads`: groups of blocks, kPadSlices CTAs each.
__device__ __forceinline__ void pad_range(int cta, int pads, int blocks, int& b0, int& b1, int& slice) {
  const int groups = pads / kPadSlices, per = (blocks + groups - 1) / groups;
  slice = cta % kPadSlices;
  b0 = min(blocks, cta / kPadSlices * per);
  b1 = min(blocks, b0 + per);
}

// ---------------------------------------------------------------- permute
// CTAs [0, pads) zero padding rows; the others take a part of a token's row
// each, one 16-byte vector a thread, whatever the type: short CTAs leave little
// work behind when the last ones run (with a CTA per token, 3.5 waves of 8 CTAs
// an SM, the last wave ran half empty).  pos and m_indices are read by coherent loads
// (and pos is not __restrict__): the layout kernel still writes them when this one
// starts.  4096 tokens x top-8 over 64 experts, 7168 bf16: 104 us with the layout
// kernel (of which some 7 us are not hidden), 588 MB with the padding rows: 0.87 of
// the measured copy bandwidth (replayed 101).
template <int kCap>
__global__ void __launch_bounds__(256) moe_permute_kernel(const uint4* __restrict__ x, int vecs, int parts, int tokens, int T,
                                                          int topk, const int32_t* pos, uint4* __restrict__ xs, int M,
                                                          int32_t* m_indices, int blocks, int pads, uint32_t* err) {
  if (static_cast<int>(blockIdx.x) < pads) {
    __shared__ uint8_t s_filled[kPadBlocks];
    int b0, b1, slice;
    pad_range(blockIdx.x, pads, blocks, b0, b1, slice);
    fp8g::grid_dependency_wait();  // m_indices
    for (int b = b0 + threadIdx.x; b < b1; b += blockDim.x) {
      int filled = 128;  // or unused
      if (__ldcg(m_indices + b) >= 0) {
        const int32_t entry = atomicAdd(m_indices + b, fp8g::moe::kBlockArrival);
        filled = fp8g::moe::block_filled(entry);
        if (fp8g::moe::block_arrivals(entry) == kPadSlices - 1) m_indices[b] = fp8g::moe::block_expert(entry);
      }
      s_filled[b - b0] = static_cast<uint8_t>(filled);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int b = b0; b < b1; ++b)
      for (int row = s_filled[b - b0] + slice + kPadSlices * warp; row < 128; row += kPadSlices * nw)
        for (int i = lane; i < vecs; i += 32) __stcs(xs + (b * 128L + row) * vecs + i, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  const int row_threads = blockDim.x / tokens, sub = threadIdx.x / row_threads, tid = threadIdx.x - sub * row_threads;
  // an item is a part of a token's row, or `tokens` short rows; memory holds fewer than 2^32 of them
  const unsigned items = (static_cast<unsigned>(T) + tokens - 1) / tokens * parts, stride = gridDim.x - pads;
  long t, at;  // of the current item: this thread's token, and its vector or -1 behind the row's end or the last token
  auto locate = [&](unsigned item) {
    const unsigned first = item / parts;
    const int j = static_cast<int>(item - first * parts) * row_threads + tid;
    t = static_cast<long>(first) * tokens + sub;
    at = j < vecs && t < T ? t * vecs + j : -1L;
  };
  unsigned i = blockIdx.x - pads;
  locate(i);
  uint4 v = at >= 0 ? __ldcs(x + at) : make_uint4(0u, 0u, 0u, 0u);  // x does not come from the layout kernel
  fp8g::grid_dependency_wait();                                     // pos does
  while (i < items) {
    const long j = at - t * vecs;
    int p[kCap];
#pragma unroll
    for (int k = 0; k < kCap; ++k) p[k] = k < topk && t < T ? pos[t * topk + k] : -1;
#pragma unroll
    for (int k = 0; k < kCap; ++k) {
      const int row = checked_pos(p[k], M, err);
      if (row >= 0 && at >= 0) __stcs(xs + static_cast<long>(row) * vecs + j, v);
    }
    i += stride;
    if (i < items) {
      locate(i);
      if (at >= 0) v = __ldcs(x + at);
    }
  }
}

// The whole sort of a small batch in one launch: every CTA counts the experts of
// all slots and its own slots' ranks itself instead of waiting for the layout
// kernel.  CTAs [0, pads) zero padding rows (they know how many every expert
// has) and write m_indices.
template <int kCap>
__global__ void __launch_bounds__(256) moe_permute_direct_kernel(const uint4* __restrict__ x, int vecs, int parts, int T,
                                                                 int topk, const int32_t* __restrict__ expert, int G,
                                                                 int32_t* __restrict__ pos, int32_t* __restrict__ m_indices,
                                                                 uint4* __restrict__ xs, int blocks, int pads,
                                                                 uint32_t* err) {
  __shared__ int32_t s_cnt[kMaxExperts], s_end[kMaxExperts];  // slots, and end of the segment in blocks
  __shared__ int32_t s_part[8][kCap];
  __shared__ int32_t s_row[kCap];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const bool pad = static_cast<int>(blockIdx.x) < pads;
  const int item = static_cast<int>(blockIdx.x) - pads, t = item / parts, part = item - t * parts;
  const int j = part * blockDim.x + threadIdx.x;
  const uint4 v = !pad && j < vecs ? __ldcs(x + static_cast<long>(t) * vecs + j) : make_uint4(0u, 0u, 0u, 0u);
  if (!pad) {
    int e[kCap];
#pragma unroll
    for (int k = 0; k < kCap; ++k) e[k] = k < topk ? fp8g::moe::expert_at(expert, G, t * topk + k, nullptr) : -1;
    fp8g::moe::count_earlier<kCap>(expert, t * topk, e, s_part);
  }
  fp8g::moe::count_experts(expert, T * topk, G, s_cnt, blockIdx.x == 0 ? err : nullptr);
  if (warp == 0) {
    // inclusive scan of the segments' blocks, 8 experts a lane
    int32_t n[kMaxExperts / 32], run = 0;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) run += (s_cnt[lane * (kMaxExperts / 32) + i] + 127) / 128, n[i] = run;
    int32_t incl = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) s_end[lane * (kMaxExperts / 32) + i] = incl - run + n[i];
  }
  __syncthreads();
  if (pad) {
    const int stride = pads * blockDim.x;
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < blocks; b += stride) {
      int g = 0;
      while (g < G && s_end[g] <= b) ++g;
      m_indices[b] = g < G ? g : -1;
    }
    // expert g's padding rows, every kPadSlices-th of them, a row per warp
    for (int it = blockIdx.x; it < G * kPadSlices; it += pads) {
      const int g = it / kPadSlices;
      const long end = 128L * s_end[g], first = end - (s_cnt[g] + 127) / 128 * 128L + s_cnt[g];
      for (long row = first + it % kPadSlices + kPadSlices * warp; row < end; row += kPadSlices * nw)
        for (int i = lane; i < vecs; i += 32) __stcs(xs + row * vecs + i, make_uint4(0u, 0u, 0u, 0u));
    }
    return;
  }
  if (static_cast<int>(threadIdx.x) < kCap) {
    const int k = threadIdx.x;
    const int g = k < topk ? fp8g::moe::expert_at(expert, G, static_cast<long>(t) * topk + k, nullptr) : -1;
    int row = -1;
    if (g >= 0) {
      row = 128 * (s_end[g] - (s_cnt[g] + 127) / 128);
      for (int i = 0; i < nw; ++i) row += s_part[i][k];
    }
    s_row[k] = row;
    if (part == 0 && k < topk) pos[t * topk + k] = row;
  }
  __syncthreads();
  if (j < vecs) {
#pragma unroll
    for (int k = 0; k < kCap; ++k)
      if (s_row[k] >= 0) __stcs(xs + static_cast<long>(s_row[k]) * vecs + j, v);
  }
}

// A CTA per token: all of a thread's row loads are issued before the first
// addition, which run in slot order.  The rows above, 529 MB: 85 us, 0.95 of the
// measured copy bandwidth (replayed 77: part of what it writes stays in L2).
template <bool kF32, int kCap>
__global__ void __launch_bounds__(256) moe_permute_backward_kernel(const void* __restrict__ dxs, int N,
                                                                   const int32_t* __restrict__ pos, int T, int topk,
                                                                   void* __restrict__ dx, int M, uint32_t* err) {
  for (long t = blockIdx.x; t < T; t += gridDim.x) {
    int p[kCap];
#pragma unroll
    for (int k = 0; k < kCap; ++k) p[k] = k < topk ? checked_pos(__ldg(pos + t * topk + k), M, err) : -1;
    for (int j = threadIdx.x; j < N / 8; j += blockDim.x) {
      Raw8<kF32> v[kCap];
#pragma unroll
      for (int k = 0; k < kCap; ++k)
        v[k] = p[k] >= 0 ? load8<kF32>(dxs, static_cast<long>(p[k]) * N + 8 * j) : zero8<kF32>();
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kCap; ++k) {
        float f[8];
        unpack8<kF32>(v[k], f);
        if (p[k] >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
      }
      store8<kF32>(dx, t * N + 8 * j, acc);
    }
  }
}

// ---------------------------------------------------------------- combine backward
// A CTA takes a token and walks its row in steps of blockDim vectors (8 columns
// a thread), four slots at a time.  A thread copies its own vectors of the next
// four slots' D rows (and of dout) into shared memory (cp.async) before it works
// on the current ones, so loads are under way all the time without holding
// registers.  The same rows, 1.06 GB with the padding: 174 us to bf16, 0.93 of the
// measured copy bandwidth; 0.80 GB to codes: 161 us, 0.76, replayed 141.  To codes
// nothing is saturated: 26 warps an SM issue in 65 % of the cycles, DRAM is at
// 64 %, and the 10.1 cycles between two instructions of a warp are spread over fixed
// latencies (1.8), waiting to be selected (1.7), the FP32 pipe (1.3), shared memory
// and shuffles (1.3), barriers (1.0) and loads (0.9); packed FP32x2 throughout.
//
// kQuant: the rows leave as e4m3 codes and 1x128 scales; 16 lanes hold a group
// of columns.  Its largest |w x| is |w| times its largest |x|, rounded once
// (rounding is monotonic), so one reduction over x serves every slot; lane k of
// the 16 forms slot k's scale and its reciprocal, and the others get them by
// shuffle: the divisions are done once per group and slot, not in every lane.
constexpr int kGroup = 4;

template <bool kQuant, int kGroups>
__global__ void __launch_bounds__(256, kGroups == 4 ? 2 : kQuant || kGroups == 1 ? 4 : 3)
    moe_combine_backward_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ D, int N,
                                const int32_t* __restrict__ pos, const float* __restrict__ w, int T, int topk,
                                uint16_t* __restrict__ dD, uint8_t* __restrict__ q, float* __restrict__ sa, int ld_sa,
                                float* __restrict__ dw, int tokens, int M, int blocks, int pads, uint32_t* err) {
  constexpr int kSlots = kGroup * kGroups;
  extern __shared__ __align__(16) uint8_t dyn[];  // two stages of kGroup + 1 vectors a thread
  struct Slots {
    long row[kSlots];  // first element of each slot's row, -1 if it is dropped
    int pos[kSlots];
    float w[kSlots];
  };
  __shared__ Slots s_slots[8];  // of each of the CTA's tokens
  __shared__ float s_dot[8][kSlots];
  if (static_cast<int>(blockIdx.x) < pads) {
    __shared__ uint32_t bits[kPadBlocks * 4];
    int b0, b1, slice;
    pad_range(blockIdx.x, pads, blocks, b0, b1, slice);
    pad_blocks(pos, static_cast<long>(T) * topk, b0, b1, slice, bits, err, [&](long row) {
      const int lane = threadIdx.x & 31;
      uint4* out = kQuant ? reinterpret_cast<uint4*>(q + row * N) : reinterpret_cast<uint4*>(dD + row * N);
      for (int i = lane; i < (kQuant ? N / 16 : N / 8); i += 32) __stcs(out + i, make_uint4(0u, 0u, 0u, 0u));
      if constexpr (kQuant)
        for (int kb = lane; kb < N / 128; kb += 32) sa[static_cast<long>(kb) * ld_sa + row] = 0.f;
    });
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int own = min(lane & 15, kSlots - 1);  // the slot whose scale this lane forms
  const int step = blockDim.x / tokens;  // threads of a token
  const int sub = threadIdx.x / step, tid = threadIdx.x - sub * step;
  Slots& slot = s_slots[sub];
  const int steps = (N / 8 + step - 1) / step;
  const uint32_t pitch = blockDim.x * 16, stage = (kGroup + 1) * pitch;
  const uint32_t slot0 = fp8g::smem_u32(dyn) + threadIdx.x * 16;
  for (long t0 = (static_cast<long>(blockIdx.x) - pads) * tokens; t0 < T; t0 += (static_cast<long>(gridDim.x) - pads) * tokens) {
    const long t = t0 + sub;
    const int slots = t < T ? topk : 0;  // behind the last token there are none
    if (tid < kSlots) {
      const int k = tid;
      const int p = k < slots ? checked_pos(__ldg(pos + t * topk + k), M, err) : -1;
      slot.pos[k] = p;
      slot.row[k] = p < 0 ? -1 : static_cast<long>(p) * N;
      slot.w[k] = k < slots && w ? __ldg(w + t * topk + k) : 1.f;
    }
    __syncthreads();
    const uint16_t* dout_t = dout + (t < T ? t * N : 0);
    long col = 8 * tid;   // this thread's columns: of the current vectors,
    int fetch_col = static_cast<int>(col);  // and of the next ones to fetch
    uint32_t put = slot0, get = slot0;
    // Copies the vectors of slots gi * kGroup ..; zeros for dropped slots and for
    // columns behind the row's end, whose products then add nothing.
    auto fetch = [&](int gi, bool there) {
      if (there) {
        const bool in = fetch_col < N;
        const int c = in ? fetch_col : 0;
        if (gi == 0) cp_async16_or_zero(put, dout_t + c, in ? 16 : 0);
        if (dw) {
#pragma unroll
          for (int k = 0; k < kGroup; ++k) {
            const long row = slot.row[gi * kGroup + k];
            cp_async16_or_zero(put + (k + 1) * pitch, D + (row < 0 ? 0 : row) + c, in && row >= 0 ? 16 : 0);
          }
        }
        if (gi == kGroups - 1) fetch_col += 8 * step;
      }
      cp_commit();
      put = put == slot0 ? slot0 + stage : slot0;
    };
    uint64_t dot[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) dot[k] = 0;
    fetch(0, true);
    for (int i = 0; i < steps; ++i, col += 8 * step) {
      const bool in = col < N;
      Pair8 g;
      float own_s = 1.f, own_y = 1.f;
      bool tiny = false;
#pragma unroll
      for (int gi = 0; gi < kGroups; ++gi) {
        fetch((gi + 1) % kGroups, gi + 1 < kGroups || i + 1 < steps);
        cp_wait<1>();
        if (gi == 0) {
          g = pairs_of<false>(load8_shared<false>(get));
          // every thread of a warp takes part in the groups' maxima and scales
          if constexpr (kQuant) {
            float x[8], amax = 0.f;
            values_of(g, x);
#pragma unroll
            for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(x[c]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            amax *= fabsf(slot.w[own]);
            tiny = __any_sync(0xffffffffu, amax > 0.f && amax < fp8g::quant::kTinyAmax);
            own_s = tiny ? fp8g::quant::scale_of(amax) : fp8g::quant::normal_scale(amax);
            own_y = __frcp_rn(own_s);
            if (in && (lane & 15) < kSlots && slot.pos[own] >= 0) sa[(col >> 7) * ld_sa + slot.pos[own]] = own_s;
          }
        }
        // Dropped slots are worked on like the others and only not stored: with
        // no branch between the slots their instructions interleave.
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
          const Pair8 d = pairs_of<false>(load8_shared<false>(get + (k + 1) * pitch));
#pragma unroll
          for (int m = 0; m < 4; ++m) dot[gi * kGroup + k] = fma2(g.v[m], d.v[m], dot[gi * kGroup + k]);
        }
        if constexpr (kQuant) {
          uint32_t c[kGroup][2];
          if (!tiny) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
              const float s = __shfl_sync(0xffffffffu, own_s, gi * kGroup + k, 16);
              const float y = __shfl_sync(0xffffffffu, own_y, gi * kGroup + k, 16);
              const uint64_t nw = both(-slot.w[gi * kGroup + k]);  // the quantiser takes negatives
              fp8g::quant::normal_codes(Pair8{mul2(g.v[0], nw), mul2(g.v[1], nw), mul2(g.v[2], nw), mul2(g.v[3], nw)}, s, y,
                                        c[k]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
              const float s = __shfl_sync(0xffffffffu, own_s, gi * kGroup + k, 16);
              const uint64_t nw = both(-slot.w[gi * kGroup + k]);
              fp8g::quant::any_codes(Pair8{mul2(g.v[0], nw), mul2(g.v[1], nw), mul2(g.v[2], nw), mul2(g.v[3], nw)}, s, c[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < kGroup; ++k) {
            const long row = slot.row[gi * kGroup + k];
            if (in && row >= 0) fp8g::quant::store_code_words(q + row + col, c[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kGroup; ++k) {
            const long row = slot.row[gi * kGroup + k];
            const uint64_t ww = both(slot.w[gi * kGroup + k]);
            float f[8];
            values_of(Pair8{mul2(g.v[0], ww), mul2(g.v[1], ww), mul2(g.v[2], ww), mul2(g.v[3], ww)}, f);
            if (in && row >= 0) store8<false>(dD, row + col, f);
          }
        }
        get = get == slot0 ? slot0 + stage : slot0;
      }
    }
    if (dw) {
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        if (k >= topk) continue;
        const float sum = warp_sum(sum2(dot[k]));
        if (lane == 0) s_dot[warp][k] = sum;
      }
    }
    const bool dropped = tid < kSlots && slot.pos[tid] < 0;
    __syncthreads();  // also: everyone has read the slots' rows and weights
    if (dw && tid < slots) {
      float sum = 0.f;
      for (int i = 0; i < step >> 5; ++i) sum += s_dot[sub * (step >> 5) + i][tid];
      dw[t * topk + tid] = dropped ? 0.f : sum;
    }
  }
}

// CTAs that zero padding rows: up to a quarter as many groups of blocks as SMs, or
// enough for their bitmaps.  In the combine's gradient each reads all of pos (to FP8,
// 4096 x top-8 x 7168: 147.7 us with half as many groups as SMs, 142.7 with a quarter,
// 139.5 with an eighth; 333 x top-4 x 4096 bf16 7.4, 7.4 and 8).
int pad_ctas(int blocks, int sms) {
  return kPadSlices * std::max((blocks + kPadBlocks - 1) / kPadBlocks, std::min(blocks, sms / 4));
}

// The kernel for a compile-time bound on topk: 4, 8 or 16.
template <typename F4, typename F8, typename F16>
void by_topk(int topk, F4 f4, F8 f8, F16 f16) {
  if (topk <= 4) f4();
  else if (topk <= 8) f8();
  else f16();
}

// Up to 256 threads that walk a row's vectors in equal steps.
int row_threads(long vecs) {
  const long steps = (vecs + 255) / 256;
  return static_cast<int>(((vecs + steps - 1) / steps + 31) / 32 * 32);
}

// Tokens of a CTA: one, or as many as give it 256 threads where the rows are
// narrow and the tokens many: a padding CTA reads every slot's position with as many
// threads as the others have (16384 x top-8, 512 bf16: combine backward to FP8 141 us
// with 64 threads, 72 with 256; sort of 65536 x top-4, 128 FP32: 76 and 70; with few
// tokens, one each spreads them over more SMs).
int cta_tokens(int T, int threads, int sms) { return T >= 8 * sms ? 256 / threads : 1; }

int check_slots(int T, int topk, int N) {
  if (T < 0 || topk < 1 || topk > kMaxTopk || N < 1 || N > 1 << 20 || static_cast<long>(T) * topk > 0x7FFFFFFFL)
    return FP8G_ERR_INVALID_ARG;
  return FP8G_OK;
}

}  // namespace

extern "C" int fp8g_moe_permute(const void* x, int x_dtype, int T, int N, const int32_t* expert, int topk, int G,
                                int blocks, void* xs, int32_t* pos, int32_t* m_indices, cudaStream_t stream) {
  if (x_dtype != FP8G_IN_BF16 && x_dtype != FP8G_IN_F32) return FP8G_ERR_INVALID_ARG;
  int rc = check_slots(T, topk, N);
  if (rc) return rc;
  if (G < 1 || G > kMaxExperts) return FP8G_ERR_INVALID_ARG;
  const long R = static_cast<long>(T) * topk;
  if (blocks < (R + 127) / 128 + G || blocks > 0x7FFFFFFF / 128) return FP8G_ERR_INVALID_ARG;
  if (N % 8 != 0) return FP8G_ERR_MISALIGNED;
  if (!m_indices || (R > 0 && (!x || !expert || !xs || !pos))) return FP8G_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(expert, 4) || !aligned(pos, 4) || !aligned(m_indices, 4))
    return FP8G_ERR_MISALIGNED;
  const int sms = sm_count();
  uint32_t* err = fp8g::device_error_word();
  if (sms <= 0 || !err) return FP8G_ERR_CUDA;
  const long vecs = static_cast<long>(N) * (x_dtype == FP8G_IN_F32 ? 4 : 2) / 16;
  const int parts = static_cast<int>((vecs + 255) / 256);
  if (R > 0 && R <= kDirectSlots && static_cast<long>(T) * parts <= 8L * sms) {
    const int pads = std::min(G * kPadSlices, 2 * sms);
    auto go = [&](auto kernel) {
      kernel<<<pads + T * parts, row_threads(vecs), 0, stream>>>(static_cast<const uint4*>(x), static_cast<int>(vecs), parts,
                                                                 T, topk, expert, G, pos, m_indices,
                                                                 static_cast<uint4*>(xs), blocks, pads, err);
    };
    by_topk(topk, [&] { go(moe_permute_direct_kernel<4>); }, [&] { go(moe_permute_direct_kernel<8>); },
            [&] { go(moe_permute_direct_kernel<kMaxTopk>); });
    if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
    return FP8G_OK;
  }
  if (fp8g::moe::launch_layout<false>(expert, static_cast<int>(R), G, 0, pos, m_indices, blocks, err, stream) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (R == 0) return FP8G_OK;
  const int pads = pad_ctas(blocks, sms);
  const int threads = row_threads(vecs), tokens = cta_tokens(T, parts == 1 ? threads : 256, sms);
  const long items = (static_cast<long>(T) + tokens - 1) / tokens * parts;
  const unsigned grid = static_cast<unsigned>(pads + std::min<long>(items, 1 << 20));
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    e = launch_behind(dim3(grid), threads * tokens, stream, kernel, static_cast<const uint4*>(x),
                                 static_cast<int>(vecs), parts, tokens, T, topk, static_cast<const int32_t*>(pos),
                                 static_cast<uint4*>(xs), blocks * 128, m_indices, blocks, pads, err);
  };
  by_topk(topk, [&] { go(moe_permute_kernel<4>); }, [&] { go(moe_permute_kernel<8>); },
          [&] { go(moe_permute_kernel<kMaxTopk>); });
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

extern "C" int fp8g_moe_permute_backward(const void* dxs, int dtype, int blocks, int N, const int32_t* pos, int T,
                                         int topk, void* dx, cudaStream_t stream) {
  if (dtype != FP8G_IN_BF16 && dtype != FP8G_IN_F32) return FP8G_ERR_INVALID_ARG;
  int rc = check_slots(T, topk, N);
  if (rc) return rc;
  if (blocks < 0 || blocks > 0x7FFFFFFF / 128) return FP8G_ERR_INVALID_ARG;
  if (N % 8 != 0) return FP8G_ERR_MISALIGNED;
  if (T == 0) return FP8G_OK;
  if ((blocks > 0 && !dxs) || !pos || !dx) return FP8G_ERR_INVALID_ARG;
  if (!aligned(dxs, 16) || !aligned(dx, 16) || !aligned(pos, 4)) return FP8G_ERR_MISALIGNED;
  const int sms = sm_count();
  uint32_t* err = fp8g::device_error_word();
  if (sms <= 0 || !err) return FP8G_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(std::min<long>(T, 32L * sms));
  auto go = [&](auto kernel) {
    kernel<<<grid, row_threads(N / 8), 0, stream>>>(dxs, N, pos, T, topk, dx, blocks * 128, err);
  };
  if (dtype == FP8G_IN_F32)
    by_topk(topk, [&] { go(moe_permute_backward_kernel<true, 4>); }, [&] { go(moe_permute_backward_kernel<true, 8>); },
            [&] { go(moe_permute_backward_kernel<true, kMaxTopk>); });
  else
    by_topk(topk, [&] { go(moe_permute_backward_kernel<false, 4>); }, [&] { go(moe_permute_backward_kernel<false, 8>); },
            [&] { go(moe_permute_backward_kernel<false, kMaxTopk>); });
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}

extern "C" int fp8g_moe_combine_backward(const uint16_t* dout, const uint16_t* D, int N, const int32_t* pos,
                                         const float* w, int T, int topk, int blocks, uint16_t* dD, uint8_t* q,
                                         float* sa, int ld_sa, float* dw, cudaStream_t stream) {
  int rc = check_slots(T, topk, N);
  if (rc) return rc;
  if (blocks < 0 || blocks > 0x7FFFFFFF / 128) return FP8G_ERR_INVALID_ARG;
  if (q && (N % 128 != 0 || ld_sa < blocks * 128L)) return FP8G_ERR_INVALID_ARG;
  if (N % 8 != 0 || (q && ld_sa % 4 != 0)) return FP8G_ERR_MISALIGNED;
  if (T == 0) return FP8G_OK;
  if (!dout || !pos || (blocks > 0 && ((dD != nullptr) == (q != nullptr) || (q && !sa) || (dw && !D))))
    return FP8G_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(D, 16) || !aligned(dD, 16) || !aligned(q, 16) || !aligned(sa, 16) ||
      !aligned(pos, 4) || !aligned(w, 4) || !aligned(dw, 4))
    return FP8G_ERR_MISALIGNED;
  const int sms = sm_count();
  uint32_t* err = fp8g::device_error_word();
  if (sms <= 0 || !err) return FP8G_ERR_CUDA;
  if (blocks == 0) D = dout;  // no row is read, but copies of no bytes name one
  const int pads = pad_ctas(blocks, sms);
  const int row = row_threads(N / 8), tokens = cta_tokens(T, row, sms), threads = row * tokens;
  const unsigned grid = static_cast<unsigned>(pads + std::min<long>((static_cast<long>(T) + tokens - 1) / tokens, 32L * sms));
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    e = allow_smem(kernel);
    if (e == cudaSuccess)
      kernel<<<grid, threads, 2 * (kGroup + 1) * threads * 16, stream>>>(dout, D, N, pos, w, T, topk, dD, q, sa, ld_sa, dw,
                                                                        tokens, blocks * 128, blocks, pads, err);
  };
  if (q)
    by_topk(topk, [&] { go(moe_combine_backward_kernel<true, 1>); }, [&] { go(moe_combine_backward_kernel<true, 2>); },
            [&] { go(moe_combine_backward_kernel<true, 4>); });
  else
    by_topk(topk, [&] { go(moe_combine_backward_kernel<false, 1>); }, [&] { go(moe_combine_backward_kernel<false, 2>); },
            [&] { go(moe_combine_backward_kernel<false, 4>); });
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}
