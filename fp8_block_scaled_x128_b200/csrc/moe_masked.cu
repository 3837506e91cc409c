// moe_masked.cu -- expert dispatch into the masked layout of decode, sm_100a.
//
// The masked grouped GEMM takes A [G][Mmax][K] and the row counts masked_m [G]
// on the device.  Routed slot r = t * topk + k takes row `rank` of its
// expert's group, rank being the number of earlier slots of that expert;
// token t is quantised once per 1x128 group and its codes and scales are
// stored into all of its rows.  pos[r] = g * Mmax + rank is the row in the
// GEMM's D seen as [G * Mmax][N], which is what the combine takes.
//
// Decode is latency: few tokens, one call per layer.  Up to kDirectSlots
// routed slots the whole dispatch is one launch: a CTA per token counts its
// slots' ranks itself, from the experts of the slots before it (a ballot per
// slot and 32 earlier slots), instead of waiting for a layout kernel; one more
// CTA counts the experts' rows.  The counting grows with T * T * topk * topk,
// so larger batches run the layout kernel first.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8gemm.h"
#include "moe_layout.cuh"
#include "quant_impl.cuh"
#include "rows.cuh"

namespace {

using namespace fp8g::quant;
using namespace fp8g::rows;
using fp8g::moe::expert_at;
using fp8g::moe::kMaxExperts;
using fp8g::moe::kMaxTopk;

constexpr int kDirectSlots = 4096;
constexpr int kThreads = 256;
constexpr int kAhead = 8;  // loads of earlier slots in flight per lane

// kDirect: ranks are counted here (grid T + 1, the last CTA counts rows per
// expert); otherwise pos and masked_m are already there.
template <bool kF32, int kCap, bool kDirect>
__global__ void __launch_bounds__(kThreads) moe_dispatch_masked_kernel(const void* __restrict__ x, int K, int T, int topk,
                                                                       const int32_t* __restrict__ expert, int G,
                                                                       int Mmax, uint8_t* __restrict__ A,
                                                                       float* __restrict__ sa, int ld_sa, int32_t* pos,
                                                                       int32_t* __restrict__ masked_m, uint32_t* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kThreads / 32;
  __shared__ int32_t s_cnt[kDirect ? kMaxExperts : 1];
  __shared__ int32_t s_part[kDirect ? kWarps : 1][kDirect ? kCap : 1];
  if constexpr (kDirect) {
    if (static_cast<int>(blockIdx.x) == T) {
      for (int g = threadIdx.x; g < G; g += kThreads) s_cnt[g] = 0;
      __syncthreads();
      for (long r = threadIdx.x; r < static_cast<long>(T) * topk; r += kThreads) {
        const int g = expert_at(expert, G, r, err);
        if (g >= 0) atomicAdd(&s_cnt[g], 1);
      }
      __syncthreads();
      for (int g = threadIdx.x; g < G; g += kThreads) {
        masked_m[g] = min(s_cnt[g], Mmax);
        if (s_cnt[g] > Mmax) atomicOr(err, FP8G_DEVERR_MASKED_OVER);
      }
      return;
    }
  }
  const size_t esz = kF32 ? 4 : 2;
  const int KB = K / 128;
  const int per_warp = (KB + kWarps - 1) / kWarps;  // K-blocks of a warp
  const int kb0 = min(KB, warp * per_warp), kb1 = min(KB, kb0 + per_warp);
  const long stride = kDirect ? T : gridDim.x;
  for (long t = blockIdx.x; t < T; t += stride) {
    int dst[kCap];
    if constexpr (kDirect) {
      int e[kCap], n[kCap];
#pragma unroll
      for (int k = 0; k < kCap; ++k) {
        e[k] = k < topk ? expert_at(expert, G, t * topk + k, nullptr) : -1;
        n[k] = 0;
      }
      // earlier slots of each of this token's experts: a share per warp
      const int before = static_cast<int>(t) * topk;
      for (int r0 = 32 * warp; r0 < before; r0 += kAhead * kThreads) {
        int g[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int r = r0 + i * kThreads + lane;
          g[i] = r < before ? __ldg(expert + r) : -1;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (r0 + i * kThreads >= before) break;  // warp-uniform
#pragma unroll
          for (int k = 0; k < kCap; ++k) n[k] += __popc(__ballot_sync(0xffffffffu, g[i] == e[k]));
        }
      }
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < kCap; ++k) s_part[warp][k] = n[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kCap; ++k) {
        int rank = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) rank += s_part[w][k];
#pragma unroll
        for (int i = 0; i < k; ++i) rank += e[i] == e[k];  // the same expert twice in a token
        dst[k] = e[k] >= 0 && rank < Mmax ? e[k] * Mmax + rank : -1;
        if (k < topk && static_cast<int>(threadIdx.x) == k) pos[t * topk + k] = dst[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < kCap; ++k) dst[k] = k < topk ? pos[t * topk + k] : -1;
    }
    if (kb0 >= kb1) continue;
    long at[kCap];  // first scale of the row in sa
#pragma unroll
    for (int k = 0; k < kCap; ++k)
      at[k] = dst[k] < 0 ? 0 : static_cast<long>(dst[k] / Mmax) * KB * ld_sa + dst[k] % Mmax;
    quantize_row_1x128<kF32>(
        static_cast<const uint8_t*>(x) + (t * K + 128L * kb0) * esz, 128 * (kb1 - kb0),
        [&](long off, const auto& c) {
#pragma unroll
          for (int k = 0; k < kCap; ++k)
            if (dst[k] >= 0) store_code_words(A + static_cast<long>(dst[k]) * K + 128L * kb0 + off, c);
        },
        [&](int kb, float s) {
#pragma unroll
          for (int k = 0; k < kCap; ++k)
            if (dst[k] >= 0) sa[at[k] + static_cast<long>(kb0 + kb) * ld_sa] = s;
        });
  }
}

}  // namespace

extern "C" int fp8g_moe_dispatch_masked(const void* x, int x_dtype, int T, int K, const int32_t* expert, int topk, int G,
                                        int Mmax, uint8_t* A, float* sa, int ld_sa, int32_t* pos, int32_t* masked_m,
                                        cudaStream_t stream) {
  if (x_dtype != FP8G_IN_BF16 && x_dtype != FP8G_IN_F32) return FP8G_ERR_INVALID_ARG;
  if (T < 0 || topk < 1 || topk > kMaxTopk || K <= 0 || K % 128 != 0 || K > 65536 || G < 1 || G > kMaxExperts)
    return FP8G_ERR_INVALID_ARG;
  const long R = static_cast<long>(T) * topk;
  if (R > 0x7FFFFFFFL || Mmax < 1 || static_cast<long>(G) * Mmax > 0x7FFFFFFFL || ld_sa < Mmax) return FP8G_ERR_INVALID_ARG;
  if (ld_sa % 4 != 0) return FP8G_ERR_MISALIGNED;
  if (!masked_m || (R > 0 && (!x || !expert || !A || !sa || !pos))) return FP8G_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(A, 16) || !aligned(sa, 16) || !aligned(expert, 4) || !aligned(pos, 4) ||
      !aligned(masked_m, 4))
    return FP8G_ERR_MISALIGNED;
  const int sms = sm_count();
  uint32_t* err = fp8g::device_error_word();
  if (sms <= 0 || !err) return FP8G_ERR_CUDA;
  const bool direct = R <= kDirectSlots;
  if (!direct && fp8g::moe::launch_layout<true>(expert, static_cast<int>(R), G, Mmax, pos, masked_m, 0, err, stream) !=
                     cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  const unsigned grid = static_cast<unsigned>(direct ? T + 1 : std::min<long>(T, 16L * sms));
  auto go = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, stream>>>(x, K, T, topk, expert, G, Mmax, A, sa, ld_sa, pos, masked_m, err);
  };
  const bool f32 = x_dtype == FP8G_IN_F32;
  if (direct) {
    if (topk <= 4) f32 ? go(moe_dispatch_masked_kernel<true, 4, true>) : go(moe_dispatch_masked_kernel<false, 4, true>);
    else if (topk <= 8) f32 ? go(moe_dispatch_masked_kernel<true, 8, true>) : go(moe_dispatch_masked_kernel<false, 8, true>);
    else f32 ? go(moe_dispatch_masked_kernel<true, kMaxTopk, true>) : go(moe_dispatch_masked_kernel<false, kMaxTopk, true>);
  } else {
    if (topk <= 4) f32 ? go(moe_dispatch_masked_kernel<true, 4, false>) : go(moe_dispatch_masked_kernel<false, 4, false>);
    else if (topk <= 8) f32 ? go(moe_dispatch_masked_kernel<true, 8, false>) : go(moe_dispatch_masked_kernel<false, 8, false>);
    else f32 ? go(moe_dispatch_masked_kernel<true, kMaxTopk, false>) : go(moe_dispatch_masked_kernel<false, kMaxTopk, false>);
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}
