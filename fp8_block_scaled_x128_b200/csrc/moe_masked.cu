// moe_masked.cu -- expert dispatch into the masked layout of decode, sm_100a.
//
// The masked grouped GEMM takes A [G][Mmax][K] and the row counts masked_m [G]
// on the device.  Routed slot r = t * topk + k takes row `rank` of its
// expert's group, rank being the number of earlier slots of that expert;
// token t is quantised once per 1x128 group and its codes and scales are
// stored into all of its rows.  pos[r] = g * Mmax + rank is the row in the
// GEMM's D seen as [G * Mmax][N], which is what the combine takes.
//
// Decode is latency: few tokens, one call per layer.  A CTA takes 2048 columns
// of a token (or 8192, once the tokens alone fill the GPU: then the ranks are
// counted once per token), 8 a thread and vector; its loads are issued first, so
// that they are under way while the slots' rows are found.  Up to kDirectSlots routed slots the whole
// dispatch is one launch: each CTA counts its slots' ranks itself, from the
// experts of the slots before it (a ballot per slot and 32 earlier slots),
// instead of waiting for a layout kernel; one more CTA counts the experts' rows.
// The counting grows with T * T * topk * topk, so larger batches run the layout
// kernel first.  K = 7168, top-8, bf16, calls back to back (and replayed in a CUDA
// graph): one token 9.3 us (2.7) and 256 tokens 9.5 (7.4; chains of three loads, the
// counting and the codes; 18.8 MB), 512 tokens 12.3 (11.1), 1024 tokens with the
// layout kernel 23.5 (21; 75 MB, 0.49 of the copy bandwidth).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "fp8gemm.h"
#include "moe_layout.cuh"
#include "quant8.cuh"
#include "rows.cuh"

namespace {

using namespace fp8g::quant;
using namespace fp8g::rows;
using fp8g::moe::expert_at;
using fp8g::moe::kMaxExperts;
using fp8g::moe::kMaxTopk;

constexpr int kDirectSlots = 4096;
constexpr int kThreads = 256;

// kDirect: ranks are counted here (the first CTA counts rows per expert);
// otherwise pos and masked_m are already there.
template <bool kF32, int V, int kCap, bool kDirect>
__global__ void __launch_bounds__(kThreads) moe_dispatch_masked_kernel(const void* __restrict__ x, int K, int parts, int T,
                                                                       int topk, const int32_t* __restrict__ expert, int G,
                                                                       int Mmax, uint8_t* __restrict__ A,
                                                                       float* __restrict__ sa, int ld_sa, int32_t* pos,
                                                                       int32_t* __restrict__ masked_m, uint32_t* err) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int32_t s_cnt[kDirect ? kMaxExperts : 1];
  __shared__ int32_t s_part[kDirect ? kWarps : 1][kCap];
  __shared__ int32_t s_row[kCap];  // each slot's row of A as [G * Mmax][K], -1 if it is dropped
  __shared__ long s_scale[kCap];   // its first scale in sa
  const int lane = threadIdx.x & 31;
  const long items = static_cast<long>(T) * parts;
  if constexpr (kDirect) {
    if (blockIdx.x == 0) {
      fp8g::moe::count_experts<kThreads>(expert, T * topk, G, s_cnt, err);
      for (int g = threadIdx.x; g < G; g += kThreads) {
        masked_m[g] = min(s_cnt[g], Mmax);
        if (s_cnt[g] > Mmax) atomicOr(err, FP8G_DEVERR_MASKED_OVER);
      }
      return;
    }
  }
  for (long i = static_cast<long>(blockIdx.x) - (kDirect ? 1 : 0); i < items; i += gridDim.x) {
    const long t = i / parts;
    const int part = static_cast<int>(i - t * parts);
    const int col0 = 8 * (part * V * kThreads + threadIdx.x);
    // K % 128 == 0: the 16 lanes of a group are all in the row or all behind it
    Raw8<kF32> raw[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = col0 + 8 * v * kThreads;
      raw[v] = col < K ? load8<kF32>(x, t * K + col) : zero8<kF32>();
    }
    if constexpr (!kDirect) fp8g::grid_dependency_wait();  // pos is the layout kernel's, x is not
    if constexpr (kDirect) {
      int e[kCap];
#pragma unroll
      for (int k = 0; k < kCap; ++k) e[k] = k < topk ? expert_at(expert, G, t * topk + k, nullptr) : -1;
      fp8g::moe::count_earlier<kCap, kThreads>(expert, static_cast<int>(t) * topk, e, s_part);
      __syncthreads();
    }
    if (static_cast<int>(threadIdx.x) < kCap) {
      const int k = threadIdx.x;
      int g = -1, rank = 0;
      if constexpr (kDirect) {
        if (k < topk) g = expert_at(expert, G, t * topk + k, nullptr);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) rank += s_part[w][k];
        if (rank >= Mmax) g = -1;
        if (part == 0 && k < topk) pos[t * topk + k] = g < 0 ? -1 : g * Mmax + rank;
      } else {
        const int p = k < topk ? pos[t * topk + k] : -1;
        if (p >= 0) g = p / Mmax, rank = p - g * Mmax;
      }
      s_row[k] = g < 0 ? -1 : g * Mmax + rank;
      s_scale[k] = static_cast<long>(g) * (K / 128) * ld_sa + rank;
    }
    // the token's codes do not depend on where they go
    uint32_t c[V][2];
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8], amax = 0.f;
      unpack8<kF32>(raw[v], f);
#pragma unroll
      for (int a = 0; a < 8; ++a) amax = fmaxf(amax, fabsf(f[a]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      Pair8 neg;
#pragma unroll
      for (int a = 0; a < 4; ++a) neg.v[a] = pack2(-f[2 * a], -f[2 * a + 1]);
      quantize8(neg, amax, s[v], c[v]);
    }
    __syncthreads();
    const int own = lane & 15;  // lane k of a group stores slot k's scale
    const bool own_live = own < kCap && s_row[own < kCap ? own : 0] >= 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = col0 + 8 * v * kThreads;
      if (col >= K) break;
#pragma unroll
      for (int k = 0; k < kCap; ++k) {
        const int row = s_row[k];
        if (row >= 0) store_code_words(A + static_cast<long>(row) * K + col, c[v]);
      }
      if (own_live) sa[s_scale[own] + static_cast<long>(col >> 7) * ld_sa] = s[v];
    }
    if (i + gridDim.x < items) __syncthreads();  // the next item writes s_row again
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
  // whole tokens per CTA once there is one for every SM (K = 7168, top-8: 256 tokens
  // 7.4 us against 8.6 with 2048 columns a CTA, 512 tokens 11.2 against 17.2)
  const int vecs = T >= sms ? 4 : 1;
  const int parts = (K / 8 + vecs * kThreads - 1) / (vecs * kThreads);
  const long items = static_cast<long>(T) * parts;
  const unsigned grid = static_cast<unsigned>(direct ? items + 1 : std::min<long>(items, 1 << 20));
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    if (direct)
      kernel<<<grid, kThreads, 0, stream>>>(x, K, parts, T, topk, expert, G, Mmax, A, sa, ld_sa, pos, masked_m, err);
    else
      e = launch_behind(dim3(grid), kThreads, stream, kernel, x, K, parts, T, topk, expert, G, Mmax, A, sa, ld_sa, pos,
                                   masked_m, err);
  };
  auto by_kind = [&](auto v) {
    constexpr int V = decltype(v)::value;
    auto by_type = [&](auto f32) {
      constexpr bool F = decltype(f32)::value;
      if (direct) {
        if (topk <= 4) go(moe_dispatch_masked_kernel<F, V, 4, true>);
        else if (topk <= 8) go(moe_dispatch_masked_kernel<F, V, 8, true>);
        else go(moe_dispatch_masked_kernel<F, V, kMaxTopk, true>);
      } else {
        if (topk <= 4) go(moe_dispatch_masked_kernel<F, V, 4, false>);
        else if (topk <= 8) go(moe_dispatch_masked_kernel<F, V, 8, false>);
        else go(moe_dispatch_masked_kernel<F, V, kMaxTopk, false>);
      }
    };
    if (x_dtype == FP8G_IN_F32) by_type(std::true_type{});
    else by_type(std::false_type{});
  };
  if (vecs == 4) by_kind(std::integral_constant<int, 4>{});
  else by_kind(std::integral_constant<int, 1>{});
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}
