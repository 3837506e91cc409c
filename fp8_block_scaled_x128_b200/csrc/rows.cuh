// rows.cuh -- what the row-wise operators (norm.cu, moe_grad.cu,
// moe_masked.cu) share: 8-element accesses of bf16 and FP32 rows, sums over a
// warp and a CTA, host checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace fp8g {

uint32_t* device_error_word();  // api.cu: this device's FP8G_DEVERR_* word

namespace rows {

// 8 consecutive elements of a row in their input format: one 16-byte vector
// of bf16, two of FP32.
template <bool kF32>
struct Raw8 {
  uint4 v[kF32 ? 2 : 1];
};

// Element index e is a multiple of 8.  Streaming loads: every row is read once.
template <bool kF32>
__device__ __forceinline__ Raw8<kF32> load8(const void* base, long e) {
  Raw8<kF32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + e * (kF32 ? 4 : 2));
  r.v[0] = __ldcs(p);
  if constexpr (kF32) r.v[1] = __ldcs(p + 1);
  return r;
}

template <bool kF32>
__device__ __forceinline__ Raw8<kF32> zero8() {
  Raw8<kF32> r;
  r.v[0] = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (kF32) r.v[1] = make_uint4(0u, 0u, 0u, 0u);
  return r;
}

template <bool kF32>
__device__ __forceinline__ void unpack8(const Raw8<kF32>& r, float (&f)[8]) {
  if constexpr (kF32) {
    f[0] = __uint_as_float(r.v[0].x), f[1] = __uint_as_float(r.v[0].y);
    f[2] = __uint_as_float(r.v[0].z), f[3] = __uint_as_float(r.v[0].w);
    f[4] = __uint_as_float(r.v[1].x), f[5] = __uint_as_float(r.v[1].y);
    f[6] = __uint_as_float(r.v[1].z), f[7] = __uint_as_float(r.v[1].w);
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// 8 FP32 values rounded once (to nearest even for bf16) and stored.
template <bool kF32>
__device__ __forceinline__ void store8(void* base, long e, const float (&f)[8]) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + e * (kF32 ? 4 : 2));
  if constexpr (kF32) {
    __stcs(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    __stcs(p + 1, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
  } else {
    __stcs(p, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7])));
  }
}

// 8 FP32 parameters (16-byte aligned), kept in cache: every row uses them.
__device__ __forceinline__ void load_param8(const float* p, long e, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + e)), b = __ldg(reinterpret_cast<const float4*>(p + e) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sums of n values over the CTA, in every thread, in a fixed order (xor
// butterflies: all lanes get the same bits).  One barrier per call: s holds two
// buffers used in turn, and a buffer is written again only after the barrier
// of the call in between, which every thread reaches after reading it.
template <int n>
struct BlockSum {
  float s[2][n][32];
};

template <int n>
__device__ __forceinline__ void block_sum(float (&v)[n], BlockSum<n>& sm, int& turn) {
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = warp_sum(v[i]);
  const int nw = (blockDim.x + 31) >> 5;
  if (nw == 1) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < n; ++i) sm.s[turn][i][w] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = warp_sum(lane < nw ? sm.s[turn][i][lane] : 0.f);
  turn ^= 1;
}

// ---------------------------------------------------------------- host
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Streaming multiprocessors of the current device, -1 if there is none.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  return n;
}

}  // namespace rows
}  // namespace fp8g
