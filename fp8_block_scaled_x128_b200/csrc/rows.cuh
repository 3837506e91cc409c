// rows.cuh -- what the row-wise operators (norm.cu, moe_grad.cu,
// moe_masked.cu) share: 8-element accesses of bf16 and FP32 rows, sums over a
// warp and a CTA, host checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>

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

// 8 FP32 values as four packed pairs: one FP32x2 instruction (sm_100) does the
// work of two, with the same rounding, which matters where the kernels are
// bound by instructions issued rather than by the FP32 pipe.
struct Pair8 {
  uint64_t v[4];
};

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void split2(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }

__device__ __forceinline__ float sum2(uint64_t p) {
  float lo, hi;
  split2(p, lo, hi);
  return lo + hi;
}

template <bool kF32>
__device__ __forceinline__ Pair8 pairs_of(const Raw8<kF32>& r) {
  float f[8];
  unpack8<kF32>(r, f);
  Pair8 p;
#pragma unroll
  for (int i = 0; i < 4; ++i) p.v[i] = pack2(f[2 * i], f[2 * i + 1]);
  return p;
}

__device__ __forceinline__ void values_of(const Pair8& p, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(p.v[i], f[2 * i], f[2 * i + 1]);
}

// 8 FP32 parameters (16-byte aligned), kept in cache: every row uses them.
__device__ __forceinline__ Pair8 load_param8(const float* p, long e) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + e)), b = __ldg(reinterpret_cast<const float4*>(p + e) + 1);
  return Pair8{pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w)};
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Four (two) sums over a warp in 6 (5) shuffles instead of 20 (10): the first
// steps halve the values a lane carries, so the lanes of octet (half) o end with
// the sum of v[o].
__device__ __forceinline__ float warp_sums(const float (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool b16 = lane & 16, b8 = lane & 8;
  float a[2], x;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    a[i] = (b16 ? v[2 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, b16 ? v[i] : v[2 + i], 16);
  x = (b8 ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, b8 ? a[0] : a[1], 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float warp_sums(const float (&v)[2]) {
  const bool b16 = threadIdx.x & 16;
  float x = (b16 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, b16 ? v[0] : v[1], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sums of n (2 or 4) values over the kC CTAs of a cluster, in every thread, in
// a fixed order that gives every thread the same bits.  At most 16 warps a CTA;
// `call` counts the calls on this sm from 0.
//
// One CTA: each warp's sums go to shared memory, one barrier, every warp adds
// them.  s holds two buffers used in turn, and a buffer is written again only
// after the barrier of the call in between, which every thread reaches after
// reading it.
//
// A cluster: each warp sends its sums into every CTA's shared memory (st.async),
// and a CTA waits until all of them have arrived on its own mbarrier.  A cluster
// barrier instead would order, and so wait for, the rows the threads have just
// stored to global memory (it cost the backward of 4096 x 7168 FP32 33 us).  A CTA
// writes a peer's buffer again only after it has the peer's sums of the call in
// between, which every warp of the peer sends after reading the buffer; and it
// leaves after all sums sent to it have arrived (sums_leave).
template <int n, int kC>
struct RowSum {
  float s[2][n][16 * kC];
  uint64_t bar[2];
};

// Limit of a cluster's waits, and the test hook that makes one run out: in call
// `withhold` (0 or 1; kNoCall: none) the last CTA of every cluster waits for an
// arrival that never comes.
constexpr uint32_t kSumWaitUs = 1000000;
constexpr unsigned kNoCall = 0xFFFFFFFFu;
struct SumWait {
  unsigned withhold;
  uint32_t limit_us;
};

// A wait on a local mbarrier, given up after the limit: the flag is recorded, and
// this thread neither waits, nor arrives, nor sends any more (its rows are undefined).
// An arrival on a phase that the last one has left open would be one too many for
// the barrier, and without this thread's sums its peers give up in turn.
__device__ __forceinline__ void wait_or_flag(uint32_t bar, uint32_t parity, uint32_t limit_us, bool& gave_up,
                                             uint32_t* err) {
  if (gave_up || mbar_try_wait_cluster(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (globaltimer_ns() - t0 > limit_us * 1000ull) {
      gave_up = true;
      atomicOr(err, 0x1u);  // FP8G_DEVERR_TIMEOUT
      return;
    }
  }
}

// Before the first row_sum, by all threads; with kC > 1 a cluster barrier has to follow.
template <int n, int kC>
__device__ __forceinline__ void row_sum_init(RowSum<n, kC>& sm, int rank, const SumWait& limits) {
  if constexpr (kC > 1) {
    if (threadIdx.x == 0) {
#pragma unroll
      for (unsigned i = 0; i < 2; ++i) mbar_init(smem_u32(&sm.bar[i]), rank == kC - 1 && i == limits.withhold ? 2 : 1);
      fence_mbar_init();
    }
  }
}

template <int n, int kC>
__device__ __forceinline__ void row_sum(float (&v)[n], RowSum<n, kC>& sm, unsigned call, int rank, const SumWait& limits,
                                        bool& gave_up, uint32_t* err) {
  constexpr int kLanes = 32 / n;  // lanes that hold the same value
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float mine = warp_sums(v);
  if (kC > 1 || nw > 1) {
    const int value = lane / kLanes, peer = lane % kLanes;
    const unsigned turn = call & 1;
    if constexpr (kC == 1) {
      if (peer == 0) sm.s[turn][value][w] = mine;
      __syncthreads();
    } else {
      const uint32_t bar = smem_u32(&sm.bar[turn]);
      if (threadIdx.x == 0 && !gave_up) mbar_arrive_expect_tx(bar, kC * nw * n * 4);
      if (peer < kC && !gave_up)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                         mapa(smem_u32(&sm.s[turn][value][16 * rank + w]), peer)),
                     "r"(__float_as_uint(mine)), "r"(mapa(bar, peer))
                     : "memory");
      wait_or_flag(bar, call >> 1 & 1, limits.limit_us, gave_up, err);
    }
    // the lanes of a value add the warps' sums of it
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int i = 0; i < 16 / kLanes; ++i)
        x += peer + kLanes * i < nw ? sm.s[turn][value][16 * c + peer + kLanes * i] : 0.f;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    mine = x;
  }
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = __shfl_sync(0xffffffffu, mine, kLanes * i);
}

// The CTAs of a cluster end together: none is gone while another, whose waits may
// have been given up, still sends to it.  Behind the barrier everything is sent; a
// CTA that has given up a wait stays some microseconds longer, since what was sent
// to it last may still be on its way.
__device__ __forceinline__ void sums_leave(bool gave_up) {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (gave_up) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 20000) {
    }
  }
}

// ---------------------------------------------------------------- asynchronous copies
// Each thread copies its own vectors of a row into shared memory and reads
// back only those, so a finished copy needs no barrier, only cp_wait.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The first `bytes` (16 or 0) of 16, zeros behind them; src is valid either way.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Until at most N committed groups of this thread are under way.
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8 elements of a row, global to shared.
template <bool kF32>
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t* src) {
  cp_async16(dst, src);
  if constexpr (kF32) cp_async16(dst + 16, src + 16);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

template <bool kF32>
__device__ __forceinline__ Raw8<kF32> load8_shared(uint32_t addr) {
  Raw8<kF32> r;
  r.v[0] = ld_shared_v4(addr);
  if constexpr (kF32) r.v[1] = ld_shared_v4(addr + 16);
  return r;
}

// ---------------------------------------------------------------- host
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Lets a kernel use all of an SM's shared memory that its static part leaves,
// once per kernel and device (the calls would cost every launch a microsecond).
template <typename... KArgs>
inline cudaError_t allow_smem(void (*kernel)(KArgs...)) {
  struct Seen {
    const void* fn;
    uint64_t devices;
  };
  static std::mutex mu;
  static Seen seen[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  Seen* at = nullptr;
  for (Seen& s : seen) {
    if (s.fn == reinterpret_cast<const void*>(kernel) || !s.fn) {
      at = &s;
      break;
    }
  }
  if (at && at->fn && dev < 64 && (at->devices >> dev & 1)) return cudaSuccess;
  int most = 0;
  cudaFuncAttributes fa;
  if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  if ((e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kernel))) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           most - static_cast<int>(fa.sharedSizeBytes));
  if (e == cudaSuccess && at && dev < 64) at->fn = reinterpret_cast<const void*>(kernel), at->devices |= 1ull << dev;
  return e;
}

// Streaming multiprocessors of the current device, -1 if there is none.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  return n;
}

// Programmatic dependent launch is on unless FP8G_DISABLE_PDL is set to a nonzero
// value in the environment (read once), as for the GEMMs.
inline bool pdl_on() {
  static const bool on = [] {
    const char* e = std::getenv("FP8G_DISABLE_PDL");
    return !(e && *e && std::strcmp(e, "0") != 0);
  }();
  return on;
}

// A launch that may take its place while the kernel before it in the stream
// still runs (once that one allows it, grid_launch_dependents): it has to wait
// (grid_dependency_wait) before it reads what that kernel writes.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_behind(dim3 grid, int threads, cudaStream_t stream, void (*kernel)(KArgs...), Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_on() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace rows
}  // namespace fp8g
