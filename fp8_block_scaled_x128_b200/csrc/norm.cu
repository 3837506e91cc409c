// norm.cu -- the norms around a block, fused with its gate, residual scale and
// residual sum, and their gradients, sm_100a.
//
// With u = y / sqrt(mean(y^2) + eps) (u = y without a post-norm), per row:
//
//   h' = h + s g w_post u           the residual stream after the block
//   z  = w_pre h' / sqrt(mean(h'^2) + eps)
//                                   the next block's input, as rows or as e4m3
//                                   codes with one FP32 scale per 1x128 group
//
// and backwards, with r1 = 1/sqrt(mean(h'^2) + eps), n = h' r1, r2 likewise
// for y, <.> the mean over the row:
//
//   dh    = dh_out + r1 (dz w_pre - n <dz w_pre n>)
//   dy    = r2 (du - u <du u>), du = s g w_post dh   (dy = du without post-norm)
//   dw_pre = sum_rows dz n,  dw_post = sum_rows s g dh u
//   dgate  = s w_post dh u, summed over rows (gate per channel) or over the
//            row (gate per token)
//
// All arithmetic is FP32; rows are rounded once, when they are stored.  z is
// formed from the unrounded h', so its error is one rounding; the backward
// pass starts from the stored h'.  Both row statistics of the backward pass
// are recomputed from h' and y, which it has to read anyway, so nothing is
// kept between the passes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fp8gemm.h"
#include "quant8.cuh"
#include "rows.cuh"

namespace {

using namespace fp8g::rows;
using fp8g::cluster_ctarank;
using fp8g::cluster_sync_all;
using fp8g::quant::quantize8;

constexpr int kMaxH = 16384;

// A row belongs to a cluster of 1, 2 or 4 CTAs, each with a run of its columns
// and a thread per 8 of them.  The rows stream through shared memory in kStages
// stages: a thread copies its own columns of a later row (cp.async) as soon as
// it has read its columns of the current one, so kStages - 1 rows are under
// way per CTA while one is worked on, without barriers or waits on other
// threads.  The parameters' values of a thread's columns stay in registers for
// all of the CTA's rows.
constexpr int kBackwardStages = 3;
__host__ __device__ constexpr int forward_stages(bool f32) { return f32 ? 3 : 4; }

struct Shape {
  int rows, H;
  int cols;      // columns of a CTA (the last of a cluster may have fewer)
  uint32_t pitch;  // bytes of one row's part in shared memory (whole warps of it)
};

struct Params {
  const float *post_w, *gate, *pre_w;
  int gate_kind;
  float scale, eps;
};

// Parameters of columns col .. col + 7: pre_w, and a = post_w times a gate per channel.
__device__ __forceinline__ void column_params(const Params& p, int col, bool in, Pair8& pre, Pair8& a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) pre.v[i] = a.v[i] = both(1.f);
  if (!in) return;
  if (p.pre_w) pre = load_param8(p.pre_w, col);
  if (p.post_w) a = load_param8(p.post_w, col);
  if (p.gate_kind == FP8G_GATE_CHANNEL) {
    const Pair8 g = load_param8(p.gate, col);
#pragma unroll
    for (int i = 0; i < 4; ++i) a.v[i] = mul2(a.v[i], g.v[i]);
  }
}

// 1 / sqrt(mean + eps): rsqrtf (within 2 units in the last place) and one Newton
// step, r + r (1 - x r^2) / 2, which leaves the roundings of its last operation.
// An IEEE division of an IEEE square root costs every thread of the CTA some
// sixty dependent instructions per row.  x is never zero (eps > 0); an infinite
// x (a row that overflows) gives 0, as the division would.
__device__ __forceinline__ float rms_factor(float sum, float inv_h, float eps) {
  const float x = fmaf(sum, inv_h, eps);
  const float r = rsqrtf(x);
  const float refined = fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r);
  return isinf(x) ? r : refined;
}

// The stages of a CTA: kTensors rows each, walked in step with its rows.  A
// thread's slots of a tensor that is not there, and all slots of a thread
// without columns, are zeroed once and never copied to, so the arithmetic needs
// no conditions.  Addresses advance by additions only: with a multiplication
// per row and tensor, a third of the instructions were address arithmetic.
template <bool kF32, int kTensors, int kStages>
struct Stream {
  const uint8_t* src[kTensors];  // this thread's columns of the next row to fetch
  uint32_t slot, stage_bytes, pitch;
  uint32_t put, get_at;  // stages to fill and to read, as offsets
  long step_bytes;       // bytes from a CTA's row to its next
  long next;             // the next row to fetch
  bool in, third, fourth;

  static constexpr int kVec = kF32 ? 32 : 16;  // bytes of 8 elements

  __device__ __forceinline__ void init(const void* const (&t)[kTensors], const uint8_t* smem, const Shape& S, int col0,
                                       bool has_columns, long row0, long step) {
    slot = fp8g::smem_u32(smem) + threadIdx.x * kVec;
    pitch = S.pitch;
    stage_bytes = kTensors * pitch;
    put = get_at = 0;
    in = has_columns;
    next = row0;
    const long row_bytes = static_cast<long>(S.H) * (kVec / 8);
    step_bytes = step * row_bytes;
#pragma unroll
    for (int i = 0; i < kTensors; ++i) {
      if (!in || !t[i]) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
          st_shared_zero16(slot + s * stage_bytes + i * pitch);
          if constexpr (kF32) st_shared_zero16(slot + s * stage_bytes + i * pitch + 16);
        }
      }
      src[i] = static_cast<const uint8_t*>(t[i]) + (row0 * row_bytes + static_cast<long>(col0) * (kVec / 8) + threadIdx.x * kVec);
    }
    third = kTensors > 2 && t[kTensors > 2 ? 2 : 0];
    fourth = kTensors > 3 && t[kTensors > 3 ? 3 : 0];
    if (kTensors == 2) third = t[1] != nullptr;  // the forward pass's residual
  }

  // Copies this thread's part of the next row, if there is one, into the next stage.
  __device__ __forceinline__ void fetch(int rows, long step) {
    if (next < rows && in) {
      const uint32_t at = slot + put;
      copy8<kF32>(at, src[0]);
      if constexpr (kTensors == 2) {
        if (third) copy8<kF32>(at + pitch, src[1]);
      } else {
        copy8<kF32>(at + pitch, src[1]);
        if (third) copy8<kF32>(at + 2 * pitch, src[2]);
        if (fourth) copy8<kF32>(at + 3 * pitch, src[3]);
      }
    }
    cp_commit();
    next += step;
#pragma unroll
    for (int i = 0; i < kTensors; ++i) src[i] += step_bytes;
    put = put == (kStages - 1) * stage_bytes ? 0 : put + stage_bytes;
  }

  __device__ __forceinline__ Pair8 get(int tensor) const {
    return pairs_of<kF32>(load8_shared<kF32>(slot + get_at + tensor * pitch));
  }

  __device__ __forceinline__ void advance() { get_at = get_at == (kStages - 1) * stage_bytes ? 0 : get_at + stage_bytes; }
};

// Stores a thread's 8 values of a row, rounded once.
template <bool kF32>
__device__ __forceinline__ void put8(uint8_t* at, const Pair8& p) {
  float f[8];
  values_of(p, f);
  store8<kF32>(at, 0, f);
}

template <bool kF32, int kC, bool kQuant>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const void* y, const void* h, Shape S, Params P, void* h_out,
                                                             void* z, uint8_t* q, float* sa, int ld_sa) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowSum<1, kC> sm;
  constexpr int D = forward_stages(kF32);
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long row0 = blockIdx.x / kC, step = gridDim.x / kC;
  const int col0 = rank * S.cols, col = col0 + 8 * threadIdx.x;
  const bool in = 8 * static_cast<int>(threadIdx.x) < S.cols && col < S.H;
  Stream<kF32, 2, D> src;
  src.init({y, h}, dyn, S, col0, in, row0, step);
#pragma unroll
  for (int s = 0; s < D - 1; ++s) src.fetch(S.rows, step);
  const long first = (row0 * S.H + col) * (src.kVec / 8);
  uint8_t *h_at = static_cast<uint8_t*>(h_out) + first, *z_at = static_cast<uint8_t*>(z) + first;
  uint8_t* q_at = q + (row0 * S.H + col);
  float* sa_at = sa + (static_cast<long>(col / 128) * ld_sa + row0);
  Pair8 pw, a;
  column_params(P, col, in, pw, a);
  if constexpr (kC > 1) cluster_sync_all();
  const float inv_h = 1.f / static_cast<float>(S.H);
  int turn = 0;
  for (long row = row0; row < S.rows; row += step) {
    src.fetch(S.rows, step);
    cp_wait<D - 1>();
    const Pair8 yv = src.get(0);
    Pair8 hv = src.get(1);
    src.advance();
    float f = P.scale;
    if (P.gate_kind == FP8G_GATE_TOKEN) f *= __ldg(P.gate + row);
    float ss[1];
    if (P.post_w) {
      uint64_t acc = mul2(yv.v[0], yv.v[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) acc = fma2(yv.v[i], yv.v[i], acc);
      ss[0] = sum2(acc);
      row_sum<1, kC>(ss, sm, turn, rank);
      f *= rms_factor(ss[0], inv_h, P.eps);
    }
    uint64_t acc = 0;
    const uint64_t ff = both(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hv.v[i] = fma2(a.v[i], mul2(yv.v[i], ff), hv.v[i]);
      acc = fma2(hv.v[i], hv.v[i], acc);
    }
    if (in) put8<kF32>(h_at, hv);
    h_at += src.step_bytes;
    ss[0] = sum2(acc);
    row_sum<1, kC>(ss, sm, turn, rank);
    const uint64_t r1 = both(rms_factor(ss[0], inv_h, P.eps));
#pragma unroll
    for (int i = 0; i < 4; ++i) hv.v[i] = mul2(pw.v[i], mul2(hv.v[i], r1));
    if constexpr (kQuant) {
      // 16 lanes hold a 1x128 group (a CTA's columns are whole groups: a half-warp is all in or all out)
      float v[8], amax = 0.f;
      values_of(hv, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float sc;
      uint32_t c[2];
      quantize8(v, amax, sc, c);
      if (in) {
        fp8g::quant::store_code_words(q_at, c);
        if ((threadIdx.x & 15) == 0) *sa_at = sc;
      }
      q_at += step * S.H;
      sa_at += step;
    } else {
      if (in) put8<kF32>(z_at, hv);
      z_at += src.step_bytes;
    }
  }
}

// Backward.  Each cluster walks its rows and keeps, per column, the two sums
// over rows that all parameter gradients come from: dz n and dh u (with the
// gate per token: g dh u).  They leave as one partial row per cluster,
// part[2][clusters][H], which norm_param_grad_kernel adds in a fixed order (no
// atomics: the same bits every run).
// kThreads: 896 (72 registers a thread, enough for its sums, parameters and
// values) or 1024.
template <bool kF32, int kC, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_residual_backward_kernel(const void* dz, const void* dh_out, const void* h,
                                                                      const void* y, Shape S, Params P, void* dh, void* dy,
                                                                      float* __restrict__ dgate, float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowSum<4, kC> sm4;
  __shared__ RowSum<1, kC> sm1;
  constexpr int D = kBackwardStages;
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long row0 = blockIdx.x / kC, step = gridDim.x / kC;
  const int col0 = rank * S.cols, col = col0 + 8 * threadIdx.x;
  const bool in = 8 * static_cast<int>(threadIdx.x) < S.cols && col < S.H;
  Stream<kF32, 4, D> src;
  src.init({h, y, dz, dh_out}, dyn, S, col0, in, row0, step);
#pragma unroll
  for (int s = 0; s < D - 1; ++s) src.fetch(S.rows, step);
  const long first = (row0 * S.H + col) * (src.kVec / 8);
  uint8_t *dh_at = static_cast<uint8_t*>(dh) + first, *dy_at = static_cast<uint8_t*>(dy) + first;
  Pair8 pw;
  // s post_w (g per channel), used once a row: kept in shared memory, which
  // leaves the registers to what every phase needs
  const uint32_t a_at = src.slot - threadIdx.x * src.kVec + D * src.stage_bytes + threadIdx.x * 32;
  {
    Pair8 a;
    column_params(P, col, in, pw, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) a.v[i] = mul2(a.v[i], both(P.scale));
    float v[8];
    values_of(a, v);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      fp8g::st_shared_v4(a_at + 16 * i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                   __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
  }
  if constexpr (kC > 1) cluster_sync_all();
  const float inv_h = 1.f / static_cast<float>(S.H);
  const bool token = P.gate_kind == FP8G_GATE_TOKEN;
  Pair8 acc_pre = {}, acc_u = {};
  int turn4 = 0, turn1 = 0;
  for (long row = row0; row < S.rows; row += step) {
    src.fetch(S.rows, step);
    cp_wait<D - 1>();
    const Pair8 hv = src.get(0);
    Pair8 yv = src.get(1), g = src.get(2);  // g: dz, then dh, then du
    uint64_t hh = 0, dn = 0, yy = 0;              // h'^2, (dz pre_w) h', y^2
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hh = fma2(hv.v[i], hv.v[i], hh);
      dn = fma2(mul2(g.v[i], pw.v[i]), hv.v[i], dn);
      yy = fma2(yv.v[i], yv.v[i], yy);
    }
    float st[4] = {sum2(hh), sum2(dn), sum2(yy), 0.f};
    row_sum<4, kC>(st, sm4, turn4, rank);
    const float r1 = rms_factor(st[0], inv_h, P.eps);
    const float r2 = P.post_w ? rms_factor(st[2], inv_h, P.eps) : 1.f;
    const float gt = token ? __ldg(P.gate + row) : 1.f;
    const Pair8 t = src.get(3);
    src.advance();
    const uint64_t rr1 = both(r1), rr2 = both(r2);
    const uint64_t rm = both(-r1 * (st[1] * r1 * inv_h));  // - r1 <dz pre_w n>
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t n = mul2(hv.v[i], rr1);
      acc_pre.v[i] = fma2(g.v[i], n, acc_pre.v[i]);
      g.v[i] = fma2(n, rm, fma2(mul2(g.v[i], pw.v[i]), rr1, t.v[i]));
    }
    if (in) put8<kF32>(dh_at, g);
    dh_at += src.step_bytes;
    const Pair8 a = pairs_of<true>(load8_shared<true>(a_at));
    uint64_t du_u = 0;  // a dh u
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      yv.v[i] = mul2(yv.v[i], rr2);
      acc_u.v[i] = fma2(token ? mul2(g.v[i], both(gt)) : g.v[i], yv.v[i], acc_u.v[i]);
      g.v[i] = mul2(g.v[i], a.v[i]);
      du_u = fma2(g.v[i], yv.v[i], du_u);
    }
    float m2 = 0.f;  // <du u>
    if (P.post_w || token) {
      float dot[1] = {sum2(du_u)};
      row_sum<1, kC>(dot, sm1, turn1, rank);
      if (P.post_w) m2 = dot[0] * gt * inv_h;
      if (dgate && token && rank == 0 && threadIdx.x == 0) dgate[row] = dot[0];
    }
    const uint64_t f = both(r2 * gt), um = both(-r2 * m2);
#pragma unroll
    for (int i = 0; i < 4; ++i) g.v[i] = fma2(g.v[i], f, mul2(yv.v[i], um));
    if (in) put8<kF32>(dy_at, g);
    dy_at += src.step_bytes;
  }
  if (part && in) {
    float* p = part + row0 * S.H + col;
    float* pu = p + step * S.H;
    float v[8];
    values_of(acc_pre, v);
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    values_of(acc_u, v);
    reinterpret_cast<float4*>(pu)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(pu)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sums of partial rows part[2][P][H] over P.  A CTA takes 32 columns and the
// partial rows of its blockIdx.y: its 8 warps every eighth row each, 8 loads
// at a time, then the warps' sums in warp order.  Many partial rows (narrow
// rows have many CTAs) are summed in two launches: to out[2][gridDim.y][H]
// first, then to the gradients (kLast).
template <bool kLast>
__global__ void __launch_bounds__(256) norm_param_grad_kernel(const float* __restrict__ part, int P, int H, int per,
                                                              float* __restrict__ out, Params prm, float* dpre,
                                                              float* dpost, float* dgate) {
  __shared__ float s[2][8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int p0 = blockIdx.y * per, p1 = min(P, p0 + per);
  float a = 0.f, b = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int p = p0 + w; p < p1; p += 8) {
      a += part[static_cast<long>(p) * H + col];
      b += part[(static_cast<long>(P) + p) * H + col];
    }
  }
  s[0][w][lane] = a;
  s[1][w][lane] = b;
  __syncthreads();
  if (w != 0 || col >= H) return;
  a = b = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a += s[0][i][lane], b += s[1][i][lane];
  if constexpr (kLast) {
    const bool channel = prm.gate_kind == FP8G_GATE_CHANNEL;
    if (dpre) dpre[col] = a;
    if (dpost) dpost[col] = prm.scale * (channel ? prm.gate[col] : 1.f) * b;
    if (dgate && channel) dgate[col] = prm.scale * (prm.post_w ? prm.post_w[col] : 1.f) * b;
  } else {
    out[static_cast<long>(blockIdx.y) * H + col] = a;
    out[(static_cast<long>(gridDim.y) + blockIdx.y) * H + col] = b;
  }
}

constexpr int kPartsPerSum = 64;   // partial rows of a CTA in the first of two launches
constexpr int kOneLaunch = 256;    // up to so many partial rows one launch sums them all

// How a row of H columns is split and how many clusters walk the rows.
struct Plan {
  Shape S;
  int ctas;      // per cluster
  int threads;
  int smem;
  long clusters;
};

constexpr int kSms = 148;
constexpr int kSmemPerSm = 225 << 10;

// tensors: rows streamed per stage.  The cluster grows until a CTA has at most
// 1024 threads and its stages fit the shared memory; narrow rows get as many
// CTAs per SM as 72 registers a thread and their stages allow.
Plan plan_of(int rows, int H, int esz, int tensors, int stages, int unit, int more_per_thread) {
  Plan p{};
  for (p.ctas = 1;; p.ctas *= 2) {
    const int units = (H / unit + p.ctas - 1) / p.ctas;
    p.threads = (units * unit / 8 + 31) / 32 * 32;
    p.S = Shape{rows, H, units * unit, static_cast<uint32_t>(p.threads * 8 * esz)};
    p.smem = tensors * stages * static_cast<int>(p.S.pitch) + more_per_thread * p.threads;
    if (p.ctas == 4 || (p.threads <= 1024 && p.smem <= kSmemPerSm)) break;
  }
  const int per_sm = std::max(1, std::min({32, 896 / p.threads, kSmemPerSm / (p.smem + 1024)}));
  p.clusters = std::max(1L, std::min<long>(rows, static_cast<long>(kSms) * per_sm / p.ctas));
  return p;
}

// Whole 1x128 groups per CTA wherever H has them, so that a row is summed in the
// same order whether it leaves as values or as codes, in either type (1 CTA up
// to H = 8192, 2 above).
Plan forward_plan(int rows, int H, int dtype) {
  return plan_of(rows, H, dtype == FP8G_IN_F32 ? 4 : 2, 2, forward_stages(dtype == FP8G_IN_F32), H % 128 == 0 ? 128 : 8, 0);
}

Plan backward_plan(int rows, int H, int dtype) {
  return plan_of(rows, H, dtype == FP8G_IN_F32 ? 4 : 2, 4, kBackwardStages, 8, 32);
}

// Launches the kernel for the plan's cluster size.
template <typename... KArgs, typename... Args>
cudaError_t launch(const Plan& p, void (*kernel)(KArgs...), cudaStream_t stream, Args... args) {
  if (p.smem > 47 << 10) {
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(p.clusters * p.ctas), 1, 1);
  cfg.blockDim = dim3(p.threads, 1, 1);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int check_rows(int dtype, int rows, int H, const float* gate, int gate_kind, float scale, float eps) {
  if (dtype != FP8G_IN_BF16 && dtype != FP8G_IN_F32) return FP8G_ERR_INVALID_ARG;
  if (rows < 0 || H <= 0 || H > kMaxH) return FP8G_ERR_INVALID_ARG;
  if (gate_kind < FP8G_GATE_NONE || gate_kind > FP8G_GATE_TOKEN || (gate_kind != FP8G_GATE_NONE) != (gate != nullptr))
    return FP8G_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(eps) || !(eps > 0.f)) return FP8G_ERR_INVALID_ARG;
  if (H % 8 != 0) return FP8G_ERR_MISALIGNED;
  return FP8G_OK;
}

bool params_aligned(const float* post_w, const float* gate, int gate_kind, const float* pre_w) {
  return aligned(post_w, 16) && aligned(pre_w, 16) && aligned(gate, gate_kind == FP8G_GATE_CHANNEL ? 16 : 4);
}

}  // namespace

extern "C" int fp8g_norm_residual(const void* y, const void* h, int dtype, int rows, int H, const float* post_w,
                                  const float* gate, int gate_kind, float scale, const float* pre_w, float eps,
                                  void* h_out, void* z, uint8_t* q, float* sa, int ld_sa, cudaStream_t stream) {
  int rc = check_rows(dtype, rows, H, gate, gate_kind, scale, eps);
  if (rc) return rc;
  if ((z != nullptr) == (q != nullptr) && rows > 0) return FP8G_ERR_INVALID_ARG;
  if (q) {
    if (H % 128 != 0 || ld_sa < rows || ld_sa < 1) return FP8G_ERR_INVALID_ARG;
    if (ld_sa % 4 != 0) return FP8G_ERR_MISALIGNED;
  }
  if (rows == 0) return FP8G_OK;
  if (!y || !h_out || (q && !sa)) return FP8G_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(h, 16) || !aligned(h_out, 16) || !aligned(z, 16) || !aligned(q, 16) ||
      (q && !aligned(sa, 16)) || !params_aligned(post_w, gate, gate_kind, pre_w))
    return FP8G_ERR_MISALIGNED;
  const Plan p = forward_plan(rows, H, dtype);
  const Params P{post_w, gate, pre_w, gate_kind, scale, eps};
  auto go = [&](auto kernel) { return launch(p, kernel, stream, y, h, p.S, P, h_out, z, q, sa, ld_sa); };
  cudaError_t e;
  if (dtype == FP8G_IN_F32)
    e = q ? (p.ctas == 1 ? go(norm_residual_kernel<true, 1, true>) : go(norm_residual_kernel<true, 2, true>))
          : (p.ctas == 1 ? go(norm_residual_kernel<true, 1, false>) : go(norm_residual_kernel<true, 2, false>));
  else
    e = q ? (p.ctas == 1 ? go(norm_residual_kernel<false, 1, true>) : go(norm_residual_kernel<false, 2, true>))
          : (p.ctas == 1 ? go(norm_residual_kernel<false, 1, false>) : go(norm_residual_kernel<false, 2, false>));
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

extern "C" size_t fp8g_norm_residual_backward_workspace_bytes(int rows, int H) {
  if (rows < 0 || H <= 0 || H > kMaxH || H % 8 != 0) return 0;
  // the larger of the two types' plans
  const long n = std::max(backward_plan(rows, H, FP8G_IN_BF16).clusters, backward_plan(rows, H, FP8G_IN_F32).clusters);
  const long sums = n > kOneLaunch ? (n + kPartsPerSum - 1) / kPartsPerSum : 0;
  return static_cast<size_t>(2 * (n + sums) * H) * sizeof(float);
}

extern "C" int fp8g_norm_residual_backward(const void* dz, const void* dh_out, const void* h_out, const void* y,
                                           int dtype, int rows, int H, const float* post_w, const float* gate,
                                           int gate_kind, float scale, const float* pre_w, float eps, void* dh, void* dy,
                                           float* dpre_w, float* dpost_w, float* dgate, void* workspace,
                                           size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_rows(dtype, rows, H, gate, gate_kind, scale, eps);
  if (rc) return rc;
  // a gradient of something that is not there
  if ((dpost_w && !post_w) || (dgate && !gate)) return FP8G_ERR_INVALID_ARG;
  const bool params = dpre_w || dpost_w || (dgate && gate_kind == FP8G_GATE_CHANNEL);
  if (params && (!workspace || workspace_bytes < fp8g_norm_residual_backward_workspace_bytes(rows, H)))
    return FP8G_ERR_INVALID_ARG;
  if (rows > 0 && ((!dz && !dh_out) || !h_out || !y || !dh || !dy)) return FP8G_ERR_INVALID_ARG;
  if (!aligned(dz, 16) || !aligned(dh_out, 16) || !aligned(h_out, 16) || !aligned(y, 16) || !aligned(dh, 16) ||
      !aligned(dy, 16) || !aligned(workspace, 16) || !aligned(dpre_w, 4) || !aligned(dpost_w, 4) || !aligned(dgate, 4) ||
      !params_aligned(post_w, gate, gate_kind, pre_w))
    return FP8G_ERR_MISALIGNED;
  if (rows == 0 && !params) return FP8G_OK;
  const Plan p = backward_plan(rows, H, dtype);
  const Params P{post_w, gate, pre_w, gate_kind, scale, eps};
  float* part = params ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    auto go = [&](auto kernel) { return launch(p, kernel, stream, dz, dh_out, h_out, y, p.S, P, dh, dy, dgate, part); };
    cudaError_t e;
    const bool wide = p.threads > 896;
    if (dtype == FP8G_IN_F32)  // a cluster of 2 or 4 has at most 512 threads a CTA
      e = p.ctas == 1   ? go(norm_residual_backward_kernel<true, 1, 896>)
          : p.ctas == 2 ? go(norm_residual_backward_kernel<true, 2, 896>)
                        : go(norm_residual_backward_kernel<true, 4, 896>);
    else if (p.ctas == 1)
      e = wide ? go(norm_residual_backward_kernel<false, 1, 1024>) : go(norm_residual_backward_kernel<false, 1, 896>);
    else
      e = wide ? go(norm_residual_backward_kernel<false, 2, 1024>) : go(norm_residual_backward_kernel<false, 2, 896>);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
  }
  if (params) {
    const unsigned groups = (H + 31) / 32;
    int n = rows > 0 ? static_cast<int>(p.clusters) : 0;
    if (n > kOneLaunch) {
      const int sums = (n + kPartsPerSum - 1) / kPartsPerSum;
      float* out = part + 2L * n * H;
      norm_param_grad_kernel<false><<<dim3(groups, sums), 256, 0, stream>>>(part, n, H, kPartsPerSum, out, P, nullptr, nullptr,
                                                                            nullptr);
      part = out;
      n = sums;
    }
    norm_param_grad_kernel<true><<<groups, 256, 0, stream>>>(part, n, H, n, nullptr, P, dpre_w, dpost_w, dgate);
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}
