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
#include "quant_impl.cuh"
#include "rows.cuh"

namespace {

using namespace fp8g::rows;
using fp8g::cluster_ctarank;
using fp8g::cluster_sync_all;
using fp8g::smem_u32;

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
  uint32_t pitch;  // bytes of one row's part in shared memory
};

struct Params {
  const float *post_w, *gate, *pre_w;
  int gate_kind;
  float scale, eps;
};

// Parameters of columns col .. col + 7: pre_w, and a = post_w times a gate per channel.
__device__ __forceinline__ void column_params(const Params& p, int col, bool in, float (&pw)[8], float (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) pw[i] = a[i] = 1.f;
  if (!in) return;
  if (p.pre_w) load_param8(p.pre_w, col, pw);
  if (p.post_w) load_param8(p.post_w, col, a);
  if (p.gate_kind == FP8G_GATE_CHANNEL) {
    float g[8];
    load_param8(p.gate, col, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= g[i];
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

template <bool kF32, int kC, bool kQuant>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const void* y, const void* h, Shape S, Params P, void* h_out,
                                                             void* z, uint8_t* q, float* sa, int ld_sa) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowSum<1, kC> sm;
  constexpr int D = forward_stages(kF32);
  constexpr int kVec = kF32 ? 32 : 16;  // bytes of 8 elements
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long row0 = blockIdx.x / kC, step = gridDim.x / kC;
  const int local = 8 * threadIdx.x;
  const int col = rank * S.cols + local;
  const bool in = local < S.cols && col < S.H;
  const uint32_t slot = smem_u32(dyn) + threadIdx.x * kVec;  // stage s: y at slot + 2 s pitch, h behind it
  auto fetch = [&](long row, int s) {
    if (in && row < S.rows) {
      copy8<kF32>(slot + 2 * s * S.pitch, y, row * S.H + col);
      if (h) copy8<kF32>(slot + (2 * s + 1) * S.pitch, h, row * S.H + col);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < D - 1; ++s) fetch(row0 + s * step, s);
  float pw[8], a[8];
  column_params(P, col, in, pw, a);
  if constexpr (kC > 1) cluster_sync_all();
  const float inv_h = 1.f / static_cast<float>(S.H);
  int turn = 0, s = 0;
  for (long row = row0; row < S.rows; row += step) {
    fetch(row + (D - 1) * step, s == 0 ? D - 1 : s - 1);
    cp_wait<D - 1>();
    float hv[8], yv[8];
    unpack8<kF32>(in ? load8_shared<kF32>(slot + 2 * s * S.pitch) : zero8<kF32>(), yv);
    unpack8<kF32>(in && h ? load8_shared<kF32>(slot + (2 * s + 1) * S.pitch) : zero8<kF32>(), hv);
    s = s == D - 1 ? 0 : s + 1;
    float f = P.scale;
    if (P.gate_kind == FP8G_GATE_TOKEN) f *= __ldg(P.gate + row);
    float ss[1] = {0.f};
    if (P.post_w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[i], yv[i], ss[0]);
      row_sum<1, kC>(ss, sm, turn, rank);
      f *= rms_factor(ss[0], inv_h, P.eps);
      ss[0] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hv[i] = fmaf(a[i], yv[i] * f, hv[i]);
      ss[0] = fmaf(hv[i], hv[i], ss[0]);
    }
    if (in) store8<kF32>(h_out, row * S.H + col, hv);
    row_sum<1, kC>(ss, sm, turn, rank);
    const float r1 = rms_factor(ss[0], inv_h, P.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) hv[i] = pw[i] * (hv[i] * r1);
    if constexpr (kQuant) {
      // 16 lanes hold a 1x128 group (a CTA's columns are whole groups: a half-warp is all in or all out)
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(hv[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float sc = fp8g::quant::scale_of(amax);
      uint32_t c[2];
      fp8g::quant::encode_group(hv, sc, c);
      if (in) {
        fp8g::quant::store_code_words(q + row * S.H + col, c);
        if ((threadIdx.x & 15) == 0) sa[static_cast<long>(col / 128) * ld_sa + row] = sc;
      }
    } else {
      if (in) store8<kF32>(z, row * S.H + col, hv);
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
  __shared__ RowSum<4, kC> sm3;
  __shared__ RowSum<1, kC> sm1;
  constexpr int D = kBackwardStages;
  constexpr int kVec = kF32 ? 32 : 16;
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long row0 = blockIdx.x / kC, step = gridDim.x / kC;
  const int local = 8 * threadIdx.x;
  const int col = rank * S.cols + local;
  const bool in = local < S.cols && col < S.H;
  const uint32_t slot = smem_u32(dyn) + threadIdx.x * kVec;  // a stage: h, y, dz, dh_out
  auto fetch = [&](long row, int s) {
    if (in && row < S.rows) {
      const uint32_t at = slot + 4 * s * S.pitch;
      const long e = row * S.H + col;
      copy8<kF32>(at, h, e);
      copy8<kF32>(at + S.pitch, y, e);
      if (dz) copy8<kF32>(at + 2 * S.pitch, dz, e);
      if (dh_out) copy8<kF32>(at + 3 * S.pitch, dh_out, e);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < D - 1; ++s) fetch(row0 + s * step, s);
  float pw[8], a[8];
  column_params(P, col, in, pw, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] *= P.scale;
  if constexpr (kC > 1) cluster_sync_all();
  const float inv_h = 1.f / static_cast<float>(S.H);
  float acc_pre[8] = {}, acc_u[8] = {};
  int turn3 = 0, turn1 = 0, s = 0;
  for (long row = row0; row < S.rows; row += step) {
    fetch(row + (D - 1) * step, s == 0 ? D - 1 : s - 1);
    cp_wait<D - 1>();
    const uint32_t at = slot + 4 * s * S.pitch;
    s = s == D - 1 ? 0 : s + 1;
    float st[4] = {0.f, 0.f, 0.f, 0.f};  // h'^2, (dz pre_w) h', y^2
    float hv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, dhv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float yv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
      unpack8<kF32>(load8_shared<kF32>(at), hv);
      unpack8<kF32>(load8_shared<kF32>(at + S.pitch), yv);
      if (dz) unpack8<kF32>(load8_shared<kF32>(at + 2 * S.pitch), dhv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        st[0] = fmaf(hv[i], hv[i], st[0]);
        st[1] = fmaf(dhv[i] * pw[i], hv[i], st[1]);
        st[2] = fmaf(yv[i], yv[i], st[2]);
      }
    }
    row_sum<4, kC>(st, sm3, turn3, rank);
    const float r1 = rms_factor(st[0], inv_h, P.eps);
    const float r2 = P.post_w ? rms_factor(st[2], inv_h, P.eps) : 1.f;
    const float m1 = st[1] * r1 * inv_h;  // <dz pre_w n>
    const float gt = P.gate_kind == FP8G_GATE_TOKEN ? __ldg(P.gate + row) : 1.f;
    float dot[1] = {0.f};  // sum of s a dh u
    if (in) {
      float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (dh_out) unpack8<kF32>(load8_shared<kF32>(at + 3 * S.pitch), t);
      const float rm = -r1 * m1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = hv[i] * r1;
        acc_pre[i] = fmaf(dhv[i], n, acc_pre[i]);
        dhv[i] = fmaf(n, rm, fmaf(dhv[i] * pw[i], r1, t[i]));
      }
      store8<kF32>(dh, row * S.H + col, dhv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        yv[i] *= r2;
        acc_u[i] = fmaf(gt * dhv[i], yv[i], acc_u[i]);
        dhv[i] *= a[i];
        dot[0] = fmaf(dhv[i], yv[i], dot[0]);
      }
    }
    float m2 = 0.f;  // <du u>
    if (P.post_w || P.gate_kind == FP8G_GATE_TOKEN) {
      row_sum<1, kC>(dot, sm1, turn1, rank);
      if (P.post_w) m2 = dot[0] * gt * inv_h;
      if (dgate && P.gate_kind == FP8G_GATE_TOKEN && rank == 0 && threadIdx.x == 0) dgate[row] = dot[0];
    }
    if (in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dhv[i] = r2 * fmaf(dhv[i], gt, -yv[i] * m2);
      store8<kF32>(dy, row * S.H + col, dhv);
    }
  }
  if (part && in) {
    float* p = part + row0 * S.H + col;
    float* pu = p + step * S.H;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      reinterpret_cast<float4*>(p)[i] = make_float4(acc_pre[4 * i], acc_pre[4 * i + 1], acc_pre[4 * i + 2], acc_pre[4 * i + 3]);
      reinterpret_cast<float4*>(pu)[i] = make_float4(acc_u[4 * i], acc_u[4 * i + 1], acc_u[4 * i + 2], acc_u[4 * i + 3]);
    }
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
constexpr int kSmemPerSm = 220 << 10;

// tensors: rows streamed per stage.  The cluster grows until a CTA has at most
// 1024 threads and its stages fit the shared memory; narrow rows get as many
// CTAs per SM as 72 registers a thread and their stages allow.
Plan plan_of(int rows, int H, int esz, int tensors, int stages, int unit) {
  Plan p{};
  for (p.ctas = 1;; p.ctas *= 2) {
    const int units = (H / unit + p.ctas - 1) / p.ctas;
    p.S = Shape{rows, H, units * unit, static_cast<uint32_t>(units * unit * esz)};
    p.threads = (p.S.cols / 8 + 31) / 32 * 32;
    p.smem = tensors * stages * static_cast<int>(p.S.pitch);
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
  return plan_of(rows, H, dtype == FP8G_IN_F32 ? 4 : 2, 2, forward_stages(dtype == FP8G_IN_F32), H % 128 == 0 ? 128 : 8);
}

Plan backward_plan(int rows, int H, int dtype) {
  return plan_of(rows, H, dtype == FP8G_IN_F32 ? 4 : 2, 4, kBackwardStages, 8);
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
