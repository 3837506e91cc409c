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

constexpr int kMaxH = 16384;

// Threads of a CTA (a row per CTA, 8 columns per thread and vector).
int threads_of(int H, int vecs) { return ((H / 8 + vecs - 1) / vecs + 31) / 32 * 32; }

template <bool kF32, int V, bool kQuant>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const void* y, const void* h, int rows, int H,
                                                             const float* __restrict__ post_w,
                                                             const float* __restrict__ gate, int gate_kind, float scale,
                                                             const float* __restrict__ pre_w, float eps, void* h_out,
                                                             void* z, uint8_t* q, float* sa, int ld_sa) {
  __shared__ BlockSum<1> sm;
  int turn = 0;
  const float inv_h = 1.f / static_cast<float>(H);
  for (long row = blockIdx.x; row < rows; row += gridDim.x) {
    float hv[V][8];
    float ss[1] = {0.f};
    float yv[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
      const bool in = col < H;
      unpack8<kF32>(in ? load8<kF32>(y, row * H + col) : zero8<kF32>(), yv[j]);
      unpack8<kF32>(in && h ? load8<kF32>(h, row * H + col) : zero8<kF32>(), hv[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[j][i], yv[j][i], ss[0]);
    }
    float f = scale;
    if (gate_kind == FP8G_GATE_TOKEN) f *= __ldg(gate + row);
    if (post_w) {
      block_sum<1>(ss, sm, turn);
      f *= 1.f / sqrtf(fmaf(ss[0], inv_h, eps));
    }
    ss[0] = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
      if (col >= H) continue;
      float a[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, t[8];
      if (post_w) load_param8(post_w, col, a);
      if (gate_kind == FP8G_GATE_CHANNEL) {
        load_param8(gate, col, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= t[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hv[j][i] = fmaf(a[i], yv[j][i] * f, hv[j][i]);
        ss[0] = fmaf(hv[j][i], hv[j][i], ss[0]);
      }
      store8<kF32>(h_out, row * H + col, hv[j]);
    }
    block_sum<1>(ss, sm, turn);
    const float r1 = 1.f / sqrtf(fmaf(ss[0], inv_h, eps));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (pre_w && col < H) load_param8(pre_w, col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= hv[j][i] * r1;
      if constexpr (kQuant) {
        // 16 lanes hold a 1x128 group (H % 128 == 0: a half-warp is all in or all out)
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(w[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float sc = fp8g::quant::scale_of(amax);
        uint32_t c[2];
        fp8g::quant::encode_group(w, sc, c);
        if (col < H) {
          fp8g::quant::store_code_words(q + row * H + col, c);
          if ((threadIdx.x & 15) == 0) sa[static_cast<long>(col / 128) * ld_sa + row] = sc;
        }
      } else {
        if (col < H) store8<kF32>(z, row * H + col, w);
      }
    }
  }
}

// Backward.  Each CTA walks its rows and keeps, per column, the two sums over
// rows that all parameter gradients come from: dz n and dh u (with the gate
// per token: g dh u).  They leave as one partial row per CTA, part[2][CTA][H],
// which norm_param_grad_kernel adds in CTA order (no atomics: the same bits
// every run).
template <bool kF32, int V>
__global__ void __launch_bounds__(1024) norm_residual_backward_kernel(
    const void* dz, const void* dh_out, const void* h, const void* y, int rows, int H,
    const float* __restrict__ post_w, const float* __restrict__ gate, int gate_kind, float scale,
    const float* __restrict__ pre_w, float eps, void* dh, void* dy, float* __restrict__ dgate, float* __restrict__ part) {
  __shared__ BlockSum<3> sm3;
  __shared__ BlockSum<1> sm1;
  int turn3 = 0, turn1 = 0;
  const float inv_h = 1.f / static_cast<float>(H);
  float acc_pre[V][8] = {}, acc_u[V][8] = {};
  for (long row = blockIdx.x; row < rows; row += gridDim.x) {
    float st[3] = {0.f, 0.f, 0.f};  // h'^2, (dz w_pre) h', y^2
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
      if (col >= H) continue;
      float hv[8], yv[8];
      unpack8<kF32>(load8<kF32>(h, row * H + col), hv);
      unpack8<kF32>(load8<kF32>(y, row * H + col), yv);
#pragma unroll
      for (int i = 0; i < 8; ++i) st[0] = fmaf(hv[i], hv[i], st[0]), st[2] = fmaf(yv[i], yv[i], st[2]);
      if (dz) {
        float d[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        unpack8<kF32>(load8<kF32>(dz, row * H + col), d);
        if (pre_w) load_param8(pre_w, col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) st[1] = fmaf(d[i] * w[i], hv[i], st[1]);
      }
    }
    block_sum<3>(st, sm3, turn3);
    const float r1 = 1.f / sqrtf(fmaf(st[0], inv_h, eps));
    const float r2 = post_w ? 1.f / sqrtf(fmaf(st[2], inv_h, eps)) : 1.f;
    const float m1 = st[1] * r1 * inv_h;  // <dz w_pre n>
    const float gt = gate_kind == FP8G_GATE_TOKEN ? __ldg(gate + row) : 1.f;
    float dhv[V][8];
    float dot[1] = {0.f};  // sum of s w_post [g per channel] dh u
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
#pragma unroll
      for (int i = 0; i < 8; ++i) dhv[j][i] = 0.f;
      if (col >= H) continue;
      float t[8];
      if (dh_out) unpack8<kF32>(load8<kF32>(dh_out, row * H + col), dhv[j]);
      if (dz) {
        float hv[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        unpack8<kF32>(load8<kF32>(dz, row * H + col), t);
        unpack8<kF32>(load8<kF32>(h, row * H + col), hv);
        if (pre_w) load_param8(pre_w, col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = hv[i] * r1;
          acc_pre[j][i] = fmaf(t[i], n, acc_pre[j][i]);
          dhv[j][i] = fmaf(r1, fmaf(t[i], w[i], -n * m1), dhv[j][i]);
        }
      }
      store8<kF32>(dh, row * H + col, dhv[j]);
      float a[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, yv[8];
      if (post_w) load_param8(post_w, col, a);
      unpack8<kF32>(load8<kF32>(y, row * H + col), yv);
      if (gate_kind == FP8G_GATE_CHANNEL) {
        load_param8(gate, col, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= t[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot[0] = fmaf(a[i] * scale * dhv[j][i], yv[i] * r2, dot[0]);
        acc_u[j][i] = fmaf(gt * dhv[j][i], yv[i] * r2, acc_u[j][i]);
      }
    }
    float m2 = 0.f;  // <du u>
    if (post_w || gate_kind == FP8G_GATE_TOKEN) {
      block_sum<1>(dot, sm1, turn1);
      if (post_w) m2 = dot[0] * gt * inv_h;
      if (dgate && gate_kind == FP8G_GATE_TOKEN && threadIdx.x == 0) dgate[row] = dot[0];
    }
    const float f = scale * gt;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
      if (col >= H) continue;
      float a[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, t[8], yv[8];
      if (post_w) load_param8(post_w, col, a);
      unpack8<kF32>(load8<kF32>(y, row * H + col), yv);
      if (gate_kind == FP8G_GATE_CHANNEL) {
        load_param8(gate, col, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= t[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = r2 * fmaf(a[i] * f, dhv[j][i], -(yv[i] * r2) * m2);
      store8<kF32>(dy, row * H + col, t);
    }
  }
  if (part) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = 8 * (threadIdx.x + j * blockDim.x);
      if (col >= H) continue;
      float* p = part + static_cast<long>(blockIdx.x) * H + col;
      float* pu = p + static_cast<long>(gridDim.x) * H;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = acc_pre[j][i], pu[i] = acc_u[j][i];
    }
  }
}

// Sums the CTAs' partial rows: a CTA takes 32 columns, its 8 warps every
// eighth partial row each; the warps' sums are added in warp order.
__global__ void __launch_bounds__(256) norm_param_grad_kernel(const float* __restrict__ part, int P, int H,
                                                              const float* __restrict__ post_w,
                                                              const float* __restrict__ gate, int gate_kind, float scale,
                                                              float* dpre, float* dpost, float* dgate) {
  __shared__ float s[2][8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float a = 0.f, b = 0.f;
  if (col < H) {
    for (int p = w; p < P; p += 8) {
      if (dpre) a += part[static_cast<long>(p) * H + col];
      if (dpost || dgate) b += part[static_cast<long>(P + p) * H + col];
    }
  }
  s[0][w][lane] = a;
  s[1][w][lane] = b;
  __syncthreads();
  if (w == 0 && col < H) {
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a += s[0][i][lane], b += s[1][i][lane];
    if (dpre) dpre[col] = a;
    const bool channel = gate_kind == FP8G_GATE_CHANNEL;
    if (dpost) dpost[col] = scale * (channel ? gate[col] : 1.f) * b;
    if (dgate && channel) dgate[col] = scale * (post_w ? post_w[col] : 1.f) * b;
  }
}

// CTAs of the backward kernel for `rows` rows of H: the partial rows of the
// workspace.  148 SMs, more CTAs per SM for narrow rows.
long partials_of(long rows, int H) {
  const long per_sm = std::max(1, std::min(8, 1024 / threads_of(H, H > 8192 ? 2 : 1)));
  return std::max(1L, std::min(rows, 148L * per_sm));
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
  const int sms = sm_count();
  if (sms <= 0) return FP8G_ERR_CUDA;
  const int V = H > 8192 ? 2 : 1;
  const int threads = threads_of(H, V);
  const unsigned grid = static_cast<unsigned>(std::min<long>(rows, static_cast<long>(sms) * std::min(32, 2048 / threads)));
  auto go = [&](auto kernel) {
    kernel<<<grid, threads, 0, stream>>>(y, h, rows, H, post_w, gate, gate_kind, scale, pre_w, eps, h_out, z, q, sa,
                                         ld_sa);
  };
  if (dtype == FP8G_IN_F32) {
    if (q) V == 2 ? go(norm_residual_kernel<true, 2, true>) : go(norm_residual_kernel<true, 1, true>);
    else V == 2 ? go(norm_residual_kernel<true, 2, false>) : go(norm_residual_kernel<true, 1, false>);
  } else {
    if (q) V == 2 ? go(norm_residual_kernel<false, 2, true>) : go(norm_residual_kernel<false, 1, true>);
    else V == 2 ? go(norm_residual_kernel<false, 2, false>) : go(norm_residual_kernel<false, 1, false>);
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}

extern "C" size_t fp8g_norm_residual_backward_workspace_bytes(int rows, int H) {
  if (rows < 0 || H <= 0 || H > kMaxH || H % 8 != 0) return 0;
  return static_cast<size_t>(2 * partials_of(rows, H) * H) * sizeof(float);
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
  const int V = H > 8192 ? 2 : 1;
  const int threads = threads_of(H, V);
  const int P = rows == 0 ? 0 : static_cast<int>(partials_of(rows, H));
  float* part = params ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    auto go = [&](auto kernel) {
      kernel<<<P, threads, 0, stream>>>(dz, dh_out, h_out, y, rows, H, post_w, gate, gate_kind, scale, pre_w, eps, dh,
                                        dy, dgate, part);
    };
    if (dtype == FP8G_IN_F32) V == 2 ? go(norm_residual_backward_kernel<true, 2>) : go(norm_residual_backward_kernel<true, 1>);
    else V == 2 ? go(norm_residual_backward_kernel<false, 2>) : go(norm_residual_backward_kernel<false, 1>);
  }
  if (params)
    norm_param_grad_kernel<<<(H + 31) / 32, 256, 0, stream>>>(part, P, H, post_w, gate, gate_kind, scale, dpre_w,
                                                              dpost_w, dgate);
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}
