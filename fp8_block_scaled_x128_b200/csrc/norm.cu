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
//
// Times in this file: calls back to back as a program makes them, into outputs of
// their own and for long enough that the power cap acts; "replayed" means the
// same calls in a short CUDA graph at full clock, whose outputs stay in L2 in part.
// Comparisons of two forms are replayed.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fp8gemm.h"
#include "fp8gemm_testing.h"
#include "quant8.cuh"
#include "rows.cuh"

namespace {

using namespace fp8g::rows;
using fp8g::cluster_ctarank;
using fp8g::cluster_sync_all;
using fp8g::quant::quantize8;
using fp8g::st_shared_v4;

constexpr int kMaxH = 16384;

// A row belongs to a cluster of 1, 2 or 4 CTAs, each with a run of its columns;
// a thread has V vectors of 8 columns, blockDim vectors apart.  The rows stream
// through shared memory in two stages: a thread copies its own columns of a later
// row (cp.async) while it works on the current one, without barriers or waits on
// other threads.  More rows under way were slower, not faster (three stages,
// backward: 8192 x 7168 bf16 118.5 us against 115.5, 8192 x 4096 79 against 74).
//
// A row needs a sum before its next row can start, and another one before it
// can end.  The two are exchanged together: while a row waits for its last sum,
// the next row's first sums are taken from its stage, which is read again
// afterwards.  So a row costs one exchange (8192 x 7168 bf16 backward: 131 us
// with two, 115.5 with one).
constexpr int kStages = 2;

struct Shape {
  int rows, H;
  int cols;        // columns of a CTA (the last of a cluster may have fewer)
  uint32_t pitch;  // bytes of one row's part in shared memory (whole vectors of all threads)
};

struct Params {
  const float *post_w, *gate, *pre_w;
  int gate_kind;
  float scale, eps;
  SumWait wait;
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
// thread's slots of a tensor that is not there, and of vectors behind the row's
// end, are zeroed once and never copied to, so the arithmetic needs no
// conditions.  Addresses advance by additions only: with a multiplication per
// row and tensor, a third of the instructions were address arithmetic.
template <bool kF32, int V, int kTensors>
struct Stream {
  uint32_t slot, pitch, put, get;  // this thread's first slot; stages to fill and to read, as offsets
  long fetch_at;                   // bytes from a tensor's start to this thread's columns of the next row to fetch
  long step_bytes;                 // from a CTA's row to its next
  long left;                       // rows that are still to be fetched
  bool in[V];

  static constexpr int kVec = kF32 ? 32 : 16;  // bytes of 8 elements
  // bytes between a thread's vectors
  __device__ __forceinline__ uint32_t apart() const { return blockDim.x * kVec; }

  __device__ __forceinline__ void init(const void* const (&t)[kTensors], const uint8_t* smem, const Shape& S, int col0,
                                       long row0, long step) {
    slot = fp8g::smem_u32(smem) + threadIdx.x * kVec;
    pitch = S.pitch;
    put = get = 0;
    fetch_at = (row0 * S.H + col0) * (kVec / 8) + threadIdx.x * kVec;
    step_bytes = step * S.H * (kVec / 8);
    left = (S.rows - row0 + step - 1) / step;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 8 * (threadIdx.x + v * blockDim.x);
      in[v] = col < S.cols && col0 + col < S.H;
#pragma unroll
      for (int i = 0; i < kTensors; ++i) {
        if (in[v] && t[i]) continue;
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
          const uint32_t at = slot + (s * kTensors + i) * pitch + v * apart();
          st_shared_v4(at, make_uint4(0u, 0u, 0u, 0u));
          if constexpr (kF32) st_shared_v4(at + 16, make_uint4(0u, 0u, 0u, 0u));
        }
      }
    }
  }

  // Copies this thread's part of the next row, if there is one, into the next
  // stage.  The first `always` tensors are there.
  __device__ __forceinline__ void fetch(const void* const (&t)[kTensors], int always) {
    if (left > 0) {
#pragma unroll
      for (int i = 0; i < kTensors; ++i) {
        if (i >= always && !t[i]) continue;
        const uint8_t* p = static_cast<const uint8_t*>(t[i]) + fetch_at;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (in[v]) copy8<kF32>(slot + put + i * pitch + v * apart(), p + v * apart());
      }
    }
    cp_commit();
    --left;
    fetch_at += step_bytes;
    put = put == (kStages - 1) * kTensors * pitch ? 0 : put + kTensors * pitch;
  }

  __device__ __forceinline__ Pair8 load(int tensor, int v) const {
    return pairs_of<kF32>(load8_shared<kF32>(slot + get + tensor * pitch + v * apart()));
  }

  __device__ __forceinline__ void advance() { get = get == (kStages - 1) * kTensors * pitch ? 0 : get + kTensors * pitch; }
};

// Stores a thread's 8 values of a row, rounded once.
template <bool kF32>
__device__ __forceinline__ void put8(void* base, long at, const Pair8& p) {
  float f[8];
  values_of(p, f);
  store8<kF32>(static_cast<uint8_t*>(base) + at, 0, f);
}

// 8 FP32 parameters of a thread's columns in its own slot of shared memory.
__device__ __forceinline__ void keep8(uint32_t at, const Pair8& p) {
  float f[8];
  values_of(p, f);
  st_shared_v4(at, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
  st_shared_v4(at + 16, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
}

__device__ __forceinline__ Pair8 kept8(uint32_t at) { return pairs_of<true>(load8_shared<true>(at)); }

// Most threads of a CTA, and the registers a thread of the backward kernel may
// use (the forward kernel: 64).  They leave nothing to be kept in local memory:
// with the stages in shared memory the L1 cache has a few KB, and six words
// spilled cost 8192 x 7168 some 50 us.
constexpr int kMaxThreads = 512;
constexpr int backward_regs(bool f32, int vecs) { return vecs == 2 ? 128 : f32 ? 88 : 80; }
// Threads of an SM whose registers fit: each of its four parts has 16384.
constexpr int threads_at(int regs) { return 128 * (16384 / (32 * regs)); }

// Forward.  Each element of y and h is read once and each of h' and z written
// once.  8192 x 7168 bf16 with post-norm and channel gate: 80 us, 5.9 TB/s, 0.90 of
// the measured copy bandwidth, replayed 76.7 (32768 x 1024: 47 us, 0.87; 4096 x 16384:
// 94 us, 0.87; 4096 x 7168 FP32: 86 us, 0.83); two CTAs share an SM, so that one
// computes while the other waits for a sum.  With codes out 90 us, 0.70, replayed
// 84: the quantisation adds a third to the instructions.  There 26 warps an SM
// fill 63 % of the issue slots and no one stall leads: of the 10.2 cycles between two
// instructions of a warp 2.3 are shared memory and shuffles, 2.0 fixed latencies,
// 0.7 barriers, 0.6 loads.  One row of 7168, decode's form: 10.5 us a call, 4.3
// replayed: two sums' latencies behind one load.
template <bool kF32, int V, int kC, bool kQuant>
__global__ void __launch_bounds__(kMaxThreads, 2)
    norm_residual_kernel(const void* y, const void* h, Shape S, Params P, void* h_out, void* z, uint8_t* q, float* sa,
                         int ld_sa, uint32_t* err) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ RowSum<2, kC> sm;
  // The next copies are issued behind the row's sum, before its output, and for
  // narrow bf16 rows before the sum (8192 x 7168 76.7 us against 87, 32768 x 1024
  // 50.2 against 45.5; 16384 x 1024 FP32 48.1 against 51)
  constexpr bool kLate = kF32 || V == 2;
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  row_sum_init(sm, rank, P.wait);
  const long row0 = blockIdx.x / kC, step = gridDim.x / kC;
  const int col0 = rank * S.cols;
  const void* const tensors[2] = {y, h};
  Stream<kF32, V, 2> src;
  src.init(tensors, dyn, S, col0, row0, step);
  long at = src.fetch_at;  // this thread's columns of the current row
#pragma unroll
  for (int s = 0; s < kStages; ++s) src.fetch(tensors, 1);
  // post_w (g per channel) stays in shared memory, pre_w in registers
  const uint32_t a_at = fp8g::smem_u32(dyn) + 2 * kStages * S.pitch + threadIdx.x * 32;
  Pair8 pw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    Pair8 a;
    column_params(P, col0 + 8 * (threadIdx.x + v * blockDim.x), src.in[v], pw[v], a);
    keep8(a_at + v * blockDim.x * 32, a);
  }
  if constexpr (kC > 1) cluster_sync_all();
  const float inv_h = 1.f / static_cast<float>(S.H);
  bool gave_up = false;
  unsigned it = 0;
  float st[2] = {};  // y^2 of the next row, h'^2 of the current one
  auto statistics = [&] {
    uint64_t yy = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Pair8 yv = src.load(0, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) yy = fma2(yv.v[i], yv.v[i], yy);
    }
    st[0] = sum2(yy);
  };
  const bool token = P.gate_kind == FP8G_GATE_TOKEN;
  auto next_row = [&] {
    cp_wait<kLate ? 0 : 1>();
    src.advance();
  };
  cp_wait<1>();
  if (P.post_w) {
    statistics();
    row_sum(st, sm, it++, rank, P.wait, gave_up, err);
  }
  for (long row = row0; row < S.rows; row += step, ++it) {
    float f = token ? P.scale * __ldg(P.gate + row) : P.scale;
    if (P.post_w) f *= rms_factor(st[0], inv_h, P.eps);
    const uint64_t ff = both(f);
    uint64_t acc = 0;
    Pair8 hv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hv[v] = src.load(1, v);
      const Pair8 yv = src.load(0, v), a = kept8(a_at + v * blockDim.x * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hv[v].v[i] = fma2(a.v[i], mul2(yv.v[i], ff), hv[v].v[i]);
        acc = fma2(hv[v].v[i], hv[v].v[i], acc);
      }
      if (src.in[v]) put8<kF32>(h_out, at + v * src.apart(), hv[v]);
    }
    // this stage is free; the next row's sum shares the exchange of this row's
    if constexpr (!kLate) src.fetch(tensors, 1);
    if (P.post_w) {
      next_row();
      if (row + step < S.rows) statistics();
    }
    st[1] = sum2(acc);
    row_sum(st, sm, it, rank, P.wait, gave_up, err);
    if (!P.post_w) next_row();
    if constexpr (kLate) src.fetch(tensors, 1);
    // the quantiser takes the negatives of its values
    const float r = rms_factor(st[1], inv_h, P.eps);
    const uint64_t r1 = both(kQuant ? -r : r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) hv[v].v[i] = mul2(pw[v].v[i], mul2(hv[v].v[i], r1));
      if constexpr (kQuant) {
        // 16 lanes hold a 1x128 group (a CTA's columns are whole groups: a half-warp is all in or all out)
        float x[8], amax = 0.f;
        values_of(hv[v], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float sc;
        uint32_t c[2];
        quantize8(hv[v], amax, sc, c);
        if (src.in[v]) {
          // a code's offset in q is its element's: at counts bytes of the input type
          fp8g::quant::store_code_words(q + (at + v * src.apart()) / (src.kVec / 8), c);
          if ((threadIdx.x & 15) == 0)
            sa[static_cast<long>((col0 + 8 * (threadIdx.x + v * blockDim.x)) / 128) * ld_sa + row] = sc;
        }
      } else {
        if (src.in[v]) put8<kF32>(z, at + v * src.apart(), hv[v]);
      }
    }
    at += src.step_bytes;
  }
  if constexpr (kC > 1) sums_leave(gave_up);
}

// Backward.  Each cluster walks its rows and keeps, per column, the two sums
// over rows that all parameter gradients come from: dz n and dh u (with the
// gate per token: g dh u).  They leave as one partial row per cluster,
// part[2][clusters][H], which norm_param_grad_kernel adds in a fixed order (no
// atomics: the same bits every run).  Those sums belong to columns, so a thread
// has to keep its columns for all rows, and a row takes the whole CTA.
//
// dh needs the row's statistics, and dy a sum over the row of a dh u, which is
// exchanged with the next row's statistics.
//
// 8192 x 7168 bf16: 130 us with the parameter sums, 5.4 TB/s, 0.83 of the measured
// copy bandwidth, replayed 116, 0.93 (8192 x 8192: 140 us, 0.88; 32768 x 1024: 82 us,
// 0.75; 4096 x 16384: 156 us, 0.79; 4096 x 7168 FP32: 138 us, 0.78; 4096 x 16384
// FP32: 334 us, 0.74), at 14 warps an SM of 128 registers.  A few rows are bound by
// latency: 1021 x 2112 FP32, 23 us a call and 19.4 replayed, has 9 warps an SM that
// issue in 21 % of the cycles and wait for shared memory and loads 6 cycles of 10,
// with 108 SMs at 8 rows and 40 at 4, and then the parameter sums on 66 CTAs
// (7 us with cold caches).  400 x 2112 FP32: 12.8 us replayed.
template <bool kF32, int V, int kC>
__global__ void __maxnreg__(backward_regs(kF32, V))
    norm_residual_backward_kernel(const void* dz, const void* dh_out, const void* h, const void* y, Shape S, Params P,
                                  void* dh, void* dy, float* __restrict__ dgate, float* __restrict__ part, uint32_t* err) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ RowSum<4, kC> sm;
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  row_sum_init(sm, rank, P.wait);
  const long row0 = blockIdx.x / kC, step = gridDim.x / kC;
  const int col0 = rank * S.cols;
  const void* const tensors[4] = {h, y, dz, dh_out};
  Stream<kF32, V, 4> src;
  src.init(tensors, dyn, S, col0, row0, step);
  long at = src.fetch_at;
#pragma unroll
  for (int s = 0; s < kStages; ++s) src.fetch(tensors, 2);
  // a = s post_w (g per channel) stays in shared memory, pre_w and the sums in registers
  const uint32_t a_at = fp8g::smem_u32(dyn) + 4 * kStages * S.pitch + threadIdx.x * 32;
  Pair8 pre[V], acc_pre[V] = {}, acc_u[V] = {};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    Pair8 a;
    column_params(P, col0 + 8 * (threadIdx.x + v * blockDim.x), src.in[v], pre[v], a);
#pragma unroll
    for (int i = 0; i < 4; ++i) a.v[i] = mul2(a.v[i], both(P.scale));
    keep8(a_at + v * blockDim.x * 32, a);
  }
  if constexpr (kC > 1) cluster_sync_all();
  if (threadIdx.x == 0) fp8g::grid_launch_dependents();  // the kernel that adds the partial rows waits for this one
  const float inv_h = 1.f / static_cast<float>(S.H);
  const bool token = P.gate_kind == FP8G_GATE_TOKEN;
  bool gave_up = false;
  unsigned it = 0;
  float st[4] = {};  // h'^2, dn h', y^2 of the next row, with dn = dz pre_w; a dh u of the current one
  auto statistics = [&] {
    uint64_t hh = 0, nh = 0, yy = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Pair8 hv = src.load(0, v), yv = src.load(1, v), z = src.load(2, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hh = fma2(hv.v[i], hv.v[i], hh);
        nh = fma2(mul2(z.v[i], pre[v].v[i]), hv.v[i], nh);
        yy = fma2(yv.v[i], yv.v[i], yy);
      }
    }
    st[0] = sum2(hh), st[1] = sum2(nh), st[2] = sum2(yy);
  };
  cp_wait<1>();
  statistics();
  row_sum(st, sm, it++, rank, P.wait, gave_up, err);
  for (long row = row0; row < S.rows; row += step, ++it) {
    const float gt = token ? __ldg(P.gate + row) : 1.f;
    const float r1 = rms_factor(st[0], inv_h, P.eps);
    const float r2 = P.post_w ? rms_factor(st[2], inv_h, P.eps) : 1.f;
    const uint64_t rr1 = both(r1), rr2 = both(r2), rm = both(-r1 * (st[1] * r1 * inv_h));  // - r1 <dn n>, n = h' r1
    Pair8 u[V], g[V];  // g: dh, then a dh
    uint64_t du_u = 0;  // a dh u
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Pair8 hv = src.load(0, v), yv = src.load(1, v), z = src.load(2, v), d = src.load(3, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t n = mul2(hv.v[i], rr1);
        acc_pre[v].v[i] = fma2(z.v[i], n, acc_pre[v].v[i]);
        g[v].v[i] = fma2(n, rm, fma2(mul2(z.v[i], pre[v].v[i]), rr1, d.v[i]));
      }
      if (src.in[v]) put8<kF32>(dh, at + v * src.apart(), g[v]);
      const Pair8 a = kept8(a_at + v * blockDim.x * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[v].v[i] = mul2(yv.v[i], rr2);
        acc_u[v].v[i] = fma2(token ? mul2(g[v].v[i], both(gt)) : g[v].v[i], u[v].v[i], acc_u[v].v[i]);
        g[v].v[i] = mul2(g[v].v[i], a.v[i]);
        du_u = fma2(g[v].v[i], u[v].v[i], du_u);
      }
    }
    // this stage is free; the next row's statistics share the exchange of this row's sum
    src.fetch(tensors, 2);
    cp_wait<1>();
    src.advance();
    if (row + step < S.rows) statistics();
    st[3] = sum2(du_u);
    row_sum(st, sm, it, rank, P.wait, gave_up, err);
    const float m2 = P.post_w ? st[3] * gt * inv_h : 0.f;  // <du u>
    if (dgate && token && rank == 0 && threadIdx.x == 0) dgate[row] = st[3];
    const uint64_t f = both(r2 * gt), um = both(-r2 * m2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) g[v].v[i] = fma2(g[v].v[i], f, mul2(u[v].v[i], um));
      if (src.in[v]) put8<kF32>(dy, at + v * src.apart(), g[v]);
    }
    at += src.step_bytes;
  }
  if (part) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!src.in[v]) continue;
      float* p = part + row0 * S.H + col0 + 8 * (threadIdx.x + v * blockDim.x);
      float* pu = p + step * S.H;
      float x[8];
      values_of(acc_pre[v], x);
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
      values_of(acc_u[v], x);
      reinterpret_cast<float4*>(pu)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(pu)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
  if constexpr (kC > 1) sums_leave(gave_up);
}

// Sums of partial rows part[2][P][H] over P.  A CTA takes 32 columns and the
// partial rows of its blockIdx.y: its 32 warps every 32nd row each, 4 loads
// at a time, then the warps' sums in warp order (8192 x 7168, 148 partial rows:
// latency of one or two rounds of loads).  Many partial rows (narrow
// rows have many CTAs) are summed in two launches: to out[2][gridDim.y][H]
// first, then to the gradients (kLast).  part is read by coherent loads: this kernel
// starts while the one that writes it still runs.
constexpr int kSumWarps = 32;

template <bool kLast>
__global__ void __launch_bounds__(32 * kSumWarps, 2) norm_param_grad_kernel(const float* part, int P, int H, int per,
                                                              float* __restrict__ out, Params prm, float* dpre,
                                                              float* dpost, float* dgate) {
  __shared__ float s[2][kSumWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int p0 = blockIdx.y * per, p1 = min(P, p0 + per);
  float a = 0.f, b = 0.f;
  fp8g::grid_dependency_wait();  // launched while the kernel that writes part still runs
  if (col < H) {
    for (int p = p0 + w; p < p1; p += 4 * kSumWarps) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = p + i * kSumWarps;
        x[i] = q < p1 ? __ldcg(part + static_cast<long>(q) * H + col) : 0.f;
        y[i] = q < p1 ? __ldcg(part + (static_cast<long>(P) + q) * H + col) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) a += x[i], b += y[i];
    }
  }
  s[0][w][lane] = a;
  s[1][w][lane] = b;
  __syncthreads();
  if (w != 0 || col >= H) return;
  a = b = 0.f;
#pragma unroll
  for (int i = 0; i < kSumWarps; ++i) a += s[0][i][lane], b += s[1][i][lane];
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

constexpr int kPartsPerSum = 128;  // partial rows of a CTA in the first of two launches
constexpr int kOneLaunch = 256;   // up to so many partial rows one launch sums them all

// How a row of H columns is split and how many clusters walk the rows.
struct Plan {
  Shape S;
  int vecs;      // vectors of 8 columns per thread
  int ctas;      // per cluster
  int threads;
  int smem;
  long clusters;
  long limit;  // clusters never exceed it, and it does not fall as the rows grow
};

constexpr int kSms = 148;
constexpr int kSmemPerSm = 224 << 10;  // of 227 KB: the static part takes up to 2.2 KB
// Rows up to so many columns get one vector a thread, wider ones two, so that half
// the warps carry the per-row work (backward of 8192 x 3000 bf16 64 us with one
// vector, 59 with two; forward of 8192 x 2048 FP32 45 us with one, 48 with two).
constexpr int kNarrow = 2048;

// tensors: rows streamed per stage.  The cluster grows until a CTA has at most
// kMaxThreads and its stages fit the shared memory; as many CTAs per SM as the
// registers of `sm_threads` threads and the stages allow.
Plan plan_of(int rows, int H, int esz, int tensors, int unit, int vecs, int sm_threads, long most_clusters) {
  Plan p{};
  p.vecs = vecs;
  for (p.ctas = 1;; p.ctas *= 2) {
    const int cols = ((H + unit - 1) / unit + p.ctas - 1) / p.ctas * unit;
    p.threads = (cols / 8 + 32 * vecs - 1) / (32 * vecs) * 32;
    p.S = Shape{rows, H, cols, static_cast<uint32_t>(p.threads * vecs * 8 * esz)};
    p.smem = tensors * kStages * static_cast<int>(p.S.pitch) + 32 * vecs * p.threads;
    if (p.ctas == 4 || (p.threads <= std::min(kMaxThreads, sm_threads) && p.smem <= kSmemPerSm)) break;
  }
  const int per_sm = std::max(1, std::min({32, sm_threads / p.threads, kSmemPerSm / p.smem}));
  // no more clusters than rows, and no more than it takes for all to have the
  // same number of rows or one less
  const long most = std::max(1L, std::min(static_cast<long>(kSms) * per_sm / p.ctas, most_clusters));
  const long rounds = std::max(1L, (rows + most - 1) / most);
  p.limit = std::max(1L, std::min(static_cast<long>(rows), most));
  p.clusters = std::max(1L, (rows + rounds - 1) / rounds);
  return p;
}

// Whole 1x128 groups per CTA wherever H has them, so that a row is summed in the
// same order whether it leaves as values or as codes, in either type (1 CTA up
// to H = 8192, 2 above).
Plan forward_plan(int rows, int H, int dtype) {
  const bool f32 = dtype == FP8G_IN_F32;
  const int vecs = H <= kNarrow ? 1 : 2;
  return plan_of(rows, H, f32 ? 4 : 2, 2, H % 128 == 0 ? 128 : 8, vecs, threads_at(64), LONG_MAX);
}

// At least 4 rows a cluster once one launch could not add the partial rows of all
// (1000 x 512 FP32: 9.2 us against 10.7 with a row each).
Plan backward_plan(int rows, int H, int dtype, long most_clusters = LONG_MAX) {
  const int vecs = H <= kNarrow ? 1 : 2;
  const bool f32 = dtype == FP8G_IN_F32;
  return plan_of(rows, H, f32 ? 4 : 2, 4, 8, vecs, threads_at(backward_regs(f32, vecs)),
                 std::min(most_clusters, std::max<long>(kOneLaunch, rows / 4)));
}

// The launch of a plan; attr is the caller's.
cudaLaunchConfig_t config(const Plan& p, cudaLaunchAttribute* attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.clusters * p.ctas), 1, 1);
  cfg.blockDim = dim3(p.threads, 1, 1);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = p.ctas;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ctas > 1 ? 1 : 0;
  return cfg;
}

// Launches the kernel for the plan's cluster size.
template <typename... KArgs, typename... Args>
cudaError_t launch(const Plan& p, void (*kernel)(KArgs...), cudaStream_t stream, Args... args) {
  const cudaError_t e = fp8g::rows::allow_smem(kernel);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(p, &attr, stream);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Clusters of 4 CTAs that the current device runs at once, 0 if it does not say.
// A quarter of its SMs is too many: a GPC's SMs beyond a multiple of four hold none
// (pairs always fit), and a cluster that does not fit starts when the others have
// walked all their rows (33 fit; 4096 x 16384 FP32: 573 us with 37, 331 with 33).
// All plans of 4 CTAs take an SM for each CTA, so one answer per device serves them.
int quad_clusters(const Plan& p) {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  auto kernel = norm_residual_backward_kernel<true, 2, 4>;
  if (fp8g::rows::allow_smem(kernel) != cudaSuccess) return 0;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(p, &attr, nullptr);
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// test hook (fp8g_testing_withhold_sum)
std::atomic<unsigned> g_test_withhold{kNoCall};
std::atomic<uint32_t> g_test_limit_us{kSumWaitUs};

SumWait sum_wait() {
  return SumWait{g_test_withhold.load(std::memory_order_relaxed), g_test_limit_us.load(std::memory_order_relaxed)};
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
  uint32_t* err = fp8g::device_error_word();
  if (!err) return FP8G_ERR_CUDA;
  const Plan p = forward_plan(rows, H, dtype);
  const Params P{post_w, gate, pre_w, gate_kind, scale, eps, sum_wait()};
  auto go = [&](auto kernel) { return launch(p, kernel, stream, y, h, p.S, P, h_out, z, q, sa, ld_sa, err); };
  auto by_split = [&](auto narrow, auto one, auto two) { return p.vecs == 1 ? go(narrow) : p.ctas == 1 ? go(one) : go(two); };
  cudaError_t e;
  if (dtype == FP8G_IN_F32)
    e = q ? by_split(norm_residual_kernel<true, 1, 1, true>, norm_residual_kernel<true, 2, 1, true>,
                     norm_residual_kernel<true, 2, 2, true>)
          : by_split(norm_residual_kernel<true, 1, 1, false>, norm_residual_kernel<true, 2, 1, false>,
                     norm_residual_kernel<true, 2, 2, false>);
  else
    e = q ? by_split(norm_residual_kernel<false, 1, 1, true>, norm_residual_kernel<false, 2, 1, true>,
                     norm_residual_kernel<false, 2, 2, true>)
          : by_split(norm_residual_kernel<false, 1, 1, false>, norm_residual_kernel<false, 2, 1, false>,
                     norm_residual_kernel<false, 2, 2, false>);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

extern "C" int fp8g_testing_withhold_sum(int call, unsigned wait_limit_us) {
  if (call < 0) {
    g_test_withhold.store(kNoCall, std::memory_order_relaxed);
    g_test_limit_us.store(kSumWaitUs, std::memory_order_relaxed);
    return FP8G_OK;
  }
  if (call > 1 || wait_limit_us < 100 || wait_limit_us > kSumWaitUs) return FP8G_ERR_INVALID_ARG;
  g_test_limit_us.store(wait_limit_us, std::memory_order_relaxed);
  g_test_withhold.store(static_cast<unsigned>(call), std::memory_order_relaxed);
  return FP8G_OK;
}

extern "C" size_t fp8g_norm_residual_backward_workspace_bytes(int rows, int H) {
  if (rows < 0 || H <= 0 || H > kMaxH || H % 8 != 0) return 0;
  // The larger of the two types' limits, not the plan's clusters: those even out the
  // rows of a cluster, so that 148 rows of 7168 have more of them (148) than 8192 (147),
  // and a workspace made for the larger batch would not do for the smaller one.
  const long n = std::max(backward_plan(rows, H, FP8G_IN_BF16).limit, backward_plan(rows, H, FP8G_IN_F32).limit);
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
  uint32_t* err = fp8g::device_error_word();
  if (!err) return FP8G_ERR_CUDA;
  Plan p = backward_plan(rows, H, dtype);
  if (p.ctas == 4) {
    const int fit = quad_clusters(p);
    if (fit < 1) {
      (void)cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
    p = backward_plan(rows, H, dtype, fit);
  }
  const Params P{post_w, gate, pre_w, gate_kind, scale, eps, sum_wait()};
  float* part = params ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    auto go = [&](auto kernel) { return launch(p, kernel, stream, dz, dh_out, h_out, y, p.S, P, dh, dy, dgate, part, err); };
    cudaError_t e;
    if (dtype == FP8G_IN_F32)  // 1 CTA up to 6144 columns, 2 up to 12288
      e = p.vecs == 1   ? go(norm_residual_backward_kernel<true, 1, 1>)
          : p.ctas == 1 ? go(norm_residual_backward_kernel<true, 2, 1>)
          : p.ctas == 2 ? go(norm_residual_backward_kernel<true, 2, 2>)
                        : go(norm_residual_backward_kernel<true, 2, 4>);
    else  // 1 CTA up to 8192 columns, 2 above
      e = p.vecs == 1   ? go(norm_residual_backward_kernel<false, 1, 1>)
          : p.ctas == 1 ? go(norm_residual_backward_kernel<false, 2, 1>)
                        : go(norm_residual_backward_kernel<false, 2, 2>);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
  }
  if (params) {
    const unsigned groups = (H + 31) / 32;
    int n = rows > 0 ? static_cast<int>(p.clusters) : 0;
    cudaError_t e = cudaSuccess;
    if (n > kOneLaunch) {
      const int sums = (n + kPartsPerSum - 1) / kPartsPerSum;
      float* out = part + 2L * n * H;
      e = fp8g::rows::launch_behind(dim3(groups, sums), 32 * kSumWarps, stream, norm_param_grad_kernel<false>, part, n, H,
                                    kPartsPerSum, out, P, nullptr, nullptr, nullptr);
      part = out;
      n = sums;
    }
    if (e == cudaSuccess)
      e = fp8g::rows::launch_behind(dim3(groups), 32 * kSumWarps, stream, norm_param_grad_kernel<true>, part, n, H, n,
                                    nullptr, P, dpre_w, dpost_w, dgate);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  return FP8G_OK;
}
