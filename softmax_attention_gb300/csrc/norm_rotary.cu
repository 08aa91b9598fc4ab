// norm_rotary.cu -- RMS norms of the queries and keys for each head, with the rotary positions in
// the same pass, and the gradient of both.
//
// With n = x r, r = (mean(x^2) + eps)^(-1/2) and R the rotation of a row's first columns,
//     y = R (n w).
// Of dy, with g = R^T dy:
//     dw = sum over rows of g n,   dx = r (g w - n mean(g w n)) = r (g w - x r^2 mean(g w x)).
// Both are bound by memory: the forward pass reads each row once and writes it once, the gradient
// reads two and writes one.  A row's units, each a lane's two 16-byte pieces (rotary.cuh describes them for
// 16-bit rows; fp32 ones are half as wide), lie in neighbouring lanes of a warp, which trade their
// sums by shuffles; a thread takes the same unit of several heads of one token, with the loads of a
// batch of heads in flight, and its sines once for all of them.
//
// Measured: 16,384 tokens of 40 heads (bf16, D = 128) 60.2 us, 5.6 TB/s, 0.83 of the copy rate; their gradient 108,
// 4.6 TB/s; the gradient of 2 x 1843 tokens of 32 heads (fp32, D = 64) 17.9, 5.1 TB/s, of which 2.7 are the weights'
// sums.  What is left is latency, with sixteen warps an SM: the forward's loads in flight and the gradient's sums
// leave no registers for more (the gradient of 16-bit rows spills a few bytes as it is).  Sums and products go two elements an instruction.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "../../include/fa.h"
#include "dependent.cuh"
#include "internal.h"
#include "rotary.cuh"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 512;
constexpr int kSumThreads = 256;

struct NormParams {
  const void* x[2];        // q, k
  const void* dy[2];       // gradient: of the outputs
  void* y[2];              // the outputs; gradient: of q and k
  int64_t xs[2][3], ds[2][3], ys[2][3];  // batch, head, token strides in elements
  const void* w[2];        // or nullptr: ones
  int w_fp32;
  const int32_t* positions;
  const double* inv_freq;
  float amplitude, eps;
  int H[2], T, D, half, units, rot_units, lanes;  // lanes: of a row
  int heads_per_thread, groups[2];  // head groups of q and of k: no group holds heads of both
  int64_t tokens;
  int blocks[2];           // gradient: blocks of q, then of k
  float* partial;          // gradient: [blocks of q + of k, D]
  float* dw[2];
};

// W elements of a row, as loaded (so that a batch of loads in flight holds no more registers than its bytes).
template <typename T, int W>
struct Raw {
  static constexpr int kWords = W * static_cast<int>(sizeof(T)) / 4;
  uint32_t v[kWords];
};

template <typename T, int W>
__device__ __forceinline__ void load(const T* src, Raw<T, W>& r) {
  if constexpr (Raw<T, W>::kWords == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    r.v[0] = x.x;
    r.v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, W>::kWords / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(src)[i];
      r.v[4 * i] = x.x;
      r.v[4 * i + 1] = x.y;
      r.v[4 * i + 2] = x.z;
      r.v[4 * i + 3] = x.w;
    }
  }
}

template <typename T, int W>
__device__ __forceinline__ void expand(const Raw<T, W>& r, float (&x)[W]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = __uint_as_float(r.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) unpack2<T>(r.v[i], x[2 * i], x[2 * i + 1]);
  }
}

template <typename T, int W>
__device__ __forceinline__ void store(T* dst, const float (&x)[W]) {
  if constexpr (sizeof(T) == 2 && W == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
  } else if constexpr (W == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    store8(dst, x);
  }
}

// The norms' weights in shared memory, as float4 [tensor][four elements of a unit][unit], so that
// neighbouring lanes read neighbouring vectors.
template <typename T, int W, bool INTERLEAVED>
__device__ __forceinline__ void fill_weights(const NormParams& p, int which, float4* w) {
  for (int i = threadIdx.x; i < p.D; i += kThreads) {
    const int u = i / (2 * W), e = i % (2 * W);
    const int col = u < p.rot_units && !INTERLEAVED ? (e < W ? W * u + e : p.half + W * u + e - W) : i;
    float v = 1.f;
    if (p.w[which]) {
      if (p.w_fp32) v = static_cast<const float*>(p.w[which])[col];
      else v = static_cast<float>(static_cast<const T*>(p.w[which])[col]);
    }
    reinterpret_cast<float*>(w + (e / 4) * p.units + u)[e % 4] = v;
  }
}

template <int W>
__device__ __forceinline__ void read_weights(const float4* w, int units, int u, float (&a)[W], float (&b)[W]) {
#pragma unroll
  for (int q = 0; q < W / 2; ++q) {
    const float4 v = w[q * units + u];
    float* to = (q < W / 4 ? a : b) + (q % (W / 4)) * 4;
    to[0] = v.x;
    to[1] = v.y;
    to[2] = v.z;
    to[3] = v.w;
  }
}

// Two elements at a time.
__device__ __forceinline__ float2 two(const float* x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ void put(float* x, float2 v) {
  x[0] = v.x;
  x[1] = v.y;
}

// A unit turned, pairs (a[i], b[i]) of the half layout two at a time.  (In the forward pass over 16-bit rows alone: 16,384
// tokens of 40 heads, D = 128, 60.2 us for 61.2; fp32 rows 116 for 106, the gradient of 16-bit ones, whose registers
// spill, 127 for 108.)
template <int W>
__device__ __forceinline__ void turn_halves(const Angles<W>& t, float (&a)[W], float (&b)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 2) {
    const float2 x = two(a + i), y = two(b + i), c = two(t.c + i), s = two(t.s + i);
    put(a + i, __ffma2_rn(x, c, __fmul2_rn(y, make_float2(-s.x, -s.y))));
    put(b + i, __ffma2_rn(y, c, __fmul2_rn(x, s)));
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Forward.  LANES: lanes of a row, the least power of two that holds its units.  Two blocks an SM that stay: 61.5 us
// for that prompt; a block a task, three an SM, 68; batches of eight heads 67.5, three blocks with batches of two 63.6.
template <typename T, int W, int LANES, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 2) norm_rotary_kernel(const NormParams p) {
  __shared__ int64_t steps[kMaxRot / 2];
  __shared__ float4 weights[2][kMaxD / 4];
  fill_weights<T, W, INTERLEAVED>(p, 0, weights[0]);
  fill_weights<T, W, INTERLEAVED>(p, 1, weights[1]);
  fill_steps(steps, p.inv_freq, p.half);
  constexpr int kSlots = kThreads / LANES;
  const int u = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const bool unit = u < p.units, rotated = u < p.rot_units;
  const int c0 = rotated && !INTERLEAVED ? W * u : 2 * W * u;
  const int c1 = rotated && !INTERLEAVED ? p.half + W * u : 2 * W * u + W;
  const float inv_d = 1.f / p.D;
  const int64_t tasks = p.tokens * (p.groups[0] + p.groups[1]), step = static_cast<int64_t>(gridDim.x) * kSlots;
  constexpr int kBatch = W * sizeof(T) == 16 ? 4 : 2;  // heads whose loads are issued together
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kSlots; base < tasks; base += step) {
    const int64_t task = base + slot;  // the loop's length is the block's: shuffles
    // every lane of a warp takes part in the shuffles, with nothing to load where it has no unit
    const bool live = unit && task < tasks;
    const int group = live ? static_cast<int>(task / p.tokens) : 0;
    const int64_t token = live ? task - group * p.tokens : 0;
    const int which = group < p.groups[0] ? 0 : 1;
    const int h0 = (which ? group - p.groups[0] : group) * p.heads_per_thread;
    const int h1 = live ? min(h0 + p.heads_per_thread, which ? p.H[1] : p.H[0]) : 0;
    const int64_t b = token / p.T, t = token - b * p.T;
    Angles<W> turn;
    if (live && rotated) fill_turn(turn, steps, u, p.positions[token], p.amplitude, false);
    const T* x = static_cast<const T*>(which ? p.x[1] : p.x[0]);
    T* y = static_cast<T*>(which ? p.y[1] : p.y[0]);
    x += which ? b * p.xs[1][0] + t * p.xs[1][2] : b * p.xs[0][0] + t * p.xs[0][2];
    y += which ? b * p.ys[1][0] + t * p.ys[1][2] : b * p.ys[0][0] + t * p.ys[0][2];
    const int64_t xh = which ? p.xs[1][1] : p.xs[0][1], yh = which ? p.ys[1][1] : p.ys[0][1];
    for (int j = 0; j < p.heads_per_thread; j += kBatch) {  // the same count for every lane: shuffles
      Raw<T, W> ra[kBatch], rb[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (h0 + j + i >= h1) continue;
        const T* src = x + (h0 + j + i) * xh;
        load<T, W>(src + c0, ra[i]);
        load<T, W>(src + c1, rb[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool ok = h0 + j + i < h1;
        float a[W] = {}, c[W] = {};
        if (ok) {
          expand<T, W>(ra[i], a);
          expand<T, W>(rb[i], c);
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < W; e += 2) sum = __ffma2_rn(two(a + e), two(a + e), __ffma2_rn(two(c + e), two(c + e), sum));
        const float r = rsqrtf(row_sum<LANES>(sum.x + sum.y) * inv_d + p.eps);
        if (!ok) continue;
        float wa[W], wc[W];
        read_weights<W>(weights[which], p.units, u, wa, wc);
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          put(a + e, __fmul2_rn(two(a + e), __fmul2_rn(make_float2(r, r), two(wa + e))));
          put(c + e, __fmul2_rn(two(c + e), __fmul2_rn(make_float2(r, r), two(wc + e))));
        }
        if (rotated) {
          if constexpr (!INTERLEAVED && sizeof(T) == 2) turn_halves(turn, a, c);
          else rotate<INTERLEAVED>(turn, a, c);
        }
        T* dst = y + (h0 + j + i) * yh;
        store<T, W>(dst + c0, a);
        store<T, W>(dst + c1, c);
      }
    }
  }
}

// Gradient.  A block belongs to q or to k and walks over (token, head group) tasks; a thread adds
// its columns' part of the weight's gradient in registers, the block its rows' parts in a fixed
// order, and weight_sum_kernel the blocks': no atomics.  (The next batch's rows loaded ahead made the registers
// spill: three times as long.)
template <typename T, int W, int LANES, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 2) norm_rotary_grad_kernel(const NormParams p) {
  let_next_start();
  __shared__ int64_t steps[kMaxRot / 2];
  __shared__ float4 weights[kMaxD / 4];
  constexpr int kSlots = kThreads / LANES;
  __shared__ float sums[kSlots * LANES * 2 * W];  // [slot][unit's columns]
  const int which = static_cast<int>(blockIdx.x) < p.blocks[0] ? 0 : 1;
  const int block = which ? blockIdx.x - p.blocks[0] : blockIdx.x;
  fill_weights<T, W, INTERLEAVED>(p, which, weights);
  fill_steps(steps, p.inv_freq, p.half);
  const int u = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const bool unit = u < p.units, rotated = u < p.rot_units;
  const int c0 = rotated && !INTERLEAVED ? W * u : 2 * W * u;
  const int c1 = rotated && !INTERLEAVED ? p.half + W * u : 2 * W * u + W;
  const int H = which ? p.H[1] : p.H[0];
  const int64_t tasks = p.tokens * (which ? p.groups[1] : p.groups[0]);
  const int64_t step = static_cast<int64_t>(which ? p.blocks[1] : p.blocks[0]) * kSlots;
  const T* x0 = static_cast<const T*>(which ? p.x[1] : p.x[0]);
  const T* d0 = static_cast<const T*>(which ? p.dy[1] : p.dy[0]);
  T* y0 = static_cast<T*>(which ? p.y[1] : p.y[0]);
  const int64_t xb = which ? p.xs[1][0] : p.xs[0][0], xh = which ? p.xs[1][1] : p.xs[0][1], xt = which ? p.xs[1][2] : p.xs[0][2];
  const int64_t db = which ? p.ds[1][0] : p.ds[0][0], dh = which ? p.ds[1][1] : p.ds[0][1], dt = which ? p.ds[1][2] : p.ds[0][2];
  const int64_t yb = which ? p.ys[1][0] : p.ys[0][0], yh = which ? p.ys[1][1] : p.ys[0][1], yt = which ? p.ys[1][2] : p.ys[0][2];
  const float inv_d = 1.f / p.D;
  float dwa[W] = {}, dwc[W] = {};
  constexpr int kBatch = W * sizeof(T) == 16 ? 2 : 1;  // heads whose loads are issued together
  for (int64_t base = static_cast<int64_t>(block) * kSlots; base < tasks; base += step) {
    const int64_t task = base + slot;  // the loop's length is the block's: shuffles
    const bool live = unit && task < tasks;
    const int group = live ? static_cast<int>(task / p.tokens) : 0;
    const int64_t token = live ? task - group * p.tokens : 0;
    const int64_t b = token / p.T, t = token - b * p.T;
    const int h0 = group * p.heads_per_thread, h1 = live ? min(h0 + p.heads_per_thread, H) : 0;
    Angles<W> turn;
    if (live && rotated) fill_turn(turn, steps, u, p.positions[token], p.amplitude, true);
    const T* x = x0 + b * xb + t * xt;
    const T* d = d0 + b * db + t * dt;
    T* y = y0 + b * yb + t * yt;
    for (int j = 0; j < p.heads_per_thread; j += kBatch) {
      Raw<T, W> ra[kBatch], rb[kBatch], rg[kBatch], rh[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + j + i;
        if (h >= h1) continue;
        load<T, W>(x + h * xh + c0, ra[i]);
        load<T, W>(x + h * xh + c1, rb[i]);
        load<T, W>(d + h * dh + c0, rg[i]);
        load<T, W>(d + h * dh + c1, rh[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + j + i;
        const bool ok = h < h1;
        float a[W] = {}, c[W] = {}, g[W] = {}, f[W] = {}, wa[W] = {}, wc[W] = {};
        if (ok) {
          expand<T, W>(ra[i], a);
          expand<T, W>(rb[i], c);
          expand<T, W>(rg[i], g);
          expand<T, W>(rh[i], f);
          if (rotated) rotate<INTERLEAVED>(turn, g, f);
          read_weights<W>(weights, p.units, u, wa, wc);
        }
        float2 x2 = make_float2(0.f, 0.f), g2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          x2 = __ffma2_rn(two(a + e), two(a + e), __ffma2_rn(two(c + e), two(c + e), x2));
          g2 = __ffma2_rn(__fmul2_rn(two(g + e), two(wa + e)), two(a + e),
                          __ffma2_rn(__fmul2_rn(two(f + e), two(wc + e)), two(c + e), g2));
        }
        const float xx = row_sum<LANES>(x2.x + x2.y), gx = row_sum<LANES>(g2.x + g2.y);
        if (!ok) continue;
        const float r = rsqrtf(xx * inv_d + p.eps);
        const float back = -r * r * gx * inv_d;
        const float2 r2 = make_float2(r, r), back2 = make_float2(back, back);
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          put(dwa + e, __ffma2_rn(two(g + e), __fmul2_rn(two(a + e), r2), two(dwa + e)));
          put(dwc + e, __ffma2_rn(two(f + e), __fmul2_rn(two(c + e), r2), two(dwc + e)));
          put(a + e, __fmul2_rn(r2, __ffma2_rn(two(a + e), back2, __fmul2_rn(two(g + e), two(wa + e)))));
          put(c + e, __fmul2_rn(r2, __ffma2_rn(two(c + e), back2, __fmul2_rn(two(f + e), two(wc + e)))));
        }
        store<T, W>(y + h * yh + c0, a);
        store<T, W>(y + h * yh + c1, c);
      }
    }
  }
  float* mine = sums + (slot * LANES + u) * 2 * W;
#pragma unroll
  for (int e = 0; e < W; ++e) {
    mine[e] = dwa[e];
    mine[W + e] = dwc[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.D; i += kThreads) {
    const int un = i / (2 * W), e = i % (2 * W);
    const int col = un < p.rot_units && !INTERLEAVED ? (e < W ? W * un + e : p.half + W * un + e - W) : i;
    float v = 0.f;
    for (int s = 0; s < kSlots; ++s) v += sums[s * LANES * 2 * W + i];
    p.partial[static_cast<int64_t>(blockIdx.x) * p.D + col] = v;
  }
}

// The blocks' parts of the weights' gradients: block = (32 columns, tensor), eight threads a column.  2.7 us of a
// call, latency (1024 threads a block: alike).
__global__ void __launch_bounds__(kSumThreads) weight_sum_kernel(const NormParams p) {
  wait_for_previous();
  __shared__ float part[8][32];
  const int which = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
  const int n = which ? p.blocks[1] : p.blocks[0];
  const float* src = p.partial + (which ? static_cast<int64_t>(p.blocks[0]) * p.D : 0);
  float v = 0.f;
  if (c < p.D) {
#pragma unroll 8
    for (int i = k; i < n; i += 8) v += src[static_cast<int64_t>(i) * p.D + c];
  }
  part[k][threadIdx.x % 32] = v;
  __syncthreads();
  float* to = which ? p.dw[1] : p.dw[0];
  if (k == 0 && c < p.D && to) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += part[i][threadIdx.x];
    to[c] = v;
  }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
int bad(int code, const char* who, const char* msg) {
  char text[240];
  snprintf(text, sizeof text, "%s: %s", who, msg);
  return set_error(code, text);
}
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

struct NormCall {  // the fields that both calls have
  int B, T, Hq, Hk, D, rot_dim;
  const int32_t* positions;
  const double* inv_freq;
  const void* q_weight;
  const void* k_weight;
  float amplitude, eps;
  fa_dtype dtype, weight_dtype;
};

bool is_type(fa_dtype t) { return t == FA_BF16 || t == FA_FP16 || t == FA_FP32; }

int check_call(const char* who, const NormCall& a) {
  if (a.B < 0 || a.T < 0 || a.Hq < 0 || a.Hk < 0) return bad(FA_ERR_INVALID_ARG, who, "need B, T, Hq, Hk >= 0");
  if (a.Hq > 65535 || a.Hk > 65535 || static_cast<int64_t>(a.B) * a.T > (1LL << 40))
    return bad(FA_ERR_UNSUPPORTED, who, "Hq and Hk must be <= 65535, B * T <= 2^40");
  if (a.D <= 0 || a.D % 16 != 0 || a.D > kMaxD)
    return bad(FA_ERR_UNSUPPORTED, who, "D must be a multiple of 16 in [16, 512]");
  if (a.rot_dim < 0 || a.rot_dim % 16 != 0 || a.rot_dim > a.D)
    return bad(FA_ERR_UNSUPPORTED, who, "rot_dim must be a multiple of 16 in [0, D]");
  if (!is_type(a.dtype)) return bad(FA_ERR_UNSUPPORTED, who, "dtype must be FA_BF16, FA_FP16 or FA_FP32");
  if (a.weight_dtype != a.dtype && a.weight_dtype != FA_FP32)
    return bad(FA_ERR_UNSUPPORTED, who, "the weights must be in dtype or FA_FP32");
  if (!isfinite(a.amplitude)) return bad(FA_ERR_INVALID_ARG, who, "amplitude must be finite");
  if (!(a.eps >= 0.f) || !isfinite(a.eps)) return bad(FA_ERR_INVALID_ARG, who, "eps must be finite and >= 0");
  return FA_OK;
}

// Address and strides of q or k (or of an output, whose rows must not overlap).
int check_rows(const char* who, const void* base, const int64_t* s, const NormCall& a, int H, bool output) {
  if (H == 0) return FA_OK;
  if (!base) return bad(FA_ERR_INVALID_ARG, who, "null pointer");
  const int64_t m = a.dtype == FA_FP32 ? 4 : 8;
  if (!aligned(base, 16) || s[0] % m != 0 || s[1] % m != 0 || s[2] % m != 0)
    return bad(FA_ERR_INVALID_ARG, who, "tensors must be 16-byte aligned, their strides multiples of 16 bytes");
  const int n[3] = {a.B, H, a.T};
  for (int i = 0; output && i < 3; ++i)
    if (n[i] > 1 && s[i] < a.D && s[i] > -a.D)
      return bad(FA_ERR_INVALID_ARG, who, "rows of an output overlap (a broadcast tensor cannot be one)");
  return FA_OK;
}

int check_tables(const char* who, const NormCall& a) {
  if (a.rot_dim > 0 && (!a.positions || !a.inv_freq)) return bad(FA_ERR_INVALID_ARG, who, "null positions or inv_freq");
  const int w = a.weight_dtype == FA_FP32 ? 4 : 2;
  if (!aligned(a.positions, 4) || !aligned(a.inv_freq, 8) || !aligned(a.q_weight, w) || !aligned(a.k_weight, w))
    return bad(FA_ERR_INVALID_ARG, who, "misaligned positions, inv_freq or weights");
  return FA_OK;
}

int sms() { return num_sms() > 0 ? num_sms() : 152; }

// Width of half a unit: 16 bytes, for fp32 rows that a warp holds that way.  (2 x 1843 tokens of 32 heads, D = 64: fp32
// with eight 26.0 us for 18.0 with four, forward 14.7 for 11.0; 16,384 tokens of 40 heads, D = 128: bf16 with eight 112
// for 117 with four, forward 64 for 68.)
int width(const NormCall& a) { return a.dtype == FA_FP32 && a.D <= 256 ? 4 : 8; }

int row_lanes(int D, int w) {
  int lanes = 1;
  while (lanes * 2 * w < D) lanes *= 2;
  return lanes;
}

// Heads a thread takes: as many as eight, so that its eight sines serve them all, but no more than leave every SM 512
// threads (128 tokens of 40 heads: 4.9 us with one a thread, 6.2 with eight; 16,384 tokens: 61.3 with eight, 67 with
// four, 176 with one, 63.6 with sixteen).
void fill_params(NormParams& p, const NormCall& a) {
  const int w = width(a), lanes = row_lanes(a.D, w);
  p.w[0] = a.q_weight;
  p.w[1] = a.k_weight;
  p.w_fp32 = a.weight_dtype == FA_FP32;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.amplitude = a.amplitude;
  p.eps = a.eps;
  p.H[0] = a.Hq;
  p.H[1] = a.Hk;
  p.T = a.T;
  p.D = a.D;
  p.half = a.rot_dim / 2;
  p.lanes = lanes;
  p.units = a.D / (2 * w);
  p.rot_units = a.rot_dim / (2 * w);
  p.tokens = static_cast<int64_t>(a.B) * a.T;
  int hpt = 8;
  while (hpt > 1 && p.tokens * lanes * ((a.Hq + a.Hk + hpt - 1) / hpt) < 512LL * sms()) hpt /= 2;
  p.heads_per_thread = hpt;
  p.groups[0] = (a.Hq + hpt - 1) / hpt;
  p.groups[1] = (a.Hk + hpt - 1) / hpt;
}

// Blocks of the gradient for q and for k: two an SM at most, shared out by their rows.
void grad_blocks(NormParams& p) {
  const int64_t slots = kThreads / p.lanes;
  const int64_t want[2] = {(p.tokens * p.groups[0] + slots - 1) / slots, (p.tokens * p.groups[1] + slots - 1) / slots};
  const int64_t most = 2LL * sms();
  for (int i = 0; i < 2; ++i) {
    int64_t n = want[0] + want[1] <= most ? want[i] : most * p.H[i] / (p.H[0] + p.H[1]);
    if (n < 1) n = 1;
    p.blocks[i] = static_cast<int>(p.H[i] == 0 ? 0 : n < want[i] ? n : want[i]);
  }
}

template <typename T, int W, int LANES>
cudaError_t launch(const NormParams& p, bool interleaved, bool grad, cudaStream_t st) {
  if (grad) {
    const unsigned n = p.blocks[0] + p.blocks[1];
    if (interleaved) norm_rotary_grad_kernel<T, W, LANES, true><<<n, kThreads, 0, st>>>(p);
    else norm_rotary_grad_kernel<T, W, LANES, false><<<n, kThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(p.dw[0] || p.dw[1])) return e;
    return launch_dependent(weight_sum_kernel, (p.D + 31) / 32, 2, kSumThreads, 0, st, p);
  } else {
    // no more blocks than are resident at once: each fills its tables once
    const int64_t threads = p.tokens * (p.groups[0] + p.groups[1]) * LANES, most = 2LL * sms();
    const int64_t want = (threads + kThreads - 1) / kThreads;
    const unsigned n = static_cast<unsigned>(want < most ? want : most);
    if (interleaved) norm_rotary_kernel<T, W, LANES, true><<<n, kThreads, 0, st>>>(p);
    else norm_rotary_kernel<T, W, LANES, false><<<n, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_lanes(const NormParams& p, bool interleaved, bool grad, cudaStream_t st) {
  if constexpr (W == 8 && sizeof(T) == 4) return launch<T, W, 32>(p, interleaved, grad, st);  // (D > 256 alone)
  if constexpr (W == 8 && sizeof(T) == 2)
    if (p.lanes == 1) return launch<T, W, 1>(p, interleaved, grad, st);  // (D = 16; of fp32 two lanes)
  switch (p.lanes) {
    case 2: return launch<T, W, 2>(p, interleaved, grad, st);
    case 4: return launch<T, W, 4>(p, interleaved, grad, st);
    case 8: return launch<T, W, 8>(p, interleaved, grad, st);
    case 16: return launch<T, W, 16>(p, interleaved, grad, st);
    default: return launch<T, W, 32>(p, interleaved, grad, st);
  }
}

int launch_type(const char* who, const NormParams& p, const NormCall& a, bool interleaved, bool grad, void* stream) {
  if (p.tokens * (p.groups[0] + p.groups[1]) * p.lanes > 2147483647LL * kThreads)
    return bad(FA_ERR_UNSUPPORTED, who, "too many rows for one launch");
  if (!device_status_ptr()) return bad(FA_ERR_CUDA, who, "no usable CUDA device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == FA_BF16   ? launch_lanes<__nv_bfloat16, 8>(p, interleaved, grad, st)
                        : a.dtype == FA_FP16 ? launch_lanes<__half, 8>(p, interleaved, grad, st)
                        : width(a) == 4      ? launch_lanes<float, 4>(p, interleaved, grad, st)
                                             : launch_lanes<float, 8>(p, interleaved, grad, st);
  return e == cudaSuccess ? FA_OK : bad(FA_ERR_CUDA, who, cudaGetErrorString(e));
}

template <typename Args>
NormCall call_of(const Args* a) {
  return NormCall{a->B, a->T, a->Hq, a->Hk, a->D, a->rot_dim, a->positions, a->inv_freq, a->q_weight, a->k_weight,
                  a->amplitude, a->eps, a->dtype, a->weight_dtype};
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_qk_norm_rotary(const fa_norm_rotary_args* a, void* stream) {
  const char* who = "fa_qk_norm_rotary";
  if (!a) return bad(FA_ERR_INVALID_ARG, who, "null argument struct");
  const NormCall c = call_of(a);
  int rc = check_call(who, c);
  if (rc != FA_OK || a->B == 0 || a->T == 0 || a->Hq + a->Hk == 0) return rc;
  if ((rc = check_rows(who, a->q, a->q_strides, c, a->Hq, false)) != FA_OK ||
      (rc = check_rows(who, a->k, a->k_strides, c, a->Hk, false)) != FA_OK ||
      (rc = check_rows(who, a->q_out, a->q_out_strides, c, a->Hq, true)) != FA_OK ||
      (rc = check_rows(who, a->k_out, a->k_out_strides, c, a->Hk, true)) != FA_OK ||
      (rc = check_tables(who, c)) != FA_OK)
    return rc;
  NormParams p{};
  fill_params(p, c);
  p.x[0] = a->q;
  p.x[1] = a->k;
  p.y[0] = a->q_out;
  p.y[1] = a->k_out;
  memcpy(p.xs[0], a->q_strides, sizeof p.xs[0]);
  memcpy(p.xs[1], a->k_strides, sizeof p.xs[1]);
  memcpy(p.ys[0], a->q_out_strides, sizeof p.ys[0]);
  memcpy(p.ys[1], a->k_out_strides, sizeof p.ys[1]);
  return launch_type(who, p, c, a->interleaved != 0, false, stream);
}

size_t fa_qk_norm_rotary_backward_workspace_size(const fa_norm_rotary_backward_args* a) {
  if (!a) return 0;
  const NormCall c = call_of(a);
  if (check_call("fa_qk_norm_rotary_backward", c) != FA_OK || a->B == 0 || a->T == 0 || a->Hq + a->Hk == 0) return 0;
  NormParams p{};
  fill_params(p, c);
  grad_blocks(p);
  return static_cast<size_t>(p.blocks[0] + p.blocks[1]) * p.D * sizeof(float);
}

int fa_qk_norm_rotary_backward(const fa_norm_rotary_backward_args* a, void* stream) {
  const char* who = "fa_qk_norm_rotary_backward";
  if (!a) return bad(FA_ERR_INVALID_ARG, who, "null argument struct");
  const NormCall c = call_of(a);
  int rc = check_call(who, c);
  if (rc != FA_OK) return rc;
  if (!aligned(a->dq_weight, 4) || !aligned(a->dk_weight, 4)) return bad(FA_ERR_INVALID_ARG, who, "misaligned weight gradient");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* const dw[2] = {a->dq_weight, a->dk_weight};
  if (a->B == 0 || a->T == 0 || a->Hq + a->Hk == 0) {
    // no row: the weights' gradients are sums of nothing
    for (int i = 0; i < 2; ++i)
      if (dw[i] && cudaMemsetAsync(dw[i], 0, a->D * sizeof(float), st) != cudaSuccess)
        return bad(FA_ERR_CUDA, who, "memset failed");
    return FA_OK;
  }
  if ((rc = check_rows(who, a->dq_out, a->dq_out_strides, c, a->Hq, false)) != FA_OK ||
      (rc = check_rows(who, a->dk_out, a->dk_out_strides, c, a->Hk, false)) != FA_OK ||
      (rc = check_rows(who, a->q, a->q_strides, c, a->Hq, false)) != FA_OK ||
      (rc = check_rows(who, a->k, a->k_strides, c, a->Hk, false)) != FA_OK ||
      (rc = check_rows(who, a->dq, a->dq_strides, c, a->Hq, true)) != FA_OK ||
      (rc = check_rows(who, a->dk, a->dk_strides, c, a->Hk, true)) != FA_OK ||
      (rc = check_tables(who, c)) != FA_OK)
    return rc;
  NormParams p{};
  fill_params(p, c);
  grad_blocks(p);
  const size_t need = static_cast<size_t>(p.blocks[0] + p.blocks[1]) * p.D * sizeof(float);
  if (!a->workspace || a->workspace_bytes < need) return bad(FA_ERR_WORKSPACE, who, "workspace too small");
  if (!aligned(a->workspace, 256)) return bad(FA_ERR_INVALID_ARG, who, "workspace must be 256-byte aligned");
  p.dy[0] = a->dq_out;
  p.dy[1] = a->dk_out;
  p.x[0] = a->q;
  p.x[1] = a->k;
  p.y[0] = a->dq;
  p.y[1] = a->dk;
  memcpy(p.ds[0], a->dq_out_strides, sizeof p.ds[0]);
  memcpy(p.ds[1], a->dk_out_strides, sizeof p.ds[1]);
  memcpy(p.xs[0], a->q_strides, sizeof p.xs[0]);
  memcpy(p.xs[1], a->k_strides, sizeof p.xs[1]);
  memcpy(p.ys[0], a->dq_strides, sizeof p.ys[0]);
  memcpy(p.ys[1], a->dk_strides, sizeof p.ys[1]);
  p.partial = static_cast<float*>(a->workspace);
  p.dw[0] = dw[0];
  p.dw[1] = dw[1];
  return launch_type(who, p, c, a->interleaved != 0, true, stream);
}

}  // extern "C"
