// delta_step.cu -- the gated delta rule token by token, on a pool of states: the decode form of
// gated_delta.cu's recurrence.
//
//     S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,   o_t = S_t (scale q_t),   a_t = e^{g_t}
//
// A row of S (one value dimension, 128 key columns) needs nothing of the other rows: with
// u = b (v - a <s, k>) its new value is a s + u k, and its output (a <s, q> + u <k, q>) scale, both
// from the row before the token, in one pass.  So the state stays in registers from the read to the
// write however many tokens there are; the state's bytes (64 KB a head, once each way, fp32) bound
// the call: 128 sequences of 32 heads, one token each, take 80.1 us, 6.74 TB/s, the measured copy rate;
// one sequence of five tokens 4.2 us, a launch, one trip to memory and five dependent tokens.  Eight lanes hold a row, sixteen columns each (four 16-byte pieces 128 bytes apart, so
// that a row's lanes read whole lines); two dot products a row and token go through three
// shuffles each.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "../../include/fa.h"
#include "internal.h"
#include "cache.cuh"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kDim = 128;      // key columns and value rows of a state
constexpr int kThreads = 256;  // 32 rows a pass

struct StepParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  float* states;
  const int32_t* read_index;   // or nullptr: sequence b's slot is b
  const int32_t* write_index;  // or nullptr: where it was read
  const int32_t* new_lens;     // or nullptr: T each
  void* out;
  int64_t qs[3], ks[3], vs[3], gs[3], bs[3], os[3];  // batch, head, token strides in elements
  int T, Hk, Hv, num_states;
  float scale;
  uint32_t* status;
};

// Sixteen columns of a key or query row: 4 * lane + 32 * i + 0..3.
template <typename T>
__device__ __forceinline__ void load_cols(const T* row, int lane8, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + 4 * lane8 + 32 * i));
    unpack2<T>(w.x, x[4 * i], x[4 * i + 1]);
    unpack2<T>(w.y, x[4 * i + 2], x[4 * i + 3]);
  }
}

__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One block: 32 * ROWS rows of one state.
template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads, ROWS == 4 ? 2 : 4) step_kernel(const StepParams p) {
  const int b = blockIdx.z, h = blockIdx.y, hk = h / (p.Hv / p.Hk);
  const int lane8 = threadIdx.x % 8;
  const int row0 = blockIdx.x * 32 * ROWS + threadIdx.x / 8;  // then every 32nd
  const int from = p.read_index ? p.read_index[b] : b;
  const int to = p.write_index ? p.write_index[b] : from;
  const int n = p.new_lens ? p.new_lens[b] : p.T;
  const bool sane = from >= 0 && from < p.num_states && to >= 0 && to < p.num_states && n >= 0 && n <= p.T;
  if (!sane && threadIdx.x == 0) record_error(p.status, kDevBounds);
  float s[ROWS][16];
  const int64_t at = (static_cast<int64_t>(h) * kDim + row0) * kDim + 4 * lane8;
  constexpr int64_t kState = static_cast<int64_t>(kDim) * kDim;
  if (sane) {
    const float* src = p.states + from * (p.Hv * kState) + at;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(src + r * 32 * kDim + 32 * i);
        s[r][4 * i] = x.x;
        s[r][4 * i + 1] = x.y;
        s[r][4 * i + 2] = x.z;
        s[r][4 * i + 3] = x.w;
      }
  }
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + hk * p.qs[1];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + hk * p.ks[1];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[1] + row0;
  const float* g = p.g + b * p.gs[0] + h * p.gs[1];
  const float* beta = p.beta + b * p.bs[0] + h * p.bs[1];
  T* out = static_cast<T*>(p.out) + b * p.os[0] + h * p.os[1] + row0;
  const int live = sane ? n : 0;
  for (int t = 0; t < live; ++t) {
    float kc[16], qc[16], vr[ROWS];
    load_cols<T>(k + t * p.ks[2], lane8, kc);
    load_cols<T>(q + t * p.qs[2], lane8, qc);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) vr[r] = static_cast<float>(v[t * p.vs[2] + 32 * r]);
    const float a = expf(g[t * p.gs[2]]), bt = beta[t * p.bs[2]];
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) kq = fmaf(kc[i], qc[i], kq);
    kq = sum8(kq);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sk = fmaf(s[r][i], kc[i], sk);
        sq = fmaf(s[r][i], qc[i], sq);
      }
      sk = sum8(sk);
      sq = sum8(sq);
      const float u = bt * (vr[r] - a * sk);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[r][i] = fmaf(u, kc[i], a * s[r][i]);
      if (lane8 == 0) out[t * p.os[2] + 32 * r] = static_cast<T>((a * sq + u * kq) * p.scale);
    }
  }
  // padding tokens
  for (int t = live; t < p.T; ++t)
    if (lane8 == 0)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) out[t * p.os[2] + 32 * r] = static_cast<T>(0.f);
  if (sane && (n > 0 || to != from)) {
    float* dst = p.states + to * (p.Hv * kState) + at;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(dst + r * 32 * kDim + 32 * i) =
            make_float4(s[r][4 * i], s[r][4 * i + 1], s[r][4 * i + 2], s[r][4 * i + 3]);
  }
}

int bad(int code, const char* msg) { return set_error(code, msg); }

template <typename T>
cudaError_t launch(const StepParams& p, int B, cudaStream_t st) {
  // A whole state a block where that gives every SM two blocks or more, else a quarter each: the
  // loads of a few states then come from four times as many SMs (one sequence of 32 heads: 4.2 us for 6.5; 128
  // sequences: 80.1 us whole, 80.9 in quarters).
  const int sms = num_sms() > 0 ? num_sms() : 152;
  if (static_cast<int64_t>(B) * p.Hv >= 2LL * sms) step_kernel<T, 4><<<dim3(1, p.Hv, B), kThreads, 0, st>>>(p);
  else step_kernel<T, 1><<<dim3(4, p.Hv, B), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" int gated_delta_step(const gated_delta_step_args* a, void* stream) {
  if (!a) return bad(FA_ERR_INVALID_ARG, "gated_delta_step: null argument struct");
  if (a->B < 0 || a->T < 0 || a->Hk <= 0 || a->Hv <= 0 || a->Hv % a->Hk != 0 || a->num_states < 0)
    return bad(FA_ERR_INVALID_ARG, "gated_delta_step: need B, T, num_states >= 0, Hk, Hv > 0, Hv % Hk == 0");
  if (a->dk != kDim || a->dv != kDim) return bad(FA_ERR_UNSUPPORTED, "gated_delta_step: dk and dv must be 128");
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16)
    return bad(FA_ERR_UNSUPPORTED, "gated_delta_step: dtype must be FA_BF16 or FA_FP16");
  if (a->B > 65535 || a->Hv > 65535) return bad(FA_ERR_UNSUPPORTED, "gated_delta_step: B and Hv must be <= 65535");
  if (!isfinite(a->scale)) return bad(FA_ERR_INVALID_ARG, "gated_delta_step: scale must be finite");
  if (!a->read_index && a->B > a->num_states)
    return bad(FA_ERR_INVALID_ARG, "gated_delta_step: without read_index the pool needs a state for each sequence");
  if (a->B == 0) return FA_OK;
  if (!a->states || (a->T > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->out)))
    return bad(FA_ERR_INVALID_ARG, "gated_delta_step: null pointer");
  auto al = [](const void* p, int m) { return (reinterpret_cast<uintptr_t>(p) & (m - 1)) == 0; };
  if (!al(a->q, 16) || !al(a->k, 16) || !al(a->v, 16) || !al(a->out, 16) || !al(a->states, 16) || !al(a->g, 4) ||
      !al(a->beta, 4) || !al(a->read_index, 4) || !al(a->write_index, 4) || !al(a->new_lens, 4))
    return bad(FA_ERR_INVALID_ARG, "gated_delta_step: q, k, v, out and states must be 16-byte aligned");
  for (int i = 0; i < 3; ++i)
    if (a->q_strides[i] % 8 != 0 || a->k_strides[i] % 8 != 0 || a->v_strides[i] % 8 != 0 || a->out_strides[i] % 8 != 0)
      return bad(FA_ERR_INVALID_ARG, "gated_delta_step: strides of q, k, v and out must be multiples of 16 bytes");
  const int n[3] = {a->B, a->Hv, a->T};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && a->out_strides[i] < kDim && a->out_strides[i] > -kDim)
      return bad(FA_ERR_INVALID_ARG, "gated_delta_step: rows of out overlap");
  uint32_t* status = device_status_ptr();
  if (!status) return bad(FA_ERR_CUDA, "gated_delta_step: no usable CUDA device");
  StepParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.g = a->g;
  p.beta = a->beta;
  p.states = a->states;
  p.read_index = a->read_index;
  p.write_index = a->write_index;
  p.new_lens = a->new_lens;
  p.out = a->out;
  memcpy(p.qs, a->q_strides, sizeof p.qs);
  memcpy(p.ks, a->k_strides, sizeof p.ks);
  memcpy(p.vs, a->v_strides, sizeof p.vs);
  memcpy(p.gs, a->g_strides, sizeof p.gs);
  memcpy(p.bs, a->beta_strides, sizeof p.bs);
  memcpy(p.os, a->out_strides, sizeof p.os);
  p.T = a->T;
  p.Hk = a->Hk;
  p.Hv = a->Hv;
  p.num_states = a->num_states;
  p.scale = a->scale;
  p.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == FA_BF16 ? launch<__nv_bfloat16>(p, a->B, st) : launch<__half>(p, a->B, st);
  if (e != cudaSuccess) return bad(FA_ERR_CUDA, cudaGetErrorString(e));
  return FA_OK;
}
