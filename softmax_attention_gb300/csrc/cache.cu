// cache.cu -- rotary positions, and the paged cache written and read back (16-bit pages, or
// e4m3 values with one power-of-two scale a row).  All three are bound by memory: every element
// is read once and written once, 16 bytes a thread and access, with nothing in shared memory
// but the table of angles a position.
//
// A row (one token of one head) is cut into units of 16 elements, one thread each:
//   - the rotated part, half layout: columns [8u, 8u+8) and [half + 8u, half + 8u+8), so that
//     one thread holds both members of its eight pairs (and may write in place);
//   - everything else: the 16 consecutive columns of the unit.
// A thread takes the same unit of several heads of one token, so that the sines and cosines of
// its eight pairs are computed once for all of them.
#include <cuda_fp8.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "../../include/fa.h"
#include "cache.cuh"
#include "internal.h"
#include "rotary.cuh"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------------------------
// Rotary positions on q and k.  Thread = (unit, token, group of heads); q's heads come first,
// then k's.  16,384 tokens of 40 heads, D = 128, half of each rotated, bf16: 60 us, 5.6 TB/s or
// 0.83 of a copy, bound by the memory's latency: 24 warps an SM (80 registers, for which the
// half-layout and the 16-bit kernels spill 12 to 24 bytes a thread) with four heads' loads in
// flight.  Two waves of blocks or fewer pay for their tables and sines instead: the fp32 gradient of
// 3,686 tokens of 32 heads, D = 64, 461 blocks where 456 fit at once, 14.4 us.
// ------------------------------------------------------------------------------------------
struct RotaryParams {
  const void* x[2];
  void* y[2];
  int64_t xs[2][3], ys[2][3];  // batch, head, token strides in elements
  int H[2];
  const int32_t* positions;
  const double* inv_freq;
  float amplitude;
  int transpose;
  int T, D, half, units, rot_units;
  int heads_per_thread, head_groups;
  uint32_t tokens;  // B * T; tokens * units * head_groups is below 2^31
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryParams p) {
  __shared__ int64_t steps[kMaxRot / 2];
  fill_steps(steps, p.inv_freq, p.half);
  const uint32_t per_group = p.tokens * p.units;
  const uint32_t idx = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t group = idx / per_group;
  if (group >= static_cast<uint32_t>(p.head_groups)) return;
  const uint32_t rem = idx - group * per_group;
  const uint32_t token = rem / p.units;
  const int u = static_cast<int>(rem - token * p.units);
  const uint32_t b = token / p.T, t = token - b * p.T;
  Turn turn;
  const bool rotated = u < p.rot_units;
  if (rotated)
    fill_turn(turn, steps, u, p.positions[token], p.amplitude, p.transpose != 0);
  // columns of the unit's two halves; a trailing unit of eight columns has no second half
  const int c0 = rotated && !INTERLEAVED ? 8 * u : 16 * u;
  const int c1 = rotated && !INTERLEAVED ? p.half + 8 * u : 16 * u + 8;
  const bool second = c1 < p.D;
  const int h0 = static_cast<int>(group) * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.H[0] + p.H[1]);
  // this token's row of head 0 in q, k and their outputs
  const T* x0 = static_cast<const T*>(p.x[0]) + b * p.xs[0][0] + t * p.xs[0][2];
  const T* x1 = static_cast<const T*>(p.x[1]) + b * p.xs[1][0] + t * p.xs[1][2];
  T* y0 = static_cast<T*>(p.y[0]) + b * p.ys[0][0] + t * p.ys[0][2];
  T* y1 = static_cast<T*>(p.y[1]) + b * p.ys[1][0] + t * p.ys[1][2];
  constexpr int kBatch = sizeof(T) == 4 ? 2 : 4;  // heads whose loads are issued together
  for (int h = h0; h < h1; h += kBatch) {
    Raw8<T> ra[kBatch], rc[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h + j >= h1) break;
      const T* src = h + j < p.H[0] ? x0 + (h + j) * p.xs[0][1] : x1 + (h + j - p.H[0]) * p.xs[1][1];
      ra[j] = load_raw8<T>(src + c0);
      if (second) rc[j] = load_raw8<T>(src + c1);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h + j >= h1) break;
      float a[8], c[8];
      expand8<T>(ra[j], a);
      expand8<T>(rc[j], c);
      if (rotated) rotate<INTERLEAVED>(turn, a, c);
      T* dst = h + j < p.H[0] ? y0 + (h + j) * p.ys[0][1] : y1 + (h + j - p.H[0]) * p.ys[1][1];
      store8(dst + c0, a);
      if (second) store8(dst + c1, c);
    }
  }
}

// ------------------------------------------------------------------------------------------
// Cache write.  Thread = (unit, token, group of heads); the D/16 threads of a row sit side by
// side in a warp and share the row's largest magnitude by shuffles.  512 tokens of eight sequences,
// 8 kv heads, D = 128, to e4m3: 8.4 us, 3.0 TB/s (10.3 us when the rows' loads waited for the page
// id); 1024 blocks of 80 registers, 456 at once, each of which loads, reduces and stores in turn.
// (The registers are the angles', which this call has none of.)  Twenty calls a graph: 6.5 us each,
// 8.8 with the rotation; one token of each of 128 sequences 2.7 and 3.6 us.
// ------------------------------------------------------------------------------------------
struct AppendParams {
  const void* x[2];            // k, v
  void* pages[2];
  uint8_t* scales[2];          // e4m3 pages only
  int64_t xs[2][3];
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* new_lens;     // or nullptr: T each
  const int32_t* positions;    // or nullptr: the cache position
  const double* inv_freq;      // or nullptr: no rotation
  float amplitude;
  int T, D, Hkv, half, rot_units, page_size, page_shift, max_pages, num_pages;
  int heads_per_thread, head_groups;
  uint32_t tokens;  // B * T; tokens * units * head_groups is below 2^31
  uint32_t* status;
};

// One row into the pages: `a`, `b` the thread's two runs of eight elements at columns c0, c1.
template <typename T, bool Q8, int UNITS>
__device__ __forceinline__ void write_row(void* pages, uint8_t* scales, int64_t row, int D, int c0,
                                          int c1, const float (&a)[8], const float (&b)[8],
                                          bool live) {
  if constexpr (Q8) {
    // Infinite and NaN elements do not count towards the row's scale: an infinity is stored
    // as +-448, a NaN as NaN.
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, finite_abs(a[i]));
      amax = fmaxf(amax, finite_abs(b[i]));
    }
#pragma unroll
    for (int o = UNITS / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!live) return;
    const int e = row_exponent(amax);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e in [-126, 120]
    uint8_t* dst = static_cast<uint8_t*>(pages) + row * D;
    const uint2 qa = make_uint2(quant4(a[0], a[1], a[2], a[3], inv), quant4(a[4], a[5], a[6], a[7], inv));
    const uint2 qb = make_uint2(quant4(b[0], b[1], b[2], b[3], inv), quant4(b[4], b[5], b[6], b[7], inv));
    if (c1 == c0 + 8) {
      *reinterpret_cast<uint4*>(dst + c0) = make_uint4(qa.x, qa.y, qb.x, qb.y);
    } else {
      *reinterpret_cast<uint2*>(dst + c0) = qa;
      *reinterpret_cast<uint2*>(dst + c1) = qb;
    }
    if (threadIdx.x % UNITS == 0) scales[row] = static_cast<uint8_t>(e + 127);
  } else {
    if (!live) return;
    T* dst = static_cast<T*>(pages) + row * D;
    store8(dst + c0, a);
    store8(dst + c1, b);
  }
}

template <typename T, bool Q8, int UNITS, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  __shared__ int64_t steps[128];  // D <= 256
  if (p.inv_freq) fill_steps(steps, p.inv_freq, p.half);
  const uint32_t per_group = p.tokens * UNITS;
  const uint32_t idx = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t group = idx / per_group;
  // a row's threads stand or fall together (UNITS divides the warp); the shuffles need them all
  bool live = group < static_cast<uint32_t>(p.head_groups);
  const uint32_t rem = live ? idx - group * per_group : 0;
  const uint32_t token = rem / UNITS;
  const int u = static_cast<int>(rem % UNITS);
  const int64_t b = token / p.T;
  const int t = static_cast<int>(token - static_cast<uint32_t>(b) * p.T);
  int pos = 0, page = 0;
  if (live) {
    const int len = p.seq_lens[b], n = p.new_lens ? p.new_lens[b] : p.T;
    const bool sane = n >= 0 && n <= p.T && len >= n &&
                      static_cast<int64_t>(len) <= static_cast<int64_t>(p.max_pages) * p.page_size;
    live = sane && t < n;
    if (!sane) record_error(p.status, kDevBounds);
    if (live) {
      pos = len - n + t;
      page = __ldg(p.page_table + b * p.max_pages + (pos >> p.page_shift));
    }
  }
  const bool rotated = p.inv_freq && u < p.rot_units;
  Turn turn;
  if (live && rotated)
    fill_turn(turn, steps, u, p.positions ? p.positions[token] : pos, p.amplitude, false);
  const int k0 = rotated && !INTERLEAVED ? 8 * u : 16 * u;
  const int k1 = rotated && !INTERLEAVED ? p.half + 8 * u : 16 * u + 8;
  const int h0 = static_cast<int>(live ? group : 0) * p.heads_per_thread;
  for (int j = 0; j < p.heads_per_thread; ++j) {  // the same count for every thread: shuffles
    const int h = h0 + j;
    const bool ok = live && h < p.Hkv;
    float ka[8] = {}, kb[8] = {}, va[8] = {}, vb[8] = {};
    if (ok) {
      const T* ks = static_cast<const T*>(p.x[0]) + b * p.xs[0][0] + h * p.xs[0][1] + t * p.xs[0][2];
      const T* vs = static_cast<const T*>(p.x[1]) + b * p.xs[1][0] + h * p.xs[1][1] + t * p.xs[1][2];
      load8(ks + k0, ka);
      load8(ks + k1, kb);
      load8(vs + 16 * u, va);
      load8(vs + 16 * u + 8, vb);
      if (rotated) rotate<INTERLEAVED>(turn, ka, kb);
    }
    // looked at here, so that the rows' loads do not wait for the page id
    const bool have_page = page >= 0 && page < p.num_pages;
    if (ok && !have_page) record_error(p.status, kDevBounds);
    const int64_t row = (static_cast<int64_t>(page) * p.Hkv + h) * p.page_size + (pos & (p.page_size - 1));
    write_row<T, Q8, UNITS>(p.pages[0], p.scales[0], row, p.D, k0, k1, ka, kb, ok && have_page);
    write_row<T, Q8, UNITS>(p.pages[1], p.scales[1], row, p.D, 16 * u, 16 * u + 8, va, vb, ok && have_page);
  }
}

// ------------------------------------------------------------------------------------------
// Cache read: dense [B,Hkv,L,D] from the pages, zeros past each sequence.  A thread keeps its
// eight columns and walks down the tokens of its block: kGatherSteps batches of kGatherBatch loads
// in flight.  Eight sequences of up to 8192 tokens, 8 kv heads, D = 128, e4m3 to bf16: 61 us, 5.7
// TB/s or 0.84 of a copy, bound by its writes (twice the bytes that it reads).
// ------------------------------------------------------------------------------------------
struct GatherParams {
  const void* pages[2];
  const uint8_t* scales[2];
  void* out[2];
  const int32_t* page_table;
  const int32_t* seq_lens;
  int Hkv, L, D, page_size, page_shift, max_pages, num_pages, B;
  uint32_t* status;
};

template <typename TIn, typename TOut, bool Q8, int kGatherBatch, int kGatherSteps>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p) {
  const int lanes = p.D / 8;                // threads a row
  const int rows = kThreads / lanes;        // rows a step
  const int c = (threadIdx.x % lanes) * 8, r = threadIdx.x / lanes;
  const int b = blockIdx.z >> 1, w = blockIdx.z & 1;
  const int h = blockIdx.y;
  const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  const int t0 = blockIdx.x * rows * kGatherBatch * kGatherSteps + r;
  // Page ids of all rows, before anything is waited for: the length, the ids and the data would
  // otherwise be three memory latencies one after another.  Entries past max_seq_len's pages are
  // not read; those past the sequence's end are read and not used.
  const int last_page = (p.L - 1) >> p.page_shift;
  int len = p.seq_lens[b];
  int id[kGatherBatch * kGatherSteps];
#pragma unroll
  for (int j = 0; j < kGatherBatch * kGatherSteps; ++j)
    id[j] = __ldg(table + min((t0 + j * rows) >> p.page_shift, last_page));
  if (len < 0 || len > p.L || static_cast<int64_t>(len) > static_cast<int64_t>(p.max_pages) * p.page_size) {
    if (threadIdx.x == 0) record_error(p.status, kDevBounds);
    len = 0;
  }
  // selected, not indexed: a kernel parameter indexed at run time is copied to local memory
  TOut* out = static_cast<TOut*>(w ? p.out[1] : p.out[0]) + (static_cast<int64_t>(b) * p.Hkv + h) * p.L * p.D;
  const void* pages = w ? p.pages[1] : p.pages[0];
  const uint8_t* scales = w ? p.scales[1] : p.scales[0];
#pragma unroll
  for (int s = 0; s < kGatherSteps; ++s) {
    uint2 q[kGatherBatch];
    uint32_t byte[kGatherBatch];
    Raw8<uint16_t> raw[kGatherBatch];
#pragma unroll
    for (int j = 0; j < kGatherBatch; ++j) {
      const int t = t0 + (s * kGatherBatch + j) * rows, page = id[s * kGatherBatch + j];
      q[j] = make_uint2(0, 0);
      byte[j] = 127;
      raw[j].v[0] = make_uint4(0, 0, 0, 0);
      if (t >= len) continue;
      if (page < 0 || page >= p.num_pages) {
        record_error(p.status, kDevBounds);
        continue;
      }
      const int64_t row = (static_cast<int64_t>(page) * p.Hkv + h) * p.page_size + (t & (p.page_size - 1));
      if constexpr (Q8) {
        q[j] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + row * p.D + c);
        byte[j] = __ldg(scales + row);
      } else {
        raw[j] = load_raw8(static_cast<const uint16_t*>(pages) + row * p.D + c);
      }
    }
#pragma unroll
    for (int j = 0; j < kGatherBatch; ++j) {
      const int t = t0 + (s * kGatherBatch + j) * rows;
      float x[8];
      if constexpr (Q8) {
        const float f = scale_of_byte(byte[j]);
        dequant4(q[j].x, f, x[0], x[1], x[2], x[3]);
        dequant4(q[j].y, f, x[4], x[5], x[6], x[7]);
      } else {
        Raw8<TIn> e;
        e.v[0] = raw[j].v[0];
        expand8<TIn>(e, x);
      }
      if (t < p.L) store8(out + static_cast<int64_t>(t) * p.D + c, x);
    }
  }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
int bad(int code, const char* msg) { return set_error(code, msg); }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int elem_size(fa_dtype t) { return t == FA_FP32 ? 4 : t == FA_E4M3 ? 1 : 2; }
bool is_float_type(fa_dtype t) { return t == FA_BF16 || t == FA_FP16 || t == FA_FP32; }

// 16-byte accesses at any (batch, head, token): every stride a multiple of 16 bytes.
bool strides_ok(const int64_t* s, fa_dtype t) {
  const int64_t m = 16 / elem_size(t);
  return s[0] % m == 0 && s[1] % m == 0 && s[2] % m == 0;
}

// Whether rows of an output [n0, n1, n2, D] are written over one another: neighbours closer than D.
bool rows_overlap(const int64_t* s, int n0, int n1, int n2, int D) {
  const int n[3] = {n0, n1, n2};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && s[i] < D && s[i] > -D) return true;
  return false;
}

int check_rot(const char* who, int rot_dim, int D) {
  char msg[200];
  if (rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > D || rot_dim > kMaxRot) {
    snprintf(msg, sizeof msg, "%s: rot_dim must be a multiple of 16 in [16, min(D, %d)] (got %d, D %d)",
             who, kMaxRot, rot_dim, D);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  return FA_OK;
}

// Heads a thread takes: as many as eight (the eight angles of a unit cost as much as several rows,
// and are then computed once for them), but no more than leave every SM 512 threads.
int heads_per_thread(int64_t unit_tokens, int H) {
  const int sms = num_sms() > 0 ? num_sms() : 152;
  int hpt = 8;
  while (hpt > 1 && unit_tokens * ((H + hpt - 1) / hpt) < 512LL * sms) hpt /= 2;
  return hpt < H ? hpt : H;
}

template <typename T>
cudaError_t run_rotary(const RotaryParams& p, bool interleaved, cudaStream_t st) {
  const uint32_t threads = p.tokens * p.units * p.head_groups;
  const unsigned grid = (threads + kThreads - 1) / kThreads;
  if (interleaved) rotary_kernel<T, true><<<grid, kThreads, 0, st>>>(p);
  else rotary_kernel<T, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, bool Q8, int UNITS>
cudaError_t run_append(const AppendParams& p, bool interleaved, cudaStream_t st) {
  const uint32_t threads = p.tokens * UNITS * p.head_groups;
  const unsigned grid = (threads + kThreads - 1) / kThreads;
  if (interleaved) append_kernel<T, Q8, UNITS, true><<<grid, kThreads, 0, st>>>(p);
  else append_kernel<T, Q8, UNITS, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, bool Q8>
cudaError_t run_append_d(const AppendParams& p, bool interleaved, cudaStream_t st) {
  switch (p.D) {
    case 64: return run_append<T, Q8, 4>(p, interleaved, st);
    case 128: return run_append<T, Q8, 8>(p, interleaved, st);
    default: return run_append<T, Q8, 16>(p, interleaved, st);
  }
}

template <typename TIn, typename TOut, bool Q8, int BATCH, int STEPS>
cudaError_t run_gather_as(const GatherParams& p, cudaStream_t st) {
  const int rows = kThreads / (p.D / 8) * BATCH * STEPS;
  const dim3 grid((p.L + rows - 1) / rows, p.Hkv, 2 * p.B);
  gather_kernel<TIn, TOut, Q8, BATCH, STEPS><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// Sixteen rows a thread, eight in flight, hide the memory's latency best (8 sequences of up to
// 8192 tokens: 61 us, against 78 with four rows a thread); two a thread give a small read more
// blocks (1021 tokens of two heads: 6 us against 10).  Sixteen once they fill every SM.
template <typename TIn, typename TOut, bool Q8>
cudaError_t run_gather_to(const GatherParams& p, cudaStream_t st) {
  const int sms = num_sms() > 0 ? num_sms() : 152;
  const int64_t blocks = static_cast<int64_t>(p.L) * (p.D / 8) / (kThreads * 16) * p.Hkv * 2 * p.B;
  return blocks >= 2 * sms ? run_gather_as<TIn, TOut, Q8, 8, 2>(p, st) : run_gather_as<TIn, TOut, Q8, 2, 1>(p, st);
}

template <typename TIn, bool Q8>
cudaError_t run_gather(const GatherParams& p, fa_dtype out, cudaStream_t st) {
  if (out == FA_BF16) return run_gather_to<TIn, __nv_bfloat16, Q8>(p, st);
  if (out == FA_FP16) return run_gather_to<TIn, __half, Q8>(p, st);
  return run_gather_to<TIn, float, Q8>(p, st);
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// What the cache calls share: pages, table, lengths.
int check_pages(const char* who, int B, int Hkv, int D, int page_size, int max_pages, int num_pages) {
  char msg[200];
  if (B < 0 || Hkv <= 0 || max_pages < 0 || num_pages < 0) {
    snprintf(msg, sizeof msg, "%s: need B, max_pages, num_pages >= 0 and Hkv > 0", who);
    return bad(FA_ERR_INVALID_ARG, msg);
  }
  if (D != 64 && D != 128 && D != 256) {
    snprintf(msg, sizeof msg, "%s: D must be 64, 128 or 256 (got %d)", who, D);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  if (page_size <= 0 || (page_size & (page_size - 1)) != 0) {
    snprintf(msg, sizeof msg, "%s: page_size must be a power of two (got %d)", who, page_size);
    return bad(FA_ERR_INVALID_ARG, msg);
  }
  if (B > 32767 || Hkv > 65535) {
    snprintf(msg, sizeof msg, "%s: B must be <= 32767 and Hkv <= 65535", who);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  if (static_cast<int64_t>(max_pages) * page_size > 2147483647LL) {
    snprintf(msg, sizeof msg, "%s: max_pages * page_size must fit in int32", who);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_rotary(const fa_rotary_args* a, void* stream) {
  if (!a) return bad(FA_ERR_INVALID_ARG, "fa_rotary: null argument struct");
  char msg[200];
  if (a->B < 0 || a->T < 0 || a->Hq < 0 || a->Hk < 0 || a->D <= 0)
    return bad(FA_ERR_INVALID_ARG, "fa_rotary: need B, T, Hq, Hk >= 0 and D > 0");
  if (a->D % 8 != 0) {
    snprintf(msg, sizeof msg, "fa_rotary: D must be a multiple of 8 (got %d)", a->D);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  int rc = check_rot("fa_rotary", a->rot_dim, a->D);
  if (rc != FA_OK) return rc;
  if (!is_float_type(a->dtype)) return bad(FA_ERR_UNSUPPORTED, "fa_rotary: dtype must be FA_BF16, FA_FP16 or FA_FP32");
  if (!(a->amplitude == a->amplitude) || isinf(a->amplitude))
    return bad(FA_ERR_INVALID_ARG, "fa_rotary: amplitude must be finite");
  if (a->B == 0 || a->T == 0 || a->Hq + a->Hk == 0) return FA_OK;
  if (!a->positions || !a->inv_freq || (a->Hq > 0 && (!a->q || !a->q_out)) || (a->Hk > 0 && (!a->k || !a->k_out)))
    return bad(FA_ERR_INVALID_ARG, "fa_rotary: null pointer");
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->q_out, 16) || !aligned(a->k_out, 16) ||
      !aligned(a->positions, 4) || !aligned(a->inv_freq, 8))
    return bad(FA_ERR_INVALID_ARG, "fa_rotary: q, k and the outputs must be 16-byte aligned");
  if (!strides_ok(a->q_strides, a->dtype) || !strides_ok(a->k_strides, a->dtype) ||
      !strides_ok(a->q_out_strides, a->dtype) || !strides_ok(a->k_out_strides, a->dtype))
    return bad(FA_ERR_INVALID_ARG, "fa_rotary: strides must be multiples of 16 bytes");
  if ((a->Hq > 0 && rows_overlap(a->q_out_strides, a->B, a->Hq, a->T, a->D)) ||
      (a->Hk > 0 && rows_overlap(a->k_out_strides, a->B, a->Hk, a->T, a->D)))
    return bad(FA_ERR_INVALID_ARG, "fa_rotary: rows of an output overlap (a broadcast tensor cannot be one)");
  if (!device_status_ptr()) return bad(FA_ERR_CUDA, "fa_rotary: no usable CUDA device");
  RotaryParams p{};
  p.x[0] = a->q;
  p.x[1] = a->k;
  p.y[0] = a->q_out;
  p.y[1] = a->k_out;
  memcpy(p.xs[0], a->q_strides, sizeof p.xs[0]);
  memcpy(p.xs[1], a->k_strides, sizeof p.xs[1]);
  memcpy(p.ys[0], a->q_out_strides, sizeof p.ys[0]);
  memcpy(p.ys[1], a->k_out_strides, sizeof p.ys[1]);
  p.H[0] = a->Hq;
  p.H[1] = a->Hk;
  p.positions = a->positions;
  p.inv_freq = a->inv_freq;
  p.amplitude = a->amplitude;
  p.transpose = a->transpose ? 1 : 0;
  p.T = a->T;
  p.D = a->D;
  p.half = a->rot_dim / 2;
  p.rot_units = a->rot_dim / 16;
  p.units = p.rot_units + (a->D - a->rot_dim + 15) / 16;
  const int64_t tokens = static_cast<int64_t>(a->B) * a->T;
  const int H = a->Hq + a->Hk;
  p.tokens = static_cast<uint32_t>(tokens);
  p.heads_per_thread = heads_per_thread(tokens * p.units, H);
  p.head_groups = (H + p.heads_per_thread - 1) / p.heads_per_thread;
  if (tokens > 2147483647LL / p.units / p.head_groups - kThreads)
    return bad(FA_ERR_UNSUPPORTED, "fa_rotary: too many rows for one launch");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->dtype == FA_BF16   ? run_rotary<__nv_bfloat16>(p, a->interleaved != 0, st)
                  : a->dtype == FA_FP16 ? run_rotary<__half>(p, a->interleaved != 0, st)
                                        : run_rotary<float>(p, a->interleaved != 0, st);
  if (e != cudaSuccess) return bad(FA_ERR_CUDA, cudaGetErrorString(e));
  return FA_OK;
}

int fa_rotary_frequencies(int rot_dim, double base, fa_rotary_scaling scaling, double factor,
                          double original_len, double fast, double slow, double* inv_freq,
                          float* amplitude) {
  if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || isinf(base) || !inv_freq || !amplitude)
    return bad(FA_ERR_INVALID_ARG, "fa_rotary_frequencies: need an even rot_dim >= 2, base > 1 and both outputs");
  if (scaling != FA_ROTARY_PLAIN && (!(factor >= 1.0) || isinf(factor)))
    return bad(FA_ERR_INVALID_ARG, "fa_rotary_frequencies: factor must be >= 1");
  float a = 1.f;
  switch (scaling) {
    case FA_ROTARY_PLAIN:
    case FA_ROTARY_LINEAR:
      break;
    case FA_ROTARY_BASE:
      if (rot_dim <= 2) return bad(FA_ERR_INVALID_ARG, "fa_rotary_frequencies: FA_ROTARY_BASE needs rot_dim > 2");
      base *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
      break;
    case FA_ROTARY_BY_PARTS:
      if (!(original_len > 0.0) || !(slow >= 0.0) || !(fast > slow))
        return bad(FA_ERR_INVALID_ARG, "fa_rotary_frequencies: need original_len > 0 and fast > slow >= 0");
      a = static_cast<float>(0.1 * log(factor) + 1.0);
      break;
    default:
      return bad(FA_ERR_INVALID_ARG, "fa_rotary_frequencies: unknown scaling");
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == FA_ROTARY_LINEAR) f /= factor;
    if (scaling == FA_ROTARY_BY_PARTS) {
      const double turns = original_len * f / 6.283185307179586477;
      const double keep = fmin(1.0, fmax(0.0, (turns - slow) / (fast - slow)));
      f = (1.0 - keep) * f / factor + keep * f;
    }
    inv_freq[i] = f;
  }
  *amplitude = a;
  return FA_OK;
}

int fa_cache_append(const fa_cache_append_args* a, void* stream) {
  if (!a) return bad(FA_ERR_INVALID_ARG, "fa_cache_append: null argument struct");
  if (a->T < 0) return bad(FA_ERR_INVALID_ARG, "fa_cache_append: T must be >= 0");
  int rc = check_pages("fa_cache_append", a->B, a->Hkv, a->D, a->page_size, a->max_pages, a->num_pages);
  if (rc != FA_OK) return rc;
  if (!is_float_type(a->dtype))
    return bad(FA_ERR_UNSUPPORTED, "fa_cache_append: dtype must be FA_BF16, FA_FP16 or FA_FP32");
  if (a->cache_dtype != FA_E4M3 && (a->cache_dtype != a->dtype || a->dtype == FA_FP32))
    return bad(FA_ERR_UNSUPPORTED, "fa_cache_append: cache_dtype must be FA_E4M3, or dtype when that has 16 bits");
  if (a->inv_freq) {
    rc = check_rot("fa_cache_append", a->rot_dim, a->D);
    if (rc != FA_OK) return rc;
    if (!(a->amplitude == a->amplitude) || isinf(a->amplitude))
      return bad(FA_ERR_INVALID_ARG, "fa_cache_append: amplitude must be finite");
  }
  if (a->B == 0 || a->T == 0) return FA_OK;
  if (!a->k || !a->v || !a->k_pages || !a->v_pages || !a->page_table || !a->seq_lens)
    return bad(FA_ERR_INVALID_ARG, "fa_cache_append: null pointer");
  if (a->cache_dtype == FA_E4M3 && (!a->k_scales || !a->v_scales))
    return bad(FA_ERR_INVALID_ARG, "fa_cache_append: an 8-bit cache needs k_scales and v_scales");
  if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_pages, 16) || !aligned(a->v_pages, 16) ||
      !aligned(a->page_table, 4) || !aligned(a->seq_lens, 4) || !aligned(a->new_lens, 4) ||
      !aligned(a->positions, 4) || !aligned(a->inv_freq, 8))
    return bad(FA_ERR_INVALID_ARG, "fa_cache_append: k, v and the pages must be 16-byte aligned");
  if (!strides_ok(a->k_strides, a->dtype) || !strides_ok(a->v_strides, a->dtype))
    return bad(FA_ERR_INVALID_ARG, "fa_cache_append: strides must be multiples of 16 bytes");
  uint32_t* status = device_status_ptr();
  if (!status) return bad(FA_ERR_CUDA, "fa_cache_append: no usable CUDA device");
  AppendParams p{};
  p.x[0] = a->k;
  p.x[1] = a->v;
  p.pages[0] = a->k_pages;
  p.pages[1] = a->v_pages;
  p.scales[0] = a->k_scales;
  p.scales[1] = a->v_scales;
  memcpy(p.xs[0], a->k_strides, sizeof p.xs[0]);
  memcpy(p.xs[1], a->v_strides, sizeof p.xs[1]);
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.new_lens = a->new_lens;
  p.positions = a->positions;
  p.inv_freq = a->inv_freq;
  p.amplitude = a->amplitude;
  p.T = a->T;
  p.D = a->D;
  p.Hkv = a->Hkv;
  p.half = a->rot_dim / 2;
  p.rot_units = a->inv_freq ? a->rot_dim / 16 : 0;
  p.page_size = a->page_size;
  p.page_shift = log2_of(a->page_size);
  p.max_pages = a->max_pages;
  p.num_pages = a->num_pages;
  const int64_t tokens = static_cast<int64_t>(a->B) * a->T;
  p.tokens = static_cast<uint32_t>(tokens);
  p.status = status;
  // without a rotation a thread has nothing to share between heads
  p.heads_per_thread = a->inv_freq ? heads_per_thread(tokens * (a->D / 16), a->Hkv) : 1;
  p.head_groups = (a->Hkv + p.heads_per_thread - 1) / p.heads_per_thread;
  if (tokens > 2147483647LL / (a->D / 16) / p.head_groups - kThreads)
    return bad(FA_ERR_UNSUPPORTED, "fa_cache_append: too many rows for one launch");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool il = a->interleaved != 0;
  cudaError_t e;
  if (a->cache_dtype == FA_E4M3)
    e = a->dtype == FA_BF16   ? run_append_d<__nv_bfloat16, true>(p, il, st)
        : a->dtype == FA_FP16 ? run_append_d<__half, true>(p, il, st)
                              : run_append_d<float, true>(p, il, st);
  else
    e = a->dtype == FA_BF16 ? run_append_d<__nv_bfloat16, false>(p, il, st)
                            : run_append_d<__half, false>(p, il, st);
  if (e != cudaSuccess) return bad(FA_ERR_CUDA, cudaGetErrorString(e));
  return FA_OK;
}

int fa_cache_gather(const fa_cache_gather_args* a, void* stream) {
  if (!a) return bad(FA_ERR_INVALID_ARG, "fa_cache_gather: null argument struct");
  int rc = check_pages("fa_cache_gather", a->B, a->Hkv, a->D, a->page_size, a->max_pages, a->num_pages);
  if (rc != FA_OK) return rc;
  if (a->max_seq_len < 0 ||
      static_cast<int64_t>(a->max_seq_len) > static_cast<int64_t>(a->max_pages) * a->page_size)
    return bad(FA_ERR_INVALID_ARG, "fa_cache_gather: max_seq_len must be in [0, max_pages * page_size]");
  if (a->cache_dtype != FA_E4M3 && a->cache_dtype != FA_BF16 && a->cache_dtype != FA_FP16)
    return bad(FA_ERR_UNSUPPORTED, "fa_cache_gather: cache_dtype must be FA_E4M3, FA_BF16 or FA_FP16");
  if (!is_float_type(a->dtype))
    return bad(FA_ERR_UNSUPPORTED, "fa_cache_gather: dtype must be FA_BF16, FA_FP16 or FA_FP32");
  if (a->B == 0 || a->max_seq_len == 0) return FA_OK;
  if (!a->k_pages || !a->v_pages || !a->page_table || !a->seq_lens || !a->k || !a->v)
    return bad(FA_ERR_INVALID_ARG, "fa_cache_gather: null pointer");
  if (a->cache_dtype == FA_E4M3 && (!a->k_scales || !a->v_scales))
    return bad(FA_ERR_INVALID_ARG, "fa_cache_gather: an 8-bit cache needs k_scales and v_scales");
  if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_pages, 16) || !aligned(a->v_pages, 16) ||
      !aligned(a->page_table, 4) || !aligned(a->seq_lens, 4))
    return bad(FA_ERR_INVALID_ARG, "fa_cache_gather: k, v and the pages must be 16-byte aligned");
  uint32_t* status = device_status_ptr();
  if (!status) return bad(FA_ERR_CUDA, "fa_cache_gather: no usable CUDA device");
  GatherParams p{};
  p.pages[0] = a->k_pages;
  p.pages[1] = a->v_pages;
  p.scales[0] = a->k_scales;
  p.scales[1] = a->v_scales;
  p.out[0] = a->k;
  p.out[1] = a->v;
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.Hkv = a->Hkv;
  p.L = a->max_seq_len;
  p.D = a->D;
  p.page_size = a->page_size;
  p.page_shift = log2_of(a->page_size);
  p.max_pages = a->max_pages;
  p.num_pages = a->num_pages;
  p.B = a->B;
  p.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->cache_dtype == FA_E4M3   ? run_gather<uint8_t, true>(p, a->dtype, st)
                  : a->cache_dtype == FA_BF16 ? run_gather<__nv_bfloat16, false>(p, a->dtype, st)
                                              : run_gather<__half, false>(p, a->dtype, st);
  if (e != cudaSuccess) return bad(FA_ERR_CUDA, cudaGetErrorString(e));
  return FA_OK;
}

}  // extern "C"
