// packed_grad.cu -- the gradients of attention over packed prompts.
//
// With P_ij = e^(scale <q_i, k_j> - lse_i), dP_ij = <dout_i, v_j>, delta_i = <dout_i, out_i> and
// dS = P (dP - delta):
//     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,   dv_j = sum_i P_ij dout_i
//
// Three kernels; the sums that a block owns stay in tensor memory, so that nothing is added by atomics
// and the same call gives the same bits:
//   - row_kernel: delta and -lse, in the form that the others use them, a pass over dout and out (and, of rows that see
//     few keys, the products themselves; fp16: what bounds dP, with a pass over v);
//   - dkv_kernel: a block holds a tile of 128 keys and walks over the query tiles that see it, all
//     heads of the group: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  With the
//     products turned, P^T and dS^T have keys as rows and go back to tensor memory as the
//     left operands of the second pair: neither ever passes through shared memory;
//   - dq_kernel: a block holds a 128-row query tile (query tokens x heads of a kv head, as in
//     packed.cu) and walks over the keys: S = Q K^T, dP = dO V^T, dQ += dS K.
// S and dP are computed in both, seven products for the five of a form that adds dq by atomics.
//
// Bound by the tensor cores where sequences are long: 8192 tokens of 16 heads in 4 groups (bf16, D = 128, causal) take
// 555 to 590 us, from board to board, 1170 to 1240 TFLOP/s counting five products and 1640 to 1740 counting the seven,
// 0.85 to 0.90 of the measured bf16 rate.
// Samples of 512 to 2048 tokens: 380 us (850 and 1190); there a work item's first tile, which waits for its loads
// and meets an empty pipe, costs some 3 us of the 7 to 20 that the item takes, and shared memory has no room to
// hold the next item's Q and dO (K and V) beside this one's.  (Loading them to L2 ahead of time: no change.)
//
// Eight warps do the element-wise work, two a row, 64 columns each.  Blocks stay for all of their work
// items, and the products are issued by whole warps from uniform registers, as in packed.cu.
//
// fp16: dS is held times a power of two, f, so that the small values that gradients have keep their
// bits (its smallest normal number is 2^-14) and the large ones stay below its largest, 65504.  No |dP_ij| passes
// b_i = sum_d |dout_id| max |v|, and no |dS_ij|, with delta_i a mean of dP_ij over j by P_ij, b_i / 2: f brings b_i to
// [2^14, 2^15), of the row and the keys that its tile sees in dq_kernel, of the sequence's keys and the largest row that may see
// the key tile in dkv_kernel, whose sums run over rows; another sequence has no part in either.
// (What |dout| alone would give, dS of values of 100 can pass.)  P is held times 2^7 there.  bf16 has fp32's
// exponents, and f = 1.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "dependent.cuh"
#include "internal.h"
#include "packed.cuh"

namespace fa {
namespace packed {
namespace {

constexpr int kBlock = kRows * 128;  // 128 rows x 64 columns of 16 bits
constexpr int kHalf = 64;            // columns of S that a warp works on

struct GradParams {
  Params f;
  const void* dout;
  const void* o;         // the forward pass's out
  const float* lse;      // [total_q, Hq]
  const void* q;
  const void* k;
  const void* v;
  int64_t q_strides[2], k_strides[2], v_strides[2];
  int64_t dout_strides[2], o_strides[2];
  void* dq;
  void* dk;
  void* dv;
  int64_t dq_strides[2], dk_strides[2], dv_strides[2];
  // A query tile's rows side by side: [Hkv, total_q, G]
  float2* rows;          // -lse log2 e (-inf where nothing is seen), delta
  float* norms;          // fp16: sum of |dout| of the row; 0 where that is no number, or infinite
  float* few;            // delta of the rows that see few keys, likewise
  int few_units, few_blocks;  // row_kernel: pieces of such rows of a sequence; blocks for them, in front
  float* maxima;         // fp16: the largest of `norms` in each block of row_kernel, [Hkv, q_blocks]
  float* v_norms;        // fp16: the largest finite |v| of each key, [Hkv, total_k]
  float* v_maxima;       // fp16: and of each of its blocks for values, [Hkv, k_blocks]
  int q_blocks, k_blocks;  // row_kernel: blocks for the rows of a kv head, behind which those for its values come
  int* taken;            // dq_kernel: work items taken so far, beyond each block's first
};

// The power of two that brings `bound` to [2^14, 2^15); 1 for 0.
__device__ __forceinline__ float power_for(float bound) {
  if (!(bound > 0.f)) return 1.f;
  const int e = static_cast<int>(__float_as_uint(bound) >> 23) - 127;  // (fp16's: -48 to 39)
  return __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack(float2 v) {
  return BF16 ? pack_bf16x2(v.x, v.y) : pack_f16x2(v.x, v.y);
}

// 32 accumulator columns of a warp's 32 rows, times f, in 16 bits to global memory; `dst`: where the
// lane's row goes, or nullptr.  Four lanes trade their 16-byte pieces first, so that each store writes
// eight rows' 64 bytes and not 16 bytes of 32 rows.
template <bool BF16>
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&o)[32], float f) {
  const int l = threadIdx.x & 3;
  uint32_t w[4][4];  // [piece][word]; in the end [row of the four][word] of piece l
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[q][e] = pack<BF16>(make_float2(__uint_as_float(o[8 * q + 2 * e]) * f, __uint_as_float(o[8 * q + 2 * e + 1]) * f));
#pragma unroll
  for (int step = 1; step <= 2; ++step) {
    const bool up = (l & step) != 0;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int lo = step == 1 ? 2 * a : a, hi = lo + step;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[lo][e] : w[hi][e], step);
        if (up) w[lo][e] = got;
        else w[hi][e] = got;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long at = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), i, 4);
    if (at) reinterpret_cast<uint4*>(at)[l] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
}

// Rows r0.. of a 128-row tile in shared memory set to zero by `n` threads.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int r0, int at, int n) {
  const int per = (kRows - r0) * 8;
  for (int i = at; i < per * (D / 64); i += n)
    *reinterpret_cast<uint4*>(tile + (i / per) * kBlock + r0 * 128 + (i % per) * 16) = make_uint4(0, 0, 0, 0);
}

// S-shaped product: D = A B^T of two tiles in shared memory, both K-major.
template <int D>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk / 4) * kBlock + (kk % 4) * 32;
    mma_ss(d, sdesc_add(a_desc, off), sdesc_add(b_desc, off), idesc, kk > 0 ? 1u : 0u);
  }
}

// Second product: D += A B, A 16-bit in tensor memory in two halves of 64 columns' worth that start
// `half` columns apart, B a 128-row tile read MN-major.
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t half, uint64_t b_desc, uint32_t idesc,
                                           bool first) {
#pragma unroll
  for (int kk = 0; kk < kRows / 16; ++kk)
    mma_ts(d, a + (kk / 4) * half + (kk % 4) * 8, sdesc_add(b_desc, kk * 2048), idesc, (!first || kk > 0) ? 1u : 0u);
}

// ------------------------------------------------------------------------------------------
// delta and lse of each row.  D / 8 lanes a row, 16 bytes of dout and of out each, four rows in flight
// a thread; bound by memory (32,768 tokens of 16 heads, D = 128: 48 us with cold caches, 279 MB, 0.87 of the copy rate).
// ------------------------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kRowBatch = 4;

constexpr int row_block(int D) { return kRowThreads / (D / 8) * kRowBatch; }  // rows of a block

// Blocks for the rows of a kv head.
unsigned row_blocks(int total_q, int G, int D) {
  const int64_t per = row_block(D);
  return static_cast<unsigned>((static_cast<int64_t>(total_q) * G + per - 1) / per);
}

// Where a row sees few keys, dP and delta are nearly alike, and the rounding of `out` in <dout, out> would show in
// dS (sequences of two to eight tokens: gradients twice as far off as by dS's own rounding, of 32 a tenth).  There
// delta is sum_j P_j dP_j / sum_j P_j, from the products themselves; and of a row that sees one key dS is 0,
// exactly, which dq_kernel sees to for the row and dkv_kernel for a sequence's only key.  (Costs 1 us of 15 for three
// short samples, 4 of 380 for samples of 512 to 2048 tokens.  Such rows' columns masked out of dS in dkv_kernel's loop:
// 18 us of 555.  32 keys, two passes: 2 us more for the short ones, and registers that slow the others.  The products
// share row_kernel's 64 registers, and spill 100 to 192 bytes.)
constexpr int kFew = 16;

// C (16 x 8, fp32) += A (16 x 16) B (16 x 8).  With g = lane / 4, t = lane % 4: a0 (row g, k 2t..), a1 (g + 8, 2t..),
// a2 (g, 2t + 8..), a3 (g + 8, 2t + 8..); b0 (k 2t.., column g), b1 (2t + 8.., g); c0, c1 (row g, columns 2t,
// 2t + 1), c2, c3 (row g + 8).
template <bool BF16>
__device__ __forceinline__ void mma_warp(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// delta of a piece of the rows of sequence b that see 1 to kFew keys.  A warp takes 16 rows at a time;
// which of a row's elements a product's k-th is does not matter as long as both sides agree, so a lane reads 16 bytes.
template <int D, bool BF16>
__device__ __forceinline__ void few_rows(const GradParams& g, int b, int piece, int hk) {
  const Params& p = g.f;
  const Seq s = load_seq(p, b);
  int first = 0, n = 0;  // tokens
  if (p.causal) {
    first = max(0, s.nq - s.nk);
    n = max(0, min(s.nq, s.nq - s.nk + kFew) - first);
  } else if (s.nk > 0 && s.nk <= kFew) {
    n = s.nq;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gr = lane / 4, t = lane % 4;
  constexpr int kPerBlock = kRowThreads / 32 * 16;
  for (int64_t r0 = static_cast<int64_t>(piece) * kPerBlock + warp * 16; r0 < static_cast<int64_t>(n) * p.G;
       r0 += static_cast<int64_t>(g.few_units) * kPerBlock) {
    const uint16_t *q[2], *dout[2];
    int sees[2];  // keys
    float nl[2];
    int64_t at[2];
    const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t r = r0 + gr + 8 * x;
      const int token = static_cast<int>(r / p.G), h = hk * p.G + static_cast<int>(r - static_cast<int64_t>(token) * p.G);
      const int i = first + token;
      const int64_t row = s.q0 + i;
      sees[x] = token >= n ? 0 : p.causal ? min(s.nk, i + s.nk - s.nq + 1) : s.nk;
      at[x] = (hk * static_cast<int64_t>(p.total_q) + row) * p.G + (h - hk * p.G);
      nl[x] = -INFINITY;
      q[x] = dout[x] = nullptr;
      if (sees[x] == 0) continue;
      q[x] = static_cast<const uint16_t*>(g.q) + row * g.q_strides[0] + h * g.q_strides[1] + 8 * t;
      dout[x] = static_cast<const uint16_t*>(g.dout) + row * g.dout_strides[0] + h * g.dout_strides[1] + 8 * t;
      const float lse = __ldg(g.lse + row * p.Hq + h);
      if (lse != -INFINITY) nl[x] = -lse * prefill::kLog2e;
    }
    float sum[2] = {0.f, 0.f}, dot[2] = {0.f, 0.f};
    {
      float sc[2][4] = {}, dp[2][4] = {};
      const uint16_t *k[2], *v[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = 8 * x + gr;
        k[x] = v[x] = nullptr;
        if (key >= s.nk) continue;
        k[x] = static_cast<const uint16_t*>(g.k) + (s.k0 + static_cast<int64_t>(key)) * g.k_strides[0] + hk * g.k_strides[1] + 8 * t;
        v[x] = static_cast<const uint16_t*>(g.v) + (s.k0 + static_cast<int64_t>(key)) * g.v_strides[0] + hk * g.v_strides[1] + 8 * t;
      }
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        auto part = [&](const uint16_t* from) { return from ? __ldg(reinterpret_cast<const uint4*>(from + c)) : none; };
        const uint4 a0 = part(q[0]), a1 = part(q[1]), d0 = part(dout[0]), d1 = part(dout[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4 kb = part(k[x]), vb = part(v[x]);
          mma_warp<BF16>(sc[x], a0.x, a1.x, a0.y, a1.y, kb.x, kb.y);
          mma_warp<BF16>(sc[x], a0.z, a1.z, a0.w, a1.w, kb.z, kb.w);
          mma_warp<BF16>(dp[x], d0.x, d1.x, d0.y, d1.y, vb.x, vb.y);
          mma_warp<BF16>(dp[x], d0.z, d1.z, d0.w, d1.w, vb.z, vb.w);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (8 * x + 2 * t + (e & 1) >= sees[e / 2]) continue;
          const float w = nl[e / 2] == -INFINITY ? 0.f : exp2_approx(fmaf(sc[x][e], p.scale_log2, nl[e / 2]));
          sum[e / 2] += w;
          dot[e / 2] = fmaf(w, dp[x][e], dot[e / 2]);
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], o);
        dot[x] += __shfl_xor_sync(0xffffffffu, dot[x], o);
      }
      if (t == 0 && sees[x] > 0) g.few[at[x]] = sum[x] == 0.f ? 0.f : dot[x] / sum[x];
    }
  }
}

// Whether tokens t0 .. t1, a block's, are to be looked at: all between the first offset and the last are (if
// offsets are broken there, nobody asks for what stands beside them); of others, padding as a rule, those of a
// sequence, by the rule that the other kernels have, for it may lie outside where those two are the broken ones.
__device__ __forceinline__ bool wanted(const int32_t* cu, int B, int total, int64_t t0, int64_t t1) {
  if (t0 >= __ldg(cu) && t1 < __ldg(cu + B)) return true;
  bool mine = false;
  for (int b = threadIdx.x; b < B; b += kRowThreads) {
    const int first = __ldg(cu + b), end = __ldg(cu + b + 1);
    mine = mine || (first >= 0 && first < end && end <= total && first <= t1 && t0 < end);
  }
  return __syncthreads_or(mine);
}

// The largest of `v`, not negative, of a block's threads, in its first one.
__device__ __forceinline__ float block_max(float v) {
  __shared__ uint32_t tops[kRowThreads / 32];
  const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(v));
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = bits;
  __syncthreads();
  return __uint_as_float(threadIdx.x < 32 ? __reduce_max_sync(0xffffffffu, threadIdx.x < kRowThreads / 32 ? tops[threadIdx.x] : 0u) : 0u);
}

// fp16: the largest finite |v| of each key of a kv head, and of the block.  (With all that the bound takes: three short
// samples 17.6 us for 16.3 without, 8 of 693 to 2005 tokens 407 for 396.)
template <int D>
__device__ __forceinline__ void value_rows(const GradParams& g, int block, int hk) {
  constexpr int kLanes = D / 8, kPerPass = kRowThreads / kLanes;
  const int lane = threadIdx.x % kLanes, end = g.f.total_k;
  const int64_t start = static_cast<int64_t>(block) * row_block(D), key0 = start + threadIdx.x / kLanes;
  if (!wanted(g.f.cu_k, g.f.B, end, start, min(start + row_block(D), static_cast<int64_t>(end)) - 1)) return;
  uint4 x[kRowBatch];
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i) {
    const int64_t key = key0 + i * kPerPass;
    x[i] = make_uint4(0, 0, 0, 0);
    if (key < end)
      x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.v) + key * g.v_strides[0] + hk * g.v_strides[1]) + lane);
  }
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;  // magnitudes: 0x7c00 and up are no numbers
      top = max(top, max(lo < 0x7c00u ? lo : 0u, hi < 0x7c00u ? hi : 0u));
    }
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float v = __half2float(__ushort_as_half(static_cast<unsigned short>(top)));
    const int64_t key = key0 + i * kPerPass;
    if (lane == 0 && key < end) g.v_norms[static_cast<int64_t>(hk) * g.f.total_k + key] = v;
    most = fmaxf(most, v);
  }
  most = block_max(most);
  if (threadIdx.x == 0) g.v_maxima[static_cast<int64_t>(hk) * g.k_blocks + block] = most;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads, 4) row_kernel(const GradParams g) {
  constexpr int kLanes = D / 8, kPerPass = kRowThreads / kLanes;
  const Params& p = g.f;
  let_next_start();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *g.taken = 0;
  const int few = g.few_blocks;  // (a sequence's piece each, or more in turn)
  if (static_cast<int>(blockIdx.x) < few) {
    for (int64_t u = blockIdx.x; u < static_cast<int64_t>(p.B) * g.few_units; u += few)
      few_rows<D, BF16>(g, static_cast<int>(u / g.few_units), static_cast<int>(u % g.few_units), blockIdx.y);
    return;
  }
  if constexpr (!BF16) {
    if (static_cast<int>(blockIdx.x) >= few + g.q_blocks) {
      value_rows<D>(g, blockIdx.x - few - g.q_blocks, blockIdx.y);
      return;
    }
  }
  const uint32_t start = (blockIdx.x - few) * row_block(D);  // of the kv head's rows
  if (!wanted(p.cu_q, p.B, p.total_q, start / p.G, min((start + row_block(D) - 1) / p.G, p.total_q - 1u))) return;
  const int lane = threadIdx.x % kLanes;
  const uint32_t row0 = start + threadIdx.x / kLanes;
  const int hk = blockIdx.y;
  uint4 a[kRowBatch], c[kRowBatch];
  int token[kRowBatch], head[kRowBatch];
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i) {
    const uint32_t row = row0 + i * kPerPass;
    token[i] = static_cast<int>(row / static_cast<uint32_t>(p.G));
    head[i] = hk * p.G + static_cast<int>(row - token[i] * p.G);
    a[i] = c[i] = make_uint4(0, 0, 0, 0);
    if (token[i] >= p.total_q) token[i] = -1;
    if (token[i] < 0) continue;
    a[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.dout) + token[i] * g.dout_strides[0] + head[i] * g.dout_strides[1]) + lane);
    c[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.o) + token[i] * g.o_strides[0] + head[i] * g.o_strides[1]) + lane);
  }
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i) {
    const int64_t row = static_cast<int64_t>(hk) * p.total_q * p.G + row0 + i * kPerPass;
    const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wc[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    float delta = 0.f, norm = 0.f;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      float2 x, y;
      if constexpr (BF16) {
        x = make_float2(__uint_as_float(wa[f] << 16), __uint_as_float(wa[f] & 0xffff0000u));
        y = make_float2(__uint_as_float(wc[f] << 16), __uint_as_float(wc[f] & 0xffff0000u));
      } else {
        x = __half22float2(*reinterpret_cast<const __half2*>(&wa[f]));
        y = __half22float2(*reinterpret_cast<const __half2*>(&wc[f]));
        norm += fabsf(x.x) + fabsf(x.y);
      }
      delta = fmaf(x.x, y.x, fmaf(x.y, y.y, delta));
    }
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) {
      delta += __shfl_xor_sync(0xffffffffu, delta, o);
      if constexpr (!BF16) norm += __shfl_xor_sync(0xffffffffu, norm, o);
    }
    if (!(norm < INFINITY)) norm = 0.f;
    most = fmaxf(most, norm);
    if (lane == 0 && token[i] >= 0) {
      const float lse = __ldg(g.lse + static_cast<int64_t>(token[i]) * p.Hq + head[i]);
      g.rows[row] = make_float2(lse == -INFINITY ? -INFINITY : -lse * prefill::kLog2e, delta);
      if constexpr (!BF16) g.norms[row] = norm;
    }
  }
  if constexpr (!BF16) {
    // (a maximum a block, which the other kernels join as they need it: one of a sequence by an atomic would have to be
    // set to 0 first, by a launch of some 4 us)
    const float top = block_max(most);
    if (threadIdx.x == 0) g.maxima[static_cast<int64_t>(blockIdx.y) * g.q_blocks + blockIdx.x - few] = top;
  }
}

// What the blocks of dq_kernel and dkv_kernel have in common: their scheduling warp's work items, and the
// clearing of rows past a sequence's end that a sum would otherwise run over.  (The copies that need it
// land on a barrier of their own, and are full when they are cleared.  One such barrier is enough: the
// next item's copies wait for the products that read this one's.)
constexpr int kThreads = 384;
constexpr int kItems = 4;

// The k-th item, copied from its place (of PLACES) in shared memory; false: no more, or a wait ran out.
template <int PLACES>
__device__ __forceinline__ bool next_item(uint32_t bar_item, uint32_t bar_item_read, const Item* items, int k, Item& item,
                                          const Params& p) {
  if (!mbar_wait(bar_item + 8u * (k % PLACES), (k / PLACES) & 1, p)) return false;
  item = items[k % PLACES];
  mbar_arrive(bar_item_read + 8u * (k % PLACES));
  return item.at >= 0;
}

// The same by a whole issuing warp, one arrival for all lanes.
template <int PLACES>
__device__ __forceinline__ bool next_item_warp(uint32_t bar_item, uint32_t bar_item_read, const Item* items, int k,
                                               Item& item, const Params& p) {
  if (!__all_sync(0xffffffffu, mbar_wait(bar_item + 8u * (k % PLACES), (k / PLACES) & 1, p))) return false;
  item = items[k % PLACES];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar_item_read + 8u * (k % PLACES));
  return __any_sync(0xffffffffu, item.at >= 0);
}

// ------------------------------------------------------------------------------------------
// dq.  Warps: 0-3 columns 0..63 of S, 4-7 columns 64..127, 8 copies, 9 issues S and dP (and owns tensor
// memory), 10 issues dS K, 11 finds the work items and clears what a last K tile holds past its
// sequence's end.  S and dP are given back as soon as they are in registers, so that S_{j+1} and
// dP_{j+1} are computed while the weights of tile j are; dS has two buffers of its own.  (With dS_j written
// over one of two S buffers S_{j+1} had to wait for dQ_{j-1}.)  Products are in the pipe in 76 % of all clocks
// (four sequences of 8192 tokens).
// ------------------------------------------------------------------------------------------
// Its work items are taken as blocks come free (a counter in the workspace; which block takes an item changes
// nothing in it), and it runs after dkv_kernel, whose blocks end far apart where sequences are long (8192 tokens: a
// key tile meets up to 256 query tiles, and the mean block 219): it fills what they leave.  dq first and both dealt
// out ahead of time: 572 us for 550 (16 heads in 4 groups, D = 128), 386 for 373 with samples of 512 to
// 2048 tokens.  An item in one place is taken as late as can be; with 2, 3 and 4 places 561, 585 and 609 us.
constexpr int kDqItems = 1;

template <int D>
struct DqLayout {
  // K_{j+1} is needed for S while the weights of tile j are computed, when dQ_{j-1}, the last to read
  // K_{j-1}, has only just been issued: three places.  V_j is given back as soon as dP_j is computed.
  static constexpr int kKeep = D == 128 ? 3 : 4, kPass = D == 128 ? 2 : 4;
  static constexpr int kTile = kBlock * (D / 64);
  static constexpr int kQ = 0, kDo = kTile, kK = 2 * kTile, kV = kK + kKeep * kTile;
  static constexpr int kBars = kV + kPass * kTile;
  static constexpr int kNumBars = 2 * kKeep + 2 * kPass + 14 + 2 * kDqItems;
  static constexpr int kAlloc = kBars + kNumBars * 8 + 1024;
  static constexpr int kS = D, kDp = D + kKeys, kDs = D + 2 * kKeys;  // tensor memory: dQ, S, dP, dS[2]
  static_assert(kAlloc <= 232448 && kDs + kKeys <= 512, "memory budgets");
};

template <int D>
struct DqBars {
  using L = DqLayout<D>;
  uint32_t at;
  __device__ __forceinline__ uint32_t one(int i) const { return at + 8u * i; }
  static constexpr int kRest = 2 * (L::kKeep + L::kPass);
  __device__ __forceinline__ uint32_t k_full(int i) const { return one(i); }
  __device__ __forceinline__ uint32_t k_empty(int i) const { return one(L::kKeep + i); }
  __device__ __forceinline__ uint32_t v_full(int i) const { return one(2 * L::kKeep + i); }
  __device__ __forceinline__ uint32_t v_empty(int i) const { return one(2 * L::kKeep + L::kPass + i); }
  __device__ __forceinline__ uint32_t tail() const { return one(kRest); }
  __device__ __forceinline__ uint32_t q() const { return one(kRest + 1); }
  __device__ __forceinline__ uint32_t q_free() const { return one(kRest + 2); }
  __device__ __forceinline__ uint32_t s() const { return one(kRest + 3); }
  __device__ __forceinline__ uint32_t s_read() const { return one(kRest + 4); }
  __device__ __forceinline__ uint32_t dp() const { return one(kRest + 5); }
  __device__ __forceinline__ uint32_t dp_read() const { return one(kRest + 6); }
  __device__ __forceinline__ uint32_t ds(int i) const { return one(kRest + 7 + i); }
  __device__ __forceinline__ uint32_t dq(int i) const { return one(kRest + 9 + i); }
  __device__ __forceinline__ uint32_t o_free() const { return one(kRest + 11); }
  __device__ __forceinline__ uint32_t done(int i) const { return one(kRest + 12 + i); }
  __device__ __forceinline__ uint32_t item() const { return one(kRest + 14); }
  __device__ __forceinline__ uint32_t item_read() const { return one(kRest + 14 + kDqItems); }
};

// The largest of the values first .. end - 1, none negative, by a whole warp: of blocks of PER by their own
// largest, of those at either end that reach beyond, one by one.  The loads start with it; the answer may be
// asked for later.
template <int PER>
class Largest {
 public:
  __device__ __forceinline__ Largest(const float* each, const float* blocks, int64_t first, int64_t end)
      : blocks_(blocks), next_((first + PER - 1) / PER + threadIdx.x % 32), end_(end / PER) {
    const int lane = threadIdx.x % 32;
    const int64_t head = min(end, (first + PER - 1) / PER * PER), tail = max(head, end_ * PER);
#pragma unroll
    for (int i = 0; i < kEdge; ++i) {
      held_[2 * i] = first + 32 * i + lane < head ? each[first + 32 * i + lane] : 0.f;
      held_[2 * i + 1] = tail + 32 * i + lane < end ? each[tail + 32 * i + lane] : 0.f;
    }
    held_[2 * kEdge] = next_ < end_ ? blocks[next_] : 0.f;
  }

  __device__ __forceinline__ float get() {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i <= 2 * kEdge; ++i) top = fmaxf(top, held_[i]);
#pragma unroll 8
    for (int64_t b = next_ + 32; b < end_; b += 32) top = fmaxf(top, blocks_[b]);
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  }

 private:
  static constexpr int kEdge = PER / 32;
  const float* blocks_;
  int64_t next_, end_;
  float held_[2 * kEdge + 1];
};

// fp16: of a kv head's keys, or rows.
template <int D>
__device__ __forceinline__ Largest<row_block(D)> largest_value(const GradParams& g, int hk, int64_t first, int64_t end) {
  return {g.v_norms + static_cast<int64_t>(hk) * g.f.total_k, g.v_maxima + static_cast<int64_t>(hk) * g.k_blocks, first, end};
}
template <int D>
__device__ __forceinline__ Largest<row_block(D)> largest_norm(const GradParams& g, int hk, int64_t first, int64_t end) {
  return {g.norms + static_cast<int64_t>(hk) * g.f.total_q * g.f.G, g.maxima + static_cast<int64_t>(hk) * g.q_blocks, first, end};
}

// A place in a ring, and how often the ring has been gone through before it.
template <int SLOTS>
struct Place {
  int slot = 0, lap = 0;
  __device__ __forceinline__ Place next() const {
    Place n;
    n.slot = slot + 1 == SLOTS ? 0 : slot + 1;
    n.lap = slot + 1 == SLOTS ? lap + 1 : lap;
    return n;
  }
};

// Key tiles that a query tile sees.
__device__ __forceinline__ int key_tiles(const Params& p, const Seq& s, int q0) {
  const int last = min(s.nq, q0 + p.q_per_tile) - 1;
  const int end = p.causal ? min(s.nk, max(0, last + s.nk - s.nq + 1)) : s.nk;
  return (end + kKeys - 1) / kKeys;
}

// fp16: the largest finite |v| of the keys that dq_kernel's item walks over.
template <int D>
__device__ __forceinline__ float largest_seen(const GradParams& g, const Item& item) {
  const int64_t n = min(item.seq.nk, key_tiles(g.f, item.seq, item.at) * kKeys);
  return largest_value<D>(g, item.head, item.seq.k0, item.seq.k0 + n).get();
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const GradParams gp) {
  using L = DqLayout<D>;
  const Params& p = gp.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint32_t tmem_slot;
  __shared__ Item items[kDqItems];
  const uint32_t s_base = smem_addr(smem);
  const DqBars<D> bars{s_base + L::kBars};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 9) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 8 * 32) {
    for (int i = 0; i < L::kKeep; ++i) {
      mbar_init(bars.k_full(i), 1);
      mbar_init(bars.k_empty(i), 1);
    }
    for (int i = 0; i < L::kPass; ++i) {
      mbar_init(bars.v_full(i), 1);
      mbar_init(bars.v_empty(i), 1);
    }
    mbar_init(bars.tail(), 1);
    mbar_init(bars.q(), 1);
    mbar_init(bars.q_free(), 1);
    mbar_init(bars.s(), 1);
    mbar_init(bars.s_read(), 256);
    mbar_init(bars.dp(), 1);
    mbar_init(bars.dp_read(), 256);
    mbar_init(bars.o_free(), 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.ds(i), 256);
      mbar_init(bars.dq(i), 1);
      mbar_init(bars.done(i), 1);
    }
    for (int i = 0; i < kDqItems; ++i) {
      mbar_init(bars.item() + 8u * i, 1);
      mbar_init(bars.item_read() + 8u * i, 256 + 3);  // weights, issuers, copies
    }
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp == 11) {
    // ------------------------------ work items, K's last rows --------------------------------
    auto pieces = [&](int s, int& n, int& first) {
      const Seq q = load_seq(p, s);
      n = (q.nq + p.q_per_tile - 1) / p.q_per_tile;
      first = (p.causal ? max(0, q.nk - q.nq) : q.nk) / p.q_per_tile;
    };
    Finder finder(p.B, !p.causal, pieces);
    int tiles = 0, tails = 0;          // key tiles of the items so far; K tiles cleared
    int clear_at = -1, clear_row = 0;  // the item before: its last key tile, first row to clear
    bool ok = true, more = true;
    for (int k = 0; ok && (more || clear_at >= 0); ++k) {
      Item item{};
      item.at = -1;
      if (more) {
        int w = blockIdx.x;
        if (k > 0) {
          if (lane == 0) w = static_cast<int>(gridDim.x) + atomicAdd(gp.taken, 1);
          w = __shfl_sync(0xffffffffu, w, 0);
        }
        int b, t;
        finder.find(w / p.Hkv, pieces, b, t);
        if (b >= 0) {
          item.seq = load_seq(p, b);
          item.at = t * p.q_per_tile;
          item.head = w % p.Hkv;
          if constexpr (!BF16) item.value = largest_seen<D>(gp, item);
        }
        if (k >= kDqItems)
          ok = __all_sync(0xffffffffu, mbar_wait(bars.item_read() + 8u * (k % kDqItems), (k / kDqItems - 1) & 1, p));
        if (ok && lane == 0) {
          items[k % kDqItems] = item;
          mbar_arrive(bars.item() + 8u * (k % kDqItems));
        }
        more = b >= 0;
      }
      if (ok && clear_at >= 0) {
        // K rows past the sequence's end: dS is 0 there, but 0 times an infinity or NaN is not
        const int slot = clear_at % L::kKeep;
        ok = __all_sync(0xffffffffu, mbar_wait(bars.tail(), tails & 1, p));
        ++tails;
        if (ok) clear_rows<D>(smem + L::kK + slot * L::kTile, clear_row, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.k_full(slot));
        clear_at = -1;
      }
      if (item.at >= 0) {
        const int n = key_tiles(p, item.seq, item.at);
        tiles += n;
        if (n > 0 && n * kKeys > item.seq.nk) {
          clear_at = tiles - 1;
          clear_row = item.seq.nk - (n - 1) * kKeys;
        }
      }
    }
  } else if (warp == 8) {
    // ---------------------------------- copies ----------------------------------------------
    if (lane == 0) {
      bool ok = true;
      int tile = 0, uses = 0, tails = 0;  // key tiles; items with any; K tiles that land on the tail's barrier
      int tail_at = -1, k_only = -1;
      Item item;
      for (int k = 0; ok && next_item<kDqItems>(bars.item(), bars.item_read(), items, k, item, p); ++k) {
        const int n = key_tiles(p, item.seq, item.at);
        if (n == 0) continue;
        if (uses > 0 && !(ok = mbar_wait(bars.q_free(), (uses - 1) & 1, p))) break;
        ++uses;
        mbar_arrive_expect_tx(bars.q(), static_cast<uint32_t>(2 * 128 * (D / 64) * p.G * p.q_per_tile));
        for (int kb = 0; kb < D / 64; ++kb) {
          tma_load_3d(s_base + L::kQ + kb * kBlock, &tm_q, bars.q(), kb * 64, item.head * p.G, item.seq.q0 + item.at);
          tma_load_3d(s_base + L::kDo + kb * kBlock, &tm_do, bars.q(), kb * 64, item.head * p.G, item.seq.q0 + item.at);
        }
        const bool tail = n * kKeys > item.seq.nk;  // the last K tile reaches past the sequence
        for (int j = 0; j < n; ++j, ++tile) {
          const int kp = tile % L::kKeep, vp = tile % L::kPass;
          if (tile >= L::kKeep && !(ok = mbar_wait(bars.k_empty(kp), (tile / L::kKeep - 1) & 1, p))) break;
          uint32_t bar = bars.k_full(kp);
          if (tail && j == n - 1) {
            bar = bars.tail();
            tail_at = tile;
            ++tails;
          }
          mbar_arrive_expect_tx(bar, L::kTile);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kK + kp * L::kTile + kb * kBlock, &tm_k, bar, kb * 64, item.head, item.seq.k0 + j * kKeys);
          k_only = tile;
          if (tile >= L::kPass && !(ok = mbar_wait(bars.v_empty(vp), (tile / L::kPass - 1) & 1, p))) break;
          mbar_arrive_expect_tx(bars.v_full(vp), L::kTile);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kV + vp * L::kTile + kb * kBlock, &tm_v, bars.v_full(vp), kb * 64, item.head,
                        item.seq.k0 + j * kKeys);
          k_only = -1;
        }
      }
      if (!ok) {
        // A wait ran out: let the copies in flight land before the block ends.  (Each wait is for the last
        // copy to its barrier.)
        if (uses > 0) mbar_wait(bars.q(), (uses - 1) & 1, nullptr);
        const int k_end = k_only >= 0 ? tile + 1 : tile;
        for (int i = max(0, k_end - L::kKeep); i < k_end; ++i) {
          if (i == tail_at) mbar_wait(bars.tail(), (tails - 1) & 1, nullptr);
          else mbar_wait(bars.k_full(i % L::kKeep), (i / L::kKeep) & 1, nullptr);
        }
        for (int i = max(0, tile - L::kPass); i < tile; ++i)
          mbar_wait(bars.v_full(i % L::kPass), (i / L::kPass) & 1, nullptr);
      }
    }
  } else if (warp == 9 || warp == 10) {
    // ------------------- issuer 9: S = Q K^T and dP = dO V^T; issuer 10: dQ += dS K -------------------
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    bool ok = true;
    auto wait = [&](uint32_t bar, int phase) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, p));
      return ok;
    };
    Place<L::kKeep> kp;
    int step = 0, uses = 0;
    Item item;
    if (warp == 9) {
      constexpr uint32_t idesc = idesc_f16(BF16, kRows, kKeys, false, false);
      const uint64_t q_desc = sdesc_sw128(s_base + L::kQ, 16, 1024), do_desc = sdesc_sw128(s_base + L::kDo, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(s_base + L::kK, 16, 1024), v_desc = sdesc_sw128(s_base + L::kV, 16, 1024);
      Place<L::kPass> vp;
      for (int k = 0; ok && next_item_warp<kDqItems>(bars.item(), bars.item_read(), items, k, item, p); ++k) {
        const int n = uniform(key_tiles(p, item.seq, item.at));
        if (n == 0) continue;
        if (!wait(bars.q(), uses++)) break;
        for (int j = 0; j < n; ++j, ++step) {
          ok = step == 0 ? wait(bars.k_full(kp.slot), kp.lap)
                         : warp_wait(bars.k_full(kp.slot), kp.lap, bars.s_read(), step - 1, p);
          if (!ok) break;
          tc_fence_after();
          if (elected()) {
            product_ss<D>(tm + L::kS, q_desc, sdesc_add(k_desc, kp.slot * L::kTile), idesc);
            tc_commit(bars.s());
          }
          __syncwarp();
          ok = step == 0 ? wait(bars.v_full(vp.slot), vp.lap)
                         : warp_wait(bars.v_full(vp.slot), vp.lap, bars.dp_read(), step - 1, p);
          if (!ok) break;
          tc_fence_after();
          if (elected()) {
            product_ss<D>(tm + L::kDp, do_desc, sdesc_add(v_desc, vp.slot * L::kTile), idesc);
            tc_commit(bars.dp());
            tc_commit(bars.v_empty(vp.slot));
            if (j == n - 1) tc_commit(bars.q_free());
          }
          __syncwarp();
          kp = kp.next();
          vp = vp.next();
        }
      }
    } else {
      constexpr uint32_t idesc = idesc_f16(BF16, kRows, D, false, true);
      const uint64_t k_desc = sdesc_sw128(s_base + L::kK, kBlock, 1024);
      for (int k = 0; ok && next_item_warp<kDqItems>(bars.item(), bars.item_read(), items, k, item, p); ++k) {
        const int n = uniform(key_tiles(p, item.seq, item.at));
        if (n == 0) continue;
        // dQ of the item before has to be read before the first product overwrites it
        if (uses > 0 && !wait(bars.o_free(), uses - 1)) break;
        ++uses;
        for (int j = 0; j < n; ++j, ++step) {
          ok = warp_wait(bars.k_full(kp.slot), kp.lap, bars.ds(step & 1), step / 2, p);
          if (!ok) break;
          tc_fence_after();
          if (elected()) {
            product_ts(tm, tm + L::kDs + (step & 1) * (kKeys / 2), kHalf / 2, sdesc_add(k_desc, kp.slot * L::kTile), idesc, j == 0);
            tc_commit(bars.dq(step & 1));
            tc_commit(bars.k_empty(kp.slot));
          }
          __syncwarp();
          kp = kp.next();
        }
      }
    }
    // every product must finish before tensor memory and the ring are given up
    if (elected()) {
      tc_commit(bars.done(warp - 9));
      mbar_wait(bars.done(warp - 9), 0, nullptr);
    }
  } else {
    // ------------------------- weights: a row and 64 columns a thread -------------------------
    const int w = warp / 4, r = threadIdx.x % 128;  // half of the columns
    const int row_token = r / p.G, row_head = r % p.G;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const float2 a2 = make_float2(p.scale_log2, p.scale_log2);
    const uint32_t tm_s = tmem + L::kS + w * kHalf + lanes, tm_dp = tmem + L::kDp + w * kHalf + lanes;
    bool ok = true;
    int step = 0;
    // The item before, whose dQ is still in tensor memory: if the first scores of the next are there, they are
    // dealt with first, so that the wait for its last product, and the stores, have work beside them.
    bool pending = false;
    uint16_t* out_row = nullptr;
    float out_scale = 0.f;
    int out_step = 0;
    bool more = true;
    for (int k = 0; ok && more; ++k) {
      Item item{};
      more = __all_sync(0xffffffffu, next_item<kDqItems>(bars.item(), bars.item_read(), items, k, item, p));
      const int n = more ? key_tiles(p, item.seq, item.at) : 0;
      const int i = item.at + row_token, h = item.head * p.G + row_head;
      const bool valid = more && r < p.G * p.q_per_tile && i < item.seq.nq;
      const int64_t row = item.seq.q0 + i;
      const int64_t at = (item.head * static_cast<int64_t>(p.total_q) + row) * p.G + row_head;
      const float2 rd = valid ? gp.rows[at] : make_float2(-INFINITY, 0.f);
      const float norm = !BF16 && valid ? gp.norms[at] : 0.f;
      // (a row of no query is not looked at by anyone: it may see everything)
      const int key_lim = !valid ? 0x7fffffff : p.causal ? min(item.seq.nk, i + item.seq.nk - item.seq.nq + 1) : item.seq.nk;
      const float delta = key_lim >= 1 && key_lim <= kFew ? gp.few[at] : rd.y;
      const float f = BF16 ? 1.f : power_for(norm * item.value);
      const float fd = key_lim == 1 ? 0.f : f;
      const float2 nl2 = make_float2(rd.x, rd.x), f2 = make_float2(fd, fd), nd2 = make_float2(-delta * fd, -delta * fd);
      for (int j = -1; j < n; ++j) {
        if (j >= 0) {
          // S_step; and dS_{step-2} read, before dS_step takes its place
          ok = step < 2 ? __all_sync(0xffffffffu, mbar_wait(bars.s(), step & 1, p))
                        : warp_wait(bars.dq(step & 1), step / 2 - 1, bars.s(), step, p);
          if (!ok) break;
          tc_fence_after();
          const int left = key_lim - (j * kKeys + w * kHalf);  // columns that the row sees
          uint32_t raw[2][32];
          tmem_ld32(tm_s, raw[0]);
          tmem_ld32(tm_s + 32, raw[1]);
          prefill::tmem_ld_wait_tied(raw[0]);
          prefill::tmem_ld_wait_tied(raw[1]);
          tc_fence_before();
          mbar_arrive(bars.s_read());
          float2 x[32];
          const bool whole = __all_sync(0xffffffffu, left >= kHalf);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 t = __ffma2_rn(make_float2(__uint_as_float(raw[c / 16][(2 * c) % 32]),
                                                    __uint_as_float(raw[c / 16][(2 * c) % 32 + 1])), a2, nl2);
            x[c] = make_float2(exp2_approx(t.x), exp2_approx(t.y));
          }
          ok = __all_sync(0xffffffffu, mbar_wait(bars.dp(), step & 1, p));
          if (!ok) break;
          tc_fence_after();
          uint32_t dp[2][32], ds[32];
          tmem_ld32(tm_dp, dp[0]);
          prefill::tmem_ld_wait_tied(dp[0]);
          tmem_ld32(tm_dp + 32, dp[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q == 1) {
              prefill::tmem_ld_wait_tied(dp[1]);
              tc_fence_before();
              mbar_arrive(bars.dp_read());
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 t = __ffma2_rn(make_float2(__uint_as_float(dp[q][2 * c]), __uint_as_float(dp[q][2 * c + 1])), f2, nd2);
              ds[16 * q + c] = pack<BF16>(__fmul2_rn(x[16 * q + c], t));
            }
          }
          if (!whole) {
            // what a hidden column holds may be another sequence's, or no number: replaced, not multiplied
#pragma unroll
            for (int c = 0; c < 32; ++c)
              ds[c] &= (2 * c < left ? 0xffffu : 0u) | (2 * c + 1 < left ? 0xffff0000u : 0u);
          }
          tmem_st32(tmem + L::kDs + (step & 1) * (kKeys / 2) + w * (kHalf / 2) + lanes, ds);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bars.ds(step & 1));
          ++step;
        }
        if (pending && (j == 0 || n == 0 || !__all_sync(0xffffffffu, mbar_test_wait(bars.s(), step & 1)))) {
          pending = false;
          ok = __all_sync(0xffffffffu, mbar_wait(bars.dq(out_step & 1), (out_step / 2) & 1, p));
          if (!ok) break;
          tc_fence_after();
          uint32_t o[D / 64][32];
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tmem_ld32(tmem + lanes + w * (D / 2) + c * 32, o[c]);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) prefill::tmem_ld_wait_tied(o[c]);
          tc_fence_before();
          mbar_arrive(bars.o_free());
#pragma unroll
          for (int c = 0; c < D / 64; ++c) store32<BF16>(out_row ? out_row + c * 32 : nullptr, o[c], out_scale);
        }
      }
      if (!ok || !more) break;
      uint16_t* dst = valid ? static_cast<uint16_t*>(gp.dq) + row * gp.dq_strides[0] + h * gp.dq_strides[1] + w * (D / 2) : nullptr;
      if (n > 0) {
        pending = true;
        out_row = dst;
        out_scale = p.scale / f;
        out_step = step - 1;
      } else if (dst) {  // rows that see no key
        for (int c = 0; c < D / 16; ++c) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  wait_for_previous();  // nothing of dkv_kernel's is read here; but what follows this kernel counts on its end
}

// ------------------------------------------------------------------------------------------
// dk and dv.  Warps: 0-3 query columns 0..63 of S^T, 4-7 columns 64..127, 8 copies, 9 issues dV and S^T
// (and owns tensor memory), 10 issues dK and dP^T, 11 finds the work items, brings each query row's
// lse and delta and clears query rows past a sequence's end.  Tensor memory is full at D = 128 (dV, dK,
// S^T, dP^T): P^T lies over S^T and dS^T over dP^T, and issuer 9 puts S^T_{i+1} right behind dV_i
// (issuer 10 dP^T_{i+1} behind dK_i), which reads what it overwrites: products of one thread and
// one shape run in order.  While the element-wise warps work on S^T the tensor cores run dK and
// dP^T, and the other way round: products are in the pipe in 75 % of all clocks (four sequences of 8192 tokens).
// Without turns of the two issuers 604 us for 575 of the whole gradient (one of 8192 tokens, dq first), with the turn
// given earlier 594, after the commits 602.  At D = 64, where the shapes differ, P^T and dS^T have columns of
// their own.
// ------------------------------------------------------------------------------------------
// fp16: the largest |v| of a sequence and head, kept from one work item to the next of both, by head.  (Found anew by
// every item: 16 queries of 24 heads in 3 groups over 2^20 keys 7977 us for 6918.)
struct Values {
  int k0, nk, head;
  float value;
};
constexpr int kKept = 16;

template <int D>
struct DkvLayout {
  // Ring of Q and dO tiles by turns.  Q_{i+1} is needed as soon as dK_{i-1}, the last to read Q_{i-1}, is
  // done: with two places for Q the load would be waited for every tile (D = 128: 3930 clocks a tile).
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kTile = kBlock * (D / 64);
  static constexpr int kK = 0, kV = kTile, kRing = 2 * kTile;
  static constexpr int kRowData = kRing + kSlots * kTile;    // [2][-lse, -delta][128] fp32
  static constexpr int kBars = kRowData + 2 * 2 * kRows * 4;
  static constexpr int kNumBars = 2 * kSlots + 15 + 2 * kItems;
  static constexpr int kShared = kBars + kNumBars * 8;       // work items, turns, tensor memory's address
  // No room is left to align the base by hand: the kernel has no static shared memory, and its dynamic
  // one is declared with this alignment.
  static constexpr int kPowers = kShared + static_cast<int>(kItems * sizeof(Item)) + 16;  // fp16: [2], beside the row data
  static constexpr int kValues = (kPowers + 2 * 4 + 15) / 16 * 16;  // fp16: [kKept]
  static constexpr int kAlloc = kValues + kKept * 16;
  static constexpr bool kApart = D == 64;
  static constexpr int kDv = 0, kDk = D, kS = 2 * D, kDp = kS + kRows;
  static constexpr int kP = kApart ? kDp + kRows : kS, kDs = kApart ? kP + kRows / 2 : kDp;
  static constexpr int kStep = kApart ? kHalf / 2 : kHalf;  // between the two halves of P^T, of dS^T
  static_assert(kAlloc <= 232448 && kDs + kRows / 2 <= 512, "memory budgets");
};

template <int D>
struct DkvBars {
  using L = DkvLayout<D>;
  uint32_t at;
  __device__ __forceinline__ uint32_t one(int i) const { return at + 8u * i; }
  __device__ __forceinline__ uint32_t full(int slot) const { return one(slot); }
  __device__ __forceinline__ uint32_t empty(int slot) const { return one(L::kSlots + slot); }
  __device__ __forceinline__ uint32_t tail() const { return one(2 * L::kSlots); }
  __device__ __forceinline__ uint32_t kv() const { return one(2 * L::kSlots + 1); }
  __device__ __forceinline__ uint32_t kv_free() const { return one(2 * L::kSlots + 2); }
  __device__ __forceinline__ uint32_t rows(int i) const { return one(2 * L::kSlots + 3 + i); }
  __device__ __forceinline__ uint32_t rows_read(int i) const { return one(2 * L::kSlots + 5 + i); }
  // x = 0: S^T, P^T, dV; 1: dP^T, dS^T, dK
  __device__ __forceinline__ uint32_t first(int x) const { return one(2 * L::kSlots + 7 + x); }
  __device__ __forceinline__ uint32_t packed(int x) const { return one(2 * L::kSlots + 9 + x); }
  __device__ __forceinline__ uint32_t second(int x) const { return one(2 * L::kSlots + 11 + x); }
  __device__ __forceinline__ uint32_t done(int x) const { return one(2 * L::kSlots + 13 + x); }
  __device__ __forceinline__ uint32_t item() const { return one(2 * L::kSlots + 15); }
  __device__ __forceinline__ uint32_t item_read() const { return one(2 * L::kSlots + 15 + kItems); }
};

// First query tile that sees a key of the tile at key0, and how many tiles from there on there are.
__device__ __forceinline__ int query_tiles(const Params& p, const Seq& s, int key0, int& first) {
  first = p.causal ? max(0, key0 - (s.nk - s.nq)) / p.q_per_tile : 0;
  return max(0, (s.nq + p.q_per_tile - 1) / p.q_per_tile - first);
}

// The issuing warp of S^T and dV (X = 0) or of dP^T and dK (X = 1).  A tile's first product reads its own
// ring entry (Q for S^T, dO for dP^T), its second the other's.
template <int D, bool BF16, int X>
__device__ __forceinline__ void issue_pair(const Params& p, uint32_t s_base, uint32_t bar_base, uint32_t tmem, const Item* items,
                                           volatile int* turns) {
  using L = DkvLayout<D>;
  const DkvBars<D> bars{bar_base};
  constexpr uint32_t idesc1 = idesc_f16(BF16, kRows, kRows, false, false);
  constexpr uint32_t idesc2 = idesc_f16(BF16, kRows, D, false, true);
  tmem = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
  const uint64_t left = sdesc_sw128(s_base + (X ? L::kV : L::kK), 16, 1024);
  const uint64_t ring1 = sdesc_sw128(s_base + L::kRing, 16, 1024), ring2 = sdesc_sw128(s_base + L::kRing, kBlock, 1024);
  const uint32_t tm1 = tmem + (X ? L::kDp : L::kS), tm2 = tmem + (X ? L::kDk : L::kDv), tm_a = tmem + (X ? L::kDs : L::kP);
  bool ok = true;
  auto wait = [&](uint32_t bar, int phase) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, p));
    return ok;
  };
  Place<L::kSlots> q;  // of the tile's Q; its dO is the next
  int step = 0, uses = 0;
  Item item;
  for (int k = 0; ok && next_item_warp<kItems>(bars.item(), bars.item_read(), items, k, item, p); ++k) {
    int first_tile;
    const int n = uniform(query_tiles(p, item.seq, item.at, first_tile));
    if (n == 0) continue;
    const Place<L::kSlots> start = X ? q.next() : q;
    if (!wait(bars.kv(), uses) || !wait(bars.full(start.slot), start.lap)) break;
    tc_fence_after();
    if (elected()) {
      product_ss<D>(tm1, left, sdesc_add(ring1, start.slot * L::kTile), idesc1);
      tc_commit(bars.first(X));
      tc_commit(bars.empty(start.slot));
      if (n == 1) tc_commit(bars.kv_free());
    }
    __syncwarp();
    for (int i = 0; i < n; ++i, ++step) {
      const Place<L::kSlots> d = q.next(), q2 = d.next();
      const Place<L::kSlots> other = X ? q : d, mine = X ? q2.next() : q2;
      q = q2;
      if (!wait(bars.full(other.slot), other.lap)) break;
      if (i + 1 < n && !wait(bars.full(mine.slot), mine.lap)) break;
      // (the sums of the item before have been read: the weights of this one's first tile come after that)
      // The other pair's turn first (dV and S^T of a tile before dK and dP^T, these before the next): one
      // pair's products are not to wait behind half of the other's.  Only an order: the wait may give up.
      for (int spin = 0; spin < 4096 && turns[1 - X] < (X ? step + 1 : step); ++spin) {}
      if (!wait(bars.packed(X), step)) break;
      tc_fence_after();
      if (elected()) {
        product_ts(tm2, tm_a, L::kStep, sdesc_add(ring2, other.slot * L::kTile), idesc2, i == 0);
        if (i + 1 < n) product_ss<D>(tm1, left, sdesc_add(ring1, mine.slot * L::kTile), idesc1);
        turns[X] = step + 1;  // (before the commits: after them the store would wait for the products)
        tc_commit(bars.second(X));
        tc_commit(bars.empty(other.slot));
        if (i + 1 < n) {
          tc_commit(bars.first(X));
          tc_commit(bars.empty(mine.slot));
          if (i + 2 == n) tc_commit(bars.kv_free());
        }
      }
      __syncwarp();
    }
    ++uses;
  }
  // every product must finish before tensor memory and the ring are given up
  if (elected()) {
    tc_commit(bars.done(X));
    mbar_wait(bars.done(X), 0, nullptr);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const GradParams gp) {
  using L = DkvLayout<D>;
  constexpr float kPower = BF16 ? 0.f : 7.f;             // P is held times 2^kPower
  constexpr float kUnpower = BF16 ? 1.f : 0.0078125f;    // 2^-kPower
  const Params& p = gp.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  Item* items = reinterpret_cast<Item*>(smem + L::kShared);
  int* turns = reinterpret_cast<int*>(items + kItems);  // pairs of products that each issuer has put into the pipe
  uint32_t& tmem_slot = reinterpret_cast<uint32_t*>(turns)[2];
  const uint32_t s_base = smem_addr(smem);
  const DkvBars<D> bars{s_base + L::kBars};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int used = p.G * p.q_per_tile;  // rows of a query tile
  if (warp == 9) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 8 * 32) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(bars.full(i), 1);
      mbar_init(bars.empty(i), 2);  // both issuers
    }
    mbar_init(bars.tail(), 1);
    mbar_init(bars.kv(), 1);
    mbar_init(bars.kv_free(), 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.rows(i), 32);
      mbar_init(bars.rows_read(i), 256);
      mbar_init(bars.first(i), 1);
      mbar_init(bars.packed(i), 256);
      mbar_init(bars.second(i), 1);
      mbar_init(bars.done(i), 1);
      turns[i] = 0;
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bars.item() + 8u * i, 1);
      mbar_init(bars.item_read() + 8u * i, 256 + 3);  // weights, issuers, copies
    }
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (used < kRows) {
    // Rows that no copy writes are summed over all the same: zero, once.
    for (int s = 0; s < L::kSlots; ++s)
      clear_rows<D>(smem + L::kRing + s * L::kTile, used, threadIdx.x, kThreads);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp == 11) {
    // --------------- work items; lse and delta of each query row; rows past the end ----------------
    wait_for_previous();  // row_kernel
    if (lane == 0) let_next_start();
    auto pieces = [&](int s, int& n, int& first) {
      const Seq q = load_seq(p, s);
      n = (q.nk + kKeys - 1) / kKeys;
      first = p.causal ? 0 : q.nq / kKeys;
    };
    Finder finder(p.B, !p.causal, pieces);
    auto find = [&](int k) {
      Item item{};
      item.at = -1;
      const int rank = dealt(k);
      int b, t;
      finder.find(rank / p.Hkv, pieces, b, t);
      if (b >= 0) {
        item.seq = load_seq(p, b);
        // a piece's work grows with its index: the first keys, which most queries see, come last
        item.at = (p.causal ? (item.seq.nk + kKeys - 1) / kKeys - 1 - t : t) * kKeys;
        item.head = rank % p.Hkv;
      }
      return item;
    };
    bool ok = true;
    auto publish = [&](int k, const Item& item) {
      if (k >= kItems)
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bars.item_read() + 8u * (k % kItems), (k / kItems - 1) & 1, p));
      if (ok && lane == 0) {
        items[k % kItems] = item;
        mbar_arrive(bars.item() + 8u * (k % kItems));
      }
    };
    float power = 1.f;  // that the item's dS is held times
    Values* kept = reinterpret_cast<Values*>(smem + L::kValues);
    if (!BF16 && lane < kKept) kept[lane].head = -1;
    __syncwarp();
    int step = 0, tails = 0;
    int token[4];  // of the tile's, of the lane's rows
#pragma unroll
    for (int e = 0; e < 4; ++e) token[e] = (lane * 4 + e) / p.G;
    Item item = find(0);
    publish(0, item);
    for (int k = 0; ok && item.at >= 0; ++k) {
      int first_tile;
      const int n = query_tiles(p, item.seq, item.at, first_tile);
      Item ahead;
      auto look_ahead = [&]() {
        ahead = find(k + 1);
        publish(k + 1, ahead);
      };
      if constexpr (BF16) {
        look_ahead();
      } else {
        // The item's power goes with the row data and not with the item, so that the first tiles' copies and products do not
        // wait for it, and what it is found from loads beside the search (after it, three short samples took 0.8 us more).
        // |v| is of all of the sequence's keys, for delta is a mean over them.
        const int64_t key = item.seq.k0, row = item.seq.q0 + static_cast<int64_t>(first_tile) * p.q_per_tile;
        Values now = kept[item.head % kKept];
        const bool known = n == 0 || (now.head == item.head && now.k0 == item.seq.k0 && now.nk == item.seq.nk);
        auto value = largest_value<D>(gp, item.head, key, known ? key : key + item.seq.nk);
        auto norm = largest_norm<D>(gp, item.head, row * p.G, n > 0 ? (item.seq.q0 + static_cast<int64_t>(item.seq.nq)) * p.G : row * p.G);
        look_ahead();
        if (!known) {
          now = {item.seq.k0, item.seq.nk, item.head, value.get()};
          if (lane == 0) kept[item.head % kKept] = now;
          __syncwarp();
        }
        power = power_for(now.value * norm.get());
      }
      const int last_rows = n > 0 ? (item.seq.nq - (first_tile + n - 1) * p.q_per_tile) * p.G : used;
      for (int i = 0; ok && i < n; ++i, ++step) {
        const int q0 = (first_tile + i) * p.q_per_tile;
        const int live = min(used, (item.seq.nq - q0) * p.G);  // rows of the tile that are a query's
        const int64_t at = (item.head * static_cast<int64_t>(p.total_q) + item.seq.q0 + q0) * p.G + lane * 4;
        float nl[4], nd[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          nl[e] = -INFINITY;  // no query: P = 0
          nd[e] = 0.f;
          if (lane * 4 + e < live) {
            const float2 rd = gp.rows[at + e];
            const int sees = p.causal ? q0 + token[e] + item.seq.nk - item.seq.nq + 1 : item.seq.nk;
            nl[e] = rd.x + kPower;
            nd[e] = sees >= 1 && sees <= kFew ? gp.few[at + e] : rd.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) nd[e] *= -kUnpower * power;
        if (step >= 2)
          ok = __all_sync(0xffffffffu, mbar_wait(bars.rows_read(step & 1), (step / 2 - 1) & 1, p));
        float* to = reinterpret_cast<float*>(smem + L::kRowData) + (step & 1) * 2 * kRows + lane * 4;
        if (ok) {
          *reinterpret_cast<float4*>(to) = make_float4(nl[0], nl[1], nl[2], nl[3]);
          *reinterpret_cast<float4*>(to + kRows) = make_float4(nd[0], nd[1], nd[2], nd[3]);
          if (!BF16 && lane == 0) reinterpret_cast<float*>(smem + L::kPowers)[step & 1] = power;
          mbar_arrive(bars.rows(step & 1));
        }
        if (ok && i == n - 1 && last_rows < used) {
          // query rows past the sequence's end, which the sums over rows must not see
          ok = __all_sync(0xffffffffu, mbar_wait(bars.tail(), tails & 1, p));
          ++tails;
          for (int x = 0; ok && x < 2; ++x)
            clear_rows<D>(smem + L::kRing + (2 * step + x) % L::kSlots * L::kTile, last_rows, lane, 32);
          fence_proxy_async_smem();
          __syncwarp();
          if (ok && lane < 2) mbar_arrive(bars.full((2 * step + lane) % L::kSlots));
        }
      }
      item = ahead;
    }
  } else if (warp == 8) {
    // ---------------------------------- copies ----------------------------------------------
    if (lane == 0) {
      bool ok = true;
      int entry = 0, uses = 0, tails = 0, tail_at = -1;
      const uint32_t bytes = static_cast<uint32_t>(128 * (D / 64) * used);
      Item item;
      for (int k = 0; ok && next_item<kItems>(bars.item(), bars.item_read(), items, k, item, p); ++k) {
        int first_tile;
        const int n = query_tiles(p, item.seq, item.at, first_tile);
        if (n == 0) continue;
        if (uses > 0 && !(ok = mbar_wait(bars.kv_free(), (uses - 1) & 1, p))) break;
        ++uses;
        mbar_arrive_expect_tx(bars.kv(), 2 * L::kTile);
        for (int kb = 0; kb < D / 64; ++kb) {
          tma_load_3d(s_base + L::kK + kb * kBlock, &tm_k, bars.kv(), kb * 64, item.head, item.seq.k0 + item.at);
          tma_load_3d(s_base + L::kV + kb * kBlock, &tm_v, bars.kv(), kb * 64, item.head, item.seq.k0 + item.at);
        }
        const bool tail = (item.seq.nq - (first_tile + n - 1) * p.q_per_tile) * p.G < used;
        for (int i = 0; ok && i < 2 * n; ++i, ++entry) {  // Q, dO, Q, dO, ...
          const int slot = entry % L::kSlots, lap = entry / L::kSlots;
          if (lap > 0 && !(ok = mbar_wait(bars.empty(slot), (lap - 1) & 1, p))) break;
          const bool in_tail = tail && i >= 2 * n - 2;
          const uint32_t bar = in_tail ? bars.tail() : bars.full(slot);
          // (the tail's barrier counts one arrival, for both of its copies)
          if (!in_tail) {
            mbar_arrive_expect_tx(bar, bytes);
          } else if (i == 2 * n - 2) {
            tail_at = entry;
            ++tails;
            mbar_arrive_expect_tx(bar, 2 * bytes);
          }
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kRing + slot * L::kTile + kb * kBlock, (i & 1) ? &tm_do : &tm_q, bar, kb * 64,
                        item.head * p.G, item.seq.q0 + (first_tile + i / 2) * p.q_per_tile);
        }
      }
      if (!ok) {
        // A wait ran out: let the copies in flight land before the block ends.  (Of the tail's two the first
        // alone may be on its way: its barrier then does not complete, and the wait's own limit, far longer
        // than a copy takes, stands for it.)
        if (uses > 0) mbar_wait(bars.kv(), (uses - 1) & 1, nullptr);
        for (int i = max(0, entry - L::kSlots); i < entry; ++i) {
          if (tail_at >= 0 && (i == tail_at || i == tail_at + 1)) mbar_wait(bars.tail(), (tails - 1) & 1, nullptr);
          else mbar_wait(bars.full(i % L::kSlots), (i / L::kSlots) & 1, nullptr);
        }
      }
    }
  } else if (warp == 9) {
    issue_pair<D, BF16, 0>(p, s_base, bars.at, tmem, items, turns);
  } else if (warp == 10) {
    issue_pair<D, BF16, 1>(p, s_base, bars.at, tmem, items, turns);
  } else {
    // -------------------- weights: a key and 64 query columns a thread ------------------------
    const int w = warp / 4, r = threadIdx.x % 128;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tm_s = tmem + L::kS + w * kHalf + lanes, tm_dp = tmem + L::kDp + w * kHalf + lanes;
    const uint32_t tm_p = tmem + L::kP + w * L::kStep + lanes, tm_ds = tmem + L::kDs + w * L::kStep + lanes;
    float f = 1.f;  // that the item's dS is held times
    float2 f2 = make_float2(kUnpower, kUnpower);
    const float2 a2 = make_float2(p.scale_log2, p.scale_log2);
    bool ok = true;
    int step = 0;
    Item item;
    for (int k = 0; ok && __all_sync(0xffffffffu, next_item<kItems>(bars.item(), bars.item_read(), items, k, item, p)); ++k) {
      int first_tile;
      const int n = query_tiles(p, item.seq, item.at, first_tile);
      const int key = item.at + r;
      // Columns below `from` are queries in front of the key.  (Held at 0 or more before the product: a context of more
      // than 2^31 / G keys would pass 32 bits.  From there down it falls by the rows of a sequence, below 2^31, at most.)
      int from = p.causal ? max(0, key - (item.seq.nk - item.seq.nq) - first_tile * p.q_per_tile) * p.G - w * kHalf : 0;
      for (int i = 0; i < n; ++i, ++step, from -= used) {
        const float4* row_data = reinterpret_cast<const float4*>(smem + L::kRowData) + (step & 1) * 64 + w * 16;
        ok = __all_sync(0xffffffffu, mbar_wait(bars.rows(step & 1), (step / 2) & 1, p));
        // (read before S^T is waited for: beside the products, which take all of shared memory's bandwidth,
        // these reads cost 250 clocks)
        float4 nl[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) nl[c] = row_data[c];
        if (!BF16 && i == 0) {
          f = reinterpret_cast<const float*>(smem + L::kPowers)[step & 1];
          f2 = make_float2(f * kUnpower, f * kUnpower);
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bars.first(0), step & 1, p));
        if (!ok) break;
        tc_fence_after();
        const bool whole = !p.causal || __all_sync(0xffffffffu, from <= 0);
        uint32_t raw[2][32];
        tmem_ld32(tm_s, raw[0]);
        tmem_ld32(tm_s + 32, raw[1]);
        prefill::tmem_ld_wait_tied(raw[0]);
        prefill::tmem_ld_wait_tied(raw[1]);
        float2 x[32];
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 t = __ffma2_rn(make_float2(__uint_as_float(raw[c / 8][(4 * c) % 32]),
                                                  __uint_as_float(raw[c / 8][(4 * c) % 32 + 1])), a2, make_float2(nl[c].x, nl[c].y));
          const float2 u = __ffma2_rn(make_float2(__uint_as_float(raw[c / 8][(4 * c) % 32 + 2]),
                                                  __uint_as_float(raw[c / 8][(4 * c) % 32 + 3])), a2, make_float2(nl[c].z, nl[c].w));
          x[2 * c] = make_float2(exp2_approx(t.x), exp2_approx(t.y));
          x[2 * c + 1] = make_float2(exp2_approx(u.x), exp2_approx(u.y));
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = make_float2(2 * c >= from ? x[c].x : 0.f, 2 * c + 1 >= from ? x[c].y : 0.f);
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = pack<BF16>(x[c]);
        // (P^T_{i-1} has been read: the commit that told of S^T_i covers dV_{i-1} before it)
        tmem_st32(tm_p, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bars.packed(0));
        ok = __all_sync(0xffffffffu, mbar_wait(bars.first(1), step & 1, p));
        if (!ok) break;
        tc_fence_after();
        uint32_t dp[2][32], ds[32];
        tmem_ld32(tm_dp, dp[0]);
        prefill::tmem_ld_wait_tied(dp[0]);
        tmem_ld32(tm_dp + 32, dp[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1) prefill::tmem_ld_wait_tied(dp[1]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float4 nd = row_data[32 + 8 * q + c];
            const float2 t = __ffma2_rn(make_float2(__uint_as_float(dp[q][4 * c]), __uint_as_float(dp[q][4 * c + 1])), f2,
                                        make_float2(nd.x, nd.y));
            const float2 u = __ffma2_rn(make_float2(__uint_as_float(dp[q][4 * c + 2]), __uint_as_float(dp[q][4 * c + 3])), f2,
                                        make_float2(nd.z, nd.w));
            ds[16 * q + 2 * c] = pack<BF16>(__fmul2_rn(x[16 * q + 2 * c], t));
            ds[16 * q + 2 * c + 1] = pack<BF16>(__fmul2_rn(x[16 * q + 2 * c + 1], u));
          }
        }
        mbar_arrive(bars.rows_read(step & 1));
        tmem_st32(tm_ds, ds);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bars.packed(1));
      }
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bars.second(w), (step - 1) & 1, p));
        tc_fence_after();
      }
      if (!ok) break;
      // dv by the first four warps, dk by the others
      const int64_t row = item.seq.k0 + key;
      uint16_t* dst = w ? static_cast<uint16_t*>(gp.dk) + row * gp.dk_strides[0] + item.head * gp.dk_strides[1]
                        : static_cast<uint16_t*>(gp.dv) + row * gp.dv_strides[0] + item.head * gp.dv_strides[1];
      if (key >= item.seq.nk) dst = nullptr;
      // (the only key of a sequence: no dS but 0)
      const float back = w ? (item.seq.nk == 1 ? 0.f : p.scale / f) : kUnpower;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(tmem + (w ? L::kDk : L::kDv) + lanes + c * 32, o);
          prefill::tmem_ld_wait_tied(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        store32<BF16>(dst ? dst + c * 32 : nullptr, o, back);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16>
cudaError_t launch(const GradParams& g, const CUtensorMap (&maps)[4], int64_t q_items, int64_t k_items, cudaStream_t st) {
  auto kq = dq_kernel<D, BF16>;
  auto kk = dkv_kernel<D, BF16>;
  cudaError_t e = ensure_smem_limit(kq, DqLayout<D>::kAlloc);
  if (e == cudaSuccess) e = ensure_smem_limit(kk, DkvLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t sms = num_sms() > 0 ? num_sms() : 152;
  auto blocks = [&](int64_t items) { return static_cast<unsigned>(items * g.f.Hkv < sms ? items * g.f.Hkv : sms); };
  if (q_items > 0) {
    row_kernel<D, BF16><<<dim3(g.few_blocks + g.q_blocks + g.k_blocks, g.f.Hkv), kRowThreads, 0, st>>>(g);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // dq_kernel reads nothing of dkv_kernel's, whose blocks let it start once row_kernel has ended: it takes
  // each SM as dkv_kernel leaves it.  (Without the one ahead, what is ahead is not known: a plain launch.)
  if (k_items > 0) {
    if (q_items > 0) {
      e = launch_dependent(kk, blocks(k_items), 1, kThreads, DkvLayout<D>::kAlloc, st, maps[0], maps[1], maps[2], maps[3], g);
      if (e != cudaSuccess) return e;
      return launch_dependent(kq, blocks(q_items), 1, kThreads, DqLayout<D>::kAlloc, st, maps[0], maps[1], maps[2], maps[3], g);
    }
    kk<<<blocks(k_items), kThreads, DkvLayout<D>::kAlloc, st>>>(maps[0], maps[1], maps[2], maps[3], g);
  } else if (q_items > 0) {
    kq<<<blocks(q_items), kThreads, DqLayout<D>::kAlloc, st>>>(maps[0], maps[1], maps[2], maps[3], g);
  }
  return cudaGetLastError();
}

size_t round_up(size_t bytes) { return (bytes + 255) / 256 * 256; }

size_t row_bytes(const fa_packed_backward_args* a) {
  return round_up(static_cast<size_t>(a->total_q) * a->Hq * sizeof(float2));
}

size_t num_maxima(const fa_packed_backward_args* a) {
  return static_cast<size_t>(row_blocks(a->total_q, a->Hq / a->Hkv, a->D)) * a->Hkv;
}

// In front: the items taken; fp16: the largest |v| of each block of keys and of each key.
size_t front_bytes(const fa_packed_backward_args* a) {
  const size_t values = a->dtype == FA_FP16 ? (static_cast<size_t>(row_blocks(a->total_k, 1, a->D)) + a->total_k) * a->Hkv : 0;
  return round_up(sizeof(int) + values * sizeof(float));
}

size_t workspace_bytes(const fa_packed_backward_args* a) {
  return front_bytes(a) + row_bytes(a) + round_up(row_bytes(a) / 2) +
         (a->dtype == FA_FP16 ? round_up(row_bytes(a) / 2) + round_up(num_maxima(a) * sizeof(float)) : 0);
}

}  // namespace
}  // namespace packed
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_packed_backward_workspace_size(const fa_packed_backward_args* a) {
  if (!a || packed::check_sizes("fa_prefill_packed_backward", a->B, a->Hq, a->Hkv, a->D, a->total_q, a->total_k,
                                a->dtype, a->scale) != FA_OK)
    return 0;
  return a->B == 0 || a->total_q + static_cast<int64_t>(a->total_k) == 0 ? 0 : packed::workspace_bytes(a);
}

int fa_prefill_packed_backward(const fa_packed_backward_args* a, void* stream) {
  const char* who = "fa_prefill_packed_backward";
  if (!a) return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed_backward: null argument struct");
  int rc = packed::check_sizes(who, a->B, a->Hq, a->Hkv, a->D, a->total_q, a->total_k, a->dtype, a->scale);
  if (rc != FA_OK || a->B == 0 || a->total_q + static_cast<int64_t>(a->total_k) == 0) return rc;
  if ((rc = packed::check_offsets(who, a->cu_seqlens_q, a->cu_seqlens_k)) != FA_OK) return rc;
  const struct {
    const char* name;
    const void* base;
    const int64_t* strides;
    int tokens, heads;
  } tensors[] = {{"dout", a->dout, a->dout_strides, a->total_q, a->Hq}, {"q", a->q, a->q_strides, a->total_q, a->Hq},
                 {"out", a->out, a->out_strides, a->total_q, a->Hq},    {"dq", a->dq, a->dq_strides, a->total_q, a->Hq},
                 {"k", a->k, a->k_strides, a->total_k, a->Hkv},         {"v", a->v, a->v_strides, a->total_k, a->Hkv},
                 {"dk", a->dk, a->dk_strides, a->total_k, a->Hkv},      {"dv", a->dv, a->dv_strides, a->total_k, a->Hkv}};
  for (const auto& t : tensors)
    if (t.tokens > 0 && (rc = packed::check_tensor(who, t.name, t.base, t.strides, t.tokens, t.heads, a->D)) != FA_OK)
      return rc;
  if (a->total_q > 0 && (!a->lse || (reinterpret_cast<uintptr_t>(a->lse) & 3u) != 0))
    return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed_backward: lse missing or misaligned");
  if (!a->workspace || a->workspace_bytes < packed::workspace_bytes(a)) {
    char msg[160];
    snprintf(msg, sizeof msg, "fa_prefill_packed_backward: workspace of %zu bytes needed (got %zu)",
             packed::workspace_bytes(a), a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
    return set_error(FA_ERR_WORKSPACE, msg);
  }
  if ((reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0)
    return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed_backward: workspace must be 256-byte aligned");
  uint32_t* status = device_status_ptr();
  if (!status) return set_error(FA_ERR_CUDA, "fa_prefill_packed_backward: no usable CUDA device");
  packed::GradParams g{};
  packed::Params& p = g.f;
  p.cu_q = a->cu_seqlens_q;
  p.cu_k = a->cu_seqlens_k;
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.total_q = a->total_q;
  p.total_k = a->total_k;
  p.q_per_tile = packed::kRows / p.G;
  p.causal = a->causal ? 1 : 0;
  p.scale = a->scale;
  p.scale_log2 = a->scale * prefill::kLog2e;
  p.status = status;
  p.wait_ns = packed::wait_limit(a->total_q, a->total_k, p.q_per_tile);
  g.dout = a->dout;
  g.o = a->out;
  g.lse = a->lse;
  g.dq = a->dq;
  g.dk = a->dk;
  g.dv = a->dv;
  memcpy(g.dout_strides, a->dout_strides, sizeof g.dout_strides);
  memcpy(g.o_strides, a->out_strides, sizeof g.o_strides);
  memcpy(g.dq_strides, a->dq_strides, sizeof g.dq_strides);
  memcpy(g.dk_strides, a->dk_strides, sizeof g.dk_strides);
  memcpy(g.dv_strides, a->dv_strides, sizeof g.dv_strides);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  g.taken = reinterpret_cast<int*>(ws);
  g.q_blocks = static_cast<int>(packed::row_blocks(a->total_q, p.G, a->D));
  g.rows = reinterpret_cast<float2*>(ws + packed::front_bytes(a));
  const size_t one = packed::round_up(packed::row_bytes(a) / 2) / sizeof(float);  // a float a row
  g.few = reinterpret_cast<float*>(ws + packed::front_bytes(a) + packed::row_bytes(a));
  // pieces of 128 rows: causal, all that a sequence can have of few keys; else, the mean sequence's
  const int64_t rows = p.causal ? static_cast<int64_t>(packed::kFew) * p.G : (static_cast<int64_t>(a->total_q) * p.G + a->B - 1) / a->B;
  g.few_units = static_cast<int>((rows + 127) / 128 > 1 ? (rows + 127) / 128 : 1);
  const int64_t few = static_cast<int64_t>(a->B) * g.few_units;
  g.few_blocks = static_cast<int>(few < (1 << 20) ? few : 1 << 20);
  g.q = a->q;
  g.k = a->k;
  g.v = a->v;
  memcpy(g.q_strides, a->q_strides, sizeof g.q_strides);
  memcpy(g.k_strides, a->k_strides, sizeof g.k_strides);
  memcpy(g.v_strides, a->v_strides, sizeof g.v_strides);
  if (a->dtype == FA_FP16) {
    g.norms = g.few + one;
    g.maxima = g.norms + one;
    g.k_blocks = static_cast<int>(packed::row_blocks(a->total_k, 1, a->D));
    g.v_maxima = reinterpret_cast<float*>(g.taken + 1);
    g.v_norms = g.v_maxima + static_cast<size_t>(g.k_blocks) * a->Hkv;
  }
  const bool bf16 = a->dtype == FA_BF16;
  // Maps of an empty side are read by nothing; they get the workspace as their address.
  const bool hq = a->total_q > 0, hk = a->total_k > 0;
  CUtensorMap maps[4];
  if (!packed::encode_rows(&maps[0], bf16, hq ? a->q : ws, a->q_strides, a->total_q, hq ? a->Hq : 1, a->D, p.q_per_tile, p.G) ||
      !packed::encode_rows(&maps[1], bf16, hq ? a->dout : ws, a->dout_strides, a->total_q, hq ? a->Hq : 1, a->D, p.q_per_tile, p.G) ||
      !packed::encode_rows(&maps[2], bf16, hk ? a->k : ws, a->k_strides, a->total_k, hk ? a->Hkv : 1, a->D, packed::kKeys, 1) ||
      !packed::encode_rows(&maps[3], bf16, hk ? a->v : ws, a->v_strides, a->total_k, hk ? a->Hkv : 1, a->D, packed::kKeys, 1))
    return set_error(FA_ERR_CUDA, "fa_prefill_packed_backward: tensor map rejected");
  const int64_t q_items = hq ? packed::most_items(a->total_q, a->B, p.q_per_tile) : 0;
  const int64_t k_items = hk ? packed::most_items(a->total_k, a->B, packed::kKeys) : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->D == 128 ? (bf16 ? packed::launch<128, true>(g, maps, q_items, k_items, st)
                                            : packed::launch<128, false>(g, maps, q_items, k_items, st))
                                    : (bf16 ? packed::launch<64, true>(g, maps, q_items, k_items, st)
                                            : packed::launch<64, false>(g, maps, q_items, k_items, st));
  if (e != cudaSuccess) return set_error(FA_ERR_CUDA, cudaGetErrorString(e));
  return FA_OK;
}

}  // extern "C"
