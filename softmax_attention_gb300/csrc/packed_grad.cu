// packed_grad.cu -- the gradients of attention over packed prompts.
//
// With P_ij = e^(scale <q_i, k_j> - lse_i), dP_ij = <dout_i, v_j>, delta_i = <dout_i, out_i> and
// dS = P (dP - delta):
//     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,   dv_j = sum_i P_ij dout_i
//
// Two kernels, each with the sums it owns resident in tensor memory, so that nothing is added by
// atomics and the same call gives the same bits:
//   - dq_kernel: a CTA holds a 128-row query tile (query tokens x heads of a kv head, as in
//     packed.cu) and walks over the keys: S = Q K^T, dP = dO V^T, dQ += dS K.  It also computes
//     delta on its way in and leaves it for the second kernel.
//   - dkv_kernel: a CTA holds a tile of 128 keys and walks over the query tiles that see it, all
//     heads of the group: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  With the
//     products turned, P^T and dS^T have keys as rows and go back to tensor memory as the
//     left operands of the second pair: neither ever passes through shared memory.
// S and dP are computed in both, seven products for the five of a form that adds dq by atomics.
//
// Eight warps do the element-wise work, two a row, 64 columns each; P and dS, packed to 16 bits, are
// written over the half of S or dP that the warp itself has read.
//
// fp16: dS is held times a power of two, f, so that the small values that gradients have keep their
// bits (its smallest normal number is 2^-14): f brings the largest |dout| to [8, 16), of the row
// in dq_kernel, of the whole call in dkv_kernel, whose sums run over rows.  P is held times 2^7
// there.  bf16 has fp32's exponents, and f = 1.
#include <math.h>
#include <stdio.h>
#include <string.h>

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
  int64_t dout_strides[2], o_strides[2];
  void* dq;
  void* dk;
  void* dv;
  int64_t dq_strides[2], dk_strides[2], dv_strides[2];
  float* delta;          // [total_q, Hq]
  uint32_t* dout_max;    // fp16: bits of the largest |dout|
};

// The power of two that brings `top` to [8, 16); 1 for 0, an infinity or NaN.
__device__ __forceinline__ float power_for(float top) {
  if (!(top > 0.f) || top == INFINITY) return 1.f;
  const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // of a subnormal: -127
  return __uint_as_float(static_cast<uint32_t>(min(max(3 - e, -100), 100) + 127) << 23);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack(float2 v) {
  return BF16 ? pack_bf16x2(v.x, v.y) : pack_f16x2(v.x, v.y);
}

// 32 accumulator columns times `f`, in 16 bits to global memory (16-byte aligned).
template <bool BF16>
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&o)[32], float f) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack<BF16>(make_float2(__uint_as_float(o[8 * q + 2 * e]) * f, __uint_as_float(o[8 * q + 2 * e + 1]) * f));
    reinterpret_cast<uint4*>(dst)[q] = make_uint4(w[0], w[1], w[2], w[3]);
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
// dq.  Warps (352 threads): 0-3 columns 0..63 of S, 4-7 columns 64..127, 8 copies, 9 issues S and dP
// (and owns tensor memory), 10 issues dS K.  S is double-buffered: S_{j+1} is computed while the
// weights of tile j are; dS_j is written over S_j.  dP has one buffer, given back as soon as it is
// in registers.
// ------------------------------------------------------------------------------------------
constexpr int kDqThreads = 352;

template <int D>
struct DqLayout {
  static constexpr int kSlots = 5;
  static constexpr int kTile = kBlock * (D / 64);
  static constexpr int kQ = 0, kDo = kTile, kRing = 2 * kTile;
  static constexpr int kBars = kRing + kSlots * kTile;
  // q, full[slots], empty[slots], tail, s[2], dp, dp_read, ds[2], dq[2], done[2]
  static constexpr int kNumBars = 2 * kSlots + 13;
  static constexpr int kAlloc = kBars + kNumBars * 8 + 1024;
  static constexpr int kS = D, kDp = D + 2 * kKeys;     // tensor memory: dQ, S[2], dP
  static_assert(kAlloc <= 232448 && kDp + kKeys <= 512, "memory budgets");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kDqThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const GradParams gp) {
  using L = DqLayout<D>;
  const Params& p = gp.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint32_t tmem_slot;
  __shared__ int item[2];
  const uint32_t s_base = smem_addr(smem), bars = s_base + L::kBars;
  const uint32_t bar_q = bars;
  auto bar_full = [&](int s) { return bars + 8u * (1 + s); };
  auto bar_empty = [&](int s) { return bars + 8u * (1 + L::kSlots + s); };
  const uint32_t bar_tail = bars + 8u * (1 + 2 * L::kSlots);
  auto bar_s = [&](int i) { return bar_tail + 8u * (1 + i); };
  const uint32_t bar_dp = bar_tail + 24u, bar_dp_read = bar_tail + 32u;
  auto bar_ds = [&](int i) { return bar_tail + 8u * (5 + i); };
  auto bar_dq = [&](int i) { return bar_tail + 8u * (7 + i); };
  auto bar_done = [&](int i) { return bar_tail + 8u * (9 + i); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = blockIdx.x % p.Hkv;
  if (warp == 0) {
    int b, t;
    auto pieces = [&](int s, int& n, int& first) {
      const Seq q = load_seq(p, s);
      n = (q.nq + p.q_per_tile - 1) / p.q_per_tile;
      first = (p.causal ? max(0, q.nk - q.nq) : q.nk) / p.q_per_tile;
    };
    const Finder finder(p.B, !p.causal, pieces);
    finder.find(blockIdx.x / p.Hkv, pieces, b, t);
    if (lane == 0) {
      item[0] = b;
      item[1] = t;
    }
  } else if (warp == 9) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 8 * 32) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_tail, 1);
    mbar_init(bar_dp, 1);
    mbar_init(bar_dp_read, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s(i), 1);
      mbar_init(bar_ds(i), 256);
      mbar_init(bar_dq(i), 1);
      mbar_init(bar_done(i), 1);
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
  const int b = item[0];
  if (b >= 0) {
    const Seq seq = load_seq(p, b);
    const int q0 = item[1] * p.q_per_tile;
    const int last = min(seq.nq, q0 + p.q_per_tile) - 1;
    const int end = p.causal ? min(seq.nk, max(0, last + seq.nk - seq.nq + 1)) : seq.nk;
    const int n = (end + kKeys - 1) / kKeys;
    auto full = [&](int i) { return mbar_wait(bar_full(i % L::kSlots), (i / L::kSlots) & 1, p.status); };
    if (warp == 8) {
      // ---------------------------------- copies ----------------------------------------
      bool ok = true;
      int issued = 0;
      const bool tail = n > 0 && n * kKeys > seq.nk;  // the last K tile reaches past the sequence
      if (lane == 0 && n > 0) {
        mbar_arrive_expect_tx(bar_q, static_cast<uint32_t>(2 * 128 * (D / 64) * p.G * p.q_per_tile));
        for (int kb = 0; kb < D / 64; ++kb) {
          tma_load_3d(s_base + L::kQ + kb * kBlock, &tm_q, bar_q, kb * 64, hk * p.G, seq.q0 + q0);
          tma_load_3d(s_base + L::kDo + kb * kBlock, &tm_do, bar_q, kb * 64, hk * p.G, seq.q0 + q0);
        }
        for (int i = 0; i < 2 * n; ++i) {  // K_0, V_0, K_1, V_1, ...
          const int slot = i % L::kSlots;
          if (i >= L::kSlots && !(ok = mbar_wait(bar_empty(slot), (i / L::kSlots - 1) & 1, p.status))) break;
          const uint32_t bar = tail && i == 2 * n - 2 ? bar_tail : bar_full(slot);
          mbar_arrive_expect_tx(bar, L::kTile);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kRing + slot * L::kTile + kb * kBlock, (i & 1) ? &tm_v : &tm_k, bar, kb * 64, hk,
                        seq.k0 + (i / 2) * kKeys);
          issued = i + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (ok && tail) {
        // K rows past the sequence's end: dS is 0 there, but 0 times an infinity or NaN is not
        ok = __all_sync(0xffffffffu, mbar_wait(bar_tail, 0, p.status));
        const int slot = (2 * n - 2) % L::kSlots;
        if (ok) clear_rows<D>(smem + L::kRing + slot * L::kTile, seq.nk - (n - 1) * kKeys, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar_full(slot));
      }
      if (lane == 0 && issued < 2 * n) {
        // A wait ran out: let the copies in flight land before the CTA ends
        mbar_wait(bar_q, 0, nullptr);
        for (int i = max(0, issued - L::kSlots); i < issued; ++i) {
          const bool in_tail = tail && i == 2 * n - 2;
          mbar_wait(in_tail ? bar_tail : bar_full(i % L::kSlots), in_tail ? 0 : (i / L::kSlots) & 1, nullptr);
        }
      }
    } else if (warp == 9) {
      // ---------------------------------- S and dP --------------------------------------
      if (lane == 0 && n > 0) {
        constexpr uint32_t idesc = idesc_f16(BF16, kRows, kKeys, false, false);
        const uint64_t q_desc = sdesc_sw128(s_base + L::kQ, 16, 1024), do_desc = sdesc_sw128(s_base + L::kDo, 16, 1024);
        const uint64_t ring = sdesc_sw128(s_base + L::kRing, 16, 1024);
        bool ok = mbar_wait(bar_q, 0, p.status);
        for (int j = 0; ok && j < n; ++j) {
          if (!(ok = full(2 * j))) break;
          if (j >= 2 && !(ok = mbar_wait(bar_dq(j & 1), (j / 2 - 1) & 1, p.status))) break;
          tc_fence_after();
          product_ss<D>(tmem + L::kS + (j & 1) * kKeys, q_desc, sdesc_add(ring, ((2 * j) % L::kSlots) * L::kTile), idesc);
          tc_commit(bar_s(j & 1));
          if (!(ok = full(2 * j + 1))) break;
          if (j >= 1 && !(ok = mbar_wait(bar_dp_read, (j - 1) & 1, p.status))) break;
          tc_fence_after();
          const int slot = (2 * j + 1) % L::kSlots;
          product_ss<D>(tmem + L::kDp, do_desc, sdesc_add(ring, slot * L::kTile), idesc);
          tc_commit(bar_dp);
          tc_commit(bar_empty(slot));
        }
        tc_commit(bar_done(0));
        mbar_wait(bar_done(0), 0, nullptr);
      }
    } else if (warp == 10) {
      // ---------------------------------- dQ += dS K ------------------------------------
      if (lane == 0 && n > 0) {
        constexpr uint32_t idesc = idesc_f16(BF16, kRows, D, false, true);
        const uint64_t ring = sdesc_sw128(s_base + L::kRing, kBlock, 1024);
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
          if (!(ok = full(2 * j))) break;
          if (!(ok = mbar_wait(bar_ds(j & 1), (j / 2) & 1, p.status))) break;
          tc_fence_after();
          const int slot = (2 * j) % L::kSlots;
          product_ts(tmem, tmem + L::kS + (j & 1) * kKeys, kHalf, sdesc_add(ring, slot * L::kTile), idesc, j == 0);
          tc_commit(bar_dq(j & 1));
          tc_commit(bar_empty(slot));
        }
        tc_commit(bar_done(1));
        mbar_wait(bar_done(1), 0, nullptr);
      }
    } else {
      // ------------------------- weights: a row and 64 columns a thread -------------------
      const int w = warp / 4, r = threadIdx.x % 128;  // half of the columns
      const int i = q0 + r / p.G, h = hk * p.G + r % p.G;
      const bool valid = r < p.G * p.q_per_tile && i < seq.nq;
      const int64_t row = seq.q0 + i;
      const int key_lim = !valid ? 0 : p.causal ? min(seq.nk, i + seq.nk - seq.nq + 1) : seq.nk;
      const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
      // delta and the largest |dout| of the row, by both of its threads: the second finds the first's
      // lines in L1, and no shared memory is left to trade halves in
      float delta = 0.f, top = 0.f, lse = -INFINITY;
      if (valid) {
        const uint4* a = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(gp.dout) + row * gp.dout_strides[0] +
                                                        h * gp.dout_strides[1]);
        const uint4* c = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(gp.o) + row * gp.o_strides[0] +
                                                        h * gp.o_strides[1]);
        lse = __ldg(gp.lse + row * p.Hq + h);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          const uint4 va = __ldg(a + e), vc = __ldg(c + e);
          const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wc[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            float2 x, y;
            if constexpr (BF16) {
              x = make_float2(__uint_as_float(wa[f] << 16), __uint_as_float(wa[f] & 0xffff0000u));
              y = make_float2(__uint_as_float(wc[f] << 16), __uint_as_float(wc[f] & 0xffff0000u));
            } else {
              x = __half22float2(*reinterpret_cast<const __half2*>(&wa[f]));
              y = __half22float2(*reinterpret_cast<const __half2*>(&wc[f]));
              top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
            delta = fmaf(x.x, y.x, fmaf(x.y, y.y, delta));
          }
        }
        if (w == 0) gp.delta[row * p.Hq + h] = delta;
      }
      float f = 1.f;
      if constexpr (!BF16) {
        f = power_for(top);
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if (w == 0 && lane == 0 && most > 0) atomicMax(gp.dout_max, most);  // a maximum: any order
      }
      const float nl = lse > -INFINITY ? -lse * prefill::kLog2e : -INFINITY;
      const float2 a2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nl, nl);
      const float2 f2 = make_float2(f, f), nd2 = make_float2(-delta * f, -delta * f);
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        const uint32_t tm_s = tmem + L::kS + (j & 1) * kKeys + w * kHalf + lanes;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s(j & 1), (j / 2) & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        const int left = key_lim - (j * kKeys + w * kHalf);  // columns that the row sees
        uint32_t raw[2][32];
        tmem_ld32(tm_s, raw[0]);
        tmem_ld32(tm_s + 32, raw[1]);
        prefill::tmem_ld_wait_tied(raw[0]);
        prefill::tmem_ld_wait_tied(raw[1]);
        float2 x[32];
        const bool whole = __all_sync(0xffffffffu, left >= kHalf);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 t = __ffma2_rn(make_float2(__uint_as_float(raw[c / 16][(2 * c) % 32]),
                                                  __uint_as_float(raw[c / 16][(2 * c) % 32 + 1])), a2, nl2);
          x[c] = make_float2(exp2_approx(t.x), exp2_approx(t.y));
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = make_float2(2 * c < left ? x[c].x : 0.f, 2 * c + 1 < left ? x[c].y : 0.f);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(bar_dp, j & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        uint32_t dp[2][32], ds[32];
        const uint32_t tm_dp = tmem + L::kDp + w * kHalf + lanes;
        tmem_ld32(tm_dp, dp[0]);
        prefill::tmem_ld_wait_tied(dp[0]);
        tmem_ld32(tm_dp + 32, dp[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1) {
            prefill::tmem_ld_wait_tied(dp[1]);
            tc_fence_before();
            mbar_arrive(bar_dp_read);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 t = __ffma2_rn(make_float2(__uint_as_float(dp[q][2 * c]), __uint_as_float(dp[q][2 * c + 1])), f2, nd2);
            float2 v = __fmul2_rn(x[16 * q + c], t);
            // a hidden column's dP may be another sequence's, or no number: selected, not multiplied
            if (!whole) v = make_float2(32 * q + 2 * c < left ? v.x : 0.f, 32 * q + 2 * c + 1 < left ? v.y : 0.f);
            ds[16 * q + c] = pack<BF16>(v);
          }
        }
        tmem_st32(tm_s, ds);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_ds(j & 1));
      }
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_dq((n - 1) & 1), ((n - 1) / 2) & 1, p.status));
        tc_fence_after();
      }
      if (ok) {
        const float back = p.scale / f;
        uint16_t* dst = static_cast<uint16_t*>(gp.dq) + row * gp.dq_strides[0] + h * gp.dq_strides[1] + w * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tmem + lanes + w * (D / 2) + c * 32, o);
            prefill::tmem_ld_wait_tied(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (valid) store32<BF16>(dst + c * 32, o, back);
        }
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

// ------------------------------------------------------------------------------------------
// dk and dv.  Warps (384 threads): 0-3 query columns 0..63 of S^T, 4-7 columns 64..127, 8 copies, 9
// issues dV and S^T (and owns tensor memory), 10 issues dK and dP^T, 11 brings each query row's lse
// and delta.  Tensor memory is full at D = 128 (dV, dK, S^T, dP^T): P^T lies over S^T and dS^T over
// dP^T, and issuer 9 puts S^T_{i+1} right behind dV_i (issuer 10 dP^T_{i+1} behind dK_i), which
// reads what it overwrites: products of one thread and one shape run in order.  While the
// element-wise warps work on S^T the tensor cores run dK and dP^T, and the other way round.  At
// D = 64, where the shapes differ, P^T and dS^T have columns of their own.
// ------------------------------------------------------------------------------------------
constexpr int kDkvThreads = 384;

template <int D>
struct DkvLayout {
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kTile = kBlock * (D / 64);
  static constexpr int kK = 0, kV = kTile, kRing = 2 * kTile;
  static constexpr int kRowData = kRing + kSlots * kTile;  // [2][-lse, -delta][128] fp32
  static constexpr int kBars = kRowData + 2 * 2 * kRows * 4;
  // kv, full[slots], empty[slots], tail, rows_full[2], rows_empty[2], s, p, dp, ds, dv, dk, done[2]
  static constexpr int kNumBars = 2 * kSlots + 14;
  static constexpr int kAlloc = kBars + kNumBars * 8 + 1024;
  static constexpr bool kApart = D == 64;
  static constexpr int kDv = 0, kDk = D, kS = 2 * D, kDp = kS + kRows;
  static constexpr int kP = kApart ? kDp + kRows : kS, kDs = kApart ? kP + kRows / 2 : kDp;
  static constexpr int kStep = kApart ? kHalf / 2 : kHalf;  // between the two halves of P^T, of dS^T
  static_assert(kAlloc <= 232448 && kDs + kRows / 2 <= 512, "memory budgets");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kDkvThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const GradParams gp) {
  using L = DkvLayout<D>;
  constexpr float kPower = BF16 ? 0.f : 7.f;  // P is held times 2^kPower
  const Params& p = gp.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint32_t tmem_slot;
  __shared__ int item[2];
  const uint32_t s_base = smem_addr(smem), bars = s_base + L::kBars;
  const uint32_t bar_kv = bars;
  auto bar_full = [&](int s) { return bars + 8u * (1 + s); };
  auto bar_empty = [&](int s) { return bars + 8u * (1 + L::kSlots + s); };
  const uint32_t bar_tail = bars + 8u * (1 + 2 * L::kSlots);
  auto bar_rows = [&](int i) { return bar_tail + 8u * (1 + i); };
  auto bar_rows_read = [&](int i) { return bar_tail + 8u * (3 + i); };
  const uint32_t bar_s = bar_tail + 40u, bar_p = bar_tail + 48u, bar_dp = bar_tail + 56u, bar_ds = bar_tail + 64u;
  const uint32_t bar_dv = bar_tail + 72u, bar_dk = bar_tail + 80u;
  auto bar_done = [&](int i) { return bar_tail + 8u * (11 + i); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = blockIdx.x % p.Hkv;
  const int used = p.G * p.q_per_tile;  // rows of a query tile
  if (warp == 0) {
    int b, t;
    auto pieces = [&](int s, int& n, int& first) {
      const Seq q = load_seq(p, s);
      n = (q.nk + kKeys - 1) / kKeys;
      first = p.causal ? 0 : q.nq / kKeys;
    };
    const Finder finder(p.B, !p.causal, pieces);
    finder.find(blockIdx.x / p.Hkv, pieces, b, t);
    if (lane == 0) {
      item[0] = b;
      item[1] = t;
    }
  } else if (warp == 9) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 8 * 32) {
    mbar_init(bar_kv, 1);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 2);  // both issuers
    }
    mbar_init(bar_tail, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_rows(i), 32);
      mbar_init(bar_rows_read(i), 256);
      mbar_init(bar_done(i), 1);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_p, 256);
    mbar_init(bar_dp, 1);
    mbar_init(bar_ds, 256);
    mbar_init(bar_dv, 1);
    mbar_init(bar_dk, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (used < kRows) {
    // Rows that no copy writes are summed over all the same: zero, once.
    for (int s = 0; s < L::kSlots; ++s)
      clear_rows<D>(smem + L::kRing + s * L::kTile, used, threadIdx.x, kDkvThreads);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int b = item[0];
  if (b >= 0) {
    const Seq seq = load_seq(p, b);
    const int off = seq.nk - seq.nq;
    // the pieces' work grows with their index: the first keys, seen by most queries, come last
    const int key0 = (p.causal ? (seq.nk + kKeys - 1) / kKeys - 1 - item[1] : item[1]) * kKeys;
    const int it0 = p.causal ? max(0, key0 - off) / p.q_per_tile : 0;  // first query tile that sees a key
    const int n = max(0, (seq.nq + p.q_per_tile - 1) / p.q_per_tile - it0);
    auto full = [&](int i) { return mbar_wait(bar_full(i % L::kSlots), (i / L::kSlots) & 1, p.status); };
    if (warp == 8) {
      // ---------------------------------- copies ----------------------------------------
      bool ok = true;
      int issued = 0;
      const int rows = n > 0 ? (seq.nq - (it0 + n - 1) * p.q_per_tile) * p.G : 0;  // of the last query tile
      const bool tail = n > 0 && rows < used;
      if (lane == 0 && n > 0) {
        mbar_arrive_expect_tx(bar_kv, 2 * L::kTile);
        for (int kb = 0; kb < D / 64; ++kb) {
          tma_load_3d(s_base + L::kK + kb * kBlock, &tm_k, bar_kv, kb * 64, hk, seq.k0 + key0);
          tma_load_3d(s_base + L::kV + kb * kBlock, &tm_v, bar_kv, kb * 64, hk, seq.k0 + key0);
        }
        const uint32_t bytes = static_cast<uint32_t>(128 * (D / 64) * used);
        for (int i = 0; i < 2 * n; ++i) {  // Q_0, dO_0, Q_1, dO_1, ...
          const int slot = i % L::kSlots;
          if (i >= L::kSlots && !(ok = mbar_wait(bar_empty(slot), (i / L::kSlots - 1) & 1, p.status))) break;
          const bool in_tail = tail && i >= 2 * n - 2;
          const uint32_t bar = in_tail ? bar_tail : bar_full(slot);
          // (the tail's barrier counts one arrival, for both of its copies)
          if (!in_tail) mbar_arrive_expect_tx(bar, bytes);
          else if (i == 2 * n - 2) mbar_arrive_expect_tx(bar, 2 * bytes);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kRing + slot * L::kTile + kb * kBlock, (i & 1) ? &tm_do : &tm_q, bar, kb * 64,
                        hk * p.G, seq.q0 + (it0 + i / 2) * p.q_per_tile);
          issued = i + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (ok && tail) {
        // query rows past the sequence's end, which the sums over rows must not see
        ok = __all_sync(0xffffffffu, mbar_wait(bar_tail, 0, p.status));
        for (int i = 2 * n - 2; ok && i < 2 * n; ++i)
          clear_rows<D>(smem + L::kRing + (i % L::kSlots) * L::kTile, rows, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        for (int i = 2 * n - 2; ok && lane == 0 && i < 2 * n; ++i) mbar_arrive(bar_full(i % L::kSlots));
      }
      if (lane == 0 && issued < 2 * n) {
        // A wait ran out: let the copies in flight land before the CTA ends (of the tail's two the
        // first alone may be on its way: its barrier then does not complete, and the wait's own
        // limit, far longer than a copy takes, stands for it)
        mbar_wait(bar_kv, 0, nullptr);
        for (int i = max(0, issued - L::kSlots); i < issued; ++i) {
          const bool in_tail = tail && i >= 2 * n - 2;
          mbar_wait(in_tail ? bar_tail : bar_full(i % L::kSlots), in_tail ? 0 : (i / L::kSlots) & 1, nullptr);
        }
      }
    } else if (warp == 9 || warp == 10) {
      // --------------------- issuer 9: S^T and dV; issuer 10: dP^T and dK ----------------
      // first = left . (ring tile of this role)^T, second += packed . (the other role's ring tile)
      const int x = warp - 9;
      if (lane == 0 && n > 0) {
        constexpr uint32_t idesc1 = idesc_f16(BF16, kRows, kRows, false, false);
        constexpr uint32_t idesc2 = idesc_f16(BF16, kRows, D, false, true);
        const uint64_t left = sdesc_sw128(s_base + (x ? L::kV : L::kK), 16, 1024);
        const uint64_t ring1 = sdesc_sw128(s_base + L::kRing, 16, 1024), ring2 = sdesc_sw128(s_base + L::kRing, kBlock, 1024);
        const uint32_t tm1 = tmem + (x ? L::kDp : L::kS), tm2 = tmem + (x ? L::kDk : L::kDv), tm_a = tmem + (x ? L::kDs : L::kP);
        const uint32_t bar1 = x ? bar_dp : bar_s, bar_a = x ? bar_ds : bar_p, bar2 = x ? bar_dk : bar_dv;
        // Q_i is ring entry 2i, dO_i 2i + 1: S^T reads Q and dV dO; dP^T reads dO and dK Q
        bool ok = mbar_wait(bar_kv, 0, p.status) && full(x);
        if (ok) {
          tc_fence_after();
          product_ss<D>(tm1, left, sdesc_add(ring1, (x % L::kSlots) * L::kTile), idesc1);
          tc_commit(bar1);
          tc_commit(bar_empty(x % L::kSlots));
        }
        for (int i = 0; ok && i < n; ++i) {
          const int mine = 2 * i + 2 + x, other = 2 * i + 1 - x;
          if (!(ok = mbar_wait(bar_a, i & 1, p.status))) break;
          if (!(ok = full(other))) break;
          if (i + 1 < n && !(ok = full(mine))) break;
          tc_fence_after();
          product_ts(tm2, tm_a, L::kStep, sdesc_add(ring2, (other % L::kSlots) * L::kTile), idesc2, i == 0);
          tc_commit(bar2);
          tc_commit(bar_empty(other % L::kSlots));
          if (i + 1 < n) {
            product_ss<D>(tm1, left, sdesc_add(ring1, (mine % L::kSlots) * L::kTile), idesc1);
            tc_commit(bar1);
            tc_commit(bar_empty(mine % L::kSlots));
          }
        }
        tc_commit(bar_done(x));
        mbar_wait(bar_done(x), 0, nullptr);
      }
    } else if (warp == 11) {
      // --------------------- lse and delta of each query row, ready for use ---------------
      float f = 1.f;
      if constexpr (!BF16) f = power_for(__uint_as_float(__ldcg(gp.dout_max))) * 0.0078125f;  // 2^-kPower
      bool ok = true;
      for (int i = 0; ok && i < n; ++i) {
        const int q0 = (it0 + i) * p.q_per_tile;
        float nl[4], nd[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = lane * 4 + e, token = q0 + r / p.G;
          nl[e] = -INFINITY;  // no query, or one that sees no key: P = 0
          nd[e] = 0.f;
          if (r < used && token < seq.nq) {
            const int64_t at = static_cast<int64_t>(seq.q0 + token) * p.Hq + hk * p.G + r % p.G;
            const float lse = __ldg(gp.lse + at);
            if (!(lse == -INFINITY)) nl[e] = kPower - lse * prefill::kLog2e;
            nd[e] = -f * __ldg(gp.delta + at);
          }
        }
        if (i >= 2) ok = __all_sync(0xffffffffu, mbar_wait(bar_rows_read(i & 1), (i / 2 - 1) & 1, p.status));
        float* to = reinterpret_cast<float*>(smem + L::kRowData) + (i & 1) * 2 * kRows + lane * 4;
        *reinterpret_cast<float4*>(to) = make_float4(nl[0], nl[1], nl[2], nl[3]);
        *reinterpret_cast<float4*>(to + kRows) = make_float4(nd[0], nd[1], nd[2], nd[3]);
        mbar_arrive(bar_rows(i & 1));
      }
    } else {
      // -------------------- weights: a key and 64 query columns a thread ------------------
      const int w = warp / 4, r = threadIdx.x % 128;
      const int key = key0 + r;
      const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
      const uint32_t tm_s = tmem + L::kS + w * kHalf + lanes, tm_dp = tmem + L::kDp + w * kHalf + lanes;
      const uint32_t tm_p = tmem + L::kP + w * L::kStep + lanes, tm_ds = tmem + L::kDs + w * L::kStep + lanes;
      float f = 1.f;
      if constexpr (!BF16) f = power_for(__uint_as_float(__ldcg(gp.dout_max)));
      const float fs = BF16 ? 1.f : f * 0.0078125f;  // 2^-kPower
      const float2 a2 = make_float2(p.scale_log2, p.scale_log2), f2 = make_float2(fs, fs);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const float4* row_data = reinterpret_cast<const float4*>(smem + L::kRowData) + (i & 1) * 64 + w * 16;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_rows(i & 1), (i / 2) & 1, p.status));
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_s, i & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        // columns below `from` are queries in front of the key
        const int from = p.causal ? (key - off - (it0 + i) * p.q_per_tile) * p.G - w * kHalf : 0;
        const bool whole = __all_sync(0xffffffffu, from <= 0);
        uint32_t raw[2][32];
        tmem_ld32(tm_s, raw[0]);
        tmem_ld32(tm_s + 32, raw[1]);
        prefill::tmem_ld_wait_tied(raw[0]);
        prefill::tmem_ld_wait_tied(raw[1]);
        float2 x[32];
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 nl = row_data[c];
          const float2 t = __ffma2_rn(make_float2(__uint_as_float(raw[c / 8][(4 * c) % 32]),
                                                  __uint_as_float(raw[c / 8][(4 * c) % 32 + 1])), a2, make_float2(nl.x, nl.y));
          const float2 u = __ffma2_rn(make_float2(__uint_as_float(raw[c / 8][(4 * c) % 32 + 2]),
                                                  __uint_as_float(raw[c / 8][(4 * c) % 32 + 3])), a2, make_float2(nl.z, nl.w));
          x[2 * c] = make_float2(exp2_approx(t.x), exp2_approx(t.y));
          x[2 * c + 1] = make_float2(exp2_approx(u.x), exp2_approx(u.y));
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = make_float2(2 * c >= from ? x[c].x : 0.f, 2 * c + 1 >= from ? x[c].y : 0.f);
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = pack<BF16>(x[c]);
        if (L::kApart && i > 0) {  // P^T_{i-1} has to be read before P^T_i takes its place
          ok = __all_sync(0xffffffffu, mbar_wait(bar_dv, (i - 1) & 1, p.status));
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st32(tm_p, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_p);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_dp, i & 1, p.status));
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
        mbar_arrive(bar_rows_read(i & 1));
        if (L::kApart && i > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar_dk, (i - 1) & 1, p.status));
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st32(tm_ds, ds);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_ds);
      }
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(w ? bar_dk : bar_dv, (n - 1) & 1, p.status));
        tc_fence_after();
      }
      if (ok) {
        // dv by the first four warps, dk by the others
        const bool valid = key < seq.nk;
        const int64_t row = seq.k0 + key;
        uint16_t* dst = w ? static_cast<uint16_t*>(gp.dk) + row * gp.dk_strides[0] + hk * gp.dk_strides[1]
                          : static_cast<uint16_t*>(gp.dv) + row * gp.dv_strides[0] + hk * gp.dv_strides[1];
        const float back = w ? p.scale / f : BF16 ? 1.f : 0.0078125f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tmem + (w ? L::kDk : L::kDv) + lanes + c * 32, o);
            prefill::tmem_ld_wait_tied(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (valid) store32<BF16>(dst + c * 32, o, back);
        }
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
  if (e == cudaSuccess && !BF16) e = cudaMemsetAsync(g.dout_max, 0, sizeof(uint32_t), st);
  if (e != cudaSuccess) return e;
  if (q_items > 0)
    kq<<<static_cast<unsigned>(q_items * g.f.Hkv), kDqThreads, DqLayout<D>::kAlloc, st>>>(maps[0], maps[1], maps[2], maps[3], g);
  if (k_items > 0)
    kk<<<static_cast<unsigned>(k_items * g.f.Hkv), kDkvThreads, DkvLayout<D>::kAlloc, st>>>(maps[0], maps[1], maps[2], maps[3], g);
  return cudaGetLastError();
}

constexpr size_t kWordBytes = 256;  // in front of delta: the largest |dout|

size_t workspace_bytes(const fa_packed_backward_args* a) {
  return kWordBytes + (static_cast<size_t>(a->total_q) * a->Hq * sizeof(float) + 255) / 256 * 256;
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
  if (!a->cu_seqlens_q || !a->cu_seqlens_k)
    return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed_backward: null cu_seqlens pointer");
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
  g.dout_max = reinterpret_cast<uint32_t*>(ws);
  g.delta = reinterpret_cast<float*>(ws + packed::kWordBytes);
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
