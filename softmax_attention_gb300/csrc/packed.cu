// packed.cu -- attention over packed prompts: sequences of different lengths behind one another
// in one tensor, grouped heads, causal or not.
//
// For a query at position i of a sequence, out = sum_j p_j v_j / l with p_j = e^(s_j - m),
// s_j = scale <q, k_j>, l = sum_j p_j and m the running maximum of the keys seen so far: one pass
// over the keys, O and l rescaled when m grows.
//
// One CTA takes two neighbouring 128-row query tiles A and B of one kv head (a tile is 128 / G
// query tokens x the G heads of the kv head, token by token, so rows past a sequence's end are
// the last ones) over all their keys.  K and V tiles of 128 keys go through one shared ring and
// serve both tiles.  Each tile has its own softmax warpgroup and its own issuing thread; tensor
// memory holds O and S of both, with P in 16 bits written over S (D = 128) or beside it (D = 64).
//
// Why two tiles: a tile's chain S_j -> softmax -> P_j V_j -> S_{j+1} leaves the tensor cores idle
// while its softmax runs; the other tile's products fill that time.  An issuer waits for P_j, V_j
// and K_{j+1} before it issues P_j V_j and S_{j+1} together: once a thread has committed products
// its next look at shared memory is held until they finish, so a wait between the two would
// drain the pipe.  S_{j+1} may be issued behind P_j V_j although it overwrites P_j: products of
// one thread and one shape run in order (D = 64, where the shapes differ, keeps P apart).
//
// The softmax works on a row 32 scores at a time against the maximum of the tiles before, and
// looks for a larger one on the way; only if a row's maximum grew by more than 2^8 (or the tile
// has masked keys, or is the first) is the tile done in two passes.  So no more than 32 scores
// and the 64 registers of packed P are held, and the maximum is not in the way of the first
// exponential.
//
// Warps (352 threads): 0-3 softmax A, 4-7 softmax B, 8 copies, 9 issuer A (and tensor memory), 10
// issuer B.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "internal.h"
#include "packed.cuh"

namespace fa {
namespace packed {
namespace {

using prefill::kLn2;
using prefill::kRescaleLog2;

constexpr int kThreads = 352;

template <int D>
struct Layout {
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kBlock = kRows * 128;          // 128 rows x 64 columns of 16 bits
  static constexpr int kTile = kBlock * (D / 64);     // a Q tile, or a ring slot of K or V
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBars = kRing + kSlots * kTile;
  // q[2], full[slots], empty[slots], tail, s[2], p[2], pv[2], done[2], turn[2]
  static constexpr int kNumBars = 2 * kSlots + 13;
  static constexpr int kAlloc = kBars + kNumBars * 8 + 1024;  // room to align the base
  // tensor memory columns
  static constexpr bool kApart = D == 64;             // P beside S
  static constexpr int kS = 2 * D, kP = kApart ? kS + 2 * kKeys : kS, kPStep = kApart ? kKeys / 2 : kKeys;
  static_assert(kAlloc <= 232448, "shared memory budget");
  static_assert(kKeys == kRows, "one block size for Q, K and V");
};

struct Tile {
  int q0, n;  // first query of the tile in its sequence, KV tiles that it sees
};

__device__ __forceinline__ Tile make_tile(const Params& p, const Seq& s, int q0) {
  Tile t{q0, 0};
  if (q0 < s.nq) {
    const int last = min(s.nq, q0 + p.q_per_tile) - 1;
    const int end = p.causal ? min(s.nk, max(0, last + s.nk - s.nq + 1)) : s.nk;
    t.n = (end + kKeys - 1) / kKeys;
  }
  return t;
}

// Thirty-two scores against the maximum m: exponentials packed, their sum added; with MASK the
// first `left` alone count.
template <bool BF16, bool MASK>
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], int left, float a, float m, float2& sum, uint32_t* pk) {
  const float2 a2 = make_float2(a, a), nm = make_float2(-m, -m);
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const float2 t = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), a2, nm);
    float2 e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
    if (MASK) e = make_float2(2 * c < left ? e.x : 0.f, 2 * c + 1 < left ? e.y : 0.f);
    sum = __fadd2_rn(sum, e);
    pk[c] = BF16 ? pack_bf16x2(e.x, e.y) : pack_f16x2(e.x, e.y);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    forward_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint32_t tmem_slot;
  __shared__ int item[2];
  const uint32_t s_base = smem_addr(smem);
  const uint32_t bars = s_base + L::kBars;
  auto bar_q = [&](int x) { return bars + 8u * x; };
  auto bar_full = [&](int s) { return bars + 8u * (2 + s); };
  auto bar_empty = [&](int s) { return bars + 8u * (2 + L::kSlots + s); };
  const uint32_t bar_tail = bars + 8u * (2 + 2 * L::kSlots);
  auto bar_s = [&](int x) { return bar_tail + 8u * (1 + x); };
  auto bar_p = [&](int x) { return bar_tail + 8u * (3 + x); };
  auto bar_pv = [&](int x) { return bar_tail + 8u * (5 + x); };
  auto bar_done = [&](int x) { return bar_tail + 8u * (7 + x); };
  auto bar_turn = [&](int x) { return bar_tail + 8u * (9 + x); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = blockIdx.x % p.Hkv;
  if (warp == 0) {
    const int width = 2 * p.q_per_tile;
    int b, t;
    find_item(p.B, blockIdx.x / p.Hkv, !p.causal, [&](int s, int& n, int& first) {
      const Seq q = load_seq(p, s);
      n = (q.nq + width - 1) / width;
      first = (p.causal ? max(0, q.nk - q.nq) : q.nk) / width;
    }, b, t);
    if (lane == 0) {
      item[0] = b;
      item[1] = t;
    }
  } else if (warp == 9) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 8 * 32) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar_q(x), 1);
      mbar_init(bar_s(x), 1);
      mbar_init(bar_p(x), 128);
      mbar_init(bar_pv(x), 1);
      mbar_init(bar_done(x), 1);
      mbar_init(bar_turn(x), 1);
    }
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 2);  // both tiles
    }
    mbar_init(bar_tail, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
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
    const int q0 = item[1] * 2 * p.q_per_tile;
    const Tile tile_a = make_tile(p, seq, q0), tile_b = make_tile(p, seq, q0 + p.q_per_tile);
    const int n = max(tile_a.n, tile_b.n);  // KV tiles through the ring
    if (warp == 8) {
      // ---------------------------------- copies ----------------------------------------
      bool ok = true;
      int issued = 0;
      const bool tail = n > 0 && n * kKeys > seq.nk;  // the last V tile reaches past the sequence
      if (lane == 0 && n > 0) {
        for (int x = 0; x < 2; ++x) {
          const Tile tile = x ? tile_b : tile_a;
          if (tile.n == 0) continue;
          mbar_arrive_expect_tx(bar_q(x), static_cast<uint32_t>(128 * (D / 64) * p.G * p.q_per_tile));
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + x * L::kTile + kb * L::kBlock, &tm_q, bar_q(x), kb * 64, hk * p.G,
                        seq.q0 + tile.q0);
        }
        for (int i = 0; i < 2 * n; ++i) {  // K_0, V_0, K_1, V_1, ...
          const int slot = i % L::kSlots;
          if (i >= L::kSlots && !(ok = mbar_wait(bar_empty(slot), (i / L::kSlots - 1) & 1, p.status))) break;
          const uint32_t bar = tail && i == 2 * n - 1 ? bar_tail : bar_full(slot);
          mbar_arrive_expect_tx(bar, L::kTile);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kRing + slot * L::kTile + kb * L::kBlock, (i & 1) ? &tm_v : &tm_k, bar,
                        kb * 64, hk, seq.k0 + (i / 2) * kKeys);
          issued = i + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (ok && tail) {
        // Rows past the sequence's end hold another sequence's values, or none: P is 0 there, but
        // 0 times an infinity or NaN would spoil O.
        ok = __all_sync(0xffffffffu, mbar_wait(bar_tail, 0, p.status));
        const int slot = (2 * n - 1) % L::kSlots, r0 = seq.nk - (n - 1) * kKeys;
        uint8_t* v = smem + L::kRing + slot * L::kTile;
        if (ok) {
          for (int i = lane; i < (kKeys - r0) * 8 * (D / 64); i += 32) {
            const int kb = i / ((kKeys - r0) * 8), at = i % ((kKeys - r0) * 8);
            *reinterpret_cast<uint4*>(v + kb * L::kBlock + r0 * 128 + at * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar_full(slot));
      }
      if (lane == 0 && issued < 2 * n) {
        // A wait ran out: let the copies in flight land before the CTA ends.  Each of these is the
        // last copy into its slot, so its phase is the barrier's current one.
        for (int x = 0; x < 2; ++x)
          if ((x ? tile_b.n : tile_a.n) > 0) mbar_wait(bar_q(x), 0, nullptr);
        for (int i = max(0, issued - L::kSlots); i < issued; ++i)
          mbar_wait(bar_full(i % L::kSlots), (i / L::kSlots) & 1, nullptr);
      }
    } else if (warp >= 9) {
      // ---------------------------------- issuers ---------------------------------------
      const int x = warp - 9, nx = x ? tile_b.n : tile_a.n, other_n = x ? tile_a.n : tile_b.n;
      if (lane == 0 && n > 0) {
        constexpr uint32_t idesc_s = idesc_f16(BF16, kRows, kKeys, false, false);
        constexpr uint32_t idesc_o = idesc_f16(BF16, kRows, D, false, true);
        const uint64_t q_desc = sdesc_sw128(s_base + x * L::kTile, 16, 1024);
        const uint64_t k_desc = sdesc_sw128(s_base + L::kRing, 16, 1024);
        const uint64_t v_desc = sdesc_sw128(s_base + L::kRing, L::kBlock, 1024);
        const uint32_t tm_o = tmem + x * D, tm_s = tmem + L::kS + x * kKeys, tm_p = tmem + L::kP + x * L::kPStep;
        auto issue_s = [&](int j) {
          const int slot = (2 * j) % L::kSlots;
          const uint64_t kd = sdesc_add(k_desc, slot * L::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * L::kBlock + (kk % 4) * 32;
            mma_ss(tm_s, sdesc_add(q_desc, off), sdesc_add(kd, off), idesc_s, kk > 0 ? 1u : 0u);
          }
        };
        auto full = [&](int i) { return mbar_wait(bar_full(i % L::kSlots), (i / L::kSlots) & 1, p.status); };
        bool ok = true;
        if (nx > 0) {
          ok = mbar_wait(bar_q(x), 0, p.status) && full(0);
          if (ok) {
            tc_fence_after();
            issue_s(0);
            tc_commit(bar_s(x));
            tc_commit(bar_empty(0));
          }
        }
        for (int j = 0; ok && j < nx; ++j) {
          if (!(ok = mbar_wait(bar_p(x), j & 1, p.status))) break;
          if (!(ok = full(2 * j + 1))) break;
          if (j + 1 < nx && !(ok = full(2 * j + 2))) break;
          // the other tile's turn before this one: its j-th pair of products for B, its (j-1)-th for A
          const int theirs = x ? j : j - 1;
          if (theirs >= 0 && theirs < other_n && !(ok = mbar_wait(bar_turn(1 - x), theirs & 1, p.status))) break;
          tc_fence_after();
          const int slot = (2 * j + 1) % L::kSlots;
          const uint64_t vd = sdesc_add(v_desc, slot * L::kTile);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts(tm_o, tm_p + kk * 8, sdesc_add(vd, kk * 2048), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
          if (j + 1 < nx) issue_s(j + 1);
          mbar_arrive(bar_turn(x));
          tc_commit(bar_pv(x));
          tc_commit(bar_empty(slot));
          if (j + 1 < nx) {
            tc_commit(bar_s(x));
            tc_commit(bar_empty((2 * j + 2) % L::kSlots));
          }
        }
        // tiles that only the other one sees: released as they land, phase by phase
        for (int i = 2 * nx; ok && i < 2 * n; ++i) {
          if (!(ok = full(i))) break;
          mbar_arrive(bar_empty(i % L::kSlots));
        }
        // every product must finish before tensor memory and the ring are given up
        tc_commit(bar_done(x));
        mbar_wait(bar_done(x), 0, nullptr);
      }
    } else {
      // --------------------------- softmax, epilogue: a row a thread ---------------------
      const int x = warp / 4, r = threadIdx.x % 128;
      const Tile tile = x ? tile_b : tile_a;
      const int nx = tile.n;
      const int i = tile.q0 + r / p.G, h = hk * p.G + r % p.G;
      const bool valid = r < p.G * p.q_per_tile && i < seq.nq;
      // a row of no query sees everything, so that it never asks for the slow path
      const int key_lim = !valid ? 0x7fffffff : p.causal ? min(seq.nk, i + seq.nk - seq.nq + 1) : seq.nk;
      const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
      const uint32_t tm_o = tmem + x * D + lanes, tm_s = tmem + L::kS + x * kKeys + lanes;
      const uint32_t tm_p = tmem + L::kP + x * L::kPStep + lanes;
      const float a = p.scale_log2;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nx; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s(x), j & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        const int key0 = j * kKeys;
        bool done = false;
        if (__all_sync(0xffffffffu, a > 0.f && key0 + kKeys <= key_lim && (m > -INFINITY || !valid))) {
          uint32_t pk[kKeys / 2];
          float2 sum = make_float2(0.f, 0.f);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t ra[32], rb[32];
          tmem_ld32(tm_s, ra);
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) {
            uint32_t(&cur)[32] = (c & 1) ? rb : ra;
            uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
            prefill::tmem_ld_wait_tied(cur);
            if (c + 1 < kKeys / 32) tmem_ld32(tm_s + (c + 1) * 32, nxt);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
#pragma unroll
              for (int f = 0; f < 4; ++f)
                mx[f] = prefill::fmax3(mx[f], __uint_as_float(cur[e + f]), __uint_as_float(cur[e + 4 + f]));
            }
            weigh<BF16, false>(cur, 32, a, m, sum, &pk[c * 16]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a;
          if (!__any_sync(0xffffffffu, valid && !(top <= m + kRescaleLog2))) {
            l += sum.x + sum.y;
            if (L::kApart && j > 0) {
              ok = __all_sync(0xffffffffu, mbar_wait(bar_pv(x), (j - 1) & 1, p.status));
              if (!ok) break;
              tc_fence_after();
            }
            prefill::store_p<kKeys>(tm_p, pk);
            done = true;
          }
        }
        if (!done) {
          // masked keys, a first tile, or a maximum that grew: its maximum first, then its weights.
          // Thirty-two columns that a whole warp sees, or that none of its rows sees, need no look at
          // each (a warp's rows are few query tokens, so that is most of them).
          float top = -INFINITY;
          uint32_t ra[32], rb[32];
          tmem_ld32(tm_s, ra);
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) {
            uint32_t(&cur)[32] = (c & 1) ? rb : ra;
            uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
            prefill::tmem_ld_wait_tied(cur);
            if (c + 1 < kKeys / 32) tmem_ld32(tm_s + (c + 1) * 32, nxt);
            const int left = key_lim - (key0 + c * 32);
            if (__all_sync(0xffffffffu, left >= 32)) {
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                top = prefill::fmax3(top, __uint_as_float(cur[e]) * a, __uint_as_float(cur[e + 1]) * a);
            } else if (__any_sync(0xffffffffu, left > 0)) {
#pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, e < left ? __uint_as_float(cur[e]) * a : -INFINITY);
            }
          }
          const float m_new = fmaxf(m, top);
          const bool need = valid && m_new > m + kRescaleLog2;
          float alpha = 1.f;
          if (need) {
            alpha = exp2_approx(m - m_new);  // 0 when m is -inf
            m = m_new;
            l *= alpha;
          }
          if (j > 0) {
            // P_{j-1} V_{j-1} has to be in O before O is rescaled, and P_{j-1} read before P_j
            ok = __all_sync(0xffffffffu, mbar_wait(bar_pv(x), (j - 1) & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            if (__any_sync(0xffffffffu, need)) prefill::rescale_o<D>(tm_o, alpha);
          }
          const float m_use = m == -INFINITY ? 0.f : m;
          float2 sum = make_float2(0.f, 0.f);
          tmem_ld32(tm_s, ra);
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) {
            uint32_t(&cur)[32] = (c & 1) ? rb : ra;
            uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
            uint32_t pk[16];
            prefill::tmem_ld_wait_tied(cur);
            if (c + 1 < kKeys / 32) tmem_ld32(tm_s + (c + 1) * 32, nxt);
            const int left = key_lim - (key0 + c * 32);
            if (__any_sync(0xffffffffu, left > 0)) {
              weigh<BF16, true>(cur, left, a, m_use, sum, pk);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            }
            // (P over S: P's columns so far are no more than the scores already in registers)
            tmem_st16(tm_p + c * 16, pk);
          }
          l += sum.x + sum.y;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_p(x));
      }
      if (ok && nx > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_pv(x), (nx - 1) & 1, p.status));
        tc_fence_after();
      }
      if (ok) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int64_t row = seq.q0 + i;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + row * p.out_strides[0] + h * p.out_strides[1];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (nx > 0) {
            tmem_ld32(tm_o + c * 32, o);
            prefill::tmem_ld_wait_tied(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (!valid) continue;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float f = __uint_as_float(o[2 * e]) * inv, g = __uint_as_float(o[2 * e + 1]) * inv;
            w[e] = BF16 ? pack_bf16x2(f, g) : pack_f16x2(f, g);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4*>(dst + c * 32)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
        if (valid && p.lse) p.lse[row * p.Hq + h] = prefill::row_lse(m, l);
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
cudaError_t launch(const Params& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   int64_t items, cudaStream_t stream) {
  auto kern = forward_kernel<D, BF16>;
  cudaError_t e = ensure_smem_limit(kern, Layout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(items * p.Hkv), kThreads, Layout<D>::kAlloc, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

int fail(int code, const char* fmt, const char* who, long a = 0, long b = 0, long c = 0) {
  char msg[256];
  snprintf(msg, sizeof msg, fmt, who, a, b, c);
  return set_error(code, msg);
}

}  // namespace

int check_sizes(const char* who, int B, int Hq, int Hkv, int D, int total_q, int total_k, fa_dtype dtype,
                float scale) {
  if (B < 0 || total_q < 0 || total_k < 0)
    return fail(FA_ERR_INVALID_ARG, "%s: need B, total_q, total_k >= 0 (got %ld, %ld, %ld)", who, B, total_q, total_k);
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
    return fail(FA_ERR_INVALID_ARG, "%s: need Hq, Hkv > 0 and Hq %% Hkv == 0 (got %ld, %ld)", who, Hq, Hkv);
  if (Hq / Hkv > kRows)
    return fail(FA_ERR_UNSUPPORTED, "%s: query heads per kv head must be <= 128 (got %ld)", who, Hq / Hkv);
  if (D != 64 && D != 128)
    return fail(FA_ERR_UNSUPPORTED, "%s: D must be 64 or 128 (got %ld)", who, D);
  if (dtype != FA_BF16 && dtype != FA_FP16)
    return fail(FA_ERR_UNSUPPORTED, "%s: dtype must be FA_BF16 or FA_FP16 (got %ld)", who, (long)dtype);
  if (!(scale == scale) || isinf(scale)) return fail(FA_ERR_INVALID_ARG, "%s: scale must be finite", who);
  const int64_t width = kRows / (Hq / Hkv);
  const int64_t most = most_items(total_q, B, width), keys = most_items(total_k, B, kKeys);
  if ((most > keys ? most : keys) * Hkv > 2147483647LL)
    return fail(FA_ERR_UNSUPPORTED, "%s: too many tiles for one launch", who);
  return FA_OK;
}

int check_tensor(const char* who, const char* name, const void* base, const int64_t* strides, int tokens, int heads,
                 int D) {
  char msg[200];
  if (!base) {
    snprintf(msg, sizeof msg, "%s: null %s pointer", who, name);
    return set_error(FA_ERR_INVALID_ARG, msg);
  }
  bool fine = (reinterpret_cast<uintptr_t>(base) & 15u) == 0;
  const int n[2] = {tokens, heads};
  for (int i = 0; i < 2; ++i)
    fine = fine && (n[i] <= 1 || (strides[i] >= D && strides[i] % 8 == 0 && strides[i] < (1LL << 38)));
  if (!fine) {
    snprintf(msg, sizeof msg,
             "%s: %s must be 16-byte aligned, its token and head strides multiples of 16 bytes and at least D", who, name);
    return set_error(FA_ERR_INVALID_ARG, msg);
  }
  return FA_OK;
}

bool encode_rows(CUtensorMap* map, bool bf16, const void* base, const int64_t* strides, int tokens, int heads, int D,
                 int box_tokens, int box_heads) {
  const uint64_t row = static_cast<uint64_t>(D) * 2;
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens > 0 ? tokens : 1)};
  // a dimension of one element may come with any stride
  const uint64_t str[2] = {heads > 1 ? static_cast<uint64_t>(strides[1]) * 2 : row,
                           tokens > 1 ? static_cast<uint64_t>(strides[0]) * 2 : row * heads};
  const uint32_t box[3] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens)};
  return encode_tiled(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims,
                      str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace packed
}  // namespace fa

using namespace fa;

extern "C" int fa_prefill_packed(const fa_packed_args* a, void* stream) {
  const char* who = "fa_prefill_packed";
  if (!a) return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed: null argument struct");
  int rc = packed::check_sizes(who, a->B, a->Hq, a->Hkv, a->D, a->total_q, a->total_k, a->dtype, a->scale);
  if (rc != FA_OK || a->B == 0 || a->total_q == 0) return rc;
  if (!a->cu_seqlens_q || !a->cu_seqlens_k)
    return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed: null cu_seqlens pointer");
  if ((rc = packed::check_tensor(who, "q", a->q, a->q_strides, a->total_q, a->Hq, a->D)) != FA_OK) return rc;
  if ((rc = packed::check_tensor(who, "out", a->out, a->out_strides, a->total_q, a->Hq, a->D)) != FA_OK) return rc;
  if (a->total_k > 0 &&
      ((rc = packed::check_tensor(who, "k", a->k, a->k_strides, a->total_k, a->Hkv, a->D)) != FA_OK ||
       (rc = packed::check_tensor(who, "v", a->v, a->v_strides, a->total_k, a->Hkv, a->D)) != FA_OK))
    return rc;
  uint32_t* status = device_status_ptr();
  if (!status) return set_error(FA_ERR_CUDA, "fa_prefill_packed: no usable CUDA device");
  packed::Params p{};
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
  p.out = a->out;
  memcpy(p.out_strides, a->out_strides, sizeof p.out_strides);
  p.lse = a->lse;
  p.status = status;
  const bool bf16 = a->dtype == FA_BF16;
  // without keys nothing reads the maps of K and V
  const void* k = a->total_k > 0 ? a->k : a->q;
  const void* v = a->total_k > 0 ? a->v : a->q;
  CUtensorMap tq, tk, tv;
  if (!packed::encode_rows(&tq, bf16, a->q, a->q_strides, a->total_q, a->Hq, a->D, p.q_per_tile, p.G) ||
      !packed::encode_rows(&tk, bf16, k, a->k_strides, a->total_k, a->total_k > 0 ? a->Hkv : 1, a->D, packed::kKeys, 1) ||
      !packed::encode_rows(&tv, bf16, v, a->v_strides, a->total_k, a->total_k > 0 ? a->Hkv : 1, a->D, packed::kKeys, 1))
    return set_error(FA_ERR_CUDA, "fa_prefill_packed: tensor map rejected");
  const int64_t items = packed::most_items(a->total_q, a->B, 2 * p.q_per_tile);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->D == 128 ? (bf16 ? packed::launch<128, true>(p, tq, tk, tv, items, st)
                                      : packed::launch<128, false>(p, tq, tk, tv, items, st))
                              : (bf16 ? packed::launch<64, true>(p, tq, tk, tv, items, st)
                                      : packed::launch<64, false>(p, tq, tk, tv, items, st));
  if (e != cudaSuccess) return set_error(FA_ERR_CUDA, cudaGetErrorString(e));
  return FA_OK;
}
