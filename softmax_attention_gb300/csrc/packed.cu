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
// serve both tiles.  Each tile has its own softmax warpgroup and its own issuing warp; tensor
// memory holds O and S of both, with P in 16 bits written over S (D = 128) or beside it (D = 64).
//
// Why two tiles: a tile's chain S_j -> softmax -> P_j V_j -> S_{j+1} leaves the tensor cores idle
// while its softmax runs; the other tile's products fill that time.  The issuers take turns, for the two
// tiles' products mixed in the pipe take longer than one after the other (a 16K-token prompt of 16 heads in 4
// groups: 995 us without turns, 761 with them, before the steps below).  An issuer waits for P_j, V_j
// and K_{j+1} before it issues P_j V_j and S_{j+1} together: once a thread has committed products
// its next look at shared memory is held until they finish, so a wait between the two would
// drain the pipe.  S_{j+1} may be issued behind P_j V_j although it overwrites P_j: products of
// one thread and one shape run in order (D = 64, where the shapes differ, keeps P apart).
//
// The softmax works on a row 32 scores at a time against the maximum so far (of the first 32 scores
// to begin with), and looks for a larger one on the way; only if a row's maximum turns out to be more
// than 2^8 times larger is the tile done again in two passes (scores of standard deviation 1: hardly ever; of 2, 4 and 8:
// a 16K-token prompt takes 760, 1190 and 1298 us for 638).  So no more than 64 scores and the 64
// registers of packed P are held, and the maximum is not in the way of the first exponential.
//
// A block stays for all of its work items: while one ends, the copies and the first scores of the
// next are under way, so that only its first item pays for set-up and an empty pipe (packed.cuh
// says how the items are dealt out).
//
// Bound by the tensor cores: that prompt takes 616 to 671 us, from board to board (1640 to 1790 TFLOP/s of its
// unmasked half, 0.85 to 0.92 of the measured bf16 rate), three quarters of all clocks with a product in the pipe and
// the exponentials' pipe busy in 38 % (counters of four sequences of 8192 tokens).  At D = 64 by the softmax instead,
// which is the same per score for half the products (four sequences of 4096 tokens: 150 us, 920 TFLOP/s).  Short
// sequences pay some 3.5 us a work item for its first and last tiles (512 to 2048 tokens: 180 us, 1100 TFLOP/s).
// Registers stand in the way of more: the softmax warps use all of their 168, and each of these spilled: runs of 32
// scores that no row of the warp sees skipped in a masked tile (180 -> 217 us), masks as words of 32 bits (293).
// Issuing by one thread in a loop that is not unrolled 1012 us, by a warp's elected lane from uniform registers 689 ->
// 650, the turn given after the commits instead of among the products 626.
//
// Warps (384 threads): 0-3 softmax A, 4-7 softmax B, 8 copies, 9 issuer A (and tensor memory), 10
// issuer B, 11 finds the work items and clears what a last V tile holds past its sequence's end.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "dependent.cuh"
#include "internal.h"
#include "packed.cuh"

namespace fa {
namespace packed {
namespace {

using prefill::kLn2;
using prefill::kRescaleLog2;

constexpr int kThreads = 384;
constexpr int kItems = 4;  // work items on their way from the scheduling warp to the others

template <int D>
struct Layout {
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kBlock = kRows * 128;          // 128 rows x 64 columns of 16 bits
  static constexpr int kTile = kBlock * (D / 64);     // a Q tile, or a ring slot of K or V
  static constexpr int kRing = 2 * kTile;
  static constexpr int kStage = kRing + kSlots * kTile;  // 32 rows x 64 columns of each softmax warp's output
  static constexpr int kBars = kStage + 8 * 32 * 128;
  // full[slots], empty[slots], tail[slots], q[2], q_free[2], s[2], p[2], pv[2], o_free[2], done[2],
  // item[items], item_read[items]
  static constexpr int kNumBars = 3 * kSlots + 14 + 2 * kItems;
  static constexpr int kAlloc = kBars + kNumBars * 8 + 1024;  // room to align the base
  // tensor memory columns
  static constexpr bool kApart = D == 64;             // P beside S
  static constexpr int kS = 2 * D, kP = kApart ? kS + 2 * kKeys : kS, kPStep = kApart ? kKeys / 2 : kKeys;
  static_assert(kAlloc <= 232448, "shared memory budget");
  static_assert(kKeys == kRows, "one block size for Q, K and V");
};

struct Tile {
  int q0, end, n;  // first query in its sequence, keys that it sees, KV tiles
};

__device__ __forceinline__ Tile make_tile(const Params& p, const Seq& s, int q0) {
  Tile t{q0, 0, 0};
  if (q0 < s.nq) {
    const int last = min(s.nq, q0 + p.q_per_tile) - 1;
    t.end = p.causal ? min(s.nk, max(0, last + s.nk - s.nq + 1)) : s.nk;
    t.n = (t.end + kKeys - 1) / kKeys;
  }
  return t;
}

// An item's two query tiles and the KV tiles that go through the ring for them: first, first + 1, ...; of
// each tile's own, n counts from there.
template <bool SPLIT>
struct Work {
  Tile a, b;
  int first, n;
  __device__ __forceinline__ Work(const Params& p, const Item& item) {
    a = make_tile(p, item.seq, item.at);
    b = make_tile(p, item.seq, item.at + p.q_per_tile);
    first = 0;
    n = max(a.n, b.n);
    if (SPLIT) {
      const int per = (n + p.splits - 1) / p.splits;
      first = min(n, item.split * per);
      const int last = min(n, first + per);
      a.n = max(0, min(a.n, last) - first);
      b.n = max(0, min(b.n, last) - first);
      n = last - first;
    }
  }
  // whether the last V tile reaches past the sequence
  __device__ __forceinline__ bool tail(const Item& item) const { return n > 0 && (first + n) * kKeys > item.seq.nk; }
};

// Thirty-two scores against the maximum m: exponentials packed, their sum added.
template <bool BF16>
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], float a, float m, float2& sum, uint32_t* pk) {
  const float2 a2 = make_float2(a, a), nm = make_float2(-m, -m);
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const float2 t = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), a2, nm);
    const float2 e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
    sum = __fadd2_rn(sum, e);
    pk[c] = BF16 ? pack_bf16x2(e.x, e.y) : pack_f16x2(e.x, e.y);
  }
}

// One pass over a row's scores of a tile against the maximum m, with the next 32 on their way while 32
// are worked on: exponentials packed, their sum added, the largest score returned.  With MASK the first
// `left` alone count (apart, because the masks' branches would cost the common pass a quarter).
template <bool BF16, bool MASK>
__device__ __forceinline__ float sweep(uint32_t tm_s, int left, float a, float m, float2& sum, uint32_t (&pk)[kKeys / 2]) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  uint32_t ra[32], rb[32];
  tmem_ld32(tm_s, ra);
#pragma unroll
  for (int c = 0; c < kKeys / 32; ++c) {
    uint32_t(&cur)[32] = (c & 1) ? rb : ra;
    uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
    prefill::tmem_ld_wait_tied(cur);
    if (c + 1 < kKeys / 32) tmem_ld32(tm_s + (c + 1) * 32, nxt);
    if (MASK) {
#pragma unroll
      for (int e = 0; e < 32; ++e) cur[e] = 32 * c + e < left ? cur[e] : 0xff800000u;  // -inf
    }
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        mx[f] = prefill::fmax3(mx[f], __uint_as_float(cur[e + f]), __uint_as_float(cur[e + 4 + f]));
    }
    weigh<BF16>(cur, a, m, sum, &pk[c * 16]);
  }
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// The barriers, by their addresses.
template <int D>
struct Bars {
  using L = Layout<D>;
  uint32_t at;
  __device__ __forceinline__ uint32_t one(int i) const { return at + 8u * i; }
  __device__ __forceinline__ uint32_t full(int slot) const { return one(slot); }
  __device__ __forceinline__ uint32_t empty(int slot) const { return one(L::kSlots + slot); }
  // of a V tile that reaches past its sequence: it lands here, and is full when its last rows are cleared
  __device__ __forceinline__ uint32_t tail(int slot) const { return one(2 * L::kSlots + slot); }
  __device__ __forceinline__ uint32_t q(int x) const { return one(3 * L::kSlots + x); }
  __device__ __forceinline__ uint32_t q_free(int x) const { return one(3 * L::kSlots + 2 + x); }
  __device__ __forceinline__ uint32_t s(int x) const { return one(3 * L::kSlots + 4 + x); }
  __device__ __forceinline__ uint32_t p(int x) const { return one(3 * L::kSlots + 6 + x); }
  __device__ __forceinline__ uint32_t pv(int x) const { return one(3 * L::kSlots + 8 + x); }
  __device__ __forceinline__ uint32_t o_free(int x) const { return one(3 * L::kSlots + 10 + x); }
  __device__ __forceinline__ uint32_t done(int x) const { return one(3 * L::kSlots + 12 + x); }
  __device__ __forceinline__ uint32_t item(int i) const { return one(3 * L::kSlots + 14 + i); }
  __device__ __forceinline__ uint32_t item_read(int i) const { return one(3 * L::kSlots + 14 + kItems + i); }
};

// The k-th item, copied from its place in shared memory; false: no more, or a wait ran out.
template <int D>
__device__ __forceinline__ bool next_item(const Bars<D>& bars, const Item* items, int k, Item& item, const Params& p) {
  if (!mbar_wait(bars.item(k % kItems), (k / kItems) & 1, p)) return false;
  item = items[k % kItems];
  mbar_arrive(bars.item_read(k % kItems));
  return item.at >= 0;
}

// The issuing warp of tile X.  All lanes wait, one issues; the order of the waits puts the last one to
// come true, for P, in front of the products.
template <int D, bool BF16, bool SPLIT, int X>
__device__ __forceinline__ void issue(const Params& p, uint32_t s_base, uint32_t bar_base, uint32_t tmem,
                                      const Item* items, volatile int* turns) {
  using L = Layout<D>;
  const Bars<D> bars{bar_base};
  tmem = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
  constexpr uint32_t idesc_s = idesc_f16(BF16, kRows, kKeys, false, false);
  constexpr uint32_t idesc_o = idesc_f16(BF16, kRows, D, false, true);
  const uint64_t q_desc = sdesc_sw128(s_base + X * L::kTile, 16, 1024);
  const uint64_t k_desc = sdesc_sw128(s_base + L::kRing, 16, 1024);
  const uint64_t v_desc = sdesc_sw128(s_base + L::kRing, L::kBlock, 1024);
  const uint32_t tm_o = tmem + X * D, tm_s = tmem + L::kS + X * kKeys, tm_p = tmem + L::kP + X * L::kPStep;
  bool ok = true;
  auto wait = [&](uint32_t bar, int phase) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, p));
    return ok;
  };
  auto issue_s = [&](int slot) {
    const uint64_t kd = sdesc_add(k_desc, slot * L::kTile);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = (kk / 4) * L::kBlock + (kk % 4) * 32;
      mma_ss(tm_s, sdesc_add(q_desc, off), sdesc_add(kd, off), idesc_s, kk > 0 ? 1u : 0u);
    }
  };
  int slot = 0, lap = 0;  // the ring entry that comes next, and how often the ring has been gone through
  auto next = [&]() {
    if (++slot == L::kSlots) {
      slot = 0;
      ++lap;
    }
  };
  int uses = 0, steps = 0, theirs = 0;  // items and KV tiles of this tile, KV tiles of the other
  for (int k = 0; ok; ++k) {
    Item got{};
    bool more = false;
    if (__all_sync(0xffffffffu, mbar_wait(bars.item(k % kItems), (k / kItems) & 1, p))) {
      got = items[k % kItems];
      __syncwarp();
      if (elected()) mbar_arrive(bars.item_read(k % kItems));
      more = got.at >= 0;
    }
    if (!__any_sync(0xffffffffu, more)) break;
    const Work<SPLIT> work(p, got);
    const int nx = uniform(X ? work.b.n : work.a.n), other_n = uniform(X ? work.a.n : work.b.n);
    const int n = uniform(work.n), end = uniform((X ? work.b.end : work.a.end) - work.first * kKeys);
    if (nx > 0) {
      if (!wait(bars.q(X), uses) || !wait(bars.full(slot), lap)) break;
      tc_fence_after();
      if (elected()) {
        issue_s(slot);
        tc_commit(bars.s(X));
        tc_commit(bars.empty(slot));
        if (nx == 1) tc_commit(bars.q_free(X));
      }
      next();
    }
    for (int j = 0; j < nx; ++j) {
      const int v_slot = slot, v_lap = lap;
      next();
      if (!wait(bars.full(v_slot), v_lap)) break;
      if (j + 1 < nx && !wait(bars.full(slot), lap)) break;
      // O of the item before has to be read before the first product overwrites it
      if (j == 0 && uses > 0 && !wait(bars.o_free(X), uses - 1)) break;
      // The other tile's turn first: its j-th pair of products before B's, its (j-1)-th before A's.  An
      // order to keep the tiles out of step, nothing that a result depends on: so the wait may give up.
      const int want = theirs + min(other_n, X ? j + 1 : j);
      for (int spin = 0; spin < 4096 && turns[1 - X] < want; ++spin) {}
      if (!wait(bars.p(X), steps + j)) break;
      tc_fence_after();
      if (elected()) {
        const uint64_t vd = sdesc_add(v_desc, v_slot * L::kTile);
        // of the last tile, no more keys than the tile sees
        const int ksteps = min(kKeys / 16, (end - j * kKeys + 15) / 16);
        if (ksteps == kKeys / 16) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts(tm_o, tm_p + kk * 8, sdesc_add(vd, kk * 2048), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < ksteps; ++kk)
            mma_ts(tm_o, tm_p + kk * 8, sdesc_add(vd, kk * 2048), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
        }
        if (j + 1 < nx) issue_s(slot);
        tc_commit(bars.pv(X));
        tc_commit(bars.empty(v_slot));
        if (j + 1 < nx) {
          tc_commit(bars.s(X));
          tc_commit(bars.empty(slot));
          if (j + 2 == nx) tc_commit(bars.q_free(X));
        }
        // After the commits, where the store is held until the products are done: with the tiles' products
        // mixed in the pipe each takes longer (16K-token prompt: 642 us with the store in front of the commits,
        // 783 and more with it among the products).
        turns[X] = steps + j + 1;
      }
      __syncwarp();
      if (j + 1 < nx) next();
    }
    if (!ok) break;
    // tiles that only the other one sees: released as they land, phase by phase
    for (int i = 2 * nx; i < 2 * n; ++i) {
      if (!wait(bars.full(slot), lap)) break;
      if (elected()) mbar_arrive(bars.empty(slot));
      next();
    }
    steps += nx;
    theirs += other_n;
    uses += nx > 0 ? 1 : 0;
  }
  // every product must finish before tensor memory and the ring are given up
  if (elected()) {
    tc_commit(bars.done(X));
    mbar_wait(bars.done(X), 0, nullptr);
  }
}

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    forward_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint32_t tmem_slot;
  __shared__ Item items[kItems];
  __shared__ int turns[2];  // pairs of products that each tile's issuer has put into the pipe
  const uint32_t s_base = smem_addr(smem);
  const Bars<D> bars{s_base + L::kBars};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 9) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 8 * 32) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bars.q(x), 1);
      mbar_init(bars.q_free(x), 1);
      mbar_init(bars.s(x), 1);
      mbar_init(bars.p(x), 128);
      mbar_init(bars.pv(x), 1);
      mbar_init(bars.o_free(x), 128);
      mbar_init(bars.done(x), 1);
      turns[x] = 0;
    }
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 2);  // both tiles
      mbar_init(bars.tail(s), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bars.item(i), 1);
      mbar_init(bars.item_read(i), 256 + 3);  // softmax, issuers, copies
    }
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp == 11) {
    // ------------------------------ work items, V's last rows --------------------------------
    const int width = 2 * p.q_per_tile;
    auto pieces = [&](int s, int& n, int& first) {
      const Seq q = load_seq(p, s);
      n = (q.nq + width - 1) / width;
      first = (p.causal ? max(0, q.nk - q.nq) : q.nk) / width;
    };
    Finder finder(p.B, !p.causal, pieces);
    int entries = 0;                // ring entries of the items so far
    uint32_t tail_phase = 0;        // of each slot's tail barrier, a bit
    int clear_at = -1, clear_row = 0;  // the item before: entry of its last V tile, first row to clear
    bool ok = true, more = true;
    for (int k = 0; ok && (more || clear_at >= 0); ++k) {
      Item item{};
      item.at = -1;
      if (more) {
        const int w = dealt(k);
        int b, t;
        finder.find(w / (SPLIT ? p.Hkv * p.splits : p.Hkv), pieces, b, t);
        if (b >= 0) {
          item.seq = load_seq(p, b);
          item.at = t * width;
          item.head = SPLIT ? w / p.splits % p.Hkv : w % p.Hkv;
          item.split = SPLIT ? w % p.splits : 0;
        }
        if (k >= kItems) ok = __all_sync(0xffffffffu, mbar_wait(bars.item_read(k % kItems), (k / kItems - 1) & 1, p));
        if (ok && lane == 0) {
          items[k % kItems] = item;
          mbar_arrive(bars.item(k % kItems));
        }
        more = b >= 0;
      }
      if (ok && clear_at >= 0) {
        // Rows past the sequence's end hold another sequence's values, or none: P is 0 there, but 0
        // times an infinity or NaN would spoil O.
        const int slot = clear_at % L::kSlots;
        ok = __all_sync(0xffffffffu, mbar_wait(bars.tail(slot), (tail_phase >> slot) & 1, p));
        tail_phase ^= 1u << slot;
        uint8_t* v = smem + L::kRing + slot * L::kTile;
        const int per = (kKeys - clear_row) * 8;
        if (ok)
          for (int i = lane; i < per * (D / 64); i += 32)
            *reinterpret_cast<uint4*>(v + (i / per) * L::kBlock + clear_row * 128 + (i % per) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.full(slot));
        clear_at = -1;
      }
      if (item.at >= 0) {
        const Work<SPLIT> work(p, item);
        entries += 2 * work.n;
        if (work.tail(item)) {
          clear_at = entries - 1;
          clear_row = item.seq.nk - (work.first + work.n - 1) * kKeys;
        }
      }
    }
  } else if (warp == 8) {
    // ---------------------------------- copies ----------------------------------------------
    if (lane == 0) {
      bool ok = true;
      int entry = 0, q_uses[2] = {0, 0};
      // a bit for each slot: the phase of its tail barrier; whether its last copy was to that one.  (One for
      // each slot: the last V of a short item may still be on its way when the next item's is copied.)
      uint32_t tail_phase = 0, to_tail = 0;
      Item item;
      for (int k = 0; ok && next_item(bars, items, k, item, p); ++k) {
        const Work<SPLIT> work(p, item);
        const int n = work.n;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const Tile tile = x ? work.b : work.a;
          if (!ok || tile.n == 0) continue;
          if (q_uses[x] > 0 && !(ok = mbar_wait(bars.q_free(x), (q_uses[x] - 1) & 1, p))) continue;
          mbar_arrive_expect_tx(bars.q(x), static_cast<uint32_t>(128 * (D / 64) * p.G * p.q_per_tile));
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + x * L::kTile + kb * L::kBlock, &tm_q, bars.q(x), kb * 64, item.head * p.G,
                        item.seq.q0 + tile.q0);
          ++q_uses[x];
        }
        const bool tail = work.tail(item);
        for (int i = 0; ok && i < 2 * n; ++i, ++entry) {      // K_0, V_0, K_1, V_1, ...
          const int slot = entry % L::kSlots;
          if (entry >= L::kSlots && !(ok = mbar_wait(bars.empty(slot), (entry / L::kSlots - 1) & 1, p))) break;
          uint32_t bar = bars.full(slot);
          to_tail &= ~(1u << slot);
          if (tail && i == 2 * n - 1) {
            bar = bars.tail(slot);
            to_tail |= 1u << slot;
            tail_phase ^= 1u << slot;
          }
          mbar_arrive_expect_tx(bar, L::kTile);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(s_base + L::kRing + slot * L::kTile + kb * L::kBlock, (i & 1) ? &tm_v : &tm_k, bar, kb * 64,
                        item.head, item.seq.k0 + (work.first + i / 2) * kKeys);
        }
      }
      if (!ok) {
        // A wait ran out: let the copies in flight land before the block ends
        for (int x = 0; x < 2; ++x)
          if (q_uses[x] > 0) mbar_wait(bars.q(x), (q_uses[x] - 1) & 1, nullptr);
        for (int i = max(0, entry - L::kSlots); i < entry; ++i) {
          const int slot = i % L::kSlots;
          if ((to_tail >> slot) & 1) mbar_wait(bars.tail(slot), ((tail_phase >> slot) & 1) ^ 1, nullptr);
          else mbar_wait(bars.full(slot), (i / L::kSlots) & 1, nullptr);
        }
      }
    }
  } else if (warp == 9) {
    issue<D, BF16, SPLIT, 0>(p, s_base, bars.at, tmem, items, turns);
  } else if (warp == 10) {
    issue<D, BF16, SPLIT, 1>(p, s_base, bars.at, tmem, items, turns);
  } else {
    // --------------------------- softmax, epilogue: a row a thread ---------------------------
    const int x = warp / 4, r = threadIdx.x % 128;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tm_o = tmem + x * D + lanes, tm_s = tmem + L::kS + x * kKeys + lanes;
    const uint32_t tm_p = tmem + L::kP + x * L::kPStep + lanes;
    const float a = p.scale_log2;
    const int row_token = r / p.G, row_head = r % p.G;
    bool ok = true;
    int steps = 0;  // KV tiles of this query tile so far
    // The item before, whose output is still in tensor memory: if the first scores of the next are there, they
    // are dealt with first, so that the wait for its last product, and the stores, have work beside them.
    bool pending = false;
    uint8_t* out_row = nullptr;
    float* lse_row = nullptr;
    float out_m = 0.f, out_l = 0.f;
    int out_step = 0;
    bool more = true;
    for (int k = 0; ok && more; ++k) {
      Item item{};
      more = __all_sync(0xffffffffu, next_item(bars, items, k, item, p));
      int first = 0;
      Tile tile;
      if (SPLIT) {
        const Work<SPLIT> work(p, item);
        tile = x ? work.b : work.a;
        first = work.first * kKeys;
      } else {
        tile = make_tile(p, item.seq, item.at + x * p.q_per_tile);
      }
      const int nx = more ? tile.n : 0;
      const int i = tile.q0 + row_token, h = item.head * p.G + row_head;
      const bool valid = more && r < p.G * p.q_per_tile && i < item.seq.nq;
      // a row of no query sees everything, so that it never asks for the slow path
      const int key_lim = !valid ? 0x7fffffff : p.causal ? min(item.seq.nk, i + item.seq.nk - item.seq.nq + 1) : item.seq.nk;
      float m = -INFINITY, l = 0.f;
      for (int j = -1; j < nx; ++j) {
        if (j >= 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(bars.s(x), steps & 1, p));
          if (!ok) break;
          tc_fence_after();
          const int left = key_lim - first - j * kKeys;  // keys of the tile that the row sees
          bool done = false;
          if (a > 0.f) {
            const bool masked = __any_sync(0xffffffffu, left < kKeys);
            if (j == 0) {
              // A first guess at the maximum: that of the first 32 scores.  Where all of them are hidden or -inf, one
              // below every score: the first that is finite then takes the slow path, however small it is.
              uint32_t raw[32];
              tmem_ld32(tm_s, raw);
              prefill::tmem_ld_wait_tied(raw);
              float top = -INFINITY;
  #pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, e < left ? __uint_as_float(raw[e]) : -INFINITY);
              m = top > -INFINITY ? top * a : -1e37f;
            }
            uint32_t pk[kKeys / 2];
            float2 sum = make_float2(0.f, 0.f);
            const float top = a * (masked ? sweep<BF16, true>(tm_s, left, a, m, sum, pk) : sweep<BF16, false>(tm_s, left, a, m, sum, pk));
            if (!__any_sync(0xffffffffu, valid && !(top <= m + kRescaleLog2))) {
              l += sum.x + sum.y;
              // (P_{j-1} has been read: the commit that told of S_j covers P_{j-1} V_{j-1} before it)
              prefill::store_p<kKeys>(tm_p, pk);
              done = true;
            }
          }
          if (!done) {
            // a maximum that grew (or a scale that is not positive): the maximum first, then the weights
            float top = -INFINITY;
  #pragma unroll 1
            for (int c = 0; c < kKeys; c += 32) {
              uint32_t raw[32];
              tmem_ld32(tm_s + c, raw);
              prefill::tmem_ld_wait_tied(raw);
  #pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, c + e < left ? __uint_as_float(raw[e]) * a : -INFINITY);
            }
            const float before = l > 0.f ? m : -INFINITY;  // (a guess that nothing was added to is none)
            const float m_new = fmaxf(before, top);
            const bool need = valid && m_new > before + kRescaleLog2;
            float alpha = 1.f;
            if (need) {
              alpha = exp2_approx(before - m_new);  // 0 when nothing was added before
              m = m_new;
              l *= alpha;
            }
            if (j > 0) {
              // P_{j-1} V_{j-1} has to be in O before O is rescaled, and P_{j-1} read before P_j
              ok = __all_sync(0xffffffffu, mbar_wait(bars.pv(x), (steps - 1) & 1, p));
              if (!ok) break;
              tc_fence_after();
              if (__any_sync(0xffffffffu, need)) prefill::rescale_o<D>(tm_o, alpha);
            }
            const float m_use = m == -INFINITY ? 0.f : m;
            float2 sum = make_float2(0.f, 0.f);
  #pragma unroll 1
            for (int c = 0; c < kKeys; c += 32) {
              uint32_t raw[32], pk[16];
              tmem_ld32(tm_s + c, raw);
              prefill::tmem_ld_wait_tied(raw);
  #pragma unroll
              for (int e = 0; e < 32; ++e) raw[e] = c + e < left ? __float_as_uint(__uint_as_float(raw[e]) * a) : 0xff800000u;
              weigh<BF16>(raw, 1.f, m_use, sum, pk);
              // (P over S: P's columns so far are no more than the scores already in registers)
              tmem_st16(tm_p + c / 2, pk);
            }
            l += sum.x + sum.y;
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bars.p(x));
          ++steps;
        }
        if (pending && (j == 0 || nx == 0 || !__all_sync(0xffffffffu, mbar_test_wait(bars.s(x), steps & 1)))) {
          pending = false;
          ok = __all_sync(0xffffffffu, mbar_wait(bars.pv(x), out_step & 1, p));
          if (!ok) break;
          tc_fence_after();
          const float inv = out_l > 0.f ? 1.f / out_l : 0.f;
          // A thread's row would be written 16 bytes at a time, each of a warp's stores touching 32 rows:
          // through shared memory (128-byte swizzle) a store writes four rows' 128 bytes.
          uint8_t* mine = smem + L::kStage + warp * (32 * 128);
          constexpr int kSlab = SPLIT ? 32 : 64;  // columns of 128 bytes
#pragma unroll 1
          for (int c = 0; c < D / kSlab; ++c) {
            uint32_t oa[32], ob[32];
            tmem_ld32(tm_o + c * kSlab, oa);
            if (!SPLIT) tmem_ld32(tm_o + c * kSlab + 32, ob);
            prefill::tmem_ld_wait_tied(oa);
            if (!SPLIT) prefill::tmem_ld_wait_tied(ob);
            if (c == D / kSlab - 1) {
              tc_fence_before();
              mbar_arrive(bars.o_free(x));
            }
            if (SPLIT) {
              prefill::stage_slab_f32(oa, inv, mine, lane);
            } else {
              prefill::stage_slab16<BF16>(oa, inv, mine, lane, 0);
              prefill::stage_slab16<BF16>(ob, inv, mine, lane, 1);
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int rr = 4 * e + lane / 8;
              const uint4 v = *reinterpret_cast<const uint4*>(mine + rr * 128 + ((lane % 8) ^ (rr & 7)) * 16);
              uint8_t* to = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out_row), rr));
              if (to) reinterpret_cast<uint4*>(to + c * 128)[lane % 8] = v;
            }
            __syncwarp();
          }
          // (no key seen: -inf; a NaN among the scores: l is NaN, and so is lse)
          if (lse_row) *lse_row = out_l == 0.f ? -INFINITY : (out_m + log2f(out_l)) * kLn2;
        }
      }
      if (!ok || !more) break;
      const int64_t row = item.seq.q0 + i;
      uint8_t* dst = nullptr;
      float* dst_lse = nullptr;
      if (valid && SPLIT) {
        const int64_t at = (row * p.Hq + h) * p.splits + item.split;
        dst = reinterpret_cast<uint8_t*>(p.o_part + at * D);
        dst_lse = p.lse_part + at;
      } else if (valid) {
        dst = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.out) + row * p.out_strides[0] + h * p.out_strides[1]);
        if (p.lse) dst_lse = p.lse + row * p.Hq + h;
      }
      if (nx > 0) {
        pending = true;
        out_row = dst;
        lse_row = dst_lse;
        out_m = m;
        out_l = l;
        out_step = steps - 1;
      } else {  // rows that see no key
        if (dst)
          for (int c = 0; c < D / (SPLIT ? 4 : 8); ++c) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
        if (dst_lse) *dst_lse = -INFINITY;
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

// Parts of the rows' keys joined (in 16 bits, by out's strides, and only the rows of a sequence): lse = ln sum_s e^{lse_s}, out = sum_s e^{lse_s - lse} o_s.  A block a
// token, a warp a head at a time, eight parts on their way at once.
constexpr int kJoinThreads = 256;
constexpr int kMaxSplits = 32;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Params p) {
  constexpr int kCols = D / 32;  // columns a lane
  const int token = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // rows of no sequence are left as they were
  bool mine = false;
  for (int b = threadIdx.x; b < p.B; b += kJoinThreads) {
    const int first = __ldg(p.cu_q + b), end = __ldg(p.cu_q + b + 1);
    mine = mine || (first >= 0 && first <= token && token < end && end <= p.total_q);
  }
  wait_for_previous();  // (by every block: what follows this kernel counts on the end of the one before it)
  if (!__syncthreads_or(mine)) return;
  for (int h = warp; h < p.Hq; h += kJoinThreads / 32) {
    const int64_t row = static_cast<int64_t>(token) * p.Hq + h;
    const float* o = p.o_part + row * p.splits * D + lane * kCols;
    const float part = lane < p.splits ? p.lse_part[row * p.splits + lane] : -INFINITY;
    float top = part;
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float m = top == -INFINITY ? 0.f : top;
    const float e = exp2_approx((part - m) * prefill::kLog2e);
    float total = 0.f, y[kCols] = {};
    for (int s0 = 0; s0 < p.splits; s0 += 8) {
      float x[8][kCols];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s0 + s >= p.splits) break;
        if constexpr (kCols == 4) {
          const float4 v = *reinterpret_cast<const float4*>(o + (s0 + s) * D);
          x[s][0] = v.x;
          x[s][1] = v.y;
          x[s][2] = v.z;
          x[s][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(o + (s0 + s) * D);
          x[s][0] = v.x;
          x[s][1] = v.y;
        }
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s0 + s >= p.splits) break;
        const float w = __shfl_sync(0xffffffffu, e, s0 + s);
        total += w;
#pragma unroll
        for (int c = 0; c < kCols; ++c) y[c] = fmaf(w, x[s][c], y[c]);
      }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;  // (a NaN stays one)
    uint16_t* to = static_cast<uint16_t*>(p.out) + token * p.out_strides[0] + h * p.out_strides[1] + lane * kCols;
    uint32_t w[kCols / 2];
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c)
      w[c] = BF16 ? pack_bf16x2(y[2 * c] * inv, y[2 * c + 1] * inv) : pack_f16x2(y[2 * c] * inv, y[2 * c + 1] * inv);
    if constexpr (kCols == 4) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(to) = w[0];
    if (lane == 0 && p.lse) p.lse[row] = total == 0.f ? -INFINITY : m + logf(total);
  }
}

template <int D, bool BF16>
cudaError_t launch(const Params& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   int64_t items, cudaStream_t stream) {
  auto kern = p.splits > 1 ? forward_kernel<D, BF16, true> : forward_kernel<D, BF16, false>;
  cudaError_t e = ensure_smem_limit(kern, Layout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t work = items * p.Hkv * p.splits, sms = num_sms() > 0 ? num_sms() : 152;
  kern<<<static_cast<unsigned>(work < sms ? work : sms), kThreads, Layout<D>::kAlloc, stream>>>(tq, tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(join_kernel<D, BF16>, static_cast<unsigned>(p.total_q), 1, kJoinThreads, 0, stream, p);
}

// Parts that the keys are split into: as many as give no SM a second work item, each of eight KV tiles of a
// mean sequence at least; so one from half as many items as SMs on.  Measured (bf16, D = 128; us): 16 queries of
// 8 heads over 65,536 keys, 1 item: 637 whole, 88 in 8 parts, 32 in 32; 512 queries of 32 heads in 8 groups over
// 32,768 keys, 64 items: 342 whole, 186 in 2, 253 in 3; two of 512 over 16,384 keys, 128 items: 180 whole, 201 in
// 2; 1024 queries over their own keys, 64 items: 19 whole, 22 in 2 (four tiles each).
int plan_splits(const fa_packed_args* a) {
  if (a->num_splits > 0) return a->num_splits;
  const int64_t sms = num_sms() > 0 ? num_sms() : 152;
  const int64_t width = 2 * (kRows / (a->Hq / a->Hkv));
  const int64_t items = (a->total_q / width + (a->B + 1) / 2) * a->Hkv;  // a sequence's last one is half full
  int64_t s = sms / items;
  const int64_t most = a->total_k / (8LL * kKeys * a->B);
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;
  return s < 2 ? 1 : static_cast<int>(s);
}

size_t part_bytes(const fa_packed_args* a, int splits) {
  return (static_cast<size_t>(a->total_q) * a->Hq * splits * a->D * sizeof(float) + 255) / 256 * 256;
}

size_t workspace_bytes(const fa_packed_args* a, int splits) {
  if (splits == 1) return 0;
  return part_bytes(a, splits) + (static_cast<size_t>(a->total_q) * a->Hq * splits * sizeof(float) + 255) / 256 * 256;
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
  if (Hkv > 65535 || static_cast<int64_t>(total_q) * Hq > 2147483647LL - 65536 ||
      static_cast<int64_t>(total_k) * Hkv > 2147483647LL - 65536)
    return fail(FA_ERR_UNSUPPORTED, "%s: Hkv must be <= 65535, total_q * Hq and total_k * Hkv below 2^31 - 2^16", who);
  const int64_t width = kRows / (Hq / Hkv);
  const int64_t most = most_items(total_q, B, width), keys = most_items(total_k, B, kKeys);
  if ((most > keys ? most : keys) * Hkv > (1LL << 30))
    return fail(FA_ERR_UNSUPPORTED, "%s: too many tiles for one launch", who);
  return FA_OK;
}

int check_offsets(const char* who, const int32_t* cu_q, const int32_t* cu_k) {
  if (!cu_q || !cu_k) return fail(FA_ERR_INVALID_ARG, "%s: null cu_seqlens pointer", who);
  if (((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) & 3u) != 0)
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned cu_seqlens pointer", who);
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

extern "C" size_t fa_packed_workspace_size(const fa_packed_args* a) {
  if (!a || packed::check_sizes("fa_prefill_packed", a->B, a->Hq, a->Hkv, a->D, a->total_q, a->total_k, a->dtype,
                                a->scale) != FA_OK)
    return 0;
  if (a->B == 0 || a->total_q == 0 || a->num_splits < 0 || a->num_splits > packed::kMaxSplits) return 0;
  return packed::workspace_bytes(a, packed::plan_splits(a));
}

extern "C" int fa_prefill_packed(const fa_packed_args* a, void* stream) {
  const char* who = "fa_prefill_packed";
  if (!a) return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed: null argument struct");
  int rc = packed::check_sizes(who, a->B, a->Hq, a->Hkv, a->D, a->total_q, a->total_k, a->dtype, a->scale);
  if (rc != FA_OK || a->B == 0 || a->total_q == 0) return rc;
  if (a->num_splits < 0 || a->num_splits > packed::kMaxSplits)
    return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed: num_splits must be in [0, 32]");
  if (a->num_splits > 1 && packed::most_items(a->total_q, a->B, 2 * (packed::kRows / (a->Hq / a->Hkv))) * a->Hkv *
                                   a->num_splits > (1LL << 30))
    return set_error(FA_ERR_UNSUPPORTED, "fa_prefill_packed: too many tiles for that many parts");
  if ((rc = packed::check_offsets(who, a->cu_seqlens_q, a->cu_seqlens_k)) != FA_OK) return rc;
  if ((reinterpret_cast<uintptr_t>(a->lse) & 3u) != 0) return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed: misaligned lse");
  if ((rc = packed::check_tensor(who, "q", a->q, a->q_strides, a->total_q, a->Hq, a->D)) != FA_OK) return rc;
  if ((rc = packed::check_tensor(who, "out", a->out, a->out_strides, a->total_q, a->Hq, a->D)) != FA_OK) return rc;
  if (a->total_k > 0 &&
      ((rc = packed::check_tensor(who, "k", a->k, a->k_strides, a->total_k, a->Hkv, a->D)) != FA_OK ||
       (rc = packed::check_tensor(who, "v", a->v, a->v_strides, a->total_k, a->Hkv, a->D)) != FA_OK))
    return rc;
  const int splits = packed::plan_splits(a);
  const size_t need = packed::workspace_bytes(a, splits);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) {
    char msg[160];
    snprintf(msg, sizeof msg, "fa_prefill_packed: workspace of %zu bytes needed (got %zu)", need,
             a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
    return set_error(FA_ERR_WORKSPACE, msg);
  }
  if (need > 0 && (reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0)
    return set_error(FA_ERR_INVALID_ARG, "fa_prefill_packed: workspace must be 256-byte aligned");
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
  p.wait_ns = packed::wait_limit(a->total_q, a->total_k, p.q_per_tile);
  p.splits = splits;
  if (splits > 1) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    p.o_part = reinterpret_cast<float*>(ws);
    p.lse_part = reinterpret_cast<float*>(ws + packed::part_bytes(a, splits));
  }
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
