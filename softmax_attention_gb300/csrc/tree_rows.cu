// tree_rows.cu -- tree attention over an 8-bit paged cache for few rows (query heads of a kv head
// times drafted tokens): the decode step, where the cache's bytes are all the time there is.
//
// The warp-level matrix instruction (m16n8k16) takes its operands from registers: e4m3 codes go
// from shared memory to registers, are converted there (one instruction a pair) and multiplied,
// so a cache byte is written to shared memory once by TMA and read once.  (The 128-row tile of the
// tcgen05 kernel passes each byte through shared memory six times and spends its tensor time on
// empty rows: there 57 sequences of 4096 tokens, 8 kv heads, D = 128, are read at 3.2 TB/s.)
// Codes are the 16-row operand and q's rows the 8-column one, in both products: S^T = K Q^T and
// O^T += V^T P^T.  Eight rows or fewer, the decode step of up to eight query heads a kv head, then
// fill their tile; nine to sixteen take two (NT).  With q as the 16-row operand a decode step's
// matrix, exponential and O instructions were half empty: 718 instructions a warp and 32 tokens
// and three CTAs of 166 registers an SM, where this takes 128 registers and four CTAs (128
// sequences of 1K to 4K tokens: 135 -> 110 us, 6.2 TB/s or 0.92 of a copy; the 57 even ones 87 ->
// 83 us).  Two tiles lose one or two per cent to the transposition of the weights.
//
// Each warp runs alone: its own ring of slices (SL tokens of K and of V), its own barriers, its
// own online softmax; four warps of a CTA take the slices of a (sequence, kv head, part) in turn
// and are combined once at the end.  Nothing in the loop waits for another warp.
//
// Numbers.  K codes are exact in fp16.  A row of q is scaled by a power of two so that its
// largest element is in [2^14, 2^15), which makes its elements exact in fp16 down to 2^-31 of the row's
// maximum for bf16 (whose eight bits end above 2^-24 from 2^-17 on) and 2^-28 for fp16.  S = q k accumulates in fp32; the scales of q's row, of the token's
// K and the softmax scale multiply it there.  V's scale 2^ev goes into the weight: with x the
// score in log2 units, O += 2^(x + ev - mo) v over the codes v, mo a running maximum of x + ev,
// while l += 2^(x - mx) with mx that of x.  (One maximum would not do: a token with a large V
// scale and no weight would push the others' weights out of fp16's range.)  The weights are
// rounded to fp16, 2^7 times larger than 1 at the maximum, which may be stale by up to 2^8: at
// most 2^15.  Below 2^-14, which is 2^-21 of the row's largest product of weight and scale, they lose
// bits: an error of 2^-32 of that product a unit of code.  It is nothing next to the row's largest
// term, but shows in a column where the tokens of large scale are 0.  O and l are fp32.
#include <math.h>
#include <type_traits>

#include "internal.h"
#include "prefill_common.cuh"
#include "tree.cuh"

namespace fa {
namespace {

constexpr int kMaxRows = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kShift = 7.f;       // weights times 2^7
constexpr float kStale = 8.f;       // O is rescaled when a maximum grows by more than 2^8
constexpr float kUnset = -3e38f;    // a maximum before the first score
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, int NT>
struct RowsLayout {
  static constexpr int kRows = 8 * NT;
  // Tokens a step, CTAs an SM and stages: what fits registers and shared memory, measured.  One
  // tile at D = 128 with slices of 32, three CTAs and two stages: 122 us where these take 110; two
  // tiles with slices of 16 and four stages: 155 for 148 (sequences of 1K to 4K tokens).  D = 64
  // with slices of 16: 150 us for 118; D = 256 with three CTAs of two stages: 115 for 113.
  static constexpr int kSlice = D == 256 || (D == 128 && NT == 1) ? 16 : 32;
  static constexpr int kStage = kSlice * D;          // bytes of K (or V) a slice
  static constexpr int kCtas = D == 256 ? 2 : NT == 1 ? 4 : 3;
  static constexpr int kStages = D == 256 || NT == 1 ? 3 : D == 64 ? 4 : 2;
  static constexpr int kRing = kStages * 2 * kStage;  // a warp's ring
  static constexpr int kQOff = kWarps * kRing;
  static constexpr int kQBytes = (D / 16) * NT * 256;  // fp16 fragments of q
  static constexpr int kBarOff = kQOff + kQBytes;
  static constexpr int kStatOff = kBarOff + kWarps * kStages * 2 * 8;
  static constexpr int kPoisonOff = kStatOff + kWarps * kRows * 3 * 4;
  static constexpr int kBytes = kPoisonOff + kMaxTree / 32 * 4 + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kRows * D * 4 <= kRing, "a warp's O goes into its ring at the end");
  static_assert(kCtas * (kAlloc + 1024) <= 228 * 1024, "shared memory of an SM");
};

// C (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).  With g = lane / 4, t = lane % 4:
// a0 (row g, k 2t..), a1 (g + 8, 2t..), a2 (g, 2t + 8..), a3 (g + 8, 2t + 8..); b0 (k 2t.., column
// g), b1 (k 2t + 8..); c0, c1 (row g, columns 2t, 2t + 1), c2, c3 (row g + 8).
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint2 b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// An 8x8 matrix of 16-bit elements, transposed (lane: row g, elements 2t, 2t + 1, in and out).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four 8x8 matrices of 16-bit units, transposed: register i of lane l holds units (row 2t, row
// 2t + 1) of column g of matrix i.  Here a unit is two neighbouring codes of one token.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Four elements of q in fp32.
template <bool BF16>
__device__ __forceinline__ void load_q4(const void* q, int64_t at, float (&x)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at);
  if constexpr (BF16) {
    unpack2<__nv_bfloat16>(w.x, x[0], x[1]);
    unpack2<__nv_bfloat16>(w.y, x[2], x[3]);
  } else {
    unpack2<__half>(w.x, x[0], x[1]);
    unpack2<__half>(w.y, x[2], x[3]);
  }
}

// NT tiles of eight rows.
template <int D, int NT, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, RowsLayout<D, NT>::kCtas)
    tree_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const TreeParams p) {
  using L = RowsLayout<D, NT>;
  constexpr int SL = L::kSlice, NS = L::kStages;
  constexpr int kSteps = D / 16;      // k steps of S, and 16-column chunks of V
  constexpr int kGroups = SL / 8;     // 8-token groups of S
  constexpr int kIn = D < 128 ? D : 128;
  constexpr int kLaneBytes = kIn / 4;  // bytes of a token's block that a lane of four holds
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_addr(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t4 = lane % 4;
  uint32_t* poison = reinterpret_cast<uint32_t*>(smem + L::kPoisonOff);
  uint32_t& failed = poison[kMaxTree / 32];

  // ---- work item: part x kv head x sequence, longest sequences first ----
  const int split = blockIdx.x % p.n_splits;
  const int hk = blockIdx.y;
  const int b = sequence_of_rank<kThreads>(p, blockIdx.z);
  int Lkv = p.kv_lens[b];
  int n_draft = p.draft_lens ? p.draft_lens[b] : p.T;
  if (Lkv < 0 || static_cast<int64_t>(Lkv) > static_cast<int64_t>(p.max_pages) * p.page_size ||
      n_draft < 0 || n_draft > p.T || n_draft > Lkv) {
    // an empty sequence without draft_lens is no error: its rows are empty
    if (threadIdx.x == 0 && !(Lkv == 0 && !p.draft_lens)) record_error(p.status, kDevBounds);
    Lkv = 0;
    n_draft = 0;
  }
  const int ctx = Lkv - n_draft;
  if (p.mask && n_draft > 0) {
    const uint64_t* words = p.mask + static_cast<int64_t>(p.mask_batches == 1 ? 0 : b) * p.T * p.words;
    for (int i = threadIdx.x * 16; i < p.T * p.words; i += kThreads * 16) prefetch_l1(words + i);
  }
  const int n_slices = n_draft > 0 ? (Lkv + SL - 1) / SL : 0;
  const int per_split = (n_slices + p.n_splits - 1) / p.n_splits;
  const int s_begin = min(n_slices, split * per_split) + warp;
  const int s_end = min(n_slices, (split + 1) * per_split);
  const int n = s_begin < s_end ? (s_end - s_begin + kWarps - 1) / kWarps : 0;  // this warp's slices

  const uint32_t ring = s_base + warp * L::kRing;
  const uint32_t bars = s_base + L::kBarOff + warp * NS * 16;
  auto bar_k = [&](int s) { return bars + 16u * s; };
  auto bar_v = [&](int s) { return bars + 16u * s + 8u; };
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_k(s), 1);
      mbar_init(bar_v(s), 1);
    }
    fence_barrier_init();
  }
  if (threadIdx.x <= kMaxTree / 32) poison[threadIdx.x] = 0;
  __syncwarp();

  // ---- copies: lane i of a slice stands for token i; the lane of a box's first token issues it
  const int box = min(p.page_size, SL), box_shift = 31 - __clz(box);
  const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  // Page id of token `lane` of this warp's slice k (0 past the end), as the table has it; checked
  // where it is first used, so that nothing waits for the load.
  auto token_page = [&](int k) {
    if (lane >= SL || k >= n) return 0;  // (a slice past the last one may pass 2^31)
    const int key = (s_begin + k * kWarps) * SL + lane;
    return key < Lkv ? __ldg(table + (key >> p.page_shift)) : 0;
  };
  auto checked = [&](int id) {
    if (id >= 0 && id < p.num_pages) return id;
    record_error(p.status, kDevBounds);
    return 0;
  };
  auto token_row = [&](int k, int id) {
    const int key = (s_begin + k * kWarps) * SL + lane;
    return (static_cast<int64_t>(id) * p.Hkv + hk) * p.page_size + (key & (p.page_size - 1));
  };
  auto copy = [&](const CUtensorMap* map, uint32_t dst, uint32_t bar, int k, int id) {
    if (lane == 0) mbar_arrive_expect_tx(bar, L::kStage);
    __syncwarp();
    if (lane < SL && (lane & (box - 1)) == 0) {
      const int key = (s_begin + k * kWarps) * SL + lane;
      tma_load_4d(dst + lane * D, map, bar, 0, key & (p.page_size - 1), 0, id * p.Hkv + hk);
    }
  };
  auto k_stage = [&](int s) { return ring + s * 2 * L::kStage; };
  auto v_stage = [&](int s) { return ring + (s * 2 + 1) * L::kStage; };
  int ids[NS + 1];
#pragma unroll
  for (int k = 0; k <= NS; ++k) ids[k] = token_page(k);
#pragma unroll
  for (int k = 0; k < NS; ++k) ids[k] = checked(ids[k]);
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    if (k >= n) break;
    copy(&tm_k, k_stage(k), bar_k(k), k, ids[k]);
    copy(&tm_v, v_stage(k), bar_v(k), k, ids[k]);
  }

  // ---- q: rows r = head * T + query, scaled and laid out as the fragments of its k steps ----
  // A lane of four holds columns [kLaneBytes t, kLaneBytes (t + 1)) of each 128-column block of a
  // token; k step kk takes four of them, in both operands (the order of k does not matter).
  const int rows = p.G * p.T;
  __shared__ float q_scale[L::kRows];  // scale_log2 times the row's power of two
  for (int r = warp * 4 + lane / 8; r < L::kRows; r += kWarps * 4) {
    // eight lanes a row: lane c takes columns 4c, 4c + 32, ...
    const int c = lane % 8;
    const bool have = r < rows && r % p.T < n_draft;  // padding rows: 0, whatever q has there
    const int head = hk * p.G + (have ? r / p.T : 0), i = have ? r % p.T : 0;
    const int64_t at = b * p.q_strides[0] + head * p.q_strides[1] + i * p.q_strides[2];
    float x[D / 32][4];
    float amax = 0.f;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
      if (have) load_q4<BF16>(p.q, at + 4 * c + 32 * u, x[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(x[u][e]));
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // 2^-eq with amax 2^-eq in [2^14, 2^15) (1 for a row of zeros)
    const int eq = amax > 0.f ? max(-112, static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14) : 0;
    const float f = __uint_as_float(static_cast<uint32_t>(127 - eq) << 23);
    if (c == 0) q_scale[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + eq) << 23);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int col = 4 * c + 32 * u, blk = col / kIn, in = col % kIn;
      const int t = in / kLaneBytes, kk = blk * (kIn / 16) + (in % kLaneBytes) / 4;
      // fragment of lane (r % 8) * 4 + t
      const int frag = kk * NT + r / 8;  // two to a 16-byte read
      uint32_t* dst = reinterpret_cast<uint32_t*>(smem + L::kQOff + frag / 2 * 512 +
                                                  ((r % 8) * 4 + t) * 16 + frag % 2 * 8);
      dst[0] = pack_f16x2(x[u][0] * f, x[u][1] * f);
      dst[1] = pack_f16x2(x[u][2] * f, x[u][3] * f);
    }
  }
  __syncthreads();

  // ---- this lane's rows: 8m + 2t and 8m + 2t + 1 of each tile m, a pair in every float2 ----
  float2 mx[NT], mo[NT], l[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    mx[m] = mo[m] = make_float2(kUnset, kUnset);
    l[m] = make_float2(0.f, 0.f);
  }
  // drafted tokens of the 32 from key0 on that row r sees
  auto seen = [&](int r, int off) {
    const int i = r < rows ? r % p.T : 0;
    TreeRow row;
    row.i = i;
    row.n = r < rows && i < n_draft ? n_draft : 0;
    row.words = p.mask && row.n
        ? p.mask + (static_cast<int64_t>(p.mask_batches == 1 ? 0 : b) * p.T + i) * p.words : nullptr;
    return row_bits(row, off);
  };
  float o[NT][kSteps][4];  // columns 16c + 2g (elements 0, 1: the two rows) and 16c + 2g + 1 (2, 3)
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[m][c][e] = 0.f;

  // shared-memory offsets inside a stage (a box holds [128-column block][token][128 bytes], 16-byte
  // chunks swizzled by the token)
  auto token_off = [&](int tok) {
    return static_cast<uint32_t>(((tok >> box_shift) << box_shift) * D + (tok & (box - 1)) * kIn);
  };
  const uint32_t blk_off = box * kIn;
  const uint32_t k_swz = D < 128 ? (g >> 1) & 3 : g;           // of tokens 8j + g
  const int v_tok = lane & 15;                                 // ldmatrix: this lane's row
  const uint32_t v_swz = D < 128 ? (v_tok >> 1) & 3 : v_tok & 7;

  // ---- one slice ----
  // scales: of token `lane`, 2^ek in bf16 above ev in bf16 (both exact)
  auto slice = [&](auto tail_c, int k, uint32_t scales, int next_id) -> bool {
    constexpr bool TAIL = decltype(tail_c)::value;
    const int st = k % NS, key0 = (s_begin + k * kWarps) * SL;
    if (!__all_sync(0xffffffffu, mbar_wait(bar_k(st), (k / NS) & 1, p.status))) return false;
    // S^T = K Q^T, a 128-column block at a time: s[.][i] are tokens 8i + g
    float2 s[NT][kGroups];
    float acc[NT][kGroups / 2][4];
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int j = 0; j < kGroups / 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
#pragma unroll
    for (int blk = 0; blk < D / kIn; ++blk) {
      uint32_t w[kGroups][kIn / 16];
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const uint32_t at = k_stage(st) + token_off(8 * j + g) + blk * blk_off;
#pragma unroll
        for (int u = 0; u < kLaneBytes / 16; ++u) {
          const uint4 v = lds128(at + (((t4 * (kLaneBytes / 16) + u) ^ k_swz) * 16));
          w[j][4 * u] = v.x;
          w[j][4 * u + 1] = v.y;
          w[j][4 * u + 2] = v.z;
          w[j][4 * u + 3] = v.w;
        }
      }
      if (blk == D / kIn - 1) {
        __syncwarp();  // every lane has read the stage
        if (k + NS < n) copy(&tm_k, k_stage(st), bar_k(st), k + NS, next_id);
      }
      uint4 qf;
#pragma unroll
      for (int kk = 0; kk < kIn / 16; ++kk) {
        const int frag = (blk * (kIn / 16) + kk) * NT;
        if (frag % 2 == 0) qf = lds128(s_base + L::kQOff + frag / 2 * 512 + lane * 16);
#pragma unroll
        for (int j = 0; j < kGroups / 2; ++j) {
          const uint32_t a0 = widen2(w[2 * j][kk]), a2 = widen2_hi(w[2 * j][kk]);
          const uint32_t a1 = widen2(w[2 * j + 1][kk]), a3 = widen2_hi(w[2 * j + 1][kk]);
#pragma unroll
          for (int m = 0; m < NT; ++m)
            mma16816(acc[m][j], a0, a1, a2, a3,
                     (frag + m) % 2 ? make_uint2(qf.z, qf.w) : make_uint2(qf.x, qf.y));
        }
      }
    }
    // the scales of this lane's tokens: 2^ek as it multiplies, ev as it is added
    float kf[kGroups], ev[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const uint32_t w = __shfl_sync(0xffffffffu, scales, 8 * i + g);
      kf[i] = __uint_as_float(w & 0xffff0000u);
      ev[i] = __uint_as_float(w << 16);
    }
    // scores in log2 units; hidden tokens get -inf
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const float2 a = make_float2(q_scale[8 * m + 2 * t4], q_scale[8 * m + 2 * t4 + 1]);
      uint32_t b0 = ~0u, b1 = ~0u;
      if constexpr (TAIL) {
        b0 = seen(8 * m + 2 * t4, key0 - ctx) >> g;
        b1 = seen(8 * m + 2 * t4 + 1, key0 - ctx) >> g;
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        float2 x = make_float2(acc[m][i / 2][2 * (i & 1)], acc[m][i / 2][2 * (i & 1) + 1]);
        x = __fmul2_rn(__fmul2_rn(x, a), make_float2(kf[i], kf[i]));
        if (TAIL && !((b0 >> (8 * i)) & 1)) x.x = -INFINITY;
        if (TAIL && !((b1 >> (8 * i)) & 1)) x.y = -INFINITY;
        s[m][i] = x;
      }
    }
    // exponents of the sums' terms (y1 = x - mx) and of the weights (y2 = x + ev - mo + kShift)
    float2 y1[NT][kGroups], y2[NT][kGroups];
    auto exponents = [&]() {
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const float2 down = make_float2(-mx[m].x, -mx[m].y);
        const float2 up = make_float2(kShift - mo[m].x, kShift - mo[m].y);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          y1[m][i] = __fadd2_rn(s[m][i], down);
          y2[m][i] = __fadd2_rn(s[m][i], __fadd2_rn(make_float2(ev[i], ev[i]), up));
        }
      }
    };
    exponents();
    // how far the scores are above the running maxima; mostly not far enough to move them
    float over1 = -INFINITY, over2 = -INFINITY;
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        over1 = prefill::fmax3(over1, y1[m][i].x, y1[m][i].y);
        over2 = prefill::fmax3(over2, y2[m][i].x, y2[m][i].y);
      }
    if (__any_sync(0xffffffffu, over1 > kStale || over2 > kStale + kShift)) {
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        float2 x1 = mx[m], x2 = mo[m];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          x1.x = fmaxf(x1.x, s[m][i].x);
          x1.y = fmaxf(x1.y, s[m][i].y);
          x2.x = fmaxf(x2.x, s[m][i].x + ev[i]);
          x2.y = fmaxf(x2.y, s[m][i].y + ev[i]);
        }
#pragma unroll
        for (int d = 4; d <= 16; d *= 2) {
          x1.x = fmaxf(x1.x, __shfl_xor_sync(0xffffffffu, x1.x, d));
          x1.y = fmaxf(x1.y, __shfl_xor_sync(0xffffffffu, x1.y, d));
          x2.x = fmaxf(x2.x, __shfl_xor_sync(0xffffffffu, x2.x, d));
          x2.y = fmaxf(x2.y, __shfl_xor_sync(0xffffffffu, x2.y, d));
        }
        l[m].x *= exp2_approx(mx[m].x - x1.x);
        l[m].y *= exp2_approx(mx[m].y - x1.y);
        const float2 alpha = make_float2(exp2_approx(mo[m].x - x2.x), exp2_approx(mo[m].y - x2.y));
        mx[m] = x1;
        mo[m] = x2;
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          o[m][c][0] *= alpha.x;
          o[m][c][1] *= alpha.y;
          o[m][c][2] *= alpha.x;
          o[m][c][3] *= alpha.y;
        }
      }
      exponents();
    }
    // weights: (token, two rows) turned to (row, two tokens), the MMA's B
    uint32_t pk[NT][kGroups];
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float2 e1 = y1[m][i], e2 = y2[m][i];
        l[m] = __fadd2_rn(l[m], make_float2(exp2_approx(e1.x), exp2_approx(e1.y)));
        pk[m][i] = transpose8x8(pack_f16x2(exp2_approx(e2.x), exp2_approx(e2.y)));
      }
    // O^T += V^T P^T: 16 tokens x 32 columns of V codes a load, transposed so that a register holds
    // two neighbouring columns of two tokens; regrouped by column they are the pairs the MMA wants.
    // Of a 16-column chunk, the A rows 0-7 are the even columns and 8-15 the odd ones.
    if (!__all_sync(0xffffffffu, mbar_wait(bar_v(st), (k / NS) & 1, p.status))) return false;
#pragma unroll
    for (int kt = 0; kt < SL / 16; ++kt) {
      const uint32_t at = v_stage(st) + token_off(16 * kt + v_tok);
#pragma unroll
      for (int c = 0; c < kSteps; c += 2) {
        const int blk = c / (kIn / 16), ci = c % (kIn / 16) + (lane >> 4);
        uint32_t r[4];
        ldmatrix4_trans(at + blk * blk_off + ((ci ^ v_swz) * 16), r);
        if constexpr (TAIL) {
          // codes past the sequence's end, and NaN of drafted tokens (noted for the epilogue):
          // 0, which a weight of 0 does not turn into NaN
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + 16 * kt + 8 * (x & 1) + 2 * t4 + e;
              if (key >= Lkv) {
                r[x] &= e ? 0x0000ffffu : 0xffff0000u;
              } else if (key >= ctx) {
#pragma unroll
                for (int by = 2 * e; by < 2 * e + 2; ++by) {
                  if (((r[x] >> (8 * by)) & 0x7fu) == 0x7fu) {
                    r[x] &= ~(0xffu << (8 * by));
                    atomicOr(&poison[(key - ctx) >> 5], 1u << ((key - ctx) & 31));
                  }
                }
              }
            }
          }
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const uint32_t u0 = __byte_perm(r[2 * cc], 0, 0x3120), u1 = __byte_perm(r[2 * cc + 1], 0, 0x3120);
          const uint32_t e0 = widen2(u0), e1 = widen2(u1), d0 = widen2_hi(u0), d1 = widen2_hi(u1);
#pragma unroll
          for (int m = 0; m < NT; ++m)
            mma16816(o[m][c + cc], e0, d0, e1, d1, make_uint2(pk[m][2 * kt], pk[m][2 * kt + 1]));
        }
      }
    }
    __syncwarp();
    if (k + NS < n) copy(&tm_v, v_stage(st), bar_v(st), k + NS, next_id);
    return true;
  };

  // ---- the loop: page ids are loaded a slice before their copies are issued, scale bytes a
  // slice before they are used ----
  auto load_bytes = [&](int k, int id, uint32_t& kb, uint32_t& vb) {
    if (k >= n || lane >= SL || (s_begin + k * kWarps) * SL + lane >= Lkv) return;
    const int64_t at = token_row(k, id);
    kb = __ldg(p.k_scales + at);
    vb = __ldg(p.v_scales + at);
  };
  int k = 0;
  bool ok = true;
  uint32_t kb = 127, vb = 127;
  load_bytes(0, ids[0], kb, vb);
  for (; ok && k < n; ++k) {
    // ids[j] is slice k + j's here, the last one not yet checked
    const float ev = static_cast<float>(static_cast<int>(vb) - 127);
    const uint32_t scales = (kb << 23) | (__float_as_uint(ev) >> 16);
    load_bytes(k + 1, ids[1], kb, vb);
    const int next_id = checked(ids[NS]);
#pragma unroll
    for (int j = 0; j < NS - 1; ++j) ids[j] = ids[j + 1];
    ids[NS - 1] = next_id;
    ids[NS] = token_page(k + NS + 1);
    if ((s_begin + k * kWarps) * SL + SL > ctx) ok = slice(std::true_type{}, k, scales, next_id);
    else ok = slice(std::false_type{}, k, scales, next_id);
  }
  if (!ok) {
    // a wait ran out: let the copies in flight land (each stage's last one) before the CTA ends
    if (lane == 0) {
      failed = 1;
      for (int j = max(0, k - 1); j < min(n, k - 1 + NS); ++j) {
        mbar_wait(bar_k(j % NS), (j / NS) & 1, nullptr);
        mbar_wait(bar_v(j % NS), (j / NS) & 1, nullptr);
      }
      // the slice that failed may have sent its next K already
      if (k - 1 + NS < n) mbar_wait(bar_k((k - 1) % NS), ((k - 1 + NS) / NS) & 1, nullptr);
    }
    __syncwarp();
  }

  // ---- combine the warps: O / l over the largest maxima ----
  float* stat = reinterpret_cast<float*>(smem + L::kStatOff);  // [warp][row][mx, mo, l]
  float* part = reinterpret_cast<float*>(smem + warp * L::kRing);
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = h ? l[m].y : l[m].x;
#pragma unroll
      for (int d = 4; d <= 16; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int r = 8 * m + 2 * t4 + h;
      if (g == 0) {
        float* at = stat + (warp * L::kRows + r) * 3;
        at[0] = h ? mx[m].y : mx[m].x;
        at[1] = h ? mo[m].y : mo[m].x;
        at[2] = sum;
      }
      // columns 16c + 2g, + 1 of row r, chunks of four swizzled by the row
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
        *reinterpret_cast<float2*>(part + r * D + ((4 * c + g / 2) ^ (r & 7)) * 4 + (g & 1) * 2) =
            make_float2(o[m][c][h], o[m][c][2 + h]);
    }
  __syncthreads();
  if (failed) return;
  bool any_poison = false;
  for (int w = 0; w < kMaxTree / 32; ++w) any_poison |= poison[w] != 0;
  constexpr int kVec = D / 4;
  for (int u = threadIdx.x; u < rows * kVec; u += kThreads) {
    const int r = u / kVec, v = u % kVec;
    float M = kUnset, Mo = kUnset;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* at = stat + (w * L::kRows + r) * 3;
      M = fmaxf(M, at[0]);
      Mo = fmaxf(Mo, at[1]);
    }
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* at = stat + (w * L::kRows + r) * 3;
      const float fo = exp2_approx(at[1] - Mo);
      sum += at[2] * exp2_approx(at[0] - M);
      const float4 x = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + w * L::kRing) + r * D + ((v ^ (r & 7)) * 4));
      acc.x = fmaf(fo, x.x, acc.x);
      acc.y = fmaf(fo, x.y, acc.y);
      acc.z = fmaf(fo, x.z, acc.z);
      acc.w = fmaf(fo, x.w, acc.w);
    }
    const int head = hk * p.G + r / p.T, i = r % p.T;
    const bool have = i < n_draft && !(sum == 0.f);  // a NaN sum stays NaN
    if (any_poison && i < n_draft) {
      TreeRow row;
      row.i = i;
      row.n = n_draft;
      row.words = p.mask ? p.mask + (static_cast<int64_t>(p.mask_batches == 1 ? 0 : b) * p.T + i) * p.words : nullptr;
      for (int d = 0; d < n_draft; ++d) {
        if (!((poison[d >> 5] >> (d & 31)) & 1) || !row_sees(row, d)) continue;
        acc.x += nonfinite_v<D, BF16, true>(p, b, hk, ctx + d, 4 * v);
        acc.y += nonfinite_v<D, BF16, true>(p, b, hk, ctx + d, 4 * v + 1);
        acc.z += nonfinite_v<D, BF16, true>(p, b, hk, ctx + d, 4 * v + 2);
        acc.w += nonfinite_v<D, BF16, true>(p, b, hk, ctx + d, 4 * v + 3);
      }
    }
    const float inv = 1.f / sum, f = exp2f(Mo - M - kShift);
    if (have) {
      acc.x = acc.x * inv * f;
      acc.y = acc.y * inv * f;
      acc.z = acc.z * inv * f;
      acc.w = acc.w * inv * f;
    } else {
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float lse = have ? (M + log2f(sum)) * kLn2 : -INFINITY;
    const int64_t flat = (static_cast<int64_t>(b) * p.Hq + head) * p.T + i;
    if constexpr (SPLIT) {
      const int64_t at = flat * p.n_splits + split;
      *reinterpret_cast<float4*>(p.o_part + at * D + 4 * v) = acc;
      // the merge takes a part of weight +inf as not a number, which a NaN part would not be
      if (v == 0) p.lse_part[at] = lse != lse ? INFINITY : lse;
    } else {
      const uint2 w = BF16 ? make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w))
                           : make_uint2(pack_f16x2(acc.x, acc.y), pack_f16x2(acc.z, acc.w));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + flat * D + 4 * v) = w;
      if (v == 0 && p.lse) p.lse[flat] = lse;
    }
  }
}

template <int D, int NT, bool BF16>
cudaError_t launch_impl(const TreeParams& p, cudaStream_t st) {
  using L = RowsLayout<D, NT>;
  CUtensorMap tk, tv;
  const uint64_t ps = static_cast<uint64_t>(p.page_size), pages = static_cast<uint64_t>(p.num_pages) * p.Hkv;
  // a page of one head: page_size rows of D bytes as (column, row, block of 128 columns)
  constexpr uint64_t in = D < 128 ? D : 128;
  const uint64_t dims[4] = {in, ps, D / in, pages}, str[3] = {D, in, ps * D};
  const uint32_t rows = p.page_size < L::kSlice ? p.page_size : L::kSlice;
  const uint32_t box[4] = {static_cast<uint32_t>(in), rows, static_cast<uint32_t>(D / in), 1};
  const CUtensorMapSwizzle swz = D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_tiled(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.k_pages, dims, str, box, swz) ||
      !encode_tiled(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.v_pages, dims, str, box, swz))
    return cudaErrorInvalidValue;
  auto kern = p.n_splits > 1 ? tree_rows_kernel<D, NT, BF16, true> : tree_rows_kernel<D, NT, BF16, false>;
  cudaError_t e = ensure_smem_limit(kern, L::kAlloc);
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.n_splits, p.Hkv, p.B), kThreads, L::kAlloc, st>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int NT, bool BF16>
cudaError_t launch_d(const TreeParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_impl<64, NT, BF16>(p, st);
    case 128: return launch_impl<128, NT, BF16>(p, st);
    default: return launch_impl<256, NT, BF16>(p, st);
  }
}

}  // namespace

// At most two tiles.  With four (17 to 32 rows, D = 128) a warp's registers spill and the loop is
// bound by its arithmetic: 38 sequences of 4096 tokens take 105 to 137 us, the 128-row kernel 100 us.
bool tree_rows_takes(int rows) { return rows <= kMaxRows; }

int tree_rows_ctas(int D, int rows) {
  const bool one = rows <= 8;
  switch (D) {
    case 64: return one ? RowsLayout<64, 1>::kCtas : RowsLayout<64, 2>::kCtas;
    case 128: return one ? RowsLayout<128, 1>::kCtas : RowsLayout<128, 2>::kCtas;
    default: return one ? RowsLayout<256, 1>::kCtas : RowsLayout<256, 2>::kCtas;
  }
}

cudaError_t launch_tree_rows(const TreeParams& p, int D, bool bf16, cudaStream_t stream) {
  if (p.G * p.T <= 8) return bf16 ? launch_d<1, true>(p, D, stream) : launch_d<1, false>(p, D, stream);
  return bf16 ? launch_d<2, true>(p, D, stream) : launch_d<2, false>(p, D, stream);
}

}  // namespace fa
