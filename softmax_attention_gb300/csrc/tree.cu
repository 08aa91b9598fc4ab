// tree.cu -- attention of a tree of drafted tokens over a paged cache, 16-bit or 8-bit, on the
// tensor cores (one drafted token: decode over an 8-bit cache).
//
// Query i of a sequence sees every token of the context (all but the sequence's last n drafted
// tokens) and the drafted tokens that bit j of its mask row names:
//   s_j = scale <q_i, k_j>,  out_i = sum_j softmax(s)_j v_j over the seen j.
// The mask touches only the KV tiles that overlap the last n tokens; every other tile runs the
// unmasked softmax.
//
// One CTA takes one 128-row tile of packed (query head, query) rows of one kv head against one
// range of KV tiles, as the paged prefill kernel does, and the two issuing threads, the three
// S/P buffers in tensor memory and the lazy rescale are the same protocol.  What differs is
// where a K or V stage comes from.  16-bit pages: TMA boxes straight into the stage.  8-bit
// pages: TMA boxes of e4m3 rows into a raw ring, from which a warpgroup of converters writes
// the 16-bit stage, one row a thread: each row's scale is a power of two, so value * 2^e is
// exact in bf16 and the product with Q is the same as on the widened cache.  Converting on
// the way costs shared-memory bandwidth (a row is written twice and read twice) but keeps the
// 16-bit queries and weights whole, which 8-bit MMAs would not.
//
// fp16 operands for bf16 queries.  e4m3 converts to fp16 in one instruction a pair, to bf16 only
// by placing bits (five, and a test for NaN codes); at 64 drafted tokens the conversion's
// instructions are what bounds the kernel.  So a CTA looks at the scale bytes of its keys
// first: if all lie in [113, 134], every value * 2^e is exact in fp16 too, the rows of Q are
// scaled by powers of two into fp16 (exact down to 2^-31 of a row's maximum, undone in the
// scores), and both products run in fp16.  Otherwise they run in bf16, which holds any scale.
//
// Values beyond the operand type.  fp16 queries meet K and V at half their size (undone in the
// scores and in the sum that O is divided by): all that fp16 rows are ever stored as, up to 65536 =
// 256 * 2^8, then fits, and a row of scale 2^-14 or more is exact.  What does not fit (fp16 from
// scale byte 136 on, bf16 at 2^128) is held at the operand's largest value, never as an infinity,
// which a weight of 0 would turn into NaN in rows that do not see the token.
//
// Measured (D = 128, 8 kv heads of four query heads, even sequences of 8192 tokens, 16-token
// pages): 16-bit cache, 32 drafted tokens of 19 sequences 103 us, 6.2 TB/s, bound by memory; 64 of
// them, two tiles a sequence, 144 us.  8-bit cache 95 and 180 us: a KV tile takes some 2450 clocks
// of converters (730 for K, 780 for V and the waits between) and softmax warps (2000 of them) side
// by side at half of the issue slots.  One row of each sequence with a scale byte outside [113, 134]
// moves its blocks to bf16 operands: 1.5 times as long (replayed twenty a graph, 88 -> 131 and 173
// -> 260 us; D = 64 238 -> 281, D = 256 190 -> 249).  fp16 queries: 83 and 163 us, 91 and 179 with
// one row a sequence that can overflow.
//
// Warp roles: 0-3 and the last four softmax + epilogue (a row of scores is shared by two
// threads), 4 TMA producer, 5 P V issuer and tensor-memory owner, 6 S issuer, and for 8-bit pages 7
// second TMA producer, 8-11 converters.
#include <float.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <type_traits>

#include "../../include/fa.h"
#include "cache.cuh"
#include "internal.h"
#include "prefill_common.cuh"
#include "sm103.cuh"
#include "tree.cuh"

namespace fa {
namespace {

using prefill::kRows;
constexpr int kNumS = 3;  // S/P buffers in tensor memory

// 5-D tiled TMA load (a 16-bit page).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3,
                                            int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
      "r"(bar)
      : "memory");
}

template <int D, int BN, int STAGES, int RAW, bool Q8>
struct Layout {
  static constexpr int kHalves = 2;                    // softmax warps a row of scores
  static constexpr int kConvertWarp = 8;               // first converter
  static constexpr int kHalfWarp = Q8 ? 12 : 8;        // first softmax warp of the second halves
  static constexpr int kThreads = (kHalfWarp + 4) * 32;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kKVBytes = BN * D * 2;   // one 16-bit K (or V) stage
  static constexpr int kRawBytes = BN * D;      // one 8-bit K (or V) stage
  static constexpr int kKOff = kQBytes;
  static constexpr int kVOff = kKOff + STAGES * kKVBytes;
  static constexpr int kRawKOff = kVOff + STAGES * kKVBytes;
  static constexpr int kRawVOff = kRawKOff + (Q8 ? RAW * kRawBytes : 0);
  static constexpr int kBarOff = kRawVOff + (Q8 ? RAW * kRawBytes : 0);
  // q_full, {k,v}_full[S], {k,v}_empty[S], s_full[3], p_full[3], pv_done[3], pv_issuer_done,
  // s_issuer_done, raw {k,v}_full[R], raw {k,v}_empty[R], q_ready
  static constexpr int kNumBars = 1 + 4 * STAGES + 3 * kNumS + 2 + (Q8 ? 4 * RAW + 1 : 0);
  static constexpr int kPoisonOff = kBarOff + kNumBars * 8 + 16;
  // what two halves of a row exchange (a maximum or a sum each), and the power of two of the row of Q
  static constexpr int kRowOff = kPoisonOff + (kMaxTree / 32) * 4;
  static constexpr int kBytes = kRowOff + 3 * kRows * 4;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base to 1024 bytes
  static_assert(D + kNumS * BN <= 512, "tensor memory budget (O and the S/P buffers)");
  static_assert(kAlloc <= 232448, "shared memory budget");
};

// ------------------------------------------------------------------------------------------
// One KV tile of the online softmax for one row, in the steps of prefill::softmax_tile but with
// a bit mask in place of the key limit and the additive mask.  raw: scores of a run of keys,
// hidden ones -inf.  a: the factor into log2 units (positive).
//
// fp16 weights are held 2^7 times larger, as are their sums: the stale maximum lets a weight grow
// to 2^8, so they still fit (2^15), and the small ones, whose rounding is absolute below 2^-14,
// keep seven more bits.
// ------------------------------------------------------------------------------------------
constexpr float kWeightLog2F16 = 7.f;

// The largest of CH scores.
template <int CH>
__device__ __forceinline__ float chunk_max(const uint32_t (&raw)[CH]) {
  float mx[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    mx[e] = prefill::fmax3(__uint_as_float(raw[e]), __uint_as_float(raw[e + 8]), -INFINITY);
#pragma unroll
  for (int c = 16; c < CH; c += 16) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      mx[e] = prefill::fmax3(mx[e], __uint_as_float(raw[c + e]), __uint_as_float(raw[c + 8 + e]));
  }
  return prefill::fmax3(prefill::fmax3(mx[0], mx[1], mx[2]), prefill::fmax3(mx[3], mx[4], mx[5]),
                        fmaxf(mx[6], mx[7]));
}

// Whether `x` holds for any thread of the named barrier's `threads`; all of them must call.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(id), "r"(threads), "r"(x ? 1u : 0u) : "memory");
  return r != 0;
}
__device__ __forceinline__ void barrier_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Weights of CH scores against the maximum m: packed pairs, and their sum added to l.
template <int CH, bool BF16>
__device__ __forceinline__ void chunk_weights(const uint32_t (&raw)[CH], float a, float m, float& l,
                                              uint32_t (&pk)[CH / 2]) {
  const float m_use = (m == -INFINITY) ? 0.f : m - (BF16 ? 0.f : kWeightLog2F16);
  const float2 a2 = make_float2(a, a), nm2 = make_float2(-m_use, -m_use);
  float2 sum2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum2[e] = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < CH / 2; ++c) {
    const float2 t = __ffma2_rn(
        make_float2(__uint_as_float(raw[2 * c]), __uint_as_float(raw[2 * c + 1])), a2, nm2);
    const float p0 = exp2_approx(t.x);
    const float p1 = exp2_approx(t.y);
    sum2[c & 3] = __fadd2_rn(sum2[c & 3], make_float2(p0, p1));
    pk[c] = BF16 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
  }
  const float2 s01 = __fadd2_rn(sum2[0], sum2[1]), s23 = __fadd2_rn(sum2[2], sum2[3]);
  l += (s01.x + s01.y) + (s23.x + s23.y);
}

// ------------------------------------------------------------------------------------------
// e4m3 -> 16 bits with the row's scale.  bf16: the byte's exponent and mantissa placed in a
// bf16 are the value times 2^-120 (subnormals included), so one product with 2^(120 + e) is
// the exact result; exponents above 7 leave bf16's range there and take a second product.  fp16:
// the hardware conversion, then the scale in two products of which only the last can round.
// ------------------------------------------------------------------------------------------
struct RowScale {
  uint32_t f1, f2;  // packed pairs; f2 is used where `two`
  bool two;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool BF16>
__device__ __forceinline__ RowScale row_scale(uint32_t byte) {
  RowScale s;
  const int e = static_cast<int>(byte) - 127;  // [-127, 128], and -128 of fp16 at half size
  if constexpr (BF16) {
    const int e1 = min(e, 7);
    const uint32_t f1 = static_cast<uint32_t>(e1 + 120 + 127) << 7;  // exponent field in [120, 254]
    const int e2 = e - e1;                                           // [0, 121]
    const uint32_t f2 = static_cast<uint32_t>(e2 + 127) << 7;
    s.f1 = f1 | (f1 << 16);
    s.f2 = f2 | (f2 << 16);
    s.two = e2 > 0;
  } else {
    // first factor in [2^-14, 2^15] (exact: an e4m3 value is a multiple of 2^-9), then the rest
    const int e1 = max(-14, min(e, 15));
    const int e2 = max(-24, min(e - e1, 15));
    const uint32_t f1 = static_cast<uint32_t>(e1 + 15) << 10;
    const uint32_t f1n = e1 == -14 ? 0x0400u : f1;
    const uint32_t f2 = e2 >= -14 ? static_cast<uint32_t>(e2 + 15) << 10 : 1u << (e2 + 24);
    s.f1 = f1n | (f1n << 16);
    s.f2 = f2 | (f2 << 16);
    s.two = e != e1;
  }
  return s;
}

// Four e4m3 codes -> two packed pairs, scaled (TWO: by both factors).
template <bool BF16, bool TWO>
__device__ __forceinline__ void widen4(uint32_t w, const RowScale& s, uint32_t& lo, uint32_t& hi) {
  if constexpr (BF16) {
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    lo = mul_bf16x2(((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), s.f1);
    hi = mul_bf16x2(((b >> 4) & 0x07f007f0u) | (b & 0x80008000u), s.f1);
    if constexpr (TWO) {
      lo = mul_bf16x2(lo, s.f2);
      hi = mul_bf16x2(hi, s.f2);
    }
  } else {
    lo = mul_f16x2(widen2(w), s.f1);
    hi = mul_f16x2(widen2_hi(w), s.f1);
    if constexpr (TWO) {
      lo = mul_f16x2(lo, s.f2);
      hi = mul_f16x2(hi, s.f2);
    }
  }
}

// ------------------------------------------------------------------------------------------
// Converters: one warpgroup, thread t taking row t % BN of a tile (for BN = 64 half its columns), K
// then V.  The row's page id is loaded two tiles ahead and its scale bytes one tile ahead;
// each 16-byte chunk of the raw row becomes two of the stage's.  Rows past the sequence's end
// become zeros.
// ------------------------------------------------------------------------------------------
// Whether some scale byte of keys [first, last) lies outside [113, 134], where every e4m3 value
// times the scale is exact in fp16 (a multiple of 2^-23, at most 448 * 2^7).  `first` is a
// multiple of eight.  THREADS threads, this one `looker`, take eight tokens at a time (a page
// holds a multiple of eight).  kBatch page ids, then kBatch scale loads are in flight together
// (the asm statements keep the compiler from joining a load to its use), and the bytes are compared
// four at a time without branches: with a branch a byte the look took 9 us of 8192 keys, so 3.
template <int THREADS>
__device__ __forceinline__ bool scales_leave_fp16(const TreeParams& p, int looker, int b, int hk, int first,
                                                  int last) {
  constexpr int kBatch = 4;
  const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  bool outside = false;
  // unsigned: the last step's keys may pass 2^31
  const uint32_t end = static_cast<uint32_t>(last);
  for (uint32_t key0 = static_cast<uint32_t>(first + looker * 8); key0 < end; key0 += THREADS * 8 * kBatch) {
    int page[kBatch];
    uint2 k[kBatch], v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t key = key0 + u * THREADS * 8;
      page[u] = key < end ? __ldg(table + (key >> p.page_shift)) : -1;
    }
    asm volatile("" : "+r"(page[0]), "+r"(page[1]), "+r"(page[2]), "+r"(page[3]));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t key = key0 + u * THREADS * 8;
      k[u] = v[u] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      const bool take = key < end;
      if (static_cast<uint32_t>(page[u]) >= static_cast<uint32_t>(p.num_pages)) page[u] = 0;  // as it is read
      const int64_t at = ((static_cast<int64_t>(page[u]) * p.Hkv + hk) << p.page_shift) + (key & (p.page_size - 1));
      if (take) k[u] = __ldg(reinterpret_cast<const uint2*>(p.k_scales + at));
      if (take) v[u] = __ldg(reinterpret_cast<const uint2*>(p.v_scales + at));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      asm volatile("" : "+r"(k[u].x), "+r"(k[u].y), "+r"(v[u].x), "+r"(v[u].y));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int left = static_cast<int>(end - (key0 + u * THREADS * 8));  // tokens from this step's first on
      const uint32_t w[4] = {k[u].x, k[u].y, v[u].x, v[u].y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // bytes past the last token become 127; x is outside if x > 134 or x < 113
        const int valid = min(4, max(0, left - 4 * (j & 1)));
        const uint32_t past = valid >= 4 ? 0u : ~0u << (8 * valid);
        const uint32_t x = (w[j] & ~past) | (0x7f7f7f7fu & past);
        outside |= (__vcmpgtu4(x, 0x86868686u) | __vcmpltu4(x, 0x71717171u)) != 0;
      }
    }
  }
  return __any_sync(0xffffffffu, outside);  // and the warp is one again
}

// Row r of the swizzled Q tile (64-column blocks of 128 rows x 128 bytes), bf16 to fp16: times
// 2^-eq such that its largest finite element lies in [2^14, 2^15).  Returns 2^eq.
template <int D>
__device__ __forceinline__ float q_row_to_fp16(uint32_t tile, int r) {
  float amax = 0.f;
#pragma unroll 8
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = lds128(tile + (c / 8) * (kRows * 128) + r * 128 + (((c % 8) ^ (r & 7)) * 16));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      unpack2<__nv_bfloat16>(w[e], lo, hi);
      amax = fmaxf(amax, fmaxf(finite_abs(lo), finite_abs(hi)));
    }
  }
  const int eq = amax > 0.f ? max(-112, static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14) : 0;
  const float f = __uint_as_float(static_cast<uint32_t>(127 - eq) << 23);
#pragma unroll 8
  for (int c = 0; c < D / 8; ++c) {
    const uint32_t at = tile + (c / 8) * (kRows * 128) + r * 128 + (((c % 8) ^ (r & 7)) * 16);
    const uint4 v = lds128(at);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      unpack2<__nv_bfloat16>(w[e], lo, hi);
      w[e] = pack_f16x2(lo * f, hi * f);
    }
    sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
  }
  return __uint_as_float(static_cast<uint32_t>(127 + eq) << 23);
}

// Least scale byte of a row whose widened values can overflow the operand type: 448 times the scale
// is 448 * 2^8 in fp16 (fp16 queries, at half size; for bf16 ones every byte is below), 1.75 * 2^128 in
// bf16.
__device__ __forceinline__ uint32_t overflow_byte(bool f16) { return f16 ? 136 : 247; }

// NaN codes of a raw row (rare): NaN in the stage, or, in a drafted token's V, zero, the token
// noted: a weight of 0 would still carry a NaN into rows that do not see the token.  Where the row
// can have overflowed (`over`), its infinities become the operand type's largest value.
template <int D, int kParts>
__device__ __noinline__ void patch_row(uint32_t raw, uint32_t raw_blk, uint32_t raw_swz, uint32_t dst,
                                       int row, int part, int draft, uint32_t* poison, bool over, bool f16) {
  constexpr int kIn = D < 128 ? D : 128, kChunks = D / 16 / kParts;
  for (int c = part * kChunks; c < (part + 1) * kChunks; ++c) {
    const int blk = c / (kIn / 16), ci = c % (kIn / 16);
    const uint4 x = lds128(raw + blk * raw_blk + ((ci ^ raw_swz) * 16));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (!over && !(nan_mark(nan_mark(nan_mark(nan_mark(0, x.x), x.y), x.z), x.w) & 0x80808080u)) continue;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int ch = (c % 4) * 2 + e / 8;
      const uint32_t at = dst + (c / 4) * 1024 + ((ch ^ (row & 7)) * 16) + (e % 8) * 2;
      if (((w[e / 4] >> (8 * (e % 4))) & 0x7fu) == 0x7fu) {
        sts16(at, draft >= 0 ? 0 : 0x7fff);
        if (draft >= 0) atomicOr(&poison[draft >> 5], 1u << (draft & 31));
      } else if (over) {
        const uint32_t h = lds16(at);
        if (nonfinite16(h, !f16)) sts16(at, (h & 0x8000u) | (f16 ? 0x7bffu : 0x7f7fu));
      }
    }
  }
}

// This thread's part of one raw row into the stage.  Returns marks of NaN codes (bf16 only: the
// conversion to fp16 keeps them).
template <int D, int kParts, bool BF16, bool TWO>
__device__ __forceinline__ uint32_t widen_row(uint32_t raw, uint32_t raw_blk, uint32_t raw_swz,
                                              uint32_t dst, int row, int part, const RowScale& s) {
  constexpr int kIn = D < 128 ? D : 128, kChunks = D / 16 / kParts;
  uint32_t marks = 0;
  // both rows start at a multiple of their swizzled run (kIn and 128 bytes), so a chunk's address
  // is the row's, its swizzle included, with the chunk's number flipped in
  const uint32_t from = raw + raw_swz * 16, to = dst + (row & 7) * 16;
  constexpr int kBatch = 4;  // chunks whose loads are issued together
#pragma unroll(BF16 ? 1 : 2)
  for (int c0 = 0; c0 < kChunks; c0 += kBatch) {
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int c = part * kChunks + c0 + u;  // 16 columns from 16c on
      w[u] = lds128((from ^ ((c % (kIn / 16)) * 16)) + (c / (kIn / 16)) * raw_blk);
    }
    const uint32_t block = to + (part * kChunks + c0) / 4 * 1024;  // 64 columns
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint4 x, y;
      widen4<BF16, TWO>(w[u].x, s, x.x, x.y);
      widen4<BF16, TWO>(w[u].y, s, x.z, x.w);
      widen4<BF16, TWO>(w[u].z, s, y.x, y.y);
      widen4<BF16, TWO>(w[u].w, s, y.z, y.w);
      if constexpr (BF16) marks = nan_mark(nan_mark(nan_mark(nan_mark(marks, w[u].x), w[u].y), w[u].z), w[u].w);
      sts128(block ^ (2 * u * 16), x);
      sts128(block ^ ((2 * u + 1) * 16), y);
    }
  }
  return marks;
}

// The barriers and rings of K or of V: raw ring (full, empty) and 16-bit ring.
struct Rings {
  uint32_t raw, full, empty, out, out_full, out_empty;
};

// BF16: the queries' type.
template <int D, int BN, int STAGES, int RAW, bool BF16>
__device__ __forceinline__ void convert_tiles(const TreeParams& p, bool f16, const Rings& k_rings,
                                              const Rings& v_rings, uint32_t* poison, int b, int hk,
                                              int t_begin, int n, int Lkv, int ctx) {
  constexpr int kParts = 128 / BN, kIn = D < 128 ? D : 128;
  constexpr int kRawBytes = BN * D, kOutBytes = BN * D * 2;
  constexpr uint32_t kRG = (D / 64) * 1024u;
  const int ct = threadIdx.x % 128, row = ct % BN, part = ct / BN;
  // this row's slot in its page is the same in every tile (BN is a multiple of the page size)
  const int pg = row >> p.page_shift, rr = row & (p.page_size - 1);
  const int64_t slot = static_cast<int64_t>(hk) * p.page_size + rr;
  const uint8_t *k_scales = p.k_scales + slot, *v_scales = p.v_scales + slot;
  const int page_stride = p.Hkv * p.page_size;
  const int32_t* entry = p.page_table + static_cast<int64_t>(b) * p.max_pages +
                         ((t_begin * BN) >> p.page_shift) + pg;
  const int tile_pages = BN >> p.page_shift;
  const int last = Lkv - t_begin * BN - row;  // tiles jj with jj * BN < last hold a token here
  // Page ids two tiles ahead, scale bytes one: nothing is computed from a load before then.
  auto page_of = [&](int jj) { return jj < n && jj * BN < last ? __ldg(entry + jj * tile_pages) : 0; };
  auto load_bytes = [&](int jj, int page, uint32_t& kb, uint32_t& vb) {
    if (jj >= n || jj * BN >= last) return;
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) page = 0;  // the producer records it
    const int64_t at = static_cast<int64_t>(page) * page_stride;
    kb = __ldg(k_scales + at);
    vb = __ldg(v_scales + at);
  };
  const uint32_t raw_row = (pg << p.page_shift) * D + rr * kIn;
  const uint32_t raw_blk = kIn << p.page_shift;
  const uint32_t raw_swz = D >= 128 ? rr & 7 : (rr >> 1) & 3;
  const uint32_t dst_row = (row / 8) * kRG + (row % 8) * 128;
  uint32_t kb = 127, vb = 127;
  load_bytes(0, page_of(0), kb, vb);
  int page = page_of(1);
  int rs = 0, stage = 0;  // raw and 16-bit slots, their phases
  uint32_t raw_phase = 0, out_phase = 1;
  for (int jj = 0; jj < n; ++jj) {
    const uint32_t k_byte = kb, v_byte = vb;
    load_bytes(jj + 1, page, kb, vb);
    page = page_of(jj + 2);
#pragma unroll 1
    for (int v = 0; v < 2; ++v) {
      const Rings& g = v ? v_rings : k_rings;
      const uint32_t byte = v ? v_byte : k_byte;
      if (!mbar_wait(g.full + 8u * rs, raw_phase, p.status)) return;
      if (jj >= STAGES && !mbar_wait(g.out_empty + 8u * stage, out_phase, p.status)) return;
      const uint32_t raw = g.raw + rs * kRawBytes + raw_row, dst = g.out + stage * kOutBytes + dst_row;
      if (jj * BN >= last) {
        // past the sequence's end: zeros, whatever the page holds
        for (int c = part * (D / 8 / kParts); c < (part + 1) * (D / 8 / kParts); ++c)
          sts128(dst + (c / 8) * 1024 + (((c % 8) ^ (row & 7)) * 16), make_uint4(0, 0, 0, 0));
      } else {
        const int key = (t_begin + jj) * BN + row;
        const int draft = v && key >= ctx ? key - ctx : -1;
        uint32_t marks;
        if (f16) {
          const RowScale s = row_scale<false>(BF16 ? byte : byte - 1);  // fp16 queries: half size
          // fp16 stands in for bf16 only where one factor holds every scale
          if (!BF16 && s.two) marks = widen_row<D, kParts, false, true>(raw, raw_blk, raw_swz, dst, row, part, s);
          else marks = widen_row<D, kParts, false, false>(raw, raw_blk, raw_swz, dst, row, part, s);
        } else {
          const RowScale s = row_scale<true>(byte);
          if (s.two) marks = widen_row<D, kParts, true, true>(raw, raw_blk, raw_swz, dst, row, part, s);
          else marks = widen_row<D, kParts, true, false>(raw, raw_blk, raw_swz, dst, row, part, s);
        }
        const bool over = byte >= overflow_byte(f16);
        if ((marks & 0x80808080u) || draft >= 0 || over)
          patch_row<D, kParts>(raw, raw_blk, raw_swz, dst, row, part, draft, poison, over, f16);
      }
      fence_proxy_async_smem();
      mbar_arrive(g.empty + 8u * rs);
      mbar_arrive(g.out_full + 8u * stage);
    }
    if (++rs == RAW) rs = 0, raw_phase ^= 1;
    if (++stage == STAGES) stage = 0, out_phase ^= 1;
  }
}

template <int D, int BN, int STAGES, int RAW, bool BF16, bool Q8, bool SPLIT>
__global__ void __launch_bounds__(Layout<D, BN, STAGES, RAW, Q8>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using L = Layout<D, BN, STAGES, RAW, Q8>;
  constexpr int kThreads = L::kThreads;
  constexpr int H = L::kHalves, CH = BN / H;  // scores of a tile that a softmax thread takes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_addr(smem);
  const uint32_t sQ = s_base, sK = s_base + L::kKOff, sV = s_base + L::kVOff;
  const uint32_t bars = s_base + L::kBarOff;
  const uint32_t bar_q = bars;
  auto bar_k = [&](int s) { return bars + 8u * (1 + s); };
  auto bar_v = [&](int s) { return bars + 8u * (1 + STAGES + s); };
  auto bar_ke = [&](int s) { return bars + 8u * (1 + 2 * STAGES + s); };
  auto bar_ve = [&](int s) { return bars + 8u * (1 + 3 * STAGES + s); };
  // per S/P buffer b (tile j with j % 3 == b): S_j computed, P_j written, P_j V_j finished
  auto bar_s = [&](int b) { return bars + 8u * (1 + 4 * STAGES + b); };
  auto bar_p = [&](int b) { return bars + 8u * (1 + 4 * STAGES + kNumS + b); };
  auto bar_pv = [&](int b) { return bars + 8u * (1 + 4 * STAGES + 2 * kNumS + b); };
  const uint32_t bar_done = bars + 8u * (1 + 4 * STAGES + 3 * kNumS);
  const uint32_t bar_sdone = bar_done + 8u;
  const uint32_t bar_raw = bar_done + 16u;
  // 8-bit pages: raw K, V landed (TMA) and read (converters)
  auto bar_rk = [&](int s) { return bar_raw + 8u * s; };
  auto bar_rv = [&](int s) { return bar_raw + 8u * (RAW + s); };
  auto bar_rke = [&](int s) { return bar_raw + 8u * (2 * RAW + s); };
  auto bar_rve = [&](int s) { return bar_raw + 8u * (3 * RAW + s); };
  const uint32_t bar_qr = bar_raw + 8u * (4 * RAW);  // Q in the operand type
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBarOff + L::kNumBars * 8);
  // drafted tokens whose V row holds a value that is not finite (see the V clearing below)
  uint32_t* poison = reinterpret_cast<uint32_t*>(smem + L::kPoisonOff);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // A 16-bit stage holds BN rows x D columns as 1024-byte SW128 atoms (8 rows x 64 columns), the
  // D/64 atoms of an 8-row group side by side, group after group (a page is whole groups).
  constexpr uint32_t kCB = 1024u;                // column-block stride
  constexpr uint32_t kRG = (D / 64) * 1024u;     // 8-row-group stride

  // ---- work item: (query tile, split) x kv head x sequence, longest sequences first ----
  const int split = blockIdx.x % p.n_splits;
  const int qt = static_cast<int>(blockIdx.x) / p.n_splits;
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
  const int q0 = qt * p.q_per_tile;
  // a tile of padding rows alone has nothing to attend
  const int n_kv_tiles = q0 < n_draft ? (Lkv + BN - 1) / BN : 0;
  const int per_split = (n_kv_tiles + p.n_splits - 1) / p.n_splits;
  const int t_begin = min(n_kv_tiles, split * per_split);
  const int n = min(n_kv_tiles, t_begin + per_split) - t_begin;
  // rows are packed head-major: r = g * q_per_tile + (i - q0); warps past them have no work
  const int rows_used = p.q_per_tile * p.G;
  const int live_warps = (rows_used + 31) / 32;

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_k(s), Q8 ? 128 : 1);
      mbar_init(bar_v(s), Q8 ? 128 : 1);
      mbar_init(bar_ke(s), 1);
      mbar_init(bar_ve(s), 1);
    }
    for (int i = 0; i < kNumS; ++i) {
      mbar_init(bar_s(i), 1);
      mbar_init(bar_p(i), H * live_warps * 32);
      mbar_init(bar_pv(i), 1);
    }
    mbar_init(bar_done, 1);
    mbar_init(bar_sdone, 1);
    if constexpr (Q8) {
      for (int s = 0; s < RAW; ++s) {
        mbar_init(bar_rk(s), 1);
        mbar_init(bar_rv(s), 1);
        mbar_init(bar_rke(s), 128);
        mbar_init(bar_rve(s), 128);
      }
      mbar_init(bar_qr, live_warps * 32);
    }
    fence_barrier_init();
  }
  if (threadIdx.x < kMaxTree / 32) poison[threadIdx.x] = 0;
  if (warp == 5) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  // Operand type of both products: the queries', or fp16 where bf16 queries meet 8-bit keys and
  // values that fp16 holds exactly.
  bool f16 = !BF16;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (Q8 && BF16) {
    // every warp but the two that copy, which have begun meanwhile
    if (warp != 4 && warp != 7) {
      constexpr int kLookers = kThreads - 64;
      const int looker = threadIdx.x - (warp > 7 ? 64 : warp > 4 ? 32 : 0);
      const int last = min(Lkv, (t_begin + n) * BN);
      f16 = !barrier_any(9, kLookers,
                         scales_leave_fp16<kLookers>(p, looker, b, hk, t_begin * BN, last));
    }
  }
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_o = tmem;           // O: columns [0, D)
  const uint32_t tm_s0 = tmem + D;      // S/P buffer b: columns [D + b*BN, D + (b+1)*BN)

  if (warp == 4 || (Q8 && warp == 7)) {
    // ------------------------------- TMA producer ---------------------------------------
    // 8-bit pages: warp 4 copies K, warp 7 V (a box takes some 80 clocks to issue, and a tile has
    // BN / page_size of each); 16-bit pages: warp 4 copies both.
    const bool do_k = warp == 4, do_v = !Q8 || warp == 7;
    if (n > 0) {
      if (do_k && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        mbar_arrive_expect_tx(bar_q, static_cast<uint32_t>(D * 2 * p.q_per_tile * p.G));
        for (int kb = 0; kb < D / 64; ++kb)
          tma_load_4d(sQ + kb * (kRows * 128), &tm_q, bar_q, kb * 64, q0, hk * p.G, b);
      }
      // A KV tile is BN / page_size pages, each one TMA box.  Lane i holds the page id of page i
      // of a tile, loaded one tile ahead, and issues that page's box itself.
      const int ps = p.page_size, tp = BN / ps;
      const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
      auto tile_page = [&](int jj) {  // pages past the sequence's end read page 0, keys hidden
        const int lp = (t_begin + jj) * tp + lane;
        return lane < tp && static_cast<int64_t>(lp) * ps < Lkv ? __ldg(table + lp) : 0;
      };
      auto checked = [&](int id) {  // where an id is used, so that nothing waits for its load
        if (id >= 0 && id < p.num_pages) return id;
        record_error(p.status, kDevBounds);
        return 0;
      };
      constexpr int kRing = Q8 ? RAW : STAGES;
      constexpr uint32_t kBytes = Q8 ? L::kRawBytes : L::kKVBytes;
      const uint32_t dst_k = Q8 ? s_base + L::kRawKOff : sK, dst_v = Q8 ? s_base + L::kRawVOff : sV;
      auto full_k = [&](int s) { return Q8 ? bar_rk(s) : bar_k(s); };
      auto full_v = [&](int s) { return Q8 ? bar_rv(s) : bar_v(s); };
      auto empty_k = [&](int s) { return Q8 ? bar_rke(s) : bar_ke(s); };
      auto empty_v = [&](int s) { return Q8 ? bar_rve(s) : bar_ve(s); };
      auto load_pages = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int id) {
        if (lane < tp) {
          const uint32_t to = dst + lane * ps * (kBytes / BN);
          if constexpr (Q8) tma_load_4d(to, map, bar, 0, 0, 0, id * p.Hkv + hk);
          else tma_load_5d(to, map, bar, 0, 0, 0, 0, id * p.Hkv + hk);
        }
      };
      int k_issued = 0, v_issued = 0;
      int ids_next = tile_page(0);
      for (int jj = 0; jj < n; ++jj) {
        const int ids = checked(ids_next);
        if (jj + 1 < n) ids_next = tile_page(jj + 1);
        const int stage = jj % kRing;
        const uint32_t par = ((jj / kRing) - 1) & 1;
        if (do_k) {
          const bool okw = jj < kRing || mbar_wait(empty_k(stage), par, p.status);
          if (!__shfl_sync(0xffffffffu, okw ? 1 : 0, 0)) break;
          if (lane == 0) mbar_arrive_expect_tx(full_k(stage), kBytes);
          __syncwarp();
          load_pages(dst_k + stage * kBytes, &tm_k, full_k(stage), ids);
          k_issued = jj + 1;
        }
        if (do_v) {
          const bool okw = jj < kRing || mbar_wait(empty_v(stage), par, p.status);
          if (!__shfl_sync(0xffffffffu, okw ? 1 : 0, 0)) break;
          if (lane == 0) mbar_arrive_expect_tx(full_v(stage), kBytes);
          __syncwarp();
          load_pages(dst_v + stage * kBytes, &tm_v, full_v(stage), ids);
          v_issued = jj + 1;
        }
      }
      if (lane == 0 && ((do_k && k_issued < n) || (do_v && v_issued < n))) {
        // A wait ran out: let the copies in flight land before the CTA exits.  Each of these is
        // the last one issued to its stage, so its parity wait is exact.
        if (do_k) mbar_wait(bar_q, 0, nullptr);
        for (int jj = max(0, k_issued - kRing); jj < k_issued; ++jj)
          mbar_wait(full_k(jj % kRing), (jj / kRing) & 1, nullptr);
        for (int jj = max(0, v_issued - kRing); jj < v_issued; ++jj)
          mbar_wait(full_v(jj % kRing), (jj / kRing) & 1, nullptr);
      }
    }
  } else if (warp == 5) {
    // ------------------------------- P V issuer -----------------------------------------
    if (lane == 0 && n > 0) {
      const uint32_t idesc_o = idesc_f16(!f16, kRows, D, false, true);
      const uint64_t v_desc = sdesc_sw128(sV, kCB, kRG);
      bool ok = true;
      for (int jj = 0; ok && jj < n; ++jj) {
        const int stage = jj % STAGES, buf = jj % kNumS;
        if (!(ok = mbar_wait(bar_p(buf), (jj / kNumS) & 1, p.status))) break;
        if (!(ok = mbar_wait(bar_v(stage), (jj / STAGES) & 1, p.status))) break;
        tc_fence_after();
        const uint64_t vd = sdesc_add(v_desc, stage * L::kKVBytes);
        const uint32_t a_p = tm_s0 + buf * BN;
        const int left = Lkv - (t_begin + jj) * BN;  // tokens from this tile's first on
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          // P (16-bit pairs) of each half lies over the first columns of its own scores.  16-bit
          // pages: steps past the sequence's end are left out, so that nothing has to clear their
          // V (92 sequences of two tokens, 8 kv heads: 43 -> 31 us with the mask's prefetch and
          // no ranking); converters write zeros there at no cost, and a branch a step costs 2 %
          if (Q8 || kk * 16 < left)
            mma_ts(tm_o, a_p + kk * 8 + (kk / (CH / 16)) * (CH / 2), sdesc_add(vd, kk * (2 * kRG)), idesc_o,
                   (jj > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bar_pv(buf));
        tc_commit(bar_ve(stage));
      }
      // Every MMA this thread issued must finish before tensor memory is released.
      tc_commit(bar_done);
      mbar_wait(bar_done, 0, nullptr);
    }
  } else if (warp == 6) {
    // --------------------------------- S issuer -----------------------------------------
    if (lane == 0 && n > 0) {
      const uint32_t idesc_s = idesc_f16(!f16, kRows, BN, false, false);
      const uint64_t k_desc = sdesc_sw128(sK, 16, kRG);
      const uint64_t q_desc = sdesc_sw128(sQ, 16, 1024);
      bool ok = mbar_wait(Q8 && BF16 && f16 ? bar_qr : bar_q, 0, p.status);
      for (int jj = 0; ok && jj < n; ++jj) {
        const int stage = jj % STAGES, buf = jj % kNumS;
        if (!(ok = mbar_wait(bar_k(stage), (jj / STAGES) & 1, p.status))) break;
        if (jj >= kNumS && !(ok = mbar_wait(bar_pv(buf), ((jj - kNumS) / kNumS) & 1, p.status))) break;
        tc_fence_after();
        const uint64_t kd = sdesc_add(k_desc, stage * L::kKVBytes);
        const uint32_t d_s = tm_s0 + buf * BN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk % 4) * 32;
          mma_ss(d_s, sdesc_add(q_desc, (kk / 4) * (kRows * 128) + off),
                 sdesc_add(kd, (kk / 4) * kCB + off), idesc_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(bar_s(buf));
        tc_commit(bar_ke(stage));
      }
      tc_commit(bar_sdone);
      mbar_wait(bar_sdone, 0, nullptr);
    }
  } else if (Q8 && warp >= L::kConvertWarp && warp < L::kHalfWarp) {
    // -------------------------------- converters ----------------------------------------
    if constexpr (Q8) {
      const Rings k{s_base + L::kRawKOff, bar_rk(0), bar_rke(0), sK, bar_k(0), bar_ke(0)};
      const Rings v{s_base + L::kRawVOff, bar_rv(0), bar_rve(0), sV, bar_v(0), bar_ve(0)};
      convert_tiles<D, BN, STAGES, RAW, BF16>(p, f16, k, v, poison, b, hk, t_begin, n, Lkv, ctx);
    }
  } else if ((warp < 4 || warp >= L::kHalfWarp) && warp % 4 < live_warps) {
    // --------------------------- softmax + epilogue -------------------------------------
    // Row r = 32 (warp % 4) + lane, of which warps 0-3 take the first CH scores of a tile and warps
    // kHalfWarp.. the last CH: two warps a sub-partition, so that one's latencies hide behind
    // the other's.  They share the row's running maximum without exchanging it: each votes on
    // whether its scores are far enough above it, and only a tile where some row's are (the
    // first, and few others) trades maxima through shared memory.
    const int half = warp >= L::kHalfWarp ? 1 : 0, wq = warp % 4;
    const int r = wq * 32 + lane, team = H * live_warps * 32;
    const int vote = 1 + wq, trade = 5 + wq;  // barriers of the two warps that share these rows
    const int g = r / p.q_per_tile, i = q0 + r % p.q_per_tile;
    const bool valid = g < p.G && i < p.T;   // a row of the output
    const bool active = valid && i < n_draft;  // a query of this sequence (else an empty row)
    const int64_t flat = (static_cast<int64_t>(b) * p.Hq + hk * p.G + g) * p.T + i;
    float* row_mem = reinterpret_cast<float*>(smem + L::kRowOff) + r;
    auto shared = [&](int h) -> float& { return row_mem[h * kRows]; };
    float& q_factor = row_mem[2 * kRows];
    TreeRow row;
    row.i = i;
    row.n = active ? n_draft : 0;
    row.words = nullptr;
    if (p.mask && active)
      row.words = p.mask + (static_cast<int64_t>(p.mask_batches == 1 ? 0 : b) * p.T + i) * p.words;
    if (row.words) prefetch_l1(row.words);
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    float m_run = -INFINITY, l_run = 0.f;
    // a > 0 goes into the exponential's argument; otherwise the scores are scaled first
    const bool pre = !(p.scale_log2 > 0.f);
    // K and V at half size (see convert_tiles)
    constexpr float kUnhalve = Q8 && !BF16 ? 2.f : 1.f;
    float to_log2 = p.scale_log2 * kUnhalve;
    // A wait that runs out leaves ok false: no more work, but every barrier is still met.
    bool ok = true;
    if constexpr (Q8 && BF16) {
      if (f16 && n > 0 && half == 0) {
        // this thread's row of Q, bf16 to fp16 times 2^-eq, in place in its swizzled tile
        ok = __all_sync(0xffffffffu, mbar_wait(bar_q, 0, p.status));
        if (ok) {
          q_factor = q_row_to_fp16<D>(sQ, r);
          fence_proxy_async_smem();
          __syncwarp();
          mbar_arrive(bar_qr);
        }
      }
    }
    for (int jj = 0; jj < n; ++jj) {
      const int buf = jj % kNumS;
      const uint32_t t_s = tm_s0 + lane_off + buf * BN;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar_s(buf), (jj / kNumS) & 1, p.status));
      if (Q8 && BF16 && f16 && jj == 0) {
        to_log2 *= q_factor;  // written before S_0 could be issued
        // never 0, which a hidden score's -inf would turn into NaN; scores are below 2^39 here
        if (!pre) to_log2 = fmaxf(to_log2, FLT_MIN);
      }
      const float a = pre ? 1.f : to_log2;
      const int key0 = (t_begin + jj) * BN;
      uint32_t raw[CH];
      float row_max = -INFINITY;
      if (ok) {
        tc_fence_after();
        prefill::load_s<CH>(t_s + half * CH, raw);
        if (pre) {
#pragma unroll
          for (int c = 0; c < CH; ++c) raw[c] = __float_as_uint(__uint_as_float(raw[c]) * to_log2);
        }
        if (key0 + BN > ctx) {
#pragma unroll
          for (int w = 0; w < CH / 32; ++w) {
            const uint32_t bits = row_bits(row, key0 + half * CH + 32 * w - ctx);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((bits >> c) & 1)) raw[32 * w + c] = 0xff800000u;  // -inf
          }
        }
        row_max = a * chunk_max(raw);
      }
      const bool raise = barrier_any(vote, H * 32, ok && row_max > m_run + prefill::kRescaleLog2);
      if (raise) {
        shared(half) = row_max;
        barrier_sync(trade, H * 32);
        const float m_new = fmaxf(m_run, fmaxf(row_max, shared(1 - half)));
        float alpha = 1.f;
        if (m_new > m_run + prefill::kRescaleLog2) {
          alpha = exp2_approx(m_run - m_new);  // 0 when m_run is -inf
          m_run = m_new;
          l_run *= alpha;
        }
        if (jj > 0) {
          // O is rescaled, half its columns each, once every earlier P V product is in it; a
          // tile with no rescale does not wait (S_j itself needed P_{j-3} V_{j-3} finished)
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar_pv((jj - 1) % kNumS), ((jj - 1) / kNumS) & 1, p.status));
          if (ok) {
            tc_fence_after();
            prefill::rescale_o<D / H>(tm_o + lane_off + half * (D / H), alpha);
          }
        }
      }
      if (!ok) continue;
      uint32_t pk[CH / 2];
      if constexpr (Q8 && BF16) {
        if (f16) chunk_weights<CH, false>(raw, a, m_run, l_run, pk);
        else chunk_weights<CH, true>(raw, a, m_run, l_run, pk);
      } else {
        chunk_weights<CH, BF16>(raw, a, m_run, l_run, pk);
      }
      prefill::store_p<CH>(t_s + half * CH, pk);
      tmem_st_wait();
      if (!Q8 && key0 + BN > ctx) {
        // The stage holds rows of drafted tokens, which some queries do not see, or rows past
        // the sequence's end.  Their weight is 0, but 0 times a V that is not finite would
        // still poison O: rows past the end are cleared, and such values of drafted tokens are
        // cleared and their token noted (the epilogue gives them to the rows that see it).
        // The parity wait for V_j is exact only once V_{j-STAGES} has landed: P_{j-1} V_{j-1}
        // finishing makes sure of it.
        const int stage = jj % STAGES;
        if (jj > 0 && !raise)
          ok = __all_sync(0xffffffffu, mbar_wait(bar_pv((jj - 1) % kNumS), ((jj - 1) / kNumS) & 1, p.status));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar_v(stage), (jj / STAGES) & 1, p.status));
        if (!ok) continue;
        const uint32_t vst = sV + stage * L::kKVBytes;
        const int r0 = max(0, ctx - key0);
        constexpr int kChunks = D / 8;  // 16-byte chunks a row
        const int r1 = min(BN, (Lkv - key0 + 15) & ~15);  // rows that P V reads
        for (int u = (half * live_warps + wq) * 32 + lane; u < (r1 - r0) * kChunks; u += team) {
          const int vr = r0 + u / kChunks, c = u % kChunks;
          const uint32_t at = vst + (vr / 8) * kRG + (c / 8) * kCB + (vr % 8) * 128 + (c % 8) * 16;
          const int d = key0 + vr - ctx;
          if (d >= n_draft) {
            sts128(at, make_uint4(0, 0, 0, 0));
            continue;
          }
          const uint4 v = lds128(at);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (nonfinite16(w[e], BF16)) w[e] &= 0xffff0000u, bad = true;
            if (nonfinite16(w[e] >> 16, BF16)) w[e] &= 0x0000ffffu, bad = true;
          }
          if (bad) {
            sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
            atomicOr(&poison[d >> 5], 1u << (d & 31));
          }
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(bar_p(buf));
    }
    if (ok && n > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_pv((n - 1) % kNumS), ((n - 1) / kNumS) & 1, p.status));
      tc_fence_after();
    }
    // the row's sum over both halves (their maxima are one)
    barrier_sync(trade, H * 32);  // the last maxima have been read
    shared(half) = l_run;
    barrier_sync(trade, H * 32);
    l_run = shared(0) + shared(1);
    if (ok) {
      // O / l, a row's slab of columns at a time, the halves in turn: staged in this warp's part of
      // the K ring (free: every MMA has finished) with 16-byte chunks swizzled by the row, then
      // written out as whole 128-byte runs, eight lanes a row.
      const bool have = active && n > 0 && !(l_run == 0.f);  // a NaN sum stays NaN
      const float inv_l = kUnhalve / l_run;
      bool any_poison = false;
      if (n > 0) {
        for (int w = 0; w < kMaxTree / 32; ++w) any_poison |= poison[w] != 0;
      }
      const uint32_t stage = sK + (half * 4 + wq) * 4096;
      constexpr int kCols = SPLIT ? 32 : 64;  // columns of a 128-byte run
      const int64_t my_row = SPLIT ? flat * p.n_splits + split : flat;
#pragma unroll 1
      for (int c0 = half * kCols; c0 < D; c0 += H * kCols) {
#pragma unroll
        for (int h = 0; h < kCols / 32; ++h) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tm_o + lane_off + c0 + 32 * h, o);
            tmem_ld_wait();
          }
          if (any_poison && active) {
            for (int d = 0; d < n_draft; ++d) {
              if (!((poison[d >> 5] >> (d & 31)) & 1) || !row_sees(row, d)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) +
                                       nonfinite_v<D, BF16, Q8>(p, b, hk, ctx + d, c0 + 32 * h + e));
            }
          }
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = have ? __uint_as_float(o[e]) * inv_l : 0.f;
#pragma unroll
          for (int ch = 0; ch < (SPLIT ? 8 : 4); ++ch) {
            uint4 w;
            if constexpr (SPLIT) {
              w = make_uint4(__float_as_uint(v[4 * ch]), __float_as_uint(v[4 * ch + 1]),
                             __float_as_uint(v[4 * ch + 2]), __float_as_uint(v[4 * ch + 3]));
            } else {
              uint32_t u[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = BF16 ? pack_bf16x2(v[8 * ch + 2 * e], v[8 * ch + 2 * e + 1])
                            : pack_f16x2(v[8 * ch + 2 * e], v[8 * ch + 2 * e + 1]);
              w = make_uint4(u[0], u[1], u[2], u[3]);
            }
            const int at = SPLIT ? ch : 4 * h + ch;
            sts128(stage + lane * 128 + ((at ^ (lane & 7)) * 16), w);
          }
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int rr = 4 * s + lane / 8, ch = lane % 8;
          const int64_t to = __shfl_sync(0xffffffffu, my_row, rr);
          const bool st = __shfl_sync(0xffffffffu, valid ? 1 : 0, rr);
          const uint4 w = lds128(stage + rr * 128 + ((ch ^ (rr & 7)) * 16));
          if (st) {
            if constexpr (SPLIT)
              *reinterpret_cast<uint4*>(p.o_part + to * D + c0 + ch * 4) = w;
            else
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to * D + c0 + ch * 8) = w;
          }
        }
        __syncwarp();
      }
      if (valid && half == 0) {
        const float lse = have ? (m_run - (f16 ? kWeightLog2F16 : 0.f) + log2f(l_run)) * prefill::kLn2 : -INFINITY;
        // the merge takes a part of weight +inf as not a number, which a NaN part would not be
        if constexpr (SPLIT) p.lse_part[my_row] = lse != lse ? INFINITY : lse;
        else if (p.lse) p.lse[my_row] = lse;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
int bad(int code, const char* msg) { return set_error(code, msg); }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

struct TreePlan {
  int G, q_per_tile, n_qtiles, n_splits;
  bool few_rows;  // the kernel of tree_rows.cu
  size_t off_lse, total;
};

constexpr int kFewRowsTokens = 256;  // least tokens of a part in the kernel for few rows

// KV tile of a head dimension: as the prefill kernels', what tensor memory holds beside O.
int block_n(int D) { return D == 256 ? 64 : 128; }

TreePlan plan_tree(const fa_tree_args* a) {
  TreePlan pl{};
  pl.G = a->Hq / a->Hkv;
  // equal query tiles, so that their rows are packed without gaps
  const int most = 128 / pl.G;
  pl.n_qtiles = (a->T + most - 1) / most;
  pl.q_per_tile = (a->T + pl.n_qtiles - 1) / pl.n_qtiles;
  pl.n_qtiles = (a->T + pl.q_per_tile - 1) / pl.q_per_tile;
  const int rows = pl.G * a->T;
  pl.few_rows = a->cache_dtype == FA_E4M3 && tree_rows_takes(rows);
  const int bn = pl.few_rows ? kFewRowsTokens : block_n(a->D);
  const int kv_tiles = (a->max_seq_len + bn - 1) / bn;
  int s = 1;
  if (a->num_splits > 0) {
    s = a->num_splits;
  } else if (pl.few_rows) {
    // its CTAs are small and several share an SM: split while the units leave half of the places
    // free, down to kFewRowsTokens tokens a part.  The busiest SM holds ceil(units s / SMs) parts
    // of length 1 / s: of the counts that fill the SMs one to `ctas` times, the one where that is
    // least, of equals the larger (4 sequences of 4096 tokens, 8 kv heads: 14 parts 12.7 us, 16
    // parts 14.4; 24 of them: 3 parts 40, 2 parts 43).
    const long units = static_cast<long>(a->Hkv) * a->B;
    const long sms = num_sms() > 0 ? num_sms() : 152;
    const int ctas = tree_rows_ctas(a->D, rows);
    if (units > 0 && units * 2 <= sms * ctas) {
      long best = 1, load = (units + sms - 1) / sms;
      for (int c = 1; c <= ctas; ++c) {
        long n = c * sms / units;
        if (n > kv_tiles) n = kv_tiles;
        if (n < 1) continue;
        const long at = (units * n + sms - 1) / sms;
        if (at * best <= load * n) {
          best = n;
          load = at;
        }
      }
      s = static_cast<int>(best);
    }
  } else if (kv_tiles > 0) {
    // as the prefill plan: split only when the tiles cover less than half the SMs
    const long tiles = static_cast<long>(pl.n_qtiles) * a->Hkv * a->B;
    const int sms = num_sms() > 0 ? num_sms() : 152;
    if (tiles * 2 <= sms) {
      s = static_cast<int>(sms / tiles);
      const int cap = kv_tiles / 4 > 1 ? kv_tiles / 4 : 1;
      if (s > cap) s = cap;
    }
  }
  if (s > kv_tiles) s = kv_tiles;
  if (s < 1) s = 1;
  pl.n_splits = s;
  if (s > 1) {
    const size_t all = static_cast<size_t>(a->B) * a->Hq * a->T;
    pl.off_lse = (all * s * a->D * sizeof(float) + 255) / 256 * 256;
    pl.total = pl.off_lse + (all * s * sizeof(float) + 255) / 256 * 256;
  }
  return pl;
}

int check_tree(const fa_tree_args* a, bool pointers) {
  char msg[200];
  if (!a) return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: null argument struct");
  if (a->B < 0 || a->T < 0 || a->Hq <= 0 || a->Hkv <= 0 || a->Hq % a->Hkv != 0 || a->max_pages < 0 ||
      a->num_pages < 0 || a->max_seq_len < 0 || a->num_splits < 0)
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: need B, T, max_pages, num_pages, max_seq_len, "
                                   "num_splits >= 0, Hq, Hkv > 0, Hq % Hkv == 0");
  if (a->Hq / a->Hkv > 128)
    return bad(FA_ERR_UNSUPPORTED, "fa_tree_decode_paged: query heads per kv head must be <= 128");
  if (a->D != 64 && a->D != 128 && a->D != 256) {
    snprintf(msg, sizeof msg, "fa_tree_decode_paged: D must be 64, 128 or 256 (got %d)", a->D);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  if (a->T > kMaxTree) {
    snprintf(msg, sizeof msg, "fa_tree_decode_paged: T must be <= %d (got %d)", kMaxTree, a->T);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16)
    return bad(FA_ERR_UNSUPPORTED, "fa_tree_decode_paged: dtype must be FA_BF16 or FA_FP16");
  if (a->cache_dtype != FA_E4M3 && a->cache_dtype != a->dtype)
    return bad(FA_ERR_UNSUPPORTED, "fa_tree_decode_paged: cache_dtype must be FA_E4M3 or dtype");
  const int bn = block_n(a->D);
  if (a->page_size < 8 || a->page_size > bn || (a->page_size & (a->page_size - 1)) != 0) {
    snprintf(msg, sizeof msg, "fa_tree_decode_paged: page_size must be a power of two in [8, %d] (got %d)",
             bn, a->page_size);
    return bad(FA_ERR_UNSUPPORTED, msg);
  }
  if (a->B > 65535 || a->Hkv > 65535)
    return bad(FA_ERR_UNSUPPORTED, "fa_tree_decode_paged: B and Hkv must be <= 65535");
  if (static_cast<int64_t>(a->num_pages) * a->Hkv > 2147483647LL ||
      static_cast<int64_t>(a->max_pages) * a->page_size > 2147483647LL - 256)  // a tile past the end
    return bad(FA_ERR_UNSUPPORTED, "fa_tree_decode_paged: num_pages * Hkv must fit in int32, and "
               "max_pages * page_size + 256");
  if (static_cast<int64_t>(a->B) * a->Hq * a->T > 2147483647LL)
    return bad(FA_ERR_UNSUPPORTED, "fa_tree_decode_paged: B * Hq * T must fit in int32");
  if (a->max_seq_len > static_cast<int64_t>(a->max_pages) * a->page_size)
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: max_seq_len exceeds max_pages * page_size");
  if (!(a->scale == a->scale) || isinf(a->scale))
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: scale must be finite");
  if (a->tree_mask && a->mask_batches != 1 && a->mask_batches != a->B)
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: mask_batches must be 1 or B");
  if (!pointers || a->B == 0 || a->T == 0) return FA_OK;
  if (!a->q || !a->out || !a->seq_lens ||
      (a->max_seq_len > 0 && (!a->k_pages || !a->v_pages || !a->page_table || a->num_pages == 0)))
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: null pointer or no pages");
  if (a->max_seq_len > 0 && a->cache_dtype == FA_E4M3 && (!a->k_scales || !a->v_scales))
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: an 8-bit cache needs k_scales and v_scales");
  if (!aligned(a->q, 16) || !aligned(a->k_pages, 16) || !aligned(a->v_pages, 16) || !aligned(a->out, 16) ||
      !aligned(a->tree_mask, 8) || !aligned(a->seq_lens, 4) || !aligned(a->draft_lens, 4) ||
      !aligned(a->page_table, 4) || !aligned(a->lse, 4) || !aligned(a->k_scales, 8) || !aligned(a->v_scales, 8))
    return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: q, the pages and out must be 16-byte aligned, "
                                   "tree_mask and the scales 8-byte aligned");
  // a tensor map takes strides of a multiple of 16 bytes, positive, below 2^40 bytes
  const int n[3] = {a->B, a->Hq, a->T};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (a->q_strides[i] % 8 != 0 || a->q_strides[i] <= 0 || a->q_strides[i] >= (1LL << 39)))
      return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: q's strides must be positive multiples of 16 bytes");
  return FA_OK;
}

template <int D, int BN, int STAGES, int RAW, bool BF16, bool Q8>
cudaError_t launch_impl(const fa_tree_args* a, const TreeParams& p, cudaStream_t st) {
  using L = Layout<D, BN, STAGES, RAW, Q8>;
  const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tq, tk, tv;
  {
    // (column, query, head, sequence); the stride of a dimension of one is never used
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.T),
                              static_cast<uint64_t>(p.Hq), static_cast<uint64_t>(p.B)};
    const uint64_t str[3] = {p.T > 1 ? static_cast<uint64_t>(a->q_strides[2]) * 2 : D * 2ull,
                             p.Hq > 1 ? static_cast<uint64_t>(a->q_strides[1]) * 2 : D * 2ull,
                             p.B > 1 ? static_cast<uint64_t>(a->q_strides[0]) * 2 : D * 2ull};
    const uint32_t box[4] = {64, static_cast<uint32_t>(p.q_per_tile), static_cast<uint32_t>(p.G), 1};
    if (!encode_tiled(&tq, dt, 4, a->q, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const uint64_t ps = static_cast<uint64_t>(p.page_size), pages = static_cast<uint64_t>(p.num_pages) * p.Hkv;
  if constexpr (Q8) {
    // a page of one head: page_size rows of D bytes as (column, row, block of 128 columns)
    constexpr uint64_t in = D < 128 ? D : 128;
    const uint64_t dims[4] = {in, ps, D / in, pages}, str[3] = {D, in, ps * D};
    const uint32_t box[4] = {static_cast<uint32_t>(in), static_cast<uint32_t>(ps), static_cast<uint32_t>(D / in), 1};
    const CUtensorMapSwizzle swz = D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!encode_tiled(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a->k_pages, dims, str, box, swz) ||
        !encode_tiled(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a->v_pages, dims, str, box, swz))
      return cudaErrorInvalidValue;
  } else {
    const uint64_t row = static_cast<uint64_t>(D) * 2;
    const uint64_t dims[5] = {64, 8, static_cast<uint64_t>(D) / 64, ps / 8, pages};
    const uint64_t str[4] = {row, 128, 8 * row, ps * row};
    const uint32_t box[5] = {64, 8, static_cast<uint32_t>(D) / 64, static_cast<uint32_t>(ps) / 8, 1};
    if (!encode_tiled(&tk, dt, 5, a->k_pages, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tiled(&tv, dt, 5, a->v_pages, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  auto kern = p.n_splits > 1 ? tree_kernel<D, BN, STAGES, RAW, BF16, Q8, true>
                             : tree_kernel<D, BN, STAGES, RAW, BF16, Q8, false>;
  cudaError_t e = ensure_smem_limit(kern, L::kAlloc);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.n_qtiles * p.n_splits, p.Hkv, p.B);
  kern<<<grid, L::kThreads, L::kAlloc, st>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_tree(const fa_tree_args* a, const TreeParams& p, cudaStream_t st) {
  if (a->cache_dtype == FA_E4M3) {
    switch (a->D) {
      case 64: return launch_impl<64, 128, 3, 3, BF16, true>(a, p, st);
      case 128: return launch_impl<128, 128, 2, 2, BF16, true>(a, p, st);
      default: return launch_impl<256, 64, 2, 1, BF16, true>(a, p, st);
    }
  }
  switch (a->D) {
    case 64: return launch_impl<64, 128, 5, 1, BF16, false>(a, p, st);
    case 128: return launch_impl<128, 128, 3, 1, BF16, false>(a, p, st);
    default: return launch_impl<256, 64, 2, 1, BF16, false>(a, p, st);
  }
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_tree_mask(const int32_t* parents, int T, uint64_t* words) {
  if (T < 0 || T > kMaxTree) return bad(FA_ERR_INVALID_ARG, "fa_tree_mask: T must be in [0, 256]");
  if (T > 0 && (!parents || !words)) return bad(FA_ERR_INVALID_ARG, "fa_tree_mask: null pointer");
  const int W = (T + 63) / 64;
  for (int i = 0; i < T; ++i) {
    const int up = parents[i];
    if (up < -1 || up >= i) return bad(FA_ERR_INVALID_ARG, "fa_tree_mask: a parent must come before its child, or be -1");
    for (int w = 0; w < W; ++w) words[i * W + w] = up >= 0 ? words[up * W + w] : 0;
    words[i * W + i / 64] |= 1ull << (i % 64);
  }
  return FA_OK;
}

size_t fa_tree_workspace_size(const fa_tree_args* a) {
  if (check_tree(a, false) != FA_OK || a->B == 0 || a->T == 0) return 0;
  return plan_tree(a).total;
}

int fa_tree_decode_paged(const fa_tree_args* a, void* stream) {
  int rc = check_tree(a, true);
  if (rc != FA_OK || a->B == 0 || a->T == 0) return rc;
  const TreePlan pl = plan_tree(a);
  char msg[200];
  if (pl.total > 0) {
    if (!a->workspace || a->workspace_bytes < pl.total) {
      snprintf(msg, sizeof msg, "fa_tree_decode_paged: workspace of %zu bytes needed (got %zu)", pl.total,
               a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
      return bad(FA_ERR_WORKSPACE, msg);
    }
    if (!aligned(a->workspace, 256))
      return bad(FA_ERR_INVALID_ARG, "fa_tree_decode_paged: workspace must be 256-byte aligned");
  }
  uint32_t* status = device_status_ptr();
  if (!status) return bad(FA_ERR_CUDA, "fa_tree_decode_paged: no usable CUDA device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MergeParams m{};
  m.out = a->out;
  m.lse = a->lse;
  m.rows = a->B * a->Hq * a->T;
  m.D = a->D;
  m.max_splits = pl.n_splits;
  m.out_dtype = static_cast<Dtype>(a->dtype);
  cudaError_t e;
  if (a->max_seq_len == 0) {  // no key anywhere: the merge alone writes the empty rows
    m.max_splits = 0;
    e = launch_merge(m, st);
    if (e != cudaSuccess) return bad(FA_ERR_CUDA, cudaGetErrorString(e));
    return FA_OK;
  }
  TreeParams p{};
  p.k_pages = a->k_pages;
  p.v_pages = a->v_pages;
  p.k_scales = a->k_scales;
  p.v_scales = a->v_scales;
  p.page_table = a->page_table;
  p.kv_lens = a->seq_lens;
  p.draft_lens = a->draft_lens;
  p.mask = a->tree_mask;
  p.out = a->out;
  p.lse = a->lse;
  p.mask_batches = a->mask_batches;
  p.words = (a->T + 63) / 64;
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = pl.G;
  p.T = a->T;
  p.q_per_tile = pl.q_per_tile;
  p.n_qtiles = pl.n_qtiles;
  p.n_splits = pl.n_splits;
  p.page_size = a->page_size;
  while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
  p.max_pages = a->max_pages;
  p.num_pages = a->num_pages;
  p.scale_log2 = a->scale * 1.44269504088896340736f;
  p.status = status;
  // the order matters where blocks wait for others to end and their lengths can differ by much
  const long units = static_cast<long>(pl.n_splits) * (pl.few_rows ? 1 : pl.n_qtiles) * a->Hkv * a->B;
  const long places = static_cast<long>(num_sms() > 0 ? num_sms() : 152) *
                      (pl.few_rows ? tree_rows_ctas(a->D, pl.G * a->T) : 1);
  p.ranked = units > places && a->max_seq_len > 512;
  if (pl.n_splits > 1) {
    p.o_part = static_cast<float*>(a->workspace);
    p.lse_part = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + pl.off_lse);
  }
  if (pl.few_rows) {
    p.q = a->q;
    p.q_strides[0] = a->B > 1 ? a->q_strides[0] : 0;
    p.q_strides[1] = a->Hq > 1 ? a->q_strides[1] : 0;
    p.q_strides[2] = a->T > 1 ? a->q_strides[2] : 0;
    e = launch_tree_rows(p, a->D, a->dtype == FA_BF16, st);
  } else {
    e = a->dtype == FA_BF16 ? launch_tree<true>(a, p, st) : launch_tree<false>(a, p, st);
  }
  if (e != cudaSuccess) {
    snprintf(msg, sizeof msg, "fa_tree_decode_paged (attention kernel): %s", cudaGetErrorString(e));
    return bad(FA_ERR_CUDA, msg);
  }
  if (pl.n_splits > 1) {
    m.o_part = p.o_part;
    m.lse_part = p.lse_part;
    e = launch_merge(m, st);
    if (e != cudaSuccess) {
      snprintf(msg, sizeof msg, "fa_tree_decode_paged (merge kernel): %s", cudaGetErrorString(e));
      return bad(FA_ERR_CUDA, msg);
    }
  }
  return FA_OK;
}

}  // extern "C"
