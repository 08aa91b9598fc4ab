// tree.cuh -- what the kernels of the tree attention share: parameters, the mask of a query row
// over the drafted tokens, and the values of V that are not finite.
#pragma once

#include <stdint.h>

#include "cache.cuh"
#include "sm103.cuh"

namespace fa {

constexpr int kMaxTree = 256;  // drafted tokens

struct TreeParams {
  const void* q;                // the kernel for few rows reads q itself: strides in elements
  int64_t q_strides[3];         // (batch, head, token)
  const void* k_pages;
  const void* v_pages;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* page_table;
  const int32_t* kv_lens;
  const int32_t* draft_lens;    // or nullptr: T each
  const uint64_t* mask;         // [mask_batches, T, words], or nullptr: a chain
  void* out;                    // [B,Hq,T,D]
  float* lse;                   // [B,Hq,T] or nullptr
  float* o_part;                // split: [B*Hq*T, n_splits, D] fp32
  float* lse_part;              // split: [B*Hq*T, n_splits]
  int mask_batches, words;
  int B, Hq, Hkv, G, T;
  int q_per_tile, n_qtiles, n_splits;
  int page_size, page_shift, max_pages, num_pages;
  int ranked;                   // blocks take the sequences in decreasing length
  float scale_log2;
  uint32_t* status;
};

// ------------------------------------------------------------------------------------------
// The mask of one query row over the drafted tokens.
// ------------------------------------------------------------------------------------------
struct TreeRow {
  const uint64_t* words;  // the row's mask words, or nullptr: a chain (tokens 0..i)
  int i, n;               // query, drafted tokens
};

__device__ __forceinline__ uint64_t row_word(const TreeRow& r, int w) {
  const int left = r.n - 64 * w;  // drafted tokens from this word on
  if (left <= 0) return 0;
  uint64_t v = ~0ull;
  if (r.words) {
    v = __ldg(reinterpret_cast<const unsigned long long*>(r.words + w));
  } else {
    const int c = r.i + 1 - 64 * w;
    v = c >= 64 ? ~0ull : c > 0 ? (1ull << c) - 1 : 0ull;
  }
  return left >= 64 ? v : v & ((1ull << left) - 1);
}

// Visibility of the 32 keys from drafted offset `off` on (negative: still in the context).
__device__ __forceinline__ uint32_t row_bits(const TreeRow& r, int off) {
  if (off <= -32) return ~0u;
  if (off < 0) return (static_cast<uint32_t>(row_word(r, 0)) << -off) | ((1u << -off) - 1);
  const int w = off >> 6, s = off & 63;
  uint64_t v = row_word(r, w) >> s;
  if (s > 32) v |= row_word(r, w + 1) << (64 - s);
  return static_cast<uint32_t>(v);
}

__device__ __forceinline__ bool row_sees(const TreeRow& r, int d) {
  return (row_word(r, d >> 6) >> (d & 63)) & 1;
}

// A NaN code (0x7f or 0xff) turns its sign bit over when one is added to every byte; a carry
// out of 0xff can only add further marks.  Sign bits of the result: some byte is NaN.
__device__ __forceinline__ uint32_t nan_mark(uint32_t acc, uint32_t w) {
  return acc | ((w + 0x01010101u) ^ w);
}

__device__ __forceinline__ bool nonfinite16(uint32_t h, bool bf16) {
  return bf16 ? (h & 0x7f80u) == 0x7f80u : (h & 0x7c00u) == 0x7c00u;
}

// Value of V at drafted token d, column c, if it is not finite (else 0): the slow path of a row
// that sees a drafted token with such a value.
template <int D, bool BF16, bool Q8>
__device__ __noinline__ float nonfinite_v(const TreeParams& p, int b, int hk, int key, int c) {
  int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + (key >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) page = 0;  // as the copies read it
  const int64_t at = ((static_cast<int64_t>(page) * p.Hkv + hk) * p.page_size + (key & (p.page_size - 1))) * D + c;
  if constexpr (Q8) {
    const uint32_t v = static_cast<const uint8_t*>(p.v_pages)[at];
    return (v & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : 0.f;
  } else {
    const uint16_t h = static_cast<const uint16_t*>(p.v_pages)[at];
    if (!nonfinite16(h, BF16)) return 0.f;
    return BF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16)
                : __half2float(__ushort_as_half(h));
  }
}

// Shared memory by its 32-bit address.  (A pointer rounded up to the swizzle's alignment is a
// generic one to the compiler, whose loads and stores take several times as long.)
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
               ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}

// Two e4m3 codes (the low or the high 16 bits) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t widen2_hi(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r) : "r"(codes));
  return r;
}

// Starts a row's mask words on their way to L1: the tiles that look at them come last.
__device__ __forceinline__ void prefetch_l1(const void* at) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
}

// The sequence that is `rank`-th in decreasing length (ties by index), so that the last blocks to
// start are short ones; past THREADS sequences, and where the order cannot matter (!p.ranked), the
// rank is the sequence.  All threads of the block must call.
template <int THREADS>
__device__ __forceinline__ int sequence_of_rank(const TreeParams& p, int rank) {
  __shared__ int found;
  if (!p.ranked || p.B == 1 || p.B > THREADS) return rank;
  if (threadIdx.x < p.B) {
    const int mine = p.kv_lens[threadIdx.x];
    int before = 0;
    for (int j = 0; j < p.B; ++j) {
      const int other = p.kv_lens[j];
      before += (other > mine || (other == mine && j < static_cast<int>(threadIdx.x))) ? 1 : 0;
    }
    if (before == rank) found = threadIdx.x;
  }
  __syncthreads();
  return found;
}

// The kernel for few rows over 8-bit pages (tree_rows.cu): takes a call if tree_rows_takes says
// so (rows = query heads per kv head times T); tree_rows_ctas is the number of its CTAs that an SM
// holds at once.
bool tree_rows_takes(int rows);
int tree_rows_ctas(int D, int rows);
cudaError_t launch_tree_rows(const TreeParams& p, int D, bool bf16, cudaStream_t stream);

}  // namespace fa
