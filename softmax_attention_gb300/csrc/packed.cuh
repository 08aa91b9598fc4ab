// packed.cuh -- what the kernels of the packed prompts share: parameters, the sequences behind
// one another in one tensor, and the order in which blocks take their work.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "prefill_common.cuh"
#include "sm103.cuh"

namespace fa {
namespace packed {

constexpr int kRows = 128;     // rows of a query tile: query tokens x the heads of a kv head
constexpr int kKeys = 128;     // keys of a KV tile

struct Params {
  const int32_t* cu_q;   // [B+1] first row of each sequence in q, and the end of the last
  const int32_t* cu_k;   // likewise in k and v
  int B, Hq, Hkv, G, total_q, total_k;
  int q_per_tile;        // query tokens of a tile: floor(128 / G)
  int causal;
  float scale, scale_log2;
  void* out;             // forward: [total_q, Hq, D] by its strides (token, head; elements)
  int64_t out_strides[2];
  float* lse;            // [total_q, Hq]; forward: or nullptr
  uint32_t* status;
};

// One sequence: its first rows and lengths.
struct Seq {
  int q0, nq, k0, nk;
};

// Offsets that do not rise, or reach out of the tensors, make an empty sequence.
__device__ __forceinline__ void load_range(const int32_t* cu, int b, int total, uint32_t* status,
                                           int& first, int& n) {
  first = __ldg(cu + b);
  const int end = __ldg(cu + b + 1);
  n = end - first;
  if (first < 0 || end < first || end > total) {
    record_error(status, kDevBounds);
    first = n = 0;
  }
}

__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  Seq s;
  load_range(p.cu_q, b, p.total_q, p.status, s.q0, s.nq);
  load_range(p.cu_k, b, p.total_k, p.status, s.k0, s.nk);
  return s;
}

// Work items.  Sequence s is cut into items(s) pieces, and a piece's work grows with its index t:
// its level is first(s) + t, or first(s) for all pieces where `flat`.  Blocks take the pieces in
// decreasing level over all sequences, so that the last blocks to start are short ones; nothing
// but the order depends on it.  The piece of a rank is found by each block itself: a binary search
// for the rank's level, a warp's lanes holding up to four sequences each (a few hundred clocks
// beside the block's set-up; no list, no kernel before this one).  Past 128 sequences the pieces
// are taken sequence by sequence.  One whole warp calls; b = -1 where the rank is past the end.
template <typename Items>
__device__ __forceinline__ void find_item(int B, int rank, bool flat, Items items, int& b, int& t) {
  const int lane = threadIdx.x & 31;
  b = -1;
  t = 0;
  if (B == 1) {
    int n, first;
    items(0, n, first);
    if (rank < n) {
      b = 0;
      t = n - 1 - rank;
    }
    return;
  }
  int before = 0;  // pieces in front of those looked at
  constexpr int kHeld = 4;
  if (B <= 32 * kHeld) {
    int n[kHeld], first[kHeld], top = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      n[i] = first[i] = 0;
      if (32 * i + lane < B) items(32 * i + lane, n[i], first[i]);
      if (n[i] > 0) top = max(top, flat ? first[i] : first[i] + n[i] - 1);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    auto at_least = [&](int level) {  // pieces of this level or above
      int c = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        c += flat ? (first[i] >= level ? n[i] : 0) : min(n[i], max(0, first[i] + n[i] - level));
      return __reduce_add_sync(0xffffffffu, c);
    };
    if (rank >= at_least(0)) return;
    int low = 0, high = top + 1;  // at_least(low) > rank >= at_least(high)
    while (high - low > 1) {
      const int mid = (low + high) / 2;
      if (at_least(mid) > rank) low = mid;
      else high = mid;
    }
    rank -= at_least(high);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int here = flat ? (first[i] == low ? n[i] : 0) : (low >= first[i] && low < first[i] + n[i] ? 1 : 0);
      int upto = here;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int other = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += other;
      }
      const bool mine = rank >= before + upto - here && rank < before + upto;
      const uint32_t who = __ballot_sync(0xffffffffu, mine);
      if (who) {
        const int src = __ffs(who) - 1;
        b = 32 * i + src;
        t = __shfl_sync(0xffffffffu, flat ? rank - (before + upto - here) : low - first[i], src);
        return;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return;
  }
  for (int base = 0; base < B; base += 32) {
    int n = 0, first = 0;
    if (base + lane < B) items(base + lane, n, first);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int other = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += other;
    }
    const bool mine = rank >= before + upto - n && rank < before + upto;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int src = __ffs(who) - 1;
      b = base + src;
      t = __shfl_sync(0xffffffffu, n - 1 - (rank - (before + upto - n)), src);
      return;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// The most pieces of `width` rows that B sequences of `total` rows together can have.
inline int64_t most_items(int64_t total, int64_t B, int64_t width) {
  return (total + B * (width - 1)) / width;
}

// Host: the checks that the calls share (argument struct fields as in fa.h).
int check_sizes(const char* who, int B, int Hq, int Hkv, int D, int total_q, int total_k, fa_dtype dtype,
                float scale);
// A [tokens, heads, D] tensor's address and strides (token, head; elements), for 16-byte accesses.
int check_tensor(const char* who, const char* name, const void* base, const int64_t* strides, int tokens,
                 int heads, int D);
// Tensor map over such a tensor, one box 64 columns x `heads` x `tokens` rows, head by head within
// a token; a tensor without rows gets a map that nothing reads.
bool encode_rows(CUtensorMap* map, bool bf16, const void* base, const int64_t* strides, int tokens, int heads,
                 int D, int box_tokens, int box_heads);

}  // namespace packed
}  // namespace fa
