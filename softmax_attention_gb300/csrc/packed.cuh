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
  // forward, keys split: normalised partial outputs [total_q, Hq, splits, D] and their lse
  int splits;
  float* o_part;
  float* lse_part;
  uint32_t* status;
  uint64_t wait_ns;      // see mbar_wait below
};

// Waits of these kernels.  Some last as long as a work item: for its last tile, or until the next one is
// asked for.  An item walks over all of a sequence's tiles, so with the longest sequences it takes seconds (a query
// tile over 400,000,000 keys: 3), and the limit grows with the tiles that there can be: 20 us each, where one takes
// 1 to 3.
using fa::mbar_wait;
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const Params& p) {
  return fa::mbar_wait(bar, parity, p.status, p.wait_ns);
}

inline uint64_t wait_limit(int total_q, int total_k, int q_per_tile) {
  const uint64_t q = static_cast<uint64_t>(total_q) / q_per_tile, k = static_cast<uint64_t>(total_k) / kKeys;
  return kWaitLimitNs + 20000 * (q > k ? q : k);
}

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
// its level is first(s) + t, or first(s) for all pieces where `flat`.  The pieces are taken in
// decreasing level over all sequences, dealt out to the blocks there and back (block i of n takes the
// ranks i, 2n-1-i, 2n+i, ...), so that every block gets about the same work and the last pieces are
// short ones; nothing but the order depends on it.  Each block finds its pieces by itself: a binary
// search for a rank's level, a warp's lanes holding up to four sequences each, a few hundred
// clocks in a warp with nothing else to do; no list, no kernel before this one.  Past 128 sequences
// the pieces are taken sequence by sequence, each search going on where the block's last one ended.
class Finder {
 public:
  template <typename Items>
  __device__ __forceinline__ Finder(int B, bool flat, Items items) : B_(B), flat_(flat), top_(0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      n_[i] = first_[i] = 0;
      if (B <= 32 * kHeld && 32 * i + lane < B) items(32 * i + lane, n_[i], first_[i]);
      if (n_[i] > 0) top_ = max(top_, flat ? first_[i] : first_[i] + n_[i] - 1);
    }
    top_ = __reduce_max_sync(0xffffffffu, top_);
  }

  // The piece of a rank, larger from call to call: sequence b and index t; b = -1 past the end.  The whole warp calls.
  template <typename Items>
  __device__ __forceinline__ void find(int rank, Items items, int& b, int& t) {
    const int lane = threadIdx.x & 31;
    b = -1;
    t = 0;
    int before = 0;  // pieces in front of those looked at
    if (B_ <= 32 * kHeld) {
      if (rank >= at_least(0)) return;
      int low = 0, high = top_ + 1;  // at_least(low) > rank >= at_least(high)
      while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (at_least(mid) > rank) low = mid;
        else high = mid;
      }
      rank -= at_least(high);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int here = flat_ ? (first_[i] == low ? n_[i] : 0) : (low >= first_[i] && low < first_[i] + n_[i] ? 1 : 0);
        if (pick(rank, before, here, 32 * i, flat_, low - first_[i], b, t)) return;
      }
      return;
    }
    for (; base_ < B_; base_ += 32) {
      int n = 0, first = 0;
      if (base_ + lane < B_) items(base_ + lane, n, first);
      before = before_;
      if (pick(rank, before, n, base_, true, 0, b, t)) {
        t = __shfl_sync(0xffffffffu, n, b - base_) - 1 - t;  // the longest first
        return;
      }
      before_ = before;
    }
  }

 private:
  static constexpr int kHeld = 4;

  __device__ __forceinline__ int at_least(int level) const {  // pieces of this level or above
    int c = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      c += flat_ ? (first_[i] >= level ? n_[i] : 0) : min(n_[i], max(0, first_[i] + n_[i] - level));
    return __reduce_add_sync(0xffffffffu, c);
  }

  // Lanes hold the counts `here` of 32 sequences from `base`; if the rank falls among them, its
  // sequence and its place there (`count`), or that lane's `index`.
  static __device__ __forceinline__ bool pick(int rank, int& before, int here, int base, bool count, int index, int& b,
                                              int& t) {
    const int lane = threadIdx.x & 31;
    int upto = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int other = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += other;
    }
    const int from = before + upto - here;
    const uint32_t who = __ballot_sync(0xffffffffu, rank >= from && rank < from + here);
    before += __shfl_sync(0xffffffffu, upto, 31);
    if (!who) return false;
    const int src = __ffs(who) - 1;
    b = base + src;
    t = __shfl_sync(0xffffffffu, count ? rank - from : index, src);
    return true;
  }

  int B_;
  bool flat_;
  int top_;
  int n_[kHeld], first_[kHeld];  // of sequences lane, lane + 32, ...
  int base_ = 0, before_ = 0;    // more sequences than that: those looked at last, and the pieces in front of them
};

// The k-th rank of this block, of `blocks` that deal them out there and back.
__device__ __forceinline__ int dealt(int k) {
  const int n = gridDim.x, i = blockIdx.x;
  return k * n + ((k & 1) ? n - 1 - i : i);
}

// One work item, as the scheduling warp hands it to the others through shared memory.
struct Item {
  Seq seq;
  int at;    // first query, or key, of the piece in its sequence; -1: no more work
  int head;  // kv head
  int split; // forward: part of the keys
  float value; // dq, fp16: the largest finite |v| of its keys
};

// A value that is the same in every lane, in a form that the compiler knows to be: the operands of
// tcgen05.mma are uniform registers, and what it cannot prove uniform is moved there before every
// product, beside softmax warps that leave an issuing warp few slots.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Waits of a whole warp for two barriers.  A look at a barrier takes some 150 clocks even when it has come
// true: both looks are on their way together.
__device__ __forceinline__ bool warp_wait(uint32_t a, int phase_a, uint32_t b, int phase_b, const Params& p) {
  const bool first = mbar_test_wait(a, phase_a & 1), second = mbar_test_wait(b, phase_b & 1);
  return __all_sync(0xffffffffu, (first || mbar_wait(a, phase_a & 1, p)) && (second || mbar_wait(b, phase_b & 1, p)));
}

// True in one lane of the warp, always the same.  (An election, not a lane's number: the compiler then
// keeps the code behind it on uniform registers.)
__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// The most pieces of `width` rows that B sequences of `total` rows together can have.
inline int64_t most_items(int64_t total, int64_t B, int64_t width) {
  return (total + B * (width - 1)) / width;
}

// Host: the checks that the calls share (argument struct fields as in fa.h).
int check_sizes(const char* who, int B, int Hq, int Hkv, int D, int total_q, int total_k, fa_dtype dtype,
                float scale);
int check_offsets(const char* who, const int32_t* cu_q, const int32_t* cu_k);
// A [tokens, heads, D] tensor's address and strides (token, head; elements), for 16-byte accesses.
int check_tensor(const char* who, const char* name, const void* base, const int64_t* strides, int tokens,
                 int heads, int D);
// Tensor map over such a tensor, one box 64 columns x `heads` x `tokens` rows, head by head within
// a token; a tensor without rows gets a map that nothing reads.
bool encode_rows(CUtensorMap* map, bool bf16, const void* base, const int64_t* strides, int tokens, int heads,
                 int D, int box_tokens, int box_heads);

}  // namespace packed
}  // namespace fa
