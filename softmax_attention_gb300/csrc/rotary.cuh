// rotary.cuh -- what the kernels that turn rows by their positions share: rows in registers, and
// the angles.
//
// A row (one token of one head) is cut into units of 16 elements, one thread each:
//   - the rotated part, half layout: columns [8u, 8u+8) and [half + 8u, half + 8u+8), so that
//     one thread holds both members of its eight pairs (and may write in place);
//   - everything else: the 16 consecutive columns of the unit.
#pragma once

#include "cache.cuh"

namespace fa {

constexpr int kMaxRot = 512;

// ------------------------------------------------------------------------------------------
// Sixteen-bit and fp32 rows in registers: eight elements.
// ------------------------------------------------------------------------------------------
// As loaded (so that a batch of loads in flight holds no more registers than its bytes).
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* src) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4*>(src)[i];
  return r;
}

template <typename T>
__device__ __forceinline__ void expand8(const Raw8<T>& r, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<T>(w[i], x[2 * i], x[2 * i + 1]);
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
  expand8<T>(load_raw8<T>(src), x);
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]),
                                                pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
  }
}

// ------------------------------------------------------------------------------------------
// Angles.  theta = position * f, needed modulo one turn to fp32 precision at any int32
// position.  The step of one position is held as a 64-bit fraction of a turn, so position *
// step modulo 2^64 is the exact phase (an integer product that wraps), and only its top 32 bits
// go to the sine.  fp64 arithmetic, slow on this part, is spent once a block and frequency:
// f / 2 pi carries a relative error of 2^-53, which at position 2^20 and f = 1 is 2^-35 turns.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ int64_t phase_step(double f) {
  const double turns = f * 0.15915494309189533577;  // 1 / (2 pi)
  const double frac = turns - rint(turns);          // [-0.5, 0.5]
  return __double2ll_rn(frac * 18446744073709551616.0);
}

__device__ __forceinline__ void angle(int64_t step, int pos, float amplitude, float& c, float& s) {
  const uint64_t phase = static_cast<uint64_t>(step) * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;
  sincospif(half_turns, &s, &c);
  s *= amplitude;
  c *= amplitude;
}

__device__ __forceinline__ void fill_steps(int64_t* steps, const double* inv_freq, int half) {
  for (int i = threadIdx.x; i < half; i += blockDim.x) steps[i] = phase_step(inv_freq[i]);
  __syncthreads();
}

// The angles of a thread's unit: W pairs, eight here (a kernel of its own may cut rows into smaller units).
template <int W>
struct Angles {
  float c[W], s[W];
};
using Turn = Angles<8>;

// Unit u of the rotated part: half layout pairs (W u + i, half + W u + i), pair index W u + i;
// interleaved pairs (2 W u + 2i, 2 W u + 2i + 1), the same pair index.
template <int W>
__device__ __forceinline__ void fill_turn(Angles<W>& t, const int64_t* steps, int u, int pos,
                                          float amplitude, bool transpose) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    angle(steps[W * u + i], pos, amplitude, t.c[i], t.s[i]);
    if (transpose) t.s[i] = -t.s[i];
  }
}

// Rotates a unit's 2 W elements: half layout a = first members, b = second; interleaved a, b =
// the 2 W consecutive elements.
template <bool INTERLEAVED, int W>
__device__ __forceinline__ void rotate(const Angles<W>& t, float (&a)[W], float (&b)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float& x = INTERLEAVED ? (2 * i < W ? a[(2 * i) % W] : b[(2 * i) % W]) : a[i];
    float& y = INTERLEAVED ? (2 * i < W ? a[(2 * i + 1) % W] : b[(2 * i + 1) % W]) : b[i];
    const float rx = x * t.c[i] - y * t.s[i];
    const float ry = y * t.c[i] + x * t.s[i];
    x = rx;
    y = ry;
  }
}

}  // namespace fa
