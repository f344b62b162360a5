// Helpers shared by the kernels that write the paged cache, take block bounds
// and select blocks: the sequence behind a work slot, 8-bit codes, ordered
// bf16 roundings.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sa_common.cuh"

namespace sa {

// Work slots over the tokens of a batch, cut into pieces of `per` positions
// (a page, a block): sequence b owns the slots [base(b), base(b + 1)) with
// base(b) = cu[b] / per + 2 b.  Its new positions touch at most
// floor(qo / per) + 2 pieces whatever their alignment, and base grows by at
// least that much, so every touched piece has a slot although the lengths
// live on the device; slots past a sequence's pieces stay idle.
__host__ __device__ __forceinline__ int64_t slot_base(int64_t cu_b, int64_t b, int per) {
#ifdef __CUDA_ARCH__
  // (a 64-bit division costs some 100 instructions; token counts rarely need it)
  if (cu_b >= 0 && cu_b < (int64_t{1} << 32))
    return static_cast<int64_t>(static_cast<uint32_t>(cu_b) / static_cast<uint32_t>(per)) + 2 * b;
#endif
  return cu_b / per + 2 * b;
}

// The largest b in [0, n) with before(b), which holds for 0 and up to some b: 32
// candidates per round.  All lanes of the warp call it.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int lane, F before) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int cand = lo + lane * step;
    const bool le = cand < hi && before(cand);
    const unsigned bal = __ballot_sync(0xffffffffu, le);   // lane 0 (cand = lo) always set
    const int last = bal ? 31 - __clz(bal) : 0;
    const int nlo = lo + last * step;
    hi = min(nlo + step, hi);
    lo = nlo;
  }
  return lo;
}

// The sequence that owns slot u (the largest b with base(b) <= u): u / 2 where
// few tokens precede it (decode batches: no search), else a search.  All lanes of
// the warp call it.
__device__ __forceinline__ int warp_slot_sequence(const int64_t* cu, int batch, int per,
                                                  int64_t u, int lane) {
  const int guess = static_cast<int>(min(u / 2, static_cast<int64_t>(batch - 1)));
  const int64_t g0 = cu[guess], g1 = cu[guess + 1];
  if (slot_base(g0, guess, per) <= u && (guess + 1 == batch || u < slot_base(g1, guess + 1, per)))
    return guess;
  return warp_search(batch, lane, [&](int b) { return slot_base(cu[b], b, per) <= u; });
}

// The new positions [p0, p1) of sequence b: right-aligned at its length lk
// (its qo new tokens end at lk); a sequence shorter than its new tokens takes
// the first lk of them.
struct NewRange {
  int64_t cu0;        // index of the sequence's first new token
  int64_t p0, p1;     // positions
};

__device__ __forceinline__ NewRange new_range(const int64_t* cu, const int32_t* used, int b,
                                              int64_t tq) {
  NewRange r;
  const int64_t lk = max(used[b], 0);
  r.cu0 = min(max(cu[b], int64_t{0}), tq);
  const int64_t end = min(max(cu[b + 1], r.cu0), tq);
  const int64_t qo = end - r.cu0;
  r.p0 = lk >= qo ? lk - qo : 0;
  r.p1 = lk;
  return r;
}

// int8: a byte b with its sign bit flipped, below the f16 exponent byte 0x64,
// is the f16 number 1024 + (b + 128); subtracting 1152 leaves b.
// `lo_sel` picks the two bytes: 0x4140 bytes 0 and 1, 0x4342 bytes 2 and 3.
__device__ __forceinline__ uint32_t int8x2_to_f16x2(uint32_t four_flipped, uint32_t lo_sel) {
  uint32_t r, d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(four_flipped), "r"(0x64646464u), "r"(lo_sel));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(r), "r"(0x64806480u));
  return d;
}

// Four codes (one 32-bit word) to two packed f16 pairs (exact for both types;
// e4m3 by the hardware conversion).
template <bool kInt8>
__device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kInt8) {
    const uint32_t f = w ^ 0x80808080u;
    lo = int8x2_to_f16x2(f, 0x4140u);
    hi = int8x2_to_f16x2(f, 0x4342u);
  } else {
    // (the 16-bit halves are operands of the conversion as they are)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// f32 to bf16 bits, rounded down (to -inf) or up (to +inf).
__device__ __forceinline__ uint32_t bf16_down(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 16) + ((u & 0xFFFFu) != 0u && (u >> 31) != 0u ? 1u : 0u);
}
__device__ __forceinline__ uint32_t bf16_up(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 16) + ((u & 0xFFFFu) != 0u && (u >> 31) == 0u ? 1u : 0u);
}

}  // namespace sa
