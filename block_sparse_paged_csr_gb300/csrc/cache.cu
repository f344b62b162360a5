// Writing the paged K/V cache and the bounds of its blocks.
//
// sa_store_kv puts the rows of new tokens into the cache's pages, in any of
// the cache's types.  The 8-bit types hold a scale for each (page, kv head):
// s = 2^e, the smallest that brings the page's largest magnitude to the
// type's range, so that x / s and code * s are exact and only the rounding to
// a code loses anything.  A page that already holds rows of its sequence and
// gets a larger value takes the larger scale, and its old codes are rounded to
// it once (for e4m3 a power of two moves the exponent only, exact but for
// subnormal codes).
//
// sa_block_bounds takes the smallest and the largest key per channel of every
// block that holds a new token.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

enum CacheType { kF32 = 0, kBf16 = 1, kE4m3 = 2, kInt8 = 3 };

// ------------------------------------------------------------------ store

struct StoreArgs {
  const void* src[2];                  // K, V rows of the new tokens
  int64_t token_stride[2], head_stride[2];   // elements
  void* pages[2];
  float* scales[2];
  int64_t num_pages;
  const int32_t* block_tables;
  const int64_t* cu;
  const int32_t* used;
  int64_t tq, slots;
  int32_t batch, hkv, head_dim, page_size, max_pages;
  int64_t* status;
};

// 8 consecutive source elements as f32.
template <bool kSrcBf16>
__device__ __forceinline__ void load8(const void* src, int64_t off, float (&x)[8]) {
  if constexpr (kSrcBf16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + off));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// Largest magnitude's bits (they order like the magnitudes; infinities and NaN
// above every number).
__device__ __forceinline__ uint32_t amax_bits(uint32_t m, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}
// The same without infinities and NaN.
__device__ __forceinline__ uint32_t amax_finite(uint32_t m, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = max(m, u < 0x7F800000u ? u : 0u);
  }
  return m;
}

// The smallest power of two s >= 2^-126 with amax <= QMAX * s (0 for amax 0).
// QMAX = 448 = 1.75 * 2^8 (e4m3) or 127 = 1.984375 * 2^6 (int8): the exponent
// of amax less 8 or 6, one more where its mantissa lies above QMAX's.
template <int kType>
__device__ __forceinline__ float scale_of(uint32_t amax) {
  if (amax == 0u) return 0.f;
  const int e = static_cast<int>(amax >> 23) - (kType == kInt8 ? 6 : 8) +
                ((amax & 0x7FFFFFu) > (kType == kInt8 ? 0x7E0000u : 0x600000u) ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// x / s for the page's scale: by the exact reciprocal where s is a power of
// two (every scale this kernel makes), by division for a caller's own.  `plain`:
// a power of two and numbers only, so that nothing has to be looked at per
// element.
struct Quant {
  float s, inv;
  bool pow2, plain;
  __device__ __forceinline__ Quant(float scale, bool numbers) : s(scale) {
    const uint32_t u = __float_as_uint(scale);
    pow2 = (u & 0x7FFFFFu) == 0u && u != 0u;
    // 2^-e has the exponent field 254 - e; e = 254 (2^127) leaves the
    // subnormal 2^-127
    const uint32_t e = u >> 23;
    inv = pow2 ? (e < 254u ? __uint_as_float((254u - e) << 23) : __uint_as_float(0x00400000u)) : 0.f;
    plain = pow2 && numbers;
  }
  __device__ __forceinline__ float divided(float x) const {
    return s == 0.f ? (x == x ? 0.f : x) : (pow2 ? x * inv : __fdiv_rn(x, s));
  }
};

// Eight values to codes, round to nearest even, beyond the range to its end;
// NaN stays NaN in e4m3 and becomes 0 in int8.
template <int kType>
__device__ __forceinline__ uint2 to_codes8(const float (&x)[8], const Quant& q) {
  uint32_t c[4];
  if constexpr (kType == kE4m3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = q.plain ? x[2 * i] * q.inv : q.divided(x[2 * i]);
      const float x1 = q.plain ? x[2 * i + 1] * q.inv : q.divided(x[2 * i + 1]);
      uint16_t r;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
      c[i] = r;
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  } else {
    // 1.5 * 2^23 + v has the integer nearest to v (|v| < 2^22) in its low bits;
    // x inv is exact, so the one rounding is that of the addition
    uint32_t b[8];
    if (q.plain) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(x[i], q.inv, 12582912.f));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = q.divided(x[i]);
        b[i] = __float_as_uint(fminf(fmaxf(v == v ? v : 0.f, -127.f), 127.f) + 12582912.f);
      }
    }
    c[0] = __byte_perm(b[0], b[1], 0x0040);
    c[1] = __byte_perm(b[2], b[3], 0x0040);
    c[2] = __byte_perm(b[4], b[5], 0x0040);
    c[3] = __byte_perm(b[6], b[7], 0x0040);
    return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
  }
}

template <int kType>
__device__ __forceinline__ void store8(void* pages, int64_t off, const float (&x)[8],
                                       const Quant& qz) {
  if constexpr (kType == kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(pages) + off);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else if constexpr (kType == kBf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pages) + off) =
        make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]),
                   pack_bf16x2_rn(x[4], x[5]), pack_bf16x2_rn(x[6], x[7]));
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + off) = to_codes8<kType>(x, qz);
  }
}

// One item: the new rows of one (page, kv head) of K or of V, by a warp
// (kItemWarps = 1: decode steps, a row or a few) or by the whole CTA (prompts:
// up to a page of rows).  A thread takes 8 elements at a time and keeps its
// first kHeld pieces in registers between the pass that finds the largest
// magnitude and the pass that writes codes, so a page of 64 x 128 is read
// once.
//
// 7000 f32 rows of 8 heads of 128, K and V, to int8 (73 MB) take 22.6 us, 3.2 TB/s.
// Neither memory (33 %) nor the issue slots (48 %) are full: at 80 registers a third
// of the warps is resident, and they wait for their rows (long scoreboard first)
// and for the maximum before they may write.  Three CTAs per SM, as four leave
// too few registers for the pieces (23.6 us).  Single bf16 rows of 64 sequences
// (128 rows of K and V, 8 heads) to e4m3: 6 us, latency.
template <int kType, bool kSrcBf16, int kItemWarps>
__global__ void __launch_bounds__(kThreads, 3) store_kv_kernel(const StoreArgs a) {
  constexpr bool kCodes = kType == kE4m3 || kType == kInt8;
  constexpr int kT = kItemWarps * 32;                 // threads per item
  constexpr int kHeld = kItemWarps == 1 ? 2 : 4;
  __shared__ uint32_t s_amax[kWarps];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int t = kItemWarps == 1 ? lane : static_cast<int>(threadIdx.x);
  const int64_t item = kItemWarps == 1 ? static_cast<int64_t>(blockIdx.x) * kWarps + warp
                                       : static_cast<int64_t>(blockIdx.x);
  const int64_t u = item / (2 * a.hkv);
  const int rest = static_cast<int>(item - u * (2 * a.hkv));
  const int h = rest >> 1;
  const int kv = rest & 1;                            // 0: K, 1: V
  if (u >= a.slots) return;
  const int b = warp_slot_sequence(a.cu, a.batch, a.page_size, u, lane);
  const NewRange nr = new_range(a.cu, a.used, b, a.tq);
  const int64_t page0 = nr.p0 / a.page_size;
  const int64_t pg = page0 + (u - slot_base(a.cu[b], b, a.page_size));
  const int64_t base = pg * a.page_size;
  // (a sequence without new rows has p0 = p1, inside a page perhaps: another
  // sequence may be writing that page and its scale)
  if (nr.p0 >= nr.p1 || pg < page0 || base >= nr.p1 || pg >= a.max_pages) return;   // the whole item
  const int id = a.block_tables[static_cast<int64_t>(b) * a.max_pages + pg];
  if (id < 0 || id >= a.num_pages) {
    if (id >= 0 && t == 0) report(a.status, SA_ERR_SHAPE);
    return;
  }
  const int r0 = static_cast<int>(max(nr.p0 - base, int64_t{0}));
  const int r1 = static_cast<int>(min(nr.p1 - base, static_cast<int64_t>(a.page_size)));
  // the new tokens end at cu0 + (p1 - p0): a sequence shorter than its new
  // tokens stores the first of them
  const int64_t tok0 = nr.cu0 + (base + r0 - nr.p0);
  const int per_row = a.head_dim >> 3;                // 8-element pieces of a row
  const int n = (r1 - r0) * per_row;
  // the thread's piece i: row r and piece c of it, without a division per piece
  const int step_r = kT / per_row, step_c = kT - step_r * per_row;
  const int first_r = t / per_row, first_c = t - first_r * per_row;
  const void* src = a.src[kv];
  const int64_t ts = a.token_stride[kv];
  const int64_t src0 = tok0 * ts + h * a.head_stride[kv];
  void* pages = a.pages[kv];
  const int64_t dst0 = ((static_cast<int64_t>(id) * a.hkv + h) * a.page_size + r0) * a.head_dim;
  auto advance = [&](int& r, int& c) {
    r += step_r;
    c += step_c;
    if (c >= per_row) {
      c -= per_row;
      ++r;
    }
  };
  auto src_at = [&](int r, int c) -> int64_t { return src0 + r * ts + c * 8; };

  float held[kHeld][8];
  uint32_t m = 0;
  int r = first_r, c = first_c;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (t + j * kT < n) load8<kSrcBf16>(src, src_at(r, c), held[j]);
    advance(r, c);
  }
  const int next_r = r, next_c = c;                    // the first piece not held
  bool numbers = true;
  float* scale_at = nullptr;
  float s_old = 0.f;
  if constexpr (kCodes) {
    scale_at = a.scales[kv] + static_cast<int64_t>(id) * a.hkv + h;
    if (r0 > 0) {
      s_old = *scale_at;
      if (!(s_old > 0.f && s_old < INFINITY)) s_old = 0.f;
    }
    auto amax = [&](bool finite_only) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (t + j * kT < n) v = finite_only ? amax_finite(v, held[j]) : amax_bits(v, held[j]);
      int ar = next_r, ac = next_c;
      for (int i = t + kHeld * kT; i < n; i += kT) {
        float x[8];
        load8<kSrcBf16>(src, src_at(ar, ac), x);
        advance(ar, ac);
        v = finite_only ? amax_finite(v, x) : amax_bits(v, x);
      }
      v = __reduce_max_sync(0xffffffffu, v);
      if constexpr (kItemWarps > 1) {
        __syncthreads();
        if (lane == 0) s_amax[warp] = v;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kItemWarps; ++w) v = max(v, s_amax[w]);
      }
      return v;
    };
    m = amax(false);
    numbers = m < 0x7F800000u;
    if (!numbers) m = amax(true);                      // (the same for the whole item)
  }
  const float s_new = kCodes ? fmaxf(s_old, scale_of<kType>(m)) : 1.f;
  const Quant qz(s_new, numbers);
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (t + j * kT < n)
      store8<kType>(pages, dst0 + static_cast<int64_t>(t + j * kT) * 8, held[j], qz);
  r = next_r;
  c = next_c;
  for (int i = t + kHeld * kT; i < n; i += kT) {
    float x[8];
    load8<kSrcBf16>(src, src_at(r, c), x);
    advance(r, c);
    store8<kType>(pages, dst0 + static_cast<int64_t>(i) * 8, x, qz);
  }
  if constexpr (kCodes) {
    if (r0 > 0 && s_new > s_old) {
      // the page's earlier rows to the larger scale
      const float ratio = __fdiv_rn(s_old, s_new);
      // (NaN codes of e4m3 stay NaN; int8 codes are numbers)
      const Quant one(1.f, true);
      uint8_t* old = static_cast<uint8_t*>(pages) + dst0 - static_cast<int64_t>(r0) * a.head_dim;
      for (int i = t; i < r0 * per_row; i += kT) {
        const uint2 w = *reinterpret_cast<const uint2*>(old + static_cast<int64_t>(i) * 8);
        uint32_t f[4];
        codes4_to_f16<kType == kInt8>(w.x, f[0], f[1]);
        codes4_to_f16<kType == kInt8>(w.y, f[2], f[3]);
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = f16x2_to_f32(f[j]);
          x[2 * j] = v.x * ratio;
          x[2 * j + 1] = v.y * ratio;
        }
        store8<kType>(old, static_cast<int64_t>(i) * 8, x, one);
      }
    }
    // every thread of the item read the old scale before the reduction above
    if (t == 0) *scale_at = s_new;
  }
}

template <int kType, bool kSrcBf16>
cudaError_t launch_store(const StoreArgs& a, bool by_warp, cudaStream_t stream) {
  const int64_t items = a.slots * a.hkv * 2;
  const int64_t grid = by_warp ? (items + kWarps - 1) / kWarps : items;
  if (grid > 0x7FFFFFFF) return cudaErrorNotSupported;
  if (by_warp)
    store_kv_kernel<kType, kSrcBf16, 1><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  else
    store_kv_kernel<kType, kSrcBf16, kWarps>
        <<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int kType>
cudaError_t launch_store_src(const StoreArgs& a, bool src_bf16, bool by_warp, cudaStream_t s) {
  return src_bf16 ? launch_store<kType, true>(a, by_warp, s)
                  : launch_store<kType, false>(a, by_warp, s);
}

// ------------------------------------------------------------------ bounds

struct BoundsArgs {
  const void* k_pages;
  const float* k_scales;
  int64_t num_pages;
  const int32_t* block_tables;
  const int64_t* cu;
  const int32_t* used;
  const int32_t* bound_tables;
  int64_t num_bounds;
  uint16_t* bounds;                    // [num_bounds, hkv, 2, head_dim] bf16
  int64_t tq, slots;
  int32_t batch, hkv, head_dim, block_size, page_size, max_pages, msb;
  int64_t* status;
};

// Elements of a 16-byte piece.
template <int kType> struct Piece { static constexpr int n = kType == kF32 ? 4 : kType == kBf16 ? 8 : 16; };

// The pieces of a row are spread over P lanes (the power of two that holds
// them, at most 32), so a warp takes 32 / P rows side by side.
template <int kType>
__host__ __device__ constexpr int lanes_per_row(int head_dim) {
  const int n = head_dim / Piece<kType>::n;
  int p = 1;
  while (p < n && p < 32) p *= 2;
  return p;
}

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Codes' minima and maxima as f16 pairs (exact, two codes an instruction).  An
// int8 code v is held as 1152 + v, whose f16 bits are 0x6400 above the byte
// v + 128, until it is read.
template <bool kI8>
struct CodeRange {
  uint32_t lo[8], hi[8];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = 0x7C007C00u;
      hi[i] = 0xFC00FC00u;
    }
  }
  __device__ __forceinline__ void add(const uint4& w) {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t f[2];
      if constexpr (kI8) {
        const uint32_t u = ww[i] ^ 0x80808080u;
        f[0] = __byte_perm(u, 0x64646464u, 0x4140);
        f[1] = __byte_perm(u, 0x64646464u, 0x4342);
      } else {
        codes4_to_f16<false>(ww[i], f[0], f[1]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {                    // (NaN codes do not count)
        asm("min.f16x2 %0, %0, %1;" : "+r"(lo[2 * i + j]) : "r"(f[j]));
        asm("max.f16x2 %0, %0, %1;" : "+r"(hi[2 * i + j]) : "r"(f[j]));
      }
    }
  }
  static __device__ __forceinline__ float2 value(uint32_t u) {
    if constexpr (kI8) asm("sub.f16x2 %0, %0, %1;" : "+r"(u) : "r"(0x64806480u));
    return f16x2_to_f32(u);
  }
};

// One warp per (block, kv head): no barrier, no shared memory, and as many
// blocks in flight as registers allow, which is what both ends of the range
// need (single tokens: the chain of lookups before the first key; prompts:
// bytes in flight).  A lane takes one 16-byte piece of every (32 / P)-th row,
// kBatch loads in flight.  Minima and maxima of codes are taken as packed f16
// (exact) and meet the scale where the page changes; they are rounded outward to
// bf16 before lanes of the same channels meet (rounding is monotonic: the
// minimum of the rounded is the rounded minimum).  Reads each key once.
//   kInPage: a batch of loads never leaves a page (page_size a multiple of its
// rows), the usual case: one lookup per batch instead of one per load.
//
// 108 MB of int8 keys, 64-key pages, 128-key blocks: 33 us, 3.3 TB/s (60 us with a
// lookup per load and rounding at every page; two loads in flight 46 us, eight 33 us
// but slower single tokens).  Neither memory (43 %) nor the issue slots (52 %) are
// full: a third of the warps is resident (80 registers), four loads each, and long
// scoreboard is the first of their stalls.  A block of 64 keys for each of 128
// sequences, 8 heads, e4m3: 10 us, latency.
constexpr int kBatch = 4;

template <int kType, bool kInPage>
__global__ void __launch_bounds__(kThreads, 3) block_bounds_kernel(const BoundsArgs a) {
  constexpr int kN = Piece<kType>::n;
  constexpr bool kCodes = kType == kE4m3 || kType == kInt8;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const unsigned u = item / static_cast<unsigned>(a.hkv);
  const int h = static_cast<int>(item - u * static_cast<unsigned>(a.hkv));
  if (u >= a.slots) return;
  const int b = warp_slot_sequence(a.cu, a.batch, a.block_size, u, lane);
  const NewRange nr = new_range(a.cu, a.used, b, a.tq);
  // (positions fit 32 bits: lengths are int32)
  const unsigned blk0 = static_cast<unsigned>(nr.p0) / static_cast<unsigned>(a.block_size);
  const int64_t blk = blk0 + (static_cast<int64_t>(u) - slot_base(nr.cu0, b, a.block_size));
  const int64_t base = blk * a.block_size;
  if (blk < blk0 || base >= nr.p1 || nr.p0 >= nr.p1 || blk >= a.msb) return;
  const int d = a.head_dim;
  const int ps = a.page_size;
  const int ppb = a.block_size / ps;
  const int keys = static_cast<int>(min(nr.p1 - base, static_cast<int64_t>(a.block_size)));
  const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_pages;
  const int row = a.bound_tables[static_cast<int64_t>(b) * a.msb + blk];

  const int lanes = lanes_per_row<kType>(d);
  const int piece = lane & (lanes - 1);
  const int sub = lane / lanes;                        // the lane's row of a load
  const int rows = 32 / lanes;                         // rows per load
  const int lps = (ps & (ps - 1)) == 0 ? __ffs(ps) - 1 : -1;
  uint32_t* out =
      reinterpret_cast<uint32_t*>(a.bounds) + (static_cast<int64_t>(max(row, 0)) * a.hkv + h) * d;
  for (int c0 = 0; c0 < d; c0 += lanes * kN) {         // (rows of more than 32 pieces: in parts)
    const int ch = c0 + piece * kN;
    const bool mine = ch < d;
    uint32_t lo[kN / 2], hi[kN / 2];                   // bf16 pairs, rounded outward
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      lo[i] = 0x7F807F80u;
      hi[i] = 0xFF80FF80u;
    }
    for (int pg0 = 0; pg0 * ps < keys; pg0 += 32) {
      // 32 pages at a time: ids and scales, one per lane
      const int64_t pg = blk * ppb + pg0 + lane;
      int id_of = pg0 + lane < ppb && (pg0 + lane) * ps < keys && pg < a.max_pages ? bt[pg] : -1;
      if (id_of >= a.num_pages) {
        report(a.status, SA_ERR_SHAPE);
        id_of = -1;
      }
      float sc_of = 0.f;
      if constexpr (kCodes)
        sc_of = id_of >= 0 ? a.k_scales[static_cast<int64_t>(id_of) * a.hkv + h] : 0.f;
      const int r1 = min(keys, (pg0 + 32) * ps);
      int cur = -1;                                    // the lane's page at hand
      float sc = 0.f;
      CodeRange<kType == kInt8> cr;
      // The page's codes times its scale.  A code has at most 8 significant bits
      // and lies in 2^-9 .. 448, so its product with a power of two of this
      // range is a bf16 number; other products are rounded outward, from f32
      // rounded outward.  A negative scale of a caller's own makes the largest
      // code the smallest key.  (A NaN product, of a scale that is 0 and a
      // channel with NaN keys only, counts as no key.)
      auto close = [&]() {
        if constexpr (kCodes) {
          const bool exact = (__float_as_uint(sc) & 0x7FFFFFu) == 0u && sc >= 0x1p-120f && sc <= 0x1p100f;
          if (exact) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 l = cr.value(cr.lo[i]);
              const float2 m = cr.value(cr.hi[i]);
              lo[i] = min_bf16x2(lo[i], __byte_perm(__float_as_uint(l.x * sc),
                                                    __float_as_uint(l.y * sc), 0x7632));
              hi[i] = max_bf16x2(hi[i], __byte_perm(__float_as_uint(m.x * sc),
                                                    __float_as_uint(m.y * sc), 0x7632));
            }
          } else {
            const bool turned = sc < 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 l = cr.value(turned ? cr.hi[i] : cr.lo[i]);
              const float2 m = cr.value(turned ? cr.lo[i] : cr.hi[i]);
              lo[i] = min_bf16x2(lo[i], bf16_down(fminf(__fmul_rd(l.x, sc), INFINITY)) |
                                            (bf16_down(fminf(__fmul_rd(l.y, sc), INFINITY)) << 16));
              hi[i] = max_bf16x2(hi[i], bf16_up(fmaxf(__fmul_ru(m.x, sc), -INFINITY)) |
                                            (bf16_up(fmaxf(__fmul_ru(m.y, sc), -INFINITY)) << 16));
            }
          }
        }
      };
      // one load's keys; `page`, its page within the block, opens the page's range
      auto open = [&](int page, float scale) {
        if constexpr (kCodes) {
          if (page == cur) return;
          if (cur >= 0) close();
          cr.reset();
          cur = page;
          sc = scale;
        }
      };
      auto add = [&](const uint4& w) {
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        if constexpr (kCodes) {
          cr.add(w);
        } else if constexpr (kType == kBf16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = min_bf16x2(lo[i], ww[i]);
            hi[i] = max_bf16x2(hi[i], ww[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x0 = __uint_as_float(ww[2 * i]), x1 = __uint_as_float(ww[2 * i + 1]);
            // (NaN keys do not count)
            lo[i] = min_bf16x2(lo[i], bf16_down(fminf(x0, INFINITY)) |
                                          (bf16_down(fminf(x1, INFINITY)) << 16));
            hi[i] = max_bf16x2(hi[i], bf16_up(fmaxf(x0, -INFINITY)) |
                                          (bf16_up(fmaxf(x1, -INFINITY)) << 16));
          }
        }
      };
      for (int k0 = pg0 * ps; k0 < r1; k0 += kBatch * rows) {
        uint4 w[kBatch];
        if constexpr (kInPage) {
          const int p = lps >= 0 ? k0 >> lps : k0 / ps;
          const int page = __shfl_sync(0xffffffffu, id_of, p - pg0);
          const float scale = kCodes ? __shfl_sync(0xffffffffu, sc_of, p - pg0) : 0.f;
          if (page < 0 || !mine) continue;
          const unsigned char* at =
              static_cast<const unsigned char*>(a.k_pages) +
              (((static_cast<int64_t>(page) * a.hkv + h) * ps + (k0 - p * ps)) * d + ch) * (16 / kN);
          const int last = r1 - 1 - k0;                // (behind it: a row that counts already)
#pragma unroll
          for (int t = 0; t < kBatch; ++t)
            w[t] = __ldg(reinterpret_cast<const uint4*>(
                at + min(t * rows + sub, last) * (d * (16 / kN))));
          open(p, scale);
#pragma unroll
          for (int t = 0; t < kBatch; ++t) add(w[t]);
        } else {
          int pw[kBatch];
#pragma unroll
          for (int t = 0; t < kBatch; ++t) {
            const int r = k0 + t * rows + sub;
            const int p = min(lps >= 0 ? r >> lps : r / ps, pg0 + 31);
            const int page = __shfl_sync(0xffffffffu, id_of, p - pg0);
            pw[t] = r < r1 && page >= 0 && mine ? p : -1;
            if (pw[t] >= 0)
              w[t] = __ldg(reinterpret_cast<const uint4*>(
                  static_cast<const unsigned char*>(a.k_pages) +
                  (((static_cast<int64_t>(page) * a.hkv + h) * ps + (r - p * ps)) * d + ch) *
                      (16 / kN)));
          }
#pragma unroll
          for (int t = 0; t < kBatch; ++t) {
            const float scale =
                kCodes ? __shfl_sync(0xffffffffu, sc_of, max(pw[t] - pg0, 0)) : 0.f;
            if (pw[t] < 0) continue;
            open(pw[t], scale);
            add(w[t]);
          }
        }
      }
      if constexpr (kCodes) {
        if (cur >= 0) close();
      }
    }
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      for (int o = lanes; o < 32; o <<= 1) {
        lo[i] = min_bf16x2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
        hi[i] = max_bf16x2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
      }
    }
    if (sub == 0 && mine && row >= 0 && row < a.num_bounds) {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        out[ch / 2 + i] = lo[i];
        out[d / 2 + ch / 2 + i] = hi[i];
      }
    }
  }
  if (row >= a.num_bounds && lane == 0) report(a.status, SA_ERR_SHAPE);
}

template <int kType>
cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t stream) {
  const int64_t grid = a.slots * a.hkv;
  if (grid > 0x7FFFFFFF) return cudaErrorNotSupported;
  const unsigned ctas = static_cast<unsigned>((grid + kWarps - 1) / kWarps);
  if (a.page_size % (kBatch * 32 / lanes_per_row<kType>(a.head_dim)) == 0)
    block_bounds_kernel<kType, true><<<ctas, kThreads, 0, stream>>>(a);
  else
    block_bounds_kernel<kType, false><<<ctas, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ checks

bool known_type(sa_dtype t) { return t >= SA_DTYPE_F32 && t <= SA_DTYPE_INT8; }

}  // namespace

}  // namespace sa

extern "C" {

sa_status sa_store_kv(const void* k, const void* v, sa_dtype src_dtype, int64_t k_token_stride,
                      int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                      void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                      int64_t num_pages, sa_dtype kv_dtype, const int32_t* block_tables,
                      int32_t max_pages, const int64_t* cu_seqlens_q_host,
                      const int64_t* cu_seqlens_q, int32_t batch, int64_t tq,
                      const int32_t* used_kv_lens, int32_t hkv, int32_t head_dim,
                      int32_t page_size, int64_t* status, void* stream) {
  if (hkv <= 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0 || page_size <= 0) return SA_ERR_BLOCK_PAGE;
  sa_status st = sa::check_lengths(cu_seqlens_q_host, batch, tq);
  if (st != SA_OK) return st;
  if (num_pages < 0 || max_pages < 0) return SA_ERR_SHAPE;
  if (src_dtype != SA_DTYPE_F32 && src_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
  if (!sa::known_type(kv_dtype)) return SA_ERR_INVALID_ARGUMENT;
  if (head_dim % (sa::eight_bit(kv_dtype) ? 16 : 8) != 0 || head_dim > 256)
    return SA_ERR_UNSUPPORTED;
  if (tq == 0) return SA_OK;
  if (!k || !v || !k_pages || !v_pages || !block_tables || !cu_seqlens_q || !used_kv_lens)
    return SA_ERR_INVALID_ARGUMENT;
  if (sa::eight_bit(kv_dtype) && (!k_scales || !v_scales)) return SA_ERR_INVALID_ARGUMENT;
  if (!sa::aligned16(k) || !sa::aligned16(v) || !sa::aligned16(k_pages) || !sa::aligned16(v_pages))
    return SA_ERR_INVALID_ARGUMENT;
  const int64_t unit = src_dtype == SA_DTYPE_BF16 ? 8 : 4;      // elements of 16 bytes
  if (k_token_stride % unit || k_head_stride % unit || v_token_stride % unit ||
      v_head_stride % unit)
    return SA_ERR_INVALID_ARGUMENT;

  sa::StoreArgs a{};
  a.src[0] = k;
  a.src[1] = v;
  a.token_stride[0] = k_token_stride;
  a.token_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  a.pages[0] = k_pages;
  a.pages[1] = v_pages;
  a.scales[0] = k_scales;
  a.scales[1] = v_scales;
  a.num_pages = num_pages;
  a.block_tables = block_tables;
  a.cu = cu_seqlens_q;
  a.used = used_kv_lens;
  a.tq = tq;
  a.slots = sa::slot_base(tq, batch, page_size);
  a.batch = batch;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.status = status;
  int64_t longest = 0;
  for (int32_t b = 0; b < batch; ++b)
    longest = std::max(longest, cu_seqlens_q_host[b + 1] - cu_seqlens_q_host[b]);
  // A warp per item while an item is at most sixteen 8-element pieces a lane: 7000
  // f32 rows of 8 heads of 128 to int8 take 18.5 us by warps and 61 us by CTAs with
  // pages of 16, 18 and 35 us with pages of 32, 20.5 and 22.6 us with pages of 64, 58
  // and 20.6 us with pages of 256; 28000 rows 69 and 123 us with pages of 32, 90 and
  // 74 us with pages of 64; one prompt of 1000 rows 10 and 8 us with pages of 32, 16
  // and 6 us with pages of 64.
  const int64_t rows = std::min<int64_t>(longest, page_size);
  const bool by_warp = rows * head_dim <= 32 * 16 * 8;
  const bool bf = src_dtype == SA_DTYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (kv_dtype) {
    case SA_DTYPE_F32: err = sa::launch_store_src<sa::kF32>(a, bf, by_warp, s); break;
    case SA_DTYPE_BF16: err = sa::launch_store_src<sa::kBf16>(a, bf, by_warp, s); break;
    case SA_DTYPE_E4M3: err = sa::launch_store_src<sa::kE4m3>(a, bf, by_warp, s); break;
    default: err = sa::launch_store_src<sa::kInt8>(a, bf, by_warp, s); break;
  }
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_block_bounds(const void* k_pages, const float* k_scales, int64_t num_pages,
                          sa_dtype kv_dtype, const int32_t* block_tables, int32_t max_pages,
                          const int64_t* cu_seqlens_q_host, const int64_t* cu_seqlens_q,
                          int32_t batch, int64_t tq, const int32_t* used_kv_lens, int32_t hkv,
                          int32_t head_dim, int32_t block_size, int32_t page_size,
                          const int32_t* bound_tables, int32_t msb, int64_t num_bounds,
                          void* bounds, int64_t* status, void* stream) {
  if (hkv <= 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0 || block_size <= 0 || page_size <= 0 || block_size % page_size != 0)
    return SA_ERR_BLOCK_PAGE;
  sa_status st = sa::check_lengths(cu_seqlens_q_host, batch, tq);
  if (st != SA_OK) return st;
  if (num_pages < 0 || max_pages < 0 || msb < 0 || num_bounds < 0) return SA_ERR_SHAPE;
  if (!sa::known_type(kv_dtype)) return SA_ERR_INVALID_ARGUMENT;
  if (head_dim % (sa::eight_bit(kv_dtype) ? 16 : 8) != 0 || head_dim > 256)
    return SA_ERR_UNSUPPORTED;
  if (tq == 0) return SA_OK;
  if (!k_pages || !block_tables || !cu_seqlens_q || !used_kv_lens || !bound_tables || !bounds)
    return SA_ERR_INVALID_ARGUMENT;
  if (sa::eight_bit(kv_dtype) && !k_scales) return SA_ERR_INVALID_ARGUMENT;
  if (!sa::aligned16(k_pages) || !sa::aligned16(bounds)) return SA_ERR_INVALID_ARGUMENT;

  sa::BoundsArgs a{};
  a.k_pages = k_pages;
  a.k_scales = k_scales;
  a.num_pages = num_pages;
  a.block_tables = block_tables;
  a.cu = cu_seqlens_q;
  a.used = used_kv_lens;
  a.bound_tables = bound_tables;
  a.num_bounds = num_bounds;
  a.bounds = static_cast<uint16_t*>(bounds);
  a.tq = tq;
  a.slots = sa::slot_base(tq, batch, block_size);
  a.batch = batch;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.msb = msb;
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (kv_dtype) {
    case SA_DTYPE_F32: err = sa::launch_bounds<sa::kF32>(a, s); break;
    case SA_DTYPE_BF16: err = sa::launch_bounds<sa::kBf16>(a, s); break;
    case SA_DTYPE_E4M3: err = sa::launch_bounds<sa::kE4m3>(a, s); break;
    default: err = sa::launch_bounds<sa::kInt8>(a, s); break;
  }
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
