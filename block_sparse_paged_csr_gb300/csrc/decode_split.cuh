// Attention of one new token per sequence over its whole paged cache, split over the
// cache's length.  Instances per cache type are in decode_f32.cu, decode_bf16.cu,
// decode_e4m3.cu and decode_int8.cu; decode.cu holds the entry point.
//
// One query row per q-head against n keys: every byte of K and V is used once for the
// few lanes of its kv head, so the floor is the cache's bytes.  The work is a flat
// list of tiles (sequence, kv head, lane group, kKT keys), cut into equal ranges,
// one per warp of a grid of one CTA per SM: whatever the batch and the lengths,
// every warp streams as many bytes as the others.  The lengths live on the device, so
// each CTA counts the tiles itself (one pass over the lengths).
//
// A warp is on its own while it streams: its lanes copy rows of K and V (16 bytes a lane
// and copy) into a ring of its own, look up pages one tile ahead, and its MMAs
// run an online softmax over the tiles.  No barrier is crossed, and no wait can hang.
// A (sequence, kv head) pair that lies whole in a warp's range is written by it; parts
// of pairs meet in the CTA (the last part of each warp through shared memory, one that
// a warp began with through the workspace), and those that cross CTAs in a second
// kernel, always in the order of the keys, so that results do not depend on timing.
#pragma once

#include <cfloat>
#include <cstdint>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {
namespace dec1 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The softmax's reference m is a whole number (log2 domain) that moves only for a
// score more than kSlack above it, so that rescaling is exact and rare.  Over 8 bits what
// meets V's codes is P times the scale of their page in two f16 parts, and o keeps a reference
// n of its own, which follows the largest such product: it moves up when m does or when
// a page's vs 2^(m - n) is above kRoom, to where the product counts 2^kTop (below
// kRoom no P of at most 2^kSlack makes a product above 2^15; f16 ends at 2^16).
constexpr float kSlack = 7.f, kTop = 4.f, kRoom = 256.f;

constexpr int kInfos = 4;            // tiles that are copied or in use at a time, at most

template <int T> struct TypeOf;
template <> struct TypeOf<SA_DTYPE_F32> { static constexpr int size = 4; };
template <> struct TypeOf<SA_DTYPE_BF16> { static constexpr int size = 2; };
template <> struct TypeOf<SA_DTYPE_E4M3> { static constexpr int size = 1; };
template <> struct TypeOf<SA_DTYPE_INT8> { static constexpr int size = 1; };

// T: the cache's type.  DP: head_dim rounded up to 64, 128 or 256 (channels behind it
// are zeros).  R: query rows of a tile, 8 or 16.  B: bf16 queries, whose Q has fewer
// parts (f32 caches take both types as they come).
template <int T, int DP, int R, bool B>
struct Cfg {
  static constexpr int kSize = TypeOf<T>::size;
  static constexpr bool kF32 = T == SA_DTYPE_F32;
  static constexpr bool k8 = kSize == 1;
  static constexpr int kRow = DP * kSize;                       // bytes of a row in the ring
  // keys of a tile: 4 KB of K where that is 8 to 32 keys
  static constexpr int kKT = 4096 / kRow < 8 ? 8 : 4096 / kRow > 32 ? 32 : 4096 / kRow;
  static constexpr int kRun = kKT < 16 ? kKT : 16;              // rows that mostly lie in one page
  static constexpr int kEntry = kKT * kRow;                     // bytes of a tile's K (or V)
  static constexpr int kNCH = kRow / 16;                        // 16-byte chunks of a row
  static constexpr int kLCH = kNCH / 4;                         // chunks of a row that a lane reads for S
  static constexpr int kEC = 16 / kSize;                        // elements of a chunk
  static constexpr int kKPC = k8 ? 4 : 2;                       // k-steps of a chunk
  static constexpr int kKS = kLCH * kKPC;                       // k-steps of a row
  static constexpr int kNT = kKT / 8;                           // n-tiles of S
  static constexpr int kKK = kF32 || kKT == 8 ? 8 : 16;         // keys of one P V k-step
  static constexpr int kVP = DP * kSize / 8 < 16 ? 8 : 16;      // bytes of a V row that a lane reads at a time
  static constexpr int kEP = kVP / kSize;                       // .. channels
  static constexpr int kNS = DP / (8 * kEP);                    // .. times
  static constexpr int kNJ = DP / 8;                            // n-tiles of o
  static constexpr int kNR = R / 8;                             // query rows of a lane
  static constexpr int kOW = 2 * kNR;                           // numbers of o of an n-tile
  // operands of Q kept per k-step (see keep_q), and of P
  static constexpr int kQP = kF32 ? 1 : k8 ? (R == 8 || B ? 1 : 2) : B ? 1 : R == 8 ? 2 : 3;
  static constexpr int kPP = kF32 ? 1 : k8 || kKK == 8 ? R / 8 : R == 8 ? 2 : 3;
  // (the third parts of R = 8 leave half of their operand zero, which is not stored)
  static constexpr bool kHalfQ = !kF32 && !k8 && R == 8 && !B;
  static constexpr int kQBytes = kF32 ? kKS / 2 * 512 : kHalfQ ? kKS * 768 : kKS * kQP * 512;
  static constexpr int kScales = k8 ? kKT * 4 : 0;              // bytes of an entry's scales
  // The ring's entries hold K and V in turn: one in use, two in flight.  (A fourth costs
  // warps, and where it costs none it gains nothing: bf16, 32 sequences of 20000 to 50000 keys, 8
  // warps: 719 us with three, 736 with four.)
  static constexpr int kNE = 3;
  static constexpr int kPerWarp = kNE * (kEntry + kScales) + kQBytes + kInfos * 16;
  static constexpr int kMost = 220 * 1024;                      // (of 227 KB, some of them static)
  // Warps hide the instructions' latencies from each other (bf16 queries, int8, 32 sequences of 20000
  // to 50000 keys: 12 warps 405 us, 8 warps 446; e4m3 with heads of 64: 16 warps 426, 12 475, 8 575).
  // Their number is a multiple of 4, as their ranges are equal and the four schedulers
  // share them (10 warps instead of 12: 1130 instead of 750 us).  bf16 keys ask for
  // few instructions; there more copies at a time only cost (64 sequences: 12 warps 732 us, 8 726).
  static constexpr int kWarpsMost = T == SA_DTYPE_BF16 ? 8 : decode_max_warps(DP, R);
  static constexpr int kWarpsSmem = kMost / kPerWarp / 4 * 4;
  static constexpr int kW = kWarpsSmem < kWarpsMost ? kWarpsSmem : kWarpsMost;      // warps
  // An SM does best with some 64 KB in flight.  Where two entries a warp would be more, V's copies
  // wait until the tile before is done with (e4m3, 64 sequences, 12 warps: 743 us, at once 755).
  static constexpr bool kLate = 2 * kW * kEntry > 64 * 1024;
  static constexpr int kThreads = 32 * kW;
  static constexpr int kSmem = kW * kPerWarp;
  // a state: o in the order of the accumulators, then m, n and l of each row
  static constexpr int kNel = R * DP;
  static constexpr int kState = kNel + 3 * R;
  static_assert(kState * 4 <= kNE * kEntry + kQBytes, "a warp's last state replaces its ring");
  static_assert(kW >= 4 && kState <= decode_state_floats(DP, R), "workspace");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^d for a whole number d up to 127 (0 below -126; some number for NaN, the difference of
// two references of nothing).
__device__ __forceinline__ float pow2_of(float d) {
  return d < -126.f ? 0.f
                    : __uint_as_float(static_cast<uint32_t>(static_cast<int>(fminf(d, 127.f)) + 127) << 23);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  const int n = there ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d += a b: m16n8k16 on f16 or bf16, m16n8k8 on tf32 (which reads the upper 19 bits).
template <int T>
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (T == SA_DTYPE_F32)
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else if constexpr (T == SA_DTYPE_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The same over 8 keys for bf16 (m16n8k8).
__device__ __forceinline__ void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// (x, y) += (a, b), one instruction.
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// (x, y) += (a, b) f, one instruction.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float f) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "mov.b64 r, {%4, %4};\n\tfma.rn.f32x2 p, q, r, p;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(f));
}

// f32 as a tf32 high part (cut) and the rest, rounded to tf32's 11 bits: 2^-21 of x
// is lost at most.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}
// Two values as f16 high parts and remainders (22 bits together).
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
  const float2 h = f16x2_to_f32(hi);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x1 - h.y), "f"(x0 - h.x));
}
// The same with the remainders times 1 / kRest: they stay in f16's normal range as long as the value
// is above 2^-25 (and below 2^15), and end at 2^-36 of the unit instead of 2^-25.
constexpr float kRest = 0x1p-11f;
__device__ __forceinline__ void split_f16_apart(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
  const float2 h = f16x2_to_f32(hi);
  float a = x0, b = x1, c = 0.f, d = 0.f;
  fma2(a, b, h.x, h.y, -1.f);
  fma2(c, d, a, b, 1.f / kRest);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(d), "f"(c));
}
// Two values as three bf16 parts (24 bits together).
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& mid,
                                           uint32_t& lo) {
  hi = pack_bf16x2_rn(x0, x1);
  const float r0 = x0 - __uint_as_float(hi << 16), r1 = x1 - __uint_as_float(hi & 0xFFFF0000u);
  mid = pack_bf16x2_rn(r0, r1);
  lo = pack_bf16x2_rn(r0 - __uint_as_float(mid << 16), r1 - __uint_as_float(mid & 0xFFFF0000u));
}

// The keys of a sequence that its query sees: [first, end).
struct Keys {
  int first, end;
};
__device__ __forceinline__ Keys keys_of(const DecodeArgs& a, int used) {
  Keys k;
  used = max(used, 0);
  k.end = min(used, a.capacity);
  // (a length may stand far past the table: a window that begins behind it holds no keys, and
  // positions stay far from 2^31)
  k.first = a.window > 0 ? min(max(used - a.window, 0), k.end) : 0;
  return k;
}
template <int KT>
__device__ __forceinline__ int tiles_of(const Keys& k) {
  return max((k.end - k.first + KT - 1) / KT, 1);             // a sequence without keys has one, of none
}

// x / y for x >= 0 (a 64-bit division is long, and rarely needed).
__device__ __forceinline__ int64_t divide(int64_t x, unsigned y) {
  return (x >> 32) == 0 ? static_cast<int64_t>(static_cast<unsigned>(x) / y) : x / y;
}

// An item: (sequence b, kv head h, lane group).  Its first query row and their number.
struct Item {
  int64_t row0;
  int rows;
};
template <int R>
__device__ __forceinline__ Item item_of(const DecodeArgs& a, int item) {
  const int b = item / a.items_per_seq, rest = item - b * a.items_per_seq;
  const int h = rest / a.groups, grp = rest - h * a.groups;
  return {static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(h) * a.qhead + grp * R,
          min(R, a.qhead - grp * R)};
}

template <int T, int DP, int R, bool B>
struct Worker {
  using C = Cfg<T, DP, R, B>;

  const DecodeArgs& a;
  unsigned char* ring;           // this warp's [kNE][kEntry]
  unsigned char* qf;             // Q's operands
  float* sc;                     // [kNE][kKT] scales
  uint4* info;                   // [kInfos]: item, live keys, flags
  int lane, g, c;

  // ---- the tile to come: where it lies
  int b, h, t, nt, first, end, next_used;     // cursor
  bool runs;                     // pages hold whole runs of kRun rows, and rows are not padded
  struct Pend {
    int pid, row, h, item;
    uint32_t flags;              // 1: the pair's first tile, 2: its last, 4: runs of rows lie in a page
  };

  // ---- state of the piece at hand
  float o[C::kNJ][C::kOW];       // columns 2 c, + 1 of row g, then of row g + 8
  float m_run[C::kNR], n_run[C::kNR], l_part[C::kNR], vfac[C::kNR], sfac[C::kNR];
  bool clamp;                    // some V scale is beyond kRoom

  __device__ __forceinline__ void seek(int b0, int64_t in_seq) {
    b = b0;
    const Keys k = keys_of(a, a.used[b]);
    first = k.first;
    end = k.end;
    nt = tiles_of<C::kKT>(k);
    h = static_cast<int>(min(divide(in_seq, static_cast<unsigned>(nt)),
                             static_cast<int64_t>(a.items_per_seq - 1)));
    t = min(static_cast<int>(in_seq - static_cast<int64_t>(h) * nt), nt - 1);
    next_used = b + 1 < a.batch ? a.used[b + 1] : 0;
  }

  // The cursor's tile: its page ids are asked for here and used a tile later.
  __device__ __forceinline__ Pend take() {
    Pend p;
    const int key = first + t * C::kKT + (lane & (C::kKT - 1));
    p.pid = -1;
    p.row = 0;
    if (key < end) {
      const int pg = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
      p.row = key - pg * a.page_size;
      p.pid = a.block_tables[static_cast<int64_t>(b) * a.max_pages + pg];
    }
    p.h = a.groups == 1 ? h : h / a.groups;
    p.item = b * a.items_per_seq + h;
    p.flags = (t == 0 ? 1u : 0u) | (t + 1 == nt ? 2u : 0u) | (runs && first % C::kRun == 0 ? 4u : 0u);
    if (++t == nt) {
      t = 0;
      if (++h == a.items_per_seq) {
        h = 0;
        if (++b < a.batch) {
          const Keys k = keys_of(a, next_used);
          first = k.first;
          end = k.end;
          nt = tiles_of<C::kKT>(k);
          if (b + 1 < a.batch) next_used = a.used[b + 1];
        } else {
          b = a.batch - 1;         // (only if the lengths change under the call: stay in bounds)
        }
      }
    }
    return p;
  }

  // Copies of one tile's K (kV false) or V rows into entry e; row: the lane's (key
  // `lane`) row of the pool, kNone where there is none (the pools have fewer rows).
  // whole: all rows are there, and every kRun of them lie side by side, so that one address serves
  // a run (a tenth of a tile's instructions less).
  static constexpr uint32_t kNone = 0xFFFFFFFFu;
  template <bool kV>
  __device__ __forceinline__ void copy_rows(int e, uint32_t row, uint32_t scale_at, bool whole) {
    const unsigned char* pool = static_cast<const unsigned char*>(kV ? a.v_pages : a.k_pages);
    const uint32_t d0 = smem_u32(ring + e * C::kEntry);
    // a lane copies chunk lane % kNCH (and + 32 ..) of rows that are 32 / kNCH apart
    constexpr int kPer = C::kNCH < 32 ? C::kNCH : 32;
    const int ch0 = lane & (kPer - 1);
    if (whole) {
      constexpr int kCopies = C::kRun * C::kNCH / 32;          // of a run
#pragma unroll
      for (int run = 0; run < C::kKT / C::kRun; ++run) {
        const uint32_t at = __shfl_sync(0xffffffffu, row, run * C::kRun);
        const unsigned char* src = pool + static_cast<uint64_t>(at) * C::kRow + 16 * lane;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int j = run * kCopies + i;
          const int r = C::kNCH <= 32 ? j * (32 / kPer) + lane / kPer : j / (C::kNCH / 32);
          const int ch = C::kNCH <= 32 ? ch0 : ch0 + 32 * (j % (C::kNCH / 32));
          const int phys = C::kNCH >= 8 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3);
          copy16(d0 + r * C::kRow + phys * 16, src + 512 * i);
        }
      }
      if constexpr (C::k8) {
        if (C::kKT == 32 || lane < C::kKT)
          copy4(smem_u32(sc + e * C::kKT + lane), (kV ? a.v_scales : a.k_scales) + scale_at, true);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < C::kKT * C::kNCH / 32; ++i) {
      const int r = C::kNCH <= 32 ? i * (32 / kPer) + lane / kPer : i / (C::kNCH / 32);
      const int ch = C::kNCH <= 32 ? ch0 : ch0 + 32 * (i % (C::kNCH / 32));
      const uint32_t at = __shfl_sync(0xffffffffu, row, r);
      const bool there = at != kNone && 16 * ch < a.row_bytes;
      const int phys = C::kNCH >= 8 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3);
      const unsigned char* src =
          pool + (there ? static_cast<uint64_t>(at) * static_cast<uint32_t>(a.row_bytes) + 16u * ch : 0);
      copy16(d0 + r * C::kRow + phys * 16, src, there);
    }
    if constexpr (C::k8) {
      if (C::kKT == 32 || lane < C::kKT) {
        const bool there = row != kNone;
        copy4(smem_u32(sc + e * C::kKT + lane), (kV ? a.v_scales : a.k_scales) + (there ? scale_at : 0u),
              there);
      }
    }
  }

  // Q's operands for an item, in the order in which the k-steps use them: lane (g, c)
  // holds row g (and g + 8) at the channels of the chunks that it reads of K's rows.
  //   8 bits: the row, scaled by a power of two into f16's range, as f16 high
  //     parts and remainders; bf16: three bf16 parts (bf16 queries: the first says all);
  //     f32: as they are, split into tf32 parts where they are used (12 operations per 16
  //     products, and half the room, which lets 12 warps in instead of 8).
  //   R = 8: rows g + 8 of the MMA's tile carry the second parts of rows g, so that they
  //     cost no product.
  // fetch_q asks for the rows, keep_q lays them out: between them other loads start.
  static constexpr int kQ4 = C::kLCH * C::kEC / 4;  // groups of 4 channels of a row that a lane holds
  struct Rows {
    uint4 x[C::kNR][kQ4];                           // f32, or bf16 in the first two words
  };
  __device__ __forceinline__ int q_channel(int i) const {
    return chunk(i / (C::kEC / 4)) * C::kEC + 4 * (i % (C::kEC / 4));
  }
  __device__ __forceinline__ void fetch_q(int item, Rows& q) const {
    const Item it = item_of<R>(a, item);
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      const bool there = g + 8 * r < it.rows;
      const int64_t at = (it.row0 + g + 8 * r) * a.head_dim;
#pragma unroll
      for (int i = 0; i < kQ4; ++i) {
        q.x[r][i] = make_uint4(0u, 0u, 0u, 0u);
        if (there && q_channel(i) < a.head_dim) {
          if (a.act_bf16) {
            const uint2 u =
                *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at + q_channel(i));
            q.x[r][i].x = u.x;
            q.x[r][i].y = u.y;
          } else {
            q.x[r][i] =
                *reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at + q_channel(i));
          }
        }
      }
    }
  }
  __device__ __forceinline__ void keep_q(const Rows& q) {
    __syncwarp();
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      float4 x[kQ4];
#pragma unroll
      for (int i = 0; i < kQ4; ++i)
        x[i] = a.act_bf16 ? bf16x4_to_f32(make_uint2(q.x[r][i].x, q.x[r][i].y))
                          : make_float4(__uint_as_float(q.x[r][i].x), __uint_as_float(q.x[r][i].y),
                                        __uint_as_float(q.x[r][i].z), __uint_as_float(q.x[r][i].w));
      float f = 1.f;
      sfac[r] = a.scale * kLog2e;
      if constexpr (C::k8) {
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < kQ4; ++i)
          am = fmaxf(am, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // largest magnitude to [2^10, 2^11): f and 1 / f kept normal
        const int ex = min(max(static_cast<int>(__float_as_uint(am) >> 23), 11), 253);
        f = __uint_as_float(static_cast<uint32_t>(264 - ex) << 23);
        sfac[r] *= __uint_as_float(static_cast<uint32_t>(ex - 10) << 23);
      }
      uint4* out = reinterpret_cast<uint4*>(qf) + lane;
#pragma unroll
      for (int i = 0; i < kQ4; ++i) {
        if constexpr (C::kF32) {
          out[32 * i] = make_uint4(__float_as_uint(x[i].x), __float_as_uint(x[i].y),
                                   __float_as_uint(x[i].z), __float_as_uint(x[i].w));
        } else {
          uint4* to = out + 32 * C::kQP * i;
          uint32_t hi[2], mid[2], lo[2] = {0u, 0u};
          if constexpr (C::k8) {
            split_f16(x[i].x * f, x[i].y * f, hi[0], mid[0]);
            split_f16(x[i].z * f, x[i].w * f, hi[1], mid[1]);
          } else {
            split_bf16(x[i].x, x[i].y, hi[0], mid[0], lo[0]);
            split_bf16(x[i].z, x[i].w, hi[1], mid[1], lo[1]);
          }
          if constexpr (R == 8) {
            if constexpr (C::kHalfQ) {
              out[32 * i] = make_uint4(hi[0], mid[0], hi[1], mid[1]);
              reinterpret_cast<uint2*>(qf + C::kKS * 512)[32 * i + lane] = make_uint2(lo[0], lo[1]);
            } else {
              to[0] = make_uint4(hi[0], mid[0], hi[1], mid[1]);
            }
          } else {
            uint32_t* w = reinterpret_cast<uint32_t*>(to) + r;
            w[0] = hi[0];
            w[2] = hi[1];
            if constexpr (C::kQP >= 2) {
              w[128] = mid[0];
              w[130] = mid[1];
            }
            if constexpr (C::kQP >= 3) {
              w[256] = lo[0];
              w[258] = lo[1];
            }
          }
        }
      }
    }
    __syncwarp();
  }

  // The chunks of a row that lane c reads for the scores: with the ring's XOR by
  // the row, eight lanes of a 16-byte read meet eight different groups of banks.
  __device__ __forceinline__ int chunk(int l) const {
    return C::kNCH == 4 ? c : 8 * (l >> 1) + 2 * c + (l & 1);
  }

  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      m_run[r] = n_run[r] = -INFINITY;
      vfac[r] = 1.f;
      l_part[r] = 0.f;
    }
    clamp = false;
#pragma unroll
    for (int j = 0; j < C::kNJ; ++j)
#pragma unroll
      for (int e = 0; e < C::kOW; ++e) o[j][e] = 0.f;
  }

  // S = Q K^T of the tile in entry e: acc[nt][i] (row g: keys 8 nt + 2 c, + 1; then row g +
  // 8).  A fragment's k index may stand for any channel as long as both operands agree,
  // so K's rows go from the ring to the MMA as they lie.  kf: the keys' scales.
  __device__ __forceinline__ void scores(int e, float (&acc)[C::kNT][4], float2 (&kf)[C::kNT]) {
    const unsigned char* kt = ring + e * C::kEntry + g * C::kRow;
    const uint4* q = reinterpret_cast<const uint4*>(qf) + lane;
    float low[C::kF32 ? C::kNT : 1][4];
#pragma unroll
    for (int n = 0; n < C::kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    if constexpr (C::kF32) {
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) low[n][i] = 0.f;
    }
#pragma unroll
    for (int l = 0; l < C::kLCH; ++l) {
      const int phys = C::kNCH >= 8 ? chunk(l) ^ g : chunk(l) ^ ((g >> 1) & 3);
      uint4 kr[C::kNT], qr;
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
        kr[n] = *reinterpret_cast<const uint4*>(kt + n * 8 * C::kRow + phys * 16);
#pragma unroll
      for (int s = 0; s < C::kKPC; ++s) {
        uint4 q0, q1, q2;
        const uint4* at = q + 32 * C::kQP * (l * C::kKPC + s);
        if constexpr (C::kF32) {
          if (s == 0) qr = q[32 * l];
          split_tf32(__uint_as_float(s ? qr.z : qr.x), q0.x, q0.y);
          split_tf32(__uint_as_float(s ? qr.w : qr.y), q0.z, q0.w);
        } else if constexpr (C::kHalfQ) {
          q0 = q[32 * (l * C::kKPC + s)];
          const uint2 low = reinterpret_cast<const uint2*>(qf + C::kKS * 512)[32 * (l * C::kKPC + s) + lane];
          q1 = make_uint4(low.x, 0u, low.y, 0u);
        } else {
          q0 = at[0];
        }
        if constexpr (C::kQP >= 2 && !C::kHalfQ) q1 = at[32];
        if constexpr (C::kQP >= 3) q2 = at[64];
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          const uint32_t w[4] = {kr[n].x, kr[n].y, kr[n].z, kr[n].w};
          uint32_t b0, b1;
          if constexpr (C::k8) {
            codes4_to_f16<T == SA_DTYPE_INT8>(w[s], b0, b1);
          } else if constexpr (C::kF32) {
            uint32_t l0, l1;
            split_tf32(__uint_as_float(w[2 * s]), b0, l0);
            split_tf32(__uint_as_float(w[2 * s + 1]), b1, l1);
            mma<T>(low[n], q0, l0, l1);
          } else {
            b0 = w[2 * s];
            b1 = w[2 * s + 1];
          }
          mma<T>(acc[n], q0, b0, b1);
          if constexpr (C::kQP >= 2) mma<T>(acc[n], q1, b0, b1);
          if constexpr (C::kQP >= 3) mma<T>(acc[n], q2, b0, b1);
        }
      }
    }
    if constexpr (C::kF32) {
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += low[n][i];
    }
    if constexpr (C::k8) {
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
        kf[n] = *reinterpret_cast<const float2*>(sc + e * C::kKT + 8 * n + 2 * c);
    }
  }

  // The online softmax of a tile whose V is in entry e: p (row g + 8 r, key 8 n + 2 c + i:
  // p[n][2 r + i]) from acc.  mask: which of the tile's keys there are (others count 0).
  __device__ __forceinline__ void softmax(int e, uint32_t mask, float (&acc)[C::kNT][4],
                                          const float2 (&kf)[C::kNT], float (&p)[C::kNT][2 * C::kNR]) {
    const float* vs = sc + e * C::kKT;
    constexpr uint32_t kAll = C::kKT == 32 ? 0xFFFFFFFFu : (1u << (C::kKT & 31)) - 1u;
    float most = -INFINITY;
    if constexpr (R == 8 && !B) {
#pragma unroll
      for (int n = 0; n < C::kNT; ++n) {                     // the remainders' row joins its own
        acc[n][0] += acc[n][2];
        acc[n][1] += acc[n][3];
      }
    }
    auto factor = [&](int n, int i) {
      const float f = sfac[i >> 1];
      if constexpr (C::k8) return f * (i & 1 ? kf[n].y : kf[n].x);
      return f;
    };
    auto missing = [&]() {
      if (mask != kAll) {
#pragma unroll
        for (int n = 0; n < C::kNT; ++n)
#pragma unroll
          for (int i = 0; i < 2 * C::kNR; ++i)
            if (!((mask >> (8 * n + 2 * c + (i & 1))) & 1u)) p[n][i] = -INFINITY;
      }
    };
#pragma unroll
    for (int n = 0; n < C::kNT; ++n)
#pragma unroll
      for (int i = 0; i < 2 * C::kNR; ++i)
        p[n][i] = fmaf(acc[n][i], factor(n, i), -m_run[i >> 1]);   // (m = -inf before the first keys)
    missing();
#pragma unroll
    for (int n = 0; n < C::kNT; ++n)
#pragma unroll
      for (int i = 0; i < 2 * C::kNR; ++i) most = fmaxf(most, p[n][i]);
    bool beyond = most > kSlack;
    if constexpr (C::k8) {
      float vm = 0.f, vf = vfac[0];
#pragma unroll
      for (int n = 0; n < C::kNT; ++n) {
        const float2 v = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c);
        vm = fmaxf(vm, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
#pragma unroll
      for (int r = 1; r < C::kNR; ++r) vf = fmaxf(vf, vfac[r]);
      beyond = beyond || vm * vf > kRoom;
    }
    clamp = false;
    if (__any_sync(0xffffffffu, beyond)) {
      clamp = true;
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int i = 0; i < 2 * C::kNR; ++i) p[n][i] = acc[n][i] * factor(n, i);
      missing();
#pragma unroll
      for (int r = 0; r < C::kNR; ++r) {
        float cm = -INFINITY, top = -INFINITY;               // largest score, largest product
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          cm = fmaxf(cm, fmaxf(p[n][2 * r], p[n][2 * r + 1]));
          if constexpr (C::k8) {
            const float2 v = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c);
            top = fmaxf(top, fmaxf(p[n][2 * r] + log2f(fabsf(v.x)), p[n][2 * r + 1] + log2f(fabsf(v.y))));
          }
        }
        cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 1));
        cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 2));
        const float m_new = fmaxf(m_run[r], ceilf(cm));
        float n_new = m_new;
        if constexpr (C::k8) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // (pages of zeros only: the lowest n whose 2^(m - n) is a number)
          n_new = fmaxf(fmaxf(n_run[r], ceilf(top) - kTop), m_new - 127.f);
          vfac[r] = pow2_of(m_new - n_new);
        }
        l_part[r] *= pow2_of(m_run[r] - m_new);
        const float beta = pow2_of(n_run[r] - n_new);
        m_run[r] = m_new;
        n_run[r] = n_new;
#pragma unroll
        for (int j = 0; j < C::kNJ; ++j)
#pragma unroll
          for (int i = 0; i < C::kOW; ++i)
            if (i / 2 == r) o[j][i] *= beta;
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          p[n][2 * r] -= m_new;
          p[n][2 * r + 1] -= m_new;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          p[n][2 * r + i] = ex2(p[n][2 * r + i]);
          sum += p[n][2 * r + i];
        }
      l_part[r] += sum;
    }
  }

  // o += P V.  V's rows too go to the MMA as they lie: n index of n-tile kEP s + i stands
  // for channel 8 kEP s + kEP n + i.
  // A tile's products are summed by the tensor cores from zero and added to o by rounding
  // additions.  The tensor cores cut a sum to 24 bits, so that an o that runs through them is
  // cut at every step, always towards zero: 1.4e-5 over 64 sequences of 4096 to 32768 bf16 keys
  // (6e-7 with the additions), 2.4e-4 over 1700 tiles of 8 bits a warp.
  // Over 8 bits what P vs loses to f16 stays in a second part, 2^11 times as large (see
  // split_f16_apart): with 8 rows in rows g + 8, with 16 in products of its own.  Together with the
  // additions this costs bf16 queries, whose output hides less, 0 to 4 % with 8 q-heads a kv head and
  // 21 to 24 % with 16 (32 sequences of 20000 to 50000 keys, heads of 128, without / with:
  // e4m3 374 / 373 and 401 / 498 us, int8 388 / 405 and 463 / 561).
  __device__ __forceinline__ void values(int e, const float (&p)[C::kNT][2 * C::kNR]) {
    constexpr int kK = C::kKT / C::kKK;            // k-steps of the tile
    const unsigned char* vt = ring + e * C::kEntry;
    const float* vs = sc + e * C::kKT;
    uint4 pa[kK][C::kPP];
#pragma unroll
    for (int kt = 0; kt < kK; ++kt) {
      if constexpr (C::kF32) {
        split_tf32(p[kt][0], pa[kt][0].x, pa[kt][0].y);
        split_tf32(p[kt][1], pa[kt][0].z, pa[kt][0].w);
      } else {
        constexpr int kX = C::kKK / 8;
        uint32_t hi[C::kNR][2] = {}, mid[C::kNR][2] = {}, lo[C::kNR][2] = {};
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          const int n = kX * kt + x;
          float2 vf = make_float2(1.f, 1.f);
          if constexpr (C::k8) vf = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c);
#pragma unroll
          for (int r = 0; r < C::kNR; ++r) {
            float p0 = p[n][2 * r], p1 = p[n][2 * r + 1];
            if constexpr (C::k8) {
              float f0 = vf.x * vfac[r], f1 = vf.y * vfac[r];
              if (clamp) {
                // (numbers: a page far above the others' scales may pass f32's range where its keys'
                // P is 0)
                f0 = fminf(fmaxf(f0, -FLT_MAX), FLT_MAX);
                f1 = fminf(fmaxf(f1, -FLT_MAX), FLT_MAX);
              }
              split_f16_apart(p0 * f0, p1 * f1, hi[r][x], mid[r][x]);
            } else {
              split_bf16(p0, p1, hi[r][x], mid[r][x], lo[r][x]);
            }
          }
        }
        if constexpr (C::kKK == 8) {
          // a step of 8 keys fills half the depth of the MMA: two parts of P lie side by side in it, over
          // the same rows of V (48 sequences, 4096 keys of 2 heads of 256: 84 us, with a product of
          // its own for the third part 93)
          if constexpr (R == 8) {
            pa[kt][0] = make_uint4(hi[0][0], mid[0][0], lo[0][0], 0u);
          } else {
            pa[kt][0] = make_uint4(hi[0][0], hi[1][0], 0u, 0u);
            pa[kt][1] = make_uint4(mid[0][0], mid[1][0], lo[0][0], lo[1][0]);
          }
        } else if constexpr (R == 8) {
          pa[kt][0] = make_uint4(hi[0][0], mid[0][0], hi[0][1], mid[0][1]);
          if constexpr (C::kPP == 2) pa[kt][1] = make_uint4(lo[0][0], 0u, lo[0][1], 0u);
        } else {
          pa[kt][0] = make_uint4(hi[0][0], hi[1][0], hi[0][1], hi[1][1]);
          if constexpr (C::kPP >= 2) pa[kt][1] = make_uint4(mid[0][0], mid[1][0], mid[0][1], mid[1][1]);
          if constexpr (C::kPP >= 3) pa[kt][2] = make_uint4(lo[0][0], lo[1][0], lo[0][1], lo[1][1]);
        }
      }
    }
    // rows of V that a lane reads per k-step
    constexpr int kVR = C::kKK == 16 ? 4 : 2;
    constexpr int kWords = C::kVP / 4;
#pragma unroll
    for (int s = 0; s < C::kNS; ++s) {
      uint32_t y[kK][kVR][kWords];
#pragma unroll
      for (int kt = 0; kt < kK; ++kt)
#pragma unroll
        for (int x = 0; x < kVR; ++x) {
          const int row = C::kKK * kt + 2 * c + (x & 1) + 8 * (x >> 1);
          const int sw = C::kNCH >= 8 ? row & 7 : (row >> 1) & 3;
          if constexpr (C::kVP == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(vt + row * C::kRow + (((8 * s + g) ^ sw) << 4));
            y[kt][x][0] = u.x;
            y[kt][x][1] = u.y;
            y[kt][x][2] = u.z;
            y[kt][x][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vt + row * C::kRow + (((g >> 1) ^ sw) << 4) +
                                                            8 * (g & 1));
            y[kt][x][0] = u.x;
            y[kt][x][1] = u.y;
          }
        }
#pragma unroll
      for (int q = 0; q < kWords; ++q) {
        constexpr int kPer = C::k8 ? 4 : C::kF32 ? 1 : 2;      // channels of a word
        float sum[kPer][4], rest[kPer][4];                     // (rest: over 8 bits with 16 rows)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) sum[i][x] = rest[i][x] = 0.f;
        if constexpr (C::kF32) {
#pragma unroll
          for (int kt = 0; kt < kK; ++kt) {
            const auto& v = y[kt];
            uint32_t h0, l0, h1, l1;
            split_tf32(__uint_as_float(v[0][q]), h0, l0);
            split_tf32(__uint_as_float(v[1][q]), h1, l1);
            mma<T>(sum[0], pa[kt][0], l0, l1);
            mma<T>(sum[0], pa[kt][0], h0, h1);
          }
        } else {
          uint32_t b[kK][kPer][2];
#pragma unroll
          for (int kt = 0; kt < kK; ++kt) {
            const auto& v = y[kt];
            if constexpr (C::k8) {
              constexpr bool kI8 = T == SA_DTYPE_INT8;
              codes4_to_f16<kI8>(__byte_perm(v[0][q], v[1][q], 0x5140), b[kt][0][0], b[kt][1][0]);
              codes4_to_f16<kI8>(__byte_perm(v[0][q], v[1][q], 0x7362), b[kt][2][0], b[kt][3][0]);
              codes4_to_f16<kI8>(__byte_perm(v[2][q], v[3][q], 0x5140), b[kt][0][1], b[kt][1][1]);
              codes4_to_f16<kI8>(__byte_perm(v[2][q], v[3][q], 0x7362), b[kt][2][1], b[kt][3][1]);
            } else {
              b[kt][0][0] = __byte_perm(v[0][q], v[1][q], 0x5410);
              b[kt][1][0] = __byte_perm(v[0][q], v[1][q], 0x7632);
              if constexpr (kVR == 4) {
                b[kt][0][1] = __byte_perm(v[2][q], v[3][q], 0x5410);
                b[kt][1][1] = __byte_perm(v[2][q], v[3][q], 0x7632);
              }
            }
          }
          // products of one channel after the other where the remainders ride along (32 sequences, heads of
          // 64, e4m3 under f32 queries: 443 us, the other way 463), of a word's channels side by side where
          // they have their own (16 q-heads a kv head, e4m3 under bf16 queries: 498 us, 523)
          constexpr int kSide = R == 16 ? kPer : 1;
#pragma unroll
          for (int i0 = 0; i0 < kPer; i0 += kSide)
#pragma unroll
            for (int x = C::kPP - 1; x >= 0; --x)                // (small parts first)
#pragma unroll
              for (int kt = 0; kt < kK; ++kt)
#pragma unroll
                for (int i = i0; i < i0 + kSide; ++i) {
                  float (&to)[4] = C::k8 && x > 0 ? rest[i] : sum[i];
                  if constexpr (C::kKK == 8 && R == 16) {
                    if (x == 0)
                      mma_k8(to, pa[kt][0].x, pa[kt][0].y, b[kt][i][0]);
                    else
                      mma<T>(to, pa[kt][x], b[kt][i][0], b[kt][i][0]);
                  } else {
                    mma<T>(to, pa[kt][x], b[kt][i][0], b[kt][i][C::kKK == 8 ? 0 : 1]);
                  }
                }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int j = C::kEP * s + kPer * q + i;
          if constexpr (R == 8) {                              // the remainders' row joins its own
            if constexpr (C::k8)
              fma2(sum[i][0], sum[i][1], sum[i][2], sum[i][3], kRest);
            else
              add2(sum[i][0], sum[i][1], sum[i][2], sum[i][3]);
            add2(o[j][0], o[j][1], sum[i][0], sum[i][1]);
          } else {
            if constexpr (C::k8) {
              fma2(sum[i][0], sum[i][1], rest[i][0], rest[i][1], kRest);
              fma2(sum[i][2], sum[i][3], rest[i][2], rest[i][3], kRest);
            }
            add2(o[j][0], o[j][1], sum[i][0], sum[i][1]);
            add2(o[j][2], o[j][3], sum[i][2], sum[i][3]);
          }
        }
      }
    }
  }

  __device__ __forceinline__ float at(int j, int r, int e) const {
    return o[j][2 * r + e];
  }
  __device__ __forceinline__ float row_sum(int r) const {
    float l = l_part[r];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    return l;
  }

  // The piece is a whole pair: its rows of the output.
  __device__ __forceinline__ void write_out(int item) {
    const Item it = item_of<R>(a, item);
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      const float l = row_sum(r);
      const int row = g + 8 * r;
      if (row >= it.rows) continue;
      const float2 f = out_factors(m_run[r], n_run[r], l);
      const int64_t out0 = (it.row0 + row) * a.head_dim;
#pragma unroll
      for (int s = 0; s < C::kNS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < C::kEP; i += 4) {
            const int ch = 8 * C::kEP * s + C::kEP * (2 * c + e) + i, j = C::kEP * s + i;
            if (ch < a.head_dim)
              store_o4(a.out, a.act_bf16, out0 + ch,
                       make_float4(at(j, r, e) * f.x * f.y, at(j + 1, r, e) * f.x * f.y,
                                   at(j + 2, r, e) * f.x * f.y, at(j + 3, r, e) * f.x * f.y));
          }
      if (c == 0 && a.lse) a.lse[it.row0 + row] = row_lse(m_run[r], l);
    }
  }
  // From o's unit 2^n to l's, 2^m, and through l, in two halves: rows with scales near the
  // ends of f32's range stay inside it.
  static __device__ __forceinline__ float2 out_factors(float m, float n, float l) {
    if (l == 0.f) return make_float2(0.f, 0.f);
    const float half = truncf(0.5f * (n - m));
    return make_float2(pow2_of(half), pow2_of(n - m - half) / l);
  }
  static __device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }

  // The state joined by another piece's (see dump).
  __device__ __forceinline__ void absorb(const float* from) {
    float f_own[C::kNR], f_other[C::kNR];
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      const float* s = from + C::kNel + g + 8 * r;
      const float m = s[0], n = s[R], l = s[2 * R];
      const float mm = fmaxf(m_run[r], m), nn = fmaxf(n_run[r], n);
      f_own[r] = pow2_of(n_run[r] - nn);
      f_other[r] = pow2_of(n - nn);
      l_part[r] = l_part[r] * pow2_of(m_run[r] - mm) + (c == 0 ? l * pow2_of(m - mm) : 0.f);
      m_run[r] = mm;
      n_run[r] = nn;
    }
#pragma unroll
    for (int j = 0; j < C::kNJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < C::kNR; ++r) {
          const float v = from[((2 * j + e) * C::kNR + r) * 32 + lane];
          const float sum = fmaf(f_other[r], v, f_own[r] * at(j, r, e));
          o[j][2 * r + e] = sum;
        }
  }

  // One element of a merged row: lane ln's, of n-tile and column je = (j, e).
  static __device__ __forceinline__ void write_element(const DecodeArgs& a, int64_t row, int ln, int je,
                                                       float sum, float m, float n, float l) {
    const int j = je >> 1, e = je & 1;
    const int ch = 8 * C::kEP * (j / C::kEP) + C::kEP * (2 * (ln & 3) + e) + j % C::kEP;
    const float2 f = out_factors(m, n, l);
    if (ch < a.head_dim) {
      const int64_t to = row * a.head_dim + ch;
      const float y = sum * f.x * f.y;
      if (a.act_bf16)
        static_cast<uint16_t*>(a.out)[to] = static_cast<uint16_t>(pack_bf16x2_rn(y, 0.f) & 0xFFFFu);
      else
        static_cast<float*>(a.out)[to] = y;
    }
    if ((ln & 3) == 0 && je == 0 && a.lse) a.lse[row] = row_lse(m, l);
  }

  // The state for a later merge.
  __device__ __forceinline__ void dump(float* to) const {
#pragma unroll
    for (int j = 0; j < C::kNJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < C::kNR; ++r) to[((2 * j + e) * C::kNR + r) * 32 + lane] = at(j, r, e);
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      const float l = row_sum(r);
      if (c == 0) {
        to[C::kNel + g + 8 * r] = m_run[r];
        to[C::kNel + R + g + 8 * r] = n_run[r];
        to[C::kNel + 2 * R + g + 8 * r] = l;
      }
    }
  }
};

// What a CTA's merge needs to know of a piece.
struct PieceInfo {
  int item;                      // -1: none
  int starts, ends;              // the pair's first, last tile is in it
};

template <int T, int DP, int R, bool B>
__global__ void __launch_bounds__(Cfg<T, DP, R, B>::kThreads, 1)
decode_split_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<T, DP, R, B>;
  using W = Worker<T, DP, R, B>;
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kChunks = 64;
  __shared__ int64_t s_chunk[kChunks];         // tiles (of one item) of pieces of the batch
  __shared__ PieceInfo s_piece[2 * C::kW];     // of warp w: [2 w] the one it began with, [2 w + 1] its last
  __shared__ int s_order[2 * C::kW];           // pieces that there are, in order
  __shared__ int4 s_group[2 * C::kW];          // groups: item, first piece, their number, 1 starts | 2 ends
  __shared__ int s_groups;
  __shared__ float s_weight[2 * C::kW][R];     // of a piece's o in its group, in that order
  __shared__ float s_stat[2 * C::kW][3][R];    // m, n, l of a group
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();

  // ---- the plan: tiles of all sequences, this warp's range and where it begins
  const int per_chunk = (a.batch + 32 * kChunks - 1) / (32 * kChunks) * 32;    // sequences
  const int chunks = (a.batch + per_chunk - 1) / per_chunk;
  auto tiles_at = [&](int b, int most) -> unsigned {
    return b < most ? static_cast<unsigned>(tiles_of<C::kKT>(keys_of(a, a.used[b]))) : 0u;
  };
#pragma unroll 1
  for (int k = warp; k < chunks; k += C::kW) {
    int64_t sum = 0;
#pragma unroll 1
    for (int i = lane; i < per_chunk; i += 32)
      sum += __reduce_add_sync(0xffffffffu, tiles_at(k * per_chunk + i, a.batch));
    if (lane == 0) s_chunk[k] = sum;
  }
  __syncthreads();
  int64_t total = 0;
#pragma unroll 1
  for (int k = 0; k < chunks; ++k) total += s_chunk[k];
  total *= a.items_per_seq;
  // CTAs that take part: as many as have a tile for each of their warps.  Where there are fewer
  // tiles than warps, four warps a CTA: fewer pieces to merge on each (4 sequences of up to 700
  // int8 keys, 2 heads of 64: 11.3 us, with all 16 warps 14.4).
  const int warps = total < static_cast<int64_t>(gridDim.x) * C::kW ? 4 : C::kW;
  const int64_t want = (total + warps - 1) / warps;
  const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), want));
  const int cta = static_cast<int>(blockIdx.x);
  if (cta >= ctas) {
    if (tid == 0) a.joins[cta] = make_int2(-1, 0);
    return;
  }
  // worker w of n: tiles floor(total w / n) on
  const unsigned workers = static_cast<unsigned>(ctas) * warps;
  const unsigned me = static_cast<unsigned>(cta) * warps + warp;
  const int64_t each = divide(total, workers);
  const unsigned rest = static_cast<unsigned>(total - each * workers);
  const int64_t t0 = each * me + rest * me / workers;
  const int64_t t1 = warp < warps ? each * (me + 1) + rest * (me + 1) / workers : t0;
  int b0 = 0;
  int64_t in_seq = t0;                         // tiles of the sequence before t0
  if (t0 < t1) {
    int k = 0;
#pragma unroll 1
    for (; in_seq >= s_chunk[k] * a.items_per_seq; ++k)        // (t0 < total)
      in_seq -= s_chunk[k] * a.items_per_seq;
    // (lengths that change under the call may leave it without an answer: then the last sequence's)
    b0 = a.batch - 1;
#pragma unroll 1
    for (int i = k * per_chunk; i < a.batch; i += 32) {
      const unsigned n = tiles_at(i + lane, a.batch);
      const int64_t all = static_cast<int64_t>(__reduce_add_sync(0xffffffffu, n)) * a.items_per_seq;
      if (in_seq < all) {
        unsigned x = n;                        // tiles of the 32 sequences up to the lane's
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned past =
            __ballot_sync(0xffffffffu, static_cast<int64_t>(x) * a.items_per_seq > in_seq);
        const int at = __ffs(past) - 1;
        b0 = i + at;
        in_seq -= static_cast<int64_t>(__shfl_sync(0xffffffffu, x - n, at)) * a.items_per_seq;
        break;
      }
      in_seq -= all;
    }
  }

  // ---- the warp's tiles
  W w{a};
  unsigned char* own = smem + warp * C::kPerWarp;
  w.ring = own;
  w.qf = own + C::kNE * C::kEntry;
  w.info = reinterpret_cast<uint4*>(w.qf + C::kQBytes);
  w.sc = reinterpret_cast<float*>(w.qf + C::kQBytes + kInfos * 16);
  w.lane = lane;
  w.g = lane >> 2;
  w.c = lane & 3;
  const int n = static_cast<int>(t1 - t0);
  if (lane < 2) s_piece[2 * warp + lane] = {-1, 0, 0};
  __syncwarp();
  int item = -1;
  bool open = false;               // the warp's range ended inside a pair
  bool started = false;            // the piece at hand holds its pair's first tile
  if (n > 0) {
    w.runs = a.head_dim == DP && a.page_size % C::kRun == 0;
    w.seek(b0, in_seq);
    item = b0 * a.items_per_seq + w.h;
    typename W::Rows q;
    w.fetch_q(item, q);
    typename W::Pend ahead = w.take();           // of the tile whose K is next to be copied
    uint32_t row = W::kNone, scale_at = 0;       // of the tile whose V is
    bool whole = false;
    int next_k = 0, next_v = 0, ne = 0;          // tiles asked for so far; the entry for the next copies
    auto end_group = [&]() {                     // (also where nothing was left to copy)
      copies_commit();
      if (++ne == C::kNE) ne = 0;
    };
    // K of a tile, and what its consumer has to know of it; then its V.
    auto issue_k = [&]() {
      if (next_k < n) {
        if (ahead.pid >= a.num_pages) {
          report(a.status, SA_ERR_SHAPE);
          ahead.pid = -1;
        }
        scale_at = static_cast<uint32_t>(ahead.pid) * static_cast<uint32_t>(a.hkv) + ahead.h;
        row = ahead.pid >= 0 ? scale_at * static_cast<uint32_t>(a.page_size) + ahead.row : W::kNone;
        const unsigned mask =
            __ballot_sync(0xffffffffu, (C::kKT == 32 || lane < C::kKT) && row != W::kNone);
        if (lane == 0)
          w.info[next_k % kInfos] = make_uint4(static_cast<uint32_t>(ahead.item), mask, ahead.flags, 0u);
        constexpr uint32_t kAll = C::kKT == 32 ? 0xFFFFFFFFu : (1u << (C::kKT & 31)) - 1u;
        whole = mask == kAll && (ahead.flags & 4u);
        w.template copy_rows<false>(ne, row, scale_at, whole);
      }
      ++next_k;
      end_group();
    };
    auto issue_v = [&]() {
      if (next_v < n) {
        w.template copy_rows<true>(ne, row, scale_at, whole);
        if (next_k < n) ahead = w.take();
      }
      ++next_v;
      end_group();
    };
    static_assert(C::kNE == 3, "a V follows a K's place");
    issue_k();
    issue_v();
    issue_k();
    // (Q of the first piece came beside the first copies)
    w.keep_q(q);
    w.begin();
    uint32_t flags = 0;
    int e = 0;
    for (int i = 0; i < n; ++i) {
      copies_wait<2>();
      __syncwarp();
      const uint4 inf = w.info[i % kInfos];
      flags = inf.z;
      if (flags & 1u) {
        started = true;
        if (i > 0) {
          item = static_cast<int>(inf.x);
          w.fetch_q(item, q);
          w.keep_q(q);
          w.begin();
        }
      }
      float acc[C::kNT][4], p[C::kNT][2 * C::kNR];
      float2 kf[C::kNT];
      if (inf.y) w.scores(e, acc, kf);
      __syncwarp();
      if constexpr (!C::kLate) issue_v();
      if (++e == C::kNE) e = 0;
      copies_wait<C::kLate ? 1 : 2>();
      __syncwarp();
      if (inf.y) {
        w.softmax(e, inf.y, acc, kf, p);
        w.values(e, p);
      }
      __syncwarp();
      if constexpr (C::kLate) issue_v();
      issue_k();
      if (++e == C::kNE) e = 0;
      if (flags & 2u) {
        if (started) {
          w.write_out(item);
        } else {
          w.dump(a.firsts + (static_cast<int64_t>(cta) * C::kW + warp) * C::kState);
          if (lane == 0) s_piece[2 * warp] = {item, 0, 1};
        }
      }
    }
    copies_wait<0>();
    __syncwarp();
    open = !(flags & 2u);
    if (open && lane == 0) s_piece[2 * warp + 1] = {item, started ? 1 : 0, 0};
  }
  __syncthreads();
  // Most pairs that are cut are cut once: a warp's last piece and the next warp's first make a
  // whole, which the warp writes from its registers.  Other last pieces go where the ring was.
  if (open) {
    if (started && warp + 1 < C::kW && s_piece[2 * warp + 2].item == item) {
      w.absorb(a.firsts + (static_cast<int64_t>(cta) * C::kW + warp + 1) * C::kState);
      w.write_out(item);
      __syncwarp();
      if (lane < 2) s_piece[2 * warp + 1 + lane].item = -1;
    } else {
      w.dump(reinterpret_cast<float*>(own));
    }
  }
  __syncthreads();

  // ---- pieces of pairs that this CTA's warps cut, in the order of the keys.  Pieces of one pair are
  // a group; groups are merged side by side: their statistics by a warp each (a lane
  // per row and piece), their elements by all warps in turn.
  static_assert(2 * C::kW <= 32, "a lane per piece");
  auto state = [&](int x) -> const float* {
    return x & 1 ? reinterpret_cast<const float*>(smem + (x >> 1) * C::kPerWarp)
                 : a.firsts + (static_cast<int64_t>(cta) * C::kW + (x >> 1)) * C::kState;
  };
  if (warp == 0) {
    PieceInfo my{-1, 0, 0};
    if (lane < 2 * C::kW) my = s_piece[lane];
    unsigned left = __ballot_sync(0xffffffffu, my.item >= 0);
    if (my.item >= 0) s_order[__popc(left & ((1u << lane) - 1u))] = lane;
    int at = 0, k = 0;
#pragma unroll 1
    for (; left; ++k) {
      const int p = __ffs(left) - 1, item = __shfl_sync(0xffffffffu, my.item, p);
      const unsigned group = __ballot_sync(0xffffffffu, my.item == item);
      const int starts = __shfl_sync(0xffffffffu, my.starts, p);
      const int ends = __shfl_sync(0xffffffffu, my.ends, 31 - __clz(group));
      if (lane == 0) s_group[k] = make_int4(item, at, __popc(group), starts | (ends << 1));
      at += __popc(group);
      left &= ~group;
    }
    if (lane == 0) s_groups = k;
  }
  __syncthreads();
  const int groups = s_groups;
  {
    constexpr int kSlots = 32 / R, kMost = (2 * C::kW + kSlots - 1) / kSlots;    // pieces: of a lane
    const int row = lane % R, slot = lane / R;
#pragma unroll 1
    for (int k = warp; k < groups; k += C::kW) {
      const int4 group = s_group[k];
      float m[kMost], n[kMost], l[kMost], mm = -INFINITY, nn = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const int x = slot + kSlots * i;
        m[i] = n[i] = -INFINITY;
        l[i] = 0.f;
        if (x < group.z) {
          const float* s = state(s_order[group.y + x]) + C::kNel + row;
          m[i] = s[0];
          n[i] = s[R];
          l[i] = s[2 * R];
        }
      }
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        mm = fmaxf(mm, m[i]);
        nn = fmaxf(nn, n[i]);
      }
#pragma unroll
      for (int o = R; o < 32; o <<= 1) {
        mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        nn = fmaxf(nn, __shfl_xor_sync(0xffffffffu, nn, o));
      }
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const int x = slot + kSlots * i;
        if (x < group.z) {
          s_weight[group.y + x][row] = pow2_of(n[i] - nn);
          sum = fmaf(pow2_of(m[i] - mm), l[i], sum);
        }
      }
#pragma unroll
      for (int o = R; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (slot == 0) {
        s_stat[k][0][row] = mm;
        s_stat[k][1][row] = nn;
        s_stat[k][2][row] = sum;
      }
    }
  }
  __syncthreads();
  auto row_of = [](int idx) {      // the query row of element idx of a state
    return ((idx & 31) >> 2) + (C::kNR == 2 ? 8 * ((idx >> 5) & 1) : 0);
  };
  // 128 elements of a group a warp at a time, four pieces in flight
  constexpr int kCols = 4, kUnits = C::kNel / (32 * kCols);
#pragma unroll 1
  for (int u = warp; u < groups * kUnits; u += C::kW) {
    const int k = u / kUnits, idx0 = (u - k * kUnits) * 32 * kCols + lane;
    const int4 group = s_group[k];
    float sum[kCols] = {};
#pragma unroll 1
    for (int x0 = 0; x0 < group.z; x0 += 4) {
      float v[4][kCols];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool in = x0 + x < group.z;
        const float* s = state(s_order[group.y + (in ? x0 + x : 0)]) + idx0;
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[x][i] = in ? s[32 * i] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x0 + x < group.z) {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            sum[i] = fmaf(s_weight[group.y + x0 + x][row_of(idx0 + 32 * i)], v[x][i], sum[i]);
        }
    }
    const bool starts = group.w & 1, all = group.w == 3;
    float* to = a.parts + (static_cast<int64_t>(cta) * 2 + (starts ? 1 : 0)) * C::kState;
    const Item it = item_of<R>(a, group.x);
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int idx = idx0 + 32 * i, je = (idx >> 5) / C::kNR, row = row_of(idx);
      const float m = s_stat[k][0][row], n = s_stat[k][1][row], l = s_stat[k][2][row];
      if (!all) {
        to[idx] = sum[i];
        if ((lane & 3) == 0 && je == 0) {
          to[C::kNel + row] = m;
          to[C::kNel + R + row] = n;
          to[C::kNel + 2 * R + row] = l;
        }
      } else if (row < it.rows) {
        W::write_element(a, it.row0 + row, lane, je, sum[i], m, n, l);
      }
    }
  }
  // the pair that goes on from the CTA before (-1: none), and whether it ends here
  if (tid == 0) {
    const int4 first = s_group[0];
    a.joins[cta] = groups > 0 && !(first.w & 1) ? make_int2(first.x, first.w >> 1) : make_int2(-1, 0);
  }
}

// Pairs whose parts lie in several CTAs.  CTA x of `joins` says which pair its first piece
// continues (-1: none) and whether it ends it; block x merges the pair that CTA x - 1
// began (its second part) and x, x + 1, .. continue (their first).  blockIdx.y: which elements.
template <int T, int DP, int R, bool B>
__global__ void __launch_bounds__(256) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<T, DP, R, B>;
  using W = Worker<T, DP, R, B>;
  constexpr int kLanes = kDecodeCtas / 32;     // pieces of a lane at most
  static_assert(kDecodeCtas % 32 == 0, "pieces by lanes");
  __shared__ float s_weight[R][kDecodeCtas];
  __shared__ float s_m[R], s_n[R], s_l[R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = static_cast<int>(gridDim.x);
  const int x = static_cast<int>(blockIdx.x);
  griddep_wait();
  if (x == 0) return;
  // the pair's last CTA: the first from x on that ends it
  const int2 before = __ldcg(a.joins + x - 1);
  int z = x, item = -1;
#pragma unroll 1
  for (int i = x;; i += 32) {
    const int2 j = i + lane < ctas ? __ldcg(a.joins + i + lane) : make_int2(-1, 1);
    if (i == x) {
      item = __shfl_sync(0xffffffffu, j.x, 0);
      if (item < 0 || before.x == item) return;
    }
    const unsigned ends = __ballot_sync(0xffffffffu, j.y != 0);
    if (ends) {
      z = min(i + __ffs(ends) - 1, ctas - 1);
      break;
    }
  }
  const int pieces = z - x + 2;
  auto state = [&](int p) -> const float* {
    return a.parts + (static_cast<int64_t>(x - 1 + p) * 2 + (p == 0 ? 1 : 0)) * C::kState;
  };
  // the first pieces' elements beside what they are weighted by
  constexpr int kEarly = 20;
  const int idx = static_cast<int>(blockIdx.y) * 256 + tid;
  float v[kEarly];
#pragma unroll
  for (int p = 0; p < kEarly; ++p) v[p] = p < pieces ? __ldcg(state(p) + idx) : 0.f;
#pragma unroll 1
  for (int row = warp; row < R; row += 8) {
    float m[kLanes], n[kLanes], l[kLanes], mm = -INFINITY, nn = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      const int p = lane + 32 * i;
      m[i] = n[i] = -INFINITY;
      l[i] = 0.f;
      if (p < pieces) {
        const float* s = state(p) + C::kNel + row;
        m[i] = __ldcg(s);
        n[i] = __ldcg(s + R);
        l[i] = __ldcg(s + 2 * R);
      }
    }
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      mm = fmaxf(mm, m[i]);
      nn = fmaxf(nn, n[i]);
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
      nn = fmaxf(nn, __shfl_xor_sync(0xffffffffu, nn, o));
    }
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      const int p = lane + 32 * i;
      if (p < pieces) {
        s_weight[row][p] = pow2_of(n[i] - nn);
        sum = fmaf(pow2_of(m[i] - mm), l[i], sum);
      }
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      s_m[row] = mm;
      s_n[row] = nn;
      s_l[row] = sum;
    }
  }
  __syncthreads();
  const Item it = item_of<R>(a, item);
  const int ln = idx & 31, rest = idx >> 5;
  const int r = rest % C::kNR, je = rest / C::kNR;
  const int row = (ln >> 2) + 8 * r;
  if (row >= it.rows) return;
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < kEarly; ++p)
    if (p < pieces) sum = fmaf(s_weight[row][p], v[p], sum);
#pragma unroll 8
  for (int p = kEarly; p < pieces; ++p) sum = fmaf(s_weight[row][p], __ldcg(state(p) + idx), sum);
  W::write_element(a, it.row0 + row, ln, je, sum, s_m[row], s_n[row], s_l[row]);
}

template <int T, int DP, int R, bool B>
cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  using C = Cfg<T, DP, R, B>;
  const void* fn = reinterpret_cast<const void*>(decode_split_kernel<T, DP, R, B>);
  static SmemLimit limit;
  cudaError_t err = limit.raise(fn, C::kSmem);
  if (err != cudaSuccess) return err;
  const int ctas = device_sm_count() < kDecodeCtas ? device_sm_count() : kDecodeCtas;
  decode_split_kernel<T, DP, R, B><<<ctas, C::kThreads, C::kSmem, stream>>>(a);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, (C::kNel + 255) / 256);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, DP, R, B>, a);
}

template <int T, int DP>
cudaError_t launch_dim(const DecodeArgs& a, int r, cudaStream_t s) {
  if constexpr (T == SA_DTYPE_F32) {
    return launch<T, DP, 8, false>(a, s);
  } else {
    if (r == 8) return a.act_bf16 ? launch<T, DP, 8, true>(a, s) : launch<T, DP, 8, false>(a, s);
    return a.act_bf16 ? launch<T, DP, 16, true>(a, s) : launch<T, DP, 16, false>(a, s);
  }
}

template <int T>
cudaError_t launch_type(const DecodeArgs& a, int dp, int r, cudaStream_t s) {
  return dp == 64 ? launch_dim<T, 64>(a, r, s) : dp == 128 ? launch_dim<T, 128>(a, r, s)
                                                           : launch_dim<T, 256>(a, r, s);
}

}  // namespace dec1
}  // namespace sa
