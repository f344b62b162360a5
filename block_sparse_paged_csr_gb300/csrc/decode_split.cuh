// Attention of one new token per sequence over its whole paged cache, split over the
// cache's length.  Instances per cache type are in decode_f32.cu, decode_bf16.cu,
// decode_e4m3.cu and decode_int8.cu; decode.cu holds the entry point and the join.
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

template <int T> struct TypeOf;
template <> struct TypeOf<SA_DTYPE_F32> { static constexpr int size = 4; };
template <> struct TypeOf<SA_DTYPE_BF16> { static constexpr int size = 2; };
template <> struct TypeOf<SA_DTYPE_E4M3> { static constexpr int size = 1; };
template <> struct TypeOf<SA_DTYPE_INT8> { static constexpr int size = 1; };

// T: the cache's type.  DP: head_dim rounded up to 64, 128 or 256 (channels behind it
// are zeros).  R: query rows of a tile, 8 or 16.
template <int T, int DP, int R>
struct Cfg {
  static constexpr int kSize = TypeOf<T>::size;
  static constexpr bool kF32 = T == SA_DTYPE_F32;
  static constexpr bool k8 = kSize == 1;
  static constexpr int kRow = DP * kSize;                       // bytes of a row in the ring
  // keys of a tile: 4 KB of K where that is 8 to 32 keys
  static constexpr int kKT = kF32 ? (DP == 64 ? 16 : 8) : k8 ? (DP == 256 ? 16 : 32) : (DP == 64 ? 32 : 16);
  static constexpr int kEntry = kKT * kRow;                     // bytes of a tile's K (or V)
  static constexpr int kST = 2;                                 // tiles of the ring
  static constexpr int kNCH = kRow / 16;                        // 16-byte chunks of a row
  static constexpr int kLCH = kNCH / 4;                         // chunks of a row that a lane reads for S
  static constexpr int kEC = 16 / kSize;                        // elements of a chunk
  static constexpr int kKPC = k8 ? 4 : 2;                       // k-steps of a chunk
  static constexpr int kKS = kLCH * kKPC;                       // k-steps of a row
  static constexpr int kNT = kKT / 8;                           // n-tiles of S
  static constexpr int kKK = kF32 ? 8 : 16;                     // keys of one P V k-step
  static constexpr int kVP = DP * kSize / 8 < 16 ? 8 : 16;      // bytes of V that a lane reads of a row at a time
  static constexpr int kEP = kVP / kSize;                       // .. channels
  static constexpr int kNS = DP / (8 * kEP);                    // .. times
  static constexpr int kNJ = DP / 8;                            // n-tiles of o
  static constexpr int kNR = R / 8;                             // query rows of a lane
  // operands of Q kept per k-step (see load_q)
  static constexpr int kQP = kF32 ? 1 : k8 ? (R == 8 ? 1 : 2) : (R == 8 ? 2 : 3);
  static constexpr int kQBytes = kKS * kQP * 512;
  static constexpr int kScales = k8 ? 2 * kST * kKT * 4 : 0;
  static constexpr int kPerWarp = 2 * kST * kEntry + kQBytes + kScales + kST * 16;
  static constexpr int kMost = 220 * 1024;
  static constexpr int kW = kMost / kPerWarp < 8 ? kMost / kPerWarp : 8;   // warps
  static constexpr int kThreads = 32 * kW;
  static constexpr int kSmem = kW * kPerWarp;
  // a state: o in the order of the accumulators, then m, n and l of each row
  static constexpr int kNel = R * DP;
  static constexpr int kState = kNel + 3 * R;
  static_assert(kState * 4 <= 2 * kST * kEntry + kQBytes, "a warp's last state replaces its ring");
  static_assert(kW >= 2 && kW <= kDecodeMaxWarps && kState <= decode_state_floats(DP, R), "workspace");
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
  k.end = min(max(used, 0), a.capacity);
  k.first = a.window > 0 ? max(used - a.window, 0) : 0;      // (used < 0: end = 0 takes all)
  return k;
}
template <int KT>
__device__ __forceinline__ int tiles_of(const Keys& k) {
  return max((k.end - k.first + KT - 1) / KT, 1);             // a sequence without keys has one, of none
}

// Four channels of query row `row` (zeros behind head_dim).
__device__ __forceinline__ float4 load_q4(const DecodeArgs& a, int64_t row, int ch, bool there) {
  if (!there || ch >= a.head_dim) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.act_bf16)
    return bf16x4_to_f32(*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) +
                                                         row * a.head_dim + ch));
  return *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + row * a.head_dim + ch);
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

template <int T, int DP, int R>
struct Worker {
  using C = Cfg<T, DP, R>;

  const DecodeArgs& a;
  unsigned char* ring;           // this warp's [2 kST][kEntry]: K, V of a tile in turn
  unsigned char* qf;             // Q's operands
  float* sc;                     // [2 kST][kKT] scales
  uint4* info;                   // [kST]: item, live keys, flags
  int lane, g, c;

  // ---- the tile to come: where it lies
  int b, h, t, nt, first, end, next_used;     // cursor
  struct Pend {
    int pid, row, h, item;
    uint32_t flags;              // 1: the pair's first tile, 2: its last
  };

  // ---- state of the piece at hand
  float o[C::kNJ][4];
  float m_run[C::kNR], n_run[C::kNR], l_part[C::kNR], vfac[C::kNR], sfac[C::kNR];

  __device__ __forceinline__ void seek(int b0, int64_t in_seq) {
    b = b0;
    const Keys k = keys_of(a, a.used[b]);
    first = k.first;
    end = k.end;
    nt = tiles_of<C::kKT>(k);
    h = static_cast<int>(in_seq / nt);
    t = static_cast<int>(in_seq - static_cast<int64_t>(h) * nt);
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
    p.flags = (t == 0 ? 1u : 0u) | (t + 1 == nt ? 2u : 0u);
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
        }
      }
    }
    return p;
  }

  // Copies of one tile's K (kV false) or V rows; off: the lane's row (key `lane`) in
  // bytes of the pool, negative where there is none; so: its scale's index.
  template <bool kV>
  __device__ __forceinline__ void copy_rows(int slot, int64_t off, int64_t so) {
    unsigned char* dst = ring + (2 * slot + (kV ? 1 : 0)) * C::kEntry;
    const unsigned char* pool = static_cast<const unsigned char*>(kV ? a.v_pages : a.k_pages);
    const uint32_t d0 = smem_u32(dst);
#pragma unroll
    for (int i = 0; i < C::kKT * C::kNCH / 32; ++i) {
      const int idx = 32 * i + lane;
      const int row = idx / C::kNCH, ch = idx & (C::kNCH - 1);
      const int64_t at = __shfl_sync(0xffffffffu, off, row);
      const bool there = at >= 0 && 16 * ch < a.row_bytes;
      const int phys = C::kNCH >= 8 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3);
      copy16(d0 + row * C::kRow + phys * 16, pool + (there ? at + 16 * ch : 0), there);
    }
    if constexpr (C::k8) {
      if (C::kKT == 32 || lane < C::kKT) {
        const float* s = kV ? a.v_scales : a.k_scales;
        copy4(smem_u32(sc + (2 * slot + (kV ? 1 : 0)) * C::kKT + lane), s + (off >= 0 ? so : 0), off >= 0);
      }
    }
  }

  // Q's operands for an item, in the order in which the k-steps use them: lane (g, c)
  // holds row g (and g + 8) at the channels of the chunks that it reads of K's rows.
  //   8 bits: the row, scaled by a power of two into f16's range, as f16 high
  //     parts and remainders; bf16: three bf16 parts (bf16 queries: the first says all);
  //     f32: tf32 parts.
  //   R = 8: rows g + 8 of the MMA's tile carry the second parts of rows g, so that they cost no product.
  __device__ __forceinline__ void load_q(int item) {
    const Item it = item_of<R>(a, item);
    uint4* out = reinterpret_cast<uint4*>(qf) + lane;
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) sfac[r] = a.scale * kLog2e;
    float f[C::kNR];
    if constexpr (C::k8) {
#pragma unroll
      for (int r = 0; r < C::kNR; ++r) {
        const int row = g + 8 * r;
        float am = 0.f;
#pragma unroll
        for (int l = 0; l < C::kLCH; ++l)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float4 x = load_q4(a, it.row0 + row, chunk(l) * 16 + 4 * s, row < it.rows);
            am = fmaxf(am, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
          }
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // largest magnitude to [2^10, 2^11): f and 1 / f kept normal
        const int ex = min(max(static_cast<int>(__float_as_uint(am) >> 23), 11), 253);
        f[r] = __uint_as_float(static_cast<uint32_t>(264 - ex) << 23);
        sfac[r] *= __uint_as_float(static_cast<uint32_t>(ex - 10) << 23);
      }
    }
    __syncwarp();
#pragma unroll
    for (int l = 0; l < C::kLCH; ++l)
#pragma unroll
      for (int s = 0; s < C::kEC / 4; ++s) {
        const int ch = chunk(l) * C::kEC + 4 * s;
        float4 x[C::kNR];
#pragma unroll
        for (int r = 0; r < C::kNR; ++r)
          x[r] = load_q4(a, it.row0 + g + 8 * r, ch, g + 8 * r < it.rows);
        if constexpr (C::kF32) {
          uint4 u, v;
          split_tf32(x[0].x, u.x, u.y);
          split_tf32(x[0].y, u.z, u.w);
          split_tf32(x[0].z, v.x, v.y);
          split_tf32(x[0].w, v.z, v.w);
          out[32 * (2 * l)] = u;
          out[32 * (2 * l + 1)] = v;
        } else {
          uint4* at = out + 32 * C::kQP * (l * C::kKPC + s);
          uint32_t hi[C::kNR][2], mid[C::kNR][2], lo[C::kNR][2];
#pragma unroll
          for (int r = 0; r < C::kNR; ++r) {
            if constexpr (C::k8) {
              split_f16(x[r].x * f[r], x[r].y * f[r], hi[r][0], mid[r][0]);
              split_f16(x[r].z * f[r], x[r].w * f[r], hi[r][1], mid[r][1]);
              lo[r][0] = lo[r][1] = 0u;
            } else {
              split_bf16(x[r].x, x[r].y, hi[r][0], mid[r][0], lo[r][0]);
              split_bf16(x[r].z, x[r].w, hi[r][1], mid[r][1], lo[r][1]);
            }
          }
          if constexpr (R == 8) {
            at[0] = make_uint4(hi[0][0], mid[0][0], hi[0][1], mid[0][1]);
            if constexpr (C::kQP == 2) at[32] = make_uint4(lo[0][0], 0u, lo[0][1], 0u);
          } else {
            at[0] = make_uint4(hi[0][0], hi[1][0], hi[0][1], hi[1][1]);
            at[32] = make_uint4(mid[0][0], mid[1][0], mid[0][1], mid[1][1]);
            if constexpr (C::kQP == 3) at[64] = make_uint4(lo[0][0], lo[1][0], lo[0][1], lo[1][1]);
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
#pragma unroll
    for (int j = 0; j < C::kNJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  }

  // S = Q K^T of a tile: acc[nt][e] (row g: keys 8 nt + 2 c, + 1; then row g + 8).
  // A fragment's k index may stand for any channel as long as both operands agree,
  // so K's rows go from the ring to the MMA as they lie.
  __device__ __forceinline__ void scores(int slot, float (&acc)[C::kNT][4]) {
    const unsigned char* kt = ring + 2 * slot * C::kEntry + g * C::kRow;
    const uint4* q = reinterpret_cast<const uint4*>(qf) + lane;
    float low[C::kF32 ? C::kNT : 1][4];
#pragma unroll
    for (int n = 0; n < C::kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    if constexpr (C::kF32) {
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) low[n][e] = 0.f;
    }
#pragma unroll
    for (int l = 0; l < C::kLCH; ++l) {
      const int phys = C::kNCH >= 8 ? chunk(l) ^ g : chunk(l) ^ ((g >> 1) & 3);
      uint4 kr[C::kNT];
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
        kr[n] = *reinterpret_cast<const uint4*>(kt + n * 8 * C::kRow + phys * 16);
#pragma unroll
      for (int s = 0; s < C::kKPC; ++s) {
        const uint4* at = q + 32 * C::kQP * (l * C::kKPC + s);
        const uint4 q0 = at[0];
        uint4 q1, q2;
        if constexpr (C::kQP >= 2) q1 = at[32];
        if constexpr (C::kQP >= 3) q2 = at[64];
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          const uint32_t w[4] = {kr[n].x, kr[n].y, kr[n].z, kr[n].w};
          if constexpr (C::k8) {
            uint32_t b0, b1;
            codes4_to_f16<T == SA_DTYPE_INT8>(w[s], b0, b1);
            mma<T>(acc[n], q0, b0, b1);
            if constexpr (C::kQP == 2)
              if (!a.act_bf16) mma<T>(acc[n], q1, b0, b1);     // (bf16 has no remainder in f16)
          } else if constexpr (C::kF32) {
            uint32_t h0, l0, h1, l1;
            split_tf32(__uint_as_float(w[2 * s]), h0, l0);
            split_tf32(__uint_as_float(w[2 * s + 1]), h1, l1);
            mma<T>(acc[n], q0, h0, h1);
            mma<T>(low[n], q0, l0, l1);
          } else {
            mma<T>(acc[n], q0, w[2 * s], w[2 * s + 1]);
            if (!a.act_bf16) {
              mma<T>(acc[n], q1, w[2 * s], w[2 * s + 1]);
              if constexpr (C::kQP == 3) mma<T>(acc[n], q2, w[2 * s], w[2 * s + 1]);
            }
          }
        }
      }
    }
    if constexpr (C::kF32) {
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] += low[n][e];
    }
    if constexpr (C::k8) {
      const float* ks = sc + 2 * slot * C::kKT;
#pragma unroll
      for (int n = 0; n < C::kNT; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(ks + 8 * n + 2 * c);
        acc[n][0] *= f.x;
        acc[n][1] *= f.y;
        acc[n][2] *= f.x;
        acc[n][3] *= f.y;
      }
    }
  }

  // The online softmax of a tile: acc becomes p (row g + 8 r, key 8 n + 2 c + e:
  // acc[n][2 r + e]).  mask: which of the tile's keys there are (others count 0).
  __device__ __forceinline__ void softmax(int slot, uint32_t mask, float (&acc)[C::kNT][4]) {
    const float* vs = sc + (2 * slot + 1) * C::kKT;
    constexpr uint32_t kAll = C::kKT == 32 ? 0xFFFFFFFFu : (1u << (C::kKT & 31)) - 1u;
    const bool whole = mask == kAll;
    bool beyond = false;
#pragma unroll
    for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
      for (int r = 0; r < C::kNR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (R = 8: the remainders' row joins its own)
          float x = (R == 8 ? acc[n][e] + acc[n][e + 2] : acc[n][2 * r + e]) * sfac[r];
          if (!whole && !((mask >> (8 * n + 2 * c + e)) & 1u)) x = -INFINITY;
          beyond = beyond || x - m_run[r] > kSlack;           // (m = -inf before the first keys)
          acc[n][2 * r + e] = x;
        }
      if constexpr (C::k8) {
        const float2 vf = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c);
        const float most = fmaxf(fabsf(vf.x), fabsf(vf.y));
#pragma unroll
        for (int r = 0; r < C::kNR; ++r) beyond = beyond || most * vfac[r] > kRoom;
      }
    }
    if (__any_sync(0xffffffffu, beyond)) {
#pragma unroll
      for (int r = 0; r < C::kNR; ++r) {
        float cm = -INFINITY, top = -INFINITY;               // largest score, largest product
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          cm = fmaxf(cm, fmaxf(acc[n][2 * r], acc[n][2 * r + 1]));
          if constexpr (C::k8) {
            const float2 vf = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c);
            // (a key that is not there: its score is -inf, its scale 0)
            top = fmaxf(top, fmaxf(acc[n][2 * r] + log2f(fabsf(vf.x)),
                                   acc[n][2 * r + 1] + log2f(fabsf(vf.y))));
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
          for (int e = 0; e < 4; ++e)
            if (R == 8 || e / 2 == r) o[j][e] *= beta;
      }
    }
#pragma unroll
    for (int r = 0; r < C::kNR; ++r) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < C::kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          acc[n][2 * r + e] = ex2(acc[n][2 * r + e] - m_run[r]);
          sum += acc[n][2 * r + e];
        }
      l_part[r] += sum;
    }
  }

  // o += P V.  V's rows too go to the MMA as they lie: n index of n-tile kEP s + i stands
  // for channel 8 kEP s + kEP n + i.
  __device__ __forceinline__ void values(int slot, const float (&p)[C::kNT][4]) {
    const unsigned char* vt = ring + (2 * slot + 1) * C::kEntry;
    const float* vs = sc + (2 * slot + 1) * C::kKT;
#pragma unroll
    for (int kt = 0; kt < C::kKT / C::kKK; ++kt) {
      uint4 a0, a1, a2;
      if constexpr (C::kF32) {
        split_tf32(p[kt][0], a0.x, a0.y);
        split_tf32(p[kt][1], a0.z, a0.w);
      } else {
        uint32_t hi[C::kNR][2], mid[C::kNR][2], lo[C::kNR][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int n = 2 * kt + x;
          float2 vf = make_float2(1.f, 1.f);
          if constexpr (C::k8) vf = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c);
#pragma unroll
          for (int r = 0; r < C::kNR; ++r) {
            float p0 = p[n][2 * r], p1 = p[n][2 * r + 1];
            if constexpr (C::k8) {
              // (a number: a page far above the others' scales may pass f32's range where its
              // keys' P is 0)
              p0 *= fminf(fmaxf(vf.x * vfac[r], -FLT_MAX), FLT_MAX);
              p1 *= fminf(fmaxf(vf.y * vfac[r], -FLT_MAX), FLT_MAX);
              split_f16(p0, p1, hi[r][x], mid[r][x]);
            } else {
              split_bf16(p0, p1, hi[r][x], mid[r][x], lo[r][x]);
            }
          }
        }
        if constexpr (R == 8) {
          a0 = make_uint4(hi[0][0], mid[0][0], hi[0][1], mid[0][1]);
          if constexpr (!C::k8) a1 = make_uint4(lo[0][0], 0u, lo[0][1], 0u);
        } else {
          a0 = make_uint4(hi[0][0], hi[1][0], hi[0][1], hi[1][1]);
          a1 = make_uint4(mid[0][0], mid[1][0], mid[0][1], mid[1][1]);
          if constexpr (!C::k8) a2 = make_uint4(lo[0][0], lo[1][0], lo[0][1], lo[1][1]);
        }
      }
#pragma unroll
      for (int s = 0; s < C::kNS; ++s) {
        auto read = [&](int row, uint32_t (&w)[4]) {
          const int sw = C::kNCH >= 8 ? row & 7 : (row >> 1) & 3;
          if constexpr (C::kVP == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(vt + row * C::kRow + (((8 * s + g) ^ sw) << 4));
            w[0] = u.x;
            w[1] = u.y;
            w[2] = u.z;
            w[3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vt + row * C::kRow + (((g >> 1) ^ sw) << 4) +
                                                            8 * (g & 1));
            w[0] = u.x;
            w[1] = u.y;
            w[2] = w[3] = 0u;
          }
        };
        uint32_t y0[4], y1[4];
        if constexpr (C::kF32) {
          read(8 * kt + 2 * c, y0);
          read(8 * kt + 2 * c + 1, y1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h0, l0, h1, l1;
            split_tf32(__uint_as_float(y0[i]), h0, l0);
            split_tf32(__uint_as_float(y1[i]), h1, l1);
            mma<T>(o[4 * s + i], a0, h0, h1);
            mma<T>(o[4 * s + i], a0, l0, l1);
          }
        } else {
          uint32_t y2[4], y3[4];
          read(16 * kt + 2 * c, y0);
          read(16 * kt + 2 * c + 1, y1);
          read(16 * kt + 2 * c + 8, y2);
          read(16 * kt + 2 * c + 9, y3);
#pragma unroll
          for (int q = 0; q < C::kVP / 4; ++q) {
            constexpr int kPer = C::k8 ? 4 : 2;              // channels of a word
            uint32_t b[kPer][2];
            if constexpr (C::k8) {
              constexpr bool kI8 = T == SA_DTYPE_INT8;
              codes4_to_f16<kI8>(__byte_perm(y0[q], y1[q], 0x5140), b[0][0], b[1][0]);
              codes4_to_f16<kI8>(__byte_perm(y0[q], y1[q], 0x7362), b[2][0], b[3][0]);
              codes4_to_f16<kI8>(__byte_perm(y2[q], y3[q], 0x5140), b[0][1], b[1][1]);
              codes4_to_f16<kI8>(__byte_perm(y2[q], y3[q], 0x7362), b[2][1], b[3][1]);
            } else {
              b[0][0] = __byte_perm(y0[q], y1[q], 0x5410);
              b[1][0] = __byte_perm(y0[q], y1[q], 0x7632);
              b[0][1] = __byte_perm(y2[q], y3[q], 0x5410);
              b[1][1] = __byte_perm(y2[q], y3[q], 0x7632);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const int j = C::kEP * s + kPer * q + i;
              mma<T>(o[j], a0, b[i][0], b[i][1]);
              if constexpr (R == 16 && C::k8) {
                // bf16 out: one f16 part of P (2^-12 of it, an eighth of the output's step)
                if (!a.act_bf16) mma<T>(o[j], a1, b[i][0], b[i][1]);
              } else if constexpr (R == 16) {
                mma<T>(o[j], a1, b[i][0], b[i][1]);
                if (!a.act_bf16) mma<T>(o[j], a2, b[i][0], b[i][1]);
              } else if constexpr (!C::k8) {
                if (!a.act_bf16) mma<T>(o[j], a1, b[i][0], b[i][1]);
              }
            }
          }
        }
      }
    }
  }

  __device__ __forceinline__ float at(int j, int r, int e) const {
    return R == 8 ? o[j][e] + o[j][e + 2] : o[j][2 * r + e];
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

template <int T, int DP, int R>
__global__ void __launch_bounds__(Cfg<T, DP, R>::kThreads, 1)
decode_split_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<T, DP, R>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[C::kThreads];
  __shared__ int64_t s_warp[C::kW];
  __shared__ PieceInfo s_piece[2 * C::kW];     // of warp w: [2 w] the one it began with, [2 w + 1] its last
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();

  // ---- the plan: tiles of all sequences, this warp's range and where it begins
  int64_t mine = 0;
  for (int b = tid; b < a.batch; b += C::kThreads) mine += tiles_of<C::kKT>(keys_of(a, a.used[b]));
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < C::kW; ++w) total += s_warp[w];
  total *= a.items_per_seq;
  // CTAs that take part: as many as have kMinTiles tiles for each of their warps
  constexpr int kMinTiles = 1;
  const int64_t want = (total + C::kW * kMinTiles - 1) / (C::kW * kMinTiles);
  const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), want));
  const int cta = static_cast<int>(blockIdx.x);
  if (cta >= ctas) {
    if (tid == 0) a.joins[cta] = make_int2(-1, 0);
    return;
  }
  const int64_t workers = static_cast<int64_t>(ctas) * C::kW;
  const int64_t me = static_cast<int64_t>(cta) * C::kW + warp;
  const int64_t t0 = total * me / workers, t1 = total * (me + 1) / workers;
  int b0 = -1;
  int64_t in_seq = 0;
  {
    int64_t before = 0;                        // tiles of the sequences before `base`, of one item
    for (int base = 0; base < a.batch; base += C::kThreads) {
      const int b = base + tid;
      const int64_t n = b < a.batch ? tiles_of<C::kKT>(keys_of(a, a.used[b])) : 0;
      int64_t x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();                         // (the last round's readers)
      if (lane == 31) s_warp[warp] = x;
      __syncthreads();
      int64_t seg = 0;
#pragma unroll
      for (int w = 0; w < C::kW; ++w) {
        if (w < warp) x += s_warp[w];
        seg += s_warp[w];
      }
      s_scan[tid] = x;
      __syncthreads();
      if (b0 < 0 && t0 < (before + seg) * a.items_per_seq) {
        for (int i = 0; i < C::kThreads && b0 < 0; i += 32) {
          const bool past = (before + s_scan[i + lane]) * a.items_per_seq > t0;
          const unsigned bal = __ballot_sync(0xffffffffu, past);
          if (bal) {
            const int at = i + __ffs(bal) - 1;
            b0 = base + at;
            in_seq = t0 - (before + (at ? s_scan[at - 1] : 0)) * a.items_per_seq;
          }
        }
      }
      before += seg;
    }
  }

  // ---- the warp's tiles
  Worker<T, DP, R> w{a};
  unsigned char* own = smem + warp * C::kPerWarp;
  w.ring = own;
  w.qf = own + 2 * C::kST * C::kEntry;
  w.info = reinterpret_cast<uint4*>(w.qf + C::kQBytes);
  w.sc = reinterpret_cast<float*>(w.qf + C::kQBytes + C::kST * 16);
  w.lane = lane;
  w.g = lane >> 2;
  w.c = lane & 3;
  const int n = static_cast<int>(t1 - t0);
  if (lane < 2) s_piece[2 * warp + lane] = {-1, 0, 0};
  __syncwarp();
  if (n > 0) {
    using Pend = typename Worker<T, DP, R>::Pend;
    w.seek(b0, in_seq);
    Pend pend[C::kST], ahead{};
    int64_t off = -1, so = 0;
    // K of a tile: what the consumer needs to know of it beside
    auto issue_k = [&](Pend& p, int slot) {
      if (p.pid >= a.num_pages) {
        report(a.status, SA_ERR_SHAPE);
        p.pid = -1;
      }
      so = static_cast<int64_t>(p.pid) * a.hkv + p.h;
      off = p.pid >= 0 ? (so * a.page_size + p.row) * a.row_bytes : -1;
      const unsigned mask = __ballot_sync(0xffffffffu, (C::kKT == 32 || lane < C::kKT) && off >= 0);
      if (lane == 0) w.info[slot] = make_uint4(static_cast<uint32_t>(p.item), mask, p.flags, 0u);
      w.template copy_rows<false>(slot, off, so);
    };
#pragma unroll
    for (int i = 0; i < C::kST; ++i)
      if (i < n) pend[i] = w.take();
    if (C::kST < n) ahead = w.take();
#pragma unroll
    for (int i = 0; i < C::kST; ++i) {
      if (i < n) issue_k(pend[i], i);
      copies_commit();
      if (i < n) w.template copy_rows<true>(i, off, so);
      copies_commit();
    }
    int item = -1;
    uint32_t flags = 0;
    bool started = false;          // the piece at hand holds its pair's first tile
    int slot = 0;
    for (int i = 0; i < n; ++i) {
      copies_wait<2 * C::kST - 1>();
      __syncwarp();
      const uint4 inf = w.info[slot];
      flags = inf.z;
      if (i == 0 || (flags & 1u)) {
        item = static_cast<int>(inf.x);
        started = (flags & 1u) != 0;
        w.begin();
        w.load_q(item);
      }
      float acc[C::kNT][4];
      if (inf.y) w.scores(slot, acc);
      __syncwarp();
      const bool more = i + C::kST < n;
      if (more) issue_k(ahead, slot);
      copies_commit();
      copies_wait<2 * C::kST - 1>();
      __syncwarp();
      if (inf.y) {
        w.softmax(slot, inf.y, acc);
        w.values(slot, acc);
      }
      __syncwarp();
      if (more) w.template copy_rows<true>(slot, off, so);
      copies_commit();
      if (i + C::kST + 1 < n) ahead = w.take();
      if (flags & 2u) {
        if (started) {
          w.write_out(item);
        } else {
          w.dump(a.firsts + me * C::kState);
          if (lane == 0) s_piece[2 * warp] = {item, 0, 1};
        }
      }
      if (++slot == C::kST) slot = 0;
    }
    copies_wait<0>();
    __syncwarp();
    if (!(flags & 2u)) {
      w.dump(reinterpret_cast<float*>(own));
      if (lane == 0) s_piece[2 * warp + 1] = {item, started ? 1 : 0, 0};
    }
  }
  __syncthreads();

  // ---- pieces of pairs that this CTA's warps cut, in the order of the keys
  bool joined = false;             // the CTA's first piece goes on from the CTA before
  int first_item = -1, first_ends = 0;
  for (int p = 0; p < 2 * C::kW;) {
    const PieceInfo head = s_piece[p];
    if (head.item < 0) {
      ++p;
      continue;
    }
    int q = p, ends = head.ends;
    while (q + 1 < 2 * C::kW && (s_piece[q + 1].item < 0 || s_piece[q + 1].item == head.item)) {
      ++q;
      if (s_piece[q].item >= 0) ends = s_piece[q].ends;
    }
    auto state = [&](int x) -> const float* {
      return x & 1 ? reinterpret_cast<const float*>(smem + (x >> 1) * C::kPerWarp)
                   : a.firsts + (static_cast<int64_t>(cta) * C::kW + (x >> 1)) * C::kState;
    };
    const bool all = head.starts && ends;
    if (!head.starts) {
      joined = true;
      first_item = head.item;
      first_ends = ends;
    }
    float* to = a.parts + (static_cast<int64_t>(cta) * 2 + (head.starts ? 1 : 0)) * C::kState;
    const Item it = item_of<R>(a, head.item);
    for (int idx = tid; idx < C::kNel; idx += C::kThreads) {
      const int ln = idx & 31, rest = idx >> 5;
      const int r = rest % C::kNR, je = rest / C::kNR;
      const int row = (ln >> 2) + 8 * r;
      float m = -INFINITY, nn = -INFINITY;
      for (int x = p; x <= q; ++x)
        if (s_piece[x].item >= 0) {
          m = fmaxf(m, state(x)[C::kNel + row]);
          nn = fmaxf(nn, state(x)[C::kNel + R + row]);
        }
      float sum = 0.f, l = 0.f;
      for (int x = p; x <= q; ++x)
        if (s_piece[x].item >= 0) {
          const float* s = state(x);
          sum = fmaf(pow2_of(s[C::kNel + R + row] - nn), s[idx], sum);
          l = fmaf(pow2_of(s[C::kNel + row] - m), s[C::kNel + 2 * R + row], l);
        }
      if (!all) {
        to[idx] = sum;
        if ((ln & 3) == 0 && je == 0) {
          to[C::kNel + row] = m;
          to[C::kNel + R + row] = nn;
          to[C::kNel + 2 * R + row] = l;
        }
      } else if (row < it.rows) {
        const int j = je >> 1, e = je & 1;
        const int ch = 8 * C::kEP * (j / C::kEP) + C::kEP * (2 * (ln & 3) + e) + j % C::kEP;
        const float2 f = Worker<T, DP, R>::out_factors(m, nn, l);
        if (ch < a.head_dim) {
          const int64_t at = (it.row0 + row) * a.head_dim + ch;
          if (a.act_bf16)
            static_cast<uint16_t*>(a.out)[at] =
                static_cast<uint16_t>(pack_bf16x2_rn(sum * f.x * f.y, 0.f) & 0xFFFFu);
          else
            static_cast<float*>(a.out)[at] = sum * f.x * f.y;
        }
        if ((ln & 3) == 0 && je == 0 && a.lse)
          a.lse[it.row0 + row] = Worker<T, DP, R>::row_lse(m, l);
      }
    }
    p = q + 1;
  }
  if (tid == 0) a.joins[cta] = make_int2(joined ? first_item : -1, first_ends);
}

// Pairs whose parts lie in several CTAs.  CTA x of `joins` says which pair its first piece
// continues (-1: none) and whether it ends it; block x merges the pair that CTA x - 1
// began (its second part) and x, x + 1, .. continue (their first).
template <int T, int DP, int R>
__global__ void __launch_bounds__(256) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<T, DP, R>;
  __shared__ int2 s_join[kDecodeCtas];
  __shared__ float s_wo[R][kDecodeCtas + 1];
  __shared__ float s_m[R], s_n[R], s_l[R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = static_cast<int>(gridDim.x);
  const int x = static_cast<int>(blockIdx.x);
  griddep_wait();
  for (int i = tid; i < ctas; i += 256) s_join[i] = __ldcg(a.joins + i);
  __syncthreads();
  const int item = s_join[x].x;
  if (x == 0 || item < 0 || s_join[x - 1].x == item) return;
  int z = x;
  while (!s_join[z].y && z + 1 < ctas) ++z;
  const int pieces = z - x + 2;
  auto state = [&](int p) -> const float* {
    return a.parts + (static_cast<int64_t>(x - 1 + p) * 2 + (p == 0 ? 1 : 0)) * C::kState;
  };
  for (int row = warp; row < R; row += 8) {
    float m = -INFINITY, n = -INFINITY;
    for (int p = lane; p < pieces; p += 32) {
      m = fmaxf(m, __ldcg(state(p) + C::kNel + row));
      n = fmaxf(n, __ldcg(state(p) + C::kNel + R + row));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    }
    float l = 0.f;
    for (int p = lane; p < pieces; p += 32) {
      s_wo[row][p] = pow2_of(__ldcg(state(p) + C::kNel + R + row) - n);
      l = fmaf(pow2_of(__ldcg(state(p) + C::kNel + row) - m), __ldcg(state(p) + C::kNel + 2 * R + row), l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      s_m[row] = m;
      s_n[row] = n;
      s_l[row] = l;
    }
  }
  __syncthreads();
  const Item it = item_of<R>(a, item);
  const int idx = static_cast<int>(blockIdx.y) * 256 + tid;
  const int ln = idx & 31, rest = idx >> 5;
  const int r = rest % C::kNR, je = rest / C::kNR;
  const int row = (ln >> 2) + 8 * r;
  if (row >= it.rows) return;
  float sum = 0.f;
#pragma unroll 8
  for (int p = 0; p < pieces; ++p) sum = fmaf(s_wo[row][p], __ldcg(state(p) + idx), sum);
  const int j = je >> 1, e = je & 1;
  const int ch = 8 * C::kEP * (j / C::kEP) + C::kEP * (2 * (ln & 3) + e) + j % C::kEP;
  const float2 f = Worker<T, DP, R>::out_factors(s_m[row], s_n[row], s_l[row]);
  if (ch < a.head_dim) {
    const int64_t at = (it.row0 + row) * a.head_dim + ch;
    if (a.act_bf16)
      static_cast<uint16_t*>(a.out)[at] =
          static_cast<uint16_t>(pack_bf16x2_rn(sum * f.x * f.y, 0.f) & 0xFFFFu);
    else
      static_cast<float*>(a.out)[at] = sum * f.x * f.y;
  }
  if ((ln & 3) == 0 && je == 0 && a.lse)
    a.lse[it.row0 + row] = Worker<T, DP, R>::row_lse(s_m[row], s_l[row]);
}

template <int T, int DP, int R>
cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  using C = Cfg<T, DP, R>;
  const void* fn = reinterpret_cast<const void*>(decode_split_kernel<T, DP, R>);
  static SmemLimit limit;
  cudaError_t err = limit.raise(fn, C::kSmem);
  if (err != cudaSuccess) return err;
  const int ctas = device_sm_count() < kDecodeCtas ? device_sm_count() : kDecodeCtas;
  decode_split_kernel<T, DP, R><<<ctas, C::kThreads, C::kSmem, stream>>>(a);
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
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, DP, R>, a);
}

template <int T>
cudaError_t launch_type(const DecodeArgs& a, int dp, int r, cudaStream_t s) {
  if constexpr (T != SA_DTYPE_F32) {
    if (r == 16)
      return dp == 64 ? launch<T, 64, 16>(a, s) : dp == 128 ? launch<T, 128, 16>(a, s)
                                                            : launch<T, 256, 16>(a, s);
  }
  return dp == 64 ? launch<T, 64, 8>(a, s) : dp == 128 ? launch<T, 128, 8>(a, s)
                                                       : launch<T, 256, 8>(a, s);
}

}  // namespace dec1
}  // namespace sa
