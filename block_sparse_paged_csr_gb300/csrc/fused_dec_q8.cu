// Fused decode attention over a cache held in 8 bits (e4m3 or int8 codes, a
// scale per page and kv head): forward and log-sum-exp combine in one kernel,
// for batches in which every sequence holds at most one query.
//
// Work is cut as in the kernel for f32 and bf16 caches (fused_dec.cu): a
// "piece" is a range of ranks of one (query, kv head) pair, normally all of
// them; its kept blocks stream through shared memory, 128 keys a stage (two
// chunks of at most 64 keys of one block), under one online softmax; pieces of a
// cut pair meet in a small global scratch and the last one to finish merges them.
//
// Half the bytes per key of a bf16 cache leave half the time per stage: what
// bounds the kernel is no longer only HBM but how fast one SM can issue a
// stage's copies and turn its codes into products.  Hence:
//   * the metadata warp leaves page rows and scales ready per piece, so that a
//     load warp spends no division and one shared-memory round trip per stage;
//     16 lanes issue its 16 page copies (K and V, 2 KB each with pages of 16);
//   * consumers wait only for stages of their own: with at most 8 query rows
//     two groups of four warps take alternate stages (a piece has an even
//     number of them; a padding stage copies nothing);
//   * a consumer warp takes 32 keys of a stage at once: twice the independent
//     products between two dependent steps of the softmax, one maximum and one
//     rescale for both halves;
//   * all that it needs of a stage (flags, live keys, scales) is one 32-byte
//     record, and one lane per warp arrives on the barriers;
//   * codes go from shared memory to the MMA's registers as they lie: see
//     consumer().
// Roles: warp 0 metadata, warps 1..NL loads, then merge, then consumers.
// Measured, with the index build beside it: 128 sequences of 65536 to 131072 keys,
// 64 blocks of 64, 64 heads on 8, pages of 16, e4m3 (970 MB): 205 us, 4.7 TB/s
// (309 us with work cut as in the kernel for wider caches); 32 heads on 8, 64
// sequences, 16 blocks (124 MB): 49 us.  From 8 to 64 blocks a query, each 16 more take
// 43 us (268 MB, 6.2 TB/s of the 6.8 that a copy reaches: 0.8 us for an SM's 128
// keys, 32 KB); with cold caches a call takes 42 us besides, for its start
// (selected ids -> page ids -> scales -> keys), its changes of piece and its end, and
// 64 us where 768 pieces make five rounds of the SMs and a short sixth.  int8 takes 6 %
// longer than e4m3 (a quarter more instructions: its conversion), f32 queries as
// long as bf16 ones.
#include <cfloat>
#include <cstdint>
#include <cuda.h>

#include "internal.h"
#include "sa_common.cuh"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kD = 128;
constexpr int kCK = 64;              // keys per chunk
constexpr int kHalf = kCK * kD;      // bytes of a chunk's K (or V)
constexpr int kStage = 4 * kHalf;    // K of two chunks, V of two chunks
constexpr int kMaxEP = 64;           // ranks per piece
constexpr int kMaxPPB = 8;           // pages per block
constexpr int kDescs = 4;            // piece descriptors in flight
constexpr int kNL = 2;               // load warps (with metadata and merge one warpgroup)
constexpr uint32_t kFirst = 1u, kLast = 2u, kDone = 4u;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The softmax's reference m is not the running maximum itself: P = 2^(s - m) is
// formed with the m at hand, and only a score more than kSlack above it moves m
// up, to the whole number above the maximum (so that rescaling is exact).  So the
// products do not wait for a maximum over lanes.
// What meets V's codes is P times their page's scale, and o keeps a reference n of
// its own for that: it holds sums of P vs 2^(m - n).  A page whose scale is far
// from the others' may carry nearly all of the softmax and little of the output,
// or the other way round, so neither m nor the largest scale will do: n follows
// the largest product.  It moves up (and o is rescaled), to where that product
// counts 2^kTop, when m moves or when a page's vs 2^(m - n) is above kRoom: below it
// no P of at most 2^kSlack makes a product above 2^15 (f16 ends at 2^16), so pages
// of up to 2^4 times the scale of the one that set n cost nothing.  The f16 parts
// of a product resolve 2^-22 of it or 2^-25, which is 2^-28 of the largest.
constexpr float kSlack = 7.f, kTop = 4.f, kRoom = 256.f;

// What differs with the number of query rows R: consumer groups, stages.
template <int R> struct Q8Cfg;
template <> struct Q8Cfg<8> { static constexpr int G = 2, S = 4; };
template <> struct Q8Cfg<16> { static constexpr int G = 1, S = 4; };
// A load warp that is about to fill stage x waits for stage x - S to be
// consumed; the wait's parity tells that phase from the one before it only if
// stage x - 2 S is known to be consumed.  The warp's own earlier fill of stage
// x - m kNL saw stage x - m kNL - S consumed, and a group consumes in order: so
// some m with m kNL <= S and m kNL a multiple of G has to exist.
template <int R>
constexpr bool parity_is_safe() {
  for (int m = kNL; m <= Q8Cfg<R>::S; m += kNL)
    if (m % Q8Cfg<R>::G == 0) return true;
  return false;
}
static_assert(parity_is_safe<8>() && parity_is_safe<16>(), "load warps against the stage ring");

struct Q8Maps {
  CUtensorMap k, v;    // rows of 128 codes
};

struct PieceDesc {
  int32_t item, k, i, h, lk, nr;
  int32_t blk[kMaxEP];               // blocks of the kept ranks, in rank order
  int32_t row[kMaxEP][kMaxPPB];      // first pool row of their pages (-1: absent)
  float ks[kMaxEP][kMaxPPB];         // their K scales
  float vs[kMaxEP][kMaxPPB];         // their V scales
};

// One consumer warp's view of a stage: per chunk its 16 keys that exist (low
// and high half of `live`) and their page's scales.
struct __align__(16) Rec {
  float ks[2], vs[2];
  uint32_t live, flags, pad0, pad1;
};

struct StageInfo {
  int32_t item, k;
};

struct Q8Layout {
  uint32_t q, rec, info, mo, mm, mn, ml, desc, bars, flag, total;
};

__host__ __device__ constexpr uint32_t up_to(uint32_t x, uint32_t a) { return (x + a - 1) / a * a; }

template <int R>
__host__ __device__ constexpr Q8Layout q8_layout() {
  constexpr int S = Q8Cfg<R>::S, NC = 4 * Q8Cfg<R>::G;
  Q8Layout L{};
  L.q = S * kStage;                                            // Q slots [S][R][128] f32
  L.rec = L.q + S * R * kD * 4;                                // Rec[S][4]
  L.info = L.rec + S * 4 * static_cast<uint32_t>(sizeof(Rec));
  L.mo = up_to(L.info + S * static_cast<uint32_t>(sizeof(StageInfo)), 16);
  L.mm = L.mo + NC * R * kD * 4;                               // merge rows [NC][R][128]
  L.mn = L.mm + NC * R * 4;
  L.ml = L.mn + NC * R * 4;
  L.desc = up_to(L.ml + NC * R * 4, 16);
  L.bars = up_to(L.desc + kDescs * static_cast<uint32_t>(sizeof(PieceDesc)), 8);
  L.flag = L.bars + (2 * S + 2 * kDescs + 2) * 8;
  L.total = L.flag + 16;
  return L;
}

struct Smem {
  uint32_t spin;
  unsigned char* base;
  float* qs;
  Rec* rec;
  StageInfo* info;
  float* mo;
  float* mm;            // l's reference
  float* mn;            // o's
  float* ml;
  PieceDesc* desc;
  uint64_t *full, *empty, *dfull, *dempty;
  uint64_t* mready;     // consumers -> merge warp: the piece's states are in mo/mm/mn/ml
  uint64_t* mfree;      // merge warp -> consumers: the states have been read
  volatile int* minfo;  // item, k of the piece being merged (-1: no more pieces)
};

// ------------------------------------------------------------------ metadata

__device__ void meta_warp(const FusedQ8Args& qa, const Smem& sm, int64_t n_pieces, int lane) {
  const FusedDecArgs& a = qa.base;
  uint32_t n = 0;
  for (int64_t g = blockIdx.x;; g += gridDim.x, ++n) {
    const int slot = static_cast<int>(n % kDescs);
    if (n >= static_cast<uint32_t>(kDescs) &&
        !mbar_wait_bounded(sm.dempty + slot, ((n / kDescs) - 1) & 1u, sm.spin)) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
      return;
    }
    PieceDesc& d = sm.desc[slot];
    if (g >= n_pieces) {
      if (lane == 0) d.item = -1;
      __syncwarp();
      mbar_arrive(sm.dfull + slot);
      return;
    }
    int64_t item;
    int k, r0, nrange;
    if (g < a.whole_items) {            // a whole pair: all its ranks
      item = g;
      k = 0;
      r0 = 0;
      nrange = a.topk;
    } else {
      const int64_t t = g - a.whole_items;
      item = a.whole_items + t / a.pieces;
      k = static_cast<int>(t - (item - a.whole_items) * a.pieces);
      r0 = k * a.ranks_per_piece;
      nrange = min(a.ranks_per_piece, a.topk - r0);
    }
    const int64_t i = item / a.hkv;
    const int h = static_cast<int>(item - i * a.hkv);
    // The selection's ids do not wait for the sequence; nor does its length
    // where every sequence so far holds one query (then b = i).
    int blk_of[kMaxEP / 32];
#pragma unroll
    for (int half = 0; half < kMaxEP / 32; ++half) {
      const int jr = 32 * half + lane;
      blk_of[half] = jr < nrange ? a.selected[(i * a.hkv + h) * a.topk + r0 + jr] : -1;
    }
    int b = static_cast<int>(min(i, static_cast<int64_t>(a.batch - 1)));
    const int64_t c0 = a.cu[b], c1 = a.cu[b + 1];
    int lk = a.used ? a.used[b] : a.msb * a.block_size;
    if (c0 > i || c1 <= i) {
      b = warp_search(a.batch, lane, [&](int x) { return a.cu[x] <= i; });
      if (a.used) lk = a.used[b];
    }
    lk = max(lk, 0);
    int nkept = 0;
#pragma unroll
    for (int half = 0; half < kMaxEP / 32; ++half) {
      // the index's rule for keeping an entry: a block id in [0, msb) whose
      // first key lies below the sequence's KV length
      const int blk = blk_of[half];
      if (blk < -1 || blk >= a.msb) report(a.status, SA_ERR_SELECTED_RANGE);
      const bool kept = blk >= 0 && blk < a.msb && static_cast<int64_t>(blk) * a.block_size < lk;
      const unsigned km = __ballot_sync(0xffffffffu, kept);
      if (kept) d.blk[nkept + __popc(km & ((1u << lane) - 1u))] = blk;
      nkept += __popc(km);
    }
    __syncwarp();
    // pages and scales, one (rank, page) per lane, four in flight
    const int ppb = a.pages_per_block;
    const int32_t* bt = a.block_tables + static_cast<int64_t>(b) * a.max_pages;
#pragma unroll 1
    for (int t0 = lane; t0 < nkept * ppb; t0 += 4 * 32) {
      int id[4], at[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = t0 + 32 * x;
        const int pos = t / ppb, p = t - pos * ppb;
        id[x] = -1;
        at[x] = pos * kMaxPPB + p;
        if (t < nkept * ppb) {
          const int64_t page = static_cast<int64_t>(d.blk[pos]) * ppb + p;
          if (page * a.page_size < lk) id[x] = bt[page];
        } else {
          at[x] = -1;
        }
      }
      float ks[4], vs[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (id[x] >= a.num_pages) {
          report(a.status, SA_ERR_SHAPE);
          id[x] = -1;
        }
        const int64_t of = static_cast<int64_t>(max(id[x], 0)) * a.hkv + h;
        ks[x] = id[x] >= 0 ? __ldg(qa.k_scales + of) : 0.f;
        vs[x] = id[x] >= 0 ? __ldg(qa.v_scales + of) : 0.f;
        if (at[x] >= 0) (&d.row[0][0])[at[x]] = id[x] >= 0 ? static_cast<int>(of * a.page_size) : -1;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (at[x] >= 0) {
          (&d.ks[0][0])[at[x]] = ks[x];
          (&d.vs[0][0])[at[x]] = vs[x];
        }
    }
    if (lane == 0) {
      d.item = static_cast<int>(item);
      d.k = k;
      d.i = static_cast<int>(i);
      d.h = h;
      d.lk = lk;
      d.nr = nkept;
    }
    __syncwarp();
    mbar_arrive(sm.dfull + slot);
  }
}

// ------------------------------------------------------------------ loads

// Load warp lw: fills the stages whose running index is lw modulo kNL.  Lane =
// (chunk, K or V, 16-key group) of the stage: it resolves its group's page
// row, live keys and scale; the first group of each page box issues its copy.
template <int R>
__device__ void load_warp(const Q8Maps& maps, const FusedQ8Args& qa, const Smem& sm, int lw,
                          int lane) {
  constexpr uint32_t S = Q8Cfg<R>::S, G = Q8Cfg<R>::G;
  const FusedDecArgs& a = qa.base;
  const int ck = a.block_size < kCK ? a.block_size : kCK;           // keys per chunk
  const int cpb = a.block_size / ck;                                // chunks per block
  const int lps = __ffs(a.page_size) - 1;                           // page_size is a power of two
  const int kb = a.page_size < ck ? a.page_size : ck;               // keys per page box
  const uint32_t box_bytes = static_cast<uint32_t>(kb) * kD;
  const uint32_t q_bytes = static_cast<uint32_t>(a.qhead) * kD * (qa.act_bf16 ? 2u : 4u);
  const int key = 16 * (lane & 3);                // first key of the lane's group
  const bool is_v = (lane & 4) != 0;
  const int half = (lane >> 3) & 1;
  const bool busy = lane < 16 && key < ck;
  const bool box_lane = busy && (key & (kb - 1)) == 0;
  const CUtensorMap* map = is_v ? &maps.v : &maps.k;
  const uint32_t dst = static_cast<uint32_t>((is_v ? 2 * kHalf : 0) + half * kHalf + key * kD);
  uint32_t n = 0, xs = 0;          // pieces, stages of all load warps
  uint32_t mine = lw;              // this warp's next stage
  bool ok = true;
  if (a.stall) return;   // test hook: no stage is ever filled, so every wait on one runs out
  for (;;) {
    const int slot = static_cast<int>(n % kDescs);
    if (!mbar_wait_bounded(sm.dfull + slot, (n / kDescs) & 1u, sm.spin)) {
      ok = false;
      break;
    }
    const PieceDesc& d = sm.desc[slot];
    const int item = d.item;
    if (item < 0) {
      // the end, told to every group
      for (uint32_t g = 0; g < G; ++g, ++xs) {
        if (xs != mine) continue;
        const uint32_t s = xs % S;
        if (xs >= S && !mbar_wait_bounded(sm.empty + s, ((xs / S) - 1) & 1u, sm.spin)) {
          ok = false;
          break;
        }
        if (lane < 4) sm.rec[s * 4 + lane].flags = kDone;
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.full + s);
        mine += kNL;
      }
      break;
    }
    const int nr = d.nr;
    const int real = nr * cpb;                    // chunks
    // stages: a multiple of G, at least one for every group
    const uint32_t need = (static_cast<uint32_t>(real) + 1) / 2;
    const uint32_t nst = need == 0 ? G : (need + G - 1) / G * G;
    if (mine < xs + nst) {
      const int lk = d.lk, h = d.h, i = d.i, kk = d.k;
      uint32_t u = mine - xs;
      int ch = 2 * static_cast<int>(u) + half;    // the lane's chunk of the piece
      int j = ch / cpb, c = ch - j * cpb;
      for (; u < nst; u += kNL, mine += kNL) {
        const uint32_t s = mine % S;
        // the stage's pages, resolved before the wait for its slot
        int live = 0;
        int row = -1;
        float sc = 0.f;
        if (busy && ch < real) {
          const int off = c * ck + key;                  // key of the block
          const int p = off >> lps;
          const int left = lk - (d.blk[j] * a.block_size + off);
          row = d.row[j][p];
          sc = is_v ? d.vs[j][p] : d.ks[j][p];
          live = row >= 0 ? min(max(left, 0), 16) : 0;
          row += off - (p << lps);
        }
        const bool copy = box_lane && live > 0;
        const unsigned pm = __ballot_sync(0xffffffffu, copy);
        const bool with_q = u < G && nr > 0;
        const uint32_t mask = (1u << live) - 1u;
        const uint32_t mask1 = __shfl_down_sync(0xffffffffu, mask, 8);   // of chunk 1
        if (mine >= S && !mbar_wait_bounded(sm.empty + s, ((mine / S) - 1) & 1u, sm.spin)) {
          ok = false;
          break;
        }
        if (lane < 16) {
          Rec& r = sm.rec[s * 4 + (lane & 3)];
          (is_v ? r.vs : r.ks)[half] = sc;
          if (lane < 4) {
            r.live = mask | (mask1 << 16);
            r.flags = (u < G ? kFirst : 0u) | (u + G >= nst ? kLast : 0u);
          }
        } else if (lane == 16) {
          sm.info[s] = StageInfo{item, kk};
        }
        __syncwarp();
        if (lane == 0)
          mbar_arrive_expect_tx(sm.full + s, static_cast<uint32_t>(__popc(pm)) * box_bytes +
                                                 (with_q ? q_bytes : 0u));
        __syncwarp();
        if (copy) tma_load_2d(sm.base + s * kStage + dst, map, 0, row, sm.full + s);
        if (with_q && lane == 16) {
          const int64_t qrow = static_cast<int64_t>(i) * a.hq + static_cast<int64_t>(h) * a.qhead;
          bulk_g2s(sm.qs + s * R * kD,
                   static_cast<const unsigned char*>(qa.q) + qrow * kD * (qa.act_bf16 ? 2 : 4),
                   q_bytes, sm.full + s);
        }
        ch += 2 * kNL;
        c += 2 * kNL;
        while (c >= cpb) {
          c -= cpb;
          ++j;
        }
      }
      if (!ok) break;
    }
    xs += nst;
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.dempty + slot);
    ++n;
  }
  if (!ok) {
    if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
    // Let this warp's copies still in flight land before the CTA can exit.
    for (uint32_t x = mine % kNL; x < mine; x += kNL)
      if (x + S >= mine) mbar_wait_bounded(sm.full + x % S, (x / S) & 1u, sm.spin);
  }
}

// 2^x (ex2.approx: relative error about 2^-22; results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ piece end

// 2^d for a whole number d up to 127 (0 below -126).
__device__ __forceinline__ float pow2_of(float d) {
  return d < -126.f ? 0.f
                    : __uint_as_float(static_cast<uint32_t>(static_cast<int>(fminf(d, 127.f)) + 127) << 23);
}

__device__ __forceinline__ void write_row(const FusedQ8Args& qa, int64_t row, int d4, float m2,
                                          float l, float4 o) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  store_o4(qa.out, qa.act_bf16, row * kD + 4 * d4,
           make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (qa.base.lse && d4 == 0) qa.base.lse[row] = l > 0.f ? (m2 + log2f(l)) * kLn2 : -INFINITY;
}

// Where consumers put 16-byte chunk c of row r of a merge row: a consumer's
// lanes hold (row, 32 consecutive channels), which without the XOR all fall
// on the same banks.
__device__ __forceinline__ int merge_chunk(int c, int r) { return c ^ (c >> 3) ^ ((r & 1) << 2); }

// The merge warp.  Per piece: merge the consumer warps' states (m and n in the
// log2 domain) row by row, lane = 4 channels; release the state buffer; then
// either write the output rows (one piece per pair) or the piece's scratch
// rows, and if this piece is the pair's last to finish (a counter per pair),
// merge the pair's scratch rows into the output.
template <int R>
__device__ void merge_warp(const FusedQ8Args& qa, const Smem& sm, int lane) {
  constexpr int NC = 4 * Q8Cfg<R>::G;
  const FusedDecArgs& a = qa.base;
  const int qhead = a.qhead;
  for (uint32_t np = 0;; ++np) {
    if (!mbar_wait_bounded(sm.mready, np & 1u, sm.spin)) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
      return;
    }
    const int item = sm.minfo[0];
    const int k = sm.minfo[1];
    if (item < 0) return;
    const int P = item < a.whole_items ? 1 : a.pieces;
    const int64_t i = item / a.hkv;
    const int h = item - static_cast<int>(i) * a.hkv;
    const int64_t row0 = i * a.hq + static_cast<int64_t>(h) * qhead;
    // scratch row of (pair, piece kk, lane r): (item * topk + kk) * qhead + r
    const int64_t prow = static_cast<int64_t>(item) * a.topk * qhead;
    for (int r = 0; r < qhead; ++r) {
      float M = -INFINITY, N = -INFINITY;
#pragma unroll
      for (int w = 0; w < NC; ++w) {
        M = fmaxf(M, sm.mm[w * R + r]);
        N = fmaxf(N, sm.mn[w * R + r]);
      }
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < NC; ++w) {
          l = fmaf(pow2_of(sm.mm[w * R + r] - M), sm.ml[w * R + r], l);
          const float e = pow2_of(sm.mn[w * R + r] - N);
          const float4 v =
              reinterpret_cast<const float4*>(sm.mo + (w * R + r) * kD)[merge_chunk(lane, r)];
          o.x = fmaf(e, v.x, o.x);
          o.y = fmaf(e, v.y, o.y);
          o.z = fmaf(e, v.z, o.z);
          o.w = fmaf(e, v.w, o.w);
        }
        // from o's unit 2^N to l's, 2^M, in two halves: the values of a row with
        // scales near the ends of f32's range stay inside it
        const float half = truncf(0.5f * (N - M));
        const float h0 = pow2_of(half), h1 = pow2_of(N - M - half);
        o = make_float4(o.x * h0 * h1, o.y * h0 * h1, o.z * h0 * h1, o.w * h0 * h1);
      }
      if (P == 1) {
        write_row(qa, row0 + r, lane, M, l, o);
      } else {
        const int64_t pr = prow + static_cast<int64_t>(k) * qhead + r;
        store_o4(a.part_o, a.part_bf16, pr * kD + 4 * lane, o);
        if (lane == 0) {
          a.part_m[pr] = M;
          a.part_l[pr] = l;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.mfree);
    if (P == 1) continue;
    __threadfence();
    __syncwarp();
    unsigned last = 0;
    if (lane == 0) {
      const unsigned old = atomicAdd(a.item_cnt + item, 1u);
      last = old == static_cast<unsigned>(P - 1);
      if (last) atomicExch(a.item_cnt + item, 0u);
    }
    last = __shfl_sync(0xffffffffu, last, 0);
    if (!last) continue;
    __threadfence();
    // The pair's P scratch rows, four GQA lanes at a time: statistics one (lane,
    // piece) row per thread, then the o rows, eight loads in flight.
    for (int r = 0; r < qhead; r += 4) {
      // lanes 8 x + y: GQA lane r + x, pieces y, y + 8, ..
      const int rr = r + (lane >> 3);
      const bool there = rr < qhead;
      float M = -INFINITY;
      for (int b = lane & 7; b < P; b += 8)
        if (there) M = fmaxf(M, __ldcg(a.part_m + prow + static_cast<int64_t>(b) * qhead + rr));
#pragma unroll
      for (int off = 4; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      float l = 0.f;
      float4 o[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int b0 = 0; b0 < P; b0 += 8) {
        const int b = b0 + (lane & 7);
        float e = 0.f;
        if (there && b < P && M != -INFINITY) {
          const int64_t pr = prow + static_cast<int64_t>(b) * qhead + rr;
          e = ex2(__ldcg(a.part_m + pr) - M);
          l = fmaf(e, __ldcg(a.part_l + pr), l);
        }
#pragma unroll 1
        for (int y = 0; y < 8 && b0 + y < P; y += 2) {
          float4 v[4][2];
          float wt[4][2];
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              wt[x][t] = __shfl_sync(0xffffffffu, e, 8 * x + y + t);
              v[x][t] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (wt[x][t] > 0.f) {
                const int64_t at =
                    (prow + static_cast<int64_t>(b0 + y + t) * qhead + r + x) * kD + 4 * lane;
                v[x][t] = a.part_bf16
                              ? bf16x4_to_f32(__ldcg(reinterpret_cast<const uint2*>(
                                    static_cast<const uint16_t*>(a.part_o) + at)))
                              : __ldcg(reinterpret_cast<const float4*>(
                                    static_cast<const float*>(a.part_o) + at));
              }
            }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              o[x].x = fmaf(wt[x][t], v[x][t].x, o[x].x);
              o[x].y = fmaf(wt[x][t], v[x][t].y, o[x].y);
              o[x].z = fmaf(wt[x][t], v[x][t].z, o[x].z);
              o[x].w = fmaf(wt[x][t], v[x][t].w, o[x].w);
            }
        }
      }
#pragma unroll
      for (int off = 4; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float mx = __shfl_sync(0xffffffffu, M, 8 * x);
        const float lx = __shfl_sync(0xffffffffu, l, 8 * x);
        if (r + x < qhead) write_row(qa, row0 + r + x, lane, mx, lx, o[x]);
      }
    }
  }
}

// ------------------------------------------------------------------ consumers

// d = a b (m16n8k16, f16 operands, f32 accumulation) from zero, and d += a b.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two values as f16 high parts and f16 remainders (22 bits together).
__device__ __forceinline__ void split2h(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
  const float2 h = f16x2_to_f32(hi);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x1 - h.y), "f"(x0 - h.x));
}

// Warp-level MMA (m16n8k16) on f16 operands.  Codes of both types are exact in
// f16; Q (its row scaled by a power of two into f16's range) and P are split
// into f16 high parts and remainders, so products lose no more than 2^-22.
// The scale of a 16-key group's page meets K on the scores and V on P (see kSlack):
// every product of the piece adds to one accumulator.
//
// Codes need no transposition and no repacking through shared memory: a
// fragment's k index may stand for any channel (scores) and its n index for
// any channel (output) as long as both operands agree.
//   scores: lane (g, c) reads the 16-byte chunks 2c and 2c + 1 of key g's row
//     (channels 32 c ..) and serves them as the k-steps' B fragments, 4 codes
//     each; Q's fragments hold the same channels.
//   output: lane (g, c) reads chunk g (channels 16 g ..) of the four keys that
//     its fragment's k indices stand for, interleaves the keys' bytes and
//     serves channel 16 g + j as n-tile j.
// Both reads are free of bank conflicts under the 128-byte swizzle.
//
// R = 8 (at most 8 query rows): rows g + 8 of the m16 tile carry the
// remainders of rows g, so the split costs no product.  R = 16: remainders in
// products of their own.
template <bool kI8, int R>
__device__ void consumer(const FusedQ8Args& qa, const Smem& sm, int warp, int lane) {
  constexpr uint32_t S = Q8Cfg<R>::S, G = Q8Cfg<R>::G;
  constexpr int NR = R / 8;                       // query rows per lane: g (and g + 8)
  const FusedDecArgs& a = qa.base;
  const int w = warp & 3;                         // the warp's 16 keys of each chunk
  const int g = lane >> 2, c = lane & 3;
  const uint32_t k_at = static_cast<uint32_t>((16 * w + g) * 128 + (((2 * c) ^ g) << 4));
  const uint32_t v_at = static_cast<uint32_t>(2 * kHalf + (16 * w + 2 * c) * 128);
  const uint32_t v_c0 = static_cast<uint32_t>((g ^ (2 * c)) << 4);
  const uint32_t v_c1 = v_c0 ^ 16u;

  float m_run[NR], n_run[NR];        // the references m and n, in the log2 domain
  float vfac[NR];                    // 2^(m - n)
  float l_part[NR], sfac[NR];
  float o[16][4];                    // [n-tile j][row g: columns 2c, 2c + 1 | row g + 8]
  uint32_t qf[8][4];                 // R = 8: high parts | remainders; R = 16: high parts
  uint32_t ql[R == 16 ? 8 : 1][4];   // R = 16: remainders
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    m_run[r] = n_run[r] = -INFINITY;
    vfac[r] = 1.f;
    l_part[r] = 0.f;
    sfac[r] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qf[j][e] = 0u;
      if constexpr (R == 16) ql[j][e] = 0u;
    }

  uint32_t handed = 0;
  for (uint32_t xc = G == 1 ? 0u : static_cast<uint32_t>(warp) >> 2;; xc += G) {
    const uint32_t s = xc % S;
    if (!mbar_wait_bounded(sm.full + s, (xc / S) & 1u, sm.spin)) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
      return;
    }
    const Rec rec = sm.rec[s * 4 + w];
    if (rec.flags & kDone) {
      if (handed == 0 || mbar_wait_bounded(sm.mfree, (handed - 1) & 1u, sm.spin)) {
        if (warp == 0 && lane == 0) sm.minfo[0] = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.mready);
      }
      return;
    }
    if (rec.flags & kFirst) {
      // Q rows g (and g + 8): lane's channels of k-step j are 32 c + 4 j ..
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int row = g + 8 * r;
        const float* q32 = sm.qs + s * R * kD + row * kD;
        const uint16_t* q16 = reinterpret_cast<const uint16_t*>(sm.qs + s * R * kD) + row * kD;
        float4 x[8];
        float am = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ch = 32 * c + 4 * j;
          x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row < a.qhead)
            x[j] = qa.act_bf16 ? bf16x4_to_f32(*reinterpret_cast<const uint2*>(q16 + ch))
                               : *reinterpret_cast<const float4*>(q32 + ch);
          am = fmaxf(am, fmaxf(fmaxf(fabsf(x[j].x), fabsf(x[j].y)),
                               fmaxf(fabsf(x[j].z), fabsf(x[j].w))));
        }
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // largest magnitude to [2^10, 2^11): f = 2^(137 - E) with E its biased
        // exponent, f and 1 / f kept normal
        const int ex = min(max(static_cast<int>(__float_as_uint(am) >> 23), 11), 253);
        const float f = __uint_as_float(static_cast<uint32_t>(264 - ex) << 23);
        sfac[r] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(ex - 10) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t h0, l0, h1, l1;
          split2h(x[j].x * f, x[j].y * f, h0, l0);
          split2h(x[j].z * f, x[j].w * f, h1, l1);
          if constexpr (R == 8) {
            qf[j][0] = h0;
            qf[j][1] = l0;
            qf[j][2] = h1;
            qf[j][3] = l1;
          } else {
            qf[j][r] = h0;
            qf[j][2 + r] = h1;
            ql[j][r] = l0;
            ql[j][2 + r] = l1;
          }
        }
        m_run[r] = n_run[r] = -INFINITY;
        vfac[r] = 1.f;
        l_part[r] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }
    // NH chunks at once; a chunk without live keys counts p = 0 (its maximum is
    // left out), and a pass without any is skipped
    constexpr int NH = R == 8 ? 2 : 1;
#pragma unroll 1
    for (int h0 = 0; h0 < 2; h0 += NH) {
      const uint32_t mk = NH == 2 ? rec.live : (rec.live >> (16 * h0)) & 0xFFFFu;
      if (mk == 0u) continue;
      constexpr uint32_t kAll = NH == 2 ? 0xFFFFFFFFu : 0xFFFFu;
      const bool whole = mk == kAll;
      const unsigned char* st = sm.base + s * kStage + h0 * kHalf;
      // (chunk 2c + 1: the XOR with g flips bit 4 of the address)
      const int32_t flip = (g & 1) ? -16 : 16;
      // ---- S = Q K^T: per n-tile of 8 keys two chains of products ----
      float part[NH][2][2][4];
      uint4 kr[NH][2][2];
#pragma unroll
      for (int hh = 0; hh < NH; ++hh)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const unsigned char* kt = st + hh * kHalf + k_at + nt * 1024;
          kr[hh][nt][0] = *reinterpret_cast<const uint4*>(kt);
          kr[hh][nt][1] = *reinterpret_cast<const uint4*>(kt + flip);
        }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int hh = 0; hh < NH; ++hh)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const uint4 u = kr[hh][nt][j >> 2];
            const uint32_t code = (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
            uint32_t b0, b1;
            codes4_to_f16<kI8>(code, b0, b1);
            if (j < 2)
              mma_first(part[hh][nt][j & 1], qf[j], b0, b1);
            else
              mma_add(part[hh][nt][j & 1], qf[j], b0, b1);
            if constexpr (R == 16) mma_add(part[hh][nt][j & 1], ql[j], b0, b1);
          }
      // ---- online softmax ----
      uint32_t pf[NH][4], pl[NH][R == 16 ? 4 : 1];
      float x[NR][NH][2][2];
      bool beyond = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float sub = -m_run[r];                     // +inf before the first keys
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          const float f = sfac[r] * rec.ks[NH == 2 ? hh : h0];
          beyond = beyond || fabsf(rec.vs[NH == 2 ? hh : h0] * vfac[r]) > kRoom;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float sum;
              if constexpr (R == 8)
                sum = (part[hh][nt][0][e] + part[hh][nt][1][e]) +
                      (part[hh][nt][0][e + 2] + part[hh][nt][1][e + 2]);
              else
                sum = part[hh][nt][0][e + 2 * r] + part[hh][nt][1][e + 2 * r];
              x[r][hh][nt][e] = fmaf(sum, f, sub);
              if (!whole && !((mk >> (16 * hh + 8 * nt + 2 * c + e)) & 1u))
                x[r][hh][nt][e] = -INFINITY;
              beyond = beyond || x[r][hh][nt][e] > kSlack;
              part[hh][nt][0][e + (R == 8 ? 0 : 2 * r)] = sum;
            }
        }
      }
      if (__any_sync(0xffffffffu, beyond)) {
        // a score well above the reference (the piece's first keys among them), or
        // a page of a large V scale
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float cm = -INFINITY, top = -INFINITY;         // largest score, largest product
#pragma unroll
          for (int hh = 0; hh < NH; ++hh) {
            const float f = sfac[r] * rec.ks[NH == 2 ? hh : h0];
            float chunk = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const bool live = (mk >> (16 * hh + 8 * nt + 2 * c + e)) & 1u;
                const float v = part[hh][nt][0][e + (R == 8 ? 0 : 2 * r)] * f;
                x[r][hh][nt][e] = live ? v : -INFINITY;
                chunk = fmaxf(chunk, x[r][hh][nt][e]);
              }
            cm = fmaxf(cm, chunk);
            top = fmaxf(top, chunk + log2f(fabsf(rec.vs[NH == 2 ? hh : h0])));
          }
          cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 1));
          cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 2));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // finite: the warp has a key
          const float m_new = fmaxf(m_run[r], ceilf(cm));
          l_part[r] *= pow2_of(m_run[r] - m_new);
          m_run[r] = m_new;
          // (pages of zeros only: the lowest n whose 2^(m - n) is a number)
          const float n_new = fmaxf(fmaxf(n_run[r], ceilf(top) - kTop), m_new - 127.f);
          const float beta = pow2_of(n_run[r] - n_new);
          n_run[r] = n_new;
          vfac[r] = pow2_of(m_new - n_new);
#pragma unroll
          for (int hh = 0; hh < NH; ++hh)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) x[r][hh][nt][e] -= m_new;
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (R == 8 || e / 2 == r) o[j][e] *= beta;
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float lsum = 0.f;
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          float p[2][2];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) p[nt][e] = ex2(x[r][hh][nt][e]);
          lsum += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
          // (a number: a page far above the others' scales may pass f32's range where
          // its keys' P is 0)
          const float vs =
              fminf(fmaxf(rec.vs[NH == 2 ? hh : h0] * vfac[r], -FLT_MAX), FLT_MAX);
          if constexpr (R == 8) {
            split2h(p[0][0] * vs, p[0][1] * vs, pf[hh][0], pf[hh][1]);
            split2h(p[1][0] * vs, p[1][1] * vs, pf[hh][2], pf[hh][3]);
          } else {
            split2h(p[0][0] * vs, p[0][1] * vs, pf[hh][r], pl[hh][r]);
            split2h(p[1][0] * vs, p[1][1] * vs, pf[hh][2 + r], pl[hh][2 + r]);
          }
        }
        l_part[r] += lsum;
      }
      // ---- o += P V (n-tile j: channels 16 n + j) ----
#pragma unroll
      for (int hh = 0; hh < NH; ++hh) {
        const unsigned char* vt = st + hh * kHalf + v_at;
        const uint4 v0 = *reinterpret_cast<const uint4*>(vt + v_c0);
        const uint4 v1 = *reinterpret_cast<const uint4*>(vt + 128 + v_c1);
        const uint4 v2 = *reinterpret_cast<const uint4*>(vt + 1024 + v_c0);
        const uint4 v3 = *reinterpret_cast<const uint4*>(vt + 1152 + v_c1);
        uint32_t y[4][4] = {{v0.x, v0.y, v0.z, v0.w}, {v1.x, v1.y, v1.z, v1.w},
                            {v2.x, v2.y, v2.z, v2.w}, {v3.x, v3.y, v3.z, v3.w}};
        if (!whole) {
          // rows behind the sequence's end hold anything (NaN codes too): zeros
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (!((mk >> (16 * hh + 2 * c + (t & 1) + 4 * (t & 2))) & 1u)) {
#pragma unroll
              for (int q = 0; q < 4; ++q) y[t][q] = 0u;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t b[4][2];
          codes4_to_f16<kI8>(__byte_perm(y[0][q], y[1][q], 0x5140), b[0][0], b[1][0]);
          codes4_to_f16<kI8>(__byte_perm(y[0][q], y[1][q], 0x7362), b[2][0], b[3][0]);
          codes4_to_f16<kI8>(__byte_perm(y[2][q], y[3][q], 0x5140), b[0][1], b[1][1]);
          codes4_to_f16<kI8>(__byte_perm(y[2][q], y[3][q], 0x7362), b[2][1], b[3][1]);
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const int j = 4 * q + jj;
            mma_add(o[j], pf[hh], b[jj][0], b[jj][1]);
            if constexpr (R == 16) mma_add(o[j], pl[hh], b[jj][0], b[jj][1]);
          }
        }
      }
    }
    __syncwarp();
    if (rec.flags & kLast) {
      const StageInfo info = sm.info[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.empty + s);
      if (handed != 0 && !mbar_wait_bounded(sm.mfree, (handed - 1) & 1u, sm.spin)) {
        if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
        return;
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float l = l_part[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = g + 8 * r;
        float4* dst = reinterpret_cast<float4*>(sm.mo + (warp * R + row) * kD);
        // (R = 8: the remainders' row joins its own)
        auto at = [&](int j, int e) {
          return R == 8 ? o[j][e] + o[j][e + 2] : o[j][2 * r + e];
        };
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[merge_chunk(8 * c + 4 * e + q, row)] =
                make_float4(at(4 * q, e), at(4 * q + 1, e), at(4 * q + 2, e), at(4 * q + 3, e));
        if (c == 0) {
          sm.mm[warp * R + row] = m_run[r];
          sm.mn[warp * R + row] = n_run[r];
          sm.ml[warp * R + row] = l;
        }
      }
      if (warp == 0 && lane == 0) {
        sm.minfo[0] = info.item;
        sm.minfo[1] = info.k;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.mready);
      ++handed;
    } else if (lane == 0) {
      mbar_arrive(sm.empty + s);
    }
  }
}

// ------------------------------------------------------------------ kernel

// Registers: 48 K of the SM's 64 K at launch, so that a CTA of the index build
// (256 threads x 64) fits beside; the first warpgroup (metadata, loads, merge)
// hands most of its share to the consumers.
template <int R> struct Q8Regs;
template <> struct Q8Regs<8> { static constexpr int kLaunch = 128, kOthers = 96, kConsumers = 144; };
template <> struct Q8Regs<16> { static constexpr int kLaunch = 192, kOthers = 96, kConsumers = 248; };
static_assert(2 + kNL == 4, "metadata, load and merge warps fill one warpgroup");
template <int R>
constexpr bool registers_fit() {
  constexpr int nc = 128 * Q8Cfg<R>::G;
  return 128 * Q8Regs<R>::kOthers + nc * Q8Regs<R>::kConsumers <= (128 + nc) * Q8Regs<R>::kLaunch &&
         (128 + nc) * Q8Regs<R>::kLaunch + 256 * 64 <= 65536;
}
static_assert(registers_fit<8>() && registers_fit<16>(), "register shares");

// (The name that sa_attention_kernel_name gives for the fused decode path.)
template <bool kI8, int R>
__global__ void __maxnreg__(Q8Regs<R>::kLaunch)
fused_dec_kernel(const __grid_constant__ Q8Maps maps, const __grid_constant__ FusedQ8Args a) {
  extern __shared__ unsigned char smem_raw[];
  constexpr Q8Layout L = q8_layout<R>();
  constexpr int S = Q8Cfg<R>::S, NC = 4 * Q8Cfg<R>::G;
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Smem sm;
  sm.spin = a.base.spin_limit ? a.base.spin_limit : kSpinLimit;
  sm.base = base;
  sm.qs = reinterpret_cast<float*>(base + L.q);
  sm.rec = reinterpret_cast<Rec*>(base + L.rec);
  sm.info = reinterpret_cast<StageInfo*>(base + L.info);
  sm.mo = reinterpret_cast<float*>(base + L.mo);
  sm.mm = reinterpret_cast<float*>(base + L.mm);
  sm.mn = reinterpret_cast<float*>(base + L.mn);
  sm.ml = reinterpret_cast<float*>(base + L.ml);
  sm.desc = reinterpret_cast<PieceDesc*>(base + L.desc);
  sm.full = reinterpret_cast<uint64_t*>(base + L.bars);
  sm.empty = sm.full + S;
  sm.dfull = sm.empty + S;
  sm.dempty = sm.dfull + kDescs;
  sm.mready = sm.dempty + kDescs;
  sm.mfree = sm.mready + 1;
  sm.minfo = reinterpret_cast<volatile int*>(base + L.flag);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(sm.full + s, 1);
      mbar_init(sm.empty + s, 4);
    }
    for (int d = 0; d < kDescs; ++d) {
      mbar_init(sm.dfull + d, 32);
      mbar_init(sm.dempty + d, kNL);
    }
    mbar_init(sm.mready, NC);
    mbar_init(sm.mfree, 1);
    fence_mbar_init();
  }
  __syncthreads();

  const int64_t n_pieces =
      a.base.whole_items + (a.base.tq * a.base.hkv - a.base.whole_items) * a.base.pieces;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Q8Regs<R>::kOthers));
    if (warp == 0)
      meta_warp(a, sm, n_pieces, lane);
    else if (warp <= kNL)
      load_warp<R>(maps, a, sm, warp - 1, lane);
    else
      merge_warp<R>(a, sm, lane);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Q8Regs<R>::kConsumers));
    consumer<kI8, R>(a, sm, warp - 4, lane);
  }
  // Launched behind the index kernel (programmatic dependent launch): finish
  // only after it, so that later work of the stream sees both complete.
  if (a.base.pdl) griddep_wait();
}

// ------------------------------------------------------------------ host

// K or V pool [num_pages, hkv, page_size, 128] as rows of one key.
bool encode_pool(const void* pool, int64_t rows, int kb, CUtensorMap* map) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {kD, static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {kD};
  const cuuint32_t box[2] = {kD, static_cast<cuuint32_t>(kb)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kI8, int R>
cudaError_t launch_q8(const FusedQ8Args& a, cudaStream_t stream) {
  constexpr size_t smem = q8_layout<R>().total + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  constexpr int threads = (2 + kNL + 4 * Q8Cfg<R>::G) * 32;
  const FusedDecArgs& b = a.base;
  const int ck = b.block_size < kCK ? b.block_size : kCK;
  const int kb = b.page_size < ck ? b.page_size : ck;
  const int64_t rows = b.num_pages * b.hkv * b.page_size;
  Q8Maps maps;
  if (!encode_pool(b.k_pages, rows, kb, &maps.k) || !encode_pool(b.v_pages, rows, kb, &maps.v))
    return cudaErrorNotSupported;
  const void* fn = reinterpret_cast<const void*>(fused_dec_kernel<kI8, R>);
  static SmemLimit limit;
  const cudaError_t err = limit.raise(fn, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int64_t n_pieces = b.whole_items + (b.tq * b.hkv - b.whole_items) * b.pieces;
  int64_t grid = device_sm_count();
  if (grid > n_pieces) grid = n_pieces;
  if (grid < 1) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = b.pdl ? 1 : 0;
  FusedQ8Args args = a;
  int site = kStallNone;
  debug_stall_setting(&site, &args.base.spin_limit);
  args.base.stall = site == kStallFusedCopies;
  return cudaLaunchKernelEx(&cfg, fused_dec_kernel<kI8, R>, maps, args);
}

}  // namespace

bool fused_dec_q8_supported(int head_dim, int block_size, int page_size, int qhead) {
  if (head_dim != kD) return false;
  // a 16-key step of a consumer lies in one page (one scale)
  if (page_size < 16 || (page_size & (page_size - 1)) != 0) return false;
  if (block_size <= 0 || block_size % page_size != 0) return false;
  if (block_size / page_size > kMaxPPB) return false;
  if (block_size > kCK && block_size % kCK != 0) return false;
  return qhead >= 1 && qhead <= 16;
}

cudaError_t launch_fused_dec_q8(const FusedQ8Args& a, cudaStream_t stream) {
  const FusedDecArgs& b = a.base;
  if (!fused_dec_q8_supported(kD, b.block_size, b.page_size, b.qhead)) return cudaErrorNotSupported;
  if (b.ranks_per_piece < 1 || b.ranks_per_piece > kMaxEP || b.pieces < 1 ||
      static_cast<int64_t>(b.pieces) * b.ranks_per_piece < b.topk || b.whole_items < 0 ||
      b.whole_items > b.tq * b.hkv || (b.whole_items > 0 && b.topk > kMaxEP))
    return cudaErrorInvalidValue;
  if (b.num_pages < 1 || b.num_pages * b.hkv * b.page_size > kFusedMaxRows)
    return cudaErrorNotSupported;
  if (b.qhead <= 8)
    return a.int8 ? launch_q8<true, 8>(a, stream) : launch_q8<false, 8>(a, stream);
  return a.int8 ? launch_q8<true, 16>(a, stream) : launch_q8<false, 16>(a, stream);
}

}  // namespace sa
