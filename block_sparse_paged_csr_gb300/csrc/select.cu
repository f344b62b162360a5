// Block selection: for every (query, kv head) the topk blocks of its sequence
// with the highest score, the input of the index build (`selected`).
//
// The score of a block is an upper bound of what its best key can add up to
// over the GQA lanes of the kv head: with lo, hi the smallest and largest key
// per channel (sa_block_bounds),
//     score = sum over lanes, channels of max(q lo, q hi)
//           = sum over channels of P hi + M lo,
//     P = sum over lanes of max(q, 0),  M = sum over lanes of min(q, 0),
// so one vector of 2 head_dim weights per (query, kv head) meets one row of
// 2 head_dim bounds per block, whatever the number of lanes.
//
// Which block comes in last may turn on the last bits of two scores, and f32
// sums in another order would choose another block.  The scores are therefore
// formed in f32 together with a bound eps of their error; a row whose k-th and
// next score lie further apart than 2 eps is decided, and in the others the
// blocks within reach of the border are scored again in f64.  Ties go to the
// lower block.  The result is that of exact scores (up to f64 rounding),
// whatever the launch shape.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kChunk = 256;            // blocks per CTA of the score kernels
constexpr int kTileQ = 64;             // queries per CTA of the tile kernel
constexpr int kTileThreads = 128;
constexpr int kTileB = 64;             // blocks in flight there
constexpr uint32_t kNoBlock = 0xFFFFFFFFu;     // a score's bits: not a candidate (a NaN)

struct SelectArgs {
  const void* q;
  int q_bf16;
  int64_t tq;
  int32_t hq, hkv, qhead, head_dim;
  const uint16_t* bounds;              // [num_bounds, hkv, 2, head_dim] bf16
  int64_t num_bounds;
  const int32_t* bound_tables;         // [batch, msb]
  int32_t msb;
  const int64_t* cu;
  int32_t batch;
  const int32_t* used;
  int32_t block_size, topk, causal, sink, local;
  int32_t* selected;                   // [tq, hkv, topk]
  int64_t row0, rows;                  // (query, kv head) rows of this launch
  int64_t slots;                       // query tiles (tile kernel)
  uint32_t* scores;                    // [rows, stride] f32 bits
  float* eps;                          // [rows, chunks]
  uint16_t* weights;                   // [rows, 2, 2 head_dim] (tile kernel)
  uint16_t* maxima;                    // [batch, hkv, chunks, 2 head_dim]
  int64_t stride;
  int32_t chunks;
  int64_t* status;
  uint32_t spin;                       // tries of a bounded wait
  int stall;                           // test hook: no copy is sent, so every wait on one runs out
};

// What a (query, kv head) row sees: its sequence and the number of blocks
// with a key it may attend to.
struct RowView {
  int i, h, b, c0, c1, lk, nblk;
};

// Blocks in sight of query i of sequence [c0, c1) of length lk.  (Rows, queries
// and positions fit 32 bits: tq hkv topk < 2^31 and int32 lengths; 64-bit
// divisions would be most of a kernel's prologue.)
__device__ __forceinline__ int blocks_in_sight(const SelectArgs& a, int i, int c0, int c1, int lk) {
  int seen = lk;
  if (a.causal) {
    const int qo = c1 - c0, ql = i - c0;
    const int pos = a.causal == 2 || lk < qo ? ql : lk - qo + ql;
    seen = min(lk, max(pos + 1, 0));
  }
  const unsigned n = (static_cast<unsigned>(seen) + static_cast<unsigned>(a.block_size) - 1u) /
                     static_cast<unsigned>(a.block_size);
  return static_cast<int>(min(n, static_cast<unsigned>(a.msb)));
}

// The sequence of query i: b = i where every sequence so far holds one query
// (decode batches: no search), else 32 candidates per round.
__device__ __forceinline__ RowView row_view(const SelectArgs& a, unsigned row, int lane) {
  RowView v;
  v.i = static_cast<int>(row / static_cast<unsigned>(a.hkv));
  v.h = static_cast<int>(row) - v.i * a.hkv;
  v.b = min(v.i, a.batch - 1);
  v.c0 = static_cast<int>(a.cu[v.b]);
  v.c1 = static_cast<int>(a.cu[v.b + 1]);
  v.lk = a.used[v.b];
  if (v.c0 > v.i || v.c1 <= v.i) {
    v.b = warp_search(a.batch, lane, [&](int b) { return a.cu[b] <= v.i; });
    v.c0 = static_cast<int>(a.cu[v.b]);
    v.c1 = static_cast<int>(a.cu[v.b + 1]);
    v.lk = a.used[v.b];
  }
  v.lk = max(v.lk, 0);
  v.nblk = blocks_in_sight(a, v.i, v.c0, v.c1, v.lk);
  return v;
}

// The bounds row of block j of sequence b (-1: none).
__device__ __forceinline__ int bound_row(const SelectArgs& a, int b, int j) {
  const int r = a.bound_tables[static_cast<int64_t>(b) * a.msb + j];
  if (r >= a.num_bounds) report(a.status, SA_ERR_SHAPE);
  return r < a.num_bounds ? r : -1;
}

__device__ __forceinline__ float q_at(const SelectArgs& a, int64_t off) {
  return a.q_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.q)[off])
                  : static_cast<const float*>(a.q)[off];
}

// ------------------------------------------------------------------ scores

// d += a b, m16n8k16, bf16 operands, f32 accumulation.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ bool special_bf16x2(uint32_t u) {
  return (u & 0x7FFFu) >= 0x7F80u || ((u >> 16) & 0x7FFFu) >= 0x7F80u;
}
// A pair without its infinities and NaNs.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t u) {
  const uint32_t l = u & 0x7FFFu, g = (u >> 16) & 0x7FFFu;
  return (l >= 0x7F80u ? 0u : l) | ((g >= 0x7F80u ? 0u : g) << 16);
}

// The error bound of a score, per unit of the sum of |weight| * largest |bound|
// (which no block's sum of |terms| exceeds).  The tensor cores add 16 exact
// products and the sum so far in one step: every addend is cut (not rounded) to
// a multiple of 2^-25 of the power of two of the largest one, two bits below
// f32's last, and the sum is cut to 24 bits.  The largest addend loses nothing,
// each of the 16 others less than 2^-25, the sum less than 2^-23: 5 * 2^-23 a
// step.  That is how GB300's tensor cores behave, found by measuring (a large
// addend of either sign, first or last product or the sum so far, beside small ones
// of 2^-20 to 2^-32, and 2 million sums of random exponents, of which the worst lost
// 3.5 * 2^-23 of its terms' magnitudes), not a documented property.  Terms just
// below 2^-25 beside two large ones take scores 62 * 2^-23 off at head_dim 128; see
// the test of small terms.
// The weights' own sums over `lanes` f32 terms and the sums of parts and chains
// lose 2^-24 each, and the weights' split `split`; the last factor covers the
// parts' magnitudes above their weight's and the error of the sum of magnitudes
// itself.  (Products and parts below 2^-133 are lost besides: nothing, unless
// all of a score's terms are below 2^-100 or so.)
__host__ __device__ constexpr float score_eps(int steps, int lanes, float split) {
  return (static_cast<float>(steps) * 0x5p-23f + static_cast<float>(lanes + 6) * 0x1p-24f + split) *
         (1.f + 0x1p-6f);
}

// The bits of a score that is not finite, or of a block without a bounds row, or
// with one that stands for no block (lo[0] > hi[0]: a block without keys holds
// lo = inf, hi = -inf): kNoBlock for the last two; else the sum over the channels
// by itself, since a part of a split weight that is 0 makes a NaN of an infinite
// bound; one NaN for all.
__device__ __noinline__ uint32_t special_bits(const SelectArgs& a, int i, int h,
                                              const uint16_t* box, bool there) {
  if (!there) return kNoBlock;
  const int d = a.head_dim;
  if (bf16_to_f32(box[0]) > bf16_to_f32(box[d])) return kNoBlock;
  float s = 0.f;
  for (int ch = 0; ch < d; ++ch) {
    float neg = 0.f, pos = 0.f;
    for (int l = 0; l < a.qhead; ++l) {
      const float v =
          q_at(a, (static_cast<int64_t>(i) * a.hq + static_cast<int64_t>(h) * a.qhead + l) * d + ch);
      neg += v != v ? v : fminf(v, 0.f);
      pos += v != v ? v : fmaxf(v, 0.f);
    }
    s = fmaf(neg, bf16_to_f32(box[ch]), s);
    s = fmaf(pos, bf16_to_f32(box[d + ch]), s);
  }
  return s != s ? 0x7FFFFFFFu : __float_as_uint(s);
}

// A sum of |terms| of the block with bounds row r: 0 where it is not finite for
// an infinite or NaN bound's sake, infinite where the terms themselves left the
// range.
__device__ __noinline__ float capped(const SelectArgs& a, float m, int r, int h) {
  if (m < INFINITY) return m;
  if (r < 0) return 0.f;
  const uint32_t* box = reinterpret_cast<const uint32_t*>(
      a.bounds + (static_cast<int64_t>(r) * a.hkv + h) * 2 * a.head_dim);
  for (int x = 0; x < a.head_dim; ++x)
    if (special_bf16x2(box[x])) return 0.f;
  return INFINITY;
}

// q values of 4 consecutive channels.  (The type is a template argument: a
// branch on it around every load would keep loads from being in flight
// together.)
template <bool kQ16>
__device__ __forceinline__ float4 q4_of(const void* q, int64_t off) {
  if constexpr (kQ16)
    return bf16x4_to_f32(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + off)));
  else
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(q) + off));
}
template <bool kQ16>
__device__ __forceinline__ float q_of(const void* q, int64_t off) {
  if constexpr (kQ16)
    return bf16_to_f32(__ldg(static_cast<const uint16_t*>(q) + off));
  else
    return __ldg(static_cast<const float*>(q) + off);
}

// A finite weight whose bf16 part may be infinite: no bound holds then.
__device__ __forceinline__ bool huge_weight(float w) {
  w = fabsf(w);
  return w >= 0x1p127f && w < INFINITY;
}

// The same of a weight in two bf16 parts.
__device__ __forceinline__ bool huge_part(uint32_t hi, uint32_t lo) {
  return (hi & 0x7FFFu) >= 0x7F00u && !((hi & 0x7FFFu) >= 0x7F80u && (lo & 0x7FFFu) > 0x7F80u);
}

// (a NaN of q stays one)
__device__ __forceinline__ float neg_part(float x) { return x != x ? x : fminf(x, 0.f); }
__device__ __forceinline__ float pos_part(float x) { return x != x ? x : fmaxf(x, 0.f); }

// Scores for few queries per sequence (decode steps): up to kNQ queries of one
// sequence against kChunk of its blocks, for one kv head.  The weights are the
// rows of the MMA's A tile, each split into three bf16 parts (rows 3 x .. 3 x +
// 2 for query x: 24 bits, all that f32 has); eight blocks are the columns.
// Reading the bounds, 4 head_dim bytes a block, is what takes time.  Every warp
// has a ring of stages of 8 rows of its own (no barrier of the CTA in the
// loop): lanes send one bulk copy per row as soon as the rows are known, the
// weights are summed while the first arrive, and a stage is refilled as soon as
// it is read.  A lane's
// 16-byte pieces of a row then go to the B fragments as they are (the k index of
// a fragment stands for whatever channel the lane read).  The sum of |terms|
// that the error bound needs comes from the same A tile: M is never positive
// and P never negative, so the columns' magnitudes, negated where they meet M,
// make every term its own magnitude.
// Measured: 128 sequences of up to 131072 keys, 64-key blocks, 8 kv heads of 128
// channels (807 MB of bounds) 152 us, 5.3 TB/s; 64 sequences of up to 32768 (77
// MB) 27 us, of which the chain length -> row ids -> bounds -> scores is a good
// part.  Two CTAs per SM at 128 registers.
//   kT: 16-byte pieces per lane and row (head_dim <= 16 kT).
constexpr int kScoreRowPad = 64;       // rows 128 k + 64 bytes apart: no bank conflicts
constexpr int kGroup = 8;              // blocks per stage (an MMA's columns)
constexpr int kStages = kChunk / kGroup / kScoreWarps;   // per warp

__host__ __device__ constexpr int score_row_bytes(int d) { return (4 * d + 127) / 128 * 128 + kScoreRowPad; }

// Stages in a warp's ring: what two CTAs per SM have room for (one above head_dim
// 128).
__host__ __device__ constexpr int score_ring(int kT) { return kT <= 8 ? 3 : 2; }

//   kSpan: chunks per CTA.  A CTA's start (sequence, row ids, weights) takes about
//   as long as a chunk's bounds, so two where there are CTAs enough: 128
//   sequences of up to 131072 keys, 64-key blocks, 8 kv heads take 178 us instead
//   of 197, but one of them 18.5 us instead of 14.4.
template <int kT, int kNQ, int kSpan, bool kQ16>
__global__ void __launch_bounds__(kScoreThreads, kT <= 8 && kNQ == 1 ? 2 : 1)
block_score_kernel(const SelectArgs a) {
  constexpr int kHalves = kNQ > 2 ? 2 : 1;             // A rows 0-7, 8-15
  constexpr int kRing = score_ring(kT);
  extern __shared__ __align__(128) unsigned char s_rows[];   // [warps][kRing][kGroup][row bytes]
  __shared__ __align__(16) uint16_t s_wb[3 * kNQ][32 * kT + 8];   // bf16 parts of M, P: rows of the A tile
  __shared__ int s_nblk[kNQ];
  __shared__ float s_l1[kNQ][kScoreWarps];
  __shared__ int s_huge[kNQ];
  __shared__ uint64_t s_bar[kScoreWarps][kRing];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int d = a.head_dim;
  // the CTA's first query (kNQ = 1: every query; else every kNQ-th of its
  // sequence), head and chunk
  const unsigned spans = static_cast<unsigned>((a.chunks + kSpan - 1) / kSpan);
  const unsigned unit = blockIdx.x / spans;
  const int chunk = static_cast<int>(blockIdx.x - unit * spans) * kSpan;
  const unsigned row = static_cast<unsigned>(a.row0) + unit;
  griddep_launch_dependents();
  if (tid < kScoreWarps * kRing) mbar_init(&s_bar[0][0] + tid, 1);
  if (tid < 32) fence_mbar_init();
  const RowView rv = row_view(a, row, lane);
  const int j0 = chunk * kChunk;
  int nq = 1;
  int nmax = rv.nblk;
  if constexpr (kNQ > 1) {
    const int w0 = static_cast<int>(a.row0) / a.hkv;
    if ((rv.i - max(rv.c0, w0)) % kNQ != 0) return;
    nq = min(kNQ, min(rv.c1, static_cast<int>(a.row0 + a.rows) / a.hkv) - rv.i);
    nmax = 0;
    for (int x = 0; x < nq; ++x) {
      const int n = blocks_in_sight(a, rv.i + x, rv.c0, rv.c1, rv.lk);
      if (n > a.topk) nmax = max(nmax, n);
      if (tid == 0) s_nblk[x] = n;
    }
  } else if (tid == 0) {
    s_nblk[0] = rv.nblk;
  }
  // (a row that takes every block it sees needs no scores)
  if (j0 >= nmax || nmax <= a.topk) return;
  const int j1 = min(j0 + kSpan * kChunk, nmax);
  // the warp's blocks: stage t holds blocks j0 + 8 (kScoreWarps t + warp) ..;
  // lane l has the row of block l & 7 of stage l / 8 of each chunk
  static_assert(kStages == 4 && kSpan <= 2, "a row id per lane and chunk");
  int ids[kSpan];
#pragma unroll
  for (int x = 0; x < kSpan; ++x) {
    const int j = j0 + kChunk * x + kGroup * (kScoreWarps * (lane >> 3) + warp) + (lane & 7);
    ids[x] = j < j1 ? bound_row(a, rv.b, j) : -1;
  }
  const int row_bytes = score_row_bytes(d);
  unsigned char* mine = s_rows + warp * kRing * kGroup * row_bytes;
  const int left = j1 - j0 - kGroup * warp;            // blocks from the warp's first on
  const int nst = left <= 0 ? 0 : (left + kGroup * kScoreWarps - 1) / (kGroup * kScoreWarps);
  __syncthreads();                                     // the barriers are there
  // rows of stage t in flight
  auto send = [&](int t) {
    if (a.stall) return;
    const int id = ids[kSpan == 1 || t < kStages ? 0 : 1];
    const bool there = (lane >> 3) == t % kStages && id >= 0;
    const unsigned present = __ballot_sync(0xffffffffu, there);
    uint64_t* bar = &s_bar[warp][t % kRing];
    if (lane == 0)
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(present)) * 4u *
                                     static_cast<uint32_t>(d));
    __syncwarp();
    if (there)
      bulk_g2s(mine + ((t % kRing) * kGroup + (lane & 7)) * row_bytes,
               a.bounds + (static_cast<int64_t>(id) * a.hkv + rv.h) * 2 * d,
               4u * static_cast<uint32_t>(d), bar);
  };
#pragma unroll
  for (int t = 0; t < kRing; ++t)
    if (t < nst) send(t);

  // The weights: a warp takes 16 channels at a time, eight GQA lanes by four
  // pieces of 4 channels over its lanes.
  if (tid < kNQ) s_huge[tid] = 0;
  __syncthreads();
  for (int qi = 0; qi < nq; ++qi) {
    for (int ch = 16 * warp + 4 * c; ch - 4 * c < d; ch += 16 * kScoreWarps) {
      const int64_t off =
          (static_cast<int64_t>(rv.i + qi) * a.hq + static_cast<int64_t>(rv.h) * a.qhead) * d + ch;
      float w[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if (ch < d) {
        for (int l = g; l < a.qhead; l += 8) {
          const float4 v = q4_of<kQ16>(a.q, off + static_cast<int64_t>(l) * d);
          const float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[0][e] += neg_part(q[e]);
            w[1][e] += pos_part(q[e]);
          }
        }
      }
      bool huge = false;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) w[half][e] += __shfl_xor_sync(0xffffffffu, w[half][e], o);
          huge = huge || huge_weight(w[half][e]);
        }
      // lanes g = 0..5: half g & 1, part g / 2
      if (g < 6 && ch < d) {
        float x0 = g & 1 ? w[1][0] : w[0][0], x1 = g & 1 ? w[1][1] : w[0][1];
        float x2 = g & 1 ? w[1][2] : w[0][2], x3 = g & 1 ? w[1][3] : w[0][3];
        uint2 u = make_uint2(0u, 0u);
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          if (part <= g / 2) {
            u = make_uint2(pack_bf16x2_rn(x0, x1), pack_bf16x2_rn(x2, x3));
            x0 -= __uint_as_float(u.x << 16);
            x1 -= __uint_as_float(u.x & 0xFFFF0000u);
            x2 -= __uint_as_float(u.y << 16);
            x3 -= __uint_as_float(u.y & 0xFFFF0000u);
          }
        }
        *reinterpret_cast<uint2*>(&s_wb[3 * qi + g / 2][(g & 1) * d + ch]) = u;
        if (huge) s_huge[qi] = 1;
      }
    }
  }
  __syncthreads();
  // A fragments: row r = 3 x + part, this lane's channels 8 (c + 4 t) + 0..7
  const int pieces = d >> 2;
  uint32_t af[kT][4][kHalves];
#pragma unroll
  for (int t = 0; t < kT; ++t)
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      const int r = g + 8 * hf, pc = c + 4 * t;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < 3 * nq && pc < pieces) w = *reinterpret_cast<const uint4*>(&s_wb[r][pc * 8]);
      af[t][0][hf] = w.x;
      af[t][1][hf] = w.y;
      af[t][2][hf] = w.z;
      af[t][3][hf] = w.w;
    }

  float l1[kNQ];                       // largest sum of |terms| so far
#pragma unroll
  for (int qi = 0; qi < kNQ; ++qi) l1[qi] = 0.f;
#pragma unroll 1
  for (int st = 0; st < nst; ++st) {
    if (!mbar_wait_bounded(&s_bar[warp][st % kRing], (st / kRing) & 1, a.spin)) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
      // (the copies in flight end before the CTA does: stages up to st + kRing - 1
      // have been sent)
      for (int x = st; x < min(st + kRing, nst); ++x)
        mbar_wait_bounded(&s_bar[warp][x % kRing], (x / kRing) & 1, a.spin);
      break;
    }
    {
      // block jw + g in column g
      const int jw = j0 + kGroup * (kScoreWarps * st + warp);
      const unsigned char* box = mine + ((st % kRing) * kGroup + g) * row_bytes + c * 16;
      float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float mag[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (c + 4 * t < pieces) x = *reinterpret_cast<const uint4*>(box + t * 64);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
        const bool hi = 8 * (c + 4 * t) >= d;
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = hi ? u[e] & 0x7FFF7FFFu : u[e] | 0x80008000u;
        // k-steps of channels 0-3 and 4-7 of the lane's piece
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t a0 = af[t][2 * k][0], a2 = af[t][2 * k + 1][0];
          const uint32_t a1 = kHalves == 2 ? af[t][2 * k][kHalves - 1] : 0u;
          const uint32_t a3 = kHalves == 2 ? af[t][2 * k + 1][kHalves - 1] : 0u;
          mma_bf16(acc[k], a0, a1, a2, a3, u[2 * k], u[2 * k + 1]);
          mma_bf16(mag[k], a0, a1, a2, a3, v[2 * k], v[2 * k + 1]);
        }
      }
      const int id = ids[kSpan == 1 || st < kStages ? 0 : 1];
      const int id0 = __shfl_sync(0xffffffffu, id, 8 * (st % kStages) + 2 * c);
      const int id1 = __shfl_sync(0xffffffffu, id, 8 * (st % kStages) + 2 * c + 1);
      // whether this lane's column (2 c + (g & 1), see below) is a block: lo[0] <= hi[0]
      const uint16_t* own = reinterpret_cast<const uint16_t*>(
          mine + ((st % kRing) * kGroup + 2 * c + (g & 1)) * row_bytes);
      const bool none = bf16_to_f32(own[0]) > bf16_to_f32(own[d]);
      // a query's score: its three rows' sums, of columns 2 c and 2 c + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[0][e] += acc[1][e];
        mag[0][e] += mag[1][e];
      }
#pragma unroll
      for (int qi = 0; qi < kNQ; ++qi) {
        if (qi < nq) {
          float s0 = 0.f, s1 = 0.f, m0 = 0.f, m1 = 0.f;
#pragma unroll
          for (int part = 2; part >= 0; --part) {
            const int r3 = 3 * qi + part;
            const int src = (r3 & 7) * 4 + c;
            s0 += __shfl_sync(0xffffffffu, r3 < 8 ? acc[0][0] : acc[0][2], src);
            s1 += __shfl_sync(0xffffffffu, r3 < 8 ? acc[0][1] : acc[0][3], src);
            m0 += __shfl_sync(0xffffffffu, r3 < 8 ? mag[0][0] : mag[0][2], src);
            m1 += __shfl_sync(0xffffffffu, r3 < 8 ? mag[0][1] : mag[0][3], src);
          }
          // (columns without a row hold what was there before)
          m0 = id0 >= 0 ? m0 : 0.f;
          m1 = id1 >= 0 ? m1 : 0.f;
          // Sums with infinite or NaN bounds (a block without keys holds
          // +-inf) do not count: their scores are infinite or NaN, in f64 as in
          // f32, and order the same.  A sum that left the range without them
          // leaves no bound.
          if (m0 < INFINITY && m1 < INFINITY)
            l1[qi] = fmaxf(l1[qi], fmaxf(m0, m1));
          else
            l1[qi] = fmaxf(l1[qi], fmaxf(capped(a, m0, id0, rv.h), capped(a, m1, id1, rv.h)));
          // lanes 0-3 write columns 2 c, lanes 4-7 columns 2 c + 1
          const int j = jw + 2 * c + (g & 1);
          const int rj = g & 1 ? id1 : id0;
          if (g < 2 && j < min(j1, s_nblk[qi])) {
            const float sv = g == 0 ? s0 : s1;
            a.scores[(static_cast<int64_t>(unit) + static_cast<int64_t>(qi) * a.hkv) * a.stride + j] =
                rj >= 0 && !none && fabsf(sv) < INFINITY
                    ? __float_as_uint(sv)
                    : special_bits(a, rv.i + qi, rv.h,
                                   a.bounds + (static_cast<int64_t>(max(rj, 0)) * a.hkv + rv.h) * 2 * d,
                                   rj >= 0);
          }
        }
      }
    }
    __syncwarp();                                      // the stage is read
    if (st + kRing < nst) send(st + kRing);
  }
#pragma unroll
  for (int qi = 0; qi < kNQ; ++qi) {
    float m = l1[qi];
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // (weights past f32's or bf16's range: no bound holds)
    if (s_huge[qi]) m = INFINITY;
    if (lane == 0) s_l1[qi][warp] = m;
  }
  __syncthreads();
  if (tid < nq) {
    float m = 0.f;
    for (int w = 0; w < kScoreWarps; ++w) m = fmaxf(m, s_l1[tid][w]);
    for (int x = chunk; x < min(chunk + kSpan, a.chunks); ++x)
      a.eps[(static_cast<int64_t>(unit) + static_cast<int64_t>(tid) * a.hkv) * a.chunks + x] =
          m * score_eps(kT, a.qhead, 0x1p-24f);
  }
}

// Scores for many queries per sequence (prompts), in three kernels: the
// weights of every (query, kv head) once, in two bf16 parts (2^-18 of a weight
// is lost, which eps counts): reads q, coalesced, at the speed of memory; the
// largest |bound| per channel of every (sequence, kv head, chunk), for eps; and
// the products, tile by tile.  For 8192 queries, 64 heads of 128 channels on 8 kv
// heads, 256 blocks: 48 us (302 MB, 6.2 TB/s), 7.5 us and 77 us.
//   weights: [rows][part][2 head_dim] bf16, M (lo channels) then P (hi)
template <bool kQ16>
__global__ void __launch_bounds__(256) block_weights_kernel(const SelectArgs a) {
  griddep_launch_dependents();
  const int d4 = a.head_dim >> 2;
  const int64_t n = a.rows * d4;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; x < n;
       x += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t lrow = x / d4;
    const int ch = static_cast<int>(x - lrow * d4) * 4;
    const int64_t off = (a.row0 + lrow) * a.qhead * a.head_dim + ch;
    float w[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 8
    for (int l = 0; l < a.qhead; ++l) {
      const float4 v = q4_of<kQ16>(a.q, off + static_cast<int64_t>(l) * a.head_dim);
      const float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[0][e] += neg_part(q[e]);
        w[1][e] += pos_part(q[e]);
      }
    }
    uint16_t* out = a.weights + lrow * 4 * a.head_dim + ch;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint2 hi, lo;
      hi.x = pack_bf16x2_rn(w[half][0], w[half][1]);
      hi.y = pack_bf16x2_rn(w[half][2], w[half][3]);
      lo.x = pack_bf16x2_rn(w[half][0] - __uint_as_float(hi.x << 16),
                            w[half][1] - __uint_as_float(hi.x & 0xFFFF0000u));
      lo.y = pack_bf16x2_rn(w[half][2] - __uint_as_float(hi.y << 16),
                            w[half][3] - __uint_as_float(hi.y & 0xFFFF0000u));
      *reinterpret_cast<uint2*>(out + half * a.head_dim) = hi;
      *reinterpret_cast<uint2*>(out + (2 + half) * a.head_dim) = lo;
    }
  }
}

// maxima: [batch][hkv][chunks][2 head_dim] bf16 magnitudes.  Infinite and NaN
// bounds do not count: the scores they enter are infinite or NaN, in f64 as in
// f32, and order the same.
__global__ void __launch_bounds__(1024) block_maxima_kernel(const SelectArgs a) {
  griddep_launch_dependents();
  static_assert(kChunk == 32 * 8, "eight rows per warp");
  __shared__ uint32_t s_max[32][128];
  const int d = a.head_dim;                            // words (channel pairs) of a row
  const unsigned bh = blockIdx.x / static_cast<unsigned>(a.chunks);
  const int chunk = static_cast<int>(blockIdx.x - bh * static_cast<unsigned>(a.chunks));
  const int b = static_cast<int>(bh / static_cast<unsigned>(a.hkv));
  const int h = static_cast<int>(bh) - b * a.hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lk = max(a.used[b], 0);
  const int j0 = chunk * kChunk;
  const int j1 = min(static_cast<int>(min((static_cast<unsigned>(lk) + a.block_size - 1u) /
                                              static_cast<unsigned>(a.block_size),
                                          static_cast<unsigned>(a.msb))),
                     j0 + kChunk);
  if (j0 >= j1) {
    griddep_wait();
    return;
  }
  const int j = j0 + 32 * (lane & 7) + warp;
  const int id = lane < 8 && j < j1 ? bound_row(a, b, j) : -1;
  for (int x0 = 0; x0 < d; x0 += 128) {
    uint32_t u[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int r = __shfl_sync(0xffffffffu, id, t);
      const uint32_t* box = reinterpret_cast<const uint32_t*>(
          a.bounds + (static_cast<int64_t>(max(r, 0)) * a.hkv + h) * 2 * d);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int w = x0 + lane + 32 * x;
        u[t][x] = r >= 0 && w < d ? __ldg(box + w) : 0u;
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t m = 0u;
#pragma unroll
      for (int t = 0; t < 8; ++t) m = __vmaxu2(m, finite_bf16x2(u[t][x]));
      s_max[warp][lane + 32 * x] = m;
    }
    __syncthreads();
    if (threadIdx.x < 128 && x0 + static_cast<int>(threadIdx.x) < d) {
      uint32_t v = 0u;
#pragma unroll 8
      for (int w = 0; w < 32; ++w) v = __vmaxu2(v, s_max[w][threadIdx.x]);
      (reinterpret_cast<uint32_t*>(a.maxima) + static_cast<int64_t>(blockIdx.x) * d)[x0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
  griddep_wait();                        // ends after the weights kernel, beside which it runs
}

// kTileQ queries of one sequence against kChunk of its blocks, for one kv head.
// Warp w holds the weights of 16 queries as A fragments in registers; the
// blocks' bounds pass through shared memory, 64 at a time, read once by each
// warp.  2 x 4 head_dim flops per (query, kv head, block).
// Bound by latency: the weights take 128 of 254 registers, so 8 warps per SM have
// to hide it (tensor pipe about 40 % busy; 92 us with copies by lanes and the
// error bound summed lane by lane).
//   kG: 32-channel groups of each bound (head_dim <= 32 kG).
template <int kG>
struct TileSmem {
  static constexpr int kRow = 4 * kG * 32 + 64;        // bytes of a bounds row: 16 banks on
  static constexpr int kBuf = kTileB * kRow;
  static constexpr int kIds = 2 * kBuf;                // int32 [kChunk]
  static constexpr int kTotal = kIds + kChunk * 4;
};

template <int kG>
__global__ void __launch_bounds__(kTileThreads, 2) block_score_tile_kernel(const SelectArgs a) {
  using L = TileSmem<kG>;
  extern __shared__ __align__(16) unsigned char s_raw[];
  int* ids = reinterpret_cast<int*>(s_raw + L::kIds);
  __shared__ uint64_t s_bar[2];                        // the two buffers' bounds are there
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int d = a.head_dim;
  griddep_launch_dependents();
  const unsigned hs = blockIdx.x / static_cast<unsigned>(a.chunks);
  const int chunk = static_cast<int>(blockIdx.x - hs * static_cast<unsigned>(a.chunks));
  const int slot = static_cast<int>(hs / static_cast<unsigned>(a.hkv));
  const int h = static_cast<int>(hs) - slot * a.hkv;
  const int b = warp_slot_sequence(a.cu, a.batch, kTileQ, slot, lane);
  const int c0 = static_cast<int>(a.cu[b]), c1 = static_cast<int>(a.cu[b + 1]);
  const int i0 = c0 + (slot - static_cast<int>(slot_base(c0, b, kTileQ))) * kTileQ;
  // this launch's queries
  const int w0 = static_cast<int>(a.row0) / a.hkv;
  const int w1 = static_cast<int>(a.row0 + a.rows) / a.hkv;
  if (i0 < c0 || i0 >= c1 || i0 >= w1 || i0 + kTileQ <= w0) {
    griddep_wait();                      // (every CTA: the kernels of the call end in order)
    return;
  }
  const int lk = max(a.used[b], 0);
  // (blocks in sight grow with the query)
  const int nmax = blocks_in_sight(a, min(i0 + kTileQ, c1) - 1, c0, c1, lk);
  const int j0 = chunk * kChunk;
  if (j0 >= nmax || nmax <= a.topk) {
    griddep_wait();
    return;
  }
  const int j1 = min(j0 + kChunk, nmax);
  if (tid < 2) mbar_init(s_bar + tid, kTileThreads / 32);
  if (tid < 32) fence_mbar_init();
  bool all_rows = true;                                // every block of the chunk has its row
  for (int j = tid; j < kChunk; j += kTileThreads) {
    const int id = j0 + j < j1 ? bound_row(a, b, j0 + j) : -1;
    ids[j] = id;
    all_rows = all_rows && (id >= 0 || j0 + j >= j1);
  }
  // channels past d: their weights are zero, so the bounds only have to be numbers
  for (int x = tid; d < 32 * kG && x < 2 * kTileB * 8 * kG; x += kTileThreads) {
    const int at = x % (8 * kG);
    if (at % (4 * kG) * 8 >= d)
      *reinterpret_cast<uint4*>(s_raw + x / (8 * kG) * L::kRow + at * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  all_rows = __syncthreads_and(all_rows);

  // A tile of bounds: a warp sends for 16 rows, a lane for the lo or the hi half
  // of one.  Blocks without a row keep what the buffer holds: their scores are
  // not taken from the MMA.
  const uint32_t half_bytes = 2u * static_cast<uint32_t>(d);
  auto load_tile = [&](int t) {
    if (a.stall) return;
    const int r = 16 * warp + (lane & 15), hi = lane >> 4;
    const int id = ids[t * kTileB + r];
    const unsigned present = __ballot_sync(0xffffffffu, id >= 0);
    uint64_t* bar = s_bar + (t & 1);
    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(present)) * half_bytes);
    __syncwarp();
    if (id >= 0)
      bulk_g2s(s_raw + (t & 1) * L::kBuf + r * L::kRow + hi * 64 * kG,
               a.bounds + ((static_cast<int64_t>(id) * a.hkv + h) * 2 + hi) * d, half_bytes, bar);
  };
  const int tiles = (j1 - j0 + kTileB - 1) / kTileB;
  load_tile(0);
  if (tiles > 1) load_tile(1);

  // the weights and the maxima are there (read past it: no read-only loads)
  griddep_wait();
  // weights of queries i0 + 16 warp + g and + 8, channels 32 x + 8 c + 0..7
  uint32_t ahi[2][kG][2][4], alo[2][kG][2][4];         // [lo, hi bound][group][k-step][fragment]
  const int iq[2] = {i0 + 16 * warp + g, i0 + 16 * warp + g + 8};
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const bool there = iq[rr] < c1 && iq[rr] >= w0 && iq[rr] < w1;
    const uint16_t* w = a.weights + static_cast<int64_t>(there ? (iq[rr] - w0) * a.hkv + h : 0) * 4 * d;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int x = 0; x < kG; ++x) {
        const int ch = 32 * x + 8 * c;
        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
        if (there && ch < d) {
          hi = __ldcg(reinterpret_cast<const uint4*>(w + half * d + ch));
          lo = __ldcg(reinterpret_cast<const uint4*>(w + (2 + half) * d + ch));
        }
        ahi[half][x][0][rr] = hi.x;
        ahi[half][x][0][2 + rr] = hi.y;
        ahi[half][x][1][rr] = hi.z;
        ahi[half][x][1][2 + rr] = hi.w;
        alo[half][x][0][rr] = lo.x;
        alo[half][x][0][2 + rr] = lo.y;
        alo[half][x][1][rr] = lo.z;
        alo[half][x][1][2 + rr] = lo.w;
      }
  }
  int nb[2];
  float* out[2];
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const bool there = iq[rr] < c1 && iq[rr] >= w0 && iq[rr] < w1;
    nb[rr] = there ? min(blocks_in_sight(a, iq[rr], c0, c1, lk), j1) : 0;
    out[rr] = reinterpret_cast<float*>(a.scores) +
              static_cast<int64_t>(there ? (iq[rr] - w0) * a.hkv + h : 0) * a.stride;
  }

  bool late = false;                                   // a wait ran out: send no more
  for (int t = 0; t < tiles; ++t) {
    if (!mbar_wait_bounded(s_bar + (t & 1), (t >> 1) & 1, a.spin)) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_TIMEOUT);
      late = true;
    }
    const unsigned char* buf = s_raw + (t & 1) * L::kBuf;
#pragma unroll 1
    for (int n = 0; n < kTileB / 16; ++n) {
      float lo0[2];                                    // lo[0] (lanes c = 0)
      bool none = false;                               // a row of these 16 with lo[0] > hi[0]
      float acc[2][2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[x][y][e] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int x = 0; x < kG; ++x)
#pragma unroll
          for (int n2 = 0; n2 < 2; ++n2) {
            const uint4 u = *reinterpret_cast<const uint4*>(
                buf + (16 * n + 8 * n2 + g) * L::kRow + (half * 4 * kG + 4 * x + c) * 16);
            if (x == 0) {
              const float first = __uint_as_float(u.x << 16);
              if (half == 0) lo0[n2] = first;
              else none = none || (c == 0 && lo0[n2] > first);
            }
            mma_bf16(acc[n2][0], ahi[half][x][0][0], ahi[half][x][0][1], ahi[half][x][0][2],
                     ahi[half][x][0][3], u.x, u.y);
            mma_bf16(acc[n2][1], alo[half][x][0][0], alo[half][x][0][1], alo[half][x][0][2],
                     alo[half][x][0][3], u.x, u.y);
            mma_bf16(acc[n2][0], ahi[half][x][1][0], ahi[half][x][1][1], ahi[half][x][1][2],
                     ahi[half][x][1][3], u.z, u.w);
            mma_bf16(acc[n2][1], alo[half][x][1][0], alo[half][x][1][1], alo[half][x][1][2],
                     alo[half][x][1][3], u.z, u.w);
          }
      float big = 0.f;                                 // largest |score|; NaN where one is
#pragma unroll
      for (int n2 = 0; n2 < 2; ++n2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[n2][0][e] += acc[n2][1][e];
          big += fabsf(acc[n2][0][e]);
        }
      const bool plain = !__any_sync(0xffffffffu, none) && all_rows && big < INFINITY;
#pragma unroll
      for (int n2 = 0; n2 < 2; ++n2) {
        const int lj = t * kTileB + 16 * n + 8 * n2 + 2 * c;   // column of the chunk
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          if (j0 + lj >= nb[rr]) continue;
          const float s0 = acc[n2][0][2 * rr], s1 = acc[n2][0][2 * rr + 1];
          uint2 bits = make_uint2(__float_as_uint(s0), __float_as_uint(s1));
          if (!plain) {
            const int id0 = ids[lj], id1 = ids[lj + 1];
            const uint16_t* r0 = reinterpret_cast<const uint16_t*>(
                buf + (16 * n + 8 * n2 + 2 * c) * L::kRow);
            const uint16_t* r1 = r0 + L::kRow / 2;
            if (id0 < 0 || !(fabsf(s0) < INFINITY) ||
                bf16_to_f32(r0[0]) > bf16_to_f32(r0[32 * kG]))
              bits.x = special_bits(
                  a, iq[rr], h, a.bounds + (static_cast<int64_t>(max(id0, 0)) * a.hkv + h) * 2 * d,
                  id0 >= 0);
            if (id1 < 0 || !(fabsf(s1) < INFINITY) ||
                bf16_to_f32(r1[0]) > bf16_to_f32(r1[32 * kG]))
              bits.y = special_bits(
                  a, iq[rr], h, a.bounds + (static_cast<int64_t>(max(id1, 0)) * a.hkv + h) * 2 * d,
                  id1 >= 0);
          }
          // (whole rows of the workspace: an even number of columns)
          *reinterpret_cast<uint2*>(out[rr] + j0 + lj) = bits;
        }
      }
    }
    if (__syncthreads_or(late)) {                      // (and the buffer is read)
      // (the copies in flight end before the CTA does)
      mbar_wait_bounded(s_bar + (t & 1), (t >> 1) & 1, a.spin);
      if (t + 1 < tiles) mbar_wait_bounded(s_bar + ((t + 1) & 1), ((t + 1) >> 1) & 1, a.spin);
      return;
    }
    if (t + 2 < tiles) load_tile(t + 2);
  }
  // eps of the chunk for every query: the sum of |weight| times the largest
  // |bound|.  M is never positive and P never negative, so it is the score of a
  // block of those maxima, negated where they meet M: one more column.
  const uint16_t* mx =
      a.maxima + ((static_cast<int64_t>(b) * a.hkv + h) * a.chunks + chunk) * 2 * d;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int x = 0; x < kG; ++x) {
      const int ch = 32 * x + 8 * c;
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (g == 0 && ch < d) {
        const uint32_t sign = half == 0 ? 0x80008000u : 0u;
        u = __ldcg(reinterpret_cast<const uint4*>(mx + half * d + ch));
        u = make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t b0 = k ? u.z : u.x, b1 = k ? u.w : u.y;
        mma_bf16(sum, ahi[half][x][k][0], ahi[half][x][k][1], ahi[half][x][k][2],
                 ahi[half][x][k][3], b0, b1);
        mma_bf16(sum, alo[half][x][k][0], alo[half][x][k][1], alo[half][x][k][2],
                 alo[half][x][k][3], b0, b1);
      }
    }
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    // (column 0 is the first lane's)
    float l1 = __shfl_sync(0xffffffffu, sum[2 * rr], lane & 28);
    if (__any_sync(0xffffffffu, !(l1 < INFINITY))) {
      // weights that are not numbers or past bf16's range: channel by channel
      l1 = 0.f;
      bool huge = false;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int x = 0; x < kG; ++x) {
          const int ch = 32 * x + 8 * c;
          if (ch >= d) continue;
          const uint4 m4 = __ldcg(reinterpret_cast<const uint4*>(mx + half * d + ch));
          const uint32_t m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t hi = ahi[half][x][e >> 1][2 * (e & 1) + rr];
            const uint32_t lo = alo[half][x][e >> 1][2 * (e & 1) + rr];
            const float a0 = fabsf(__uint_as_float(hi << 16) + __uint_as_float(lo << 16));
            const float a1 = fabsf(__uint_as_float(hi & 0xFFFF0000u) +
                                   __uint_as_float(lo & 0xFFFF0000u));
            l1 += a0 < INFINITY ? a0 * __uint_as_float(m[e] << 16) : 0.f;
            l1 += a1 < INFINITY ? a1 * __uint_as_float(m[e] & 0xFFFF0000u) : 0.f;
            // (a weight past bf16's range has an infinite part and an infinite
            // remainder of the other sign; an infinite weight's remainder is NaN)
            huge = huge || huge_part(hi, lo) || huge_part(hi >> 16, lo >> 16);
          }
        }
      if (huge) l1 = INFINITY;
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }
    if (c == 0 && iq[rr] < c1 && iq[rr] >= w0 && iq[rr] < w1)
      a.eps[static_cast<int64_t>((iq[rr] - w0) * a.hkv + h) * a.chunks + chunk] =
          l1 * score_eps(4 * kG, a.qhead, 0x1p-18f);
  }
}

// ------------------------------------------------------------------ pick

// Scores as unsigned keys that order like them; 0: not a candidate, 1: NaN.
__device__ __forceinline__ uint32_t score_key(uint32_t bits) {
  if (bits == kNoBlock) return 0u;
  if ((bits & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  return (bits >> 31) ? ~bits : bits | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t key) {
  if (key <= 1u) return -INFINITY;
  return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long score_key64(double x) {
  if (x != x) return 1ull;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x));
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

constexpr uint32_t kForced = 0xFFFFFFFFu;   // key of a block that comes in whatever its score

// The threads of one row: a warp, or a CTA of eight.
template <int kWarps>
struct RowGroup {
  int* red;              // [2][kWarps] (CTA rows)
  int par = 0;
  __device__ __forceinline__ explicit RowGroup(int* r) : red(r) {}
  __device__ __forceinline__ void sync() const {
    if constexpr (kWarps == 1)
      __syncwarp();
    else
      __syncthreads();
  }
  // Alternating buffers: a thread that writes one again has passed the barrier
  // after everyone's read of it.
  __device__ __forceinline__ int sum(int x) {
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (kWarps > 1) {
      int* buf = red + (par ^= 1) * kWarps;
      if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
      __syncthreads();
      x = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x += buf[w];
    }
    return x;
  }
  __device__ __forceinline__ uint32_t max(uint32_t x) {
    x = __reduce_max_sync(0xffffffffu, x);
    if constexpr (kWarps > 1) {
      int* buf = red + (par ^= 1) * kWarps;
      if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = static_cast<int>(x);
      __syncthreads();
      x = 0u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x = ::max(x, static_cast<uint32_t>(buf[w]));
    }
    return x;
  }
};

// One warp's f64 score of block j: the weights from shared memory.
__device__ __forceinline__ double score64(const SelectArgs& a, const RowView& rv, const double* w64,
                                          int j, int lane) {
  const int d = a.head_dim;
  const int r = bound_row(a, rv.b, j);
  double s = 0.0;
  if (r >= 0) {
    const uint32_t* br = reinterpret_cast<const uint32_t*>(
        a.bounds + (static_cast<int64_t>(r) * a.hkv + rv.h) * 2 * d);
    for (int x = lane; x < d; x += 32) {
      const uint32_t u = __ldg(br + x);
      s = fma(w64[2 * x], static_cast<double>(__uint_as_float(u << 16)), s);
      s = fma(w64[2 * x + 1], static_cast<double>(__uint_as_float(u & 0xFFFF0000u)), s);
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// Sum of f32 values with the rounding errors kept beside it (two f32: error
// 2^-48 of the values' sum of magnitudes; f64 adds would cost 30 times as
// much here).
struct TwoSum {
  float s = 0.f, e = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(s, v), bb = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, bb)), __fsub_rn(v, bb)));
    s = t;
  }
  __device__ __forceinline__ double value() const {
    return fabsf(s) < INFINITY ? static_cast<double>(s) + static_cast<double>(e)
                               : static_cast<double>(s);
  }
};

// The f64 weights of a row: M (with lo) then P (with hi).  Where an f32 sum
// leaves the range, in f64 throughout.
template <bool kQ16>
__device__ __forceinline__ void weights64(const SelectArgs& a, const RowView& rv, double* w64,
                                          int t, int nt) {
  const int d = a.head_dim;
  for (int x = t * 4; x < d; x += nt * 4) {
    const int64_t off =
        (static_cast<int64_t>(rv.i) * a.hq + static_cast<int64_t>(rv.h) * a.qhead) * d + x;
    TwoSum neg[4], pos[4];
#pragma unroll 8
    for (int g = 0; g < a.qhead; ++g) {
      const float4 v = q4_of<kQ16>(a.q, off + static_cast<int64_t>(g) * d);
      const float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        neg[e].add(neg_part(q[e]));
        pos[e].add(pos_part(q[e]));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double n = neg[e].value(), p = pos[e].value();
      if (!(fabs(n) < INFINITY) || !(fabs(p) < INFINITY)) {
        n = p = 0.0;
        for (int g = 0; g < a.qhead; ++g) {
          const float q = q_of<kQ16>(a.q, off + e + static_cast<int64_t>(g) * d);
          n += neg_part(q);
          p += pos_part(q);
        }
      }
      w64[x + e] = n;
      w64[d + x + e] = p;
    }
  }
}

// The topk of one row: keys in registers (block t * threads + thread),
// bisection over the keys' range until just k lie above (a dozen counts), the
// border check against eps, f64 scores where it asks for them, and the ids
// written in ascending order.  A CTA of one or eight warps per row (two rows of a
// warp each in a CTA are a tenth slower in the case below: a row whose border
// has to be settled in f64 takes several times as long and holds the other's place).
// What it costs is instructions and the latency of the counts, so the fewest
// threads that hold a row's keys in registers take it.  65536 rows of 256 blocks,
// 32 of them chosen: 101 us, of which the 15 % of rows that f32 leaves open take 40,
// the bisection 18, reading the scores 29; 512 rows of up to 512 blocks, 16
// chosen: 17.5 us; 1024 rows of up to 2048, 64 chosen: 26 us.  (Cuts by
// interpolation need as many counts as bisection; border scores four blocks at a
// time are slower, since most open rows have two or three.)
template <int kWarps, int kKeys, bool kQ16>
__global__ void __launch_bounds__(32 * kWarps) block_pick_kernel(const SelectArgs a) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int kList = 32;
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ int s_red[2 * kWarps];
  __shared__ int s_amb[kList];
  __shared__ int s_namb;
  __shared__ int s_cnt[kWarps == 1 ? 1 : kKeys * kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = static_cast<int>(threadIdx.x);
  const int64_t lrow = blockIdx.x;
  RowGroup<kWarps> grp(s_red);
  const RowView rv = row_view(a, static_cast<unsigned>(a.row0 + lrow), lane);
  const int n = rv.nblk;
  int32_t* out = a.selected + (a.row0 + lrow) * a.topk;
  double* w64 = reinterpret_cast<double*>(s_raw);                                 // [2 d]
  unsigned long long* key64 =
      reinterpret_cast<unsigned long long*>(w64 + 2 * a.head_dim);                // [msb]

  griddep_wait();                        // the scores are there
  uint32_t key[kKeys];
  int n_cand = 0;
  uint32_t kmax = 0u, kinv = 0u;                       // kinv: maximum of ~key
#pragma unroll
  for (int t = 0; t < kKeys; ++t) {
    const int j = t * kThreads + tid;
    key[t] = j < n && n > a.topk ? __ldcg(a.scores + lrow * a.stride + j) : kNoBlock;
  }
  // rows of numbers only, without blocks that come in whatever their score,
  // are the usual case
  bool odd = n <= a.topk || (a.sink | a.local) != 0;
#pragma unroll
  for (int t = 0; t < kKeys; ++t)
    odd = odd || (t * kThreads + tid < n && (key[t] & 0x7FFFFFFFu) > 0x7F800000u);
  if (!grp.max(odd ? 1u : 0u)) {
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      const uint32_t u = key[t];
      key[t] = t * kThreads + tid < n ? u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u)
                                      : 0u;
      kmax = max(kmax, key[t]);
      kinv = max(kinv, t * kThreads + tid < n ? ~key[t] : 0u);
    }
    n_cand = n;
  } else {
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      const int j = t * kThreads + tid;
      uint32_t k = score_key(key[t]);
      if (n <= a.topk && j < n) {
        const int r = bound_row(a, rv.b, j);
        if (r >= 0) {
          const uint16_t* br =
              a.bounds + (static_cast<int64_t>(r) * a.hkv + rv.h) * 2 * a.head_dim;
          k = bf16_to_f32(br[0]) > bf16_to_f32(br[a.head_dim]) ? 0u : 2u;
        }
      }
      if (k != 0u && (j < a.sink || j >= n - a.local)) k = kForced;
      key[t] = k;
      if (k != 0u) {
        ++n_cand;
        kmax = max(kmax, k);
        kinv = max(kinv, ~k);
      }
    }
    n_cand = grp.sum(n_cand);
  }
  const int want = min(n_cand, a.topk);
  uint32_t take_from = 1u;               // keys >= take_from come in
  if (n_cand > a.topk) {
    // bisect for a cut with `want` keys at or above it: count(>= bot) = c_lo >=
    // want, the cut at most top
    uint32_t bot = ~grp.max(kinv), top = grp.max(kmax);
    int c_lo = n_cand;
    while (c_lo != want && bot < top) {
      const uint32_t mid = bot + (top - bot + 1u) / 2u;
      int c = 0;
#pragma unroll
      for (int t = 0; t < kKeys; ++t) c += key[t] >= mid ? 1 : 0;
      c = grp.sum(c);
      if (c >= want) {
        bot = mid;
        c_lo = c;
      } else {
        top = mid - 1u;
      }
    }
    take_from = bot;
    // s_k: the smallest key of the `want` largest; s_next: the largest other
    // (equal to s_k where the cut runs through equal keys)
    uint32_t mk = 0u, mn = 0u;
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      if (key[t] >= take_from)
        mk = max(mk, ~key[t]);
      else
        mn = max(mn, key[t]);
    }
    const uint32_t s_k = ~grp.max(mk);
    uint32_t s_next = grp.max(mn);
    if (c_lo != want) s_next = s_k;
    // eps of the row
    float e = 0.f;
    const int used_chunks = (n + kChunk - 1) / kChunk;
    for (int c = tid; c < used_chunks; c += kThreads)
      e = fmaxf(e, __ldcg(a.eps + lrow * a.chunks + c));
    e = __uint_as_float(grp.max(__float_as_uint(e)));
    const float fk = key_score(s_k), fn = key_score(s_next);
    // (forced blocks lie above every score; NaN and infinite scores are exact
    // unless sums of this size leave f32's range)
    const bool decided = s_k != s_next && (s_k == kForced || (s_next <= 1u && e < INFINITY) ||
                                           fk - fn > 2.f * e);
    if (!decided) {
      // Blocks within 2 eps of the border: those whose rank the f32 scores
      // leave open.  More come in for certain (above) or stay out (below).
      const bool finite = fabsf(fk) < INFINITY && fabsf(fn) < INFINITY && e < INFINITY;
      const float above = finite ? fn + 2.f * e : INFINITY;
      const float below = finite ? fk - 2.f * e : -INFINITY;
      // equal scores with eps = 0, or infinite ones, are exact ties
      const bool exact_tie =
          s_k == s_next && e < INFINITY && (e == 0.f || s_k <= 1u || !(fabsf(fk) < INFINITY));
      int n_in = 0, n_amb = 0;
      if (tid == 0) s_namb = 0;
#pragma unroll
      for (int t = 0; t < kKeys; ++t) {
        const uint32_t k = key[t];
        uint32_t f = 0u;                                // out
        if (exact_tie) {
          f = k > s_k ? 2u : (k == s_k ? 1u : 0u);
        } else if (k == kForced) {
          f = 2u;
        } else if (k != 0u) {
          const float sc = key_score(k);
          const bool in = finite && sc > above && k != 1u;
          const bool outside = finite && (sc < below || k == 1u);
          f = in ? 2u : (outside ? 0u : 1u);
        }
        key[t] = f;
        n_in += f == 2u ? 1 : 0;
        n_amb += f == 1u ? 1 : 0;
      }
      n_in = grp.sum(n_in);
      n_amb = grp.sum(n_amb);
      const int need = want - n_in;                     // 1 <= need < n_amb
      if (!exact_tie) {
        weights64<kQ16>(a, rv, w64, tid, kThreads);
        grp.sync();
#pragma unroll 1
        for (int t = 0; t < kKeys; ++t) {
          uint32_t kt = 0u;
#pragma unroll
          for (int x = 0; x < kKeys; ++x) kt = x == t ? key[x] : kt;
          unsigned m = __ballot_sync(0xffffffffu, kt == 1u);
          while (m) {
            const int j = t * kThreads + warp * 32 + __ffs(m) - 1;
            m &= m - 1;
            const double sc = score64(a, rv, w64, j, lane);
            if (lane == 0) {
              key64[j] = score_key64(sc);
              const int at = atomicAdd(&s_namb, 1);
              if (at < kList) s_amb[at] = j;
            }
          }
        }
        grp.sync();
      }
      if (!exact_tie && n_amb <= kList) {
        // every warp ranks the list: a block comes in with fewer than `need`
        // better ones
        const int j = lane < n_amb ? s_amb[lane] : -1;
        const unsigned long long kj = j >= 0 ? key64[j] : 0ull;
        int rank = 0;
        for (int t = 0; t < n_amb; ++t) {
          const int jt = __shfl_sync(0xffffffffu, j, t);
          const unsigned long long kt = __shfl_sync(0xffffffffu, kj, t);
          rank += (kt > kj || (kt == kj && jt < j)) ? 1 : 0;
        }
        const bool in = j >= 0 && rank < need;
        unsigned m = __ballot_sync(0xffffffffu, in);
        while (m) {
          const int src = __ffs(m) - 1;
          m &= m - 1;
          const int js = __shfl_sync(0xffffffffu, j, src);
#pragma unroll
          for (int t = 0; t < kKeys; ++t)
            if (js == t * kThreads + tid) key[t] = 2u;
        }
      } else {
        // the need-th largest key, bit by bit, then the lowest ids among its
        // equals (key64 is the thread's own here)
        unsigned long long cut = 0ull;
        if (!exact_tie) {
          for (int bit = 63; bit >= 0; --bit) {
            const unsigned long long mid = cut | (1ull << bit);
            int c = 0;
#pragma unroll
            for (int t = 0; t < kKeys; ++t)
              if (key[t] == 1u) c += key64[t * kThreads + tid] >= mid ? 1 : 0;
            if (grp.sum(c) >= need) cut = mid;
          }
        }
        int c = 0;
#pragma unroll
        for (int t = 0; t < kKeys; ++t)
          if (key[t] == 1u && !exact_tie) {
            const unsigned long long kt = key64[t * kThreads + tid];
            if (kt > cut) {
              key[t] = 2u;
              ++c;
            } else if (kt < cut) {
              key[t] = 0u;
            }
          }
        int left = need - grp.sum(c);
        // the first `left` of the remaining equals, 32 kWarps blocks at a time
#pragma unroll
        for (int t = 0; t < kKeys; ++t) {
          const bool eq = key[t] == 1u;
          const unsigned m = __ballot_sync(0xffffffffu, eq);
          int before = 0, all = __popc(m);
          if constexpr (kWarps > 1) {
            int* buf = s_red + (grp.par ^= 1) * kWarps;
            if (lane == 0) buf[warp] = all;
            __syncthreads();
            all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              if (w < warp) before += buf[w];
              all += buf[w];
            }
          }
          if (eq) key[t] = before + __popc(m & ((1u << lane) - 1u)) < left ? 2u : 0u;
          left -= all;
        }
      }
      take_from = 2u;
    }
  }

  // ids in ascending order
  int at = 0;
  if constexpr (kWarps > 1) {
    grp.sync();
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      const unsigned m = __ballot_sync(0xffffffffu, key[t] >= take_from);
      if (lane == 0) s_cnt[t * kWarps + warp] = __popc(m);
    }
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < kKeys; ++t) {
    const bool in = key[t] >= take_from;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    int before = 0, all = __popc(m);
    if constexpr (kWarps > 1) {
      all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int x = s_cnt[t * kWarps + w];
        if (w < warp) before += x;
        all += x;
      }
    }
    const int pos = at + before + __popc(m & ((1u << lane) - 1u));
    if (in && pos < a.topk) out[pos] = t * kThreads + tid;
    at += all;
  }
  for (int r = want + tid; r < a.topk; r += kThreads) out[r] = -1;
}

// ------------------------------------------------------------------ host

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Scores and weights of at most this many bytes at a time; larger problems run
// in parts.
constexpr size_t kScoreBytes = size_t{256} << 20;

struct SelectLayout {
  int64_t stride;        // scores per row
  int32_t chunks;
  int64_t rows;          // rows per launch
  size_t eps, weights, maxima, total;
};

SelectLayout select_layout(int64_t tq, int32_t batch, int32_t hkv, int32_t head_dim, int32_t msb) {
  SelectLayout l{};
  l.stride = std::max<int64_t>((msb + 31) / 32 * 32, 32);
  l.chunks = std::max((msb + kChunk - 1) / kChunk, 1);
  const int64_t all = tq * hkv;
  const int64_t row_bytes = l.stride * 4 + 8 * static_cast<int64_t>(head_dim);
  l.rows = std::min<int64_t>(
      all, std::max<int64_t>(static_cast<int64_t>(kScoreBytes) / row_bytes / hkv, 1) * hkv);
  l.rows = std::max<int64_t>(l.rows, 1);
  l.eps = up256(static_cast<size_t>(l.rows) * l.stride * 4);
  l.weights = l.eps + up256(static_cast<size_t>(l.rows) * l.chunks * 4);
  l.maxima = l.weights + up256(static_cast<size_t>(l.rows) * 8 * head_dim);
  l.total = l.maxima + up256(static_cast<size_t>(batch) * hkv * l.chunks * 4 * head_dim);
  return l;
}

// Calls f with the type of q as a constant.
template <typename F>
auto by_q_type(const SelectArgs& a, F f) {
  return a.q_bf16 ? f(std::true_type{}) : f(std::false_type{});
}

template <int kT, int kNQ, int kSpan>
cudaError_t launch_score(const SelectArgs& a, cudaStream_t s) {
  return by_q_type(a, [&](auto q16) {
    auto fn = block_score_kernel<kT, kNQ, kSpan, decltype(q16)::value>;
    const int smem = kScoreWarps * score_ring(kT) * kGroup * score_row_bytes(a.head_dim);
    static SmemLimit limit;
    const cudaError_t err = limit.raise(reinterpret_cast<const void*>(fn), smem);
    if (err != cudaSuccess) return err;
    const int64_t spans = (a.chunks + kSpan - 1) / kSpan;
    fn<<<static_cast<unsigned>(a.rows * spans), kScoreThreads, smem, s>>>(a);
    return cudaGetLastError();
  });
}

template <int kT>
cudaError_t launch_score_nq(const SelectArgs& a, bool one, cudaStream_t s) {
  if (!one) return launch_score<kT, 5, 1>(a, s);
  // (two CTAs per SM are there at a time)
  return a.rows * a.chunks <= 2 * device_sm_count() ? launch_score<kT, 1, 1>(a, s)
                                                    : launch_score<kT, 1, 2>(a, s);
}

template <int kG>
cudaError_t launch_tile(const SelectArgs& a, cudaStream_t s) {
  const int64_t grid = a.slots * a.hkv * a.chunks;
  if (grid > 0x7FFFFFFF) return cudaErrorNotSupported;
  const int64_t work = a.rows * (a.head_dim / 4);
  const unsigned g = static_cast<unsigned>(
      std::min<int64_t>((work + 255) / 256, static_cast<int64_t>(device_sm_count()) * 16));
  by_q_type(a, [&](auto q16) {
    block_weights_kernel<decltype(q16)::value><<<g, 256, 0, s>>>(a);
    return 0;
  });
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  static SmemLimit limit;
  err = limit.raise(reinterpret_cast<const void*>(block_score_tile_kernel<kG>), TileSmem<kG>::kTotal);
  if (err != cudaSuccess) return err;
  // The maxima beside the weights, and the tiles' first bounds beside both
  // (11 us less for the case of 8192 queries): the weights kernel starts after all
  // earlier work, so the bounds that the others read meanwhile are there.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.hkv * a.chunks);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, block_maxima_kernel, a);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = TileSmem<kG>::kTotal;
  return cudaLaunchKernelEx(&cfg, block_score_tile_kernel<kG>, a);
}

template <int kWarps, int kKeys>
cudaError_t launch_pick(const SelectArgs& a, bool behind_scores, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(2) * a.head_dim * 8 + static_cast<size_t>(a.msb) * 8;
  return by_q_type(a, [&](auto q16) {
    auto fn = block_pick_kernel<kWarps, kKeys, decltype(q16)::value>;
    if (smem > 32 * 1024) {            // (the default limit counts the static part too)
      static SmemLimit limit;
      const cudaError_t err =
          limit.raise(reinterpret_cast<const void*>(fn), static_cast<int>(smem));
      if (err != cudaSuccess) return err;
    }
    // Behind a score kernel its prologue overlaps that kernel's end.  (Behind
    // another it would overlap work that may still write its inputs.)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind_scores ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, a);
  });
}

// `longest`: most queries of one sequence.
cudaError_t launch_select(SelectArgs a, const SelectLayout& l, int64_t longest, cudaStream_t s) {
  cudaError_t err;
  // The tile kernel from 8 queries of a sequence on, where its weights fit in
  // registers (16 sequences, 8 heads of 128 channels, 256 blocks: 4 queries 41 us
  // with it, 31 us without; 8: 43 and 51; 32: 47 and 147).
  const bool tile = longest >= kTileQ / 8 && a.head_dim <= 128;
  a.slots = slot_base(a.tq, a.batch, kTileQ);
  const int64_t all = a.tq * a.hkv;
  for (int64_t r0 = 0; r0 < all; r0 += l.rows) {
    a.row0 = r0;
    a.rows = std::min<int64_t>(l.rows, all - r0);
    if (a.rows * a.chunks > 0x7FFFFFFF) return cudaErrorNotSupported;
    // (no scores where no query can see more blocks than it takes)
    if (a.msb > a.topk) {
      const bool one = longest <= 1;
      if (tile)
        err = a.head_dim <= 32   ? launch_tile<1>(a, s)
              : a.head_dim <= 64 ? launch_tile<2>(a, s)
                                 : launch_tile<4>(a, s);
      else
        err = a.head_dim <= 32    ? launch_score_nq<2>(a, one, s)
              : a.head_dim <= 64  ? launch_score_nq<4>(a, one, s)
              : a.head_dim <= 128 ? launch_score_nq<8>(a, one, s)
                                  : launch_score_nq<16>(a, one, s);
      if (err != cudaSuccess) return err;
    }
    // A warp per row while a row's keys fit in its registers: 65536 rows of 256
    // blocks take 101 us, some 700 us with a CTA of eight warps per row; 32 rows of 512
    // blocks the same time either way (13 and 14 us with their scores).
    if (a.msb <= 256) err = launch_pick<1, 8>(a, a.msb > a.topk, s);
    else if (a.msb <= 512) err = launch_pick<1, 16>(a, a.msb > a.topk, s);
    else if (a.msb <= 2048) err = launch_pick<8, 8>(a, a.msb > a.topk, s);
    else if (a.msb <= 4096) err = launch_pick<8, 16>(a, a.msb > a.topk, s);
    else err = launch_pick<8, 64>(a, a.msb > a.topk, s);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace

}  // namespace sa

extern "C" {

sa_status sa_select_workspace_size(int64_t tq, int32_t batch, int32_t hkv, int32_t head_dim,
                                   int32_t msb, size_t* bytes) {
  if (bytes == nullptr) return SA_ERR_INVALID_ARGUMENT;
  if (hkv <= 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0) return SA_ERR_BLOCK_PAGE;
  if (batch < 1) return SA_ERR_CU_SEQLENS;
  if (tq < 0 || msb < 0) return SA_ERR_SHAPE;
  if (msb > sa::kMaxMsb || head_dim % 8 != 0 || head_dim > 256) return SA_ERR_UNSUPPORTED;
  *bytes = sa::select_layout(tq, batch, hkv, head_dim, msb).total;
  return SA_OK;
}

sa_status sa_select_blocks(const void* q, sa_dtype q_dtype, int64_t tq, int32_t hq, int32_t hkv,
                           int32_t head_dim, const void* bounds, int64_t num_bounds,
                           const int32_t* bound_tables, int32_t msb,
                           const int64_t* cu_seqlens_q_host, const int64_t* cu_seqlens_q,
                           int32_t batch, const int32_t* used_kv_lens, int32_t block_size,
                           int32_t topk, int32_t causal, int32_t sink_blocks,
                           int32_t local_blocks, int32_t* selected, void* workspace,
                           size_t workspace_bytes, int64_t* status, void* stream) {
  if (hkv <= 0 || hq <= 0 || hq % hkv != 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0 || block_size <= 0) return SA_ERR_BLOCK_PAGE;
  if (tq == 0 || topk == 0) return SA_ERR_EMPTY;
  if (tq < 0 || topk < 0 || msb < 0 || num_bounds < 0) return SA_ERR_SHAPE;
  const sa_status st = sa::check_lengths(cu_seqlens_q_host, batch, tq);
  if (st != SA_OK) return st;
  if (q_dtype != SA_DTYPE_F32 && q_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
  if (causal < 0 || causal > 2) return SA_ERR_INVALID_ARGUMENT;
  if (sink_blocks < 0 || local_blocks < 0 ||
      static_cast<int64_t>(sink_blocks) + local_blocks > topk)
    return SA_ERR_INVALID_ARGUMENT;
  if (head_dim % 8 != 0 || head_dim > 256 || msb > sa::kMaxMsb ||
      tq * hkv * static_cast<int64_t>(topk) >= (int64_t{1} << 31))
    return SA_ERR_UNSUPPORTED;
  if (!q || !bounds || !bound_tables || !cu_seqlens_q || !used_kv_lens || !selected || !workspace)
    return SA_ERR_INVALID_ARGUMENT;
  if (!sa::aligned16(q) || !sa::aligned16(bounds) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return SA_ERR_INVALID_ARGUMENT;
  const sa::SelectLayout l = sa::select_layout(tq, batch, hkv, head_dim, msb);
  if (workspace_bytes < l.total) return SA_ERR_INVALID_ARGUMENT;

  sa::SelectArgs a{};
  a.q = q;
  a.q_bf16 = q_dtype == SA_DTYPE_BF16 ? 1 : 0;
  a.tq = tq;
  a.hq = hq;
  a.hkv = hkv;
  a.qhead = hq / hkv;
  a.head_dim = head_dim;
  a.bounds = static_cast<const uint16_t*>(bounds);
  a.num_bounds = num_bounds;
  a.bound_tables = bound_tables;
  a.msb = msb;
  a.cu = cu_seqlens_q;
  a.batch = batch;
  a.used = used_kv_lens;
  a.block_size = block_size;
  a.topk = topk;
  a.causal = causal;
  a.sink = sink_blocks;
  a.local = local_blocks;
  a.selected = selected;
  a.scores = static_cast<uint32_t*>(workspace);
  a.eps = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + l.eps);
  a.weights = reinterpret_cast<uint16_t*>(static_cast<unsigned char*>(workspace) + l.weights);
  a.maxima = reinterpret_cast<uint16_t*>(static_cast<unsigned char*>(workspace) + l.maxima);
  a.stride = l.stride;
  a.chunks = l.chunks;
  a.status = status;
  int site = sa::kStallNone;
  sa::debug_stall_setting(&site, &a.spin);
  if (a.spin == 0) a.spin = sa::kSpinLimit;
  a.stall = site == sa::kStallSelectCopies ? 1 : 0;
  int64_t longest = 0;
  for (int32_t b = 0; b < batch; ++b)
    longest = std::max(longest, cu_seqlens_q_host[b + 1] - cu_seqlens_q_host[b]);
  const cudaError_t err = sa::launch_select(a, l, longest, static_cast<cudaStream_t>(stream));
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
