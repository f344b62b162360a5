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

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kChunk = 128;            // blocks per CTA of the score kernel
constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;
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
  uint32_t* scores;                    // [rows, stride] f32 bits
  float* eps;                          // [rows, chunks]
  int64_t stride;
  int32_t chunks;
  int64_t* status;
};

// What a (query, kv head) row sees: its sequence and the number of blocks
// with a key it may attend to.
struct RowView {
  int64_t i;
  int h, b, nblk;
};

__device__ __forceinline__ RowView row_view(const SelectArgs& a, int64_t row, int lane) {
  RowView v;
  v.i = row / a.hkv;
  v.h = static_cast<int>(row - v.i * a.hkv);
  // the sequence of query i: slots of one position each, without the slack
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int cand = lo + lane * step;
    const bool le = cand < hi && a.cu[cand] <= v.i;
    const unsigned bal = __ballot_sync(0xffffffffu, le);
    const int last = bal ? 31 - __clz(bal) : 0;
    const int nlo = lo + last * step;
    hi = min(nlo + step, hi);
    lo = nlo;
  }
  v.b = lo;
  const int64_t c0 = a.cu[lo], qo = a.cu[lo + 1] - c0;
  const int64_t lk = max(a.used[lo], 0);
  int64_t seen = lk;
  if (a.causal) {
    const int64_t ql = v.i - c0;
    const int64_t pos = a.causal == 2 || lk < qo ? ql : lk - qo + ql;
    seen = min(lk, max(pos + 1, int64_t{0}));
  }
  v.nblk = static_cast<int>(min((seen + a.block_size - 1) / a.block_size,
                                static_cast<int64_t>(a.msb)));
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

// Scores of kChunk blocks for one row.  Reads 4 head_dim bytes per block, a
// group of kW lanes per bounds row (16 bytes each), and little else: the time
// is that of reading the bounds.
template <int kW, int kPieces>
__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(const SelectArgs a) {
  constexpr int kRows = 32 / kW;                       // bounds rows per warp load
  constexpr int kBatch = 8;                            // loads in flight per lane
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int64_t lrow = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - lrow * a.chunks);
  const RowView rv = row_view(a, a.row0 + lrow, lane);
  const int j0 = chunk * kChunk;
  // (a row that takes every block it sees needs no scores)
  if (j0 >= rv.nblk || rv.nblk <= a.topk) return;
  const int j1 = min(j0 + kChunk, rv.nblk);
  const int d = a.head_dim;
  const int pieces = d >> 2;                           // 8-channel pieces of a row
  const int sub = lane / kW;
  const int p = lane % kW;

  // the row's weights on this lane's channels
  float w[kPieces][8];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c][e] = 0.f;
    const int pc = p + c * kW;
    if (pc < pieces) {
      const bool is_hi = pc * 8 >= d;
      const int ch = pc * 8 - (is_hi ? d : 0);
      for (int g = 0; g < a.qhead; ++g) {
        const int64_t off =
            (rv.i * a.hq + static_cast<int64_t>(rv.h) * a.qhead + g) * d + ch;
        float x[8];
        if (a.q_bf16) {
          const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + off);
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(uu[e] << 16);
            x[2 * e + 1] = __uint_as_float(uu[e] & 0xFFFF0000u);
          }
        } else {
          const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + off);
          const float4 u0 = f[0], u1 = f[1];
          x[0] = u0.x; x[1] = u0.y; x[2] = u0.z; x[3] = u0.w;
          x[4] = u1.x; x[5] = u1.y; x[6] = u1.z; x[7] = u1.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          // (a NaN of q stays one)
          w[c][e] += x[e] != x[e] ? x[e] : (is_hi ? fmaxf(x[e], 0.f) : fminf(x[e], 0.f));
      }
    }
  }

  uint32_t bmax[kPieces][4];           // largest |bound| per channel, packed bf16
#pragma unroll
  for (int c = 0; c < kPieces; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) bmax[c][e] = 0u;

  const int per_warp = kChunk / kScoreWarps;
  const int jw0 = j0 + warp * per_warp;
  const int jw1 = min(jw0 + per_warp, j1);
  for (int jb = jw0; jb < jw1; jb += kBatch * kRows) {
    uint4 x[kBatch][kPieces];
    int rr[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const int j = jb + t * kRows + sub;
      rr[t] = j < jw1 ? bound_row(a, rv.b, j) : -1;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const int pc = p + c * kW;
        x[t][c] = make_uint4(0u, 0u, 0u, 0u);
        if (rr[t] >= 0 && pc < pieces)
          x[t][c] = __ldg(reinterpret_cast<const uint4*>(
              a.bounds + (static_cast<int64_t>(rr[t]) * a.hkv + rv.h) * 2 * d + pc * 8));
      }
    }
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const uint32_t u[4] = {x[t][c].x, x[t][c].y, x[t][c].z, x[t][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(w[c][2 * e], __uint_as_float(u[e] << 16), s);
          s = fmaf(w[c][2 * e + 1], __uint_as_float(u[e] & 0xFFFF0000u), s);
          // magnitudes order like their bits: a packed 16-bit maximum
          bmax[c][e] = __vmaxu2(bmax[c][e], u[e] & 0x7FFF7FFFu);
        }
      }
#pragma unroll
      for (int off = kW / 2; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const int j = jb + t * kRows + sub;
      if (p == 0 && j < jw1) {
        uint32_t bits = __float_as_uint(s);
        if (!(fabsf(s) < INFINITY)) {
          if (s != s) bits = 0x7FFFFFFFu;
          // a block without keys holds lo = inf, hi = -inf
          if (rr[t] >= 0) {
            const uint16_t* br = a.bounds + (static_cast<int64_t>(rr[t]) * a.hkv + rv.h) * 2 * d;
            if (bf16_to_f32(br[0]) > bf16_to_f32(br[d])) bits = kNoBlock;
          }
        }
        a.scores[lrow * a.stride + j] = rr[t] >= 0 ? bits : kNoBlock;
      }
    }
  }

  // Infinite and NaN bounds (a block without keys holds +-inf) do not count:
  // the scores they enter are infinite or NaN, in f64 as in f32, and order the
  // same.  Where a lane met one, its maxima are taken again without them.
  bool special = false;
#pragma unroll
  for (int c = 0; c < kPieces; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      special = special || (bmax[c][e] & 0xFFFFu) >= 0x7F80u || (bmax[c][e] >> 16) >= 0x7F80u;
  if (special) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) bmax[c][e] = 0u;
    for (int j = jw0 + sub; j < jw1; j += kRows) {
      const int r = bound_row(a, rv.b, j);
      if (r < 0) continue;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const int pc = p + c * kW;
        if (pc >= pieces) continue;
        const uint4 x = *reinterpret_cast<const uint4*>(
            a.bounds + (static_cast<int64_t>(r) * a.hkv + rv.h) * 2 * d + pc * 8);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t l = u[e] & 0x7FFFu, g = (u[e] >> 16) & 0x7FFFu;
          l = l >= 0x7F80u ? 0u : l;
          g = g >= 0x7F80u ? 0u : g;
          bmax[c][e] = __vmaxu2(bmax[c][e], l | (g << 16));
        }
      }
    }
  }
  // eps of this chunk: (terms added in a chain) * 2^-24 of the sum of
  // |weight| * largest |bound|, which no block's sum of |terms| exceeds.
  float l1 = 0.f;
#pragma unroll
  for (int c = 0; c < kPieces; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w0 = fabsf(w[c][2 * e]), w1 = fabsf(w[c][2 * e + 1]);
      l1 += w0 < INFINITY ? w0 * __uint_as_float(bmax[c][e] << 16) : 0.f;
      l1 += w1 < INFINITY ? w1 * __uint_as_float(bmax[c][e] & 0xFFFF0000u) : 0.f;
    }
#pragma unroll
  for (int off = kW / 2; off; off >>= 1) l1 += __shfl_xor_sync(0xffffffffu, l1, off);
#pragma unroll
  for (int off = 16; off >= kW; off >>= 1) l1 = fmaxf(l1, __shfl_xor_sync(0xffffffffu, l1, off));
  __shared__ float s_l1[kScoreWarps];
  if (lane == 0) s_l1[warp] = l1;
  __syncthreads();
  if (threadIdx.x == 0) {
    float m = 0.f;
    for (int k = 0; k < kScoreWarps; ++k) m = fmaxf(m, s_l1[k]);
    a.eps[lrow * a.chunks + chunk] =
        m * (static_cast<float>(a.qhead + 8 * kPieces + 16) * 0x1p-24f);
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

// Sum over the CTA (all threads call; result to all).
__device__ __forceinline__ int cta_sum(int x, int* s_red) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = x;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) t += s_red[w];
  return t;
}
__device__ __forceinline__ uint32_t cta_max(uint32_t x, uint32_t* s_red) {
  x = __reduce_max_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) t = max(t, s_red[w]);
  return t;
}

// One warp's f64 score of block j: the weights from shared memory.
__device__ __forceinline__ double score64(const SelectArgs& a, const RowView& rv, const double* w64,
                                          int j, int lane) {
  const int d = a.head_dim;
  const int r = bound_row(a, rv.b, j);
  double s = 0.0;
  if (r >= 0) {
    const uint16_t* br = a.bounds + (static_cast<int64_t>(r) * a.hkv + rv.h) * 2 * d;
    for (int x = lane; x < 2 * d; x += 32) s += w64[x] * static_cast<double>(bf16_to_f32(br[x]));
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// The f64 weights of a row: M (with lo) then P (with hi).
__device__ __forceinline__ void weights64(const SelectArgs& a, const RowView& rv, double* w64,
                                          int t, int nt) {
  const int d = a.head_dim;
  for (int x = t; x < d; x += nt) {
    double neg = 0.0, pos = 0.0;
    for (int g = 0; g < a.qhead; ++g) {
      const float q = q_at(a, (rv.i * a.hq + static_cast<int64_t>(rv.h) * a.qhead + g) * d + x);
      if (q != q) {
        neg += q;
        pos += q;
      } else {
        neg += fminf(q, 0.f);
        pos += fmaxf(q, 0.f);
      }
    }
    w64[x] = neg;
    w64[d + x] = pos;
  }
}

// The topk of one row, one CTA per row: keys in shared memory; bisection over
// the keys' range until just k lie above (a handful of counts), the border
// check against eps, f64 scores where it asks for them, and the ids written
// in ascending order.
__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ int s_cnt[kPickWarps];
  __shared__ uint32_t s_red[kPickWarps];
  __shared__ int s_amb[32];
  __shared__ int s_namb;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t lrow = blockIdx.x;
  const RowView rv = row_view(a, a.row0 + lrow, lane);
  const int n = rv.nblk;
  int32_t* out = a.selected + (a.row0 + lrow) * a.topk;
  double* w64 = reinterpret_cast<double*>(s_raw);                       // [2 d]
  unsigned long long* key64 = reinterpret_cast<unsigned long long*>(w64 + 2 * a.head_dim);  // [msb]
  uint32_t* key = reinterpret_cast<uint32_t*>(key64 + a.msb);          // [msb]

  // keys
  int n_cand = 0;
  uint32_t kmax = 0u, kinv = 0u;                       // kinv: maximum of ~key
  for (int j = tid; j < n; j += kPickThreads) {
    uint32_t k;
    if (n <= a.topk) {
      const int r = bound_row(a, rv.b, j);
      k = 0u;
      if (r >= 0) {
        const uint16_t* br =
            a.bounds + (static_cast<int64_t>(r) * a.hkv + rv.h) * 2 * a.head_dim;
        k = bf16_to_f32(br[0]) > bf16_to_f32(br[a.head_dim]) ? 0u : 2u;
      }
    } else {
      k = score_key(__ldcg(a.scores + lrow * a.stride + j));
    }
    if (k != 0u && (j < a.sink || j >= n - a.local)) k = kForced;
    key[j] = k;
    if (k != 0u) {
      ++n_cand;
      kmax = max(kmax, k);
      kinv = max(kinv, ~k);
    }
  }
  n_cand = cta_sum(n_cand, s_cnt);
  const int want = min(n_cand, a.topk);
  uint32_t take_from = 1u;               // keys >= take_from come in
  if (n_cand > a.topk) {
    // bisect for a cut with `want` keys at or above it; lo keeps count >= want,
    // hi count < want
    uint32_t lo = ~cta_max(kinv, s_red), hi = cta_max(kmax, s_red);
    // count(>= lo) = n_cand >= want; the cut may lie at hi itself
    int c_lo = n_cand;
    unsigned long long top = static_cast<unsigned long long>(hi) + 1ull;   // count(>= top) = 0
    unsigned long long bot = lo;
    while (c_lo != want && top - bot > 1ull) {
      const uint32_t mid = static_cast<uint32_t>(bot + (top - bot) / 2ull);
      int c = 0;
      for (int j = tid; j < n; j += kPickThreads) c += key[j] >= mid ? 1 : 0;
      c = cta_sum(c, s_cnt);
      if (c >= want) {
        bot = mid;
        c_lo = c;
      } else {
        top = mid;
      }
    }
    take_from = static_cast<uint32_t>(bot);
    // s_k: the smallest key of the `want` largest; s_next: the largest other
    // (equal to s_k where the cut runs through equal keys)
    uint32_t mk = 0u, mn = 0u;
    for (int j = tid; j < n; j += kPickThreads) {
      const uint32_t k = key[j];
      if (k >= take_from) mk = max(mk, ~k);
      else mn = max(mn, k);
    }
    const uint32_t s_k = ~cta_max(mk, s_red);
    uint32_t s_next = cta_max(mn, s_red);
    if (c_lo != want) s_next = s_k;
    // eps of the row
    float e = 0.f;
    const int used_chunks = (n + kChunk - 1) / kChunk;
    for (int c = tid; c < used_chunks; c += kPickThreads)
      e = fmaxf(e, __ldcg(a.eps + lrow * a.chunks + c));
    e = __uint_as_float(cta_max(__float_as_uint(e), s_red));
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
      __syncthreads();
      for (int j = tid; j < n; j += kPickThreads) {
        const uint32_t k = key[j];
        uint32_t f = 0u;                                // out
        if (exact_tie) {
          f = k > s_k ? 2u : (k == s_k ? 1u : 0u);
        } else if (k == kForced) {
          f = 2u;
        } else if (k != 0u) {
          const float s = key_score(k);
          // rounding of the borders outward: one more ulp either way
          const bool in = finite && s > above && k != 1u;
          const bool outside = finite && (s < below || k == 1u);
          f = in ? 2u : (outside ? 0u : 1u);
        }
        key[j] = f;
        n_in += f == 2u ? 1 : 0;
        n_amb += f == 1u ? 1 : 0;
      }
      n_in = cta_sum(n_in, s_cnt);
      n_amb = cta_sum(n_amb, s_cnt);
      const int need = want - n_in;                     // 1 <= need < n_amb
      if (exact_tie) {
        for (int j = tid; j < n; j += kPickThreads) key64[j] = 0ull;
        __syncthreads();
      } else {
        weights64(a, rv, w64, tid, kPickThreads);
        __syncthreads();
        for (int jb = warp * 32; jb < n; jb += kPickThreads) {
          unsigned m = __ballot_sync(0xffffffffu, jb + lane < n && key[jb + lane] == 1u);
          while (m) {
            const int j = jb + __ffs(m) - 1;
            m &= m - 1;
            const double s = score64(a, rv, w64, j, lane);
            if (lane == 0) {
              key64[j] = score_key64(s);
              const int at = atomicAdd(&s_namb, 1);
              if (at < 32) s_amb[at] = j;
            }
          }
        }
        __syncthreads();
      }
      if (!exact_tie && n_amb <= 32) {
        if (warp == 0) {
          const int j = lane < n_amb ? s_amb[lane] : -1;
          const unsigned long long kj = j >= 0 ? key64[j] : 0ull;
          int rank = 0;
          for (int t = 0; t < n_amb; ++t) {
            const int jt = __shfl_sync(0xffffffffu, j, t);
            const unsigned long long kt = __shfl_sync(0xffffffffu, kj, t);
            rank += (kt > kj || (kt == kj && jt < j)) ? 1 : 0;
          }
          if (j >= 0) key[j] = rank < need ? 2u : 0u;
        }
        __syncthreads();
      } else {
        // the need-th largest key, bit by bit, then the lowest ids among its
        // equals
        unsigned long long cut = 0ull;
        if (!exact_tie) {
          for (int bit = 63; bit >= 0; --bit) {
            const unsigned long long mid = cut | (1ull << bit);
            int c = 0;
            for (int j = tid; j < n; j += kPickThreads)
              c += key[j] == 1u && key64[j] >= mid ? 1 : 0;
            if (cta_sum(c, s_cnt) >= need) cut = mid;
          }
        }
        int c = 0;
        for (int j = tid; j < n; j += kPickThreads) {
          if (key[j] == 1u && key64[j] > cut) {
            key[j] = 2u;
            ++c;
          }
        }
        const int left = need - cta_sum(c, s_cnt);
        // the first `left` of the remaining equals: count per warp range
        const int span = (n + kPickWarps - 1) / kPickWarps;
        const int a0 = min(warp * span, n), a1 = min(a0 + span, n);
        int mine = 0;
        for (int jb = a0; jb < a1; jb += 32) {
          const int j = jb + lane;
          const bool eq = j < a1 && key[j] == 1u && key64[j] == cut;
          mine += __popc(__ballot_sync(0xffffffffu, eq));
        }
        __syncthreads();
        if (lane == 0) s_cnt[warp] = mine;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += s_cnt[w];
        for (int jb = a0; jb < a1; jb += 32) {
          const int j = jb + lane;
          const bool eq = j < a1 && key[j] == 1u && key64[j] == cut;
          const unsigned m = __ballot_sync(0xffffffffu, eq);
          if (eq) key[j] = before + __popc(m & ((1u << lane) - 1u)) < left ? 2u : 0u;
          before += __popc(m);
        }
        __syncthreads();
      }
      take_from = 2u;
    }
  }

  // ids in ascending order
  const int span = (n + kPickWarps - 1) / kPickWarps;
  const int a0 = min(warp * span, n), a1 = min(a0 + span, n);
  int mine = 0;
  for (int jb = a0; jb < a1; jb += 32) {
    const int j = jb + lane;
    mine += __popc(__ballot_sync(0xffffffffu, j < a1 && key[j] >= take_from));
  }
  __syncthreads();
  if (lane == 0) s_cnt[warp] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += s_cnt[w];
  for (int jb = a0; jb < a1; jb += 32) {
    const int j = jb + lane;
    const bool in = j < a1 && key[j] >= take_from;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const int pos = at + __popc(m & ((1u << lane) - 1u));
    if (in && pos < a.topk) out[pos] = j;
    at += __popc(m);
  }
  for (int r = want + tid; r < a.topk; r += kPickThreads) out[r] = -1;
}

// ------------------------------------------------------------------ host

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Scores of at most this many bytes at a time; larger problems run in parts.
constexpr size_t kScoreBytes = size_t{256} << 20;

struct SelectLayout {
  int64_t stride;        // scores per row
  int32_t chunks;
  int64_t rows;          // rows per launch
  size_t eps, total;
};

SelectLayout select_layout(int64_t tq, int32_t hkv, int32_t msb) {
  SelectLayout l{};
  l.stride = std::max<int64_t>((msb + 31) / 32 * 32, 32);
  l.chunks = std::max((msb + kChunk - 1) / kChunk, 1);
  const int64_t all = tq * hkv;
  l.rows = std::min<int64_t>(
      all, std::max<int64_t>(static_cast<int64_t>(kScoreBytes / (l.stride * 4)) / hkv, 1) * hkv);
  l.rows = std::max<int64_t>(l.rows, 1);
  l.eps = up256(static_cast<size_t>(l.rows) * l.stride * 4);
  l.total = l.eps + up256(static_cast<size_t>(l.rows) * l.chunks * 4);
  return l;
}

template <int kW, int kPieces>
void launch_score(const SelectArgs& a, cudaStream_t s) {
  block_score_kernel<kW, kPieces>
      <<<static_cast<unsigned>(a.rows * a.chunks), kScoreThreads, 0, s>>>(a);
}

size_t pick_smem(int head_dim, int msb) {
  return static_cast<size_t>(2) * head_dim * 8 + static_cast<size_t>(msb) * 12;
}

cudaError_t launch_select(SelectArgs a, const SelectLayout& l, cudaStream_t s) {
  const size_t smem = pick_smem(a.head_dim, a.msb);
  cudaError_t err = cudaFuncSetAttribute(block_pick_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(std::max<size_t>(smem, 48 * 1024)));
  if (err != cudaSuccess) return err;
  const int64_t all = a.tq * a.hkv;
  for (int64_t r0 = 0; r0 < all; r0 += l.rows) {
    a.row0 = r0;
    a.rows = std::min<int64_t>(l.rows, all - r0);
    if (a.rows * a.chunks > 0x7FFFFFFF) return cudaErrorNotSupported;
    const int pieces = a.head_dim / 4;
    if (pieces <= 2) launch_score<2, 1>(a, s);
    else if (pieces <= 4) launch_score<4, 1>(a, s);
    else if (pieces <= 8) launch_score<8, 1>(a, s);
    else if (pieces <= 16) launch_score<16, 1>(a, s);
    else if (pieces <= 32) launch_score<32, 1>(a, s);
    else launch_score<32, 2>(a, s);
    block_pick_kernel<<<static_cast<unsigned>(a.rows), kPickThreads, smem, s>>>(a);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
  *bytes = sa::select_layout(tq, hkv, msb).total;
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
  if (cu_seqlens_q_host == nullptr || batch < 1 || cu_seqlens_q_host[0] != 0)
    return SA_ERR_CU_SEQLENS;
  for (int32_t b = 1; b <= batch; ++b)
    if (cu_seqlens_q_host[b] < cu_seqlens_q_host[b - 1]) return SA_ERR_CU_SEQLENS;
  if (cu_seqlens_q_host[batch] != tq) return SA_ERR_SHAPE;
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
  const sa::SelectLayout l = sa::select_layout(tq, hkv, msb);
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
  a.stride = l.stride;
  a.chunks = l.chunks;
  a.status = status;
  const cudaError_t err = sa::launch_select(a, l, static_cast<cudaStream_t>(stream));
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
