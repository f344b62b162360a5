// Head norms and position rotation of queries and keys in one pass.
//
// Per (token, head) row x of d channels: y = x / sqrt(mean(x^2) + eps) * w (y = x
// without a weight), then pair i of the first rot channels turns by the angle
// p f_i, p the token's position on the pair's axis: (a, b) -> (a cos - b sin,
// a sin + b cos).  The pairs are (i, i + rot / 2), or (2 i, 2 i + 1).
//
// Angles: f32 products p f lose the angle (p = 131072 leaves 2^-7 radians), so
// f / (2 pi) is taken as a 64-bit fraction of a turn.  Its product with the integer p
// wraps at whole turns by itself; the error is |p| (1 + |f| / 256) 2^-64 turns.  What lies beyond the
// nearest quarter of a turn, an eighth at most, goes to sincospif in f32 (2^-28 turns; a
// whole turn in f32 would be rounded by 2^-26), and the quarters turn its results.
#include <cstdint>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;                 // tokens per CTA
// Rows that a lane has in flight, and CTAs per SM that the registers have to leave room for, by the
// source's type and the channels of a piece.
template <bool kSrcBf16, int kC>
constexpr int kRowsOf = kSrcBf16 && kC == 4 ? 4 : 3;
template <int kC>
constexpr int kMinCtas = kC == 8 ? 3 : 4;
// Tokens of a CTA that walks over their heads, as a power of two: more of them make fewer CTAs with
// longer tails, fewer of them fewer rows after the angles.  1 / 2 / 4 tokens, heads of 128, us: f32 8192
// tokens of 64 + 8 heads 93.1 / 93.3 / 97.8, 800 of 32 + 8 10.5 / 8.5 / 11.3, 5000 44.4 / 38.6 / 40.5;
// bf16 to f32 8192 of 64 + 8 80.4 / 76.4 / 79.4; bf16 70.6 / 66.1 / 59.1, 5000 of 32 + 8 41.4 / 33.5 /
// 27.2, 800 7.7 / 6.2 / 7.1 (8 tokens: 27.9 and 9.1).
template <int kC>
constexpr int kLogTokens = kC == 8 ? 2 : 1;

struct RopeArgs {
  const void* src[2];                         // q, k
  void* dst[2];
  int64_t token_stride[2], head_stride[2];    // elements
  int64_t dst_token_stride[2], dst_head_stride[2];
  const void* weight[2];                      // nullable
  int32_t heads[2];
  int32_t weight_bf16;
  float eps;
  const float* inv_freq;
  const int32_t* freq_axes;                   // nullable: axis 0
  const int32_t* positions;                   // nullable: from cu and used
  int64_t axis_stride;
  int32_t n_axes;
  const int64_t* cu;
  const int32_t* used;
  int32_t batch;
  int64_t tq;
  int32_t head_dim, rot, interleaved;
  int64_t* status;
};

// f / (2 pi) as a fraction of a turn, times 2^64 (whole turns dropped).  With f = M
// 2^(e - 150) and C = 2^66 / (2 pi) (the 64 bits kept are 2^-6 off): M C 2^(e - 152), formed as the
// upper half of (M 2^40) C, shifted by e - 128; a shift up (f of 2 and more) brings in the lower half.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>((u >> 23) & 0xFFu);
  const uint64_t m = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  constexpr uint64_t kC = 0xA2F9836E4E44152Aull;
  const uint64_t hi = __umul64hi(m << 40, kC), lo = (m << 40) * kC;
  const int s = (e ? e : 1) - 128;
  const uint64_t v = s <= -64 || s >= 64 ? 0ull : s < 0 ? hi >> -s : s == 0 ? hi : hi << s | lo >> (64 - s);
  return (u >> 31) ? 0ull - v : v;
}

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int pos) {
  const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint64_t quarters = (t + (1ull << 61)) >> 62;
  float s, c;
  sincospif(__ll2float_rn(static_cast<int64_t>(t - (quarters << 62))) * 0x1p-63f, &s, &c);
  const float x = quarters & 1 ? s : c, y = quarters & 1 ? c : s;
  // (cosine's sign turns in the second and third quarter, sine's in the third and fourth)
  return make_float2((quarters + 1) & 2 ? -x : x, quarters & 2 ? -y : y);
}

// Position of token `tok` where the call gives lengths: its sequence's last tokens
// are the new ones.  All lanes of the warp call it.
__device__ __forceinline__ int position_of(const RopeArgs& a, int64_t tok, int lane) {
  // (every sequence so far holds one token: no search)
  int b = static_cast<int>(min(tok, static_cast<int64_t>(a.batch - 1)));
  if (a.cu[b] > tok || a.cu[b + 1] <= tok)
    b = warp_search(a.batch, lane, [&](int x) { return a.cu[x] <= tok; });
  const NewRange r = new_range(a.cu, a.used, b, a.tq);
  return static_cast<int>(r.p0 + (tok - r.cu0));
}

__device__ __forceinline__ int axis_position(const RopeArgs& a, int64_t tok, int pair) {
  int axis = a.freq_axes ? a.freq_axes[pair] : 0;
  if (axis < 0 || axis >= a.n_axes) {
    report(a.status, SA_ERR_SHAPE);
    axis = 0;
  }
  return a.positions[axis * a.axis_stride + tok];
}

// Two f32 numbers side by side, and operations on both at once.
using pair_t = unsigned long long;
__device__ __forceinline__ pair_t make_pair(float lo, float hi) {
  pair_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 both(pair_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ pair_t mul2(pair_t x, pair_t y) {
  pair_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ pair_t fma2(pair_t x, pair_t y, pair_t z) {
  pair_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}

// kC channels of a row as they lie (8 or 16 bytes of bf16, 16 of f32), and as values.
template <bool kBf16, int kC>
struct Raw {
  static constexpr int kWords = kC * (kBf16 ? 2 : 4) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t off) {
    const unsigned char* at = static_cast<const unsigned char*>(p) + off * (kBf16 ? 2 : 4);
    if constexpr (kWords == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(at);
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(at);
      w[0] = u.x;
      w[1] = u.y;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ pair_t pair(int i) const {          // channels 2 i, 2 i + 1
    if constexpr (kBf16)
      return make_pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    else
      return make_pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
};

template <bool kBf16, int kC>
__device__ __forceinline__ void store_piece(void* p, int64_t off, const pair_t (&x)[kC / 2]) {
  float2 v[kC / 2];
#pragma unroll
  for (int i = 0; i < kC / 2; ++i) v[i] = both(x[i]);
  if constexpr (kBf16 && kC == 8) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off) =
        make_uint4(pack_bf16x2_rn(v[0].x, v[0].y), pack_bf16x2_rn(v[1].x, v[1].y),
                   pack_bf16x2_rn(v[2].x, v[2].y), pack_bf16x2_rn(v[3].x, v[3].y));
  } else {
#pragma unroll
    for (int i = 0; i < kC / 4; ++i)
      store_o4(p, kBf16, off + 4 * i, make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y));
  }
}

// A row is spread over kLanes lanes, a lane holding 2 kC channels in two pieces of kC that
// hold whole pairs: channels kC u and rot / 2 + kC u on (or 2 kC u on, where pairs are
// adjacent), so that the rotation needs no other lane.  Either way the pieces' pairs are
// kC u on.  A group of kLanes lanes keeps one token and walks over its heads, kRows of them
// at a time, all asked for before the first is used: angles are made once per
// token and pair, by the CTA, and stay in registers; weights come from shared memory.
//
// Bound by memory from some thousand tokens on: 8192 of 64 + 8 heads of 128 in f32 (604 MB) 93 us,
// 6.5 TB/s, 32768 350 us, 6.9; 32768 in bf16 (1.2 GB) 210 us, 5.7 TB/s.  bf16 stands between: 8192
// tokens keep issue and DRAM 55 % busy each, with 80 registers and a third of the warps; fewer
// instructions helped (4 channels a piece and one number an operation: 288 us for 32768, 8 and two
// numbers 210), what is left is latency.  Rows in flight against CTAs an SM:
//   bf16, 8 channels, 32768 tokens: 3 rows and 3 CTAs 211 us, 2 and 3 221, 2 and 4 211, 3 and 2 248;
// and, with four tokens a CTA,
//   f32, 2048 tokens / 8192: 3 and 4 29.7 / 97.5, 3 and 3 37.4 / 99.7, 2 and 4 29.5 / 100.5, 2 and
//   5 (spilling) 30.6 / 98.2, 4 and 3 36.7 / 98.6;
//   bf16 to f32, 4 channels, 32768: 4 and 4 282, 3 and 4 292, 2 and 4 313.
template <bool kSrcBf16, bool kDstBf16, int kC, int kLanes>
__global__ void __launch_bounds__(kThreads, kMinCtas<kC>)
norm_rope_kernel(const RopeArgs a, int log_tokens, int heads_per_cta) {
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kRows = kRowsOf<kSrcBf16, kC>;
  __shared__ int s_pos[kMaxTokens];
  __shared__ __align__(16) float s_cos[kMaxTokens * 128], s_sin[kMaxTokens * 128];
  __shared__ __align__(16) float s_w[2][256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tokens = 1 << log_tokens;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) << log_tokens;
  const int n_pairs = a.rot >> 1;
  const int group = tid / kLanes, u = tid % kLanes;
  const int64_t tok = tok0 + (group & (tokens - 1));
  const int step = kGroups >> log_tokens;              // heads between a group's rows
  const int total = a.heads[0] + a.heads[1];
  const int end = min(total, static_cast<int>(blockIdx.y + 1) * heads_per_cta);
  int head = static_cast<int>(blockIdx.y) * heads_per_cta + (group >> log_tokens);
  const bool rotated = u < a.rot / (2 * kC);
  const int ca = rotated && !a.interleaved ? kC * u : 2 * kC * u;
  const int cb = rotated && !a.interleaved ? n_pairs + kC * u : ca + kC;
  const bool mine = 2 * kC * u < a.head_dim;
  const bool live = tok < a.tq;

  Raw<kSrcBf16, kC> xa[kRows], xb[kRows];
  auto load_rows = [&](int first) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int h = first + i * step;
      xa[i].zero();
      xb[i].zero();
      if (live && mine && h < end) {
        const int kind = h >= a.heads[0] ? 1 : 0;
        const int64_t at = tok * a.token_stride[kind] +
                           static_cast<int64_t>(h - (kind ? a.heads[0] : 0)) * a.head_stride[kind];
        xa[i].load(a.src[kind], at + ca);
        xb[i].load(a.src[kind], at + cb);
      }
    }
  };
  load_rows(head);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (a.weight[k] != nullptr && tid < a.head_dim)
      s_w[k][tid] = a.weight_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.weight[k])[tid])
                                  : static_cast<const float*>(a.weight[k])[tid];

  if (n_pairs > 0) {
    if (a.positions == nullptr) {
      if (warp < tokens && tok0 + warp < a.tq) {
        const int p = position_of(a, tok0 + warp, lane);
        if (lane == 0) s_pos[warp] = p;
      }
      __syncthreads();
    }
    for (int i = tid; i < tokens * n_pairs; i += kThreads) {
      const int t = i / n_pairs, pair = i - t * n_pairs;
      if (tok0 + t < a.tq) {
        const int p = a.positions ? axis_position(a, tok0 + t, pair) : s_pos[t];
        const float2 turn = cos_sin(turn_fraction(a.inv_freq[pair]), p);
        s_cos[i] = turn.x;
        s_sin[i] = turn.y;
      }
    }
  }
  __syncthreads();
  if (!live) return;
  pair_t co[kC / 2], si[kC / 2];                       // of the lane's pairs, two by two
#pragma unroll
  for (int j = 0; j < kC / 2; ++j) {
    co[j] = make_pair(1.f, 1.f);
    si[j] = make_pair(0.f, 0.f);
    if (rotated) {
      const int at = (group & (tokens - 1)) * n_pairs + kC * u + 2 * j;
      co[j] = *reinterpret_cast<const pair_t*>(s_cos + at);
      si[j] = *reinterpret_cast<const pair_t*>(s_sin + at);
    }
  }
  const unsigned mask = kLanes == 32 ? 0xffffffffu
                                     : ((1u << (kLanes & 31)) - 1u) << ((lane / kLanes) * kLanes);
  for (;;) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int h = head + i * step;
      if (h >= end) return;
      const int kind = h >= a.heads[0] ? 1 : 0;
      pair_t x[kC / 2], y[kC / 2];
#pragma unroll
      for (int c = 0; c < kC / 2; ++c) {
        x[c] = xa[i].pair(c);
        y[c] = xb[i].pair(c);
      }
      // (the same for all lanes of a group, and a group's lanes lie in one warp)
      if (a.weight[kind] != nullptr) {
        pair_t ss2 = make_pair(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kC / 2; ++c) ss2 = fma2(y[c], y[c], fma2(x[c], x[c], ss2));
        float ss = both(ss2).x + both(ss2).y;
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float r = rsqrtf(ss / static_cast<float>(a.head_dim) + a.eps);
        const pair_t rr = make_pair(r, r);
        if (mine) {
          const ulonglong2* wa = reinterpret_cast<const ulonglong2*>(s_w[kind] + ca);
          const ulonglong2* wb = reinterpret_cast<const ulonglong2*>(s_w[kind] + cb);
#pragma unroll
          for (int c = 0; c < kC / 4; ++c) {
            const ulonglong2 p = wa[c], q = wb[c];
            x[2 * c] = mul2(mul2(x[2 * c], rr), p.x);
            x[2 * c + 1] = mul2(mul2(x[2 * c + 1], rr), p.y);
            y[2 * c] = mul2(mul2(y[2 * c], rr), q.x);
            y[2 * c + 1] = mul2(mul2(y[2 * c + 1], rr), q.y);
          }
        }
      }
      if (rotated) {
        if (a.interleaved) {
          // x[c] is pair kC u + c, y[c] pair kC u + kC / 2 + c
          auto turn = [](pair_t& v, float co1, float si1) {
            const float2 p = both(v);
            v = make_pair(p.x * co1 - p.y * si1, p.x * si1 + p.y * co1);
          };
#pragma unroll
          for (int c = 0; c < kC / 4; ++c) {
            const float2 c0 = both(co[c]), s0 = both(si[c]);
            const float2 c1 = both(co[kC / 4 + c]), s1 = both(si[kC / 4 + c]);
            turn(x[2 * c], c0.x, s0.x);
            turn(x[2 * c + 1], c0.y, s0.y);
            turn(y[2 * c], c1.x, s1.x);
            turn(y[2 * c + 1], c1.y, s1.y);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kC / 2; ++c) {
            const pair_t minus = si[c] ^ 0x8000000080000000ull;
            const pair_t p = x[c];
            x[c] = fma2(y[c], minus, mul2(p, co[c]));
            y[c] = fma2(p, si[c], mul2(y[c], co[c]));
          }
        }
      }
      if (mine) {
        const int64_t at =
            tok * a.dst_token_stride[kind] +
            static_cast<int64_t>(h - (kind ? a.heads[0] : 0)) * a.dst_head_stride[kind];
        store_piece<kDstBf16, kC>(a.dst[kind], at + ca, x);
        store_piece<kDstBf16, kC>(a.dst[kind], at + cb, y);
      }
    }
    head += kRows * step;
    load_rows(head);
  }
}

// Any sizes, strides and alignment: a warp per row, a lane per pair (and per
// channel behind the rotated ones), angles made where they are used (8192 tokens of 64 + 8
// heads in f32 whose rows start off 16 bytes: 411 us, the other kernel 93).
template <bool kSrcBf16, bool kDstBf16>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const RopeArgs a) {
  constexpr int kPairs = 4, kRest = 8;                 // of a lane: head_dim <= 256
  const int lane = threadIdx.x & 31;
  const int total = a.heads[0] + a.heads[1];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.tq * total) return;
  const int64_t tok = row / total;
  const int h = static_cast<int>(row - tok * total);
  const int kind = h >= a.heads[0] ? 1 : 0;
  const int hh = h - (kind ? a.heads[0] : 0);
  const int64_t from = tok * a.token_stride[kind] + hh * a.head_stride[kind];
  const int64_t to = tok * a.dst_token_stride[kind] + hh * a.dst_head_stride[kind];
  const int n_pairs = a.rot >> 1, rest = a.head_dim - a.rot;
  auto get = [&](int c) {
    if constexpr (kSrcBf16)
      return bf16_to_f32(static_cast<const uint16_t*>(a.src[kind])[from + c]);
    else
      return static_cast<const float*>(a.src[kind])[from + c];
  };
  auto put = [&](int c, float v) {
    if constexpr (kDstBf16)
      static_cast<uint16_t*>(a.dst[kind])[to + c] =
          static_cast<uint16_t>(pack_bf16x2_rn(v, 0.f) & 0xFFFFu);
    else
      static_cast<float*>(a.dst[kind])[to + c] = v;
  };
  auto weight = [&](int c) {
    return a.weight_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.weight[kind])[c])
                         : static_cast<const float*>(a.weight[kind])[c];
  };
  auto first = [&](int pair) { return a.interleaved ? 2 * pair : pair; };
  auto second = [&](int pair) { return a.interleaved ? 2 * pair + 1 : pair + n_pairs; };
  float p[kPairs], q[kPairs], r[kRest];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int pair = lane + 32 * i;
    p[i] = q[i] = 0.f;
    if (pair < n_pairs) {
      p[i] = get(first(pair));
      q[i] = get(second(pair));
    }
    ss = fmaf(p[i], p[i], fmaf(q[i], q[i], ss));
  }
#pragma unroll
  for (int i = 0; i < kRest; ++i) {
    r[i] = lane + 32 * i < rest ? get(a.rot + lane + 32 * i) : 0.f;
    ss = fmaf(r[i], r[i], ss);
  }
  const bool norm = a.weight[kind] != nullptr;
  float inv = 1.f;
  if (norm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    inv = rsqrtf(ss / static_cast<float>(a.head_dim) + a.eps);
  }
  const int pos = a.positions == nullptr && n_pairs > 0 ? position_of(a, tok, lane) : 0;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int pair = lane + 32 * i;
    if (pair < n_pairs) {
      const float2 t = cos_sin(turn_fraction(a.inv_freq[pair]),
                               a.positions ? axis_position(a, tok, pair) : pos);
      float x = p[i], y = q[i];
      if (norm) {
        x = x * inv * weight(first(pair));
        y = y * inv * weight(second(pair));
      }
      put(first(pair), x * t.x - y * t.y);
      put(second(pair), x * t.y + y * t.x);
    }
  }
#pragma unroll
  for (int i = 0; i < kRest; ++i) {
    const int c = a.rot + lane + 32 * i;
    if (c < a.head_dim) put(c, norm ? r[i] * inv * weight(c) : r[i]);
  }
}

template <bool kSrcBf16, bool kDstBf16, int kC>
cudaError_t launch_wide(const RopeArgs& a, cudaStream_t stream) {
  const int total = a.heads[0] + a.heads[1];
  const int units = a.head_dim / (2 * kC);
  const int lanes = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
  const int groups = kThreads / lanes;
  constexpr int kRows = kRowsOf<kSrcBf16, kC>;
  // Prompts: two or four tokens a CTA, whose groups walk over the heads in `turns` turns of kRows.
  // Few tokens: one, and its heads over several CTAs, so that a row is all that a group does.  A turn
  // takes about half as long as a round of CTAs: 32 + 8 heads of 128, several tokens / one token a
  // CTA, us: f32 64 tokens (2 turns, 1 round) 5.2 / 3.8, 128 (1 round) 5.4 / 4.2, 256 (2 rounds) 5.7 /
  // 6.2, 800 (4 rounds) 8.7 / 12.3; bf16 (2 turns) 64 (1 round) 5.6 / 3.5, 256 (2 rounds) 5.8 / 6.0,
  // 800 7.3 / 10.9; 8 + 1 heads (1 turn): bf16 500 tokens (2 rounds) 4.3 / 5.8.
  const int64_t slots = static_cast<int64_t>(kMinCtas<kC>) * device_sm_count();
  const int64_t rounds = (a.tq * ((total + groups - 1) / groups) + slots - 1) / slots;
  const int64_t turns =
      ((static_cast<int64_t>(total) << kLogTokens<kC>) + kRows * groups - 1) / (kRows * groups);
  const bool few = 2 * rounds <= turns + 1;
  const int log_tokens = few ? 0 : kLogTokens<kC>;
  const int heads_per_cta = few ? groups : total;
  const int64_t gx = (a.tq + (int64_t{1} << log_tokens) - 1) >> log_tokens;
  const int64_t gy = (total + heads_per_cta - 1) / heads_per_cta;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a, log_tokens, heads_per_cta); };
  if (lanes == 4)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, kC, 4>);
  else if (lanes == 8)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, kC, 8>);
  else if (lanes == 16)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, kC, 16>);
  else if constexpr (kC == 4)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, kC, 32>);
  return cudaGetLastError();
}

// piece: channels of a piece that sizes, strides and alignment allow (8, 4, or 0: none).
template <bool kSrcBf16, bool kDstBf16>
cudaError_t launch_rope(const RopeArgs& a, int piece, cudaStream_t stream) {
  if (piece == 0) {
    const int64_t rows = a.tq * (a.heads[0] + a.heads[1]);
    const int64_t ctas = (rows + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 0x7FFFFFFF) return cudaErrorNotSupported;
    norm_rope_any_kernel<kSrcBf16, kDstBf16>
        <<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  // 4 channels of f32 fill the 16 bytes of an access: 8 would make two half-filled ones of each (3900
  // tokens of 28 + 4 heads, bf16 to f32: 20.7 us with 4, 24.4 with 8)
  if constexpr (kSrcBf16 && kDstBf16)
    if (piece == 8) return launch_wide<kSrcBf16, kDstBf16, 8>(a, stream);
  return launch_wide<kSrcBf16, kDstBf16, 4>(a, stream);
}

bool activation_type(sa_dtype t) { return t == SA_DTYPE_F32 || t == SA_DTYPE_BF16; }

}  // namespace

}  // namespace sa

extern "C" sa_status sa_norm_rope(
    const void* q, const void* k, sa_dtype src_dtype, int64_t q_token_stride,
    int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride, const void* q_weight,
    const void* k_weight, sa_dtype weight_dtype, float eps, const float* inv_freq,
    int32_t rot_dim, const int32_t* freq_axes, int32_t interleaved, const int32_t* positions,
    int32_t n_axes, int64_t axis_stride, const int64_t* cu_seqlens_q_host,
    const int64_t* cu_seqlens_q, int32_t batch, const int32_t* used_kv_lens, int64_t tq,
    int32_t hq, int32_t hkv, int32_t head_dim, void* q_out, void* k_out, sa_dtype out_dtype,
    int64_t q_out_token_stride, int64_t q_out_head_stride, int64_t k_out_token_stride,
    int64_t k_out_head_stride, int64_t* status, void* stream) {
  if (hq < 0 || hkv < 0 || hq + static_cast<int64_t>(hkv) == 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0)
    return SA_ERR_HEAD_DIM;
  if (tq < 0) return SA_ERR_SHAPE;
  if (n_axes < 0) return SA_ERR_SHAPE;
  const bool by_lengths = rot_dim > 0 && n_axes == 0;
  if (by_lengths) {
    const sa_status st = sa::check_lengths(cu_seqlens_q_host, batch, tq);
    if (st != SA_OK) return st;
  }
  if (!sa::activation_type(src_dtype) || !sa::activation_type(out_dtype) ||
      !sa::activation_type(weight_dtype) || !(eps >= 0.f))
    return SA_ERR_INVALID_ARGUMENT;
  if (freq_axes != nullptr && n_axes == 0) return SA_ERR_INVALID_ARGUMENT;
  if (head_dim > 256) return SA_ERR_UNSUPPORTED;
  if (tq == 0) return SA_OK;
  if ((hq > 0 && (!q || !q_out)) || (hkv > 0 && (!k || !k_out)) || (rot_dim > 0 && !inv_freq) ||
      (rot_dim > 0 && n_axes > 0 && !positions) || (by_lengths && (!cu_seqlens_q || !used_kv_lens)))
    return SA_ERR_INVALID_ARGUMENT;
  // (with one token or one head its stride says nothing, and may be anything)
  if (tq == 1) q_token_stride = k_token_stride = q_out_token_stride = k_out_token_stride = 0;
  if (hq == 1) q_head_stride = q_out_head_stride = 0;
  if (hkv == 1) k_head_stride = k_out_head_stride = 0;
  if (sa::rows_overlap(tq, hq, head_dim, q_out_token_stride, q_out_head_stride) ||
      sa::rows_overlap(tq, hkv, head_dim, k_out_token_stride, k_out_head_stride))
    return SA_ERR_INVALID_ARGUMENT;

  sa::RopeArgs a{};
  a.src[0] = q;
  a.src[1] = k;
  a.dst[0] = q_out;
  a.dst[1] = k_out;
  a.token_stride[0] = q_token_stride;
  a.token_stride[1] = k_token_stride;
  a.head_stride[0] = q_head_stride;
  a.head_stride[1] = k_head_stride;
  a.dst_token_stride[0] = q_out_token_stride;
  a.dst_token_stride[1] = k_out_token_stride;
  a.dst_head_stride[0] = q_out_head_stride;
  a.dst_head_stride[1] = k_out_head_stride;
  a.weight[0] = hq > 0 ? q_weight : nullptr;
  a.weight[1] = hkv > 0 ? k_weight : nullptr;
  a.heads[0] = hq;
  a.heads[1] = hkv;
  a.weight_bf16 = weight_dtype == SA_DTYPE_BF16;
  a.eps = eps;
  a.inv_freq = inv_freq;
  a.freq_axes = freq_axes;
  a.positions = by_lengths ? nullptr : positions;
  a.axis_stride = axis_stride;
  a.n_axes = n_axes;
  a.cu = cu_seqlens_q;
  a.used = used_kv_lens;
  a.batch = batch;
  a.tq = tq;
  a.head_dim = head_dim;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.status = status;
  // loads and stores of pieces of 4 or 8 channels, at most 16 bytes: everything a multiple of them
  auto fits = [&](int c) {
    auto whole = [&](const void* p, sa_dtype type) {
      const uintptr_t bytes = c * (type == SA_DTYPE_BF16 ? 2 : 4);
      return (reinterpret_cast<uintptr_t>(p) & ((bytes < 16 ? bytes : 16) - 1)) == 0;
    };
    bool ok = head_dim % (2 * c) == 0 && rot_dim % (2 * c) == 0;
    for (int i = 0; i < 2; ++i)
      ok = ok && (a.heads[i] == 0 ||
                  (whole(a.src[i], src_dtype) && whole(a.dst[i], out_dtype) &&
                   ((a.token_stride[i] | a.head_stride[i] | a.dst_token_stride[i] | a.dst_head_stride[i]) &
                    (c - 1)) == 0));
    return ok;
  };
  const int piece = fits(8) ? 8 : fits(4) ? 4 : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (src_dtype == SA_DTYPE_BF16)
    err = out_dtype == SA_DTYPE_BF16 ? sa::launch_rope<true, true>(a, piece, s)
                                     : sa::launch_rope<true, false>(a, piece, s);
  else
    err = out_dtype == SA_DTYPE_BF16 ? sa::launch_rope<false, true>(a, piece, s)
                                     : sa::launch_rope<false, false>(a, piece, s);
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
