// Head norms and position rotation of queries and keys in one pass.
//
// Per (token, head) row x of d channels: y = x / sqrt(mean(x^2) + eps) * w (y = x
// without a weight), then pair i of the first rot channels turns by the angle
// p f_i, p the token's position on the pair's axis: (a, b) -> (a cos - b sin,
// a sin + b cos).  The pairs are (i, i + rot / 2), or (2 i, 2 i + 1).
//
// Angles: f32 products p f lose the angle (p = 131072 leaves 2^-7 radians), so
// f / (2 pi) is taken as a 64-bit fraction of a turn.  Its product with the integer p
// wraps at whole turns by itself; the error is |p| 2^-64 turns, and the upper 32 bits
// of the product go to sincospif.
#include <cstdint>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;                 // tokens per CTA

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
// 2^(e - 150) and C = 2^66 / (2 pi): M C 2^(e - 152), formed as the upper half of
// (M 2^40) C, shifted by e - 128.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>((u >> 23) & 0xFFu);
  const uint64_t m = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const uint64_t hi = __umul64hi(m << 40, 0xA2F9836E4E44152Aull);
  const int s = (e ? e : 1) - 128;
  const uint64_t v = s <= -64 || s >= 64 ? 0ull : s < 0 ? hi >> -s : hi << s;
  return (u >> 31) ? 0ull - v : v;
}

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int pos) {
  const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const int half_turns = static_cast<int>(static_cast<int64_t>(t) >> 32);
  float2 r;
  sincospif(__int2float_rn(half_turns) * 0x1p-31f, &r.y, &r.x);
  return r;
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

// Four channels as they lie, and as values.
template <bool kBf16> struct Raw4;
template <> struct Raw4<true> {
  uint2 u;
  __device__ __forceinline__ void load(const void* p, int64_t off) {
    u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + off);
  }
  __device__ __forceinline__ void zero() { u = make_uint2(0u, 0u); }
  __device__ __forceinline__ float4 values() const { return bf16x4_to_f32(u); }
};
template <> struct Raw4<false> {
  float4 u;
  __device__ __forceinline__ void load(const void* p, int64_t off) {
    u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + off);
  }
  __device__ __forceinline__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float4 values() const { return u; }
};

// A row is spread over kLanes lanes, a lane holding 8 channels in two pieces of 4 that
// hold whole pairs: channels 4 u and rot / 2 + 4 u on (or 8 u on, where pairs are
// adjacent), so that the rotation needs no other lane.  Either way the pieces' pairs are
// 4 u .. 4 u + 3.  A group of kLanes lanes keeps one token and walks over its heads, kRows of them
// at a time, all asked for before the first is used: angles are made once per
// token and pair, by the CTA, and stay in registers, as the weights do.
template <bool kSrcBf16, bool kDstBf16, int kLanes>
__global__ void __launch_bounds__(kThreads, 3)
norm_rope_kernel(const RopeArgs a, int log_tokens, int heads_per_cta) {
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kRows = 3;
  __shared__ int s_pos[kMaxTokens];
  __shared__ __align__(16) float2 s_turn[kMaxTokens * 128];
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
  const int rot_units = a.rot >> 3;
  const bool rotated = u < rot_units;
  const int ca = rotated ? (a.interleaved ? 8 * u : 4 * u) : 8 * u;
  const int cb = rotated && !a.interleaved ? n_pairs + 4 * u : ca + 4;
  const bool mine = 8 * u < a.head_dim;
  const bool live = tok < a.tq;

  Raw4<kSrcBf16> xa[kRows], xb[kRows];
  auto load_rows = [&]() {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int h = head + i * step;
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
  load_rows();
  float4 w[2][2];                                      // of q and k: both pieces
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    w[k][0] = w[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.weight[k] != nullptr && mine) {
      if (a.weight_bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(a.weight[k]);
        w[k][0] = bf16x4_to_f32(*reinterpret_cast<const uint2*>(p + ca));
        w[k][1] = bf16x4_to_f32(*reinterpret_cast<const uint2*>(p + cb));
      } else {
        const float* p = static_cast<const float*>(a.weight[k]);
        w[k][0] = *reinterpret_cast<const float4*>(p + ca);
        w[k][1] = *reinterpret_cast<const float4*>(p + cb);
      }
    }
  }

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
        s_turn[i] = cos_sin(turn_fraction(a.inv_freq[pair]), p);
      }
    }
    __syncthreads();
  }
  if (!live) return;
  float co[4], si[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    float4 t = make_float4(1.f, 0.f, 1.f, 0.f);
    if (rotated)
      t = *reinterpret_cast<const float4*>(s_turn + (group & (tokens - 1)) * n_pairs + 4 * u + j);
    co[j] = t.x;
    si[j] = t.y;
    co[j + 1] = t.z;
    si[j + 1] = t.w;
  }
  const unsigned mask = kLanes == 32 ? 0xffffffffu
                                     : ((1u << (kLanes & 31)) - 1u) << ((lane / kLanes) * kLanes);
  for (; head < end; head += kRows * step) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int h = head + i * step;
      if (h >= end) break;
      const int kind = h >= a.heads[0] ? 1 : 0;
      const float4 p4 = xa[i].values(), q4 = xb[i].values();
      float x[8] = {p4.x, p4.y, p4.z, p4.w, q4.x, q4.y, q4.z, q4.w};
      // (the same for all lanes of a group, and a group's lanes lie in one warp)
      if (a.weight[kind] != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) ss = fmaf(x[c], x[c], ss);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float r = rsqrtf(ss / static_cast<float>(a.head_dim) + a.eps);
        const float4 wa = kind ? w[1][0] : w[0][0], wb = kind ? w[1][1] : w[0][1];
        const float ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = x[c] * r * ww[c];
      }
      if (rotated) {
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = x[2 * j], q = x[2 * j + 1];
            x[2 * j] = p * co[j] - q * si[j];
            x[2 * j + 1] = p * si[j] + q * co[j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = x[j], q = x[4 + j];
            x[j] = p * co[j] - q * si[j];
            x[4 + j] = p * si[j] + q * co[j];
          }
        }
      }
      if (mine) {
        const int64_t at =
            tok * a.dst_token_stride[kind] +
            static_cast<int64_t>(h - (kind ? a.heads[0] : 0)) * a.dst_head_stride[kind];
        store_o4(a.dst[kind], kDstBf16, at + ca, make_float4(x[0], x[1], x[2], x[3]));
        store_o4(a.dst[kind], kDstBf16, at + cb, make_float4(x[4], x[5], x[6], x[7]));
      }
    }
    if (head + kRows * step < end) {
      head += kRows * step;
      load_rows();
      head -= kRows * step;
    }
  }
}

// Any sizes, strides and alignment: a warp per row, a lane per pair (and per
// channel behind the rotated ones), angles made where they are used (8192 tokens of 64 + 8
// heads in f32 whose rows start off 16 bytes: 411 us, the other kernel 100).
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

template <bool kSrcBf16, bool kDstBf16>
cudaError_t launch_rope(const RopeArgs& a, bool wide, cudaStream_t stream) {
  const int total = a.heads[0] + a.heads[1];
  if (!wide) {
    const int64_t ctas = (a.tq * total + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 0x7FFFFFFF) return cudaErrorNotSupported;
    norm_rope_any_kernel<kSrcBf16, kDstBf16>
        <<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const int units = a.head_dim / 8;
  const int lanes = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
  const int groups = kThreads / lanes;
  // Prompts: four tokens a CTA, whose groups walk over the heads in `turns` turns of kRows.  Few
  // tokens: one, and its heads over several CTAs, so that a row is all that a group does.  A turn
  // takes about half as long as a round of CTAs: 32 + 8 heads of 128 in bf16, four tokens / one token
  // a CTA: 64 tokens (4 turns, 1 round) 7.4 / 3.5 us, 256 (2 rounds) 7.7 / 6.2, 400 (3 rounds) 7.6 /
  // 8.1, 2000 19.7 / 31.8; 8 + 1 heads (1 turn): 500 tokens (2 rounds) 4.2 / 5.8.
  const int64_t slots = 3ll * device_sm_count();
  const int64_t rounds = (a.tq * ((total + groups - 1) / groups) + slots - 1) / slots;
  const int64_t turns = (4ll * total + 3 * groups - 1) / (3 * groups);
  const bool few = 2 * rounds <= turns + 1;
  const int log_tokens = few ? 0 : 2;
  const int heads_per_cta = few ? groups : total;
  const int64_t gx = (a.tq + (int64_t{1} << log_tokens) - 1) >> log_tokens;
  const int64_t gy = (total + heads_per_cta - 1) / heads_per_cta;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a, log_tokens, heads_per_cta); };
  if (lanes == 4)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, 4>);
  else if (lanes == 8)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, 8>);
  else if (lanes == 16)
    go(norm_rope_kernel<kSrcBf16, kDstBf16, 16>);
  else
    go(norm_rope_kernel<kSrcBf16, kDstBf16, 32>);
  return cudaGetLastError();
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
  // loads and stores of 4-channel pieces (8 or 16 bytes): everything a multiple of them
  auto whole = [](const void* p, sa_dtype type) {
    return (reinterpret_cast<uintptr_t>(p) & (type == SA_DTYPE_BF16 ? 7u : 15u)) == 0;
  };
  bool wide = head_dim % 8 == 0 && rot_dim % 8 == 0;
  for (int i = 0; i < 2; ++i) {
    if (a.heads[i] == 0) continue;
    wide = wide && whole(a.src[i], src_dtype) && whole(a.dst[i], out_dtype) &&
           whole(a.weight[i], weight_dtype) &&
           ((a.token_stride[i] | a.head_stride[i] | a.dst_token_stride[i] | a.dst_head_stride[i]) & 3) == 0;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (src_dtype == SA_DTYPE_BF16)
    err = out_dtype == SA_DTYPE_BF16 ? sa::launch_rope<true, true>(a, wide, s)
                                     : sa::launch_rope<true, false>(a, wide, s);
  else
    err = out_dtype == SA_DTYPE_BF16 ? sa::launch_rope<false, true>(a, wide, s)
                                     : sa::launch_rope<false, false>(a, wide, s);
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
