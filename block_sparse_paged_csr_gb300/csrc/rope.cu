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
constexpr int kMaxTokens = 8;                 // tokens per CTA

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

template <bool kBf16>
__device__ __forceinline__ void load8f(const void* p, int64_t off, float* x) {
  if constexpr (kBf16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + off);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(p) + off);
    const float4 l = v[0], h = v[1];
    x[0] = l.x; x[1] = l.y; x[2] = l.z; x[3] = l.w;
    x[4] = h.x; x[5] = h.y; x[6] = h.z; x[7] = h.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store8f(void* p, int64_t off, const float* x) {
  if constexpr (kBf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off) =
        make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]),
                   pack_bf16x2_rn(x[4], x[5]), pack_bf16x2_rn(x[6], x[7]));
  } else {
    float4* v = reinterpret_cast<float4*>(static_cast<float*>(p) + off);
    v[0] = make_float4(x[0], x[1], x[2], x[3]);
    v[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// A row is spread over kLanes lanes, a lane holding 16 channels in two pieces of 8
// that hold whole pairs: channels 8 u and rot / 2 + 8 u on (or 16 u on, where pairs
// are adjacent), so that the rotation needs no other lane.  Either way the pieces'
// pairs are 8 u .. 8 u + 7.  A group of kLanes lanes keeps one token and walks over
// its heads: angles are made once per token and pair, by the CTA, and stay in
// registers, as the weights do.
template <bool kSrcBf16, bool kDstBf16, int kLanes>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const RopeArgs a, int log_tokens, int heads_per_cta) {
  constexpr int kGroups = kThreads / kLanes;
  __shared__ int s_pos[kMaxTokens];
  __shared__ float2 s_turn[kMaxTokens * 128];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tokens = 1 << log_tokens;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) << log_tokens;
  const int n_pairs = a.rot >> 1;
  const int group = tid / kLanes, u = tid % kLanes;
  const int64_t tok = tok0 + (group & (tokens - 1));
  const int step = kGroups >> log_tokens;              // heads between a group's rows
  const int head0 = static_cast<int>(blockIdx.y) * heads_per_cta + (group >> log_tokens);
  const int total = a.heads[0] + a.heads[1];
  const int end = min(total, static_cast<int>(blockIdx.y + 1) * heads_per_cta);
  const int rot_units = a.rot >> 4;
  const bool rotated = u < rot_units;
  const int ca = rotated ? (a.interleaved ? 16 * u : 8 * u) : a.rot + 16 * (u - rot_units);
  const int cb = rotated && !a.interleaved ? n_pairs + 8 * u : ca + 8;
  const bool has_a = ca < a.head_dim, has_b = has_a && cb < a.head_dim;

  float x[16];
  auto load_row = [&](int h, float (&v)[16]) {
    const int kind = h >= a.heads[0] ? 1 : 0;
    const int64_t at = tok * a.token_stride[kind] +
                       static_cast<int64_t>(h - (kind ? a.heads[0] : 0)) * a.head_stride[kind];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    if (has_a) load8f<kSrcBf16>(a.src[kind], at + ca, v);
    if (has_b) load8f<kSrcBf16>(a.src[kind], at + cb, v + 8);
  };
  const bool live = tok < a.tq;
  if (live && head0 < end) load_row(head0, x);

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
  float co[8], si[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    co[j] = 1.f;
    si[j] = 0.f;
    if (rotated) {
      const float2 t = s_turn[(group & (tokens - 1)) * n_pairs + 8 * u + j];
      co[j] = t.x;
      si[j] = t.y;
    }
  }
  float w[16];
  int have = -1;                                       // whose weights w holds
  for (int h = head0; h < end; h += step) {
    float next[16];
    if (h + step < end) load_row(h + step, next);
    const int kind = h >= a.heads[0] ? 1 : 0;
    // (the same for all lanes of a group, and a group's lanes lie in one warp)
    if (a.weight[kind] != nullptr) {
      if (have != kind) {
        have = kind;
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 0.f;
        if (a.weight_bf16) {
          if (has_a) load8f<true>(a.weight[kind], ca, w);
          if (has_b) load8f<true>(a.weight[kind], cb, w + 8);
        } else {
          if (has_a) load8f<false>(a.weight[kind], ca, w);
          if (has_b) load8f<false>(a.weight[kind], cb, w + 8);
        }
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      const unsigned mask = kLanes == 32 ? 0xffffffffu
                                         : ((1u << kLanes) - 1u) << ((lane / kLanes) * kLanes);
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float r = rsqrtf(ss / static_cast<float>(a.head_dim) + a.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
    }
    if (rotated) {
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = x[2 * j], q = x[2 * j + 1];
          x[2 * j] = p * co[j] - q * si[j];
          x[2 * j + 1] = p * si[j] + q * co[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = x[j], q = x[8 + j];
          x[j] = p * co[j] - q * si[j];
          x[8 + j] = p * si[j] + q * co[j];
        }
      }
    }
    const int64_t at = tok * a.dst_token_stride[kind] +
                       static_cast<int64_t>(h - (kind ? a.heads[0] : 0)) * a.dst_head_stride[kind];
    if (has_a) store8f<kDstBf16>(a.dst[kind], at + ca, x);
    if (has_b) store8f<kDstBf16>(a.dst[kind], at + cb, x + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = next[i];
  }
}

// Any sizes, strides and alignment: a warp per row, a lane per pair (and per
// channel behind the rotated ones), angles made where they are used.
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
  const int units = (a.head_dim + 15) / 16;
  const int lanes = units <= 4 ? 4 : units <= 8 ? 8 : 16;
  const int groups = kThreads / lanes;
  // Prompts: four tokens a CTA.  Few tokens: one, and its heads over several CTAs,
  // so that a row is all that a group does.
  const int64_t sms = device_sm_count();
  const bool few = a.tq * total <= 4 * sms * groups;
  const int log_tokens = few ? 0 : 2;
  const int heads_per_cta = few ? groups : total;
  const int64_t gx = (a.tq + (int64_t{1} << log_tokens) - 1) >> log_tokens;
  const int64_t gy = (total + heads_per_cta - 1) / heads_per_cta;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (lanes == 4)
    norm_rope_kernel<kSrcBf16, kDstBf16, 4>
        <<<grid, kThreads, 0, stream>>>(a, log_tokens, heads_per_cta);
  else if (lanes == 8)
    norm_rope_kernel<kSrcBf16, kDstBf16, 8>
        <<<grid, kThreads, 0, stream>>>(a, log_tokens, heads_per_cta);
  else
    norm_rope_kernel<kSrcBf16, kDstBf16, 16>
        <<<grid, kThreads, 0, stream>>>(a, log_tokens, heads_per_cta);
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
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
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
  // 16-byte loads and stores of 8-channel pieces: everything a multiple of them
  const int64_t src_unit = src_dtype == SA_DTYPE_BF16 ? 8 : 4;
  const int64_t dst_unit = out_dtype == SA_DTYPE_BF16 ? 8 : 4;
  bool wide = head_dim % 8 == 0 && rot_dim % 16 == 0;
  for (int i = 0; i < 2; ++i) {
    if (a.heads[i] == 0) continue;
    wide = wide && sa::aligned16(a.src[i]) && sa::aligned16(a.dst[i]) &&
           (a.weight[i] == nullptr || sa::aligned16(a.weight[i])) &&
           a.token_stride[i] % src_unit == 0 && a.head_stride[i] % src_unit == 0 &&
           a.dst_token_stride[i] % dst_unit == 0 && a.dst_head_stride[i] % dst_unit == 0;
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
