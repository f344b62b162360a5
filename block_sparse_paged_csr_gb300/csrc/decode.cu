// Attention of one new token per sequence over its whole paged cache (or the last
// `window` keys of it).
#include <cstdint>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct DecodeArgs {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const float* k_scales;
  const float* v_scales;
  int64_t num_pages;
  const int32_t* block_tables;
  const int32_t* used;
  int32_t batch, hq, hkv, qhead, head_dim, page_size, max_pages, window, q_bf16, kv_type;
  float scale;
  void* out;
  float* lse;
  int64_t* status;
};

__device__ __forceinline__ float cached(const void* p, int64_t at, int type) {
  if (type == SA_DTYPE_F32) return static_cast<const float*>(p)[at];
  if (type == SA_DTYPE_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
  const uint32_t w = static_cast<const uint8_t*>(p)[at];
  uint32_t lo, hi;
  if (type == SA_DTYPE_INT8)
    codes4_to_f16<true>(w, lo, hi);
  else
    codes4_to_f16<false>(w, lo, hi);
  return f16x2_to_f32(lo).x;
}

// A CTA per (sequence, q-head): a key per warp at a time, a lane holding channels
// lane, lane + 32, ..; the warps' states meet in shared memory.
__global__ void __launch_bounds__(kThreads) decode_attention_kernel(const DecodeArgs a) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / a.hq);
  const int h = static_cast<int>(row - static_cast<int64_t>(b) * a.hq) / a.qhead;
  const int64_t lk = min(static_cast<int64_t>(max(a.used[b], 0)),
                         static_cast<int64_t>(a.max_pages) * a.page_size);
  const int64_t first = a.window > 0 ? max(static_cast<int64_t>(a.used[b]) - a.window, int64_t{0}) : 0;
  const bool eight = a.kv_type == SA_DTYPE_E4M3 || a.kv_type == SA_DTYPE_INT8;
  float q[8], o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = lane + 32 * i;
    o[i] = 0.f;
    q[i] = c >= a.head_dim ? 0.f
           : a.q_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.q)[row * a.head_dim + c])
                      : static_cast<const float*>(a.q)[row * a.head_dim + c];
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t key = first + warp; key < lk; key += kWarps) {
    const int64_t pg = key / a.page_size;
    const int id = a.block_tables[static_cast<int64_t>(b) * a.max_pages + pg];
    if (id >= a.num_pages && lane == 0) report(a.status, SA_ERR_SHAPE);
    if (id < 0 || id >= a.num_pages) continue;
    const int64_t at =
        ((static_cast<int64_t>(id) * a.hkv + h) * a.page_size + (key - pg * a.page_size)) *
        a.head_dim;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.head_dim)
        s = fmaf(q[i], cached(a.k_pages, at + lane + 32 * i, a.kv_type), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    float vs = 1.f;
    if (eight) {
      s *= a.k_scales[static_cast<int64_t>(id) * a.hkv + h];
      vs = a.v_scales[static_cast<int64_t>(id) * a.hkv + h];
    }
    const float top = fmaxf(m, s);
    const float e = m == top ? 1.f : expf(m - top), p = expf(s - top);
    m = top;
    l = l * e + p;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.head_dim)
        o[i] = o[i] * e + p * vs * cached(a.v_pages, at + lane + 32 * i, a.kv_type);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s_o[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  const int c = threadIdx.x;
  for (int w = 0; w < kWarps; ++w) {
    const float e = s_l[w] == 0.f ? 0.f : expf(s_m[w] - top);
    sum += e * s_l[w];
    acc += e * s_o[w][c];
  }
  if (c < a.head_dim) {
    const float y = sum == 0.f ? 0.f : acc / sum;
    if (a.q_bf16)
      static_cast<uint16_t*>(a.out)[row * a.head_dim + c] =
          static_cast<uint16_t>(pack_bf16x2_rn(y, 0.f) & 0xFFFFu);
    else
      static_cast<float*>(a.out)[row * a.head_dim + c] = y;
  }
  if (c == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

}  // namespace sa

extern "C" {

sa_status sa_decode_workspace_size(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim,
                                   size_t* bytes) {
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0) return SA_ERR_HEAD_DIM;
  if (batch < 0) return SA_ERR_SHAPE;
  if (bytes == nullptr) return SA_ERR_INVALID_ARGUMENT;
  *bytes = 16;
  return SA_OK;
}

sa_status sa_decode_attention(const void* q, sa_dtype q_dtype, const void* k_pages,
                              const void* v_pages, const float* k_scales, const float* v_scales,
                              int64_t num_pages, sa_dtype kv_dtype, const int32_t* block_tables,
                              int32_t max_pages, const int32_t* used_kv_lens, int32_t batch,
                              int32_t hq, int32_t hkv, int32_t head_dim, int32_t page_size,
                              float softmax_scale, int32_t window, void* out, float* lse,
                              void* workspace, size_t workspace_bytes, int64_t* status,
                              void* stream) {
  size_t need = 0;
  const sa_status st = sa_decode_workspace_size(batch, hq, hkv, head_dim, &need);
  if (st != SA_OK) return st;
  if (page_size <= 0) return SA_ERR_BLOCK_PAGE;
  if (num_pages < 0 || max_pages < 0 || window < 0) return SA_ERR_SHAPE;
  if (q_dtype != SA_DTYPE_F32 && q_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
  if (kv_dtype < SA_DTYPE_F32 || kv_dtype > SA_DTYPE_INT8) return SA_ERR_INVALID_ARGUMENT;
  if (head_dim % (sa::eight_bit(kv_dtype) ? 16 : 8) != 0 || head_dim > 256)
    return SA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * hq > 0x7FFFFFFF) return SA_ERR_UNSUPPORTED;
  if (batch == 0) return SA_OK;
  // (a cache without pages or columns may have no memory either)
  if (!q || !out || !used_kv_lens || !workspace || (max_pages > 0 && !block_tables) ||
      (num_pages > 0 && (!k_pages || !v_pages)))
    return SA_ERR_INVALID_ARGUMENT;
  if (sa::eight_bit(kv_dtype) && num_pages > 0 && (!k_scales || !v_scales))
    return SA_ERR_INVALID_ARGUMENT;
  if (!sa::aligned16(q) || !sa::aligned16(out) || !sa::aligned16(k_pages) ||
      !sa::aligned16(v_pages) || !sa::aligned16(workspace) || workspace_bytes < need)
    return SA_ERR_INVALID_ARGUMENT;
  sa::DecodeArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.num_pages = num_pages;
  a.block_tables = block_tables;
  a.used = used_kv_lens;
  a.batch = batch;
  a.hq = hq;
  a.hkv = hkv;
  a.qhead = hq / hkv;
  a.head_dim = head_dim;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.window = window;
  a.q_bf16 = q_dtype == SA_DTYPE_BF16;
  a.kv_type = kv_dtype;
  a.scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  a.status = status;
  sa::decode_attention_kernel<<<static_cast<unsigned>(batch * hq), sa::kThreads, 0,
                                static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
