// Reading rows of the paged K/V cache back: the rows that a store with the same
// lengths writes, as f32 or bf16 (value = code * scale of the page and kv head).
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "seq_common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

enum CacheType { kF32 = 0, kBf16 = 1, kE4m3 = 2, kInt8 = 3 };

struct LoadArgs {
  void* dst[2];                        // K, V rows
  int64_t token_stride[2], head_stride[2];   // elements
  const void* pages[2];
  const float* scales[2];
  int64_t num_pages;
  const int32_t* block_tables;
  const int64_t* cu;
  const int32_t* used;
  int64_t tq, slots;
  int32_t batch, hkv, head_dim, page_size, max_pages;
  int32_t part_rows, items_per_slot;   // a warp's rows of a page; warps of a page
  int64_t* status;
};

// A piece: 16 bytes of the output row, which is what a lane handles at a time, so
// that a warp's stores fill whole lines whatever the cache's type.
template <bool kDstBf16> struct Out { static constexpr int n = kDstBf16 ? 8 : 4; };

// The n cached elements of one piece as they lie (raw), and as values.
template <int kType, int kN>
struct Raw {
  static constexpr int bytes = kN * (kType == kF32 ? 4 : kType == kBf16 ? 2 : 1);
  uint32_t w[bytes / 4];
  __device__ __forceinline__ void load(const void* p, int64_t elem) {
    const unsigned char* at =
        static_cast<const unsigned char*>(p) + elem * (kType == kF32 ? 4 : kType == kBf16 ? 2 : 1);
    if constexpr (bytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    } else if constexpr (bytes == 8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(at));
      w[0] = u.x;
      w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < bytes / 16; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(at) + i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < bytes / 4; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void values(float scale, float (&x)[kN]) const {
    if constexpr (kType == kF32) {
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = __uint_as_float(w[i]);
    } else if constexpr (kType == kBf16) {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        uint32_t lo, hi;
        codes4_to_f16<kType == kInt8>(w[i], lo, hi);
        const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
        x[4 * i] = a.x * scale;
        x[4 * i + 1] = a.y * scale;
        x[4 * i + 2] = b.x * scale;
        x[4 * i + 3] = b.y * scale;
      }
    }
  }
};

// One warp per (part of a page of a sequence, kv head, K or V): its rows lie side by side
// in the page and go to rows of the output.  kBatch pieces a lane in flight.
//
// Bound by memory: 105000 rows of 8 heads of 128 from e4m3 to bf16 (664 MB) take 103 us, 6.5 TB/s;
// 7000 rows of 4 heads of 256 from bf16 to f32 (91 MB) 18.5 us.  A part of 4096 elements
// is the best of both ends: whole pages of 64 x 128 and 32 x 256 took 105 and 26 us (few
// warps), parts of 2048 112 and 19 us, of 1024 172 and 18 us (lookups); 4 pieces in flight
// 104 and 21 us.
template <int kType, bool kDstBf16>
__global__ void __launch_bounds__(kThreads) load_kv_kernel(const LoadArgs a) {
  constexpr int kN = Out<kDstBf16>::n;
  constexpr int kBatch = 8;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t u = item / a.items_per_slot;
  const int rest = static_cast<int>(item - u * a.items_per_slot);
  const int part = rest / (2 * a.hkv), hv = rest - part * (2 * a.hkv);
  const int h = hv >> 1;
  const int kv = hv & 1;
  if (u >= a.slots) return;
  const int b = warp_slot_sequence(a.cu, a.batch, a.page_size, u, lane);
  const NewRange nr = new_range(a.cu, a.used, b, a.tq);
  const int64_t p1 = nr.p0 + (min(max(a.cu[b + 1], nr.cu0), a.tq) - nr.cu0);   // end of the rows asked for
  const int64_t page0 = nr.p0 / a.page_size;
  const int64_t pg = page0 + (u - slot_base(a.cu[b], b, a.page_size));
  const int64_t base = pg * a.page_size;
  if (nr.p0 >= p1 || pg < page0 || base >= p1) return;
  int id = pg < a.max_pages ? a.block_tables[static_cast<int64_t>(b) * a.max_pages + pg] : -1;
  if (id >= a.num_pages) {
    if (lane == 0) report(a.status, SA_ERR_SHAPE);
    id = -1;
  }
  // the part's rows of the page that are asked for
  const int64_t part0 = static_cast<int64_t>(part) * a.part_rows;
  const int r0 = static_cast<int>(max(nr.p0 - base, part0));
  const int r1 = static_cast<int>(min(min(p1 - base, static_cast<int64_t>(a.page_size)), part0 + a.part_rows));
  if (r0 >= r1) return;
  // rows that the cache holds (the others become 0)
  const int held = id < 0 ? 0 : static_cast<int>(min(max(nr.p1 - (base + r0), int64_t{0}),
                                                     static_cast<int64_t>(r1 - r0)));
  const int per_row = a.head_dim / kN;
  const int n = (r1 - r0) * per_row, n_held = held * per_row;
  const int64_t tok0 = nr.cu0 + (base + r0 - nr.p0);
  const int64_t src0 =
      ((static_cast<int64_t>(max(id, 0)) * a.hkv + h) * a.page_size + r0) * a.head_dim;
  const void* src = a.pages[kv];
  float scale = 1.f;
  if constexpr (kType == kE4m3 || kType == kInt8)
    scale = id >= 0 ? __ldg(a.scales[kv] + static_cast<int64_t>(id) * a.hkv + h) : 0.f;
  void* dst = a.dst[kv];
  const int64_t ts = a.token_stride[kv];
  const int64_t dst0 = tok0 * ts + h * a.head_stride[kv];
  // the lane's piece: row r and piece c of it, without a division per piece
  const int step_r = 32 / per_row, step_c = 32 - step_r * per_row;
  int r = lane / per_row, c = lane - r * per_row;
  for (int i0 = lane; i0 < n; i0 += 32 * kBatch) {
    Raw<kType, kN> raw[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 32 * j;
      if (i < n_held)
        raw[j].load(src, src0 + static_cast<int64_t>(i) * kN);
      else
        raw[j].zero();
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + 32 * j < n) {
        float x[kN];
        raw[j].values(i0 + 32 * j < n_held ? scale : 0.f, x);
        const int64_t at = dst0 + r * ts + c * kN;
        if constexpr (kDstBf16)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + at) =
              make_uint4(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]),
                         pack_bf16x2_rn(x[4], x[5]), pack_bf16x2_rn(x[6], x[7]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(dst) + at) =
              make_float4(x[0], x[1], x[2], x[3]);
      }
      r += step_r;
      c += step_c;
      if (c >= per_row) {
        c -= per_row;
        ++r;
      }
    }
  }
}

template <int kType>
cudaError_t launch_load(const LoadArgs& a, bool dst_bf16, cudaStream_t stream) {
  const int64_t ctas = (a.slots * a.items_per_slot + kWarps - 1) / kWarps;
  if (ctas > 0x7FFFFFFF) return cudaErrorNotSupported;
  if (dst_bf16)
    load_kv_kernel<kType, true><<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(a);
  else
    load_kv_kernel<kType, false><<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

}  // namespace sa

extern "C" sa_status sa_load_kv(const void* k_pages, const void* v_pages, const float* k_scales,
                                const float* v_scales, int64_t num_pages, sa_dtype kv_dtype,
                                const int32_t* block_tables, int32_t max_pages,
                                const int64_t* cu_seqlens_host, const int64_t* cu_seqlens,
                                int32_t batch, int64_t tq, const int32_t* used_kv_lens,
                                int32_t hkv, int32_t head_dim, int32_t page_size, void* k, void* v,
                                sa_dtype dst_dtype, int64_t k_token_stride, int64_t k_head_stride,
                                int64_t v_token_stride, int64_t v_head_stride, int64_t* status,
                                void* stream) {
  if (hkv <= 0) return SA_ERR_HEAD_COUNT;
  if (head_dim <= 0 || page_size <= 0) return SA_ERR_BLOCK_PAGE;
  const sa_status st = sa::check_lengths(cu_seqlens_host, batch, tq);
  if (st != SA_OK) return st;
  if (num_pages < 0 || max_pages < 0) return SA_ERR_SHAPE;
  if (dst_dtype != SA_DTYPE_F32 && dst_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
  if (kv_dtype < SA_DTYPE_F32 || kv_dtype > SA_DTYPE_INT8) return SA_ERR_INVALID_ARGUMENT;
  if (head_dim % (sa::eight_bit(kv_dtype) ? 16 : 8) != 0 || head_dim > 256)
    return SA_ERR_UNSUPPORTED;
  if (tq == 0) return SA_OK;
  if (!k || !v || !k_pages || !v_pages || !block_tables || !cu_seqlens || !used_kv_lens)
    return SA_ERR_INVALID_ARGUMENT;
  if (sa::eight_bit(kv_dtype) && (!k_scales || !v_scales)) return SA_ERR_INVALID_ARGUMENT;
  if (!sa::aligned16(k) || !sa::aligned16(v) || !sa::aligned16(k_pages) || !sa::aligned16(v_pages))
    return SA_ERR_INVALID_ARGUMENT;
  // (with one token or one head its stride says nothing, and may be anything)
  if (tq == 1) k_token_stride = v_token_stride = 0;
  if (hkv == 1) k_head_stride = v_head_stride = 0;
  const int64_t unit = dst_dtype == SA_DTYPE_BF16 ? 8 : 4;      // elements of 16 bytes
  if (k_token_stride % unit || k_head_stride % unit || v_token_stride % unit ||
      v_head_stride % unit)
    return SA_ERR_INVALID_ARGUMENT;
  if (sa::rows_overlap(tq, hkv, head_dim, k_token_stride, k_head_stride) ||
      sa::rows_overlap(tq, hkv, head_dim, v_token_stride, v_head_stride))
    return SA_ERR_INVALID_ARGUMENT;

  sa::LoadArgs a{};
  a.dst[0] = k;
  a.dst[1] = v;
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
  a.cu = cu_seqlens;
  a.used = used_kv_lens;
  a.tq = tq;
  a.slots = sa::slot_base(tq, batch, page_size);
  a.batch = batch;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.part_rows = std::max(4096 / head_dim, 1);
  const int64_t items = static_cast<int64_t>((page_size - 1) / a.part_rows + 1) * hkv * 2;
  if (items > 0x7FFFFFFF) return SA_ERR_UNSUPPORTED;
  a.items_per_slot = static_cast<int32_t>(items);
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = dst_dtype == SA_DTYPE_BF16;
  cudaError_t err;
  switch (kv_dtype) {
    case SA_DTYPE_F32: err = sa::launch_load<sa::kF32>(a, bf, s); break;
    case SA_DTYPE_BF16: err = sa::launch_load<sa::kBf16>(a, bf, s); break;
    case SA_DTYPE_E4M3: err = sa::launch_load<sa::kE4m3>(a, bf, s); break;
    default: err = sa::launch_load<sa::kInt8>(a, bf, s); break;
  }
  if (err == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
