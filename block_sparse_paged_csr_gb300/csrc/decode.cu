// Entry point of the attention of one new token per sequence over its whole cache; the
// kernels are in decode_split.cuh.
#include <algorithm>
#include <cstdint>

#include "internal.h"

namespace sa {

namespace {

int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

// Bytes of the workspace's regions, each a multiple of 256.
struct Workspace {
  size_t firsts, parts, joins;
  size_t total() const { return firsts + parts + joins; }
};
Workspace decode_workspace(int qhead, int head_dim) {
  const int dp = padded_dim(std::min(head_dim, 256));
  // (the larger of what the two row counts need: f32 caches keep 8 rows)
  auto bytes = [&](int r) {
    return sizeof(float) * static_cast<size_t>(decode_max_warps(dp, r)) * decode_state_floats(dp, r);
  };
  const size_t state = sizeof(float) * decode_state_floats(dp, qhead <= 8 ? 8 : 16);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  return {up(kDecodeCtas * std::max(bytes(8), qhead <= 8 ? 0 : bytes(16))), up(kDecodeCtas * 2 * state),
          up(kDecodeCtas * sizeof(int2))};
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
  *bytes = sa::decode_workspace(hq / hkv, head_dim).total();
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
  // (row numbers of the pools are 32-bit, as are the tiles of 32 sequences)
  if (static_cast<int64_t>(batch) * hq > 0x7FFFFFFF ||
      static_cast<int64_t>(max_pages) * page_size > (int64_t{1} << 29) ||
      (num_pages > 0 && num_pages > int64_t{0xFFFFFFFE} / page_size / hkv))
    return SA_ERR_UNSUPPORTED;
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
  const int qhead = hq / hkv;
  // Query rows of a tile: 16 where a kv head has more than 8 q-heads (f32 caches keep 8: their
  // operands come in two parts each, which fill the rows), in several groups where that is
  // not enough.  Each group reads K and V (f32, 32 sequences of 20000 to 50000 keys: 8 q-heads a kv
  // head 1390 us, 16 2750).
  const int r = qhead <= 8 || kv_dtype == SA_DTYPE_F32 ? 8 : 16;
  const sa::Workspace ws = sa::decode_workspace(qhead, head_dim);
  unsigned char* base = static_cast<unsigned char*>(workspace);
  sa::DecodeArgs a{};
  a.q = q;
  // (copies of rows that are not there name the pools' start and read nothing: some address)
  a.k_pages = num_pages > 0 ? k_pages : workspace;
  a.v_pages = num_pages > 0 ? v_pages : workspace;
  a.k_scales = num_pages > 0 ? k_scales : static_cast<const float*>(workspace);
  a.v_scales = num_pages > 0 ? v_scales : static_cast<const float*>(workspace);
  a.num_pages = num_pages;
  a.block_tables = block_tables;
  a.used = used_kv_lens;
  a.batch = batch;
  a.hq = hq;
  a.hkv = hkv;
  a.qhead = qhead;
  a.groups = (qhead + r - 1) / r;
  a.items_per_seq = hkv * a.groups;
  a.head_dim = head_dim;
  a.row_bytes = head_dim * (kv_dtype == SA_DTYPE_F32 ? 4 : kv_dtype == SA_DTYPE_BF16 ? 2 : 1);
  a.page_size = page_size;
  a.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(page_size) : -1;
  a.max_pages = max_pages;
  a.capacity = max_pages * page_size;
  a.window = window;
  a.act_bf16 = q_dtype == SA_DTYPE_BF16;
  a.scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.firsts = reinterpret_cast<float*>(base);
  a.parts = reinterpret_cast<float*>(base + ws.firsts);
  a.joins = reinterpret_cast<int2*>(base + ws.firsts + ws.parts);
  const int dp = sa::padded_dim(head_dim);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (kv_dtype) {
    case SA_DTYPE_F32: err = sa::launch_decode_f32(a, dp, r, s); break;
    case SA_DTYPE_BF16: err = sa::launch_decode_bf16(a, dp, r, s); break;
    case SA_DTYPE_E4M3: err = sa::launch_decode_e4m3(a, dp, r, s); break;
    default: err = sa::launch_decode_int8(a, dp, r, s); break;
  }
  return err == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
