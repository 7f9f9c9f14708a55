// Host side of msa_cache_append: argument validation (all of it before any HIP
// call) and one launch on the caller's stream.
#include "msa_index_score.h"

#include <algorithm>
#include <cstdint>

#include "msa_append.hpp"
#include "msa_host.hpp"

namespace {

using msa::AppendItem;
using msa::AppendParams;

static_assert(msa::kAppendItems == MSA_APPEND_MAX_ITEMS && msa::kLayoutRows == MSA_LAYOUT_ROWS,
              "the kernel's constants are the header's");

// Waves per token: as few as keep 8192 waves (the chip holds half as many at
// once) and 16 steps a wave.  A wave begins with three dependent reads (its
// request, its page and angles, its rows), so long runs pay: 14000 tokens of
// 23 steps take 140 us in runs of 12, 145 in runs of 8 and 200 in runs of 2;
// 4096 tokens of 15 steps 35 us in runs of 8, 57 in single steps.
int groups_for(int64_t T, int steps) {
  const int64_t g = std::max<int64_t>((steps + 15) / 16, (8192 + T - 1) / T);
  return (int)std::min<int64_t>(g, steps);
}

msa_status_t item_for(const msa_append_item_t& in, int64_t T, AppendItem& a) {
  const msa_tensor_t& src = in.src;
  const msa_tensor_t& dst = in.dst;
  if (in.layout < MSA_LAYOUT_TND || in.layout > MSA_LAYOUT_ROWS) return MSA_ERR_LAYOUT;
  if (in.rotate != 0 && in.rotate != 1) return MSA_ERR_ATTR;
  const int eb = msa::elem_bytes(dst.dtype);
  if (eb == 0 || (eb == 2 && dst.dtype != src.dtype)) return MSA_ERR_DTYPE;
  const bool i8 = dst.dtype == MSA_DTYPE_I8, mx = dst.dtype == MSA_DTYPE_MXFP4;
  if (T > 0 && (i8 || mx) != (in.scale != nullptr)) return MSA_ERR_SCALE;
  if (src.ndim != 3 || src.shape[0] != T || src.shape[1] < 1 || src.shape[1] > 65536 ||
      src.shape[2] != msa::kD)
    return MSA_ERR_SHAPE;
  const int64_t H = src.shape[1], last = mx ? msa::kD / 2 : msa::kD;
  a.src_row = (T > 1 ? src.stride[0] : 0) * 2;
  a.src_head = (H > 1 ? src.stride[1] : 0) * 2;
  if (src.stride[2] != 1 || a.src_row < 0 || a.src_head < 0 || a.src_row % 16 || a.src_head % 16 ||
      !msa::aligned16(src.data))
    return MSA_ERR_STRIDE;
  if (in.layout == MSA_LAYOUT_ROWS) {
    if (dst.ndim != 3 || dst.shape[0] != T || dst.shape[1] != H || dst.shape[2] != last)
      return MSA_ERR_SHAPE;
    a.row = (T > 1 ? dst.stride[0] : 0) * eb;
    a.head = (H > 1 ? dst.stride[1] : 0) * eb;
    // (rows that overlap would be written by two waves: a token's heads lie
    // within its stride, or a head's tokens within the head's)
    const int64_t len = last * eb;
    if (dst.stride[2] != 1 || (T > 1 && a.row < len) || (H > 1 && a.head < len) ||
        (T > 1 && H > 1 && a.row < a.head * (H - 1) + len && a.head < a.row * (T - 1) + len) ||
        a.row % 16 || a.head % 16 || !msa::aligned16(dst.data))
      return MSA_ERR_STRIDE;
    a.s_head = 4;                      // [T, H] floats, or [T, H, 4] bytes
    a.s_row = H * 4;
    a.limit = T;
  } else {
    msa::CacheView v;
    const msa_status_t st = msa::cache_view(dst, in.layout, last, msa::kP, false, v);
    if (st != MSA_OK) return st;
    if (v.heads != H) return MSA_ERR_SHAPE;
    // (pages that overlap, likewise)
    if (in.layout != MSA_LAYOUT_TND && v.pages > 1 && v.page < H * msa::kP * last * eb)
      return MSA_ERR_STRIDE;
    a.page = v.page;
    a.row = v.row;
    a.head = v.head;
    a.limit = v.pages;
    // scale: int8 [NP, H, 128] or [T2, H] floats; MXFP4 the layout's own
    // shape with 4 bytes a row
    const bool heads_first = in.layout == MSA_LAYOUT_BNBD || (i8 && in.layout != MSA_LAYOUT_TND);
    a.s_page = in.layout == MSA_LAYOUT_TND ? 0 : H * msa::kP * 4;
    a.s_row = heads_first ? 4 : H * 4;
    a.s_head = heads_first ? msa::kP * 4 : 4;
  }
  if (reinterpret_cast<uintptr_t>(in.scale) & 3u) return MSA_ERR_STRIDE;
  if (T > 0 && (!src.data || (!dst.data && a.limit > 0))) return MSA_ERR_NULL;
  a.src = static_cast<const uint8_t*>(src.data);
  a.dst = static_cast<uint8_t*>(const_cast<void*>(dst.data));
  a.scale = static_cast<uint8_t*>(in.scale);
  a.heads = (int32_t)H;
  a.steps = (int32_t)((H + 3) / 4);
  a.kind = dst.dtype;
  a.layout = in.layout;
  a.rotate = in.rotate;
  return MSA_OK;
}

// Position axes of a call (axes 0: none).
struct Axes {
  const int32_t* positions;
  int32_t axes;
  const uint8_t* of_pair;
};

msa_status_t append(const msa_append_item_t* items, int32_t num_items, const float* cos,
                    const float* sin, int64_t positions, int32_t rotary_dim, int32_t interleaved,
                    const Axes& ax, const int32_t* block_table, int64_t max_blocks,
                    const int32_t* cu_seqlens_q, const int32_t* kv_len, int32_t batch,
                    int32_t block_size, void* stream) {
  if (!items || !cu_seqlens_q) return MSA_ERR_NULL;
  if (batch > 0 && !kv_len) return MSA_ERR_NULL;
  if (num_items < 1 || num_items > MSA_APPEND_MAX_ITEMS) return MSA_ERR_ATTR;
  const int32_t dt = items[0].src.dtype;
  if (dt != MSA_DTYPE_F16 && dt != MSA_DTYPE_BF16) return MSA_ERR_DTYPE;
  if (items[0].src.ndim != 3) return MSA_ERR_SHAPE;
  const int64_t T = items[0].src.shape[0];
  if (T < 0 || T > INT32_MAX || batch < 0 || batch > (1 << 30) || block_size != msa::kP ||
      max_blocks < 0 || max_blocks > (1 << 24) || positions < 0)
    return MSA_ERR_SHAPE;
  if (batch == 0 && T > 0) return MSA_ERR_SHAPE;

  AppendParams p{};
  bool rotated = false, paged = false;
  for (int i = 0; i < num_items; ++i) {
    if (items[i].src.dtype != dt) return MSA_ERR_DTYPE;
    const msa_status_t st = item_for(items[i], T, p.item[i]);
    if (st != MSA_OK) return st;
    rotated = rotated || p.item[i].rotate;
    paged = paged || items[i].layout == MSA_LAYOUT_BBND || items[i].layout == MSA_LAYOUT_BNBD;
    if (items[i].layout == MSA_LAYOUT_TND) p.packed = 1;
    p.steps += p.item[i].steps;
  }
  if (interleaved != 0 && interleaved != 1) return MSA_ERR_ATTR;
  if (rotated) {
    if (rotary_dim < 16 || rotary_dim > msa::kD || rotary_dim % 16) return MSA_ERR_ATTR;
    if (T > 0 && positions > 0 && (!cos || !sin)) return MSA_ERR_NULL;
    if (!msa::aligned16(cos) || !msa::aligned16(sin)) return MSA_ERR_STRIDE;
    if (ax.axes > 0) {
      if (!ax.of_pair || (T > 0 && !ax.positions)) return MSA_ERR_NULL;
      if (reinterpret_cast<uintptr_t>(ax.positions) & 3u) return MSA_ERR_STRIDE;
      for (int r = 0; r < rotary_dim / 2; ++r) {
        if (ax.of_pair[r] >= ax.axes) return MSA_ERR_ATTR;
        p.pair_axis[r >> 5] |= (uint64_t)ax.of_pair[r] << (2 * (r & 31));
      }
      p.axis_pos = ax.positions;
      p.axes = ax.axes;
    }
  }
  if (paged) {
    if (max_blocks < 1) return MSA_ERR_SHAPE;
    if (!block_table && batch > 0) return MSA_ERR_NULL;
  }
  if (T == 0) return MSA_OK;

  p.cos = cos;
  p.sin = sin;
  p.block_table = paged ? block_table : nullptr;
  p.cu_q = cu_seqlens_q;
  p.kv_len = kv_len;
  p.positions = positions;
  p.T = T;
  p.B = batch;
  p.MB = (int32_t)max_blocks;
  p.half = rotated ? rotary_dim / 2 : 0;
  p.interleaved = interleaved;
  p.groups = groups_for(T, p.steps);
  p.per_wave = (p.steps + p.groups - 1) / p.groups;
  const int64_t grid = (T * p.groups + msa::kAppendWaves - 1) / msa::kAppendWaves;
  // (a launch holds less than 2^32 threads)
  if (grid * 64 * msa::kAppendWaves > (int64_t)UINT32_MAX) return MSA_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 gr((unsigned)grid), bl(64 * msa::kAppendWaves);
  const bool bf = dt == MSA_DTYPE_BF16;
  const hipError_t e =
      p.axes > 0 ? bf ? msa::launch_kernel(msa::append_kernel<true, true>, gr, bl, s, p)
                      : msa::launch_kernel(msa::append_kernel<false, true>, gr, bl, s, p)
      : bf ? msa::launch_kernel(msa::append_kernel<true, false>, gr, bl, s, p)
           : msa::launch_kernel(msa::append_kernel<false, false>, gr, bl, s, p);
  return e == hipSuccess ? MSA_OK : MSA_ERR_HIP;
}

}  // namespace

extern "C" {

msa_status_t msa_cache_append(const msa_append_item_t* items, int32_t num_items, const float* cos,
                              const float* sin, int64_t positions, int32_t rotary_dim,
                              int32_t interleaved, const int32_t* block_table, int64_t max_blocks,
                              const int32_t* cu_seqlens_q, const int32_t* kv_len, int32_t batch,
                              int32_t block_size, void* stream) {
  return append(items, num_items, cos, sin, positions, rotary_dim, interleaved, Axes{}, block_table,
                max_blocks, cu_seqlens_q, kv_len, batch, block_size, stream);
}

msa_status_t msa_cache_append_axes(const msa_append_item_t* items, int32_t num_items,
                                   const float* cos, const float* sin, int64_t positions,
                                   int32_t rotary_dim, int32_t interleaved,
                                   const int32_t* axis_positions, int32_t axes,
                                   const uint8_t* pair_axes, const int32_t* block_table,
                                   int64_t max_blocks, const int32_t* cu_seqlens_q,
                                   const int32_t* kv_len, int32_t batch, int32_t block_size,
                                   void* stream) {
  if (axes < 1 || axes > MSA_APPEND_MAX_AXES) return MSA_ERR_ATTR;
  return append(items, num_items, cos, sin, positions, rotary_dim, interleaved,
                Axes{axis_positions, axes, pair_axes}, block_table, max_blocks, cu_seqlens_q,
                kv_len, batch, block_size, stream);
}

}  // extern "C"
