// Host helpers that the C ABI's entry points share.
#pragma once

#include "msa_index_score.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <tuple>

namespace msa {

inline int elem_bytes(int32_t dt) {
  switch (dt) {
    case MSA_DTYPE_F16:
    case MSA_DTYPE_BF16: return 2;
    case MSA_DTYPE_I8:
    case MSA_DTYPE_F8E4M3:
    case MSA_DTYPE_F8E5M2:
    case MSA_DTYPE_MXFP4: return 1;   // MXFP4: a byte holds two elements
    default: return 0;
  }
}

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// Extent-1 axes are never addressed, so their strides are not compared.
inline bool compact_axis(int64_t extent, int64_t stride, int64_t want) {
  return extent <= 1 || stride == want;
}

// Launch `kern` with these arguments (converted to its parameter types) and
// return the status of this launch alone.  (hipGetLastError after a
// triple-chevron launch would also return, and clear, an error left pending
// by earlier unrelated HIP calls of the caller.)
template <typename... KA, typename... A>
hipError_t launch_kernel(void (*kern)(KA...), dim3 grid, dim3 block, hipStream_t s, A... a) {
  static_assert(sizeof...(KA) == sizeof...(A), "one value per kernel parameter");
  std::tuple<KA...> vals{static_cast<KA>(a)...};
  void* ptrs[sizeof...(KA)];
  std::apply([&](auto&... v) {
    int i = 0;
    ((ptrs[i++] = static_cast<void*>(&v)), ...);
  }, vals);
  return hipLaunchKernel(reinterpret_cast<const void*>(kern), grid, block, ptrs, 0, s);
}

// Shape and byte strides of a paged or packed cache tensor.  The axes other
// than the first are compact; a packed tensor's token stride is free where
// `free_tokens` says so (rows that lie in a wider projection's rows).
struct CacheView {
  int64_t pages = 0;       // NP (paged) or T2 (packed)
  int64_t heads = 0;
  int64_t page = 0, row = 0, head = 0;   // bytes
};

inline msa_status_t cache_view(const msa_tensor_t& t, int32_t layout, int64_t last, int64_t block,
                               bool free_tokens, CacheView& v) {
  const int64_t* s = t.stride;
  const int64_t* n = t.shape;
  const int eb = elem_bytes(t.dtype);
  int64_t page = 0, row = 0, head = 0;
  if (layout == MSA_LAYOUT_TND) {
    if (t.ndim != 3 || n[0] < 0 || n[1] < 1 || n[2] != last) return MSA_ERR_SHAPE;
    if (!compact_axis(n[2], s[2], 1) || !compact_axis(n[1], s[1], last)) return MSA_ERR_STRIDE;
    row = n[0] > 1 ? s[0] : n[1] * last;
    if (free_tokens ? row < n[1] * last : row != n[1] * last) return MSA_ERR_STRIDE;
    v.pages = n[0];
    v.heads = n[1];
    head = last;
  } else if (layout == MSA_LAYOUT_BBND && t.ndim == 3) {
    if (n[0] < 1 || n[1] != block || n[2] != last) return MSA_ERR_SHAPE;
    if (!compact_axis(n[2], s[2], 1) || !compact_axis(n[1], s[1], last)) return MSA_ERR_STRIDE;
    v.pages = n[0];
    v.heads = 1;
    page = s[0];
    row = last;
  } else {
    const bool bbnd = layout == MSA_LAYOUT_BBND;
    if (t.ndim != 4) return MSA_ERR_SHAPE;
    const int64_t P = bbnd ? n[1] : n[2];
    v.pages = n[0];
    v.heads = bbnd ? n[2] : n[1];
    if (n[0] < 1 || v.heads < 1 || P != block || n[3] != last) return MSA_ERR_SHAPE;
    row = bbnd ? v.heads * last : last;
    head = bbnd ? last : P * last;
    page = s[0];
    if (!compact_axis(n[3], s[3], 1) || !compact_axis(v.heads, bbnd ? s[2] : s[1], head) ||
        !compact_axis(P, bbnd ? s[1] : s[2], row))
      return MSA_ERR_STRIDE;
  }
  if (layout != MSA_LAYOUT_TND) {
    if (v.pages > 1 && page < 1) return MSA_ERR_STRIDE;
    if (v.pages == 1) page = 0;
  }
  if ((page * eb) % 16 || (row * eb) % 16 || !aligned16(t.data)) return MSA_ERR_STRIDE;
  // 32-bit offsets within a block of one head
  if ((block - 1) * row * eb + last * eb > INT32_MAX || head * eb > INT32_MAX || v.heads > 65536 ||
      v.pages > INT32_MAX)
    return MSA_ERR_SHAPE;
  v.page = page * eb;
  v.row = row * eb;
  v.head = v.heads > 1 ? head * eb : 0;
  return MSA_OK;
}

}  // namespace msa
