// Launches of the dense attention kernels in the other forms of the scores
// (capped, biased, narrowed by a range of keys per token): compiled apart from the
// plain ones, a type each, as they are many.
#pragma once

#include "msa_attention.hpp"
#include "msa_host.hpp"

namespace msa {

// Launches `form` (a sum of ScoreForms, not 0) with tiles of `rows` rows.
template <int KK>
hipError_t launch_form(const AttnParams& p, int rows, int form, dim3 grid, hipStream_t s);

template <int KK, int F>
hipError_t launch_rows_of(const AttnParams& p, int rows, dim3 grid, hipStream_t s) {
  if (rows == kAttnRows)
    return launch_kernel(attn_rows_kernel<KK, false, F>, grid, dim3(256), s, p);
  if (rows == 256) return launch_kernel(attn_tile_kernel<KK, 8, F>, grid, dim3(512), s, p);
  return launch_kernel(attn_tile_kernel<KK, 4, F>, grid, dim3(256), s, p);
}

template <int KK>
hipError_t launch_form_of(const AttnParams& p, int rows, int form, dim3 grid, hipStream_t s) {
  switch (form & (kCap | kBias)) {
    case 0: return launch_rows_of<KK, kRange>(p, rows, grid, s);
    case kCap: return launch_rows_of<KK, kRange | kCap>(p, rows, grid, s);
    case kBias: return launch_rows_of<KK, kRange | kBias>(p, rows, grid, s);
    default: return launch_rows_of<KK, kRange | kCap | kBias>(p, rows, grid, s);
  }
}

}  // namespace msa
