// The dense attention kernels' other forms of the scores, f16.
#include "msa_attention_forms.hpp"

template <>
hipError_t msa::launch_form<msa::KF16>(const AttnParams& p, int rows, int form, dim3 grid,
                                      hipStream_t s) {
  return launch_form_of<KF16>(p, rows, form, grid, s);
}
