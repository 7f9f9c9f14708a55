// The dense attention kernels' other forms of the scores, bf16.
#include "msa_attention_forms.hpp"

template <>
hipError_t msa::launch_form<msa::KBF16>(const AttnParams& p, int rows, int form, dim3 grid,
                                      hipStream_t s) {
  return launch_form_of<KBF16>(p, rows, form, grid, s);
}
