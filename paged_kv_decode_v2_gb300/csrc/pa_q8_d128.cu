// Attention kernels over an 8-bit cache, head_dim 128.
#include "pa_q8.cuh"

namespace pa {
PA_DEFINE_Q8_OPS(q8_ops_d128, 128)
} // namespace pa
