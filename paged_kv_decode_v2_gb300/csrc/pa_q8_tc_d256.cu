// Attention over an 8-bit cache on the tcgen05 tensor cores, head_dim 256.
#include "pa_q8_tc.cuh"

namespace pa {

Q8TcKernel q8_tc_d256(int rows, int dtype, int mode)
{
    switch (rows) {
    case 8: return q8_tc_pick<256, 8>(dtype, mode);
    case 16: return q8_tc_pick<256, 16>(dtype, mode);
    case 32: return q8_tc_pick<256, 32>(dtype, mode);
    default: return {nullptr, 0, 0, 0};
    }
}

} // namespace pa
