// Attention over an 8-bit cache on the tcgen05 tensor cores, head_dim 128.
#include "pa_q8_tc.cuh"

namespace pa {

Q8TcKernel q8_tc_d128(int rows, int dtype, int mode)
{
    switch (rows) {
    case 8: return q8_tc_pick<128, 8>(dtype, mode);
    case 16: return q8_tc_pick<128, 16>(dtype, mode);
    case 32: return q8_tc_pick<128, 32>(dtype, mode);
    case 64: return q8_tc_pick<128, 64>(dtype, mode);
    default: return {nullptr, 0, 0, 0};
    }
}

} // namespace pa
