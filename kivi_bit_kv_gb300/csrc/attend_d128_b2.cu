// attend_d128_b2.cu -- sparse and tree attention, head dimension 128, 2-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(128, 2)

}  // namespace kivi
