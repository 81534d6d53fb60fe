// attend_d256_b2.cu -- sparse and tree attention, head dimension 256, 2-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(256, 2)

}  // namespace kivi
