// attend_d256_b4.cu -- sparse and tree attention, head dimension 256, 4-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(256, 4)

}  // namespace kivi
