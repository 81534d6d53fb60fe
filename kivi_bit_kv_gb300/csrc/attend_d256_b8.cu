// attend_d256_b8.cu -- sparse and tree attention, head dimension 256, 8-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(256, 8)

}  // namespace kivi
