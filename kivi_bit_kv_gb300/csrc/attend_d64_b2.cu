// attend_d64_b2.cu -- sparse and tree attention, head dimension 64, 2-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(64, 2)

}  // namespace kivi
