// attend_d64_b4.cu -- sparse and tree attention, head dimension 64, 4-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(64, 4)

}  // namespace kivi
