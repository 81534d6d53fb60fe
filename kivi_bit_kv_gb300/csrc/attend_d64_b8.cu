// attend_d64_b8.cu -- sparse and tree attention, head dimension 64, 8-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(64, 8)

}  // namespace kivi
