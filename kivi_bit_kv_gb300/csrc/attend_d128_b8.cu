// attend_d128_b8.cu -- sparse and tree attention, head dimension 128, 8-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(128, 8)

}  // namespace kivi
