// attend_d128_b4.cu -- sparse and tree attention, head dimension 128, 4-bit codes.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(128, 4)

}  // namespace kivi
