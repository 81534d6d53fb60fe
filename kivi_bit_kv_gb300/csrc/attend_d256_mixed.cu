// attend_d256_mixed.cu -- sparse and tree attention, head dimension 256, key and value widths that differ.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(256, 0)

}  // namespace kivi
