// attend_d64_mixed.cu -- sparse and tree attention, head dimension 64, key and value widths that differ.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(64, 0)

}  // namespace kivi
