// attend_d128_mixed.cu -- sparse and tree attention, head dimension 128, key and value widths that differ.
#include "attend_launch.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(128, 0)

}  // namespace kivi
