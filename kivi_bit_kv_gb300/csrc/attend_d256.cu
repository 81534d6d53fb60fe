// attend_d256.cu -- sparse and tree attention, head dimension 256.
#include "attend.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(256)

#ifdef KIVI_CHECKS
int32_t check_word_attend_d256() { return take_check_word(); }
#endif

}  // namespace kivi
