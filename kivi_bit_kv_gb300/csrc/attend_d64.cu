// attend_d64.cu -- sparse and tree attention, head dimension 64.
#include "attend.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(64)

#ifdef KIVI_CHECKS
int32_t check_word_attend_d64() { return take_check_word(); }
#endif

}  // namespace kivi
