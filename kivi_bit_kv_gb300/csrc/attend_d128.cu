// attend_d128.cu -- sparse and tree attention, head dimension 128.
#include "attend.cuh"

namespace kivi {

KIVI_ATTEND_INSTANTIATE(128)

#ifdef KIVI_CHECKS
int32_t check_word_attend_d128() { return take_check_word(); }
#endif

}  // namespace kivi
