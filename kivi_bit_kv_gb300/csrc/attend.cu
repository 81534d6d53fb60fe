// attend.cu -- dispatch of kivi_sparse_attention and kivi_tree_attention
// (kernels in attend.cuh, one translation unit per head dimension and width).
#include "attend_plan.h"
#include "kivi_launch.h"

namespace kivi {

size_t attend_ws_bytes(const kivi_cache& c, int Hq, int N)
{
    const int M = Hq / c.H * N;
    const bool warp = attend_by_warp(c.D, M);
    const size_t pieces = warp ? kAttMaxRanges : kAttMaxCTAs;
    const size_t floats = warp ? warp_part_floats(c.D, M) : (size_t)attend_rows(c.D, M) * (c.D + 2);
    return (kAttHeaderFloats + pieces * (kAttCutInts + 2 * floats)) * sizeof(float);
}

size_t attend_ws_bytes_upto(const kivi_cache& c, int Hq, int N)
{
    // the warp kernel has more and smaller pieces than the tcgen05 kernel, so a
    // call for more drafts may need less
    size_t most = 0;
    for (int n = 1; n <= N; ++n)
        most = attend_ws_bytes(c, Hq, n) > most ? attend_ws_bytes(c, Hq, n) : most;
    return most;
}

template <int D>
static cudaError_t launch_attend_d(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s)
{
    switch (c.bits_k == c.bits_v ? c.bits_k : 0) {
    case 2: return launch_attend_b<D, 2>(c, a, ws, s);
    case 4: return launch_attend_b<D, 4>(c, a, ws, s);
    case 8: return launch_attend_b<D, 8>(c, a, ws, s);
    default: return launch_attend_b<D, 0>(c, a, ws, s);
    }
}

cudaError_t launch_attend(const kivi_cache& c, const AttendArgs& a, void* ws, cudaStream_t s)
{
    float* w = static_cast<float*>(ws);
    switch (c.D) {
    case 64: return launch_attend_d<64>(c, a, w, s);
    case 128: return launch_attend_d<128>(c, a, w, s);
    default: return launch_attend_d<256>(c, a, w, s);
    }
}

#ifdef KIVI_CHECKS
// The first failed check of any unit; every unit's word is read and cleared.
template <int D>
static void check_words(int32_t& first)
{
    for (const int32_t w : {check_word_attend_b<D, 0>(), check_word_attend_b<D, 2>(), check_word_attend_b<D, 4>(),
                            check_word_attend_b<D, 8>()})
        if (first == KIVI_OK || w == KIVI_ECUDA)
            first = w;
}
int32_t check_word_attend()
{
    int32_t first = KIVI_OK;
    check_words<64>(first);
    check_words<128>(first);
    check_words<256>(first);
    return first;
}
#endif

}  // namespace kivi
