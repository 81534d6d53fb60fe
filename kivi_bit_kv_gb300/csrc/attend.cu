// attend.cu -- dispatch of kivi_sparse_attention and kivi_tree_attention
// (kernels in attend.cuh, one translation unit per head dimension).
#include "attend.cuh"

namespace kivi {

size_t attend_ws_bytes(const kivi_cache& c, int Hq, int N)
{
    const int NR = attend_rows(c.D, Hq / c.H * N);
    return ((size_t)kAttHeaderFloats + (size_t)kAttMaxCTAs * kAttCutInts +
            (size_t)kAttMaxCTAs * 2 * NR * (c.D + 2)) * sizeof(float);
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

}  // namespace kivi
