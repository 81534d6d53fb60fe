// attend_launch.cuh -- which kernel serves a call of kivi_sparse_attention or
// kivi_tree_attention.
#pragma once

#include "attend_warp.cuh"

namespace kivi {

// Up to 16 query rows of a KV head (8 at D = 256) go to the warp kernel, more
// to the tcgen05 kernel, whose products cost the same up to 32 rows.  Beyond,
// the warp kernel would need the registers of 24 rows' O (16 at D = 256).  Both
// sides in us, warp kernel against tcgen05 kernel, int2:
//     rows of a KV head                     1           8         16
//     B 8, H 32, D 128, T 4096      77 / 165    82 / 172  124 / 176
//     B 4, H 8, D 128, T 32768     107 / 161   113 / 171  157 / 173
//     B 1, H 8, D 128, T 2048       17 /  25    21 /  41   28 /  41
//     B 1, H 1, D 128, T 32768      73 / 103    78 / 315  113 / 310
//     B 1, H 8, D 128, T 32768      79 /  66    84 / 100  122 / 101
//     B 8, H 32, D 64, T 4096       47 / 119    50 / 125   63 / 129
//     B 8, H 32, D 256, T 4096     193 / 229   200 / 241
//     B 1, H 8, D 256, T 32768     148 /  74   157 / 113
// The rule goes by rows alone.  Where few long rows fill neither kernel (the
// fifth and the last line) the other side is faster: the warp kernel takes
// ranges longer than it would need to (warp_locate).
template <int D, int B>
cudaError_t launch_attend_b(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s)
{
    KIVI_SET_CHECK_RANGES(c, s, {{a.q, (size_t)c.B * a.Hq * a.N * D * 2}, {a.out, (size_t)c.B * a.Hq * a.N * D * 4},
                                 {a.k ? a.k : (const void*)a.blocks,  // a call has drafts or a list of groups
                                  (size_t)c.B * c.H * (a.k ? (size_t)a.N * D * 2 : (size_t)a.n_keep * 4)},
                                 {a.v, (size_t)c.B * c.H * a.N * D * 2},
                                 {a.mask, (size_t)c.B * a.N * ((a.N + 63) / 64) * 8}, {a.n_draft, (size_t)c.B * 4},
                                 {ws, attend_ws_bytes(c, a.Hq, a.N)}});
    const int M = a.Hq / c.H * a.N;
    if (attend_by_warp(D, M)) {
        if constexpr (D != 256)
            if (M > 8)
                return attend_warp_launch<D, 2, B>(c, a, ws, s);
        return attend_warp_launch<D, 1, B>(c, a, ws, s);
    }
    switch (attend_rows(D, M)) {
    case 32: return attend_launch_rows<D, 32, B>(c, a, ws, s);
    case 64:
        if constexpr (D != 256)
            return attend_launch_rows<D, 64, B>(c, a, ws, s);
        break;
    default:
        if constexpr (D != 256)
            return attend_launch_rows<D, 128, B>(c, a, ws, s);
        break;
    }
    return cudaErrorInvalidValue;
}

// Instantiates the kernels of one head dimension and code width (0: mixed), a
// translation unit each, so that they compile in parallel.
#ifdef KIVI_CHECKS
#define KIVI_ATTEND_INSTANTIATE(DIM, B)                                                                       \
    template cudaError_t launch_attend_b<DIM, B>(const kivi_cache&, const AttendArgs&, float*, cudaStream_t); \
    template <>                                                                                               \
    int32_t check_word_attend_b<DIM, B>()                                                                     \
    {                                                                                                         \
        return take_check_word();                                                                             \
    }
#else
#define KIVI_ATTEND_INSTANTIATE(DIM, B) \
    template cudaError_t launch_attend_b<DIM, B>(const kivi_cache&, const AttendArgs&, float*, cudaStream_t);
#endif

}  // namespace kivi
