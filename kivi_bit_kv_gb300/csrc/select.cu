// select.cu -- kivi_block_select: which key groups a query may attend, from the
// cache's own statistics.
//
// A group's zero and zero + M scale are its smallest and largest key per
// channel, so sum_d max(q_d lo_d, q_d hi_d) bounds q . k over the group
// without reading a code.  With q+ = max(q, 0) and q- = min(q, 0) one of
// q+ hi and q- lo is zero and their sum is the larger product, rounded once:
// one multiply and one fused multiply-add per channel and head.  The sum over
// channels is pairwise over neighbours: inside a lane first (a lane holds
// D / 32 neighbouring channels), then lane pairs 1, 2, 4, 8, 16 apart.
#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

constexpr int kScoreThreads = 256;
constexpr int kSelectThreads = 256;

__device__ __forceinline__ int cache_len(const kivi_cache& c, int b)
{
    return min(max(ld_checked(c.len + b), 0), c.Tmax);
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads)
block_score_kernel(kivi_cache c, const uint16_t* __restrict__ q, int gq, float M, float* __restrict__ scores)
{
    constexpr int CPL = D / 32;  // channels per lane
    const int bh = blockIdx.y, b = bh / c.H;
    const int nb = quantized_tokens(cache_len(c, b), c.G, c.R) / c.G;
    const int NB = c.Tmax / c.G;
    const int lane = threadIdx.x & 31;
    const int g = blockIdx.x * (kScoreThreads / 32) + threadIdx.x / 32;
    if (g >= nb)
        return;
    const size_t so = ((size_t)bh * NB + g) * D + lane * CPL;
    float lo[CPL], hi[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        lo[i] = ldg_checked(c.kzero + so + i);
        hi[i] = __fadd_rn(lo[i], __fmul_rn(ldg_checked(c.kscale + so + i), M));
    }
    float best = -INFINITY;
    for (int hq = 0; hq < gq; ++hq) {
        const uint16_t* qp = q + ((size_t)bh * gq + hq) * D + lane * CPL;
        float t[CPL];
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            const float x = __half2float(__ushort_as_half(ldg_checked(qp + i)));
            t[i] = __fmaf_rn(fmaxf(x, 0.0f), hi[i], __fmul_rn(fminf(x, 0.0f), lo[i]));
        }
#pragma unroll
        for (int n = CPL / 2; n > 0; n /= 2)
#pragma unroll
            for (int i = 0; i < n; ++i)
                t[i] = __fadd_rn(t[2 * i], t[2 * i + 1]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            t[0] = __fadd_rn(t[0], __shfl_xor_sync(0xffffffffu, t[0], o));
        best = hq == 0 ? t[0] : fmaxf(best, t[0]);
    }
    if (lane == 0)
        st_checked(scores + (size_t)bh * NB + g, best);
}

// Order-preserving 32-bit key of a score: larger score, larger key; -0 counts
// as +0 and NaN as the lowest.
__device__ __forceinline__ uint32_t score_key(float s)
{
    const uint32_t u = __float_as_uint(s + 0.0f);
    if (isnan(s))
        return 0u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One CTA per (b, h): a radix select finds the key of the n_keep-th largest
// score in four passes of eight bits, then one ordered pass writes the indices
// above it and the first of those equal to it.
__global__ void __launch_bounds__(kSelectThreads)
block_pick_kernel(kivi_cache c, const float* __restrict__ scores, int32_t* __restrict__ blocks, int n_keep)
{
    constexpr int T = kSelectThreads, W = T / 32;
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_digit, s_need;
    __shared__ uint32_t wsum[2][W];
    const int bh = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int nb = quantized_tokens(cache_len(c, bh / c.H), c.G, c.R) / c.G;
    const float* sc = scores + (size_t)bh * (c.Tmax / c.G);
    int32_t* dst = blocks + (size_t)bh * n_keep;
    const int m = min(n_keep, nb);
    for (int i = m + tid; i < n_keep; i += T)
        st_checked(dst + i, -1);
    if (m == nb) {
        for (int i = tid; i < nb; i += T)
            st_checked(dst + i, i);
        return;
    }
    uint32_t prefix = 0, need = (uint32_t)m;  // need of the keys that start with prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < nb; i += T) {
            const uint32_t key = score_key(ld_checked(sc + i));
            if (shift == 24 || (key >> (shift + 8)) == prefix)
                atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t above = 0;
            int d = 255;
            for (; d > 0 && above + hist[d] < need; --d)
                above += hist[d];
            s_digit = (uint32_t)d;
            s_need = need - above;
        }
        __syncthreads();
        prefix = (prefix << 8) | s_digit;
        need = s_need;
    }
    // keys above `prefix`, and the first `need` of those equal to it, in order
    uint32_t eq_seen = 0, out_at = 0;
    for (int i0 = 0; i0 < nb; i0 += T) {
        const int i = i0 + tid;
        const uint32_t key = i < nb ? score_key(ld_checked(sc + i)) : 0u;
        const bool gt = i < nb && key > prefix, eq = i < nb && key == prefix;
        const uint32_t beq = __ballot_sync(0xffffffffu, eq);
        if (lane == 0)
            wsum[0][warp] = __popc(beq);
        __syncthreads();
        uint32_t before = eq_seen, all = 0;
        for (int w = 0; w < W; ++w) {
            before += w < warp ? wsum[0][w] : 0u;
            all += wsum[0][w];
        }
        const bool take = gt || (eq && before + __popc(beq & ((1u << lane) - 1u)) < need);
        const uint32_t bt = __ballot_sync(0xffffffffu, take);
        if (lane == 0)
            wsum[1][warp] = __popc(bt);
        __syncthreads();
        uint32_t at = out_at, tall = 0;
        for (int w = 0; w < W; ++w) {
            at += w < warp ? wsum[1][w] : 0u;
            tall += wsum[1][w];
        }
        if (take)
            st_checked(dst + at + __popc(bt & ((1u << lane) - 1u)), i);
        eq_seen += all;
        out_at += tall;
        __syncthreads();
    }
}

cudaError_t launch_block_select(const kivi_cache& c, const uint16_t* q, int Hq, int32_t* blocks, int n_keep,
                                float* scores, cudaStream_t s)
{
    const int NB = c.Tmax / c.G, BH = c.B * c.H;
    KIVI_SET_CHECK_RANGES(c, s, {{q, (size_t)c.B * Hq * c.D * 2}, {blocks, (size_t)BH * n_keep * 4},
                                 {scores, (size_t)BH * NB * 4}});
    const dim3 grid((NB + kScoreThreads / 32 - 1) / (kScoreThreads / 32), BH);
    const float M = (float)((1 << c.bits_k) - 1);
    switch (c.D) {
    case 64: block_score_kernel<64><<<grid, kScoreThreads, 0, s>>>(c, q, Hq / c.H, M, scores); break;
    case 128: block_score_kernel<128><<<grid, kScoreThreads, 0, s>>>(c, q, Hq / c.H, M, scores); break;
    default: block_score_kernel<256><<<grid, kScoreThreads, 0, s>>>(c, q, Hq / c.H, M, scores); break;
    }
    block_pick_kernel<<<BH, kSelectThreads, 0, s>>>(c, scores, blocks, n_keep);
    return cudaGetLastError();
}

#ifdef KIVI_CHECKS
int32_t check_word_select() { return take_check_word(); }
#endif

}  // namespace kivi
