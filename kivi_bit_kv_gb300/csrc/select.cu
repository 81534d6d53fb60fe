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
//
// Bound by the statistics' bytes (8 D a group).  A warp scores eight
// neighbouring groups (four at D = 256), so that sixteen loads a lane are in
// flight, and reduces the eight sums together: a lane keeps half of what it
// holds at each of the first three exchanges, nine shuffles instead of forty.
#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

constexpr int kScoreThreads = 256;
// groups of a warp: sixteen or more 16-byte loads a lane in flight within 128
// registers
__host__ __device__ constexpr int score_groups(int D) { return D == 256 ? 4 : 8; }
constexpr int kSelectThreads = 256;
constexpr int kSelectKeys = 8;    // keys a thread keeps in registers
static_assert(kSelectThreads == 256, "one histogram bin per thread");

__device__ __forceinline__ int cache_len(const kivi_cache& c, int b)
{
    return min(max(ld_checked(c.len + b), 0), c.Tmax);
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads)
block_score_kernel(kivi_cache c, const uint16_t* __restrict__ q, int gq, float M, float* __restrict__ scores)
{
    constexpr int CPL = D / 32;  // channels per lane: 2, 4 or 8
    constexpr int V = CPL < 4 ? CPL : 4, NV = CPL / V;
    constexpr int NG = score_groups(D);
    // q+ and q- of the heads
    __shared__ float2 s_q[16 * D];
    asm volatile("griddepcontrol.launch_dependents;");
    const int NB = c.Tmax / c.G, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int chunks = (NB + NG * (kScoreThreads / 32) - 1) / (NG * (kScoreThreads / 32));
    const size_t bh = blockIdx.x / chunks;
    const int nb = quantized_tokens(cache_len(c, (int)(bh / c.H)), c.G, c.R) / c.G;
    const int first = (int)(blockIdx.x % chunks) * NG * (kScoreThreads / 32);
    if (first >= nb)
        return;
    for (int i = threadIdx.x; i < gq * D; i += kScoreThreads) {
        const float x = __half2float(__ushort_as_half(ldg_checked(q + bh * gq * D + i)));
        s_q[i] = make_float2(fmaxf(x, 0.0f), fminf(x, 0.0f));
    }
    __syncthreads();
    const int g0 = first + warp * NG;
    if (g0 >= nb)
        return;
    float lo[NG][CPL], hi[NG][CPL];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        const size_t at = (bh * NB + min(g0 + k, nb - 1)) * D + lane * CPL;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (V == 4) {
                const float4 z = ld_nc_f4(c.kzero + at + 4 * v), s = ld_nc_f4(c.kscale + at + 4 * v);
                lo[k][4 * v] = z.x, lo[k][4 * v + 1] = z.y, lo[k][4 * v + 2] = z.z, lo[k][4 * v + 3] = z.w;
                hi[k][4 * v] = s.x, hi[k][4 * v + 1] = s.y, hi[k][4 * v + 2] = s.z, hi[k][4 * v + 3] = s.w;
            } else {
                const float2 z = ldg_checked(reinterpret_cast<const float2*>(c.kzero + at));
                const float2 s = ldg_checked(reinterpret_cast<const float2*>(c.kscale + at));
                lo[k][0] = z.x, lo[k][1] = z.y;
                hi[k][0] = s.x, hi[k][1] = s.y;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int i = 0; i < CPL; ++i)
            hi[k][i] = __fadd_rn(lo[k][i], __fmul_rn(hi[k][i], M));
    float best = 0.0f;
#pragma unroll 1
    for (int h = 0; h < gq; ++h) {
        float2 x[CPL];
#pragma unroll
        for (int i = 0; i < CPL; ++i)
            x[i] = s_q[h * D + lane * CPL + i];
        float t[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            float y[CPL];
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                y[i] = __fmaf_rn(x[i].x, hi[k][i], __fmul_rn(x[i].y, lo[k][i]));
#pragma unroll
            for (int n = CPL / 2; n > 0; n /= 2)
#pragma unroll
                for (int i = 0; i < n; ++i)
                    y[i] = __fadd_rn(y[2 * i], y[2 * i + 1]);
            t[k] = y[0];
        }
        // the lane with the bit clear keeps the first half of the groups
#pragma unroll
        for (int o = 1, half = NG / 2; o < 32; o <<= 1, half /= 2) {
            if (half == 0)
                t[0] = __fadd_rn(t[0], __shfl_xor_sync(0xffffffffu, t[0], o));
#pragma unroll
            for (int k = 0; k < half; ++k) {
                const float give = lane & o ? t[k] : t[k + half], keep = lane & o ? t[k + half] : t[k];
                t[k] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, o));
            }
        }
        best = h == 0 ? t[0] : fmaxf(best, t[0]);
    }
    int k = 0;  // the group that this lane holds
#pragma unroll
    for (int o = 1, half = NG / 2; half > 0; o <<= 1, half /= 2)
        k += lane & o ? half : 0;
    if (lane < NG && g0 + k < nb)
        st_checked(scores + bh * NB + g0 + k, best);
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

// Exclusive prefix sums of n <= 64 counters, by one warp.
__device__ __forceinline__ void scan_words(uint32_t* w, int n)
{
    const int lane = threadIdx.x & 31;
    const uint32_t a = 2 * lane < n ? w[2 * lane] : 0u, b = 2 * lane + 1 < n ? w[2 * lane + 1] : 0u;
    uint32_t inc = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
        inc += lane >= o ? t : 0u;
    }
    if (2 * lane < n)
        w[2 * lane] = inc - a - b;
    if (2 * lane + 1 < n)
        w[2 * lane + 1] = inc - b;
}

// One CTA per (b, h): a radix select finds the key of the n_keep-th largest
// score in four passes of eight bits, then one ordered pass writes the indices
// above it and the first of those equal to it.  Bound by latency: per pass a
// histogram in shared memory and one warp's scan of it, with up to 2048 keys
// in registers throughout (a longer row reads its scores again).
__global__ void __launch_bounds__(kSelectThreads)
block_pick_kernel(kivi_cache c, const float* __restrict__ scores, int32_t* __restrict__ blocks, int n_keep)
{
    constexpr int T = kSelectThreads, W = T / 32, K = kSelectKeys;
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_digit, s_need, s_base[2];
    __shared__ uint32_t s_eq[W * K], s_take[W * K];
    const int bh = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int nb = quantized_tokens(cache_len(c, bh / c.H), c.G, c.R) / c.G;
    const float* sc = scores + (size_t)bh * (c.Tmax / c.G);
    int32_t* dst = blocks + (size_t)bh * n_keep;
    const int m = min(n_keep, nb);
    for (int i = m + tid; i < n_keep; i += T)
        st_checked(dst + i, -1);
    if (m == nb)
        for (int i = tid; i < nb; i += T)
            st_checked(dst + i, i);
    // the scores are written; every CTA waits, so that none of what follows in
    // the stream starts before them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (m == nb)
        return;
    const bool kept = nb <= T * K;
    uint32_t key[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = tid + k * T;
        key[k] = kept && i < nb ? score_key(ld_checked(sc + i)) : 0u;
    }
    uint32_t prefix = 0, need = (uint32_t)m;  // need of the keys that start with prefix
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        auto count = [&](uint32_t x) {
            if (shift == 24 || (x >> (shift + 8)) == prefix)
                atomicAdd(&hist[(x >> shift) & 255u], 1u);
        };
        if (kept) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (tid + k * T < nb)
                    count(key[k]);
        } else {
            for (int i = tid; i < nb; i += T)
                count(score_key(ld_checked(sc + i)));
        }
        __syncthreads();
        if (warp == 0) {  // lane: bins 255 - 8 lane downwards
            uint32_t n[8], sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum += n[k] = hist[255 - 8 * lane - k];
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
                inc += lane >= o ? t : 0u;
            }
            uint32_t above = inc - sum;
            if (above < need && need <= inc) {  // exactly one lane
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (above < need && need <= above + n[k]) {
                        s_digit = (uint32_t)(255 - 8 * lane - k);
                        s_need = need - above;
                    }
                    above += n[k];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | s_digit;
        need = s_need;
    }
    // keys above `prefix`, and the first `need` of those equal to it, in order,
    // T K at a time
    if (tid < 2)
        s_base[tid] = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < nb; i0 += T * K) {
        uint32_t eq[K], take[K];
        __syncthreads();
        const uint32_t eq_base = s_base[0], out_base = s_base[1];
        // word k W + warp of a mask: indices i0 + 32 (k W + warp) .. + 31
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = i0 + tid + k * T;
            if (!kept)
                key[k] = i < nb ? score_key(ld_checked(sc + i)) : 0u;
            eq[k] = __ballot_sync(0xffffffffu, i < nb && key[k] == prefix);
            if (lane == 0)
                s_eq[k * W + warp] = __popc(eq[k]);
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t last = s_eq[W * K - 1];
            __syncwarp();
            scan_words(s_eq, W * K);
            __syncwarp();
            if (lane == 0)
                s_base[0] = eq_base + s_eq[W * K - 1] + last;
        }
        __syncthreads();
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = i0 + tid + k * T;
            const bool is_eq = (eq[k] >> lane) & 1u;
            take[k] = __ballot_sync(0xffffffffu, i < nb && (key[k] > prefix ||
                                                            (is_eq && eq_base + s_eq[k * W + warp] + __popc(eq[k] & below) < need)));
            if (lane == 0)
                s_take[k * W + warp] = __popc(take[k]);
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t last = s_take[W * K - 1];
            __syncwarp();
            scan_words(s_take, W * K);
            __syncwarp();
            if (lane == 0)
                s_base[1] = out_base + s_take[W * K - 1] + last;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((take[k] >> lane) & 1u)
                st_checked(dst + out_base + s_take[k * W + warp] + __popc(take[k] & below), i0 + tid + k * T);
    }
}

cudaError_t launch_block_select(const kivi_cache& c, const uint16_t* q, int Hq, int32_t* blocks, int n_keep,
                                float* scores, cudaStream_t s)
{
    const int NB = c.Tmax / c.G, BH = c.B * c.H;
    KIVI_SET_CHECK_RANGES(c, s, {{q, (size_t)c.B * Hq * c.D * 2}, {blocks, (size_t)BH * n_keep * 4},
                                 {scores, (size_t)BH * NB * 4}});
    const int per = score_groups(c.D) * (kScoreThreads / 32);
    const dim3 grid((unsigned)BH * (unsigned)((NB + per - 1) / per));
    const float M = (float)((1 << c.bits_k) - 1);
    switch (c.D) {
    case 64: block_score_kernel<64><<<grid, kScoreThreads, 0, s>>>(c, q, Hq / c.H, M, scores); break;
    case 128: block_score_kernel<128><<<grid, kScoreThreads, 0, s>>>(c, q, Hq / c.H, M, scores); break;
    default: block_score_kernel<256><<<grid, kScoreThreads, 0, s>>>(c, q, Hq / c.H, M, scores); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    // the choice's CTAs are scheduled while the scores drain
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(BH);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_pick_kernel, c, (const float*)scores, blocks, n_keep);
}

#ifdef KIVI_CHECKS
int32_t check_word_select() { return take_check_word(); }
#endif

}  // namespace kivi
