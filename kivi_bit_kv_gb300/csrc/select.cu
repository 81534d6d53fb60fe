// select.cu -- kivi_block_select: which key groups a query may attend, from the
// cache's own statistics.
//
// A group's zero and zero + M scale are its smallest and largest key per
// channel, so sum_d max(q_d lo_d, q_d hi_d) bounds q . k over the group
// without reading a code.  lo <= hi, so the larger product is q hi for q >= 0
// and q lo otherwise: a select and a multiply per channel and head.  A NaN of
// the query or of either statistic stays one (lo is NaN where hi is, and the
// maxima carry it), so that a broken row cannot look like an ordinary choice;
// four query heads and more are 2 to 8 % faster than with max(q, 0) hi +
// min(q, 0) lo, one head the same.  The sum over
// channels is pairwise over neighbours: inside a lane first (a lane holds
// D / 32 neighbouring channels), then lane pairs 1, 2, 4, 8, 16 apart.
//
// Bound by the statistics' bytes (8 D a group).  A warp scores 512 / D
// neighbouring groups at a time while the next ones' statistics are on their
// way to its part of shared memory (cp.async: no lane reads what another
// copied, so nothing waits at a barrier), and reduces their sums together: a lane keeps half of
// what it holds at each of the first exchanges (four groups: six shuffles
// instead of twenty).
//
// Measured: 64 ragged sequences of 32 heads (295 MB of statistics): 50 us for
// the scores, 5.9 TB/s, and 14 us for the choice, 62 us together; four sequences
// of 1020 groups and 8 heads (34 MB): 11 and 8 us, 14 us together.
#include "kivi_device.cuh"
#include "kivi_launch.h"

#include <algorithm>
#include <type_traits>

namespace kivi {

constexpr int kScoreThreads = 256, kScoreWarps = kScoreThreads / 32;
constexpr int kScoreStages = 3;     // a warp's ring of statistics
constexpr int kScoreStage = 4096;   // bytes: the two statistics of score_groups(D) groups
constexpr int kScoreRing = kScoreWarps * kScoreStages * kScoreStage;
// groups of a warp at a time: 16 values of each statistic a lane
__host__ __device__ constexpr int score_groups(int D) { return 512 / D; }

// The larger and the smaller of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float min_nan(float x, float y)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// Threads that choose for one row, and the keys each keeps in registers.
struct PickWarp { static constexpr int T = 32, K = 16; };
struct PickCta { static constexpr int T = 256, K = 8; };

__device__ __forceinline__ int cache_len(const kivi_cache& c, int b)
{
    return min(max(ld_checked(c.len + b), 0), c.Tmax);
}

// cp_async16, or its 8-byte form.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const float* src)
{
    if constexpr (BYTES == 16) {
        cp_async16(dst, src);
    } else {
        if (KIVI_IN_RANGE(src, BYTES))
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                         "l"(src), "n"(BYTES)
                         : "memory");
    }
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads)
block_score_kernel(kivi_cache c, const uint16_t* __restrict__ q, int gq, int iters, float M,
                   float* __restrict__ scores)
{
    constexpr int CPL = D / 32;  // channels per lane: 2, 4 or 8
    constexpr int V = CPL < 4 ? CPL : 4, NV = CPL / V;
    constexpr int NG = score_groups(D);
    extern __shared__ __align__(16) uint8_t s_ring[];
    float* s_q = reinterpret_cast<float*>(s_ring + kScoreRing);  // [gq][D]
    asm volatile("griddepcontrol.launch_dependents;");
    const int NB = c.Tmax / c.G, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int per = iters * NG * kScoreWarps, chunks = (NB + per - 1) / per;
    const size_t bh = blockIdx.x / chunks;
    const int nb = quantized_tokens(cache_len(c, (int)(bh / c.H)), c.G, c.R) / c.G;
    const int first = (int)(blockIdx.x % chunks) * per, end = min(first + per, nb);
    if (first >= nb)
        return;
    // lane's share of a vector: NV pieces of V channels, 32 lanes' pieces side by side
    uint8_t* mine = s_ring + warp * kScoreStages * kScoreStage + lane * (4 * V);
    constexpr int kPiece = 32 * 4 * V;
    auto issue = [&](int it) {
        const int g0 = first + (it * kScoreWarps + warp) * NG;
        if (g0 < end) {
            uint8_t* dst = mine + it % kScoreStages * kScoreStage;
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                const size_t at = (bh * NB + min(g0 + k, nb - 1)) * D + lane * CPL;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    copy_async<4 * V>(dst + (2 * k * NV + v) * kPiece, c.kzero + at + V * v);
                    copy_async<4 * V>(dst + ((2 * k + 1) * NV + v) * kPiece, c.kscale + at + V * v);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int it = 0; it < kScoreStages - 1; ++it)
        issue(it);
    for (int i = threadIdx.x; i < gq * D; i += kScoreThreads)
        s_q[i] = __half2float(__ushort_as_half(ldg_checked(q + bh * gq * D + i)));
    __syncthreads();
#pragma unroll 1
    for (int it = 0;; ++it) {
        const int now = first + (it * kScoreWarps + warp) * NG;
        if (now >= end)
            break;
        issue(it + kScoreStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 1) : "memory");
        // a lane reads what it copied itself
        const uint8_t* src = mine + it % kScoreStages * kScoreStage;
        float l[NG][CPL], hi[NG][CPL];
#pragma unroll
        for (int k = 0; k < NG; ++k)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                using Vec = typename std::conditional<V == 4, float4, float2>::type;
                const Vec z = *reinterpret_cast<const Vec*>(src + (2 * k * NV + v) * kPiece);
                const Vec s = *reinterpret_cast<const Vec*>(src + ((2 * k + 1) * NV + v) * kPiece);
                const float* zp = reinterpret_cast<const float*>(&z);
                const float* sp = reinterpret_cast<const float*>(&s);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    hi[k][V * v + i] = __fadd_rn(zp[i], __fmul_rn(sp[i], M));
                    l[k][V * v + i] = min_nan(zp[i], hi[k][V * v + i]);
                }
            }
        float best = 0.0f;
#pragma unroll 1
        for (int h = 0; h < gq; ++h) {
            float x[CPL];
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                x[i] = s_q[h * D + lane * CPL + i];
            float t[NG];
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                float y[CPL];
#pragma unroll
                for (int i = 0; i < CPL; ++i)
                    y[i] = __fmul_rn(x[i], x[i] >= 0.0f ? hi[k][i] : l[k][i]);
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
            best = h == 0 ? t[0] : max_nan(best, t[0]);
        }
        int k = 0;  // the group that this lane holds
#pragma unroll
        for (int o = 1, half = NG / 2; half > 0; o <<= 1, half /= 2)
            k += lane & o ? half : 0;
        if (lane < NG && now + k < nb)
            st_checked(scores + bh * NB + now + k, best);
    }
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
// histogram in shared memory and one warp's scan of it, with up to T K keys in
// registers throughout (a longer row reads its scores again).
template <class P>
__global__ void __launch_bounds__(P::T)
block_pick_kernel(kivi_cache c, const float* __restrict__ scores, int32_t* __restrict__ blocks, int n_keep)
{
    constexpr int T = P::T, W = T / 32, K = P::K;
    static_assert(W * K <= 64, "scan_words takes 64 counters");
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
        for (int i = tid; i < 256; i += T)
            hist[i] = 0;
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

template <int D>
static cudaError_t launch_score(const kivi_cache& c, dim3 grid, int smem, const uint16_t* q, int gq, int iters,
                                float M, float* scores, cudaStream_t s)
{
    static int allowed[64];
    const cudaError_t e = allow_smem(block_score_kernel<D>, kScoreRing + 16 * D * 4, allowed);
    if (e != cudaSuccess)
        return e;
    block_score_kernel<D><<<grid, kScoreThreads, smem, s>>>(c, q, gq, iters, M, scores);
    return cudaGetLastError();
}

cudaError_t launch_block_select(const kivi_cache& c, const uint16_t* q, int Hq, int32_t* blocks, int n_keep,
                                float* scores, cudaStream_t s)
{
    const int NB = c.Tmax / c.G, BH = c.B * c.H;
    KIVI_SET_CHECK_RANGES(c, s, {{q, (size_t)c.B * Hq * c.D * 2}, {blocks, (size_t)BH * n_keep * 4},
                                 {scores, (size_t)BH * NB * 4}});
    // A row's groups go to equal chunks: as many as keep two CTAs an SM busy once,
    // with eight steps of a warp at most.
    const int units = (NB + score_groups(c.D) * kScoreWarps - 1) / (score_groups(c.D) * kScoreWarps);
    const long long waves = ((long long)BH * units + 2 * sm_count() - 1) / (2 * sm_count());
    const int most = (int)std::min(8ll, waves), iters = (units + (units + most - 1) / most - 1) / ((units + most - 1) / most);
    const dim3 grid((unsigned)BH * (unsigned)((units + iters - 1) / iters));
    const int gq = Hq / c.H, smem = kScoreRing + gq * c.D * 4;
    const float M = (float)((1 << c.bits_k) - 1);
    cudaError_t e;
    switch (c.D) {
    case 64: e = launch_score<64>(c, grid, smem, q, gq, iters, M, scores, s); break;
    case 128: e = launch_score<128>(c, grid, smem, q, gq, iters, M, scores, s); break;
    default: e = launch_score<256>(c, grid, smem, q, gq, iters, M, scores, s); break;
    }
    if (e != cudaSuccess)
        return e;
    // the choice's CTAs are scheduled while the scores drain
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(BH);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // A warp's registers hold a row of up to 512 groups.  With many rows a warp a
    // row takes less of the machine, with few a CTA a row is sooner done.  Both
    // kernels in us, a warp against a CTA a row, D = 128:
    //     rows             4          608         640        2048
    //     64 groups    9.2/7.2   17.7/13.3   16.1/17.9   38.3/46.3
    //     256 groups  11.9/7.5   39.4/32.7   41.2/37.5   94.4/99.7
    //     500 groups  15.7/7.9   66.4/55.1   68.6/61.5   170/172
    // The border, four rows an SM, is the one of short rows.
    if (NB <= PickWarp::T * PickWarp::K && BH > 4 * sm_count()) {
        cfg.blockDim = dim3(PickWarp::T);
        return cudaLaunchKernelEx(&cfg, block_pick_kernel<PickWarp>, c, (const float*)scores, blocks, n_keep);
    }
    cfg.blockDim = dim3(PickCta::T);
    return cudaLaunchKernelEx(&cfg, block_pick_kernel<PickCta>, c, (const float*)scores, blocks, n_keep);
}

#ifdef KIVI_CHECKS
int32_t check_word_select() { return take_check_word(); }
#endif

}  // namespace kivi
