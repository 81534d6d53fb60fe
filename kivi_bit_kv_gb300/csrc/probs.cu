// probs.cu -- probabilities of rows of logits, one temperature per sequence
// (kivi_token_probs).
//
// A row is read once into the registers of a cluster of CTAs: each thread keeps a
// running maximum and sum of its own values, the pairs are joined over warp, CTA and
// cluster, and the quotients are written from the registers.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <limits.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

namespace cg = cooperative_groups;

constexpr int kProbsThreads = 512, kProbsWarps = kProbsThreads / 32;
constexpr int kProbsCluster = 8;  // most CTAs of a row

// log2(e) / T as hi + lo with lo > 0, so that a distance of -infinity gives
// -infinity through both.  An infinite T gives equal weights to all finite logits, a
// tiny one only to the largest: hi stays between the smallest normal and the largest
// finite number.  NaN for a NaN T.
struct Scale {
    float hi, lo;
};
__device__ __forceinline__ Scale inverse_temperature(float T)
{
    constexpr double kLog2e = 1.44269504088896340736;
    constexpr float L = 1.44269502f;  // below log2(e)
    static_assert((double)L < kLog2e, "");
    if (isinf(T))
        return {0x1p-126f, 0x1p-149f};
    const float hi = fmaxf(__fdiv_rz(L, T), 0x1p-126f);
    const float lo = __fdiv_rn(__fmaf_rn(-hi, T, L) + (float)(kLog2e - (double)L), T);
    return {isnan(T) ? T : hi, fminf(fmaxf(lo, 0x1p-149f), hi * 0x1p-22f)};
}

__device__ __forceinline__ float exp2_ftz(float y)
{
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(y));
    return w;
}

// Two fp32 values in one operation.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 pack2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 both(float a) { return pack2(a, a); }

// Scale and reference of a row as the loops below use them, twice each.
struct Scale2 {
    F2 hi, lo, minus_ref;
};
__device__ __forceinline__ Scale2 twice(Scale c, float ref) { return {both(c.hi), both(c.lo), both(-ref)}; }

// 2^(d (hi + lo)) of distances d = l - ref <= 0 from the largest logit; NaN for a NaN
// d, 0 for -infinity.  For sums, whose terms' roundings cancel.
__device__ __forceinline__ F2 weights_sum(F2 l, const Scale2& c)
{
    const F2 d = add2(l, c.minus_ref);
    const float2 y = unpack2(fma2(d, c.lo, mul2(d, c.hi)));
    return pack2(exp2_ftz(y.x), exp2_ftz(y.y));
}

// The same times f, with the rounding of the exponent (half a unit of 2^-24 of up to
// 126) made good: 2^(y + e) = 2^y (1 + e ln 2).  e is NaN or infinite only where 2^y
// is 0 or where the row's sum, and so f, is NaN.
__device__ __forceinline__ F2 weights(F2 l, const Scale2& c, F2 f)
{
    const F2 d = add2(l, c.minus_ref);
    const float2 y = unpack2(mul2(d, c.hi));
    const float2 e = unpack2(fma2(d, c.lo, fma2(d, c.hi, pack2(-y.x, -y.y))));
    const F2 w = mul2(pack2(exp2_ftz(y.x), exp2_ftz(y.y)), f);
    return fma2(w, mul2(pack2(fminf(e.x, 1.0f), fminf(e.y, 1.0f)), both(0.693147181f)), w);
}
__device__ __forceinline__ float weight(float d, Scale c)
{
    return unpack2(weights(both(d), twice(c, 0.0f), both(1.0f))).x;
}

// Four neighbouring logits as loaded: pair(i) in fp32.
template <class T>
struct Raw4 {
    uint2 v;
    __device__ __forceinline__ void load(const T* p)
    {
        if (KIVI_IN_RANGE(p, 8))
            v = __ldg(reinterpret_cast<const uint2*>(p));
    }
    __device__ __forceinline__ void load_each(const T* p)
    {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        v.x = ldg_checked(q) | (uint32_t)ldg_checked(q + 1) << 16;
        v.y = ldg_checked(q + 2) | (uint32_t)ldg_checked(q + 3) << 16;
    }
    __device__ __forceinline__ void clear()  // to -infinity
    {
        constexpr uint32_t w = std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
        v = make_uint2(w, w);
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        const uint32_t w = i ? v.y : v.x;
        if constexpr (std::is_same<T, __half>::value)
            return __half22float2(as_h2(w));
        else
            return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <>
struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = ld_nc_f4(p); }
    __device__ __forceinline__ void load_each(const float* p)
    {
        v = make_float4(ldg_checked(p), ldg_checked(p + 1), ldg_checked(p + 2), ldg_checked(p + 3));
    }
    __device__ __forceinline__ void clear() { v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ float2 pair(int i) const { return i ? make_float2(v.z, v.w) : make_float2(v.x, v.y); }
};
template <class T>
__device__ __forceinline__ float largest(const Raw4<T>& v)
{
    const float2 a = v.pair(0), b = v.pair(1);
    return fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
}
template <class T>
__device__ __forceinline__ F2 pair2(const Raw4<T>& v, int i)
{
    const float2 f = v.pair(i);
    return pack2(f.x, f.y);
}
// The first of four logits at x .. x + 3 that is m; none is past all of them.
template <class T>
__device__ __forceinline__ int where(const Raw4<T>& v, float m, int x, int none)
{
    const float2 a = v.pair(0), b = v.pair(1);
    return a.x == m ? x : a.y == m ? x + 1 : b.x == m ? x + 2 : b.y == m ? x + 3 : none;
}
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// A largest logit, the sum of weights relative to it, and where it is first met
// (found for temperature 0 alone).
struct Stat {
    float m, l;
    int first;
};
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }
// Of all lanes.
__device__ __forceinline__ Stat join(Stat s, Scale c, bool greedy)
{
    float m = s.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = s.l * weight(s.m - reference(m), c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, o);
    int first = s.first;
    if (greedy)
        first = __reduce_min_sync(0xffffffffu, s.m == m ? s.first : INT_MAX);
    return {m, l, first};
}

struct ProbsSmem {
    Stat warp[kProbsWarps], slot[kProbsCluster];
};

// A cluster per row; CTA r takes the row's vectors of four logits [r per, (r + 1) per),
// the last one also the up to three logits after them.  The first NV vectors of a
// thread stay in registers, what lies beyond is read again.  The order of a row's sum
// does not depend on where the row lies.
template <class T, int NV>
__global__ void __launch_bounds__(kProbsThreads, 2)
token_probs_kernel(ProbsArgs a, int per)
{
    __shared__ ProbsSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = (int)(blockIdx.x / C), b = row / a.N, i = row % a.N;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, V = a.V;
    // Every CTA comes to both barriers and does the same between them whatever it
    // reads; one of a row that is left as it is has no logits.
    const bool left = a.n_rows && i >= ldg_checked(a.n_rows + b);
    auto arrived = cluster.barrier_arrive();  // this CTA's shared memory may be written
    const T* src = static_cast<const T*>(a.logits) + b * a.batch_stride + i * a.row_stride;
    float* dst = a.probs + (size_t)row * V;
    const int nvec = V / 4;
    const int j0 = left ? nvec : min(rank * per, nvec), j1 = min(j0 + per, nvec);
    const bool aligned = ((uintptr_t)src & (4 * sizeof(T) - 1)) == 0;
    auto load = [&](int j) {
        Raw4<T> v;
        if (j >= j1)
            v.clear();
        else if (aligned)
            v.load(src + 4 * j);
        else
            v.load_each(src + 4 * j);
        return v;
    };
    Raw4<T> keep[NV];
#pragma unroll
    for (int r = 0; r < NV; ++r)
        keep[r] = load(j0 + tid + r * kProbsThreads);
    const int edge = 4 * nvec + tid;  // one of the logits after the vectors
    const bool has_edge = !left && rank == C - 1 && edge < V;
    const float edge_l = has_edge ? to_float(ldg_checked(src + edge)) : -INFINITY;
    const float temp = a.temperature ? ldg_checked(a.temperature + b) : 1.0f;
    const bool greedy = temp <= 0.0f;
    const Scale c = inverse_temperature(greedy ? 1.0f : temp);
    Stat s = {edge_l, 0.0f, has_edge ? edge : INT_MAX};
#pragma unroll
    for (int r = 0; r < NV; ++r)
        if (j0 + r * kProbsThreads < j1)
            s.m = fmaxf(s.m, largest(keep[r]));
    {
        const Scale2 c2 = twice(c, reference(s.m));
        F2 l = weights_sum(pack2(edge_l, -INFINITY), c2);
#pragma unroll
        for (int r = 0; r < NV; ++r)
            if (j0 + r * kProbsThreads < j1) {
                l = add2(l, weights_sum(pair2(keep[r], 0), c2));
                l = add2(l, weights_sum(pair2(keep[r], 1), c2));
            }
        s.l = unpack2(l).x + unpack2(l).y;
    }
    if (greedy) {
        s.first = s.m == edge_l ? s.first : INT_MAX;
#pragma unroll
        for (int r = 0; r < NV; ++r)
            s.first = min(s.first, where(keep[r], s.m, 4 * (j0 + tid + r * kProbsThreads), INT_MAX));
    }
    for (int j = j0 + tid + NV * kProbsThreads; j < j1; j += kProbsThreads) {
        const Raw4<T> v = load(j);
        const float m = fmaxf(s.m, largest(v));
        const int x = where(v, m, 4 * j, INT_MAX);
        const Scale2 c2 = twice(c, reference(m));
        const float2 l = unpack2(add2(weights_sum(pair2(v, 0), c2), weights_sum(pair2(v, 1), c2)));
        s = {m, s.l * weight(s.m - reference(m), c) + (l.x + l.y), m == s.m ? min(s.first, x) : x};
    }
    s = join(s, c, greedy);
    if (lane == 0)
        sm.warp[warp] = s;
    __syncthreads();
    s = join(lane < kProbsWarps ? sm.warp[lane] : Stat{-INFINITY, 0.0f, INT_MAX}, c, greedy);
    cluster.barrier_wait(std::move(arrived));
    if (tid < C)
        cluster.map_shared_rank(&sm, tid)->slot[rank] = s;
    cluster.sync();
    s = join(lane < C ? sm.slot[lane] : Stat{-INFINITY, 0.0f, INT_MAX}, c, greedy);
    // Outputs of vector j of this lane; all lanes have neighbouring vectors.  Where an
    // aligned vector begins with output `ahead` of them, its end is the next lane's.
    const int ahead = (int)((0 - (uintptr_t)dst / 4) & 3);
    auto store = [&](int j, F2 p, F2 q) {
        const float2 x = unpack2(p), y = unpack2(q);
        float4 v = make_float4(x.x, x.y, y.x, y.y);
        float* to = dst + 4 * j;
        if (ahead != 0) {  // the same for the whole row
            const float4 n = make_float4(__shfl_down_sync(0xffffffffu, v.x, 1), __shfl_down_sync(0xffffffffu, v.y, 1),
                                         __shfl_down_sync(0xffffffffu, v.z, 1), 0.0f);
            const bool last = lane == 31 || j + 1 == j1;
            if (j < j1) {
                if (lane == 0 || last) {
                    if (lane == 0 ? true : ahead < 1)
                        st_checked(to, v.x);
                    if (lane == 0 ? ahead > 1 || last : last && ahead <= 1)
                        st_checked(to + 1, v.y);
                    if (lane == 0 ? ahead > 2 || last : last && ahead <= 2)
                        st_checked(to + 2, v.z);
                    if (last)
                        st_checked(to + 3, v.w);
                }
                if (last)
                    return;
            }
            v = ahead == 1 ? make_float4(v.y, v.z, v.w, n.x)
                           : ahead == 2 ? make_float4(v.z, v.w, n.x, n.y) : make_float4(v.w, n.x, n.y, n.z);
            to += ahead;
        }
        if (j < j1 && KIVI_IN_RANGE(to, 16))
            __stcs(reinterpret_cast<float4*>(to), v);
    };
    if (greedy) {
        const float zero = isnan(s.l) ? s.l : 0.0f, one = s.l == 0.0f ? 0.0f : 1.0f + zero;
        for (int base = j0; base < j1; base += kProbsThreads) {
            const int j = base + tid, x = 4 * j;
            store(j, pack2(x == s.first ? one : zero, x + 1 == s.first ? one : zero),
                  pack2(x + 2 == s.first ? one : zero, x + 3 == s.first ? one : zero));
        }
        if (has_edge)
            st_checked(dst + edge, edge == s.first ? one : zero);
        return;
    }
    const Scale2 c2 = twice(c, reference(s.m));
    const F2 inv = both(s.l == 0.0f ? 0.0f : 1.0f / s.l);  // NaN for a NaN sum
#pragma unroll
    for (int r = 0; r < NV; ++r)
        if (j0 + r * kProbsThreads < j1)
            store(j0 + tid + r * kProbsThreads, weights(pair2(keep[r], 0), c2, inv), weights(pair2(keep[r], 1), c2, inv));
    for (int base = j0 + NV * kProbsThreads; base < j1; base += kProbsThreads) {
        const int j = base + tid;
        const Raw4<T> v = load(j);
        store(j, weights(pair2(v, 0), c2, inv), weights(pair2(v, 1), c2, inv));
    }
    if (has_edge)
        st_checked(dst + edge, unpack2(weights(both(edge_l), c2, inv)).x);
}

#ifdef KIVI_CHECKS
static size_t extent(const ProbsArgs& a)
{
    const int64_t last = (a.B > 1 ? (a.B - 1) * a.batch_stride : 0) + (a.N > 1 ? (a.N - 1) * a.row_stride : 0) + a.V;
    return (size_t)last * (a.dtype == KIVI_F32 ? 4 : 2);
}
#endif

template <class T, int NV>
static cudaError_t launch_probs(const ProbsArgs& a, cudaStream_t s)
{
    const long long rows = (long long)a.B * a.N;
    const int nvec = a.V / 4;
    int C = 1;
    while (C < kProbsCluster && (nvec > C * NV * kProbsThreads || (rows * C < 2 * sm_count() && nvec > C * kProbsThreads)))
        C *= 2;
    const int per = ((nvec + C - 1) / C + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kProbsThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, token_probs_kernel<T, NV>, a, per);
}

cudaError_t launch_token_probs(const ProbsArgs& a, cudaStream_t s)
{
    KIVI_SET_CHECK_BUFFERS(s, {{a.logits, extent(a)}, {a.temperature, (size_t)a.B * 4}, {a.n_rows, (size_t)a.B * 4},
                               {a.probs, (size_t)a.B * a.N * a.V * 4}});
    switch (a.dtype) {
    case KIVI_F16: return launch_probs<__half, 16>(a, s);
    case KIVI_BF16: return launch_probs<__nv_bfloat16, 16>(a, s);
    default: return launch_probs<float, 8>(a, s);
    }
}

#ifdef KIVI_CHECKS
int32_t check_word_probs() { return take_check_word(); }
#endif

}  // namespace kivi
