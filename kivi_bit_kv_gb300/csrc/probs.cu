// probs.cu -- probabilities of rows of logits, one temperature per sequence
// (kivi_token_probs).
//
// A row is read once, into the shared memory of a cluster of CTAs: each thread keeps a
// running maximum and sum of its own values, the pairs are joined over the cluster, and
// the quotients are formed from the values kept.
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

constexpr int kProbsThreads = 256, kProbsWarps = kProbsThreads / 32, kProbsCtas = 5;
constexpr int kProbsCluster = 8;    // most CTAs of a row
constexpr int kProbsBytes = 32768;  // shared memory for a CTA's logits

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
    F2 hi, lo, minus_ref, minus_hi, minus_lo;
};
__device__ __forceinline__ Scale2 twice(Scale c, float ref)
{
    return {both(c.hi), both(c.lo), both(-ref), both(-c.hi), both(-c.lo)};
}

// 2^(d (hi + lo)) of distances d = l - ref <= 0 from the largest logit; NaN for a NaN
// d, 0 for -infinity.  For sums, whose terms' roundings cancel.
__device__ __forceinline__ F2 weights_sum(F2 l, const Scale2& c)
{
    const F2 d = add2(l, c.minus_ref);
    const float2 y = unpack2(fma2(d, c.lo, mul2(d, c.hi)));
    return pack2(exp2_ftz(y.x), exp2_ftz(y.y));
}

// The same times f, with the rounding of the exponent (half a unit of 2^-24 of up to
// 126) made good: 2^(y + e) = 2^y (1 + e ln 2).  -e is NaN or infinite only where 2^y
// is 0 or where the row's sum, and so f, is NaN.
__device__ __forceinline__ F2 weights(F2 l, const Scale2& c, F2 f)
{
    const F2 d = add2(l, c.minus_ref), y = mul2(d, c.hi);
    const float2 e = unpack2(fma2(d, c.minus_lo, fma2(d, c.minus_hi, y)));
    const F2 w = mul2(pack2(exp2_ftz(unpack2(y).x), exp2_ftz(unpack2(y).y)), f);
    return fma2(w, mul2(pack2(fmaxf(e.x, -1.0f), fmaxf(e.y, -1.0f)), both(-0.693147181f)), w);
}
__device__ __forceinline__ float weight(float d, Scale c)
{
    return unpack2(weights(both(d), twice(c, 0.0f), both(1.0f))).x;
}

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// Four neighbouring logits: pair(i) in fp32.
template <class T>
struct Raw4 {
    uint2 v;
    static constexpr int BYTES = 8;
    __device__ __forceinline__ void load_each(const T* p)
    {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        v.x = ldg_checked(q) | (uint32_t)ldg_checked(q + 1) << 16;
        v.y = ldg_checked(q + 2) | (uint32_t)ldg_checked(q + 3) << 16;
    }
    // From the two aligned vectors that hold them, `mis` logits into the first.
    __device__ __forceinline__ void load_shifted(const T* p, int mis)
    {
        const uint2* q = reinterpret_cast<const uint2*>(p - mis);
        const uint2 a = ldg_checked(q), b = ldg_checked(q + 1);
        const unsigned long long lo = (unsigned long long)a.y << 32 | a.x, hi = (unsigned long long)b.y << 32 | b.x;
        const unsigned long long w = lo >> (16 * mis) | hi << (64 - 16 * mis);
        v = make_uint2((uint32_t)w, (uint32_t)(w >> 32));
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
    static constexpr int BYTES = 16;
    __device__ __forceinline__ void load_each(const float* p)
    {
        v = make_float4(ldg_checked(p), ldg_checked(p + 1), ldg_checked(p + 2), ldg_checked(p + 3));
    }
    __device__ __forceinline__ void load_shifted(const float* p, int) { load_each(p); }
    __device__ __forceinline__ void clear() { v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ float2 pair(int i) const { return i ? make_float2(v.z, v.w) : make_float2(v.x, v.y); }
};
// An aligned vector on its way to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_vector(void* dst, const void* src)
{
    if (KIVI_IN_RANGE(src, BYTES)) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
        if constexpr (BYTES == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(src) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(src) : "memory");
    }
}
// The largest logit of U vectors, NaN apart.
template <class T, int U>
__device__ __forceinline__ float largest(const Raw4<T> (&v)[U])
{
    if constexpr (std::is_same<T, float>::value) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
            m = fmaxf(fmaxf(m, fmaxf(v[u].v.x, v[u].v.y)), fmaxf(v[u].v.z, v[u].v.w));
        return m;
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        T2 m = *reinterpret_cast<const T2*>(&v[0].v.x);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u)
                m = __hmax2(m, *reinterpret_cast<const T2*>(&v[u].v.x));
            m = __hmax2(m, *reinterpret_cast<const T2*>(&v[u].v.y));
        }
        const float a = to_float(m.x), b = to_float(m.y);
        return fmaxf(fmaxf(a, b), -INFINITY);  // -infinity for NaN alone
    }
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

// A largest logit, the sum of weights relative to it, and where it is first met
// (found for temperature 0 alone).
struct Stat {
    float m, l;
    int first;
};
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }
// Whole numbers in the order of finite and infinite fp32 values.
__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
// Of all lanes.
__device__ __forceinline__ Stat join(Stat s, Scale c, bool greedy)
{
    const int top = __reduce_max_sync(0xffffffffu, ordered(s.m + 0.0f));
    const float m = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
    float l = s.l * weight(s.m - reference(m), c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, o);
    int first = s.first;
    if (greedy)
        first = __reduce_min_sync(0xffffffffu, s.m == m ? s.first : INT_MAX);
    return {m, l, first};
}

// A cluster per row; CTA r takes the row's vectors of four logits [r per, (r + 1) per),
// the last one also the up to three logits after them.  The first `room` vectors of a
// CTA stay in its shared memory, what lies beyond is read again.  The order of a row's
// sum does not depend on where the row lies.
template <class T>
__global__ void __launch_bounds__(kProbsThreads, kProbsCtas)
token_probs_kernel(ProbsArgs a, int per, int room)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ Stat s_stat[kProbsCluster * kProbsWarps];  // of all warps of the cluster
    Raw4<T>* const kept = reinterpret_cast<Raw4<T>*>(s_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = (int)(blockIdx.x / C), b = row / a.N, i = row % a.N;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, V = a.V;
    auto arrived = cluster.barrier_arrive();  // this CTA's shared memory may be written
    // Every CTA comes to both barriers and does the same between them whatever it
    // reads; one of a row that is left as it is has no logits.
    const bool left = a.n_rows && i >= ldg_checked(a.n_rows + b);
    const T* src = static_cast<const T*>(a.logits) + b * a.batch_stride + i * a.row_stride;
    float* dst = a.probs + (size_t)row * V;
    const int nvec = V / 4, j0 = left ? nvec : min(rank * per, nvec), j1 = min(j0 + per, nvec), jr = min(j0 + room, j1);
    const int mis = (int)(((uintptr_t)src / sizeof(T)) & 3);  // logits past an aligned vector
    if (mis == 0) {
#pragma unroll 4
        for (int j = j0 + tid; j < jr; j += kProbsThreads)
            copy_vector<Raw4<T>::BYTES>(kept + (j - j0), src + 4 * j);
    } else {
#pragma unroll 4
        for (int j = j0 + tid; j < jr; j += kProbsThreads) {
            Raw4<T> v;
            if (j > 0 && 4 * j + 8 - mis <= V)
                v.load_shifted(src + 4 * j, mis);
            else
                v.load_each(src + 4 * j);
            kept[j - j0] = v;
        }
    }
    const int edge = 4 * nvec + tid;  // one of the logits after the vectors
    const bool has_edge = !left && rank == C - 1 && edge < V;
    const float edge_l = has_edge ? to_float(ldg_checked(src + edge)) : -INFINITY;
    const float temp = a.temperature ? ldg_checked(a.temperature + b) : 1.0f;
    const bool greedy = temp <= 0.0f;
    const Scale c = inverse_temperature(greedy ? 1.0f : temp);
    // The U vectors of this thread from j on; -infinity past the end of the CTA's.
    constexpr int U = 4;
    auto fetch = [&](int j, Raw4<T> (&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = j + u * kProbsThreads;
            if (x < jr)
                v[u] = kept[x - j0];
            else if (x < j1)
                v[u].load_each(src + 4 * x);
            else
                v[u].clear();
        }
    };
    Stat s = {-INFINITY, 0.0f, INT_MAX};
    asm volatile("cp.async.wait_all;" ::: "memory");  // a thread reads what it copied itself
    auto take = [&](const Raw4<T> (&v)[U], int j) {
        const float m = largest(v);
        if (m > s.m) {
            s.l *= weight(s.m - m, c);
            s.m = m;
            if (greedy) {
                s.first = INT_MAX;
#pragma unroll
                for (int u = U - 1; u >= 0; --u)
                    s.first = where(v[u], m, 4 * (j + u * kProbsThreads), s.first);
            }
        }
        const Scale2 c2 = twice(c, reference(s.m));
        F2 l = weights_sum(pair2(v[0], 0), c2);
        l = add2(l, weights_sum(pair2(v[0], 1), c2));
#pragma unroll
        for (int u = 1; u < U; ++u) {
            l = add2(l, weights_sum(pair2(v[u], 0), c2));
            l = add2(l, weights_sum(pair2(v[u], 1), c2));
        }
        s.l += unpack2(l).x + unpack2(l).y;
    };
    // chunks of all threads' U vectors each that are kept, then the rest
    const int chunks = (jr - j0) / (U * kProbsThreads), jc = j0 + chunks * U * kProbsThreads;
#pragma unroll 1
    for (int j = tid; j < chunks * U * kProbsThreads; j += U * kProbsThreads) {
        Raw4<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = kept[j + u * kProbsThreads];
        take(v, j0 + j);
    }
#pragma unroll 1
    for (int j = jc + tid; j < j1; j += U * kProbsThreads) {
        Raw4<T> v[U];
        fetch(j, v);
        take(v, j);
    }
    if (has_edge) {  // a thread's last logit
        const float m = fmaxf(s.m, edge_l), r = reference(m);
        s = {m, s.l * weight(s.m - r, c) + weight(edge_l - r, c), edge_l > s.m ? edge : s.first};
    }
    s = join(s, c, greedy);
    cluster.barrier_wait(std::move(arrived));
    if (lane < C)
        cluster.map_shared_rank(s_stat, lane)[rank * kProbsWarps + warp] = s;
    cluster.sync();
    s = {-INFINITY, 0.0f, INT_MAX};
    for (int k = lane; k < C * kProbsWarps; k += 32) {
        const Stat t = s_stat[k];
        const float m = fmaxf(s.m, t.m), r = reference(m);
        s = {m, s.l * weight(s.m - r, c) + t.l * weight(t.m - r, c),
             s.m == t.m ? min(s.first, t.first) : s.m > t.m ? s.first : t.first};
    }
    s = join(s, c, greedy);
    // Outputs of vector j of this lane; all lanes have neighbouring vectors.  Where an
    // aligned vector begins with output AHEAD of them, its end is the next lane's.
    const int ahead = (int)((0 - (uintptr_t)dst / 4) & 3);
    auto store = [&](auto known, int j, F2 p, F2 q) {
        constexpr int AHEAD = decltype(known)::value;
        const float2 x = unpack2(p), y = unpack2(q);
        float o[8] = {x.x, x.y, y.x, y.y};
        bool whole = j < j1;
        if constexpr (AHEAD > 0) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                o[4 + k] = __shfl_down_sync(0xffffffffu, o[k], 1);
            const bool last = lane == 31 || j + 1 == j1;
            if (whole && (lane == 0 || last)) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < AHEAD ? lane == 0 : last)
                        st_checked(dst + 4 * j + k, o[k]);
            }
            whole = whole && !last;
        }
        if (whole && KIVI_IN_RANGE(dst + 4 * j + AHEAD, 16))
            __stcs(reinterpret_cast<float4*>(dst + 4 * j + AHEAD),
                   make_float4(o[AHEAD], o[AHEAD + 1], o[AHEAD + 2], o[AHEAD + 3]));
    };
    auto by_alignment = [&](auto all) {
        switch (ahead) {
        case 0: all(std::integral_constant<int, 0>()); break;
        case 1: all(std::integral_constant<int, 1>()); break;
        case 2: all(std::integral_constant<int, 2>()); break;
        default: all(std::integral_constant<int, 3>()); break;
        }
    };
    if (greedy) {
        const float zero = isnan(s.l) ? s.l : 0.0f, one = s.l == 0.0f ? 0.0f : 1.0f + zero;
        by_alignment([&](auto known) {
#pragma unroll 1
            for (int base = j0; base < j1; base += kProbsThreads) {
                const int j = base + tid, x = 4 * j;
                store(known, j, pack2(x == s.first ? one : zero, x + 1 == s.first ? one : zero),
                      pack2(x + 2 == s.first ? one : zero, x + 3 == s.first ? one : zero));
            }
        });
        if (has_edge)
            st_checked(dst + edge, edge == s.first ? one : zero);
        return;
    }
    const Scale2 c2 = twice(c, reference(s.m));
    const F2 inv = both(s.l == 0.0f ? 0.0f : 1.0f / s.l);  // NaN for a NaN sum
    if (ahead == 0) {
        float* to = dst + 4 * (j0 + tid);
#pragma unroll 1
        for (int j = tid; j < chunks * U * kProbsThreads; j += U * kProbsThreads, to += 4 * U * kProbsThreads) {
            Raw4<T> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = kept[j + u * kProbsThreads];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float2 x = unpack2(weights(pair2(v[u], 0), c2, inv)), y = unpack2(weights(pair2(v[u], 1), c2, inv));
                if (KIVI_IN_RANGE(to + 4 * u * kProbsThreads, 16))
                    __stcs(reinterpret_cast<float4*>(to + 4 * u * kProbsThreads), make_float4(x.x, x.y, y.x, y.y));
            }
        }
    }
    by_alignment([&](auto known) {
#pragma unroll 1
        for (int base = decltype(known)::value == 0 ? jc : j0; base < j1; base += U * kProbsThreads) {
            Raw4<T> v[U];
            fetch(base + tid, v);
#pragma unroll
            for (int u = 0; u < U; ++u)
                store(known, base + tid + u * kProbsThreads, weights(pair2(v[u], 0), c2, inv),
                      weights(pair2(v[u], 1), c2, inv));
        }
    });
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

template <class T>
static cudaError_t launch_probs(const ProbsArgs& a, cudaStream_t s)
{
    constexpr int kMost = kProbsBytes / Raw4<T>::BYTES;  // vectors a CTA keeps
    static int allowed[64];
    const cudaError_t e = allow_smem(token_probs_kernel<T>, kProbsBytes, allowed);
    if (e != cudaSuccess)
        return e;
    const long long rows = (long long)a.B * a.N;
    const int nvec = a.V / 4;
    int C = 1;
    while (C < kProbsCluster && (nvec > C * kMost || (rows * C < 2 * sm_count() && nvec > C * kProbsThreads)))
        C *= 2;
    const int per = ((nvec + C - 1) / C + 31) / 32 * 32, room = std::min(per, kMost);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kProbsThreads);
    cfg.dynamicSmemBytes = (size_t)room * Raw4<T>::BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, token_probs_kernel<T>, a, per, room);
}

cudaError_t launch_token_probs(const ProbsArgs& a, cudaStream_t s)
{
    KIVI_SET_CHECK_BUFFERS(s, {{a.logits, extent(a)}, {a.temperature, (size_t)a.B * 4}, {a.n_rows, (size_t)a.B * 4},
                               {a.probs, (size_t)a.B * a.N * a.V * 4}});
    switch (a.dtype) {
    case KIVI_F16: return launch_probs<__half>(a, s);
    case KIVI_BF16: return launch_probs<__nv_bfloat16>(a, s);
    default: return launch_probs<float>(a, s);
    }
}

#ifdef KIVI_CHECKS
int32_t check_word_probs() { return take_check_word(); }
#endif

}  // namespace kivi
