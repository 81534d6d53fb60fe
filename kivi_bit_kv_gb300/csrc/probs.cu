// probs.cu -- probabilities of rows of logits, one temperature per sequence
// (kivi_token_probs).
//
// A row is read into the shared memory of a cluster of CTAs: each thread keeps a running
// maximum and sum of its own values, the pairs are joined over the cluster, and the
// quotients are formed from the values kept.  What the shared memory of sixteen CTAs does
// not hold (of rows above 131072 fp32 or 262144 16-bit values) is read again for them.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <limits.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "kivi_device.cuh"
#include "kivi_f32x2.cuh"
#include "kivi_launch.h"

namespace kivi {

namespace cg = cooperative_groups;

// 128 threads a CTA, six CTAs an SM.  In us for 512 rows of 131072 bf16 logits (128 x 6;
// 5 or 7 CTAs are within 1 %): 256 x 5 73, 512 x 2 77, 1024 x 1 84, 64 x 6 76.  A CTA for
// one row, without the walk over rows, took 74 (256 threads); clusters of four with
// twice the shared memory 74.
constexpr int kProbsThreads = 128, kProbsWarps = kProbsThreads / 32, kProbsCtas = 6;
constexpr int kProbsCluster = 16;   // most CTAs of a row
constexpr int kProbsBytes = 32768;  // logits a CTA keeps in shared memory

// A distance d = l - ref <= 0 of a logit from the largest weighs 2^(d log2(e) / T).  Where T
// is far from 1 the distance is formed as `unit` times itself, unit a power of two, and
// log2(e) / (unit T) taken, so that neither leaves the range of fp32: from 2^100 on logits
// near both ends of the range have a finite distance, below 2^-100 the quotient is finite.
// log2(e) / (unit T) as hi + lo with lo > 0, so that a distance of -infinity gives -infinity
// through both.  With an infinite T all finite distances (below 2^65 in their unit) weigh
// 2^-0.  NaN for a NaN T.
struct Scale {
    float hi, lo, unit;
};
__device__ __forceinline__ Scale inverse_temperature(float T)
{
    constexpr double kLog2e = 1.44269504088896340736;
    constexpr float L = 1.44269502f;  // below log2(e)
    static_assert((double)L < kLog2e, "");
    const float unit = T >= 0x1p100f ? 0x1p-64f : T < 0x1p-100f ? 0x1p64f : 1.0f, t = T * unit;
    const float hi = __fdiv_rz(L, t);
    const float lo = __fdiv_rn(__fmaf_rn(-hi, t, L) + (float)(kLog2e - (double)L), t);
    return isinf(T) ? Scale{0x1p-126f, 0x1p-149f, unit} : Scale{hi, fmaxf(lo, 0x1p-149f), unit};
}
// Distances from ref as l unit + minus.  A large unit is 1 where l would overflow: distances
// other than 0 are 2^36 or more there, and weigh 0.
struct Ref {
    float unit, minus;
};
__device__ __forceinline__ Ref ref_at(const Scale& c, float ref)
{
    const float unit = fabsf(ref) < 0x1p60f ? c.unit : fminf(c.unit, 1.0f);
    return {unit, -ref * unit};
}

__device__ __forceinline__ float exp2_ftz(float y)
{
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(y));
    return w;
}

// Scale and reference of a row as the loops below use them, twice each.
struct Scale2 {
    F2 hi, lo, unit, minus_ref, minus_hi, minus_lo;
    __device__ __forceinline__ F2 distance(F2 l) const { return fma2(l, unit, minus_ref); }
};
__device__ __forceinline__ Scale2 twice(const Scale& c, Ref ref)
{
    return {both(c.hi), both(c.lo), both(ref.unit), both(ref.minus), both(-c.hi), both(-c.lo)};
}

// 2^(d (hi + lo)) of distances d = l - ref <= 0 from the largest logit; NaN for a NaN
// d, 0 for -infinity.  For sums, whose terms' roundings cancel.
__device__ __forceinline__ F2 weights_sum(F2 l, const Scale2& c)
{
    const F2 d = c.distance(l);
    const float2 y = unpack2(fma2(d, c.lo, mul2(d, c.hi)));
    return pack2(exp2_ftz(y.x), exp2_ftz(y.y));
}

// The same times f (1 + rest), with the rounding of the exponent (half a unit of 2^-24 of
// up to 126) made good: 2^(y + e) = 2^y (1 + e ln 2).  -e is NaN or infinite only where
// 2^y is 0 or where the row's sum, and so f, is NaN.
__device__ __forceinline__ F2 weights(F2 l, const Scale2& c, F2 f, F2 rest)
{
    const F2 d = c.distance(l), y = mul2(d, c.hi);
    const float2 e = unpack2(fma2(d, c.minus_lo, fma2(d, c.minus_hi, y)));
    const F2 w = mul2(pack2(exp2_ftz(unpack2(y).x), exp2_ftz(unpack2(y).y)), f);
    return fma2(w, fma2(pack2(fmaxf(e.x, -1.0f), fmaxf(e.y, -1.0f)), both(-0.693147181f), rest), w);
}
// The same of one value with f = 1: the factor between sums relative to l and to ref.  Every
// new maximum waits for it; in single operations it takes 1 to 3 % less of a short row's time.
__device__ __forceinline__ float weight(float l, Ref ref, const Scale& c)
{
    const float d = __fmaf_rn(l, ref.unit, ref.minus), y = __fmul_rn(d, c.hi);
    const float e = __fmaf_rn(d, -c.lo, __fmaf_rn(d, -c.hi, y)), w = exp2_ftz(y);
    return __fmaf_rn(w, __fmul_rn(fmaxf(e, -1.0f), -0.693147181f), w);
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
        v.x = ld_prior(q) | (uint32_t)ld_prior(q + 1) << 16;
        v.y = ld_prior(q + 2) | (uint32_t)ld_prior(q + 3) << 16;
    }
    __device__ __forceinline__ void load(const T* p) { v = ld_prior(reinterpret_cast<const uint2*>(p)); }
    // Four of the eight logits of a and b, from number `skip` (1 to 3) on.
    __device__ __forceinline__ void shifted(const Raw4& a, const Raw4& b, int skip)
    {
        const uint32_t x = skip >= 2 ? a.v.y : a.v.x, y = skip >= 2 ? b.v.x : a.v.y, z = skip >= 2 ? b.v.y : b.v.x;
        const int bits = skip % 2 * 16;
        v = make_uint2(__funnelshift_r(x, y, bits), __funnelshift_r(y, z, bits));
    }
    __device__ __forceinline__ Raw4 of_next_lane() const
    {
        Raw4 r;
        r.v = make_uint2(__shfl_down_sync(0xffffffffu, v.x, 1), __shfl_down_sync(0xffffffffu, v.y, 1));
        return r;
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
        v = make_float4(ld_prior(p), ld_prior(p + 1), ld_prior(p + 2), ld_prior(p + 3));
    }
    __device__ __forceinline__ void load(const float* p) { v = ld_prior(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void clear() { v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ float2 pair(int i) const { return i ? make_float2(v.z, v.w) : make_float2(v.x, v.y); }
};
// Aligned bytes on their way to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_bytes(void* dst, const void* src)
{
    if (KIVI_IN_RANGE(src, BYTES)) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
        if constexpr (BYTES == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(src) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(to), "l"(src), "n"(BYTES) : "memory");
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
__device__ __forceinline__ Stat join(Stat s, const Scale& c, bool greedy)
{
    const int top = __reduce_max_sync(0xffffffffu, ordered(s.m + 0.0f));
    const float m = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
    float l = s.l * weight(s.m, ref_at(c, reference(m)), c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, o);
    int first = s.first;
    if (greedy)
        first = __reduce_min_sync(0xffffffffu, s.m == m ? s.first : INT_MAX);
    return {m, l, first};
}

// Place of a CTA's vector k in its shared memory: the 32 of a warp are followed by one
// more, for rows that are not aligned.
__host__ __device__ constexpr int slot_of(int k) { return k + k / 32; }

// A row's logits as a CTA's threads keep and read them.  A thread reads what it copied
// itself, so it needs no barrier, and its share of the next row is on its way as soon as
// its share of this one has been used.
//   fp32 and aligned rows: slot k holds vector k.
//   16-bit rows that begin `skip` logits past an aligned vector: slot k holds the aligned
// vector with the first of vector k's logits; the rest are in the next one, which the
// next lane has.  The last lane of a warp, and the one with the CTA's last vector, have
// that in the slot after.
template <class T>
struct Kept {
    Raw4<T>* slots;
    int j0, count, V;  // first vector of the CTA, vectors kept, logits of a row

    __device__ __forceinline__ static int skip_of(const T* row) { return (int)(((uintptr_t)row / sizeof(T)) & 3); }
    __device__ __forceinline__ bool reads_slot_after(int k) const { return (threadIdx.x & 31) == 31 || k == count - 1; }

    // an aligned vector of a row from logit x on, of which some may lie outside the row
    __device__ __forceinline__ void copy_aligned(int slot, const T* row, int x) const
    {
        if (x >= 0 && x + 4 <= V) {
            copy_bytes<Raw4<T>::BYTES>(slots + slot, row + x);
        } else {
            T* to = reinterpret_cast<T*>(slots + slot);
            for (int i = 0; i < 4; ++i)
                if (x + i >= 0 && x + i < V)
                    to[i] = ld_prior(row + x + i);
        }
    }
    // vectors n + tid, n + tid + kProbsThreads .. below end
    __device__ __forceinline__ void copy(const T* row, int n, int end) const
    {
        const int skip = skip_of(row);
#pragma unroll 4
        for (int k = n + (int)threadIdx.x; k < end; k += kProbsThreads) {
            const int x = 4 * (j0 + k);
            if (skip == 0) {
                copy_bytes<Raw4<T>::BYTES>(slots + slot_of(k), row + x);
            } else if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    copy_bytes<4>(reinterpret_cast<float*>(slots + slot_of(k)) + i, row + x + i);
            } else {
                copy_aligned(slot_of(k), row, x - skip);
                if (reads_slot_after(k))
                    copy_aligned(slot_of(k) + 1, row, x - skip + 4);
            }
        }
    }
    // the same of U vectors from n + tid on, n a multiple of 32, all below count
    template <int U>
    __device__ __forceinline__ void copy_chunk(const T* row, int n) const
    {
        const int skip = skip_of(row), x = 4 * (j0 + n);
        // the aligned vectors of the whole chunk lie in the row
        const bool inside = sizeof(T) == 2 && x >= skip && x + 4 * U * kProbsThreads + 4 - skip <= V;
        if (skip != 0 && !inside) {
            copy(row, n, n + U * kProbsThreads);
            return;
        }
        Raw4<T>* to = slots + slot_of(threadIdx.x) + slot_of(n);
        const T* from = row + x - skip + 4 * (int)threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u)
            copy_bytes<Raw4<T>::BYTES>(to + slot_of(u * kProbsThreads), from + 4 * u * kProbsThreads);
        if (skip != 0 && (threadIdx.x & 31) == 31)
#pragma unroll
            for (int u = 0; u < U; ++u)
                copy_bytes<Raw4<T>::BYTES>(to + slot_of(u * kProbsThreads) + 1, from + 4 * u * kProbsThreads + 4);
    }
    // U vectors, as above, of a row that needs shifting or of one that does not
    template <bool SHIFT, int U>
    __device__ __forceinline__ void read_chunk(int n, int skip, Raw4<T> (&v)[U]) const
    {
        const Raw4<T>* from = slots + slot_of(threadIdx.x) + slot_of(n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = from[slot_of(u * kProbsThreads)];
            if constexpr (SHIFT) {
                Raw4<T> after = v[u].of_next_lane();
                if ((threadIdx.x & 31) == 31)
                    after = from[slot_of(u * kProbsThreads) + 1];
                v[u].shifted(v[u], after, skip);
            }
        }
    }
    // vector k < count of the row; called by all lanes, with neighbouring k
    __device__ __forceinline__ Raw4<T> read(int k, int skip) const
    {
        Raw4<T> v = slots[slot_of(k)];
        if constexpr (sizeof(T) == 2)
            if (skip != 0) {
                Raw4<T> after = v.of_next_lane();
                if (reads_slot_after(k))
                    after = slots[slot_of(k) + 1];
                v.shifted(v, after, skip);
            }
        return v;
    }
};

// Clusters walk over the rows; CTA r takes a row's vectors of four logits [r per,
// (r + 1) per), the last one also the up to three logits after them.  The first `room`
// vectors of a CTA stay in its shared memory, what lies beyond is read again.  The order
// of a row's sum does not depend on where the row lies.
template <class T>
__global__ void __launch_bounds__(kProbsThreads, kProbsCtas)
token_probs_kernel(ProbsArgs a, int per, int room)
{
    constexpr int U = 4;  // vectors a thread works on at a time
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ Stat s_stat[2][kProbsCluster * kProbsWarps];  // of all warps of the cluster, for two rows in turn
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int rows = a.B * a.N, stride = (int)(gridDim.x / C);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, V = a.V;
    auto arrived = cluster.barrier_arrive();  // this CTA's shared memory may be written
    // A programmatic dependent: its CTAs may be scheduled while the kernel before it ends,
    // and read and write nothing until that is done.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int nvec = V / 4, j0 = min(rank * per, nvec), all = min(per, nvec - j0);
    const Kept<T> kept = {reinterpret_cast<Raw4<T>*>(s_raw), j0, min(room, all), V};
    // chunks of all threads' U vectors each that are kept
    const int chunked = kept.count / (U * kProbsThreads) * (U * kProbsThreads);
    struct Row {
        const T* src;
        bool on;  // there is such a row, and it is not left as it is
        float temperature;
    };
    auto row_of = [&](int row) {
        Row r = {nullptr, row < rows, 1.0f};
        if (r.on) {
            const int b = row / a.N, i = row % a.N;
            r.src = static_cast<const T*>(a.logits) + b * a.batch_stride + i * a.row_stride;
            r.on = !(a.n_rows && i >= ld_prior(a.n_rows + b));
            if (a.temperature)
                r.temperature = ld_prior(a.temperature + b);
        }
        return r;
    };
    Row next = row_of((int)(blockIdx.x / C));
    if (next.on)
        kept.copy(next.src, 0, kept.count);
    cluster.barrier_wait(std::move(arrived));
    // Every CTA of a cluster comes to the barrier of every row and does the same before
    // it whatever it reads.
#pragma unroll 1
    for (int row = (int)(blockIdx.x / C), turn = 0; row < rows; row += stride, turn ^= 1) {
        const Row now = next;
        const T* src = now.src;
        float* dst = a.probs + (size_t)row * V;
        next = row_of(row + stride);
        const int edge = 4 * nvec + tid;  // one of the logits after the vectors
        const bool has_edge = now.on && rank == C - 1 && edge < V;
        const float edge_l = has_edge ? to_float(ld_prior(src + edge)) : -INFINITY;
        const bool greedy = now.temperature <= 0.0f;
        const Scale c = inverse_temperature(greedy ? 1.0f : now.temperature);
        const int skip = Kept<T>::skip_of(src);
        auto by_shift = [&](auto body) {
            if (sizeof(T) == 4 || skip == 0)
                body(std::false_type());
            else
                body(std::integral_constant<bool, sizeof(T) == 2>());
        };
        // The U vectors of this thread from vector n + tid on: kept, read again, or past
        // the end: -infinity.
        auto fetch = [&](int n, Raw4<T> (&v)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = n + tid + u * kProbsThreads;
                v[u] = kept.read(min(k, room - 1), skip);
                if (k >= kept.count) {
                    if (k >= all)
                        v[u].clear();
                    else if (skip == 0)
                        v[u].load(src + 4 * (j0 + k));
                    else
                        v[u].load_each(src + 4 * (j0 + k));
                }
            }
        };
        Stat s = {-INFINITY, 0.0f, INT_MAX};
        Ref ref = ref_at(c, reference(s.m));
        asm volatile("cp.async.wait_all;" ::: "memory");
        auto take = [&](const Raw4<T> (&v)[U], int n) {
            const float m = largest(v);
            if (m > s.m) {
                ref = ref_at(c, m);
                s.l *= weight(s.m, ref, c);
                s.m = m;
                if (greedy) {
                    s.first = INT_MAX;
#pragma unroll
                    for (int u = U - 1; u >= 0; --u)
                        s.first = where(v[u], m, 4 * (j0 + n + tid + u * kProbsThreads), s.first);
                }
            }
            const Scale2 c2 = twice(c, ref);
            F2 l = weights_sum(pair2(v[0], 0), c2);
            l = add2(l, weights_sum(pair2(v[0], 1), c2));
#pragma unroll
            for (int u = 1; u < U; ++u) {
                l = add2(l, weights_sum(pair2(v[u], 0), c2));
                l = add2(l, weights_sum(pair2(v[u], 1), c2));
            }
            s.l += unpack2(l).x + unpack2(l).y;
        };
        if (now.on) {
            by_shift([&](auto shift) {
#pragma unroll 1
                for (int n = 0; n < chunked; n += U * kProbsThreads) {
                    Raw4<T> v[U];
                    kept.template read_chunk<decltype(shift)::value>(n, skip, v);
                    take(v, n);
                }
            });
#pragma unroll 1
            for (int n = chunked; n < all; n += U * kProbsThreads) {
                Raw4<T> v[U];
                fetch(n, v);
                take(v, n);
            }
        }
        if (has_edge) {  // a thread's last logit
            const float m = fmaxf(s.m, edge_l);
            const Ref r = ref_at(c, reference(m));
            s = {m, s.l * weight(s.m, r, c) + weight(edge_l, r, c), edge_l > s.m ? edge : s.first};
        }
        s = join(s, c, greedy);
        if (lane < C)
            cluster.map_shared_rank(&s_stat[turn][0], lane)[rank * kProbsWarps + warp] = s;
        cluster.sync();
        static_assert(kProbsCluster * kProbsWarps <= 64, "a lane for two warps of the cluster");
        s = lane < C * kProbsWarps ? s_stat[turn][lane] : Stat{-INFINITY, 0.0f, INT_MAX};
        if (lane + 32 < C * kProbsWarps) {
            const Stat t = s_stat[turn][lane + 32];
            const float m = fmaxf(s.m, t.m);
            const Ref r = ref_at(c, reference(m));
            s = {m, s.l * weight(s.m, r, c) + t.l * weight(t.m, r, c),
                 s.m == t.m ? min(s.first, t.first) : s.m > t.m ? s.first : t.first};
        }
        s = join(s, c, greedy);
        if (!now.on) {
            if (next.on)
                kept.copy(next.src, 0, kept.count);
            continue;
        }
        // Outputs of vector k of this lane; all lanes have neighbouring vectors.  Where an
        // aligned vector begins with output AHEAD of them, its end is the next lane's; the
        // first lane's outputs before it and the last one's after it go out one by one.
        auto store = [&](auto known, int k, F2 p, F2 q) {
            constexpr int AHEAD = decltype(known)::value;
            const float2 x = unpack2(p), y = unpack2(q);
            float o[8] = {x.x, x.y, y.x, y.y};
            float* to = dst + 4 * (j0 + k);
            bool whole = k < all;
            if constexpr (AHEAD > 0) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    o[4 + i] = __shfl_down_sync(0xffffffffu, o[i], 1);
                const bool last = lane == 31 || k + 1 == all;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (whole && (i < AHEAD ? lane == 0 : last))
                        st_checked(to + i, o[i]);
                whole = whole && !last;
            }
            if (whole && KIVI_IN_RANGE(to + AHEAD, 16))
                __stcs(reinterpret_cast<float4*>(to + AHEAD), make_float4(o[AHEAD], o[AHEAD + 1], o[AHEAD + 2], o[AHEAD + 3]));
        };
        auto by_alignment = [&](auto body) {
            switch ((0 - (uintptr_t)dst / 4) & 3) {
            case 0: body(std::integral_constant<int, 0>()); break;
            case 1: body(std::integral_constant<int, 1>()); break;
            case 2: body(std::integral_constant<int, 2>()); break;
            default: body(std::integral_constant<int, 3>()); break;
            }
        };
        if (greedy) {
            if (next.on)
                kept.copy(next.src, 0, kept.count);
            const float zero = isnan(s.l) ? s.l : 0.0f, one = s.l == 0.0f ? 0.0f : 1.0f + zero;
            by_alignment([&](auto known) {
                // (512 rows of 131072 bf16 logits: 73.3 us, 73.8 without unrolling)
#pragma unroll 4
                for (int n = 0; n < all; n += kProbsThreads) {
                    const int x = 4 * (j0 + n + tid);
                    store(known, n + tid, pack2(x == s.first ? one : zero, x + 1 == s.first ? one : zero),
                          pack2(x + 2 == s.first ? one : zero, x + 3 == s.first ? one : zero));
                }
            });
            if (has_edge)
                st_checked(dst + edge, edge == s.first ? one : zero);
            continue;
        }
        const Scale2 c2 = twice(c, ref_at(c, reference(s.m)));
        // the sum's inverse, NaN for a NaN sum, and what its rounding left, which would
        // be the same for all of the row
        const float inv1 = s.l == 0.0f ? 0.0f : 1.0f / s.l;
        const F2 inv = both(inv1), rest = both(s.l == 0.0f ? 0.0f : __fmaf_rn(-inv1, s.l, 1.0f));
        by_alignment([&](auto known) {
            constexpr int AHEAD = decltype(known)::value;
            by_shift([&](auto shift) {
                float* to = dst + 4 * (j0 + tid);
#pragma unroll 1
                for (int n = 0; n < chunked; n += U * kProbsThreads, to += 4 * U * kProbsThreads) {
                    Raw4<T> v[U];
                    kept.template read_chunk<decltype(shift)::value>(n, skip, v);
#pragma unroll
                    for (int u = 0; u < U; ++u) {  // as `store`, with all vectors there
                        const float2 x = unpack2(weights(pair2(v[u], 0), c2, inv, rest));
                        const float2 y = unpack2(weights(pair2(v[u], 1), c2, inv, rest));
                        float o[8] = {x.x, x.y, y.x, y.y};
                        float* at = to + 4 * u * kProbsThreads;
#pragma unroll
                        for (int i = 0; i < AHEAD; ++i)
                            o[4 + i] = __shfl_down_sync(0xffffffffu, o[i], 1);
                        if constexpr (AHEAD > 0)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (lane == (i < AHEAD ? 0 : 31))
                                    st_checked(at + i, o[i]);
                        if ((AHEAD == 0 || lane != 31) && KIVI_IN_RANGE(at + AHEAD, 16))
                            __stcs(reinterpret_cast<float4*>(at + AHEAD),
                                   make_float4(o[AHEAD], o[AHEAD + 1], o[AHEAD + 2], o[AHEAD + 3]));
                    }
                    if (next.on)  // these slots have been read
                        kept.template copy_chunk<U>(next.src, n);
                }
            });
#pragma unroll 1
            for (int n = chunked; n < all; n += U * kProbsThreads) {
                Raw4<T> v[U];
                fetch(n, v);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    store(known, n + tid + u * kProbsThreads, weights(pair2(v[u], 0), c2, inv, rest),
                          weights(pair2(v[u], 1), c2, inv, rest));
                if (next.on)
                    kept.copy(next.src, n, min(n + U * kProbsThreads, kept.count));
            }
        });
        if (has_edge)
            st_checked(dst + edge, unpack2(weights(both(edge_l), c2, inv, rest)).x);
    }
}

#ifdef KIVI_CHECKS
// The logits that a call may read.
static CallBuf logits_of(const ProbsArgs& a)
{
    const int32_t dims[2] = {a.B, a.N};
    const int64_t strides[2] = {a.batch_stride, a.row_stride};
    const Span s = strided_span(a.logits, dims, strides, 2, a.V, a.dtype == KIVI_F32 ? 4 : 2);
    return {reinterpret_cast<const void*>(s.lo), s.hi - s.lo};
}
#endif

template <class T>
static cudaError_t launch_probs(const ProbsArgs& a, cudaStream_t s)
{
    constexpr int kMost = kProbsBytes / Raw4<T>::BYTES;  // vectors a CTA keeps
    constexpr int kMostSmem = (slot_of(kMost - 1) + 2) * Raw4<T>::BYTES;
    static int allowed[64], wide[64], resident[64][kProbsCluster + 1];
    cudaError_t e = allow_smem(token_probs_kernel<T>, kMostSmem, allowed);
    if (e != cudaSuccess || (e = allow_wide_clusters(token_probs_kernel<T>, wide)) != cudaSuccess)
        return e;
    // As few CTAs a row as keep all of it; up to eight where fewer leave SMs idle and a
    // thread has more than two vectors; sixteen also where each of them has an SM.  In us
    // with eight and with sixteen, fp32 rows of 131072: 8 rows 7.7 and 5.2, 512 rows (half
    // of which eight would read again) 98.7 and 93.4; 32 bf16 rows 7.6 and 8.4.
    const int rows = a.B * a.N, nvec = a.V / 4;
    int C = 1;
    while (C < kProbsCluster &&
           (nvec > C * kMost || (nvec > C * 2 * kProbsThreads &&
                                 (C < 8 ? (long long)rows * C < 2 * sm_count() : (long long)rows * 2 * C <= sm_count()))))
        C *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kProbsThreads);
    cfg.dynamicSmemBytes = kMostSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    // The clusters that are resident at once, asked for once per device; where none of
    // sixteen CTAs is, smaller ones do.
    int dev = 0, clusters = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess)
        return e;
    for (;; C /= 2) {
        at[0].val.clusterDim.x = (unsigned)C;
        cfg.gridDim = dim3((unsigned)C);
        clusters = dev < 64 ? __atomic_load_n(&resident[dev][C], __ATOMIC_RELAXED) : 0;
        if (clusters == 0) {
            if ((e = cudaOccupancyMaxActiveClusters(&clusters, token_probs_kernel<T>, &cfg)) != cudaSuccess)
                return e;
            if (clusters == 0)
                clusters = C > 8 ? -1 : 1;
            if (dev < 64)
                __atomic_store_n(&resident[dev][C], clusters, __ATOMIC_RELAXED);
        }
        if (clusters > 0)
            break;
    }
    const int per = ((nvec + C - 1) / C + 31) / 32 * 32, room = std::max(1, std::min(per, kMost));
    cfg.gridDim = dim3((unsigned)(std::min(rows, clusters) * C));
    cfg.dynamicSmemBytes = (size_t)(slot_of(room - 1) + 2) * Raw4<T>::BYTES;
    return cudaLaunchKernelEx(&cfg, token_probs_kernel<T>, a, per, room);
}

cudaError_t launch_token_probs(const ProbsArgs& a, cudaStream_t s)
{
    KIVI_SET_CHECK_BUFFERS(s, {logits_of(a), {a.temperature, (size_t)a.B * 4}, {a.n_rows, (size_t)a.B * 4},
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
