// verify.cu -- verification of drafted tokens against the target's probabilities
// from given random numbers (kivi_verify_tree).
//
// A cluster of CTAs verifies a sequence: the walk down the tree is a few tests of
// single probabilities, and every sum over a row of the vocabulary (after a
// rejection, and for the next token) is shared by the cluster.  Weights are whole
// numbers, so neither the split nor the order of a sum shows in a result.
#include <cooperative_groups.h>

#include <algorithm>

#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 16;  // warps of a CTA
constexpr int kMaxCluster = 8;

typedef unsigned long long u64;

__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }  // NaN to 0

// Probabilities as multiples of 2^-42, rounded half to even: sums of up to 2^20 of these
// are exact.  The conversion to 64 bits is slow (it shares the fp64 pipe), so a value
// below 4 is split in fp32: r + 4 rounds it to a = A 2^-21, r - a is exact and at most
// 2^-22, and (r - a) 2^42 + 1.5 2^23 rounds that to a whole number B.  As A 2^21 is
// even, A 2^21 + B is the rounded r 2^42.  The numbers add up as the bits of the
// rounded sums; two of 32 bits hold those of 1024 values below 2 (of 1365 below 1.5).
struct Whole {
    uint32_t a = 0, b = 0;
    template <int N>
    __device__ __forceinline__ void add(const float (&r)[N])
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = __fadd_rn(r[i], 4.0f);
            const float u = __fmaf_rn(__fsub_rn(r[i], __fsub_rn(t, 4.0f)), 0x1p42f, 0x1.8p23f);
            a += __float_as_uint(t);
            b += __float_as_uint(u);
        }
        a -= N * 0x40800000u;
        b -= N * 0x4b400000u;
    }
    __device__ __forceinline__ u64 sum() const { return ((u64)a << 21) + (u64)(long long)(int)b; }
    // of all lanes
    __device__ __forceinline__ u64 warp_sum() const
    {
        Whole w;
        w.a = __reduce_add_sync(0xffffffffu, a);
        w.b = __reduce_add_sync(0xffffffffu, b);
        return w.sum();
    }
};
__device__ __forceinline__ u64 whole(float r)
{
    const float x[1] = {r};
    Whole w;
    w.add(x);
    return w.sum();
}

// The fp32 rounding of the fp64 rounding of 2^42 / z, z <= 2^62 (0 for 0).  In fp32 with
// z as h + l and the quotient as q0 + q1, each in two terms: off by some 2^-46 of it.
// The rounded sum s is right where what it leaves is not that near half a unit of s;
// the division in 64 bits, far slower, is left for the rest.  (Below a power of two the
// unit is half as large.)
__device__ __forceinline__ float scale_of(u64 z)
{
    if (z == 0)
        return 0.0f;
    const float a = (float)(uint32_t)(z >> 38) * 0x1p38f, b = (float)((uint32_t)(z >> 14) & 0xffffffu) * 0x1p14f;
    const float ab = __fadd_rn(a, b);  // a is 0 or above b: what the sum leaves is b - (ab - a)
    const float rest = __fadd_rn(__fsub_rn(b, __fsub_rn(ab, a)), (float)((uint32_t)z & 0x3fffu));
    const float h = __fadd_rn(ab, rest), l = __fsub_rn(rest, __fsub_rn(h, ab));
    const float r = __frcp_rn(h), q0 = __fmul_rn(r, 0x1p42f);
    const float q1 = __fmul_rn(__fmaf_rn(-q0, l, __fmaf_rn(-q0, h, 0x1p42f)), r);
    const float s = __fadd_rn(q0, q1), left = __fsub_rn(q1, __fsub_rn(s, q0));
    const float half = __fmul_rn(__uint_as_float(__float_as_uint(s) & 0x7f800000u), 0x1p-24f);
    const bool low = (__float_as_uint(s) & 0x7fffffu) == 0 && left < 0.0f;
    if (fabsf(left) > half * (low ? 0.5f - 0x1p-13f : 1.0f - 0x1p-12f))
        return (float)__ddiv_rn(0x1p42, (double)z);
    return s;
}

// Over all lanes, of numbers whose sum is below 2^63.
__device__ __forceinline__ u64 warp_sum(u64 x)
{
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)x & 0xffffffu);
    const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 24) & 0xffffffu);
    const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 48));
    return ((u64)c << 48) + ((u64)b << 24) + a;
}

// The tree of a sequence and the single probabilities its tests need: rank 0 of
// the cluster reads them and gives every CTA a copy, so that all of them take the
// same way whatever happens to the inputs meanwhile.
struct VerifyTree {
    int n;                       // nodes
    int parent[KIVI_MAX_DRAFT];  // -1: never accepted
    int token[KIVI_MAX_DRAFT];
    float u[KIVI_MAX_DRAFT];
    float p[KIVI_MAX_DRAFT], q[KIVI_MAX_DRAFT];  // of the token, after its parent
};

struct VerifySmem {
    VerifyTree tree;
    int path[KIVI_MAX_DRAFT];
    float scale[KIVI_MAX_DRAFT];  // s after k rejections
    int gone[KIVI_MAX_DRAFT];     // rejected tokens, and their weights (0: rejected before)
    u64 gone_w[KIVI_MAX_DRAFT];
    u64 part[2][kMaxCluster * kMaxWarps];  // sums of the runs, of the last two passes in turn
};

// Residual of a value after k rejections of drawn tokens.
__device__ __forceinline__ float residual(float r, float q, const float* scale, int k)
{
    for (int n = 0; n < k; ++n)
        r = fmaxf(__fsub_rn(__fmul_rn(r, scale[n]), q), 0.0f);
    return r;
}

// A row of probabilities, counted from the aligned vector that holds its first: place
// y is token y - off.
struct Row {
    const float *p, *q;  // at place 0; q NULL without a draft
    int off, end;        // tokens at places off .. end
};

// Four neighbouring places at an end of a row or run, 0 where there is no token.
__device__ __forceinline__ float4 load_edge(const float* row, const Row& at, int y, int y1)
{
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int end = min(at.end, y1);
    if (y >= at.off && y < end)
        v.x = ld_prior(row + y);
    if (y + 1 >= at.off && y + 1 < end)
        v.y = ld_prior(row + y + 1);
    if (y + 2 >= at.off && y + 2 < end)
        v.z = ld_prior(row + y + 2);
    if (y + 3 >= at.off && y + 3 < end)
        v.w = ld_prior(row + y + 3);
    return v;
}

// Residuals of U lines of 128 places from y on, up to place y1: a lane has four
// neighbours of each.
template <int U>
__device__ __forceinline__ void load_lines(const Row& at, int y, int y1, const float* scale, int k, float (&r)[U][4])
{
    const bool both = at.q && k > 0;
    const int mine = y + 4 * (threadIdx.x & 31);
    float4 p[U], q[U];
    if (y >= at.off && y + 128 * U <= min(at.end, y1)) {  // all loads at once
#pragma unroll
        for (int i = 0; i < U; ++i)
            p[i] = ld_prior(reinterpret_cast<const float4*>(at.p + mine + i * 128));
        if (both)
#pragma unroll
            for (int i = 0; i < U; ++i)
                q[i] = ld_prior(reinterpret_cast<const float4*>(at.q + mine + i * 128));
    } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            p[i] = load_edge(at.p, at, mine + i * 128, y1);
            if (both)
                q[i] = load_edge(at.q, at, mine + i * 128, y1);
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
        r[i][0] = clamp01(p[i].x), r[i][1] = clamp01(p[i].y), r[i][2] = clamp01(p[i].z), r[i][3] = clamp01(p[i].w);
    if (both) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            q[i] = make_float4(clamp01(q[i].x), clamp01(q[i].y), clamp01(q[i].z), clamp01(q[i].w));
#pragma unroll 1
        for (int n = 0; n < k; ++n) {
            const float s = scale[n];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                r[i][0] = fmaxf(__fsub_rn(__fmul_rn(r[i][0], s), q[i].x), 0.0f);
                r[i][1] = fmaxf(__fsub_rn(__fmul_rn(r[i][1], s), q[i].y), 0.0f);
                r[i][2] = fmaxf(__fsub_rn(__fmul_rn(r[i][2], s), q[i].z), 0.0f);
                r[i][3] = fmaxf(__fsub_rn(__fmul_rn(r[i][3], s), q[i].w), 0.0f);
            }
        }
    }
}

// The first node from `from` on whose parent is cur; n if there is none.
__device__ __forceinline__ int next_child(const VerifyTree& t, int cur, int from)
{
    for (int base = from & ~31; base < t.n; base += 32) {
        const int i = base + (threadIdx.x & 31);
        const unsigned hit = __ballot_sync(0xffffffffu, i >= from && i < t.n && t.parent[i] == cur);
        if (hit)
            return base + __ffs(hit) - 1;
    }
    return t.n;
}

// Warp w of CTA r sums the run of neighbouring places r (warps of a CTA) + w.
template <int TH>
__global__ void __launch_bounds__(TH, 1024 / TH)
verify_tree_kernel(VerifyArgs a, int run)
{
    constexpr int U = 4;  // lines of a run loaded at a time
    __shared__ VerifySmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = (int)(blockIdx.x / C), tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    constexpr int threads = TH, warps = TH / 32;
    const int N = a.N, V = a.V;
    const size_t row0 = (size_t)b * N;
    const bool drawn = a.draft != nullptr;
    auto arrived = cluster.barrier_arrive();  // this CTA's shared memory may be written
    // A programmatic dependent: its CTAs may be scheduled while the kernel before it ends,
    // and read and write nothing until that is done.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int g = rank * warps + warp;
    const int y0 = (int)min((long long)g * run, (long long)V + 3), y1 = y0 + run;
    auto row_of = [&](int node) {
        const size_t at = (row0 + node) * V;
        const int off = (int)(at & 3);
        return Row{a.target + at - off, drawn ? a.draft + at - off : nullptr, off, off + V};
    };
    if (rank == 0) {
        VerifyTree& t = sm.tree;
        const int n = a.n_draft ? min(max(ld_prior(a.n_draft + b), 0), N) : N;
        for (int i = tid; i < N; i += threads) {
            int par = i ? ld_prior(a.parent + row0 + i) : -1;
            const int x = i ? ld_prior(a.tokens + row0 + i) : -1;
            if (par < 0 || par >= i || x < 0 || x >= V)
                par = -1;
            t.parent[i] = par;
            t.token[i] = x;
            t.u[i] = ld_prior(a.u + row0 + i);
            if (par >= 0 && i < n) {
                t.p[i] = clamp01(ld_prior(a.target + (row0 + par) * V + x));
                t.q[i] = drawn ? clamp01(ld_prior(a.draft + (row0 + par) * V + x)) : 1.0f;
            }
        }
        if (tid == 0)
            t.n = n;
        __syncthreads();
    }
    if (tid == 0) {
        sm.path[0] = 0;
        sm.scale[0] = 1.0f;
    }
    cluster.barrier_wait(std::move(arrived));
    if (rank == 0)
        for (int i = tid; i < 1 + 5 * N; i += threads) {  // n, then N words of each of the five arrays
            const int at = i == 0 ? 0 : 1 + (i - 1) / N * KIVI_MAX_DRAFT + (i - 1) % N;
            const int x = reinterpret_cast<const int*>(&sm.tree)[at];
            for (int r = 1; r < C; ++r)
                reinterpret_cast<int*>(&cluster.map_shared_rank(&sm, r)->tree)[at] = x;
        }
    cluster.sync();
    const VerifyTree& t = sm.tree;
    int pass = 0;
    // Sum of the runs before run n in the last pass.
    auto runs_before = [&](int n) {
        u64 z = 0;
        for (int i = lane; i < n; i += 32)
            z += sm.part[pass][i];
        return warp_sum(z);
    };
    // Sum of w(rho) at node cur after k rejections, rejected tokens included if they
    // were not drawn.  A part is written again two passes later, when every CTA has
    // come to the barrier between and so has read it.
    auto sum = [&](int cur, int k) {
        const Row at = row_of(cur);
        u64 z = 0;
#pragma unroll 1
        for (int y = y0; y < y1 && y < at.end; y += 128 * U) {
            float r[U][4];
            load_lines<U>(at, y, y1, sm.scale, k, r);
            Whole w;  // of up to 512 values of the warp
#pragma unroll
            for (int i = 0; i < U; ++i)
                w.add(r[i]);
            z += w.warp_sum();
        }
        pass ^= 1;
        if (lane < C)
            cluster.map_shared_rank(&sm, lane)->part[pass][g] = z;
        cluster.sync();
        return runs_before(C * warps);
    };
    int cur = 0, k = 0, count = t.n > 0 ? 1 : 0;
    u64 z = 0;
    auto accept = [&](int i) {
        cur = i;
        k = 0;
        if (tid == 0)
            sm.path[count] = i;
        ++count;
    };
    if (drawn) {
        // A scale is written after the barriers of the sum that it comes from, which
        // every warp reaches when it has read the scales of the node before.
        for (int i = 1; (i = next_child(t, cur, i)) < t.n; ++i) {
            if (k > 0) {  // a sibling is left to be tested
                if (tid == 0)
                    sm.scale[k] = scale_of(z);
                __syncthreads();
            }
            const float r = residual(t.p[i], t.q[i], sm.scale, k);
            if (__fmul_rn(t.u[i], t.q[i]) < __fmul_rn(r, sm.scale[k]))
                accept(i);
            else
                z = sum(cur, ++k);
        }
    } else {
        // Nothing but the sum of the row is needed to test all siblings after the first
        // at once: a lane has one of 32 nodes, and the weights of those before it in a
        // prefix sum.  All warps do the same and write the same lists.
        for (int i = 1; (i = next_child(t, cur, i)) < t.n;) {
            if (t.u[i] < t.p[i]) {
                accept(i++);
                continue;
            }
            z = sum(cur, 0);
            sm.gone[0] = t.token[i];
            sm.gone_w[0] = whole(t.p[i]);
            z -= whole(t.p[i]);
            k = 1;
            int taken = t.n;
            for (int base = i + 1; base < t.n && taken == t.n; base += 32) {
                const int c = base + lane;
                const bool child = c < t.n && t.parent[c] == cur;
                const unsigned those = __ballot_sync(0xffffffffu, child), before = (1u << lane) - 1;
                if (those == 0)
                    continue;
                __syncwarp();
                const int x = child ? t.token[c] : -1 - lane;
                bool again = (__match_any_sync(0xffffffffu, x) & before) != 0;
                for (int m = 0; m < k; ++m)
                    again |= sm.gone[m] == x;
                const float r = child && !again ? t.p[c] : 0.0f;
                const u64 w = whole(r);
                u64 upto = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
                    upto += lane >= o ? y : 0;
                }
                const bool ok = child && t.u[c] < __fmul_rn(r, scale_of(z - (upto - w)));
                const unsigned hits = __ballot_sync(0xffffffffu, ok);
                if (hits) {
                    taken = base + __ffs(hits) - 1;
                } else {
                    if (child) {
                        sm.gone[k + __popc(those & before)] = x;
                        sm.gone_w[k + __popc(those & before)] = w;
                    }
                    z -= __shfl_sync(0xffffffffu, upto, 31);
                    k += __popc(those);
                }
            }
            if (taken == t.n)
                break;
            accept(taken);
            i = taken + 1;
        }
    }
    if (t.n > 0 && k == 0)
        z = sum(cur, 0);
    if (t.n > 0 && z == 0 && k > 0) {
        k = 0;
        z = sum(cur, 0);
    }
    __syncthreads();  // of the path and the lists
    if (rank == 0 && warp == warps - 1) {
        for (int i = lane; i < N; i += 32)
            st_checked(a.path + row0 + i, i < count ? sm.path[i] : -1);
        if (lane == 0) {
            st_checked(a.counts + b, count);
            if (z == 0)
                st_checked(a.next + b, -1);
        }
    }
    if (z == 0)
        return;
    // The run in which the running sum passes `target`, then its line, then the token.
    const float u0 = t.u[0];
    const unsigned d = u0 >= 1.0f ? 0xffffffffu : u0 > 0.0f ? (unsigned)(u0 * 0x1p32f) : 0u;
    const u64 target = __umul64hi(z, (u64)d << 32);
    const Row row = row_of(cur);
    u64 at = runs_before(g), mine = sm.part[pass][g];
    if (!drawn)
        for (int m = 0; m < k; ++m) {
            const int home = (sm.gone[m] + row.off) / run;
            at -= home < g ? sm.gone_w[m] : 0;
            mine -= home == g ? sm.gone_w[m] : 0;
        }
    if (target < at || target - at >= mine)
        return;
#pragma unroll 1
    for (int y = y0; y < y1 && y < row.end; y += 128 * U) {
        float r[U][4];
        load_lines<U>(row, y, y1, sm.scale, k, r);
        if (!drawn)
#pragma unroll 1
            for (int m = 0; m < k; ++m) {
                const int x = sm.gone[m] + row.off - y - 4 * lane;
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        r[i][j] = x == i * 128 + j ? 0.0f : r[i][j];
            }
        // the line: the first whose sum takes `at` past the target
        u64 line[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            Whole w;
            w.add(r[i]);
            line[i] = w.warp_sum();
        }
        int hit = U;
        float f[4] = {};
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (hit == U) {
                if (target - at < line[i]) {
                    hit = i;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[j] = r[i][j];
                } else {
                    at += line[i];
                }
            }
        if (hit == U)
            continue;
        // the lane: sums of the lanes before it
        Whole w;
        w.add(f);
        Whole upto = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t ya = __shfl_up_sync(0xffffffffu, upto.a, o), yb = __shfl_up_sync(0xffffffffu, upto.b, o);
            upto.a += lane >= o ? ya : 0;
            upto.b += lane >= o ? yb : 0;
        }
        u64 here = at + upto.sum() - w.sum();
        if (target >= here && target - here < w.sum()) {
            int j = 0;
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                here += whole(f[n]);
                j += here <= target;
            }
            st_checked(a.next + b, y + 4 * lane - row.off + hit * 128 + j);
        }
        return;
    }
}

cudaError_t launch_verify_tree(const VerifyArgs& a, cudaStream_t s)
{
    const size_t BN = (size_t)a.B * a.N;
    (void)BN;
    KIVI_SET_CHECK_BUFFERS(s, {{a.tokens, BN * 4}, {a.parent, BN * 4}, {a.n_draft, (size_t)a.B * 4}, {a.u, BN * 4},
                               {a.target, BN * a.V * 4}, {a.draft, BN * a.V * 4}, {a.path, BN * 4},
                               {a.counts, (size_t)a.B * 4}, {a.next, (size_t)a.B * 4}});
    // As many CTAs a sequence as leave all of them resident at once (four of 256
    // threads an SM) and give a thread four places; of 512 threads where every CTA has
    // an SM for itself and more than 32 places a thread.  In us, CTAs x threads, for 1
    // sequence of 32000 tokens, 16 and 64 of 131072, 32 of 50001:
    //              1       16      64      32
    //     8x256   6.0     14.5    17.4    9.0
    //     8x512   6.9     12.7    21.8    9.2
    //     4x512   6.4     16.8    17.7    9.2
    //     4x256   6.6     21.4    20.5    9.8
    //     1x512   9.0     44.4    30.6   14.0
    int C = kMaxCluster;
    while (C > 1 && ((long long)a.B * C > 4 * sm_count() || a.V < C * 1024))
        C /= 2;
    const int threads = (long long)a.B * C <= sm_count() && a.V > C * 256 * 32 ? 512 : 256;
    const int warps = C * threads / 32, places = a.V % 4 ? a.V + 3 : a.V, run = ((places + warps - 1) / warps + 127) / 128 * 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * C));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    return threads == 512 ? cudaLaunchKernelEx(&cfg, verify_tree_kernel<512>, a, run)
                          : cudaLaunchKernelEx(&cfg, verify_tree_kernel<256>, a, run);
}

#ifdef KIVI_CHECKS
int32_t check_word_verify() { return take_check_word(); }
#endif

}  // namespace kivi
