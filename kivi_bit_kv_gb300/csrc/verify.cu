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

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;

typedef unsigned long long u64;

__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }  // NaN to 0

// Probabilities as multiples of 2^-42, rounded half to even: sums of up to 2^20 of these
// are exact.  The conversion to 64 bits is slow (it shares the fp64 pipe), so a value
// below 4 is split in fp32: r + 4 rounds it to a = A 2^-21, r - a is exact and at most
// 2^-22, and (r - a) 2^42 + 1.5 2^23 rounds that to a whole number B.  As A 2^21 is
// even, A 2^21 + B is the rounded r 2^42.  The numbers add up as the bits of the
// rounded sums; two of 32 bits hold those of some hundred values.
struct Whole {
    uint32_t a = 0, b = 0, n = 0;
    __device__ __forceinline__ void add(float r)
    {
        const float t = __fadd_rn(r, 4.0f);
        const float u = __fmaf_rn(__fsub_rn(r, __fsub_rn(t, 4.0f)), 0x1p42f, 0x1.8p23f);
        a += __float_as_uint(t);
        b += __float_as_uint(u);
        ++n;  // a constant after unrolling
    }
    __device__ __forceinline__ u64 sum() const
    {
        return ((u64)(a - n * 0x40800000u) << 21) + (u64)(long long)(int)(b - n * 0x4b400000u);
    }
};
__device__ __forceinline__ u64 whole(float r)
{
    Whole w;
    w.add(r);
    return w.sum();
}

__device__ __forceinline__ float scale_of(u64 z) { return z ? (float)__ddiv_rn(0x1p42, (double)z) : 0.0f; }

__device__ __forceinline__ u64 warp_sum(u64 x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
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
    u64 part[2][kVerifyWarps];    // sums of the warps' runs, of the last two passes in turn
    u64 slot[2][kMaxCluster];     // the CTAs' sums
};

// Residual of a value after k rejections of drawn tokens.
__device__ __forceinline__ float residual(float r, float q, const float* scale, int k)
{
    for (int n = 0; n < k; ++n)
        r = fmaxf(__fsub_rn(__fmul_rn(r, scale[n]), q), 0.0f);
    return r;
}

// W neighbouring probabilities of a row, those from V on as 0.
template <int W>
__device__ __forceinline__ void load_probs(const float* row, int x, int end, float (&r)[W])
{
    if constexpr (W == 4) {
        const float4 v = x < end ? ld_nc_f4(row + x) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        r[0] = clamp01(v.x), r[1] = clamp01(v.y), r[2] = clamp01(v.z), r[3] = clamp01(v.w);
    } else {
        r[0] = x < end ? clamp01(ldg_checked(row + x)) : 0.0f;
    }
}

// Weights of U lines of 32 W tokens from x on: a lane takes W neighbours of each.
template <int W, int U>
__device__ __forceinline__ void load_lines(const float* p, const float* q, int x, int end, const float* scale, int k,
                                           float (&r)[U][W])
{
#pragma unroll
    for (int i = 0; i < U; ++i)
        load_probs<W>(p, x + i * 32 * W, end, r[i]);
    if (q && k > 0) {
        float d[U][W];
#pragma unroll
        for (int i = 0; i < U; ++i)
            load_probs<W>(q, x + i * 32 * W, end, d[i]);
        for (int n = 0; n < k; ++n) {
            const float s = scale[n];
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    r[i][j] = fmaxf(__fsub_rn(__fmul_rn(r[i][j], s), d[i][j]), 0.0f);
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

// Warp w of CTA r sums the run of neighbouring tokens r kVerifyWarps + w.
template <int W>
__global__ void __launch_bounds__(kVerifyThreads)
verify_tree_kernel(VerifyArgs a, int run)
{
    constexpr int U = W == 4 ? 4 : 8;
    __shared__ VerifySmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = (int)(blockIdx.x / C), tid = threadIdx.x, lane = tid & 31, warp = tid / 32, N = a.N, V = a.V;
    const size_t row0 = (size_t)b * N;
    const bool drawn = a.draft != nullptr;
    auto arrived = cluster.barrier_arrive();  // this CTA's shared memory may be written
    if (rank == 0) {
        VerifyTree& t = sm.tree;
        const int n = a.n_draft ? min(max(ldg_checked(a.n_draft + b), 0), N) : N;
        for (int i = tid; i < N; i += kVerifyThreads) {
            int par = i ? ldg_checked(a.parent + row0 + i) : -1;
            const int x = i ? ldg_checked(a.tokens + row0 + i) : -1;
            if (par < 0 || par >= i || x < 0 || x >= V)
                par = -1;
            t.parent[i] = par;
            t.token[i] = x;
            t.u[i] = ldg_checked(a.u + row0 + i);
            if (par >= 0 && i < n) {
                t.p[i] = clamp01(ldg_checked(a.target + (row0 + par) * V + x));
                t.q[i] = drawn ? clamp01(ldg_checked(a.draft + (row0 + par) * V + x)) : 1.0f;
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
        for (int i = tid; i < 1 + 5 * N; i += kVerifyThreads) {  // n, then N words of each of the five arrays
            const int at = i == 0 ? 0 : 1 + (i - 1) / N * KIVI_MAX_DRAFT + (i - 1) % N;
            const int x = reinterpret_cast<const int*>(&sm.tree)[at];
            for (int r = 1; r < C; ++r)
                reinterpret_cast<int*>(&cluster.map_shared_rank(&sm, r)->tree)[at] = x;
        }
    cluster.sync();
    const VerifyTree& t = sm.tree;
    const int g = rank * kVerifyWarps + warp;
    const int x0 = (int)min((long long)g * run, (long long)V), x1 = min(x0 + run, V);
    int pass = 0;
    // Sum of w(rho) at node cur after k rejections, rejected tokens included if they
    // were not drawn.  A slot is written again two passes later, when every CTA has
    // come to the barrier between and so has read it.
    auto sum = [&](int cur, int k) {
        const float *p = a.target + (row0 + cur) * V, *q = drawn ? a.draft + (row0 + cur) * V : nullptr;
        u64 z = 0;
        for (int x = x0 + lane * W; x < x1; x += 32 * W * U) {
            float r[U][W];
            load_lines<W, U>(p, q, x, x1, sm.scale, k, r);
            Whole w;
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    w.add(r[i][j]);
            z += w.sum();
        }
        z = warp_sum(z);
        pass ^= 1;
        if (lane == 0)
            sm.part[pass][warp] = z;
        __syncthreads();
        if (tid < C) {
            z = 0;
            for (int w = 0; w < kVerifyWarps; ++w)
                z += sm.part[pass][w];
            cluster.map_shared_rank(&sm, tid)->slot[pass][rank] = z;
        }
        cluster.sync();
        z = 0;
        for (int r = 0; r < C; ++r)
            z += sm.slot[pass][r];
        return z;
    };
    int cur = 0, k = 0, count = t.n > 0 ? 1 : 0;
    u64 z = 0;
    for (int i = 1; (i = next_child(t, cur, i)) < t.n; ++i) {
        if (k > 0) {  // s after a rejection, where a sibling is left to be tested
            if (tid == 0)
                sm.scale[k] = scale_of(z);
            __syncthreads();
        }
        float r = t.p[i];
        if (drawn)
            r = residual(r, t.q[i], sm.scale, k);
        else
            for (int m = 0; m < k; ++m)
                r = sm.gone[m] == t.token[i] ? 0.0f : r;
        if (__fmul_rn(t.u[i], t.q[i]) < __fmul_rn(r, sm.scale[k])) {
            cur = i;
            k = 0;
            if (tid == 0)
                sm.path[count] = i;
            ++count;
            continue;
        }
        if (drawn)
            z = sum(cur, k + 1);
        else
            z = (k == 0 ? sum(cur, 0) : z) - whole(r);
        __syncthreads();  // the scales and lists are read before they grow
        if (tid == 0) {
            sm.gone[k] = t.token[i];
            sm.gone_w[k] = whole(r);
        }
        __syncthreads();
        ++k;
    }
    if (t.n > 0 && k == 0)
        z = sum(cur, 0);
    if (t.n > 0 && z == 0 && k > 0) {
        k = 0;
        z = sum(cur, 0);
    }
    __syncthreads();
    if (rank == 0) {
        for (int i = tid; i < N; i += kVerifyThreads)
            st_checked(a.path + row0 + i, i < count ? sm.path[i] : -1);
        if (tid == 0) {
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
    u64 at = 0, mine = sm.part[pass][warp];
    for (int r = 0; r < rank; ++r)
        at += sm.slot[pass][r];
    for (int w = 0; w < warp; ++w)
        at += sm.part[pass][w];
    if (!drawn)
        for (int m = 0; m < k; ++m) {
            const int home = sm.gone[m] / run;
            at -= home < g ? sm.gone_w[m] : 0;
            mine -= home == g ? sm.gone_w[m] : 0;
        }
    if (target < at || target - at >= mine)
        return;
    const float *p = a.target + (row0 + cur) * V, *q = drawn ? a.draft + (row0 + cur) * V : nullptr;
    for (int x = x0 + lane * W; x - lane * W < x1; x += 32 * W * U) {
        float r[U][W];
        load_lines<W, U>(p, q, x, x1, sm.scale, k, r);
        u64 line[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            Whole w;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (!drawn)
                    for (int m = 0; m < k; ++m)
                        r[i][j] = sm.gone[m] == x + i * 32 * W + j ? 0.0f : r[i][j];
                w.add(r[i][j]);
            }
            line[i] = w.sum();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const u64 all = warp_sum(line[i]);
            if (target - at < all) {
                u64 upto = line[i];  // of this lane and those before it
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
                    upto += lane >= o ? y : 0;
                }
                u64 here = at + upto - line[i];
                if (target >= here && target - here < line[i]) {
                    int j = 0;
#pragma unroll
                    for (int y = 0; y < W - 1; ++y) {
                        here += whole(r[i][y]);
                        j += here <= target;
                    }
                    st_checked(a.next + b, x + i * 32 * W + j);
                }
                return;
            }
            at += all;
        }
    }
}

cudaError_t launch_verify_tree(const VerifyArgs& a, cudaStream_t s)
{
    const size_t BN = (size_t)a.B * a.N;
    (void)BN;
    KIVI_SET_CHECK_BUFFERS(s, {{a.tokens, BN * 4}, {a.parent, BN * 4}, {a.n_draft, (size_t)a.B * 4}, {a.u, BN * 4},
                               {a.target, BN * a.V * 4}, {a.draft, BN * a.V * 4}, {a.path, BN * 4},
                               {a.counts, (size_t)a.B * 4}, {a.next, (size_t)a.B * 4}});
    int C = kMaxCluster;
    while (C > 1 && ((long long)a.B * C > 4 * sm_count() || a.V < C * kVerifyThreads))
        C /= 2;
    const int warps = C * kVerifyWarps, run = ((a.V + warps - 1) / warps + 127) / 128 * 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * C));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return a.V % 4 == 0 ? cudaLaunchKernelEx(&cfg, verify_tree_kernel<4>, a, run)
                        : cudaLaunchKernelEx(&cfg, verify_tree_kernel<1>, a, run);
}

#ifdef KIVI_CHECKS
int32_t check_word_verify() { return take_check_word(); }
#endif

}  // namespace kivi
