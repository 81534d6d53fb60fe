// verify.cu -- verification of drafted tokens against the target's probabilities
// from given random numbers (kivi_verify_tree).
#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;

__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }  // NaN to 0

// A probability as a multiple of 2^-42: sums of up to 2^20 of these are exact.
__device__ __forceinline__ unsigned long long whole(float r)
{
    return (unsigned long long)__float2ll_rn(r * 0x1p42f);
}

__device__ __forceinline__ float scale_of(unsigned long long z)
{
    return z ? (float)__ddiv_rn(0x1p42, (double)z) : 0.0f;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

struct VerifySmem {
    int parent[KIVI_MAX_DRAFT], token[KIVI_MAX_DRAFT], path[KIVI_MAX_DRAFT], gone[KIVI_MAX_DRAFT];
    float u[KIVI_MAX_DRAFT], p[KIVI_MAX_DRAFT], q[KIVI_MAX_DRAFT];
    float scale[KIVI_MAX_DRAFT];  // s after k rejections
    unsigned long long part[kVerifyWarps];
};

// Residual of a value after k rejections of drawn tokens.
__device__ __forceinline__ float residual(float r, float q, const float* scale, int k)
{
    for (int n = 0; n < k; ++n)
        r = fmaxf(__fsub_rn(__fmul_rn(r, scale[n]), q), 0.0f);
    return r;
}

// One CTA per sequence; a warp sums a run of neighbouring tokens.
__global__ void __launch_bounds__(kVerifyThreads)
verify_tree_kernel(VerifyArgs a)
{
    __shared__ VerifySmem sm;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid / 32, N = a.N, V = a.V;
    const int n = a.n_draft ? min(max(ldg_checked(a.n_draft + b), 0), N) : N;
    const size_t row0 = (size_t)b * N;
    const bool drawn = a.draft != nullptr;
    for (int i = tid; i < n; i += kVerifyThreads) {
        int par = i ? ldg_checked(a.parent + row0 + i) : -1;
        const int x = i ? ldg_checked(a.tokens + row0 + i) : -1;
        if (par < 0 || par >= i || x < 0 || x >= V)
            par = -1;
        sm.parent[i] = par;
        sm.token[i] = x;
        sm.u[i] = ldg_checked(a.u + row0 + i);
        if (par >= 0) {
            sm.p[i] = clamp01(ldg_checked(a.target + (row0 + par) * V + x));
            sm.q[i] = drawn ? clamp01(ldg_checked(a.draft + (row0 + par) * V + x)) : 1.0f;
        }
    }
    if (tid == 0) {
        sm.path[0] = 0;
        sm.scale[0] = 1.0f;
    }
    __syncthreads();
    const int run = ((V + kVerifyWarps - 1) / kVerifyWarps + 31) / 32 * 32;
    const int x0 = min(warp * run, V), x1 = min(x0 + run, V);
    const float *p = a.target, *q = a.draft;
    // Sum of w(rho) at node cur after k rejections, rejected tokens included if they
    // were not drawn.
    auto sum = [&](int cur, int k) {
        p = a.target + (row0 + cur) * V;
        q = a.draft + (row0 + cur) * V;
        unsigned long long z = 0;
        for (int x = x0 + lane; x < x1; x += 32)
            z += whole(drawn ? residual(clamp01(ldg_checked(p + x)), clamp01(ldg_checked(q + x)), sm.scale, k)
                             : clamp01(ldg_checked(p + x)));
        z = warp_sum(z);
        __syncthreads();
        if (lane == 0)
            sm.part[warp] = z;
        __syncthreads();
        z = 0;
        for (int w = 0; w < kVerifyWarps; ++w)
            z += sm.part[w];
        return z;
    };
    int cur = 0, k = 0, count = n > 0 ? 1 : 0;
    unsigned long long z = 0;
    for (int i = 1; i < n; ++i) {
        if (sm.parent[i] != cur)
            continue;
        float r = sm.p[i];
        if (drawn)
            r = residual(r, sm.q[i], sm.scale, k);
        else
            for (int m = 0; m < k; ++m)
                r = sm.gone[m] == sm.token[i] ? 0.0f : r;
        if (__fmul_rn(sm.u[i], sm.q[i]) < __fmul_rn(r, sm.scale[k])) {
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
            sm.gone[k] = sm.token[i];
            sm.scale[k + 1] = scale_of(z);
        }
        __syncthreads();
        ++k;
    }
    if (n > 0 && k == 0)
        z = sum(cur, 0);
    if (n > 0 && z == 0 && k > 0) {
        k = 0;
        z = sum(cur, 0);
    }
    __syncthreads();
    if (warp == 0) {
        if (lane == 0) {
            a.counts[b] = count;
            int next = -1;
            if (n > 0 && z > 0) {
                const float u0 = sm.u[0];
                const unsigned d = u0 >= 1.0f ? 0xffffffffu : u0 > 0.0f ? (unsigned)(u0 * 0x1p32f) : 0u;
                const unsigned long long t = (__umul64hi(z, (unsigned long long)d << 32));
                unsigned long long at = 0;
                for (int x = 0; x < V; ++x) {
                    float r = clamp01(ldg_checked(p + x));
                    if (drawn)
                        r = residual(r, clamp01(ldg_checked(q + x)), sm.scale, k);
                    else
                        for (int m = 0; m < k; ++m)
                            r = sm.gone[m] == x ? 0.0f : r;
                    at += whole(r);
                    if (at > t) {
                        next = x;
                        break;
                    }
                }
            }
            a.next[b] = next;
        }
    }
    for (int i = tid; i < N; i += kVerifyThreads)
        st_checked(a.path + row0 + i, i < count ? sm.path[i] : -1);
}

cudaError_t launch_verify_tree(const VerifyArgs& a, cudaStream_t s)
{
    const size_t BN = (size_t)a.B * a.N;
    (void)BN;
    KIVI_SET_CHECK_BUFFERS(s, {{a.tokens, BN * 4}, {a.parent, BN * 4}, {a.n_draft, (size_t)a.B * 4}, {a.u, BN * 4},
                               {a.target, BN * a.V * 4}, {a.draft, BN * a.V * 4}, {a.path, BN * 4},
                               {a.counts, (size_t)a.B * 4}, {a.next, (size_t)a.B * 4}});
    verify_tree_kernel<<<a.B, kVerifyThreads, 0, s>>>(a);
    return cudaGetLastError();
}

#ifdef KIVI_CHECKS
int32_t check_word_verify() { return take_check_word(); }
#endif

}  // namespace kivi
