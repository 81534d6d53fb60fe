// probs.cu -- probabilities of rows of logits, one temperature per sequence
// (kivi_token_probs).
#include <cuda_bf16.h>

#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

constexpr int kProbsThreads = 512;

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// log2(e) / T, kept between the smallest normal and the largest finite number so
// that neither 0 * infinity nor infinity * 0 appears below: an infinite T gives
// equal weights, a tiny one only those of the largest logit.  NaN for a NaN T.
__device__ __forceinline__ float inverse_temperature(float T)
{
    constexpr float kLog2e = 1.44269504088896340736f;
    const float c = kLog2e / T;
    return isnan(c) ? c : fminf(fmaxf(c, 0x1p-126f), 0x1.fffffep127f);
}

// Weight of a logit; 0 for one of -infinity, and NaN for a NaN or for an infinite
// largest logit.
__device__ __forceinline__ float weight(float l, float m, float c) { return exp2f((l - m) * c); }

// One CTA per row: the largest logit, the sum of the weights, the quotients.
template <class T>
__global__ void __launch_bounds__(kProbsThreads)
token_probs_kernel(ProbsArgs a)
{
    __shared__ float s_m[kProbsThreads / 32], s_l[kProbsThreads / 32];
    __shared__ int s_first;
    const int b = blockIdx.x / a.N, i = blockIdx.x % a.N, tid = threadIdx.x;
    if (a.n_rows && i >= ldg_checked(a.n_rows + b))
        return;
    const T* src = static_cast<const T*>(a.logits) + b * a.batch_stride + i * a.row_stride;
    float* dst = a.probs + (size_t)blockIdx.x * a.V;
    const float temp = a.temperature ? ldg_checked(a.temperature + b) : 1.0f;
    const bool greedy = temp <= 0.0f;
    const float c = inverse_temperature(greedy ? 1.0f : temp);
    float m = -INFINITY;
    for (int x = tid; x < a.V; x += kProbsThreads)
        m = fmaxf(m, to_float(ldg_checked(src + x)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (tid % 32 == 0)
        s_m[tid / 32] = m;
    if (tid == 0)
        s_first = a.V;
    __syncthreads();
    for (int w = 0; w < kProbsThreads / 32; ++w)
        m = fmaxf(m, s_m[w]);
    float l = 0.0f;
    int first = a.V;
    const float ref = m == -INFINITY ? 0.0f : m;
    for (int x = tid; x < a.V; x += kProbsThreads) {
        const float v = to_float(ldg_checked(src + x));
        l += weight(v, ref, c);
        if (v == m)
            first = min(first, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, o);
    if (tid % 32 == 0)
        s_l[tid / 32] = l;
    if (first < a.V)
        atomicMin(&s_first, first);
    __syncthreads();
    l = 0.0f;
    for (int w = 0; w < kProbsThreads / 32; ++w)
        l += s_l[w];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a NaN sum stays
    for (int x = tid; x < a.V; x += kProbsThreads) {
        const float v = to_float(ldg_checked(src + x));
        float p = weight(v, ref, c) * inv;
        if (greedy && !isnan(l))
            p = l > 0.0f && x == s_first ? 1.0f : 0.0f;
        st_checked(dst + x, isnan(l) ? NAN : p);
    }
}

#ifdef KIVI_CHECKS
static size_t extent(const ProbsArgs& a)
{
    const int64_t last = (a.B > 1 ? (a.B - 1) * a.batch_stride : 0) + (a.N > 1 ? (a.N - 1) * a.row_stride : 0) + a.V;
    return (size_t)last * (a.dtype == KIVI_F32 ? 4 : 2);
}
#endif

cudaError_t launch_token_probs(const ProbsArgs& a, cudaStream_t s)
{
    KIVI_SET_CHECK_BUFFERS(s, {{a.logits, extent(a)}, {a.temperature, (size_t)a.B * 4}, {a.n_rows, (size_t)a.B * 4},
                               {a.probs, (size_t)a.B * a.N * a.V * 4}});
    const unsigned grid = (unsigned)a.B * (unsigned)a.N;
    switch (a.dtype) {
    case KIVI_F16: token_probs_kernel<__half><<<grid, kProbsThreads, 0, s>>>(a); break;
    case KIVI_BF16: token_probs_kernel<__nv_bfloat16><<<grid, kProbsThreads, 0, s>>>(a); break;
    default: token_probs_kernel<float><<<grid, kProbsThreads, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

#ifdef KIVI_CHECKS
int32_t check_word_probs() { return take_check_word(); }
#endif

}  // namespace kivi
