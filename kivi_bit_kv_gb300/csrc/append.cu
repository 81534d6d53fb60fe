// append.cu -- append one decoded token per sequence, flushing the oldest G
// residual tokens into the packed cache when the residual reaches R + G
// (CacheForge README, "How it works": recent tokens stay at higher precision;
// the quantization flow during decoding).
//
// Kernel 1, one CTA per (h, b): writes k, v into ring slot len mod (R+G) and,
// on a flush step, quantizes the G oldest ring tokens exactly like a prefix
// group (same lane quantizers as the encode kernels).  Kernel 2 advances
// len[b]; it runs after every CTA of kernel 1 has read the old length, so no
// CTA can observe a half-updated count.
#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

template <int BV, int G>
__device__ __forceinline__ void flush_values(const kivi_cache& c, size_t bh, int Tq)
{
    const int D = c.D, NG = D / G, RG = c.R + c.G;
    for (int task = threadIdx.x; task < G * NG; task += blockDim.x) {
        const int gi = task % NG, r = task / NG;
        const int t = Tq + r;
        const uint16_t* src = c.vres + (bh * RG + t % RG) * D + gi * G;
        uint4 raw[G / 8];
#pragma unroll
        for (int v = 0; v < G / 8; ++v)
            raw[v] = ld_checked(reinterpret_cast<const uint4*>(src + v * 8));
        quant_store_value_group<BV, G>(c, bh, t, gi, raw);
    }
}

// Keys of a flushed group: one G-token group per channel, lanes (s, j) with s
// fastest (S = G/16 lanes per channel column).
template <int BK, int S>
__device__ __forceinline__ void flush_keys(const kivi_cache& c, size_t bh, int Tq)
{
    const int D = c.D, RG = c.R + c.G, NC = D / kLaneChans;
    const int lane = threadIdx.x & 31;
    const unsigned smask = (((1u << S) - 1u) << (lane & ~(S - 1)));
    for (int task = threadIdx.x; task < S * NC; task += blockDim.x) {
        const int s = task % S, j = task / S;
        const int t0 = Tq + s * kLaneTokens;
        uint4 raw[kLaneTokens];
#pragma unroll
        for (int i = 0; i < kLaneTokens; ++i)
            raw[i] = ld_checked(reinterpret_cast<const uint4*>(c.kres + (bh * RG + (t0 + i) % RG) * D +
                                                                (size_t)j * kLaneChans));
        // RG and t0 are multiples of 16: the lane's 16 ring rows never wrap
        quant_store_key_lane<BK, S>(c, bh, t0, Tq / c.G, j, s, smask, raw,
                                    c.kres + (bh * RG + t0 % RG) * D + (size_t)j * kLaneChans, D);
    }
}

template <int BK, int BV>
__global__ void __launch_bounds__(128)
append_kernel(kivi_cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
              int32_t* status)
{
    const size_t bh = blockIdx.x;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    const int L = ld_checked(c.len + b);
    if (L + 1 > c.Tmax) {
        if (h == 0 && threadIdx.x == 0)
            atomicExch(status, KIVI_ECAPACITY);
        return;
    }
    const int D = c.D, G = c.G, RG = c.R + c.G;
    const int slot = L % RG;
    for (int i = threadIdx.x; i < D / kLaneChans; i += blockDim.x) {
        const size_t o = (bh * RG + slot) * D + (size_t)i * kLaneChans;
        const size_t in = bh * D + (size_t)i * kLaneChans;
        st_checked(reinterpret_cast<uint4*>(c.kres + o), ld_checked(reinterpret_cast<const uint4*>(k + in)));
        st_checked(reinterpret_cast<uint4*>(c.vres + o), ld_checked(reinterpret_cast<const uint4*>(v + in)));
    }
    const int Tq = quantized_tokens(L, G, c.R);
    if (L + 1 - Tq != RG)
        return;  // uniform over the CTA
    __syncthreads();  // the new token is visible to every thread of the CTA

    // keys, then values: G token rows x D/G channel groups, one lane per group
    switch (G) {
    case 32:
        flush_keys<BK, 2>(c, bh, Tq);
        flush_values<BV, 32>(c, bh, Tq);
        break;
    case 64:
        flush_keys<BK, 4>(c, bh, Tq);
        flush_values<BV, 64>(c, bh, Tq);
        break;
    default:
        flush_keys<BK, 8>(c, bh, Tq);
        flush_values<BV, 128>(c, bh, Tq);
        break;
    }
}

__global__ void advance_len_kernel(int32_t* len, int B, int Tmax)
{
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B) {
        const int L = ld_checked(len + b);
        if (L + 1 <= Tmax)
            st_checked(len + b, L + 1);
    }
}

template <int BK>
static void launch_append_bk(const kivi_cache& c, const uint16_t* k, const uint16_t* v,
                             int32_t* status, cudaStream_t s)
{
    const dim3 grid(c.B * c.H);
    switch (c.bits_v) {
    case 2: append_kernel<BK, 2><<<grid, 128, 0, s>>>(c, k, v, status); break;
    case 4: append_kernel<BK, 4><<<grid, 128, 0, s>>>(c, k, v, status); break;
    default: append_kernel<BK, 8><<<grid, 128, 0, s>>>(c, k, v, status); break;
    }
}

cudaError_t launch_append(const kivi_cache& c, const uint16_t* k, const uint16_t* v,
                          int32_t* status, cudaStream_t s)
{
    KIVI_SET_CHECK_RANGES(c, s, {{k, (size_t)c.B * c.H * c.D * 2}, {v, (size_t)c.B * c.H * c.D * 2}, {status, 4}});
    switch (c.bits_k) {
    case 2: launch_append_bk<2>(c, k, v, status, s); break;
    case 4: launch_append_bk<4>(c, k, v, status, s); break;
    default: launch_append_bk<8>(c, k, v, status, s); break;
    }
    advance_len_kernel<<<(c.B + 127) / 128, 128, 0, s>>>(c.len, c.B, c.Tmax);
    return cudaGetLastError();
}

// ------------------------------------------------------------ append path ---

// Status of appending the first n = counts[b] nodes of path row b to a
// sequence of L tokens; every thread of the warp calls it and gets the result.
__device__ __forceinline__ int path_status(const kivi_cache& c, int L, int n, const int32_t* row, int N, int P)
{
    if (L < 0 || n < 0 || n > P)
        return KIVI_EINVAL;
    bool bad = false;
    for (int i = threadIdx.x & 31; i < n; i += 32) {
        const int node = ldg_checked(row + i);
        bad |= node < 0 || node >= N;
    }
    if (__any_sync(0xffffffffu, bad))
        return KIVI_EINVAL;
    return (long long)L + n > c.Tmax ? KIVI_ECAPACITY : KIVI_OK;
}

// One CTA per (b, h).  The accepted tokens enter the ring in runs that end
// where the residual reaches R + G; there the oldest G tokens are flushed as
// append_kernel flushes them, and the next run reuses their slots.  Bound by
// latency: a dependent chain of length, path and token loads, then one store
// (16 x 8 B of D = 128 channels per token and head).  With the second
// kernel 3.6 us for one small sequence; 13 us for 64 sequences of 32 heads that
// keep up to eight tokens each, nine of which flush a group (16.5 MB).
template <int BK, int BV>
__global__ void __launch_bounds__(128)
append_path_kernel(kivi_cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int N,
                   const int32_t* __restrict__ path, int P, const int32_t* __restrict__ counts, int32_t* status)
{
    asm volatile("griddepcontrol.launch_dependents;");
    const size_t bh = blockIdx.x;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    const int L = ld_checked(c.len + b);
    const int n = ldg_checked(counts + b);
    const int32_t* row = path + (size_t)b * P;
    const int st = path_status(c, L, n, row, N, P);
    if (st != KIVI_OK) {  // uniform over the CTA
        if (st == KIVI_ECAPACITY && h == 0 && threadIdx.x == 0)
            atomicExch(status, st);
        return;
    }
    const int D = c.D, G = c.G, RG = c.R + c.G, NC = D / kLaneChans;
    for (int done = 0; done < n;) {
        const int Tq = quantized_tokens(L + done, G, c.R);
        const int res = L + done - Tq;  // < R + G
        const int m = min(RG - res, n - done);
        for (int i = threadIdx.x; i < m * NC; i += blockDim.x) {
            const int j = i / NC, ch = (i % NC) * kLaneChans;
            const size_t o = (bh * RG + (L + done + j) % RG) * D + ch;
            const size_t in = (bh * N + ldg_checked(row + done + j)) * D + ch;
            st_checked(reinterpret_cast<uint4*>(c.kres + o), ldg_checked(reinterpret_cast<const uint4*>(k + in)));
            st_checked(reinterpret_cast<uint4*>(c.vres + o), ldg_checked(reinterpret_cast<const uint4*>(v + in)));
        }
        done += m;
        if (res + m == RG) {
            __syncthreads();  // the ring is full and visible to every thread of the CTA
            switch (G) {
            case 32:
                flush_keys<BK, 2>(c, bh, Tq);
                flush_values<BV, 32>(c, bh, Tq);
                break;
            case 64:
                flush_keys<BK, 4>(c, bh, Tq);
                flush_values<BV, 64>(c, bh, Tq);
                break;
            default:
                flush_keys<BK, 8>(c, bh, Tq);
                flush_values<BV, 128>(c, bh, Tq);
                break;
            }
            __syncthreads();  // the flushed slots are read before the next run reuses them
        }
    }
}

// One warp per sequence: adds the tokens append_path_kernel appended.  Its CTAs
// start with that kernel's, which read `len`, and write once it has ended.  That
// kernel reports full sequences and this one bad arguments, so that the status
// of a call with both does not depend on which CTA is last.
__global__ void __launch_bounds__(128)
advance_path_kernel(kivi_cache c, int N, const int32_t* __restrict__ path, int P,
                    const int32_t* __restrict__ counts, int32_t* status)
{
    const int b = (int)(blockIdx.x * 4 + threadIdx.x / 32);
    if (b >= c.B)
        return;
    const int L = ld_checked(c.len + b), n = ldg_checked(counts + b);
    const int st = path_status(c, L, n, path + (size_t)b * P, N, P);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((threadIdx.x & 31) != 0)
        return;
    if (st == KIVI_OK)
        st_checked(c.len + b, L + n);
    else if (st == KIVI_EINVAL)
        atomicExch(status, st);
}

template <int BK>
static void launch_append_path_bk(const kivi_cache& c, const uint16_t* k, const uint16_t* v, int N,
                                  const int32_t* path, int P, const int32_t* counts, int32_t* status,
                                  cudaStream_t s)
{
    const dim3 grid(c.B * c.H);
    switch (c.bits_v) {
    case 2: append_path_kernel<BK, 2><<<grid, 128, 0, s>>>(c, k, v, N, path, P, counts, status); break;
    case 4: append_path_kernel<BK, 4><<<grid, 128, 0, s>>>(c, k, v, N, path, P, counts, status); break;
    default: append_path_kernel<BK, 8><<<grid, 128, 0, s>>>(c, k, v, N, path, P, counts, status); break;
    }
}

cudaError_t launch_append_path(const kivi_cache& c, const uint16_t* k, const uint16_t* v, int N,
                               const int32_t* path, int P, const int32_t* counts, int32_t* status,
                               cudaStream_t s)
{
    KIVI_SET_CHECK_RANGES(c, s, {{k, (size_t)c.B * c.H * N * c.D * 2}, {v, (size_t)c.B * c.H * N * c.D * 2},
                                 {path, (size_t)c.B * P * 4}, {counts, (size_t)c.B * 4}, {status, 4}});
    switch (c.bits_k) {
    case 2: launch_append_path_bk<2>(c, k, v, N, path, P, counts, status, s); break;
    case 4: launch_append_path_bk<4>(c, k, v, N, path, P, counts, status, s); break;
    default: launch_append_path_bk<8>(c, k, v, N, path, P, counts, status, s); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((c.B + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, advance_path_kernel, c, N, path, P, counts, status);
}

#ifdef KIVI_CHECKS
int32_t check_word_append() { return take_check_word(); }
#endif

}  // namespace kivi
