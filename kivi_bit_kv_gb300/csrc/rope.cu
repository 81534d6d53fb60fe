// rope.cu -- queries, keys and values out of a layer's projections: head norms,
// rotary positions of one or several axes and the head-major layout of the
// other entry points, in one pass (kivi_norm_rope).
#include <cuda_bf16.h>

#include <algorithm>

#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

constexpr int kRopeWarps = 8;

// Sixteen channels of a head in fp32: two vectors of eight.
struct Chans {
    float x[2][8];
};

__device__ __forceinline__ void load8(const __half* p, float (&x)[8])
{
    const uint4 v = ld_nc(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(as_h2(u4_word(v, i)));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8])
{
    const uint4 v = ld_nc(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u4_word(v, i) << 16);
        x[2 * i + 1] = __uint_as_float(u4_word(v, i) & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = ld_nc_f4(p), b = ld_nc_f4(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8])
{
    uint4 v;
    v.x = h2_bits(__floats2half2_rn(x[0], x[1]));
    v.y = h2_bits(__floats2half2_rn(x[2], x[3]));
    v.z = h2_bits(__floats2half2_rn(x[4], x[5]));
    v.w = h2_bits(__floats2half2_rn(x[6], x[7]));
    st_checked(reinterpret_cast<uint4*>(p), v);
}

// (cos, sin) of position * f.  The angle in half turns, a = position f / pi, is
// formed in two terms: f / pi as hi + lo (1 / pi in two terms itself), the position
// as a multiple of 4096 and a rest, both exact in fp32, and each product's rounding
// error from an fma.  Whole turns leave every term before the terms are added, so
// that the sum keeps an absolute error near 2^-24 for |a| below 2^24.
__device__ __forceinline__ float2 turn(int position, float f)
{
    constexpr float kInvPiHi = 0.318309886183790671538f;
    constexpr float kInvPiLo = (float)(0.318309886183790671538 - (double)kInvPiHi);
    const float hi = __fmul_rn(f, kInvPiHi);
    const float lo = __fmaf_rn(f, kInvPiLo, __fmaf_rn(f, kInvPiHi, -hi));
    float sum = 0.0f, err = 0.0f;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        const float x = part == 0 ? (float)(position >> 12) * 4096.0f : (float)(position & 4095);
        const float t = __fmul_rn(x, hi);
        err += __fmaf_rn(x, lo, __fmaf_rn(x, hi, -t));
        sum += t - 2.0f * rintf(0.5f * t);
    }
    float2 cs;
    sincospif(sum + err, &cs.y, &cs.x);
    return cs;
}

// One warp per token and run of `per` steps; a step is 32 / (D/16) heads, a lane
// 16 channels of one.  In pairs of halves a lane's two vectors of eight are
// (8j, rot/2 + 8j), beyond the rotated channels their successors; interleaved
// pairs lie inside a lane's 16 neighbouring channels.
template <class T, int D, bool INTER>
__global__ void __launch_bounds__(32 * kRopeWarps)
norm_rope_kernel(kivi_heads a, int B, int H, int per)
{
    constexpr int L = D / 16, HS = 32 / L;  // lanes a head, heads a step
    __shared__ float2 s_turn[kRopeWarps][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const long long w = (long long)blockIdx.x * kRopeWarps + warp;
    const int tokens = B * a.N;
    const int token = (int)(w % tokens), b = token / a.N, i = token % a.N;
    const int qs = a.q_in ? (a.Hq + HS - 1) / HS : 0, ks = a.k_in ? (H + HS - 1) / HS : 0;
    const int vs = a.v_in ? (H + HS - 1) / HS : 0;
    const int first = (int)min(w / tokens * per, (long long)(qs + ks + vs)), end = min(first + per, qs + ks + vs);
    if (first >= end || (a.n_tok && i >= ldg_checked(a.n_tok + b)))
        return;
    const int half = a.rot / 2, j = lane % L;
    if (first < qs + ks) {
        const int base = a.base ? ldg_checked(a.base + b) : 0;
        for (int p = lane; p < half; p += 32) {
            int at = i;
            if (a.pos) {
                const int ax = a.axis ? min(max(ldg_checked(a.axis + p), 0), a.n_axes - 1) : 0;
                at = ldg_checked(a.pos + (size_t)ax * tokens + token);
            }
            s_turn[warp][p] = turn((int)((unsigned)at + (unsigned)base), ldg_checked(a.inv_freq + p));
        }
        __syncwarp();
    }
    const bool turned = 16 * j < a.rot;
    const int c0 = INTER ? 16 * j : turned ? 8 * j : a.rot + 16 * (j - a.rot / 16);
    const int c1 = !INTER && turned ? half + 8 * j : c0 + 8;
    for (int s = first; s < end; ++s) {
        const int group = s < qs ? 0 : s < qs + ks ? 1 : 2;
        const int heads = group == 0 ? a.Hq : H;
        const int h = (s - (group == 0 ? 0 : group == 1 ? qs : qs + ks)) * HS + lane / L;
        const int64_t* st = group == 0 ? a.q_strides : group == 1 ? a.k_strides : a.v_strides;
        const T* in = static_cast<const T*>(group == 0 ? a.q_in : group == 1 ? a.k_in : a.v_in);
        const float* weight = group == 0 ? a.q_weight : group == 1 ? a.k_weight : nullptr;
        uint16_t* out = group == 0 ? a.q : group == 1 ? a.k : a.v;
        Chans y = {};
        if (h < heads) {
            const T* src = in + b * st[0] + i * st[1] + h * st[2];
            load8(src + c0, y.x[0]);
            load8(src + c1, y.x[1]);
        }
        if (weight) {
            float ss = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                ss = fmaf(y.x[k / 8][k % 8], y.x[k / 8][k % 8], ss);
#pragma unroll
            for (int o = 1; o < L; o <<= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const float4 wt = ld_nc_f4(weight + (v ? c1 : c0) + k);
                    y.x[v][k] *= r * wt.x, y.x[v][k + 1] *= r * wt.y;
                    y.x[v][k + 2] *= r * wt.z, y.x[v][k + 3] *= r * wt.w;
                }
        }
        if (group < 2 && turned) {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float2 cs = s_turn[warp][8 * j + p];
                float& u = INTER ? y.x[p / 4][2 * p % 8] : y.x[0][p];
                float& v = INTER ? y.x[p / 4][2 * p % 8 + 1] : y.x[1][p];
                const float u0 = u;
                u = u0 * cs.x - v * cs.y;
                v = v * cs.x + u0 * cs.y;
            }
        }
        if (h < heads) {
            uint16_t* dst = out + (((size_t)b * heads + h) * a.N + i) * D;
            store8(dst + c0, y.x[0]);
            store8(dst + c1, y.x[1]);
        }
    }
}

template <class T, int D>
static cudaError_t launch_rope(const kivi_cache& c, const kivi_heads& a, cudaStream_t s)
{
    constexpr int HS = 512 / D;
    const int steps = (a.q_in ? (a.Hq + HS - 1) / HS : 0) + (a.k_in ? (c.H + HS - 1) / HS : 0) +
                      (a.v_in ? (c.H + HS - 1) / HS : 0);
    const long long tokens = (long long)c.B * a.N;
    const int per = (int)std::max(1ll, std::min((long long)steps, tokens * steps / (32ll * sm_count())));
    const long long warps = tokens * ((steps + per - 1) / per);
    const unsigned grid = (unsigned)((warps + kRopeWarps - 1) / kRopeWarps);
    if (a.interleaved)
        norm_rope_kernel<T, D, true><<<grid, 32 * kRopeWarps, 0, s>>>(a, c.B, c.H, per);
    else
        norm_rope_kernel<T, D, false><<<grid, 32 * kRopeWarps, 0, s>>>(a, c.B, c.H, per);
    return cudaGetLastError();
}

template <class T>
static cudaError_t launch_rope_d(const kivi_cache& c, const kivi_heads& a, cudaStream_t s)
{
    switch (c.D) {
    case 64: return launch_rope<T, 64>(c, a, s);
    case 128: return launch_rope<T, 128>(c, a, s);
    default: return launch_rope<T, 256>(c, a, s);
    }
}

#ifdef KIVI_CHECKS
// Bytes from the first to the last element of a strided input.
static size_t extent(const kivi_cache& c, const kivi_heads& a, const int64_t* st, int heads)
{
    const int64_t last = (c.B - 1) * st[0] * (c.B > 1) + (a.N - 1) * st[1] * (a.N > 1) +
                         (heads - 1) * st[2] * (heads > 1) + c.D;
    return (size_t)last * (a.dtype == KIVI_F32 ? 4 : 2);
}
#endif

cudaError_t launch_norm_rope(const kivi_cache& c, const kivi_heads& a, cudaStream_t s)
{
    const size_t out = (size_t)c.B * a.N * c.D * 2;
    (void)out;
    KIVI_SET_CHECK_BUFFERS(s, {{a.q_in, extent(c, a, a.q_strides, a.Hq)}, {a.k_in, extent(c, a, a.k_strides, c.H)},
                               {a.v_in, extent(c, a, a.v_strides, c.H)}, {a.q_weight, (size_t)c.D * 4},
                               {a.k_weight, (size_t)c.D * 4}, {a.inv_freq, (size_t)a.rot * 2},
                               {a.axis, (size_t)a.rot * 2}, {a.pos, (size_t)a.n_axes * c.B * a.N * 4},
                               {a.base, (size_t)c.B * 4}, {a.n_tok, (size_t)c.B * 4}, {a.q, out * a.Hq},
                               {a.k, out * c.H}, {a.v, out * c.H}});
    switch (a.dtype) {
    case KIVI_F16: return launch_rope_d<__half>(c, a, s);
    case KIVI_BF16: return launch_rope_d<__nv_bfloat16>(c, a, s);
    default: return launch_rope_d<float>(c, a, s);
    }
}

#ifdef KIVI_CHECKS
int32_t check_word_rope() { return take_check_word(); }
#endif

}  // namespace kivi
