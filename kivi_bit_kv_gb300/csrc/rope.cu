// rope.cu -- queries, keys and values out of a layer's projections: head norms,
// rotary positions of one or several axes and the head-major layout of the
// other entry points, in one pass (kivi_norm_rope).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "kivi_device.cuh"
#include "kivi_f32x2.cuh"
#include "kivi_launch.h"

namespace kivi {

// Four warps a CTA and eight CTAs an SM (64 registers a thread): with 32 warps an SM
// and one step of each on its way the kernel is bound by DRAM.  In us, for the prompts
// of a layer (8 x 4096 tokens, 96 heads of 128 channels, fp16) and for 4260 fp32 tokens
// of 48 heads of 256 channels, interleaved:
//     warps a CTA, CTAs an SM, steps on their way    layer    fp32
//     4, 8, 1                                         246      49.5
//     4, 7 or 6, 1 (fewer warps, no spills)           254      50.4
//     8, 4, 1                                         249      50.0
//     16, 2, 1                                        254      51.1
//     8, 2, 2                                         294      55.3
// With pairs of halves the fp32 kernels keep 12 bytes a thread in local memory at 64
// registers, none with seven CTAs.  In us with eight, seven and six CTAs, for the same
// fp32 tokens: D = 256 50.2, 50.6, 51.7; D = 128 (96 heads) 50.8, 51.1, 52.2; D = 64
// (192 heads) 51.6, 50.7, 51.8.
constexpr int kRopeWarps = 4, kRopeCtas = 8;

// One 16-byte vector of channels: VW of them, as pairs of fp32.
template <class T>
struct Vec {
    static constexpr int VW = 16 / sizeof(T);
    uint4 raw;
    __device__ __forceinline__ F2 pair(int i) const
    {
        if constexpr (std::is_same<T, float>::value) {
            return i ? pack2(__uint_as_float(raw.z), __uint_as_float(raw.w))
                     : pack2(__uint_as_float(raw.x), __uint_as_float(raw.y));
        } else {
            const uint32_t w = u4_word(raw, i);
            if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(as_h2(w));
                return pack2(f.x, f.y);
            } else {
                return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            }
        }
    }
};

__device__ __forceinline__ uint32_t half_pair(F2 a)
{
    const float2 f = unpack2(a);
    return h2_bits(__floats2half2_rn(f.x, f.y));
}
// VW channels of a head in fp16.
template <int VW>
__device__ __forceinline__ void store_chans(uint16_t* p, const F2 (&x)[VW / 2])
{
    if constexpr (VW == 8)
        st_checked(reinterpret_cast<uint4*>(p), make_uint4(half_pair(x[0]), half_pair(x[1]), half_pair(x[2]), half_pair(x[3])));
    else
        st_checked(reinterpret_cast<uint2*>(p), make_uint2(half_pair(x[0]), half_pair(x[1])));
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

// Steps (of 32 / (D/16) heads) of one group of heads.
struct RopeGroup {
    const void* in;
    int64_t sequence, token, head;  // strides
    const float* weight;            // or NULL
    uint16_t* out;
    int heads, steps;
};
struct RopeArgs {
    RopeGroup g[3];  // queries, keys, values
    const float* inv_freq;
    const int32_t *axis, *pos, *base, *n_tok;
    float eps;
    int B, N, rot, n_axes;
    int per;         // steps of a warp
};

// One warp per token and run of `per` steps; neighbouring warps take neighbouring
// tokens.  A lane holds 16 channels of a head, in vectors of 16 bytes so placed that a
// load of the warp reads whole lines: with pairs of halves two vectors whose channels
// pair with one another (p and p + rot/2; beyond the rotated channels any two),
// interleaved each vector has its pairs in itself.  The next step is on its way while
// one is worked on.
template <class T, int D, bool INTER>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeCtas)
norm_rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int L = D / 16, HS = 32 / L;  // lanes a head, heads a step
    constexpr int VW = Vec<T>::VW, NV = 16 / VW, HW = VW / 2;
    __shared__ __align__(16) float s_cos[kRopeWarps][D / 2];
    __shared__ __align__(16) float s_sin[kRopeWarps][D / 2];
    // A programmatic dependent: its CTAs may be scheduled while the kernel before it ends,
    // and read and write nothing until that is done.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const long long w = (long long)blockIdx.x * kRopeWarps + warp;
    const int tokens = a.B * a.N;
    const int token = (int)(w % tokens), b = token / a.N, i = token % a.N;
    const int qk = a.g[0].steps + a.g[1].steps, all = qk + a.g[2].steps;
    const int first = (int)min(w / tokens * a.per, (long long)all), end = min(first + a.per, all);
    if (first >= end || (a.n_tok && i >= ld_prior(a.n_tok + b)))
        return;
    const int half = a.rot / 2, j = lane % L, hl = lane / L;
    // channels of the lane's vectors, and of their first pair in the table of turns
    int chan[NV], pair[NV];
    bool turned[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (INTER) {
            chan[v] = VW * (j + L * v);
            pair[v] = chan[v] / 2;
            turned[v] = chan[v] < a.rot;
        } else {
            const int p = VW * (j + L * (v / 2));  // first channel of the pair of vectors
            turned[v] = p < half;
            const int mate = turned[v] ? half : (D - a.rot) / 2;
            chan[v] = (turned[v] ? p : half + p) + (v % 2) * mate;
            pair[v] = p;
        }
    }
    // where a step's heads are, and the vectors of a step
    auto load = [&](int s, Vec<T> (&x)[NV]) {
        if (s >= end)
            return;
        const int n = s < a.g[0].steps ? 0 : s < qk ? 1 : 2;
        const RopeGroup& g = a.g[n];
        const int h = min((s - (n == 0 ? 0 : n == 1 ? a.g[0].steps : qk)) * HS + hl, g.heads - 1);
        const T* src = static_cast<const T*>(g.in) + (b * g.sequence + i * g.token + h * g.head);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            x[v].raw = ld_prior(reinterpret_cast<const uint4*>(src + chan[v]));
    };
    Vec<T> next[NV];
    load(first, next);
    if (first < qk && half > 0) {
        const int base = a.base ? ld_prior(a.base + b) : 0;
        for (int p = lane; p < half; p += 32) {
            int at = i;
            if (a.pos) {
                const int ax = a.axis ? min(max(ld_prior(a.axis + p), 0), a.n_axes - 1) : 0;
                at = ld_prior(a.pos + (size_t)ax * tokens + token);
            }
            const float2 cs = turn((int)((unsigned)at + (unsigned)base), ld_prior(a.inv_freq + p));
            s_cos[warp][p] = cs.x;
            s_sin[warp][p] = cs.y;
        }
        __syncwarp();
    }
    auto work = [&](int s, const Vec<T> (&x)[NV]) {
        const int n = s < a.g[0].steps ? 0 : s < qk ? 1 : 2;
        const RopeGroup& g = a.g[n];
        const int h = (s - (n == 0 ? 0 : n == 1 ? a.g[0].steps : qk)) * HS + hl;
        F2 y[NV][HW];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int k = 0; k < HW; ++k)
                y[v][k] = x[v].pair(k);
        if (g.weight) {
            F2 ss = mul2(y[0][0], y[0][0]);
#pragma unroll
            for (int k = 1; k < NV * HW; ++k)
                ss = fma2(y[k / HW][k % HW], y[k / HW][k % HW], ss);
            float sum = unpack2(ss).x + unpack2(ss).y;
#pragma unroll
            for (int o = 1; o < L; o <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const F2 r = both(rsqrtf(sum * (1.0f / D) + a.eps));
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int k = 0; k < HW; k += 2) {
                    const float4 wt = ld_prior(reinterpret_cast<const float4*>(g.weight + chan[v] + 2 * k));
                    y[v][k] = mul2(y[v][k], mul2(r, pack2(wt.x, wt.y)));
                    y[v][k + 1] = mul2(y[v][k + 1], mul2(r, pack2(wt.z, wt.w)));
                }
        }
        if (n < 2) {
#pragma unroll
            for (int v = 0; v < NV; v += INTER ? 1 : 2) {
                if (!turned[v])
                    continue;
                const float *c = &s_cos[warp][pair[v]], *sn = &s_sin[warp][pair[v]];
                if constexpr (INTER) {
#pragma unroll
                    for (int k = 0; k < HW; ++k) {
                        const float2 u = unpack2(y[v][k]);
                        y[v][k] = fma2(pack2(u.y, u.x), pack2(-sn[k], sn[k]), mul2(y[v][k], both(c[k])));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < HW; ++k) {
                        const F2 cc = pack2(c[2 * k], c[2 * k + 1]), ss = pack2(sn[2 * k], sn[2 * k + 1]);
                        const F2 u = y[v][k], z = y[v + 1][k];
                        y[v][k] = fma2(z, minus(ss), mul2(u, cc));
                        y[v + 1][k] = fma2(u, ss, mul2(z, cc));
                    }
                }
            }
        }
        if (h < g.heads) {
            uint16_t* dst = g.out + (((size_t)b * g.heads + h) * a.N + i) * D;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                store_chans<VW>(dst + chan[v], y[v]);
        }
    };
    for (int s = first; s < end; ++s) {
        Vec<T> x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v)
            x[v] = next[v];
        load(s + 1, next);
        work(s, x);
    }
}

template <class T, int D>
static cudaError_t launch_rope(const kivi_cache& c, const kivi_heads& h, cudaStream_t s)
{
    constexpr int HS = 512 / D;
    RopeArgs a = {};
    a.g[0] = {h.q_in, h.q_strides[0], h.q_strides[1], h.q_strides[2], h.q_weight, h.q, h.Hq, 0};
    a.g[1] = {h.k_in, h.k_strides[0], h.k_strides[1], h.k_strides[2], h.k_weight, h.k, c.H, 0};
    a.g[2] = {h.v_in, h.v_strides[0], h.v_strides[1], h.v_strides[2], nullptr, h.v, c.H, 0};
    int steps = 0;
    for (RopeGroup& g : a.g)
        steps += g.steps = g.in ? (g.heads + HS - 1) / HS : 0;
    a.inv_freq = h.inv_freq;
    a.axis = h.axis;
    a.pos = h.pos;
    a.base = h.base;
    a.n_tok = h.n_tok;
    a.eps = h.eps;
    a.B = c.B;
    a.N = h.N;
    a.rot = h.rot;
    a.n_axes = h.n_axes;
    const long long tokens = (long long)c.B * h.N;
    // Steps of a warp: as many as leave 128 warps an SM, four times what is resident.  A
    // long run forms its angles once; short ones end more evenly (the fp32 tokens
    // above: 49.5 us with 128, 50.9 with 32, 51.4 with 256; the layer takes all its 24
    // steps with any).
    a.per = (int)std::max(1ll, std::min((long long)steps, tokens * steps / (128ll * sm_count())));
    const long long warps = tokens * ((steps + a.per - 1) / a.per);
    const unsigned grid = (unsigned)((warps + kRopeWarps - 1) / kRopeWarps);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * kRopeWarps);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return h.interleaved ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, D, true>, a)
                         : cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, D, false>, a);
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
// The values of a strided input that a call may read.
static CallBuf heads_of(const kivi_cache& c, const kivi_heads& a, const void* in, const int64_t* strides, int heads)
{
    const int32_t dims[3] = {c.B, a.N, heads};
    const Span s = strided_span(in, dims, strides, 3, c.D, a.dtype == KIVI_F32 ? 4 : 2);
    return {reinterpret_cast<const void*>(s.lo), s.hi - s.lo};
}
#endif

cudaError_t launch_norm_rope(const kivi_cache& c, const kivi_heads& a, cudaStream_t s)
{
    const size_t out = (size_t)c.B * a.N * c.D * 2;
    (void)out;
    KIVI_SET_CHECK_BUFFERS(s, {heads_of(c, a, a.q_in, a.q_strides, a.Hq), heads_of(c, a, a.k_in, a.k_strides, c.H),
                               heads_of(c, a, a.v_in, a.v_strides, c.H), {a.q_weight, (size_t)c.D * 4},
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
