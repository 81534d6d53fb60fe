// attend.cu -- kivi_sparse_attention and kivi_tree_attention.
//
// The tokens a row attends form one sequence of "virtual" tokens: the tokens
// of its quantized groups (all of them, or the listed ones), the residual
// tokens, the drafted tokens.
#include "kivi_device.cuh"
#include "kivi_launch.h"

namespace kivi {

constexpr int kAttendThreads = 128;

__device__ __forceinline__ float hat(uint32_t code, float scale, float zero)
{
    return __half2float(__float2half_rn(__fmaf_rn((float)code, scale, zero)));
}

__global__ void __launch_bounds__(kAttendThreads)
attend_kernel(kivi_cache c, AttendArgs a, int* ws)
{
    constexpr int T = kAttendThreads;
    __shared__ float p_s[T], q_s[256];
    __shared__ long long src_s[T];
    __shared__ float red[T / 32];
    const int N = a.N, D = c.D, G = c.G, RG = c.R + c.G, gq = a.Hq / c.H;
    const int n = blockIdx.x % N, hq = (blockIdx.x / N) % a.Hq, b = blockIdx.x / N / a.Hq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const size_t bh = (size_t)b * c.H + hq / gq;
    if (blockIdx.x == 0 && tid == 0)
        ws[0] = KIVI_OK;
    const int nd = a.k ? (a.n_draft ? min(max(a.n_draft[b], 0), N) : N) : 0;
    if (a.k && n >= nd)
        return;
    const int len = min(max(c.len[b], 0), c.Tmax);
    const int Tq = quantized_tokens(len, G, c.R);
    const int nq = a.blocks ? min(a.n_keep, Tq / G) * G : Tq;
    const int total = nq + (len - Tq) + nd;
    const size_t row = ((size_t)b * a.Hq + hq) * N + n;
    for (int d = tid; d < D; d += T)
        q_s[d] = __half2float(__ushort_as_half(a.q[row * D + d]));
    __syncthreads();
    const int Pk = 32 / c.bits_k, Pv = 32 / c.bits_v;
    const uint32_t Mk = (1u << c.bits_k) - 1, Mv = (1u << c.bits_v) - 1;
    float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
    for (int v0 = 0; v0 < total; v0 += T) {
        const int vt = v0 + tid;
        float s = -INFINITY;
        long long src = -1;  // >= 0: token; ring slots and drafts follow at Tmax, Tmax + RG
        if (vt < nq) {
            int t = vt;
            if (a.blocks) {
                const int g = a.blocks[bh * a.n_keep + vt / G];
                t = g >= 0 && g < Tq / G ? g * G + vt % G : -1;
            }
            src = t;
        } else if (vt < nq + len - Tq) {
            src = c.Tmax + (Tq + vt - nq) % RG;
        } else if (vt < total) {
            const int j = vt - nq - (len - Tq);
            if (a.mask[((size_t)b * N + n) * ((N + 63) / 64) + j / 64] >> (j % 64) & 1)
                src = (long long)c.Tmax + RG + j;
        }
        if (src >= 0) {
            s = 0.0f;
            if (src < c.Tmax) {
                const size_t st = (bh * (c.Tmax / G) + src / G) * D;
                const int32_t* w = c.kq + (bh * (c.Tmax / Pk) + src / Pk) * D;
                const int sh = (int)(src % Pk) * c.bits_k;
                for (int d = 0; d < D; ++d)
                    s = fmaf(q_s[d], hat((uint32_t)w[d] >> sh & Mk, c.kscale[st + d], c.kzero[st + d]), s);
            } else {
                const uint16_t* r = src < c.Tmax + RG ? c.kres + (bh * RG + src - c.Tmax) * D
                                                      : a.k + (bh * N + src - c.Tmax - RG) * D;
                for (int d = 0; d < D; ++d)
                    s = fmaf(q_s[d], __half2float(__ushort_as_half(r[d])), s);
            }
            s *= a.sm_scale;
        }
        float mx = s;
        for (int i = 16; i > 0; i >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        if (lane == 0)
            red[warp] = mx;
        __syncthreads();
        float mn = m;
        for (int i = 0; i < T / 32; ++i)
            mn = fmaxf(mn, red[i]);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float alpha = expf(m - ref);
        p_s[tid] = expf(s - ref);
        src_s[tid] = src;
        m = mn;
        l *= alpha;
        o[0] *= alpha;
        o[1] *= alpha;
        __syncthreads();
        float lc = 0.0f, oc[2] = {0.0f, 0.0f};  // the chunk's sums: no chain of additions is longer than a chunk
        for (int i = 0; i < min(T, total - v0); ++i) {
            const float p = p_s[i];
            const long long t = src_s[i];
            lc += p;
            if (t < 0)
                continue;
            for (int k = 0, d = tid; d < D; d += T, ++k) {
                float x;
                if (t < c.Tmax) {
                    const size_t r = bh * c.Tmax + t;
                    x = hat((uint32_t)c.vq[r * (D / Pv) + d / Pv] >> (d % Pv * c.bits_v) & Mv,
                            c.vscale[r * (D / G) + d / G], c.vzero[r * (D / G) + d / G]);
                } else {
                    x = __half2float(__ushort_as_half(t < c.Tmax + RG ? c.vres[(bh * RG + t - c.Tmax) * D + d]
                                                                      : a.v[(bh * N + t - c.Tmax - RG) * D + d]));
                }
                oc[k] = fmaf(p, x, oc[k]);
            }
        }
        l += lc;
        o[0] += oc[0];
        o[1] += oc[1];
        __syncthreads();
    }
    for (int k = 0, d = tid; d < D; d += T, ++k)
        a.out[row * D + d] = l > 0.0f ? o[k] / l : 0.0f;
}

size_t attend_ws_bytes(const kivi_cache&, int, int) { return 16; }

cudaError_t launch_attend(const kivi_cache& c, const AttendArgs& a, void* ws, cudaStream_t s)
{
    attend_kernel<<<c.B * a.Hq * a.N, kAttendThreads, 0, s>>>(c, a, static_cast<int*>(ws));
    return cudaGetLastError();
}

#ifdef KIVI_CHECKS
int32_t check_word_attend() { return KIVI_OK; }
#endif

}  // namespace kivi
