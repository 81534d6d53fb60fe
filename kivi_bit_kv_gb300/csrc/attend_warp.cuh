// attend_warp.cuh -- kivi_sparse_attention and kivi_tree_attention for up to
// sixteen query rows of a KV head: a decode step of a grouped-query set, a
// small tree.
//
// The mathematics is attend.cuh's (softmax over "virtual" tokens, K_hat and
// V_hat exactly as kivi_dequant materializes them, weights as two fp16 terms,
// a lazily moved reference maximum, fp32 sums).  With few rows the time goes
// into rebuilding K_hat and V_hat from codes, not into the products, and the
// hand-offs of a tcgen05 pipeline (operands through shared memory to the
// tensor core, TMEM back, several barriers a tile) cost more than the
// warp-level products they feed: this kernel takes one third of the
// instructions per token and no barrier at all.
//
// Work.  A unit is 32 virtual tokens.  Every warp of the grid takes a
// contiguous range of the units of all rows (row: a sequence's KV head), so no
// two warps ever wait for one another.  A row inside one range is finished
// there; a row that ranges cut leaves partial (o, m, l) in the workspace,
// merged by attend_warp_combine_kernel.  The split and every sum's order depend
// only on sizes and lengths.
//
// A warp's unit: lanes 0 .. 2 have bulk copies (codes, scales, zeros) of the
// next unit's keys and values under way, each into its one buffer as soon as
// this unit's has been read;
//   keys    lane = channel: 32 codes -> 64 bytes of K_hat [channel][token];
//   S^T     m16n8k16, A = K_hat (ldmatrix.trans), B = the rows' Q in registers;
//   P^T     in registers, turned into B operands by movmatrix;
//   values  lane = token: a row of V_hat [token][channel], over K_hat;
//   O^T     m16n8k16, A = V_hat^T (ldmatrix.trans), B = P^T, both terms.
// Tokens and channels keep attend.cuh's order inside runs of 16.
//
// Every wait on an mbarrier gives up after some two seconds: it records
// KIVI_ETIMEOUT in the workspace's status word; the warp then leaves once its
// copies have landed (a bounded wait as well).
//
// Measured: one row a KV head over 1024 listed tokens and the residual of 64
// ragged int2 sequences of 32 heads (418 MB): 161 us, 2.6 TB/s; 8 rows over a
// 2065-token int4 prefix of 32 x 32 heads (420 MB): 170 us, 2.5 TB/s; 16 rows
// over eight int2 sequences of 4096 tokens (152 MB): 124 us.  Chains of
// dependent instructions bound it: some 1200 instructions a unit of 4096
// elements of K and of V each, issued in 52 % of the cycles by the four warps
// that a scheduler's registers and shared memory hold; ALU and shared memory are
// busy half of the time.  Deeper unrolling made it slower (instruction fetch).
#pragma once

#include "attend.cuh"

namespace kivi {

// A sequence's counts, in units: quantized units, then fp16 ones.
struct WarpSeq {
    int Tq, nq, res, nd, nu, nt;
};
__device__ __forceinline__ WarpSeq warp_seq(const kivi_cache& c, const AttendArgs& a, int lgG, int b)
{
    const AttSeq q = att_seq(c, a, lgG, b);
    WarpSeq s;
    s.Tq = q.Tq;
    s.nq = q.nq;
    s.res = q.len - q.Tq;
    s.nd = q.nd;
    s.nu = q.nq >> 5;
    s.nt = q.nt == 0 ? 0 : max(1, s.nu + ((s.res + s.nd + 31) >> 5));
    return s;
}
struct WarpWalk {
    int b, h, j;
    WarpSeq s;
};
__device__ __forceinline__ void warp_next(WarpWalk& w, const kivi_cache& c, const AttendArgs& a, int lgG)
{
    if (++w.j < w.s.nt)
        return;
    w.j = 0;
    if (++w.h < c.H)
        return;
    w.h = 0;
#pragma unroll 1
    while (++w.b < c.B) {
        w.s = warp_seq(c, a, lgG, w.b);
        if (w.s.nt > 0)
            return;
    }
    w.b = c.B - 1;  // only if a length was changed meanwhile: stay inside the arrays
}

// The split of all units into ranges of `base` units, the first `rem` of them
// one longer, and where this warp's lies.  32 bits hold every unit number: the
// codes of a unit take 1 KB of device memory at least, a row's ring more.
struct WarpRange {
    int first, n, base, rem;
    // the range that unit u lies in
    __device__ __forceinline__ int of(int u) const
    {
        const int longer = rem * (base + 1);
        return u < longer ? u / (base + 1) : rem + (u - longer) / base;
    }
};

// Range `index` of up to `count` (empty beyond the last) and the position of its
// first unit.  One warp.
static __device__ __noinline__ void warp_locate(const kivi_cache* c, const AttendArgs* a, int lgG, int index, int count,
                                                WarpRange* range, WarpWalk* first)
{
    const int lane = threadIdx.x & 31;
    int total = 0;
    WarpWalk w;
    w.b = lane;
    w.s.nt = 0;
#pragma unroll 1
    for (int b = lane; b - lane < c->B; b += 32) {
        if (b < c->B)
            w.s = warp_seq(*c, *a, lgG, b);
        total += __reduce_add_sync(0xffffffffu, b < c->B ? w.s.nt * c->H : 0);
    }
    // A unit a range or more, and 40 ranges a row on average: past that merging
    // the pieces costs more than the warps save (four sequences of 8 heads and
    // 69 units: 17.7 us with a unit each, 16.6 with two).  For few rows that are
    // long it is too few: the ranges of one sequence of 32768 tokens have 26 units
    // (8 query rows: 78 us with one KV head, 84 with eight).
    const unsigned least = total > 0 ? (total - 1) / 40u / (unsigned)(c->B * c->H) + 1 : 1;
    count = min(count, least > 1 ? (int)((total - 1) / least + 1) : total);
    WarpRange r = {0, 0, 1, 0};
    if (index < count) {
        r.base = (int)((unsigned)total / (unsigned)count);
        r.rem = total - r.base * count;
        r.first = index * r.base + min(index, r.rem);
        r.n = r.base + (index < r.rem);
    }
    if (lane == 0)
        *range = r;
    __syncwarp();
    if (r.n == 0)
        return;
    int before = 0;
#pragma unroll 1
    for (; w.b - lane < c->B; w.b += 32) {
        if (c->B > 32 && w.b < c->B)  // else as in the first pass
            w.s = warp_seq(*c, *a, lgG, w.b);
        const int n = w.b < c->B ? w.s.nt * c->H : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o);
            inc += lane >= o ? t : 0;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, r.first < before + inc);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                const unsigned at = r.first - (before + inc - n);
                w.h = (int)(at / (unsigned)w.s.nt);
                w.j = (int)(at - (unsigned)w.h * w.s.nt);
                *first = w;
            }
            __syncwarp();
            return;
        }
        before = __shfl_sync(0xffffffffu, before + inc, 31);
    }
    // first < total, so only if a length was changed meanwhile
    if (lane == 0)
        range->n = 0;
    __syncwarp();
}

// An 8 x 8 matrix of halves, transposed across the warp.
__device__ __forceinline__ uint32_t mov_trans(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// K_hat of a unit from its stage: lane = channel (and 32, 64, ... further);
// rows of 64 bytes per channel, 16-byte chunk c at c ^ (channel / 2) % 4, so
// that eight neighbouring channels' chunks fall in eight different columns.
template <int D, int BITS>
__device__ __forceinline__ void warp_keys(const uint8_t* st, uint8_t* hat, int lane, int kub)
{
    const float* sc = reinterpret_cast<const float*>(st + kub);
#pragma unroll 2
    for (int ch = lane; ch < D; ch += 32) {
        const float s = sc[ch], z = sc[D + ch];
        uint8_t* row = hat + ch * 64;
        const int x = ((ch >> 1) & 3) << 4;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[BITS / 2], h[8];
            run_words<BITS>(st + hf * (BITS / 2) * D * 4 + ch * 4, D * 4, w);
            hat16<BITS>(w, s, z, h);
            *reinterpret_cast<uint4*>(row + ((32 * hf) ^ x)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(row + ((32 * hf + 16) ^ x)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
}

// V_hat of a unit: lane = token position; rows of 2 D bytes per token, chunk c
// at c ^ token % 8.  A lane takes 16 bytes of codes at a time, starting at a
// chunk of its own, so that eight lanes read different banks whatever the
// bytes of a token.
template <int D, int BITS>
__device__ __forceinline__ void warp_values(const uint8_t* st, uint8_t* hat, int lane, int vub, int lgG)
{
    constexpr int ROW = D * BITS / 8, NCH = ROW / 16, CPC = 128 / BITS;  // code bytes, chunks, channels of a chunk
    constexpr int SH = ROW <= 16 ? 3 : ROW == 32 ? 2 : ROW == 64 ? 1 : 0;
    const int tok = run16(lane), NG = D >> lgG;
    const float* sc = reinterpret_cast<const float*>(st + vub) + tok * NG;
    const float* zr = sc + 32 * NG;
    uint8_t* row = hat + lane * (2 * D);
    const int x = (lane & 7) << 4;
#pragma unroll 1
    for (int j = 0; j < NCH; ++j) {
        const int ck = (j + (lane >> SH)) & (NCH - 1);
        const uint4 v = *reinterpret_cast<const uint4*>(st + tok * ROW + ck * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        constexpr int RUNS = CPC < 32 ? 1 : 2;  // runs of 16 channels that share statistics (G >= 32)
#pragma unroll
        for (int p = 0; p < CPC / (16 * RUNS); ++p) {
            const int g = (ck * CPC + 32 * p) >> lgG;
            const float sv = sc[g], zv = zr[g];
#pragma unroll
            for (int r = RUNS * p; r < RUNS * (p + 1); ++r) {
                uint32_t y[BITS / 2], h[8];
#pragma unroll
                for (int k = 0; k < BITS / 2; ++k)
                    y[k] = w[r * (BITS / 2) + k];
                hat16<BITS>(y, sv, zv, h);
                uint8_t* dst = row + ck * (CPC * 2);
                if constexpr (CPC >= 64) {  // a chunk covers whole 128-byte lines: the swizzle stays inside them
                    *reinterpret_cast<uint4*>(dst + ((32 * r) ^ x)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(dst + ((32 * r + 16) ^ x)) = make_uint4(h[4], h[5], h[6], h[7]);
                } else {
                    const int c0 = ck * (CPC * 2) + 32 * r;
                    *reinterpret_cast<uint4*>(row + (c0 ^ x)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(row + ((c0 + 16) ^ x)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
            }
        }
    }
}

// The fp16 token at a lane's position (null: none, or no row attends it) as a
// row [token][channel] laid out like V_hat's: its keys in channel order, its
// values in run order.
template <int D>
static __device__ __noinline__ void warp_fp16_keys(const uint16_t* src, uint8_t* hat, int lane)
{
    uint8_t* row = hat + lane * (2 * D);
    const int x = (lane & 7) << 4;
#pragma unroll 8
    for (int c = 0; c < 2 * D; c += 16) {
        if (src)
            cp_async16(row + (c ^ x), reinterpret_cast<const uint8_t*>(src) + c);
        else
            *reinterpret_cast<uint4*>(row + (c ^ x)) = make_uint4(0u, 0u, 0u, 0u);
    }
    cp_async_commit();
    cp_async_wait_all();
}
template <int D, bool DRAFTS>
static __device__ __noinline__ bool warp_fp16_values(const uint16_t* src, uint8_t* hat, int lane, bool draft)
{
    bool cleared = false;
    uint8_t* row = hat + lane * (2 * D);
    const int x = (lane & 7) << 4;
#pragma unroll 2
    for (int c0 = 0; c0 < D; c0 += 16) {
        uint4 y = make_uint4(0u, 0u, 0u, 0u), z = y;
        if (src) {
            y = ldg_checked(reinterpret_cast<const uint4*>(src + c0));
            z = ldg_checked(reinterpret_cast<const uint4*>(src + c0) + 1);
        }
        uint32_t q[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
        if (DRAFTS && draft)
            cleared |= clear_nonfinite(q);
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int sel = k & 1 ? 0x7632 : 0x5410;
            o[2 * k] = __byte_perm(q[k >> 1], q[2 + (k >> 1)], sel);
            o[2 * k + 1] = __byte_perm(q[4 + (k >> 1)], q[6 + (k >> 1)], sel);
        }
        *reinterpret_cast<uint4*>(row + ((c0 * 2) ^ x)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(row + ((c0 * 2 + 16) ^ x)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    return cleared;
}
// Four 8 x 8 b16 matrices, not transposed.
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// Adds to the M rows of output at dst the values that are not finite of the
// drafts which they attend.
template <int D>
static __device__ __noinline__ void warp_add_nonfinite(const AttendArgs* a, const uint16_t* v, int b, int nd, int M,
                                                       float* dst, int lane)
{
    __syncwarp();  // the rows are stored
#pragma unroll 1
    for (int x = lane; x < nd * D; x += 32) {
        const int j = x / D, ch = x % D;
        const float y = nonfinite(v + x);
        if (y == 0.0f)
            continue;
#pragma unroll 1
        for (int row = 0; row < M; ++row) {
            const int i = row % a->N;
            if (i < nd && (ldg_checked(a->mask + (size_t)b * a->N + i) >> j) & 1)
                st_checked(dst + (size_t)row * D + ch, ld_checked(dst + (size_t)row * D + ch) + y);
        }
    }
}

template <int D, int NT, int B>
__global__ void __launch_bounds__(32 * WarpCfg<D, NT>::WARPS, 1)
attend_warp_kernel(const __grid_constant__ kivi_cache c, const __grid_constant__ AttendArgs a,
                   const __grid_constant__ WarpPlan pl, float* __restrict__ ws)
{
    using C = WarpCfg<D, NT>;
    constexpr int NCOL = 2 * NT;  // rows (columns of S^T) of a lane
    extern __shared__ __align__(128) uint8_t att_smem[];
    __shared__ uint64_t s_full[C::WARPS][2];
    __shared__ WarpWalk s_walk[C::WARPS];
    __shared__ WarpRange s_range[C::WARPS];
    __shared__ int s_abort[C::WARPS], s_dirty[C::WARPS];  // dirty: values of some draft were cleared
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int g = lane >> 2, tq = lane & 3;
    // neighbouring ranges on different SMs: few ranges, or the longer ones, are
    // spread over all of them
    const int index = warp * gridDim.x + blockIdx.x, count = gridDim.x * pl.warps;
    int* status = reinterpret_cast<int*>(ws);
    if (lane == 0) {
        mbar_init(&s_full[warp][0], 1);
        mbar_init(&s_full[warp][1], 1);
        s_abort[warp] = s_dirty[warp] = 0;
        if (index == 0)
            st_checked(status, KIVI_OK);
        mbar_fence_init();
    }
    warp_locate(&c, &a, pl.lgG, index, count, &s_range[warp], &s_walk[warp]);
    const int n = s_range[warp].n;
    int4* cuts = reinterpret_cast<int4*>(ws + kAttHeaderFloats);
    if (!pl.by_row && lane == 0)
        st_checked(cuts + index, make_int4(-1, 0, 0, 0));
    asm volatile("griddepcontrol.launch_dependents;");
    if (n == 0)
        return;
    uint8_t* hat = att_smem + (size_t)warp * pl.bytes;
    uint8_t* const stage[2] = {hat + C::HAT, hat + C::HAT + pl.kst};
    const float sl2 = a.sm_scale * 1.4426950408889634f;

    WarpWalk w = s_walk[warp], x = w;  // this unit, the next one
    const bool starts_mid = w.j > 0;
    const int b0 = w.b, h0 = w.h;
    int phase[2] = {0, 0};
    bool go = false, xgo = false;      // quantized and attended: its copies are issued
    int xt0 = 0;                       // first token of the next unit
    bool ok = true;

    // Where unit x of the walk lies: its list entry is loaded well before it
    // decides whether the unit is copied, and from which token.
    int entry = 0;
    auto place = [&]() {
        if (a.blocks && x.j < x.s.nu)
            entry = ldg_checked(a.blocks + ((size_t)x.b * c.H + x.h) * a.n_keep + (x.j * 32 >> pl.lgG));
    };
    auto resolve = [&]() {
        xgo = x.j < x.s.nu;
        xt0 = x.j * 32;
        if (a.blocks) {
            xgo = xgo && entry >= 0 && entry < x.s.Tq >> pl.lgG;
            xt0 = (entry << pl.lgG) + (xt0 & (c.G - 1));
        }
    };
    // Copies of its keys (0) or values (1): codes, scales and zeros by lanes 0, 1
    // and 2, whose pointers into the next unit's row are kept.
    const uint8_t* row_at[2] = {nullptr, nullptr};
    const uint32_t kbytes = lane == 0 ? pl.kub : D * 4, vbytes = lane == 0 ? pl.vub : 32 * (D >> pl.lgG) * 4;
    const uint32_t koff = lane == 0 ? 0 : pl.kub + (lane - 1) * kbytes, voff = lane == 0 ? 0 : pl.vub + (lane - 1) * vbytes;
    const int klg = lane == 0 ? 5 : pl.lgG;
    auto row_start = [&]() {
        const size_t bh = (size_t)x.b * c.H + x.h;
        const void* k = lane == 0 ? (const void*)c.kq : lane == 1 ? (const void*)c.kscale : (const void*)c.kzero;
        const void* v = lane == 0 ? (const void*)c.vq : lane == 1 ? (const void*)c.vscale : (const void*)c.vzero;
        row_at[0] = static_cast<const uint8_t*>(k) + bh * (c.Tmax >> klg) * kbytes;
        row_at[1] = static_cast<const uint8_t*>(v) + bh * (c.Tmax >> 5) * vbytes;
    };
    auto issue = [&](int which) {
        uint64_t* bar = &s_full[warp][which];
        if (lane == 0)
            mbar_arrive_tx(bar, which == 0 ? pl.kst : pl.vst);
        __syncwarp();
        if (lane < 3) {
            const uint32_t bytes = which == 0 ? kbytes : vbytes;
            const uint8_t* src = row_at[which] + (size_t)(xt0 >> (which == 0 ? klg : 5)) * bytes;
            if (KIVI_IN_RANGE(src, bytes))
                bulk_g2s(stage[which] + (which == 0 ? koff : voff), src, bytes, bar);
        }
    };
    auto wait = [&](int which) {
        if (!__all_sync(0xffffffffu, att_wait(&s_full[warp][which], phase[which] & 1, &s_abort[warp], status)))
            ok = false;
        ++phase[which];
    };
    // the fp16 token at this lane's position of unit w, or null
    auto fp16_src = [&](const uint16_t* ringp, const uint16_t* draft) -> const uint16_t* {
        const int f = (w.j - w.s.nu) * 32 + lane, j = f - w.s.res, RG = c.R + c.G;
        const size_t bh = (size_t)w.b * c.H + w.h;
        if (j < 0) {
            int s = w.s.Tq % RG + f;
            s = s >= RG ? s - RG : s;
            return ringp + (bh * RG + s) * D;
        }
        if (j >= w.s.nd)
            return nullptr;
        bool seen = false;  // by any row (N <= 16 here: one word a row)
#pragma unroll 1
        for (int i = 0; i < w.s.nd; ++i)
            seen |= (ldg_checked(a.mask + (size_t)w.b * a.N + i) >> j) & 1;
        return seen ? draft + (bh * a.N + j) * D : nullptr;
    };

    float o[D / 16][NT][4];
    float l[NCOL], ref[NCOL];
    uint32_t q[D / 16][NT][2];

    row_start();
    place();
    resolve();
    if (xgo) {
        issue(0);
        issue(1);
    }
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
        go = xgo;
        const bool first = i == 0 || w.j == 0;
        x = w;
        if (i + 1 < n) {
            warp_next(x, c, a, pl.lgG);
            if (x.j == 0)
                row_start();
            place();
        }
        if (__builtin_expect(first, 0)) {
            // rows 8 nt + g, channels 16 k + 2 tq (+ 1), + 8
            const uint16_t* base = a.q + ((size_t)w.b * a.Hq + (size_t)w.h * (a.Hq / c.H)) * a.N * D + 2 * tq;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = 8 * nt + g;
                const bool have = row < pl.M && (!a.k || row % a.N < w.s.nd);
                const uint32_t* p = reinterpret_cast<const uint32_t*>(base + (size_t)(have ? row : 0) * D);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    q[k][nt][0] = have ? ldg_checked(p + 8 * k) : 0u;
                    q[k][nt][1] = have ? ldg_checked(p + 8 * k + 4) : 0u;
                }
            }
#pragma unroll
            for (int k = 0; k < NCOL; ++k) {
                l[k] = 0.0f;
                ref[k] = kAttNoRef;
            }
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[m][nt][k] = 0.0f;
        }
        const bool quant = w.j < w.s.nu;
        if (go || !quant) {
            if (go) {
                wait(0);
                switch (B ? B : c.bits_k) {
                case 2: warp_keys<D, B ? B : 2>(stage[0], hat, lane, pl.kub); break;
                case 4: warp_keys<D, B ? B : 4>(stage[0], hat, lane, pl.kub); break;
                default: warp_keys<D, B ? B : 8>(stage[0], hat, lane, pl.kub); break;
                }
            } else {
                warp_fp16_keys<D>(fp16_src(c.kres, a.k), hat, lane);
            }
            __syncwarp();
            xgo = false;
            if (i + 1 < n)
                resolve();
            if (xgo)
                issue(0);

            // S^T: tokens 16 m + g (+ 8), rows 8 nt + 2 tq (+ 1).  The tensor core
            // truncates its sums: a chain of n steps of 16 channels loses some (n + 1) / 2
            // units of 2^-23 of its sum.  Chains of 64 channels side by side, added
            // with rounding, lose 2.5 at every D; one chain through all channels loses
            // 8.5 at D = 256, where it is also slower (203 against 200 us, 8 rows of B 8,
            // H 32, T 4096), and 4.5 at D = 128 (169.6 against 170.8 us, 8 int4 rows).
            float s[2][NT][4];
            auto scores = [&](auto&& load) {
                constexpr int KC = 4, NC = D / 16 / KC;  // steps of a chain, chains
                float y[NC][2][NT][4];
#pragma unroll
                for (int x = 0; x < NC; ++x)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[x][m][nt][k] = 0.0f;
#pragma unroll
                for (int k = 0; k < KC; ++k)
#pragma unroll
                    for (int x = 0; x < NC; ++x)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t f[4];
                            load(f, k + x * KC, m);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(y[x][m][nt], f[0], f[1], f[2], f[3], q[k + x * KC][nt][0], q[k + x * KC][nt][1]);
                        }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
#pragma unroll
                            for (int x = 1; x < NC; ++x)
                                add_pair(y[0][m][nt] + k, y[x][m][nt] + k);
                            s[m][nt][k] = y[0][m][nt][k];
                            s[m][nt][k + 1] = y[0][m][nt][k + 1];
                        }
            };
            if (__builtin_expect(!go, 0)) {
                // fp16 keys: blocks token + 8 (lane / 8) % 2, channel chunk lane / 16
                const int tok = (lane & 7) + (lane & 8), ck = lane >> 4;
                const uint32_t at = smem_addr(hat) + tok * (2 * D), sw = (tok & 7) << 4;
                scores([&](uint32_t (&f)[4], int k, int m) { ldsm_x4(f, at + m * (32 * D) + (((2 * k + ck) << 4) ^ sw)); });
            } else {
                // lane's row address of the four 8 x 8 blocks: channels + 8 (lane / 16), token chunk (lane / 8) % 2
                const int r = lane & 7, chb = r + ((lane >> 4) << 3), ck = (lane >> 3) & 1;
                const uint32_t at = smem_addr(hat) + chb * 64, sw = ((chb >> 1) & 3) << 4;
                scores([&](uint32_t (&f)[4], int k, int m) { ldsm_x4_t(f, at + k * 1024 + ((((2 * m + ck) << 4)) ^ sw)); });
            }
            // logits in log2 units; -inf where the row does not attend the token
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; k += 2)
                        mul_pair(s[m][nt] + k, sl2);
            const int f0 = (w.j - w.s.nu) * 32;
            if (__builtin_expect(!quant && f0 + 32 > w.s.res, 0)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = (8 * nt + 2 * tq + e) % a.N;
                        const uint64_t word =
                            a.k && row < w.s.nd ? ldg_checked(a.mask + (size_t)w.b * a.N + row) : 0ull;
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const int j = f0 + 16 * m + 8 * hf + g - w.s.res;
                                if (j >= 0 && !(j < w.s.nd && (word >> j) & 1))
                                    s[m][nt][2 * hf + e] = -INFINITY;
                            }
                    }
                __syncwarp();
            }
            float top = -INFINITY;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        float y[2] = {s[m][nt][k], s[m][nt][k + 1]};
                        sub_pair(y, ref + 2 * nt);
                        top = fmaxf(top, fmaxf(y[0], y[1]));
                    }
            if (__builtin_expect(__any_sync(0xffffffffu, top > kAttLimit), 0)) {
                // the references move to the rows' maxima so far
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                        const float old = ref[2 * nt + e];
                        const float next = fmaxf(old, fabsf(m) < 1048576.0f ? m - kAttShift : m);
                        const float alpha = next == old ? 1.0f : ex2_ftz(old - next);
                        ref[2 * nt + e] = next;
                        l[2 * nt + e] *= alpha;
#pragma unroll
                        for (int t = 0; t < D / 16; ++t) {
                            o[t][nt][e] *= alpha;
                            o[t][nt][2 + e] *= alpha;
                        }
                    }
            }
            // weights, and the operands of the second product
            uint32_t ph[2][NT][2], pl2[2][NT][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float p[2] = {s[m][nt][2 * hf], s[m][nt][2 * hf + 1]};
                        sub_pair(p, ref + 2 * nt);
                        p[0] = ex2_ftz(p[0]);
                        p[1] = ex2_ftz(p[1]);
                        add_pair(l + 2 * nt, p);
                        uint32_t hi, lo;
                        split_pair(p, hi, lo);
                        ph[m][nt][hf] = mov_trans(hi);
                        pl2[m][nt][hf] = mov_trans(lo);
                    }
            __syncwarp();  // K_hat has been read

            if (go) {
                wait(1);
                switch (B ? B : c.bits_v) {
                case 2: warp_values<D, B ? B : 2>(stage[1], hat, lane, pl.vub, pl.lgG); break;
                case 4: warp_values<D, B ? B : 4>(stage[1], hat, lane, pl.vub, pl.lgG); break;
                default: warp_values<D, B ? B : 8>(stage[1], hat, lane, pl.vub, pl.lgG); break;
                }
            } else {
                if (f0 + 32 <= w.s.res)
                    warp_fp16_values<D, false>(fp16_src(c.vres, a.v), hat, lane, false);
                else if (warp_fp16_values<D, true>(fp16_src(c.vres, a.v), hat, lane, f0 + lane >= w.s.res))
                    s_dirty[warp] = 1;
            }
            __syncwarp();
            if (xgo)
                issue(1);
            {
                // blocks: token + 8 (lane / 16), channel chunk (lane / 8) % 2
                const int tok = (lane & 7) + ((lane >> 4) << 3), ck = (lane >> 3) & 1;
                const uint32_t at = smem_addr(hat) + tok * (2 * D), sw = (tok & 7) << 4;
                // The unit's sums start at zero and are added to the row's with rounded
                // additions: the tensor core truncates, and a chain through every unit
                // of a long row would lose in one direction.  TG tiles at a time, so
                // that their products do not wait for one another.
                constexpr int TG = NT == 1 ? 4 : 2;  // 8 int4 rows: 169 us with 4, 172 with 2; 16 rows lack registers
#pragma unroll
                for (int t0 = 0; t0 < D / 16; t0 += TG) {
                    uint32_t f[2][TG][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int t = 0; t < TG; ++t)
                            ldsm_x4_t(f[m][t], at + m * (32 * D) + (((2 * (t0 + t) + ck) << 4) ^ sw));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float sum[TG][4];
#pragma unroll
                        for (int t = 0; t < TG; ++t)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                sum[t][k] = 0.0f;
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
#pragma unroll
                            for (int t = 0; t < TG; ++t)
                                mma_f16(sum[t], f[m][t][0], f[m][t][1], f[m][t][2], f[m][t][3], ph[m][nt][0], ph[m][nt][1]);
#pragma unroll
                            for (int t = 0; t < TG; ++t)
                                mma_f16(sum[t], f[m][t][0], f[m][t][1], f[m][t][2], f[m][t][3], pl2[m][nt][0], pl2[m][nt][1]);
                        }
#pragma unroll
                        for (int t = 0; t < TG; ++t)
#pragma unroll
                            for (int k = 0; k < 4; k += 2)
                                add_pair(o[t0 + t][nt] + k, sum[t] + k);
                    }
                }
            }
            __syncwarp();  // V_hat has been read
        } else {  // a skipped unit: the next one's copies all the same
            xgo = false;
            if (i + 1 < n)
                resolve();
            if (xgo) {
                issue(0);
                issue(1);
            }
        }
        const bool tail = w.j == w.s.nt - 1;
        if (__builtin_expect(tail || i == n - 1, 0)) {
            const bool mid = starts_mid && w.b == b0 && w.h == h0;
            float scale[NCOL];
#pragma unroll
            for (int k = 0; k < NCOL; ++k) {
#pragma unroll
                for (int e = 4; e < 32; e <<= 1)
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], e);
                scale[k] = 1.0f;
            }
            float* dst;
            if (tail && !mid) {
                dst = a.out + ((size_t)w.b * a.Hq + (size_t)w.h * (a.Hq / c.H)) * a.N * D;
#pragma unroll
                for (int k = 0; k < NCOL; ++k)
                    scale[k] = row_scale(l[k]);
                if (pl.by_row && lane == 0)
                    st_checked(cuts + w.b * c.H + w.h, make_int4(-1, 0, 0, 0));
            } else {
                dst = warp_part(ws, D, pl.M, index, mid ? 0 : 1);
                if (g == 0) {
#pragma unroll
                    for (int k = 0; k < NCOL; ++k) {
                        const int row = 8 * (k >> 1) + 2 * tq + (k & 1);
                        if (row < pl.M) {
                            st_checked(dst + pl.M * D + row, ref[k]);
                            st_checked(dst + pl.M * D + pl.M + row, copysignf(l[k], s_dirty[warp] ? -1.0f : 1.0f));
                        }
                    }
                }
                if (!tail && !mid && lane == 0) {
                    // the row starts in this range; where its last unit lies
                    const WarpRange& r = s_range[warp];
                    st_checked(cuts + (pl.by_row ? w.b * c.H + w.h : index),
                               make_int4(r.of(r.first + n - 1 + (w.s.nt - 1 - w.j)), index, w.b, w.h));
                }
            }
#pragma unroll
            for (int k = 0; k < NCOL; ++k) {
                const int row = 8 * (k >> 1) + 2 * tq + (k & 1);
                if (row < pl.M && (!(tail && !mid) || !a.k || row % a.N < w.s.nd)) {
                    float* p = dst + (size_t)row * D;
#pragma unroll
                    for (int t = 0; t < D / 16; ++t) {
                        st_checked(p + run16(16 * t + g), o[t][k >> 1][k & 1] * scale[k]);
                        st_checked(p + run16(16 * t + g + 8), o[t][k >> 1][2 + (k & 1)] * scale[k]);
                    }
                }
            }
            if (__builtin_expect(s_dirty[warp] && tail && !mid, 0))
                warp_add_nonfinite<D>(&a, a.v + ((size_t)w.b * c.H + w.h) * a.N * D, w.b, w.s.nd, pl.M, dst, lane);
        }
        w = x;
    }
    // copies in flight have landed before the warp ends (none unless a wait gave up)
    if (!ok) {
        if (lane == 0)
            s_abort[warp] = 0;
        __syncwarp();
        for (int k = 0; k < 2; ++k)
            att_wait(&s_full[warp][k], phase[k] & 1, &s_abort[warp], nullptr);
    }
}

// Adds to the stored output of row (b, h), M query rows, the values that are
// not finite of the drafts which they attend.  All threads of the block.
static __device__ __noinline__ void warp_merge_nonfinite(const kivi_cache* c, const AttendArgs* a, int b, int h, int nd,
                                                         int M)
{
    const int D = c->D;
    float* dst = a->out + ((size_t)b * a->Hq + (size_t)h * M / a->N) * a->N * D;
    const uint16_t* v = a->v + ((size_t)b * c->H + h) * a->N * D;
    __syncthreads();  // the row is stored
#pragma unroll 1
    for (int x = threadIdx.x; x < M * D; x += blockDim.x) {
        const int i = x / D % a->N, ch = x % D;
        if (i >= nd)
            continue;
        const uint64_t word = ldg_checked(a->mask + (size_t)b * a->N + i);  // (N <= 16 here: one word a row)
        float y = 0.0f;
#pragma unroll 1
        for (int j = 0; j < nd; ++j)
            if ((word >> j) & 1)
                y += nonfinite(v + j * D + ch);
        if (y != 0.0f)
            st_checked(dst + x, ld_checked(dst + x) + y);
    }
}

// Merges the pieces of the rows that ranges cut, piece by piece in order: block
// (h, b) takes row (b, h) (few rows, 512 threads: each has many pieces), or
// block i the row that starts in range i and ends in a later one (256 threads).
//
// A record by row is written by the range in which its row ends or is cut, so
// one whose row has no unit (a sequence without drafts) holds whatever the
// workspace held: the block takes its row from its own index and leaves before
// it reads one.  Records by range are all written, and name their row.
template <bool BY_ROW>
__global__ void __launch_bounds__(BY_ROW ? 512 : 256)
attend_warp_combine_kernel(const __grid_constant__ kivi_cache c, const __grid_constant__ AttendArgs a, int M,
                           int ranges, float* __restrict__ ws)
{
    constexpr int T = BY_ROW ? 512 : 256;
    const int D = c.D;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 cut = ld_checked(reinterpret_cast<const int4*>(ws + kAttHeaderFloats) +
                                (BY_ROW ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x));
    const int last = cut.x, i = cut.y, b = BY_ROW ? blockIdx.y : cut.z, h = BY_ROW ? blockIdx.x : cut.w;
    // a kernel that gave up leaves its records as they were: stay inside the arrays
    const bool merge = i >= 0 && last > i && last < ranges;
    if (!BY_ROW && !(merge && b >= 0 && b < c.B && h >= 0 && h < c.H))
        return;
    const int nd = a.k ? (a.n_draft ? min(max(ldg_checked(a.n_draft + b), 0), a.N) : a.N) : 1;
    if (BY_ROW && !(merge && nd > 0))
        return;
    // 64 pieces at a time: their weights (a warp per row, a lane per two pieces),
    // then the weighted sum of their outputs, four channels a thread and the
    // pieces spread over the threads that are left
    constexpr int P = 64;
    __shared__ float s_w[16][P], s_m[16], s_l[16], s_f[16];
    __shared__ float4 s_o[T];
    const int t = threadIdx.x, lane = t & 31, n4 = M * D / 4;
    const int groups = n4 < T ? T / n4 : 1;
    bool dirty = false;  // some piece cleared values of drafts
    if (t < M) {
        s_m[t] = -INFINITY;
        s_l[t] = 0.0f;
    }
    float4 o[2];  // M D / 4 <= 16 x 128 / 4, 8 x 256 / 4: up to two a thread
#pragma unroll
    for (int k = 0; k < 2; ++k)
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = i; k0 <= last; k0 += P) {
        const int np = min(P, last + 1 - k0);
        bool cleared = false;
        __syncthreads();
#pragma unroll 1
        for (int r = t >> 5; r < M; r += T / 32) {
            float m[2], l[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int q = lane + 32 * k;
                const float* p = warp_part(ws, D, M, k0 + q, k0 + q == i) + M * D + r;
                m[k] = q < np ? ld_checked(p) : -INFINITY;
                l[k] = q < np ? ld_checked(p + M) : 0.0f;
                cleared |= signbit(l[k]);
                l[k] = fabsf(l[k]);
            }
            const float old = s_m[r], mx = fmaxf(old, redux_max(fmaxf(m[0], m[1])));
            float L = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float wk = m[k] == -INFINITY ? 0.0f : ex2_ftz(m[k] - mx);
                s_w[r][lane + 32 * k] = wk;
                L = fmaf(l[k], wk, L);
            }
#pragma unroll
            for (int e = 16; e > 0; e >>= 1)
                L += __shfl_xor_sync(0xffffffffu, L, e);
            const float f = old == mx ? 1.0f : ex2_ftz(old - mx);
            if (lane == 0) {
                s_l[r] = s_l[r] * f + L;
                s_m[r] = mx;
                s_f[r] = f;
            }
            __syncwarp();
        }
        dirty |= __syncthreads_or(cleared);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e4 = (t + k * T) % (groups * n4) % n4, grp = groups > 1 ? t / n4 : 0;
            if (grp >= groups || (k > 0 && t + k * T >= n4))
                continue;
            const int r = e4 * 4 / D;
            const float f = s_f[r];
            float4 x = make_float4(o[k].x * f, o[k].y * f, o[k].z * f, o[k].w * f);
#pragma unroll 8
            for (int q = grp; q < np; q += groups) {
                const float4 v =
                    ld_checked(reinterpret_cast<const float4*>(warp_part(ws, D, M, k0 + q, k0 + q == i) + 4 * e4));
                const float wq = s_w[r][q];
                x.x = fmaf(v.x, wq, x.x);
                x.y = fmaf(v.y, wq, x.y);
                x.z = fmaf(v.z, wq, x.z);
                x.w = fmaf(v.w, wq, x.w);
            }
            o[k] = x;
        }
    }
    if (groups > 1) {  // the groups' sums, in order
        s_o[t] = o[0];
        __syncthreads();
        if (t < n4)
            for (int k = 1; k < groups; ++k) {
                const float4 v = s_o[t + k * n4];
                o[0].x += v.x;
                o[0].y += v.y;
                o[0].z += v.z;
                o[0].w += v.w;
            }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e4 = t + k * T, r = e4 * 4 / D;
        if (e4 < n4 && r % a.N < nd) {
            const float inv = row_scale(s_l[r]);
            st_checked(reinterpret_cast<float4*>(
                           a.out + (((size_t)b * a.Hq + (size_t)h * (a.Hq / c.H)) * a.N) * D) + e4,
                       make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv));
        }
    }
    if (__builtin_expect(dirty, 0))
        warp_merge_nonfinite(&c, &a, b, h, nd, M);
}

// ----------------------------------------------------------------- launch ---

template <int D, int NT, int B>
cudaError_t attend_warp_launch(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s)
{
    using C = WarpCfg<D, NT>;
    auto kern = attend_warp_kernel<D, NT, B>;
    WarpPlan pl = warp_plan<D, NT>(c.G, c.bits_k, c.bits_v, a.Hq / c.H * a.N);
    if (pl.warps < 1)
        return cudaErrorInvalidConfiguration;
    const int smem = pl.warps * pl.bytes;
    static int allowed[64];
    cudaError_t e = allow_smem(kern, kAttSmem - kWarpStatic, allowed);
    if (e != cudaSuccess)
        return e;
    const int N = cmin(sm_count(), kAttMaxCTAs / 2);
    pl.by_row = (long long)c.B * c.H <= 2 * N;  // few rows: a block per row merges them, else one per range
    kern<<<N, 32 * pl.warps, smem, s>>>(c, a, pl, ws);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    // the combine's CTAs are scheduled while the attention drains
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = pl.by_row ? dim3(c.H, c.B) : dim3(N * pl.warps);
    cfg.blockDim = dim3(pl.by_row ? 512 : 256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pl.by_row ? attend_warp_combine_kernel<true> : attend_warp_combine_kernel<false>, c, a,
                              pl.M, N * pl.warps, ws);
}

}  // namespace kivi
