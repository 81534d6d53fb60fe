// attend.cuh -- kivi_sparse_attention and kivi_tree_attention as one
// persistent kernel on the 5th-generation tensor cores.
//
// Mathematics.  The tokens a KV head's queries attend form one sequence of
// "virtual" tokens: those of its quantized groups (all, or the listed ones),
// the residual's, the drafted ones.  A row tile is NR query rows of one KV
// head (query heads x drafted tokens; they share every key and value), a tile
// 128 virtual tokens.  Per tile
//     S^T [128 tokens x NR rows] = K_hat Q^T       (tcgen05.mma, fp16 in, fp32 sum)
//     P^T = 2^(S^T log2e sm_scale - m + 13), m the running row maximum
//     O^T [D channels x NR rows] = V_hat^T P^T
// with K_hat, V_hat = fp16_rne(fmaf(code, scale, zero)) exactly as
// kivi_dequant materializes them.  P is split into two fp16 terms (about 22
// significant bits; the factor 2^13 keeps the second term of small weights out
// of fp16's subnormals) and the sums of P, the maxima and the output stay in
// fp32: a tile's O^T is read back from TMEM and added to the running output
// in registers, so no long chain of tensor-core additions builds up.
//
// Tokens lie on the M axis (TMEM lanes) of both products and rows on the N
// axis, so one row costs as little as one column: a decode step (one to
// sixteen rows) and a verified tree (up to 128 rows per tile) run the same
// code.  What a tile costs whatever the rows is rebuilding 2 x 128 x D fp16
// operands from codes.
//
// Work.  One CTA per SM takes a contiguous range of the tiles of all row
// tiles in order; a row tile cut by a range boundary leaves partial (o, m, l)
// in the workspace, merged by attend_combine_kernel.  The split and every
// sum's order depend only on sizes and lengths.
//
// Pipeline.  Sixteen worker warps share every step; a seventeenth issues the
// bulk copies of the packed codes and statistics into a ring of stages (one
// stage = the keys or the values of a tile).  Per tile i the workers
//     softmax of S(i) -> P; barrier, P(i) V(i) issued;
//     rebuild K(i+2);       barrier, K(i+2) Q issued;      [overlaps P V]
//     add O(i); rebuild V(i+1)                             [overlaps K Q]
// so both products run under the workers' arithmetic.  Worker warp w reads
// TMEM lanes 32 (w % 4) .. + 31 (tokens, later channels) and the NR/4 rows
// w / 4 of them: a row's state (m, the factor of the last tile, its share of
// l and o) never leaves the warps that own the row.
//
// Every wait on an mbarrier gives up after two seconds: it sets the abort
// flag and records KIVI_ETIMEOUT in the workspace's status word; the CTA then
// runs through without waiting, waits (bounded) for its copies, frees its
// TMEM and ends.
#pragma once

#include "decode_stream.cuh"

namespace kivi {

constexpr int kAttTile = 128;                 // tokens per tile
constexpr int kAttWorkers = 512;              // worker threads (16 warps)
constexpr int kAttThreads = kAttWorkers + 32; // and the copy warp
constexpr int kAttMaxCTAs = 160;              // workspace bound on the grid
constexpr int kAttMaxStages = 16;
constexpr int kAttDescs = 8;                  // tile descriptors kept in shared memory
constexpr int kAttCutInts = 8;
constexpr int kAttHeaderFloats = 4;
constexpr int kAttAtom = kAttTile * 128;      // bytes of 64 channels (128 B) of a tile's tokens
constexpr int kAttStaticSmem = 8 * 1024;      // bound on the kernel's static shared arrays
constexpr float kAttShift = 13.0f;            // weights are scaled by 2^13

// Rows per row tile for M query rows of a KV head: the next of 32, 64, 128,
// or 32 for D = 256, whose operands leave no shared memory for more.
inline int attend_rows(int D, int M) { return M <= 32 || D == 256 ? 32 : M <= 64 ? 64 : 128; }

// Workspace: header (status word), a cut descriptor per CTA, two partial
// (o [NR][D], m [NR], l [NR]) slots per CTA: slot 0 for a row tile that an
// earlier CTA started, slot 1 for one that starts here and ends later.
__host__ __device__ inline float* att_part(float* ws, int D, int NR, int cta, int slot)
{
    return ws + kAttHeaderFloats + kAttMaxCTAs * kAttCutInts + ((size_t)cta * 2 + slot) * NR * (D + 2);
}

template <int D, int NR>
struct AttCfg {
    static constexpr int NA = D / 64;                  // 64-channel atoms of a key row
    static constexpr int NAV = D == 64 ? 2 : D / 64;   // of a value row (M = 128 spans two)
    static constexpr int MH = D == 256 ? 2 : 1;        // 128-channel halves of the output
    static constexpr int NC = NR / 4;                  // rows of a warp
    static constexpr int CH = NC < 16 ? NC : 16;       // rows of one TMEM read
    static constexpr bool STACK = NR == 32;            // both terms of P side by side in one product
    static constexpr int PN = STACK ? 64 : NR;         // columns of the second product
    static constexpr int PASSES = STACK ? 1 : 2;
    static constexpr int PATOMS = STACK ? 1 : 2 * NR / 64;
    static constexpr int QBYTES = NA * NR * 128;
    static constexpr int O_K = 0;
    static constexpr int O_V = O_K + NA * kAttAtom;
    static constexpr int O_P = O_V + NAV * kAttAtom;
    static constexpr int O_Q = O_P + PATOMS * kAttAtom;  // two buffers
    static constexpr int O_RING = O_Q + 2 * QBYTES;
    static constexpr int TM_S = 0;                     // TMEM columns: S(even), S(odd), O
    static constexpr int TM_O = 2 * NR;
    static constexpr int TM_USED = 2 * NR + MH * PN;
    static constexpr int TM_COLS = TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;
    static constexpr int RING = kStreamSmemBytes - kAttStaticSmem - 1024 - O_RING;  // 1024: base alignment
    static_assert(D != 256 || NR == 32, "shared memory");
    static_assert(O_Q % 1024 == 0 && QBYTES % 1024 == 0, "operand alignment");
};

// Sizes the kernel needs besides the descriptor's.
struct AttPlan {
    int lgG, M, RT;       // log2 G, query rows of a KV head, row tiles
    int ns;               // ring stages
    int stage;            // bytes of a stage
    int kub, vub;         // code bytes of 32 tokens: keys, values
};

// ------------------------------------------------------------------ PTX ---

__device__ __forceinline__ void tc_alloc(uint32_t* dst, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_dealloc(uint32_t tm, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// N columns of this thread's TMEM lane; the values are there after tc_wait_ld,
// which names them so that no use can be scheduled before it.
__device__ __forceinline__ void tc_ld(float (&r)[8], uint32_t a)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void tc_ld(float (&r)[16], uint32_t a)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(a));
}
template <int N>
__device__ __forceinline__ void tc_wait_ld(float (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+f"(r[i]));
}

// Largest value over the warp, in every lane.
__device__ __forceinline__ float redux_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Shared-memory matrix descriptor, 128-byte swizzle (8 rows of 128 bytes per
// kilobyte): version 1 (bit 46), layout 2 (bits 61-63), byte offsets in
// sixteenths.  lead: stride between 64-element columns of an operand whose M
// or N axis is contiguous (unused for one whose K axis is).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp16 operands, fp32 sums, M = 128; mn: the M / N
// axes of both operands are contiguous in shared memory.
__host__ __device__ constexpr uint32_t mma_idesc(int n, bool mn)
{
    return (1u << 4) | (mn ? (1u << 15) | (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// ---------------------------------------------------------------- walker ---

// A sequence's token counts: quantized tokens attended, residual, drafts, and
// the tiles of each of its row tiles (0: nothing to write).
struct AttSeq {
    int len, Tq, nq, nd, total, nt;
};
__device__ __forceinline__ AttSeq att_seq(const kivi_cache& c, const AttendArgs& a, int lgG, int b)
{
    AttSeq s;
    s.len = min(max(ldg_checked(c.len + b), 0), c.Tmax);
    s.Tq = quantized_tokens(s.len, c.G, c.R);
    s.nq = a.blocks ? min(a.n_keep, s.Tq >> lgG) << lgG : s.Tq;
    s.nd = 0;
    if (a.k)
        s.nd = a.n_draft ? min(max(ldg_checked(a.n_draft + b), 0), a.N) : a.N;
    s.total = s.nq + (s.len - s.Tq) + s.nd;
    s.nt = a.k && s.nd == 0 ? 0 : max(1, (s.total + kAttTile - 1) / kAttTile);
    return s;
}

// Position in the sequence of tiles: sequence b, row rr = h RT + row tile,
// tile j of it.
struct AttWalk {
    int b, rr, j;
    AttSeq s;
};
__device__ __forceinline__ void att_next(AttWalk& w, const kivi_cache& c, const AttendArgs& a, int lgG, int RB)
{
    if (++w.j < w.s.nt)
        return;
    w.j = 0;
    if (++w.rr < RB)
        return;
    w.rr = 0;
    while (++w.b < c.B) {
        w.s = att_seq(c, a, lgG, w.b);
        if (w.s.nt > 0)
            return;
    }
}

// One warp: the tiles of all rows, and the position of tile `p` (any p with
// 0 <= p < total; p is a function of the total).
template <class F>
__device__ __forceinline__ long long att_locate(const kivi_cache& c, const AttendArgs& a, int lgG, int RB, F p_of,
                                                AttWalk& w)
{
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int b0 = 0; b0 < c.B; b0 += 32) {
        long long n = b0 + lane < c.B ? (long long)att_seq(c, a, lgG, b0 + lane).nt * RB : 0;
        for (int o = 16; o > 0; o >>= 1)
            n += __shfl_xor_sync(0xffffffffu, n, o);
        total += n;
    }
    const long long p = p_of(total);
    long long before = 0;
    w.b = w.rr = w.j = 0;
    for (int b0 = 0; b0 < c.B; b0 += 32) {
        const long long n = b0 + lane < c.B ? (long long)att_seq(c, a, lgG, b0 + lane).nt * RB : 0;
        long long inc = n;
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            inc += lane >= o ? t : 0;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, p < before + inc);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const long long at = __shfl_sync(0xffffffffu, before + inc - n, l);
            w.b = b0 + l;
            w.s = att_seq(c, a, lgG, w.b);
            w.rr = (int)((p - at) / w.s.nt);
            w.j = (int)((p - at) % w.s.nt);
            return total;
        }
        before = __shfl_sync(0xffffffffu, before + inc, 31);
    }
    return total;
}

// What the workers need of a tile.
struct AttDesc {
    int b, rr, v0;            // v0: its first virtual token
    int nuq;                  // 32-token units of quantized tokens, 0 .. 4
    int nq, Tq, res, nd;
    int first, last;          // first / last tile of a row tile within this CTA's range
    int tail, mid;            // the row tile ends here / an earlier CTA started it
    int qbuf;
    unsigned umask;           // quantized units to attend (the others' entries are skipped)
};

// ---------------------------------------------------------------- rebuild ---

// Sixteen 2-bit codes of word w through the table x[c] = fp16(c s + z), as
// eight half pairs of neighbouring codes.  The byte (2c) | (2c + 1) << 4 is a
// PRMT selector of x[c] in the four-entry table: the word's codes are spread
// to bytes, turned into selectors by one multiply-add per four codes and
// paired by PRMT -- two instructions a code, against four and a half for
// extracting, converting, scaling and rounding each.
__device__ __forceinline__ void codes2_to_half(uint32_t w, float s, float z, uint32_t (&h)[8])
{
    const uint32_t t01 = h2_bits(__floats2half2_rn(__fmaf_rn(0.0f, s, z), __fmaf_rn(1.0f, s, z)));
    const uint32_t t23 = h2_bits(__floats2half2_rn(__fmaf_rn(2.0f, s, z), __fmaf_rn(3.0f, s, z)));
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = ((w >> (2 * i)) & 0x03030303u) * 0x22u + 0x10101010u;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        h[2 * b] = __byte_perm(t01, t23, __byte_perm(q[0], q[1], b | (4 + b) << 4));
        h[2 * b + 1] = __byte_perm(t01, t23, __byte_perm(q[2], q[3], b | (4 + b) << 4));
    }
}
// Code i of a byte quadruple as a float: the byte becomes the mantissa of
// 2^23, which one exact subtraction removes.
__device__ __forceinline__ float byte_float(uint32_t bytes, int i)
{
    return __fsub_rn(__uint_as_float(__byte_perm(bytes, 0x4B000000u, 0x7540 | i)), 8388608.0f);
}
// The codes of word w of width BITS (4 or 8) as floats, in order.
template <int BITS>
__device__ __forceinline__ void codes_float(uint32_t w, float (&f)[32 / BITS])
{
    if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = byte_float(w, i);
    } else {
        const uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = byte_float(e, i);
            f[2 * i + 1] = byte_float(o, i);
        }
    }
}

// Keys of the stage at `st` into the operand at kb: a task is 16 tokens of two
// neighbouring channels (one 4-byte store per token; a warp's 32 tasks cover
// a token's 128-byte row, so the stores are free of bank conflicts).
template <int D, int BITS>
__device__ __forceinline__ void rebuild_keys(const uint8_t* st, uint8_t* kb, int nuq, unsigned umask, int kub)
{
    constexpr int P = 32 / BITS, WR = 16 / P;  // word-rows of 16 tokens
    const float* sc = reinterpret_cast<const float*>(st + 4 * kub);
    const float* zr = sc + 4 * D;
#pragma unroll 1
    for (int task = threadIdx.x; task < 4 * D; task += kAttWorkers) {
        const int cp = task % (D / 2), hu = task / (D / 2), u = hu >> 1;
        if (u >= nuq || !((umask >> u) & 1u))
            continue;  // uniform over the warp
        const float2 s = *reinterpret_cast<const float2*>(sc + u * D + 2 * cp);
        const float2 z = *reinterpret_cast<const float2*>(zr + u * D + 2 * cp);
        const uint2* wp = reinterpret_cast<const uint2*>(st + u * kub) + (size_t)((hu & 1) * WR) * (D / 2) + cp;
        const int c8 = (cp & 31) >> 2;
        uint8_t* dst = kb + (cp >> 5) * kAttAtom + hu * 16 * 128 + (cp & 3) * 4;
        if constexpr (BITS == 2) {
            const uint2 w = wp[0];
            uint32_t h0[8], h1[8];
            codes2_to_half(w.x, s.x, z.x, h0);
            codes2_to_half(w.y, s.y, z.y, h1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                *reinterpret_cast<uint32_t*>(dst + (2 * k) * 128 + ((c8 ^ ((2 * k) & 7)) << 4)) =
                    __byte_perm(h0[k], h1[k], 0x5410);
                *reinterpret_cast<uint32_t*>(dst + (2 * k + 1) * 128 + ((c8 ^ ((2 * k + 1) & 7)) << 4)) =
                    __byte_perm(h0[k], h1[k], 0x7632);
            }
        } else {
#pragma unroll
            for (int r = 0; r < WR; ++r) {
                const uint2 w = wp[(size_t)r * (D / 2)];
                float f0[P], f1[P];
                codes_float<BITS>(w.x, f0);
                codes_float<BITS>(w.y, f1);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int t = r * P + i;
                    *reinterpret_cast<uint32_t*>(dst + t * 128 + ((c8 ^ (t & 7)) << 4)) =
                        dequant_h2(f0[i], f1[i], s.x, z.x, s.y, z.y);
                }
            }
        }
    }
}

// Values: a task is 16 channels of one token, two 16-byte stores.  Lanes of
// odd 64-channel columns store their second chunk first, so that the eight
// lanes of a store phase touch eight different 16-byte columns.
template <int D, int BITS>
__device__ __forceinline__ void rebuild_values(const uint8_t* st, uint8_t* vb, int nuq, unsigned umask, int vub,
                                               int lgG)
{
    constexpr int W = D / 16, WB = 2 * BITS;  // tasks per token, code bytes of a task
    const int lgNG = (D == 64 ? 6 : D == 128 ? 7 : 8) - lgG;
    const float* sc = reinterpret_cast<const float*>(st + 4 * vub);
    const float* zr = sc + (kAttTile << lgNG);
#pragma unroll 2
    for (int task = threadIdx.x; task < kAttTile * W; task += kAttWorkers) {
        const int w = task % W, t = task / W;
        if ((t >> 5) >= nuq)
            continue;
        uint32_t h[8];
        if ((umask >> (t >> 5)) & 1u) {
            const int g = (16 * w) >> lgG;
            const float s = sc[(t << lgNG) + g], z = zr[(t << lgNG) + g];
            const uint8_t* src = st + (size_t)t * (D * BITS / 8) + w * WB;
            if constexpr (BITS == 2) {
                codes2_to_half(*reinterpret_cast<const uint32_t*>(src), s, z, h);
            } else if constexpr (BITS == 4) {
                const uint2 x = *reinterpret_cast<const uint2*>(src);
                float f[8];
                codes_float<4>(x.x, f);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[k] = dequant_h2(f[2 * k], f[2 * k + 1], s, z, s, z);
                codes_float<4>(x.y, f);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[4 + k] = dequant_h2(f[2 * k], f[2 * k + 1], s, z, s, z);
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(src);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[4];
                    codes_float<8>(u4_word(x, i), f);
                    h[2 * i] = dequant_h2(f[0], f[1], s, z, s, z);
                    h[2 * i + 1] = dequant_h2(f[2], f[3], s, z, s, z);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                h[k] = 0u;  // a skipped group: its weights are 0, its values must be finite
        }
        const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
        uint8_t* row = vb + (w >> 2) * kAttAtom + t * 128;
        const int c = 2 * (w & 3), odd = (w >> 2) & 1;
        *reinterpret_cast<uint4*>(row + (((c + odd) ^ (t & 7)) << 4)) = odd ? hi : lo;
        *reinterpret_cast<uint4*>(row + (((c + 1 - odd) ^ (t & 7)) << 4)) = odd ? lo : hi;
    }
}

// ----------------------------------------------------------------- kernel ---

template <int D, int NR>
__global__ void __launch_bounds__(kAttThreads, 1)
attend_kernel(const kivi_cache c, const AttendArgs a, const AttPlan pl, float* __restrict__ ws)
{
    using C = AttCfg<D, NR>;
    constexpr int NC = C::NC, CH = C::CH, MH = C::MH;
    extern __shared__ uint8_t att_smem[];
    __shared__ AttDesc s_desc[kAttDescs];
    __shared__ unsigned long long s_seen[4][4];   // drafts any row attends, by tile and word
    __shared__ __align__(16) float s_red[2][4][NC][4];  // maxima, sums: [row group][row][lane quadrant]
    __shared__ uint64_t s_full[kAttMaxStages], s_empty[kAttMaxStages], s_sbar[2], s_obar;
    __shared__ unsigned s_umask[kAttMaxStages];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_never;
    __shared__ AttWalk s_walk;
    __shared__ long long s_range[3];
    uint8_t* sm = att_smem + ((1024u - (smem_addr(att_smem) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int RB = c.H * pl.RT;
    int* status = reinterpret_cast<int*>(ws);
    const long long ctas = gridDim.x, cta = blockIdx.x;

    if (warp == 0) {
        AttWalk w;
        long long p0 = 0;
        const long long total = att_locate(c, a, pl.lgG, RB, [&](long long t) { return p0 = t * cta / ctas; }, w);
        if (lane == 0) {
            s_range[0] = p0;
            s_range[1] = total * (cta + 1) / ctas;
            s_range[2] = total;
            s_walk = w;
            s_abort = s_never = 0;
            if (cta == 0)
                *status = KIVI_OK;
            for (int i = 0; i < pl.ns; ++i) {
                mbar_init(&s_full[i], 1);
                mbar_init(&s_empty[i], kAttWorkers / 32);
            }
            mbar_init(&s_sbar[0], 1);
            mbar_init(&s_sbar[1], 1);
            mbar_init(&s_obar, 1);
            mbar_fence_init();
        }
    } else if (warp == 1) {
        tc_alloc(&s_tmem, C::TM_COLS);
    }
    if constexpr (D == 64) {  // the second 64 rows of V^T are not channels: zero
        for (int i = tid; i < kAttAtom / 16; i += kAttThreads)
            reinterpret_cast<uint4*>(sm + C::O_V + kAttAtom)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;
    const int n = (int)(s_range[1] - s_range[0]);
    int* cut = reinterpret_cast<int*>(ws + kAttHeaderFloats) + (size_t)cta * kAttCutInts;
    if (tid == 0)
        cut[0] = 0;

    if (warp == kAttWorkers / 32) {
        // ------------------------------------------------------ copies ---
        // in the order the workers consume: K0, K1, V0, K2, V1, ...
        AttWalk w[2] = {s_walk, s_walk};  // next tile whose keys / values are copied
        int at[2] = {0, 0};
        int sp = 0;
        uint8_t* ring = sm + C::O_RING;
        while (at[1] < n) {
            const int which = at[0] < n && at[0] < at[1] + 2 ? 0 : 1;
            AttWalk& x = w[which];
            const int v0 = x.j * kAttTile;
            const int nuq = min(max((x.s.nq - v0) >> 5, 0), 4);
            if (nuq > 0) {
                const int slot = sp % pl.ns, round = sp / pl.ns;
                bool ok = true;
                if (round > 0)
                    ok = mbar_wait_bounded(&s_empty[slot], (round - 1) & 1, &s_abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    if (lane == 0 && atomicExch(&s_abort, 1) == 0)
                        atomicExch(status, KIVI_ETIMEOUT);
                    break;
                }
                const size_t bh = (size_t)x.b * c.H + x.rr / pl.RT;
                const int v = v0 + 32 * lane;  // this lane's unit
                int t0 = v;
                bool go = lane < nuq;
                if (go && a.blocks) {
                    const int g = ldg_checked(a.blocks + bh * a.n_keep + (v >> pl.lgG));
                    go = g >= 0 && g < x.s.Tq >> pl.lgG;
                    t0 = (g << pl.lgG) + (v & (c.G - 1));
                }
                const unsigned mask = __ballot_sync(0xffffffffu, go);
                const uint32_t stat = which == 0 ? D * 4 : 32 * (D >> pl.lgG) * 4;
                const uint32_t code = which == 0 ? pl.kub : pl.vub;
                if (lane == 0) {
                    s_umask[slot] = mask;
                    mbar_arrive_tx(&s_full[slot], __popc(mask) * (code + 2 * stat));
                }
                __syncwarp();
                if (go) {
                    const uint8_t* src;
                    const float *ss, *zz;
                    if (which == 0) {
                        const int P = 32 / c.bits_k;
                        src = reinterpret_cast<const uint8_t*>(c.kq + (bh * (c.Tmax / P) + t0 / P) * D);
                        const size_t so = (bh * (c.Tmax >> pl.lgG) + (t0 >> pl.lgG)) * D;
                        ss = c.kscale + so;
                        zz = c.kzero + so;
                    } else {
                        src = reinterpret_cast<const uint8_t*>(c.vq) + (bh * c.Tmax + t0) * (D * c.bits_v / 8);
                        const size_t so = (bh * c.Tmax + t0) * (D >> pl.lgG);
                        ss = c.vscale + so;
                        zz = c.vzero + so;
                    }
                    uint8_t* d = ring + (size_t)slot * pl.stage;
                    if (KIVI_IN_RANGE(src, code) && KIVI_IN_RANGE(ss, stat) && KIVI_IN_RANGE(zz, stat)) {
                        bulk_g2s(d + lane * code, src, code, &s_full[slot]);
                        bulk_g2s(d + 4 * code + lane * stat, ss, stat, &s_full[slot]);
                        bulk_g2s(d + 4 * code + 4 * stat + lane * stat, zz, stat, &s_full[slot]);
                    }
                }
                ++sp;
            }
            ++at[which];
            att_next(x, c, a, pl.lgG, RB);
        }
        // every copy has landed before the CTA may end (the workers have
        // consumed them all unless a wait gave up)
        for (int s = max(0, sp - pl.ns); s < sp; ++s)
            mbar_wait_bounded(&s_full[s % pl.ns], (s / pl.ns) & 1, &s_never);
    } else if (n > 0) {
        // ----------------------------------------------------- workers ---
        const int qd = warp & 3, wg = warp >> 2;
        const uint32_t lanes = (uint32_t)(qd * 32) << 16;
        const float sl2 = a.sm_scale * 1.4426950408889634f;
        const int RG = c.R + c.G;
        int sc = 0;                        // stages consumed
        float m = -INFINITY, alpha = 1.0f; // of row wg NC + lane, lane < NC
        float l[NC], o[MH][NC];

        auto wait = [&](uint64_t* bar, int phase) {
            if (!mbar_wait_bounded(bar, phase & 1, &s_abort))
                if (atomicExch(&s_abort, 1) == 0)
                    atomicExch(status, KIVI_ETIMEOUT);
        };
        auto barrier = [&]() { named_bar(1, kAttWorkers); };

        // tile descriptors, written by thread 0 two tiles before their first use
        AttWalk dw = s_walk;
        int dn = 0, dq = 0;
        auto describe = [&]() {
            if (dn >= n)
                return;
            AttDesc& d = s_desc[dn & (kAttDescs - 1)];
            const int v0 = dw.j * kAttTile;
            d.b = dw.b;
            d.rr = dw.rr;
            d.v0 = v0;
            d.nuq = min(max((dw.s.nq - v0) >> 5, 0), 4);
            d.nq = dw.s.nq;
            d.Tq = dw.s.Tq;
            d.res = dw.s.len - dw.s.Tq;
            d.nd = dw.s.nd;
            d.tail = dw.j == dw.s.nt - 1;
            d.mid = s_walk.j > 0 && dw.b == s_walk.b && dw.rr == s_walk.rr;
            d.first = dw.j == 0 || dn == 0;
            d.last = d.tail || dn == n - 1;
            if (d.first)
                dq ^= 1;
            d.qbuf = dq;
            if (dn == n - 1 && !d.tail && !d.mid) {
                // the row starts in this range and ends in a later one
                const long long end = s_range[1] + (dw.s.nt - 1 - dw.j);
                int k = (int)cta + 1;
                while (s_range[2] * (k + 1) / ctas < end)
                    ++k;
                cut[1] = dw.b;
                cut[2] = dw.rr;
                cut[3] = k;
                cut[4] = (int)(s_range[2] & 0x7fffffff);
                cut[5] = (int)(s_range[2] >> 31);
                cut[0] = 1;
            }
            ++dn;
            att_next(dw, c, a, pl.lgG, RB);
        };

        // fp16 rows of a tile (residual and drafts) into an operand buffer
        auto copy_rows = [&](const AttDesc& d, int ti, const uint16_t* ringp, const uint16_t* draft, uint8_t* dst) {
            const int e0 = 32 * d.nuq, NCH = D / 8;
            const size_t bh = (size_t)d.b * c.H + d.rr / pl.RT;
            const int s0 = d.Tq % RG;
#pragma unroll 4
            for (int i = tid; i < (kAttTile - e0) * NCH; i += kAttWorkers) {
                const int ch = i % NCH, e = e0 + i / NCH;
                const int f = d.v0 + e - d.nq;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (f < d.res) {
                    const int slot = s0 + f >= RG ? s0 + f - RG : s0 + f;
                    x = ldg_checked(reinterpret_cast<const uint4*>(ringp + (bh * RG + slot) * D) + ch);
                } else {
                    const int j = f - d.res;
                    if (j < d.nd && (s_seen[ti & 3][j >> 6] >> (j & 63)) & 1)
                        x = ldg_checked(reinterpret_cast<const uint4*>(draft + (bh * a.N + j) * D) + ch);
                }
                *reinterpret_cast<uint4*>(dst + (ch >> 3) * kAttAtom + e * 128 + (((ch & 7) ^ (e & 7)) << 4)) = x;
            }
        };

        // K operand (and a new row tile's Q) of tile i
        auto keys = [&](int i) {
            AttDesc& d = s_desc[i & (kAttDescs - 1)];
            const int h = d.rr / pl.RT, rt = d.rr - h * pl.RT;
            const int gq = a.Hq / c.H;
            const bool drafts = d.nd > 0 && d.v0 + kAttTile > d.nq + d.res;
            if (drafts) {  // which drafts any row attends
                if (tid < 4)
                    s_seen[i & 3][tid] = 0ull;
                barrier();
                const int W = (a.N + 63) >> 6;
                for (int x = tid; x < d.nd * W; x += kAttWorkers)
                    atomicOr(&s_seen[i & 3][x % W],
                             (unsigned long long)ldg_checked(a.mask + ((size_t)d.b * a.N + x / W) * W + x % W));
                barrier();
            }
            if (d.first) {
                uint8_t* qb = sm + C::O_Q + d.qbuf * C::QBYTES;
                constexpr int NCH = D / 8;
#pragma unroll 2
                for (int x = tid; x < NR * NCH; x += kAttWorkers) {
                    const int ch = x % NCH, r = x / NCH, row = rt * NR + r;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (row < pl.M && (!a.k || row % a.N < d.nd))
                        v = ldg_checked(reinterpret_cast<const uint4*>(
                                            a.q + (((size_t)d.b * a.Hq + (size_t)h * gq) * a.N + row) * D) + ch);
                    *reinterpret_cast<uint4*>(qb + (ch >> 3) * (NR * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
                }
            }
            if (d.nuq > 0) {
                const int slot = sc % pl.ns;
                wait(&s_full[slot], sc / pl.ns);
                const unsigned um = s_umask[slot];
                if (tid == 0)
                    d.umask = um;
                const uint8_t* st = sm + C::O_RING + (size_t)slot * pl.stage;
                switch (c.bits_k) {
                case 2: rebuild_keys<D, 2>(st, sm + C::O_K, d.nuq, um, pl.kub); break;
                case 4: rebuild_keys<D, 4>(st, sm + C::O_K, d.nuq, um, pl.kub); break;
                default: rebuild_keys<D, 8>(st, sm + C::O_K, d.nuq, um, pl.kub); break;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s_empty[slot]);
                ++sc;
            }
            if (d.nuq < 4)
                copy_rows(d, i, c.kres, a.k, sm + C::O_K);
        };
        auto values = [&](int i) {
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
            if (d.nuq > 0) {
                const int slot = sc % pl.ns;
                wait(&s_full[slot], sc / pl.ns);
                const uint8_t* st = sm + C::O_RING + (size_t)slot * pl.stage;
                switch (c.bits_v) {
                case 2: rebuild_values<D, 2>(st, sm + C::O_V, d.nuq, s_umask[slot], pl.vub, pl.lgG); break;
                case 4: rebuild_values<D, 4>(st, sm + C::O_V, d.nuq, s_umask[slot], pl.vub, pl.lgG); break;
                default: rebuild_values<D, 8>(st, sm + C::O_V, d.nuq, s_umask[slot], pl.vub, pl.lgG); break;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s_empty[slot]);
                ++sc;
            }
            if (d.nuq < 4)
                copy_rows(d, i, c.vres, a.v, sm + C::O_V);
        };
        auto publish = [&]() {  // operands in shared memory, TMEM reads done
            fence_async_smem();
            tc_fence_before();
            barrier();
        };
        auto issue_s = [&](int i) {
            if (tid != 0)
                return;
            tc_fence_after();
            const uint32_t kb = smem_addr(sm + C::O_K);
            const uint32_t qb = smem_addr(sm + C::O_Q + s_desc[i & (kAttDescs - 1)].qbuf * C::QBYTES);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                tc_mma(tm + C::TM_S + (i & 1) * NR, smem_desc(kb + (k >> 2) * kAttAtom + (k & 3) * 32, 16),
                       smem_desc(qb + (k >> 2) * (NR * 128) + (k & 3) * 32, 16), mma_idesc(NR, false), k > 0);
            tc_commit(&s_sbar[i & 1]);
        };
        auto issue_o = [&]() {
            if (tid != 0)
                return;
            tc_fence_after();
            const uint32_t vb = smem_addr(sm + C::O_V), pb = smem_addr(sm + C::O_P);
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
                for (int x = 0; x < C::PASSES * (kAttTile / 16); ++x) {
                    const int pass = x / (kAttTile / 16), k = x % (kAttTile / 16);
                    tc_mma(tm + C::TM_O + h * C::PN, smem_desc(vb + h * 2 * kAttAtom + k * 2048, kAttAtom),
                           smem_desc(pb + pass * (C::PATOMS / 2) * kAttAtom + k * 2048, kAttAtom),
                           mma_idesc(C::PN, true), x > 0);
                }
            tc_commit(&s_obar);
        };

        // P of tile i
        auto softmax = [&](int i) {
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
            const int rt = d.rr % pl.RT;
            if (d.first) {
                m = -INFINITY;
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    l[k] = 0.0f;
            }
            // tokens of this warp's lanes: a quantized unit, or fp16 tokens
            const bool quant = qd < d.nuq;
            const bool off = quant && !((d.umask >> qd) & 1u);
            const int f = d.v0 + 32 * qd + lane - d.nq;          // fp16 token
            const int j = f - d.res;                             // draft
            const uint32_t src = tm + C::TM_S + (i & 1) * NR + wg * NC + lanes;
            float y[CH];
            auto load = [&](int k0) {
                tc_ld(y, src + k0);
                tc_wait_ld(y);
#pragma unroll
                for (int k = 0; k < CH; ++k)
                    y[k] *= sl2;
                if (off || (!quant && f >= d.res)) {
                    const int W = (a.N + 63) >> 6;
                    const bool draft = !off && j < d.nd;
                    int row = (rt * NR + wg * NC + k0) % a.N;
#pragma unroll
                    for (int k = 0; k < CH; ++k) {
                        bool see = false;
                        if (draft && row < d.nd)
                            see = (ldg_checked(a.mask + ((size_t)d.b * a.N + row) * W + (j >> 6)) >> (j & 63)) & 1;
                        if (!see)
                            y[k] = -INFINITY;
                        if (++row == a.N)
                            row = 0;
                    }
                }
                __syncwarp();
            };
            float mine = -INFINITY;
#pragma unroll
            for (int k0 = 0; k0 < NC; k0 += CH) {
                load(k0);
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const float x = redux_max(y[k]);
                    if (lane == k0 + k)
                        mine = x;
                }
            }
            if (lane < NC)
                s_red[0][wg][lane][qd] = mine;
            named_bar(2 + wg, 128);
            const float4 r = *reinterpret_cast<const float4*>(s_red[0][wg][lane < NC ? lane : 0]);
            const float mn = fmaxf(fmaxf(m, fmaxf(r.x, r.y)), fmaxf(r.z, r.w));
            const float ref = mn == -INFINITY ? 0.0f : mn;
            alpha = m == mn ? 1.0f : ex2(m - ref);
            m = mn;
            const float sub = ref - kAttShift;
            const bool grew = __any_sync(0xffffffffu, alpha != 1.0f && lane < NC);
            uint8_t* prow = sm + C::O_P + (32 * qd + lane) * 128;
            const int sw = lane & 7;  // token % 8
#pragma unroll
            for (int k0 = 0; k0 < NC; k0 += CH) {
                if (NC > CH)
                    load(k0);
                uint32_t hi[CH / 2], lo[CH / 2];
#pragma unroll
                for (int k = 0; k < CH; k += 2) {
                    const float p0 = ex2(y[k] - __shfl_sync(0xffffffffu, sub, k0 + k));
                    const float p1 = ex2(y[k + 1] - __shfl_sync(0xffffffffu, sub, k0 + k + 1));
                    if (grew) {
                        l[k0 + k] *= __shfl_sync(0xffffffffu, alpha, k0 + k);
                        l[k0 + k + 1] *= __shfl_sync(0xffffffffu, alpha, k0 + k + 1);
                    }
                    l[k0 + k] += p0;
                    l[k0 + k + 1] += p1;
                    split_hi_lo(p0, p1, hi[k / 2], lo[k / 2]);
                }
#pragma unroll
                for (int k = 0; k < CH; k += 8) {
                    const int r0 = wg * NC + k0 + k;  // first of eight rows: one 16-byte chunk of each term
                    uint8_t* h0 = prow + (r0 >> 6) * kAttAtom;
                    const uint4 vh = make_uint4(hi[k / 2], hi[k / 2 + 1], hi[k / 2 + 2], hi[k / 2 + 3]);
                    const uint4 vl = make_uint4(lo[k / 2], lo[k / 2 + 1], lo[k / 2 + 2], lo[k / 2 + 3]);
                    *reinterpret_cast<uint4*>(h0 + ((((r0 >> 3) & 7) ^ sw) << 4)) = vh;
                    if constexpr (C::STACK)
                        *reinterpret_cast<uint4*>(h0 + (((4 + (r0 >> 3)) ^ sw) << 4)) = vl;
                    else
                        *reinterpret_cast<uint4*>(h0 + (C::PATOMS / 2) * kAttAtom + ((((r0 >> 3) & 7) ^ sw) << 4)) = vl;
                }
            }
        };

        // O of tile i joins the running output; the row tile's last one writes it
        auto output = [&](int i) {
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
            const bool grew = __any_sync(0xffffffffu, alpha != 1.0f && lane < NC);
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
                for (int k0 = 0; k0 < NC; k0 += CH) {
                    float t[CH];
                    const uint32_t src = tm + C::TM_O + h * C::PN + wg * NC + k0 + lanes;
                    tc_ld(t, src);
                    if constexpr (C::STACK) {
                        float t2[CH];
                        tc_ld(t2, src + 32);
                        tc_wait_ld(t);
                        tc_wait_ld(t2);
#pragma unroll
                        for (int k = 0; k < CH; ++k)
                            t[k] += t2[k];
                    } else {
                        tc_wait_ld(t);
                    }
                    if (d.first) {
#pragma unroll
                        for (int k = 0; k < CH; ++k)
                            o[h][k0 + k] = t[k];
                    } else if (grew) {
#pragma unroll
                        for (int k = 0; k < CH; ++k)
                            o[h][k0 + k] = fmaf(o[h][k0 + k], __shfl_sync(0xffffffffu, alpha, k0 + k), t[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < CH; ++k)
                            o[h][k0 + k] += t[k];
                    }
                }
            if (!d.last)
                return;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float x = l[k];
#pragma unroll
                for (int s = 16; s > 0; s >>= 1)
                    x += __shfl_xor_sync(0xffffffffu, x, s);
                if (lane == k)
                    sum = x;
            }
            if (lane < NC)
                s_red[1][wg][lane][qd] = sum;
            named_bar(2 + wg, 128);
            const float4 r = *reinterpret_cast<const float4*>(s_red[1][wg][lane < NC ? lane : 0]);
            const float L = (r.x + r.y) + (r.z + r.w);
            const int h = d.rr / pl.RT, r0 = (d.rr - h * pl.RT) * NR + wg * NC;
            const int ch = 32 * qd + lane;
            const bool owns = D >= 128 || qd < 2;  // D = 64: the upper lanes hold no channels
            if (d.tail && !d.mid) {
                const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                float* dst = a.out + (((size_t)d.b * a.Hq + (size_t)h * (a.Hq / c.H)) * a.N + r0) * D + ch;
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float f = __shfl_sync(0xffffffffu, inv, k);
                    if (owns && r0 + k < pl.M && (!a.k || (r0 + k) % a.N < d.nd))
#pragma unroll
                        for (int x = 0; x < MH; ++x)
                            st_checked(dst + (size_t)k * D + 128 * x, o[x][k] * f);
                }
            } else {
                // a piece: slot 0 for a row tile that an earlier CTA starts, else 1
                float* part = att_part(ws, D, NR, (int)cta, d.mid ? 0 : 1);
                if (owns) {
#pragma unroll
                    for (int k = 0; k < NC; ++k)
#pragma unroll
                        for (int x = 0; x < MH; ++x)
                            part[(size_t)(wg * NC + k) * D + ch + 128 * x] = o[x][k];
                }
                if (qd == 0 && lane < NC) {
                    part[(size_t)NR * D + wg * NC + lane] = m;
                    part[(size_t)NR * D + NR + wg * NC + lane] = L;
                }
            }
        };

        if (tid == 0)
            for (int i = 0; i < 4; ++i)
                describe();
        barrier();
        keys(0);
        publish();
        issue_s(0);
        if (n > 1) {
            wait(&s_sbar[0], 0);
            keys(1);
            publish();
            issue_s(1);
        }
        values(0);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (tid == 0)
                describe();  // tile i + 4
            wait(&s_sbar[i & 1], i >> 1);
            tc_fence_after();
            softmax(i);
            publish();
            issue_o();
            if (i + 2 < n) {
                wait(&s_sbar[(i + 1) & 1], (i + 1) >> 1);
                keys(i + 2);
                publish();
                issue_s(i + 2);
            }
            wait(&s_obar, i);
            tc_fence_after();
            output(i);
            if (i + 1 < n)
                values(i + 1);
        }
        if (*(volatile int*)&s_abort) {  // products in flight end before their TMEM is freed
            mbar_wait_bounded(&s_sbar[(n - 1) & 1], ((n - 1) >> 1) & 1, &s_never);
            mbar_wait_bounded(&s_obar, (n - 1) & 1, &s_never);
        }
        tc_fence_before();
    }
    asm volatile("griddepcontrol.launch_dependents;");
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tc_dealloc(tm, C::TM_COLS);
    }
}

// ---------------------------------------------------------------- combine ---

// Merges the pieces of the row tiles that CTA ranges cut: block (i, y) takes
// eight rows of the row tile that starts in range i and ends in a later one,
// piece by piece in order (empty ranges hold none).
constexpr int kAttCombineThreads = 256;
constexpr int kAttCombineRows = 8;
static __global__ void __launch_bounds__(kAttCombineThreads)
attend_combine_kernel(const kivi_cache c, const AttendArgs a, const AttPlan pl, int NR, float* __restrict__ ws)
{
    const int D = c.D, i = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int* cut = reinterpret_cast<const int*>(ws + kAttHeaderFloats) + (size_t)i * kAttCutInts;
    if (cut[0] == 0)
        return;
    const int b = cut[1], rr = cut[2], last = cut[3];
    const long long total = (long long)cut[4] | (long long)cut[5] << 31, N = gridDim.x;
    const int h = rr / pl.RT, rt = rr - h * pl.RT;
    const int nd = a.k ? (a.n_draft ? min(max(ldg_checked(a.n_draft + b), 0), a.N) : a.N) : 1;
    for (int e = threadIdx.x; e < kAttCombineRows * D; e += kAttCombineThreads) {
        const int r = blockIdx.y * kAttCombineRows + e / D, d = e % D, row = rt * NR + r;
        if (row >= pl.M || row % a.N >= nd)
            continue;
        float M = -INFINITY, L = 0.0f, o = 0.0f;
        for (int k = i; k <= last; ++k) {
            if (total * k / N == total * (k + 1) / N)
                continue;
            const float* p = att_part(ws, D, NR, k, k == i);
            const float m = p[(size_t)NR * D + r], l = p[(size_t)NR * D + NR + r], x = p[(size_t)r * D + d];
            if (m == -INFINITY)
                continue;
            const float Mn = fmaxf(M, m), f = ex2(M - Mn), g = ex2(m - Mn);
            L = L * f + l * g;
            o = o * f + x * g;
            M = Mn;
        }
        st_checked(a.out + (((size_t)b * a.Hq + (size_t)h * (a.Hq / c.H)) * a.N + row) * D + d, L > 0.0f ? o / L : 0.0f);
    }
}

// ----------------------------------------------------------------- launch ---

template <int D, int NR>
cudaError_t attend_launch_rows(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s)
{
    using C = AttCfg<D, NR>;
    auto kern = attend_kernel<D, NR>;
    AttPlan pl;
    pl.lgG = c.G == 32 ? 5 : c.G == 64 ? 6 : 7;
    pl.M = a.Hq / c.H * a.N;
    pl.RT = (pl.M + NR - 1) / NR;
    pl.kub = 4 * D * c.bits_k;
    pl.vub = 4 * D * c.bits_v;
    pl.stage = cmax(4 * pl.kub + 32 * D, 4 * pl.vub + 1024 * (D / c.G));
    pl.ns = cmin(C::RING / pl.stage, kAttMaxStages);
    const int smem = 1024 + C::O_RING + pl.ns * pl.stage;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    const int N = cmin(sm_count(), kAttMaxCTAs);
    kern<<<N, kAttThreads, smem, s>>>(c, a, pl, ws);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    // the combine's CTAs are scheduled while the attention drains
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(N, (cmin(pl.M, NR) + kAttCombineRows - 1) / kAttCombineRows);
    cfg.blockDim = dim3(kAttCombineThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_combine_kernel, c, a, pl, NR, ws);
}

template <int D>
cudaError_t launch_attend_d(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s)
{
    KIVI_SET_CHECK_RANGES(c, s, {{a.q, (size_t)c.B * a.Hq * a.N * D * 2}, {a.out, (size_t)c.B * a.Hq * a.N * D * 4},
                                 {a.k, (size_t)c.B * c.H * a.N * D * 2}, {a.v, (size_t)c.B * c.H * a.N * D * 2},
                                 {a.mask, (size_t)c.B * a.N * ((a.N + 63) / 64) * 8}, {a.n_draft, (size_t)c.B * 4},
                                 {a.blocks, (size_t)c.B * c.H * a.n_keep * 4}});
    switch (attend_rows(D, a.Hq / c.H * a.N)) {
    case 32: return attend_launch_rows<D, 32>(c, a, ws, s);
    case 64:
        if constexpr (D != 256)
            return attend_launch_rows<D, 64>(c, a, ws, s);
        break;
    default:
        if constexpr (D != 256)
            return attend_launch_rows<D, 128>(c, a, ws, s);
        break;
    }
    return cudaErrorInvalidValue;
}

#define KIVI_ATTEND_INSTANTIATE(DIM) \
    template cudaError_t launch_attend_d<DIM>(const kivi_cache&, const AttendArgs&, float*, cudaStream_t);

}  // namespace kivi
