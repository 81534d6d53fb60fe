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
// axis, so that a row costs one column and a tile has as many as there are (32,
// 64 or 128; attend_warp.cuh serves fewer than 17).  What a tile costs whatever
// the rows is rebuilding 2 x 128 x D fp16 operands from codes.
//
// Work.  A CTA (one or two per SM) takes a contiguous range of the tiles of all
// row tiles in order; a row tile cut by a range boundary leaves partial (o, m, l)
// in the workspace, merged by attend_combine_kernel.  The split and every
// sum's order depend only on sizes and lengths.
//
// Roles.  Eight or sixteen worker warps share every step of a tile; two copy warps bring
// the packed codes and statistics of keys and values into rings of stages, and
// one warp issues the products.  Per tile i the workers
//     turn S(i) into P(i);        barrier, O(i) = V P is issued;
//     rebuild the keys of i + 2;  barrier, S(i + 2) = K Q is issued;
//     add O(i) to the running output and, at a row's end, store it;
//     rebuild the values of i + 1;
// so both products run under the workers' arithmetic.  All workers run the same
// code at the same time on purpose: with a warpgroup per step (475 us for 8
// rows of an int4 prefix, against 263) each group fetched its own instruction
// stream once per tile, and instruction fetch, not the arithmetic, set the pace.
// The widths are template arguments and the cold paths are functions for the
// same reason.  Worker warp w reads TMEM lanes 32 (w % 4) .. + 31
// (tokens, later channels) and the NC rows w / 4 of the tile.
//
// The softmax keeps one reference maximum per row and does not move it while
// the weights stay below 2^15.9: the exact maximum of a tile (warp reductions
// and an exchange between the four warps of a row) is only formed when some
// weight would pass that, which the row's first tile does and few later ones.
//
// Order inside 16.  A K or V operand is stored with its contiguous axis cut
// into runs of 16 -- tokens of a key channel, channels of a value token -- and
// element x of a run sits at position 4 (x % 4) + x / 4: the order in which
// byte-wise extraction delivers the codes of a word, so no instruction
// transposes them.  Tokens of a run take the same positions in V, and the
// channel positions are undone when the output is stored.
//
// Every wait on an mbarrier gives up after some two seconds: it sets the abort
// flag and records KIVI_ETIMEOUT in the workspace's status word; the CTA then
// runs through without waiting, waits (bounded) for its copies and products,
// frees its TMEM and ends.
//
// Measured: 128 query rows over four int2 contexts of 32768 tokens and eight KV
// heads, D = 128: 300 us, 222 TFLOP/s of the two products (66.6 GFLOP) and 139
// MB read once.  The chain of steps between barriers bounds it: the
// schedulers issue in 56 % of the cycles, 35 instructions per weight, of which
// six rebuild the operands; the tensor cores are busy 17 % of the time and DRAM
// 7 %.
#pragma once

#include "attend_plan.h"
#include "decode_stream.cuh"

namespace kivi {

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
// Issued by the one lane with issue != 0; the whole warp runs through, so that
// the descriptors are computed once for the warp (uniform registers).
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t issue)
{
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %4, 0; setp.ne.u32 q, %5, 0;"
        "  @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t issue)
{
    asm volatile(
        "{ .reg .pred q; setp.ne.u32 q, %1, 0;"
        "  @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(smem_addr(bar)),
        "r"(issue)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r;
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
// Instruction descriptor: fp16 operands, fp32 sums, M = 128; mn_a, mn_b: the
// M / N axis of that operand is contiguous in shared memory.
__host__ __device__ constexpr uint32_t mma_idesc(int n, bool mn_a, bool mn_b)
{
    return (1u << 4) | (mn_a ? 1u << 15 : 0u) | (mn_b ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((128u >> 4) << 24);
}
// Whether any of the warpgroup's 128 threads says so (a barrier as well).
__device__ __forceinline__ bool group_any(int id, bool x)
{
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 q, %2, 0; bar.red.or.pred p, %1, 128, q; selp.u32 %0, 1, 0, p; }"
                 : "=r"(r)
                 : "r"(id), "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}
// A row's reference before its first token: below every logit, and finite, so
// that a logit of -inf less it is -inf.
constexpr float kAttNoRef = -3e38f;

// 2^x, 0 below 2^-126 (a weight that small is nothing beside the largest, which
// is 1 or more).
__device__ __forceinline__ float ex2_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two rounded operations in one instruction: x += y, x -= y, x *= f.
__device__ __forceinline__ void put_pair(float* x, float2 r)
{
    x[0] = r.x;
    x[1] = r.y;
}
__device__ __forceinline__ void add_pair(float* x, const float* y)
{
    put_pair(x, __fadd2_rn(make_float2(x[0], x[1]), make_float2(y[0], y[1])));
}
__device__ __forceinline__ void sub_pair(float* x, const float* y)
{
    put_pair(x, __ffma2_rn(make_float2(y[0], y[1]), make_float2(-1.0f, -1.0f), make_float2(x[0], x[1])));
}
__device__ __forceinline__ void mul_pair(float* x, float f)
{
    put_pair(x, __fmul2_rn(make_float2(x[0], x[1]), make_float2(f, f)));
}
// What a row's output is multiplied by, given the sum of its weights: 0 if it
// attends nothing.  A NaN sum (a NaN logit, or an infinite one) stays NaN.
__device__ __forceinline__ float row_scale(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
// p = hi + lo as two fp16 pairs: the upper 11 bits, and what is left of them.
__device__ __forceinline__ void split_pair(float* p, uint32_t& hi, uint32_t& lo)
{
    const float h[2] = {__uint_as_float(__float_as_uint(p[0]) & 0xFFFFE000u),
                        __uint_as_float(__float_as_uint(p[1]) & 0xFFFFE000u)};
    hi = h2_bits(__floats2half2_rn(h[0], h[1]));
    sub_pair(p, h);
    lo = h2_bits(__floats2half2_rn(p[0], p[1]));
}
// A value that is not finite must not reach the product: its weight of 0 in a
// row that does not attend its token would still make the row NaN.  The fp16
// values of drafted tokens are cleared of such halves here (true if there were
// any) and added to the stored rows that attend them, once and after the
// division by the row's sum: a row in one piece by its worker, a cut one by the
// merge.  A piece says that it cleared some by the sign of its rows' sums (its
// own weight may be 0, which would make NaN of them).
__device__ __forceinline__ bool clear_nonfinite(uint32_t (&q)[8])
{
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        any |= (q[k] & 0x7C007C00u) + 0x04000400u;  // bits 15, 31: an exponent of all ones
    if (!(any & 0x80008000u))
        return false;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        q[k] &= ~(((((q[k] & 0x7C007C00u) + 0x04000400u) & 0x80008000u) >> 15) * 0xFFFFu);
    return true;
}
// An fp16 value if it is not finite, else 0.
__device__ __forceinline__ float nonfinite(const uint16_t* p)
{
    const float x = __half2float(__ushort_as_half(ldg_checked(p)));
    return isfinite(x) ? 0.0f : x;
}
// Waits for the phase of parity `parity` of mbarrier b; false, with the abort
// flag set and the timeout recorded in *status (unless null), if it has not
// completed within kAttWaitTries attempts (some four microseconds each) or *abort
// was set.  An iteration count and not the clock, to keep it to a few
// instructions: every role of the kernel runs through its code once per tile,
// so what bounds the kernel first is how much of that code the instruction
// cache holds (inlined waits with a timer and everything unrolled to 150 KB
// ran at a third of this speed, 44% of the instruction fetches missing).
constexpr uint32_t kAttWaitTries = 1u << 19;
__device__ __forceinline__ bool att_wait(uint64_t* b, uint32_t parity, int* abort, int* status)
{
    const uint32_t bar = smem_addr(b);
#pragma unroll 1
    for (uint32_t it = 0; it < kAttWaitTries; ++it) {
        uint32_t done;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000; selp.u32 %0, 1, 0, p; }"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done)
            return true;
        if ((it & 63u) == 63u && *(volatile int*)abort)
            return false;
    }
    if (status && atomicExch(abort, 1) == 0)
        atomicExch(status, KIVI_ETIMEOUT);
    return false;
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
    s.Tq = max(s.len - c.R, 0) >> lgG << lgG;
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
#pragma unroll 1
    while (++w.b < c.B) {
        w.s = att_seq(c, a, lgG, w.b);
        if (w.s.nt > 0)
            return;
    }
    w.b = c.B - 1;  // only if a length was changed meanwhile: stay inside the arrays
}

// One warp: the CTA's range of tiles [range[0], range[1]) of range[2], one of
// range[3] = min(CTAs, total) ranges (none for a CTA beyond them), and the
// position of its first tile.
static __device__ __noinline__ void att_locate(const kivi_cache* c, const AttendArgs* a, const AttPlan* pl,
                                               long long* range, AttWalk* first)
{
    const int lane = threadIdx.x & 31;
    const long long RB = (long long)c->H * pl->RT;
    long long total = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < c->B; b0 += 32) {
        long long n = b0 + lane < c->B ? att_seq(*c, *a, pl->lgG, b0 + lane).nt * RB : 0;
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1)
            n += __shfl_xor_sync(0xffffffffu, n, o);
        total += n;
    }
    const long long index = blockIdx.x, count = min((long long)gridDim.x, total);
    const long long p = index < count ? total * index / count : total;
    if (lane == 0) {
        range[0] = p;
        range[1] = index < count ? total * (index + 1) / count : total;
        range[2] = total;
        range[3] = count;
    }
    if (p == total)
        return;
    long long before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < c->B; b0 += 32) {
        const long long n = b0 + lane < c->B ? att_seq(*c, *a, pl->lgG, b0 + lane).nt * RB : 0;
        long long inc = n;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            inc += lane >= o ? t : 0;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, p < before + inc);
        if (hit) {
            const int l = __ffs(hit) - 1;
            if (lane == l) {
                AttWalk w;
                w.b = b0 + l;
                w.s = att_seq(*c, *a, pl->lgG, w.b);
                const long long at = p - (before + inc - n);
                w.rr = (int)(at / w.s.nt);
                w.j = (int)(at % w.s.nt);
                *first = w;
            }
            return;
        }
        before = __shfl_sync(0xffffffffu, before + inc, 31);
    }
    // p < total, so only if a length was changed meanwhile
    if (lane == 0)
        range[1] = p;
}

// What the workers need of a tile, written by the copy warp.  Aligned, so
// that its fields may be read several at a time (128 rows: 300 against 302 us).
struct alignas(16) AttDesc {
    int b, rr;
    int nuq;                  // 32-token units of quantized tokens, 0 .. 4
    int f0;                   // fp16 token (residual, then drafts) at position 0 of the tile; negative before them
    int Tq, res, nd;
    int first, last;          // first / last tile of a row tile within this CTA's range
    int tail, mid;            // the row tile ends here / an earlier CTA started it
    unsigned umask;           // quantized units to attend (the others' entries are skipped)
};


// ---------------------------------------------------------------- rebuild ---

// Position of element x of a run of 16 (its own inverse).
__device__ __forceinline__ int run16(int x) { return (x & ~15) | (x & 3) << 2 | (x >> 2 & 3); }

// Sixteen codes (BITS / 2 words) as fp16_rne(fmaf(code, s, z)), in run order:
// h[2i] = elements i, 4 + i; h[2i + 1] = elements 8 + i, 12 + i.
//
// Two-bit codes go through the table x[c]: the byte (2c) | (2c + 1) << 4 is a
// PRMT selector of x[c] among the table's four halves, so the word's codes
// are masked to bytes, turned into selectors by one multiply-add per four
// codes, and one PRMT per pair looks both values up: 28 instructions for 16
// codes, against 72 that extract, convert, scale and round each.  Wider codes:
// a byte placed in the mantissa of 2^23 by PRMT is its float plus 2^23, which
// one exact subtraction removes.
template <int BITS>
__device__ __forceinline__ void hat16(const uint32_t (&w)[BITS / 2], float s, float z, uint32_t (&h)[8])
{
    if constexpr (BITS == 2) {
        const uint32_t t01 = h2_bits(__floats2half2_rn(__fmaf_rn(0.0f, s, z), __fmaf_rn(1.0f, s, z)));
        const uint32_t t23 = h2_bits(__floats2half2_rn(__fmaf_rn(2.0f, s, z), __fmaf_rn(3.0f, s, z)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t q = ((w[0] >> (2 * i)) & 0x03030303u) * 0x22u + 0x10101010u;
            h[2 * i] = __byte_perm(t01, t23, q);
            h[2 * i + 1] = __byte_perm(t01, t23, q >> 16);
        }
    } else {
        float f[16];
        auto bytes = [&](uint32_t x, int first, int step) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                f[first + step * b] =
                    __fsub_rn(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7540 | b)), 8388608.0f);
        };
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) {
            if constexpr (BITS == 8) {
                bytes(w[j], 4 * j, 1);
            } else {
                bytes(w[j] & 0x0F0F0F0Fu, 8 * j, 2);
                bytes((w[j] >> 4) & 0x0F0F0F0Fu, 8 * j + 1, 2);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[2 * i] = dequant_h2(f[i], f[4 + i], s, z, s, z);
            h[2 * i + 1] = dequant_h2(f[8 + i], f[12 + i], s, z, s, z);
        }
    }
}

// Words of a run of 16 codes at p, word r at p + r step.
template <int BITS>
__device__ __forceinline__ void run_words(const uint8_t* p, int step, uint32_t (&w)[BITS / 2])
{
#pragma unroll
    for (int r = 0; r < BITS / 2; ++r)
        w[r] = *reinterpret_cast<const uint32_t*>(p + r * step);
}

// Keys of a stage (its first nuq units): a task is 32 tokens of a channel, 64
// contiguous bytes of the K operand, whose token axis is contiguous (rows of
// 64 tokens per channel).  Eight neighbouring channels' stores fall in eight
// different 16-byte columns of the swizzle.
template <int D, int WORKERS, int BITS>
__device__ __forceinline__ void rebuild_keys(const uint8_t* st, uint8_t* kb, int t, int su, int nuq, unsigned umask,
                                             int kub)
{
    const float* sc = reinterpret_cast<const float*>(st + su * kub);
    const float* zr = sc + su * D;
#pragma unroll 1
    for (int task = t; task < D * nuq; task += WORKERS) {
        const int ch = task % D, u = task / D;
        if (!((umask >> u) & 1u))
            continue;  // uniform over the warp
        const float s = sc[task], z = zr[task];
        const uint8_t* wp = st + u * kub + ch * 4;
        uint8_t* row = kb + ((u >> 1) * D + ch) * 128;
        const int c0 = (u & 1) * 64, x = (ch & 7) << 4;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[BITS / 2], h[8];
            run_words<BITS>(wp + hf * (BITS / 2) * D * 4, D * 4, w);
            hat16<BITS>(w, s, z, h);
            *reinterpret_cast<uint4*>(row + ((c0 + 32 * hf) ^ x)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(row + ((c0 + 32 * hf + 16) ^ x)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
}

// Values of a stage (its first nuq units): KVW neighbouring threads rebuild the
// token at one position, 32 channels (a statistic group, or part of one) at a
// time, into the V operand, whose channel axis is contiguous (rows of 64
// channels per token).
template <int D, int WORKERS, int BITS>
__device__ __forceinline__ void rebuild_values(const uint8_t* st, uint8_t* vb, int x, int su, int nuq, unsigned umask,
                                               int vub, int lgG)
{
    const int lgT = (WORKERS == 512 ? 2 : 1) + (su == 2 ? 1 : 0);  // threads per token
    const int t = x >> lgT;
    if ((t >> 5) >= nuq)
        return;
    const int tok = run16(t), lgNG = (D == 64 ? 6 : D == 128 ? 7 : 8) - lgG;
    const bool live = (umask >> (t >> 5)) & 1u;
    const float* sc = reinterpret_cast<const float*>(st + su * vub) + (tok << lgNG);
    const float* zr = sc + (32 * su << lgNG);
    const uint8_t* src = st + tok * (D * BITS / 8);
    uint8_t* row = vb + t * 128;
    const int sw = (t & 7) << 4;
#pragma unroll 1
    for (int c = 32 * (x & ((1 << lgT) - 1)); c < D; c += 32 << lgT) {
        const float s = sc[c >> lgG], z = zr[c >> lgG];
        uint8_t* dst = row + (c >> 6) * (kAttTile * 128);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[BITS / 2], h[8];
            run_words<BITS>(src + (c + 16 * hf) * BITS / 8, 4, w);
            hat16<BITS>(w, s, z, h);
            if (!live) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    h[k] = 0u;  // a skipped group: its weights are 0, its values must be finite
            }
            const int c0 = (c & 32) * 2 + 32 * hf;
            *reinterpret_cast<uint4*>(dst + (c0 ^ sw)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + ((c0 + 16) ^ sw)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
}

// ----------------------------------------------------------------- kernel ---

// ------------------------------------------------------------- cold paths ---
// Out of line, so that a worker's loop over whole quantized tiles stays small
// and contiguous: instruction fetch is what bounds it first.

// Q of a new row tile, rows beyond the problem's zero.
template <int D, int NR, int WORKERS>
static __device__ __noinline__ void att_load_q(const kivi_cache* c, const AttendArgs* a, const AttPlan* pl,
                                               const AttDesc* d, uint8_t* qs, int t)
{
    const int h = d->rr / pl->RT, rt = d->rr - h * pl->RT;
    const uint4* q =
        reinterpret_cast<const uint4*>(a->q + ((size_t)d->b * a->Hq + (size_t)h * (a->Hq / c->H)) * a->N * D);
#pragma unroll 1
    for (int x = t; x < NR * D / 8; x += WORKERS) {
        const int ch = x % (D / 8), r = x / (D / 8), row = rt * NR + r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < pl->M && (!a->k || row % a->N < d->nd))
            v = ldg_checked(q + (size_t)row * (D / 8) + ch);
        *reinterpret_cast<uint4*>(qs + (ch >> 3) * (NR * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
    }
}

// Which drafts any row attends, into seen[4]; every worker calls it.
template <int WORKERS>
static __device__ __noinline__ void att_seen(const AttendArgs* a, const AttDesc* d, unsigned long long* seen, int t)
{
    const int W = (a->N + 63) >> 6;
    if (t < 4)
        seen[t] = 0ull;
    named_bar(2, WORKERS);
#pragma unroll 1
    for (int x = t; x < d->nd * W; x += WORKERS)
        atomicOr(&seen[x % W],
                 (unsigned long long)ldg_checked(a->mask + ((size_t)d->b * a->N + x / W) * W + x % W));
    named_bar(2, WORKERS);
}

// The fp16 tokens (residual, then drafts) of a tile into the K (which = 0) or V
// operand; zero where no row attends one.  A thread takes D / GROUPS channels
// of a token: an element of each channel's row of K, run order in V.
template <int D, int GROUPS>
static __device__ __noinline__ void att_fp16_rows(const kivi_cache* c, const AttendArgs* a, const AttPlan* pl,
                                                  const AttDesc* d, const unsigned long long* seen, int* dirty,
                                                  uint8_t* dst, int which, int t)
{
    const int e = which == 0 ? t & 127 : t / GROUPS, part = which == 0 ? t >> 7 : t % GROUPS;
    if (e < 32 * d->nuq)
        return;
    const int f = d->f0 + e, j = f - d->res, RG = c->R + c->G;
    const size_t bh = (size_t)d->b * c->H + d->rr / pl->RT;
    const uint16_t* src = nullptr;
    if (j < 0) {
        int s = d->Tq % RG + f;
        s = s >= RG ? s - RG : s;
        src = (which == 0 ? c->kres : c->vres) + (bh * RG + s) * D;
    } else if (j < d->nd && (seen[j >> 6] >> (j & 63)) & 1) {
        src = (which == 0 ? a->k : a->v) + (bh * a->N + j) * D;
    }
    uint8_t* kd = dst + (e >> 6) * D * 128 + (e & 7) * 2;
    uint8_t* vd = dst + e * 128;
    const int kx = ((e >> 3) & 7) << 4, vx = (e & 7) << 4;
#pragma unroll 1
    for (int c0 = part * (D / GROUPS); c0 < (part + 1) * (D / GROUPS); c0 += 16) {
        uint4 y = make_uint4(0u, 0u, 0u, 0u), z = y;
        if (src) {
            y = ldg_checked(reinterpret_cast<const uint4*>(src + c0));
            z = ldg_checked(reinterpret_cast<const uint4*>(src + c0) + 1);
        }
        if (which == 0) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                *reinterpret_cast<uint16_t*>(kd + (c0 + k) * 128 + (kx ^ ((k & 7) << 4))) = u4_half(k < 8 ? y : z, k & 7);
        } else {
            uint32_t q[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
            if (j >= 0 && clear_nonfinite(q))
                *dirty = 1;
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int sel = k & 1 ? 0x7632 : 0x5410;
                o[2 * k] = __byte_perm(q[k >> 1], q[2 + (k >> 1)], sel);
                o[2 * k + 1] = __byte_perm(q[4 + (k >> 1)], q[6 + (k >> 1)], sel);
            }
            uint8_t* run = vd + (c0 >> 6) * (kAttTile * 128);
            const int cc = (c0 & 63) * 2;
            *reinterpret_cast<uint4*>(run + (cc ^ vx)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(run + ((cc + 16) ^ vx)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// Adds to a thread's stored channels ch, ch + 128 of the rows r0 + k (bit k of
// `rows`) the values that are not finite of the drafts which those rows attend.
template <int D, int MH>
static __device__ __noinline__ void att_add_nonfinite(const AttendArgs* a, const AttDesc* d, const uint16_t* v, int r0,
                                                      uint32_t rows, int ch, float* dst)
{
    const int W = (a->N + 63) >> 6;
    if (ch >= D)
        return;
#pragma unroll 1
    for (int x = 0; x < d->nd * MH; ++x) {
        const int j = x / MH, half = 128 * (x % MH);
        const float y = nonfinite(v + (size_t)j * D + ch + half);
        if (y == 0.0f)
            continue;
#pragma unroll 1
        for (uint32_t left = rows; left; left &= left - 1) {
            const int k = __ffs(left) - 1, i = (r0 + k) % a->N;
            if (i < d->nd && (ldg_checked(a->mask + ((size_t)d->b * a->N + i) * W + (j >> 6)) >> (j & 63)) & 1)
                st_checked(dst + k * D + half, ld_checked(dst + k * D + half) + y);
        }
    }
}

// B: the codes' width if keys and values have the same (it then is a constant
// of the kernel, and its loops hold no other width's code), else 0.
template <int D, int NR, int B>
__global__ void __launch_bounds__(AttCfg<D, NR>::THREADS, AttCfg<D, NR>::CTAS)
attend_kernel(const __grid_constant__ kivi_cache c, const __grid_constant__ AttendArgs a,
              const __grid_constant__ AttPlan pl, float* __restrict__ ws)
{
    using C = AttCfg<D, NR>;
    constexpr int NC = C::NC, CH = C::CH, MH = C::MH;
    constexpr int kCopyWarp = C::WORKERS / 32, kMmaWarp = kCopyWarp + 2;
    extern __shared__ uint8_t att_smem[];
    __shared__ AttDesc s_desc[kAttDescs];
    __shared__ unsigned long long s_seen[4][4];                // drafts any row attends, by tile
    __shared__ int s_dirty;                                    // values of some draft were cleared (of any row tile so far)
    __shared__ __align__(16) float s_red[C::GROUPS][NC][4];            // maxima: [row group][row][lane quadrant]
    __shared__ float s_part[C::GROUPS][128];
    __shared__ __align__(16) float s_ref[C::GROUPS][C::REG_REF ? 1 : NC];
    __shared__ uint64_t s_full[2][kAttMaxStages], s_empty[2][kAttMaxStages];
    __shared__ uint64_t s_sdone[2], s_odone;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_never;
    __shared__ AttWalk s_walk;
    __shared__ long long s_range[4];
    uint8_t* sm = att_smem + ((1024u - (smem_addr(att_smem) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int RB = c.H * pl.RT;
    int* status = reinterpret_cast<int*>(ws);
    const long long cta = blockIdx.x;

    if (warp == kCopyWarp) {
        att_locate(&c, &a, &pl, s_range, &s_walk);
    } else if (warp == kMmaWarp) {
        tc_alloc(&s_tmem, C::TM_COLS);
        if (lane == 0) {
            s_abort = s_never = s_dirty = 0;
            if (cta == 0)
                st_checked(status, KIVI_OK);
            for (int i = 0; i < pl.ns; ++i) {
                for (int x = 0; x < 2; ++x) {
                    mbar_init(&s_full[x][i], 1);
                    mbar_init(&s_empty[x][i], C::WORKERS / 32);
                }
            }
            mbar_init(&s_sdone[0], 1);
            mbar_init(&s_sdone[1], 1);
            mbar_init(&s_odone, 1);
            mbar_fence_init();
        }
    }
    if constexpr (D == 64) {  // the second 64 rows of V^T are not channels: zero
        for (int i = tid; i < C::VATOM / 16; i += C::THREADS)
            reinterpret_cast<uint4*>(sm + C::O_V + C::VATOM)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;
    const int n = (int)(s_range[1] - s_range[0]);
    auto wait = [&](uint64_t* bar, int phase) { return att_wait(bar, phase & 1, &s_abort, status); };

    if (warp >= kCopyWarp && warp < kMmaWarp) {
        // ---------------------------------------------------------- copy ---
        const int which = warp - kCopyWarp;  // 0: keys, 1: values
        AttWalk w = s_walk;
        const bool starts_mid = w.j > 0;
        const int b0 = w.b, rr0 = w.rr;
        int* cut = reinterpret_cast<int*>(ws + kAttHeaderFloats) + (size_t)cta * kAttCutInts;
        if (warp == kCopyWarp && lane == 0)
            st_checked(cut, 0);
        // a unit: 32 tokens' codes, then its scales, then its zeros, at these
        // byte strides per 32 tokens (keys: statistics per group)
        const uint32_t code = which == 0 ? pl.kub : pl.vub;
        const uint32_t stat = which == 0 ? D * 4 : 32 * (D >> pl.lgG) * 4;
        const uint8_t* codes = reinterpret_cast<const uint8_t*>(which == 0 ? c.kq : c.vq);
        const uint8_t* scales = reinterpret_cast<const uint8_t*>(which == 0 ? c.kscale : c.vscale);
        const uint8_t* zeros = reinterpret_cast<const uint8_t*>(which == 0 ? c.kzero : c.vzero);
        const int lgs = which == 0 ? pl.lgG : 5;  // tokens of a statistic unit
        uint8_t* ring = sm + C::O_RING + (which == 0 ? 0 : pl.ns * pl.kst);
        const int stage = which == 0 ? pl.kst : pl.vst;
        int slot = 0, round = 0, sent = 0;
        bool alive = true;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int v0 = w.j * kAttTile;
            const int nuq = min(max((w.s.nq - v0) >> 5, 0), 4);
            const size_t bh = (size_t)w.b * c.H + w.rr / pl.RT;
            const int v = v0 + 32 * lane;  // this lane's unit of 32 tokens
            int t0 = v;
            bool go = lane < nuq;
            if (go && a.blocks) {
                const int g = ldg_checked(a.blocks + bh * a.n_keep + (v >> pl.lgG));
                go = g >= 0 && g < w.s.Tq >> pl.lgG;
                t0 = (g << pl.lgG) + (v & (c.G - 1));
            }
            const unsigned mask = __ballot_sync(0xffffffffu, go);
#pragma unroll 1
            for (int u0 = 0; u0 < 4; u0 += pl.su) {
                if (round > 0 && !__all_sync(0xffffffffu, wait(&s_empty[which][slot], round - 1))) {
                    alive = false;
                    break;
                }
                uint64_t* bar = &s_full[which][slot];
                const unsigned pmask = mask >> u0 & ((1u << pl.su) - 1);
                if (lane == 0) {
                    if (which == 0 && u0 == 0) {
                        AttDesc& d = s_desc[i & (kAttDescs - 1)];
                        d.b = w.b;
                        d.rr = w.rr;
                        d.nuq = nuq;
                        d.f0 = v0 - w.s.nq;
                        d.Tq = w.s.Tq;
                        d.res = w.s.len - w.s.Tq;
                        d.nd = w.s.nd;
                        d.tail = w.j == w.s.nt - 1;
                        d.mid = starts_mid && w.b == b0 && w.rr == rr0;
                        d.first = w.j == 0 || i == 0;
                        d.last = d.tail || i == n - 1;
                        d.umask = mask;
                        if (__builtin_expect(i == n - 1 && !d.tail && !d.mid, 0)) {
                            // the row tile starts in this range and its last tile, end - 1, is in range
                            // `last`: the first with total (last + 1) / count >= end
                            const long long end = s_range[1] + (w.s.nt - 1 - w.j);
                            st_checked(cut + 1, w.b);
                            st_checked(cut + 2, w.rr);
                            st_checked(cut + 3, (int)((end * s_range[3] + s_range[2] - 1) / s_range[2] - 1));
                            st_checked(cut, 1);
                        }
                    }
                    mbar_arrive_tx(bar, __popc(pmask) * (code + 2 * stat));
                }
                __syncwarp();
                const int u = lane - u0;  // unit of the stage
                if (go && u >= 0 && u < pl.su) {
                    const uint8_t* src = codes + (bh * (c.Tmax >> 5) + (t0 >> 5)) * code;
                    const size_t so = (bh * (c.Tmax >> lgs) + (t0 >> lgs)) * stat;
                    uint8_t* d = ring + slot * stage;
                    if (KIVI_IN_RANGE(src, code) && KIVI_IN_RANGE(scales + so, stat) && KIVI_IN_RANGE(zeros + so, stat)) {
                        bulk_g2s(d + u * code, src, code, bar);
                        bulk_g2s(d + pl.su * code + u * stat, scales + so, stat, bar);
                        bulk_g2s(d + pl.su * (code + stat) + u * stat, zeros + so, stat, bar);
                    }
                }
                ++sent;
                if (++slot == pl.ns) {
                    slot = 0;
                    ++round;
                }
            }
            if (!alive)
                break;
            att_next(w, c, a, pl.lgG, RB);
        }
        // every copy has landed before the CTA may end (the groups have
        // consumed them all unless a wait gave up)
#pragma unroll 1
        for (int s = max(0, sent - pl.ns); s < sent; ++s)
            att_wait(&s_full[which][s % pl.ns], (s / pl.ns) & 1, &s_never, nullptr);
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------- MMA ---
        const uint32_t one = elect_lane();
        const uint64_t kd = smem_desc(smem_addr(sm + C::O_K), D * 128);
        const uint64_t qd = smem_desc(smem_addr(sm + C::O_Q), 16);
        const uint64_t vd = smem_desc(smem_addr(sm + C::O_V), C::VATOM);
        const uint64_t pd = smem_desc(smem_addr(sm + C::O_P), C::PATOM);
        // S(0), S(1), then O(i) and S(i + 2)
        auto scores = [&](int i) {
            named_bar(1, C::WORKERS + 32);
            tc_fence_after();
            const uint32_t dst = tm + C::TM_S + (i & 1) * NR;
#pragma unroll 1
            for (int a64 = 0; a64 < D / 64; ++a64)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma(dst, kd + ((a64 * 4 + k) * 2048 >> 4), qd + ((a64 * (NR * 128) + k * 32) >> 4),
                           mma_idesc(NR, true, false), a64 + k > 0, one);
            tc_commit(&s_sdone[i & 1], one);
        };
#pragma unroll 1
        for (int i = -2; i < n; ++i) {
            if (i >= 0) {  // O(i)
                named_bar(1, C::WORKERS + 32);
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < MH * C::PASSES; ++x) {
                    const int h = x / C::PASSES, pass = x % C::PASSES;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma(tm + C::TM_O + h * C::PN, vd + ((h * 2 * C::VATOM + k * 2048) >> 4),
                               pd + ((pass * C::PTERM + k * 2048) >> 4), mma_idesc(C::PN, true, true), pass + k > 0, one);
                }
                tc_commit(&s_odone, one);
            }
            if (i + 2 < n)
                scores(i + 2);
        }
        // every product has ended before the TMEM is freed
        if (n > 0) {
            att_wait(&s_sdone[(n - 1) & 1], ((n - 1) >> 1) & 1, &s_never, nullptr);
            att_wait(&s_odone, (n - 1) & 1, &s_never, nullptr);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- workers ---
        const int qd = warp & 3, wg = warp >> 2, t = tid;
        const uint32_t lanes = (uint32_t)(qd * 32) << 16;
        const float sl2 = a.sm_scale * 1.4426950408889634f;
        const int W = (a.N + 63) >> 6;
        int slot[2] = {0, 0}, round[2] = {0, 0};  // of the key and the value ring

        auto release = [&](int which) {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s_empty[which][slot[which]]);
            if (++slot[which] == pl.ns) {
                slot[which] = 0;
                ++round[which];
            }
        };
        auto keys = [&](int i) {
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
#pragma unroll 1
            for (int u0 = 0; u0 < 4; u0 += pl.su) {
                wait(&s_full[0][slot[0]], round[0]);  // (the first stage brings the tile's descriptor)
                const uint8_t* st = sm + C::O_RING + slot[0] * pl.kst;
                uint8_t* kb = sm + C::O_K + u0 * D * 64;
                const int nu = min(d.nuq - u0, pl.su);
                const unsigned um = d.umask >> u0;
                switch (B ? B : c.bits_k) {
                case 2: rebuild_keys<D, C::WORKERS, B ? B : 2>(st, kb, t, pl.su, nu, um, pl.kub); break;
                case 4: rebuild_keys<D, C::WORKERS, B ? B : 4>(st, kb, t, pl.su, nu, um, pl.kub); break;
                default: rebuild_keys<D, C::WORKERS, B ? B : 8>(st, kb, t, pl.su, nu, um, pl.kub); break;
                }
                release(0);
            }
            if (__builtin_expect(d.first, 0))
                att_load_q<D, NR, C::WORKERS>(&c, &a, &pl, &d, sm + C::O_Q, t);
            if (__builtin_expect(d.nuq < 4, 0)) {
                if (d.nd > 0 && d.f0 + kAttTile > d.res)
                    att_seen<C::WORKERS>(&a, &d, s_seen[i & 3], t);
                att_fp16_rows<D, C::GROUPS>(&c, &a, &pl, &d, s_seen[i & 3], &s_dirty, sm + C::O_K, 0, t);
            }
        };
        auto values = [&](int i) {
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
#pragma unroll 1
            for (int u0 = 0; u0 < 4; u0 += pl.su) {
                wait(&s_full[1][slot[1]], round[1]);
                const uint8_t* st = sm + C::O_RING + pl.ns * pl.kst + slot[1] * pl.vst;
                uint8_t* vb = sm + C::O_V + u0 * 32 * 128;
                const int nu = min(d.nuq - u0, pl.su);
                const unsigned um = d.umask >> u0;
                switch (B ? B : c.bits_v) {
                case 2: rebuild_values<D, C::WORKERS, B ? B : 2>(st, vb, t, pl.su, nu, um, pl.vub, pl.lgG); break;
                case 4: rebuild_values<D, C::WORKERS, B ? B : 4>(st, vb, t, pl.su, nu, um, pl.vub, pl.lgG); break;
                default: rebuild_values<D, C::WORKERS, B ? B : 8>(st, vb, t, pl.su, nu, um, pl.vub, pl.lgG); break;
                }
                release(1);
            }
            if (__builtin_expect(d.nuq < 4, 0))
                att_fp16_rows<D, C::GROUPS>(&c, &a, &pl, &d, s_seen[i & 3], &s_dirty, sm + C::O_V, 1, t);
        };
        auto publish = [&]() {  // operands in shared memory, TMEM reads done: the MMA warp goes on
            fence_async_smem();
            tc_fence_before();
            named_bar(1, C::WORKERS + 32);
        };

        // A row's weights are 2^(S sl2 - ref); -inf before its first token.  All
        // threads of a row hold its reference: in registers up to 16 rows, in
        // shared memory beyond.
        float ref[C::REG_REF ? NC : 1];
        float l[NC], o[MH][NC];
        auto my_ref = [&]() {  // of row `lane`
            float x = -INFINITY;
            if constexpr (C::REG_REF) {
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    x = lane == k ? ref[k] : x;
            } else {
                x = s_ref[wg][lane % NC];
            }
            return x;
        };

        // the row tile that ends with tile i: its output, or a piece of it
        auto finish = [&](int i) {
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
            // sums of the weights over the 128 tokens, through P's buffer (its
            // product is done): each thread's row of NC, then 128 / NC partial
            // sums a row
            const int x = tid & 127;
            float* own = reinterpret_cast<float*>(sm + C::O_P) + (wg * 128 + x) * NC;
#pragma unroll
            for (int k = 0; k < NC; k += 4)
                *reinterpret_cast<float4*>(own + k) = make_float4(l[k], l[k + 1], l[k + 2], l[k + 3]);
            named_bar(3 + wg, 128);
            const float* col = reinterpret_cast<float*>(sm + C::O_P) + (wg * 128 + x / NC * NC) * NC + x % NC;
            float part = 0.0f;
#pragma unroll 4
            for (int k = 0; k < NC; ++k)
                part += col[k * NC];
            s_part[wg][x] = part;
            named_bar(3 + wg, 128);
            float L = 0.0f;
#pragma unroll
            for (int k = 0; k < 128; k += NC)
                L += s_part[wg][k + lane % NC];
            const int h = d.rr / pl.RT, r0 = (d.rr - h * pl.RT) * NR + wg * NC;
            float *dst, scale = 1.0f;
            bool mine = lane < NC;  // row `lane` is stored
            if (d.tail && !d.mid) {
                scale = row_scale(L);
                mine = mine && r0 + lane < pl.M && (!a.k || (r0 + lane) % a.N < d.nd);
                dst = a.out + (((size_t)d.b * a.Hq + (size_t)h * (a.Hq / c.H)) * a.N + r0) * D;
            } else {
                float* piece = att_part(ws, D, NR, (int)cta, d.mid ? 0 : 1);
                dst = piece + wg * NC * D;
                const float rf = my_ref();
                if (qd == 0 && lane < NC) {
                    st_checked(piece + (size_t)NR * D + wg * NC + lane, rf);
                    st_checked(piece + (size_t)NR * D + NR + wg * NC + lane, copysignf(L, s_dirty ? -1.0f : 1.0f));
                }
            }
            uint32_t rows = __ballot_sync(0xffffffffu, mine);
            if (D == 64 && qd >= 2)
                rows = 0;  // the upper lanes hold no channels
            dst += run16(32 * qd + lane);
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const float f = __shfl_sync(0xffffffffu, scale, k);
                if ((rows >> k) & 1u)
#pragma unroll
                    for (int x = 0; x < MH; ++x)
                        st_checked(dst + k * D + 128 * x, o[x][k] * f);
            }
            if (__builtin_expect(s_dirty && d.tail && !d.mid, 0))
                att_add_nonfinite<D, MH>(&a, &d, a.v + ((size_t)d.b * c.H + h) * a.N * D, r0, rows, run16(32 * qd + lane), dst);
        };

#pragma unroll 1
        for (int i = -2; i < n; ++i) {  // -2 and -1: the keys of tiles 0 and 1, the values of 0
            const AttDesc& d = s_desc[i & (kAttDescs - 1)];
            if (i >= 0) {
                if (i + 1 >= n)  // else it was waited for before the keys of tile i + 1
                    wait(&s_sdone[i & 1], i >> 1);
                tc_fence_after();
                if (__builtin_expect(d.first, 0)) {
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        if constexpr (C::REG_REF)
                            ref[k] = kAttNoRef;
                        l[k] = 0.0f;
#pragma unroll
                        for (int h = 0; h < MH; ++h)
                            o[h][k] = 0.0f;
                    }
                    if constexpr (!C::REG_REF) {
                        named_bar(3 + wg, 128);  // the previous row tile's are no longer read
                        if (qd == 0)
                            s_ref[wg][lane % NC] = kAttNoRef;
                        named_bar(3 + wg, 128);
                    }
                }
                // this warp's tokens: a quantized unit, or fp16 tokens
                const bool quant = qd < d.nuq;
                const bool skip = quant && !((d.umask >> qd) & 1u);
                const int j = d.f0 + 32 * qd + lane - d.res;  // draft, at or past 0
                const bool masked = skip || (!quant && j >= 0);
                uint32_t sees = 0u;                           // rows (bits) that attend this lane's token
                if (__builtin_expect(masked && !skip && j < d.nd, 0)) {
                    const uint64_t* mw = a.mask + (size_t)d.b * a.N * W + (j >> 6);
                    int row = ((d.rr % pl.RT) * NR + wg * NC) % a.N;
#pragma unroll 2
                    for (int k = 0; k < NC; ++k) {
                        if (row < d.nd)
                            sees |= (uint32_t)((ldg_checked(mw + (size_t)row * W) >> (j & 63)) & 1) << k;
                        if (++row == a.N)
                            row = 0;
                    }
                }
                __syncwarp();
                const uint32_t src = tm + C::TM_S + (i & 1) * NR + wg * NC + lanes;
                float y[CH];
                // -inf where the row does not attend the lane's token
                auto apply_mask = [&](int k0) {
                    if (__builtin_expect(masked, 0)) {
#pragma unroll
                        for (int k = 0; k < CH; ++k)
                            y[k] = (sees >> (k0 + k)) & 1u ? y[k] : -INFINITY;
                    }
                    __syncwarp();
                };
                auto exponents = [&](int k0) {
                    tc_ld(y, src + k0);
                    tc_wait_ld(y);
#pragma unroll
                    for (int k = 0; k < CH; k += 2)
                        mul_pair(y + k, sl2);
                    if constexpr (C::REG_REF) {
#pragma unroll
                        for (int k = 0; k < CH; k += 2)
                            sub_pair(y + k, ref + k0 + k);
                    } else {
#pragma unroll
                        for (int k = 0; k < CH; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(&s_ref[wg][k0 + k]);
                            sub_pair(y + k, &f.x);
                            sub_pair(y + k + 2, &f.z);
                        }
                    }
                    apply_mask(k0);
                };
                // the second time round, after the references moved, no weight passes the limit
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
                    float top = -INFINITY;
#pragma unroll
                    for (int k0 = 0; k0 < NC; k0 += CH) {
                        exponents(k0);
#pragma unroll
                        for (int k = 0; k < CH; ++k)
                            top = fmaxf(top, y[k]);
                    }
                    if (__builtin_expect(pass == 1 || !group_any(3 + wg, top > kAttLimit), 1))
                        break;
                    float mine = -INFINITY;  // the warp's largest logit of row `lane`
#pragma unroll
                    for (int k0 = 0; k0 < NC; k0 += CH) {
                        tc_ld(y, src + k0);
                        tc_wait_ld(y);
#pragma unroll
                        for (int k = 0; k < CH; k += 2)
                            mul_pair(y + k, sl2);
                        apply_mask(k0);
#pragma unroll
                        for (int k = 0; k < CH; ++k) {
                            const float x = redux_max(y[k]);
                            mine = lane == k0 + k ? x : mine;
                        }
                    }
                    const float old = my_ref();
                    if (lane < NC)
                        s_red[wg][lane][qd] = mine;
                    named_bar(3 + wg, 128);
                    const float4 r = *reinterpret_cast<const float4*>(s_red[wg][lane < NC ? lane : 0]);
                    const float m = fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w));
                    // a maximum beyond 2^20 is its own reference: 13 would be lost in it
                    const float next = fmaxf(old, fabsf(m) < 1048576.0f ? m - kAttShift : m);
                    const float alpha = next == old ? 1.0f : ex2_ftz(old - next);
                    if constexpr (!C::REG_REF) {
                        if (qd == 0)
                            s_ref[wg][lane % NC] = next;  // every warp has read the old one
                        named_bar(3 + wg, 128);
                    }
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        if constexpr (C::REG_REF)
                            ref[k] = __shfl_sync(0xffffffffu, next, k);
                        const float f = __shfl_sync(0xffffffffu, alpha, k);
                        l[k] *= f;
#pragma unroll
                        for (int h = 0; h < MH; ++h)
                            o[h][k] *= f;
                    }
                }
                uint8_t* prow = sm + C::O_P + (32 * qd + lane) * 128;
                const int sw = lane & 7;  // token position % 8
#pragma unroll
                for (int k0 = 0; k0 < NC; k0 += CH) {
                    if (NC > CH)
                        exponents(k0);
                    uint32_t hi[CH / 2], lo[CH / 2];
#pragma unroll
                    for (int k = 0; k < CH; k += 2) {
                        y[k] = ex2_ftz(y[k]);
                        y[k + 1] = ex2_ftz(y[k + 1]);
                        add_pair(l + k0 + k, y + k);
                        split_pair(y + k, hi[k / 2], lo[k / 2]);
                    }
                    const int r0 = wg * NC + k0;
#pragma unroll
                    for (int k = 0; k < CH; k += 8) {  // eight rows: a 16-byte chunk of each term
                        const int ck = (r0 + k) >> 3;
                        uint8_t* row = prow + (ck >> 3) * C::PATOM;
                        const uint4 vh = make_uint4(hi[k / 2], hi[k / 2 + 1], hi[k / 2 + 2], hi[k / 2 + 3]);
                        const uint4 vl = make_uint4(lo[k / 2], lo[k / 2 + 1], lo[k / 2 + 2], lo[k / 2 + 3]);
                        *reinterpret_cast<uint4*>(row + (((ck & 7) ^ sw) << 4)) = vh;
                        if constexpr (C::STACK)
                            *reinterpret_cast<uint4*>(row + (((NR / 8 + ck) ^ sw) << 4)) = vl;
                        else
                            *reinterpret_cast<uint4*>(row + C::PTERM + (((ck & 7) ^ sw) << 4)) = vl;
                    }
                }
                publish();  // O(i) is issued
            }
            if (i + 2 < n) {
                if (i >= -1)
                    wait(&s_sdone[(i + 1) & 1], (i + 1) >> 1);
                keys(i + 2);
                publish();  // S(i + 2) is issued
            }
            if (i >= 0) {
                wait(&s_odone, i);
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < MH; ++h)
#pragma unroll
                    for (int k0 = 0; k0 < NC; k0 += 8) {
                        float y[8];
                        const uint32_t src = tm + C::TM_O + h * C::PN + wg * NC + k0 + lanes;
                        tc_ld(y, src);
                        if constexpr (C::STACK) {
                            float z[8];
                            tc_ld(z, src + NR);
                            tc_wait_ld(y);
                            tc_wait_ld(z);
#pragma unroll
                            for (int k = 0; k < 8; k += 2)
                                add_pair(y + k, z + k);
                        } else {
                            tc_wait_ld(y);
                        }
#pragma unroll
                        for (int k = 0; k < 8; k += 2)
                            add_pair(o[h] + k0 + k, y + k);
                    }
                if (__builtin_expect(d.last, 0)) {
                    finish(i);
                    named_bar(2, C::WORKERS);  // P's buffer, where the sums went, may be written
                }
            }
            if (i >= -1 && i + 1 < n)
                values(i + 1);
        }
        tc_fence_before();
    }
    asm volatile("griddepcontrol.launch_dependents;");
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tc_dealloc(tm, C::TM_COLS);
    }
}

// ---------------------------------------------------------------- combine ---

// Merges the pieces of the row tiles that CTA ranges cut: block (i, y) takes
// eight rows of the row tile that starts in range i and ends in a later one,
// piece by piece in order.
constexpr int kAttCombineThreads = 256;
constexpr int kAttCombineRows = 8;

// Adds to this block's rows of the row tile that starts with row `row0` and has
// `rows` rows the values that are not finite of the drafts which they attend.  A
// thread takes the elements that it stored.
static __device__ __noinline__ void att_merge_nonfinite(const kivi_cache* c, const AttendArgs* a, int b, int h, int nd,
                                                        int row0, int rows)
{
    const int D = c->D, W = (a->N + 63) >> 6;
    const uint16_t* v = a->v + ((size_t)b * c->H + h) * a->N * D;
    float* dst = a->out + (((size_t)b * a->Hq + (size_t)h * (a->Hq / c->H)) * a->N + row0) * D;
#pragma unroll 1
    for (int e = threadIdx.x; e < kAttCombineRows * D; e += kAttCombineThreads) {
        const int r = blockIdx.y * kAttCombineRows + e / D, d = e % D, q = (row0 + r) % a->N;
        if (r >= rows || q >= nd)
            continue;
        const uint64_t* words = a->mask + ((size_t)b * a->N + q) * W;
        float y = 0.0f;
#pragma unroll 1
        for (int j = 0; j < nd; ++j)
            if ((ldg_checked(words + (j >> 6)) >> (j & 63)) & 1)
                y += nonfinite(v + (size_t)j * D + d);
        if (y != 0.0f)
            st_checked(dst + (size_t)r * D + d, ld_checked(dst + (size_t)r * D + d) + y);
    }
}

static __global__ void __launch_bounds__(kAttCombineThreads)
attend_combine_kernel(const __grid_constant__ kivi_cache c, const __grid_constant__ AttendArgs a,
                      const __grid_constant__ AttPlan pl, int NR, float* __restrict__ ws)
{
    const int D = c.D, i = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int* cut = reinterpret_cast<const int*>(ws + kAttHeaderFloats) + (size_t)i * kAttCutInts;
    if (ld_checked(cut) == 0)
        return;
    const int b = ld_checked(cut + 1), rr = ld_checked(cut + 2), last = ld_checked(cut + 3);
    const int h = rr / pl.RT, rt = rr - h * pl.RT;
    const int nd = a.k ? (a.n_draft ? min(max(ldg_checked(a.n_draft + b), 0), a.N) : a.N) : 1;
    // negative: a piece cleared values of drafts, which lie in the last three tiles
    int sign[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int piece = max(last - k, i);
        sign[k] = __float_as_int(ld_checked(att_part(ws, D, NR, piece, piece == i) + (size_t)NR * D + NR));
    }
#pragma unroll 1
    for (int e = threadIdx.x; e < kAttCombineRows * D; e += kAttCombineThreads) {
        const int r = blockIdx.y * kAttCombineRows + e / D, d = e % D, row = rt * NR + r;
        if (row >= pl.M || row % a.N >= nd)
            continue;
        float M = kAttNoRef, L = 0.0f, o = 0.0f;
#pragma unroll 1
        for (int k = i; k <= last; ++k) {
            const float* p = att_part(ws, D, NR, k, k == i);
            const float m = ld_checked(p + (size_t)NR * D + r), l = fabsf(ld_checked(p + (size_t)NR * D + NR + r)),
                        x = ld_checked(p + (size_t)r * D + d);
            const float Mn = fmaxf(M, m), f = ex2_ftz(M - Mn), g = ex2_ftz(m - Mn);
            L = L * f + l * g;
            o = o * f + x * g;
            M = Mn;
        }
        st_checked(a.out + (((size_t)b * a.Hq + (size_t)h * (a.Hq / c.H)) * a.N + row) * D + d, L == 0.0f ? 0.0f : o / L);
    }
    if (__builtin_expect((sign[0] | sign[1] | sign[2]) < 0, 0))
        att_merge_nonfinite(&c, &a, b, h, nd, rt * NR, min(NR, pl.M - rt * NR));
}

// ----------------------------------------------------------------- launch ---

template <int D, int NR, int B>
cudaError_t attend_launch_rows(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s)
{
    using C = AttCfg<D, NR>;
    auto kern = attend_kernel<D, NR, B>;
    const AttPlan pl = att_plan<D, NR>(c.G, c.bits_k, c.bits_v, a.Hq / c.H * a.N);
    if (pl.ns < 1)
        return cudaErrorInvalidConfiguration;
    const int smem = att_smem_bytes<D, NR>(pl);
    static int allowed[64];
    cudaError_t e = allow_smem(kern, kAttSmem - C::STATIC, allowed);
    if (e != cudaSuccess)
        return e;
    const int N = cmin(C::CTAS * sm_count(), kAttMaxCTAs);
    kern<<<N, C::THREADS, smem, s>>>(c, a, pl, ws);
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

}  // namespace kivi
