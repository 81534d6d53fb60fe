// attend_plan.h -- shapes of the sparse and tree attention kernels (attend.cuh,
// attend_warp.cuh): shared memory, TMEM and workspace.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define KIVI_HD __host__ __device__
#else
#define KIVI_HD
#endif

namespace kivi {

constexpr int kAttSmem = 227 * 1024;          // shared memory of one CTA alone on its SM
constexpr int kAttTile = 128;                 // tokens per tile
constexpr int kAttMaxCTAs = 320;              // bound on the grid, which sizes the workspace
constexpr int kAttMaxStages = 8;              // of each ring
constexpr int kAttDescs = 16;                 // tile descriptors kept in shared memory
constexpr int kAttCutInts = 4;                 // of a cut row tile: set, sequence, head or row tile, last range
constexpr int kAttHeaderFloats = 4;
constexpr float kAttShift = 13.0f;            // a row's largest weight is 2^13 when its reference is set ...
constexpr float kAttLimit = 15.9f;            // ... and stays below 2^15.9, inside fp16

// Whether M query rows of a KV head go to the warp kernel (attend_warp.cuh),
// whose registers hold O of 16 rows (8 at D = 256).
inline bool attend_by_warp(int D, int M) { return M <= (D == 256 ? 8 : 16); }

// Rows per row tile of the tcgen05 kernel (attend.cuh) for M query rows: the
// smallest tile that holds them, up to 128; shared memory holds 32 at D = 256.
// In us with tiles of 32 / 64 / 128 rows, B 8, H 32, T 4096, int2:
//     M             48                65               128               256
//     D 128  340/233/315       495/426/324       659/447/349      1443/948/749
//     D 64   243/199/281       354/364/284       480/382/301      1079/802/642
// and past 128 rows the whole tiles of 128 are the same or better too, but for
// one sequence of few heads (160 rows, B 1, H 8, T 32768: 211/173/184).
inline int attend_rows(int D, int M) { return M <= 32 || D == 256 ? 32 : M <= 64 ? 64 : 128; }

// Workspace: header (status word), a cut descriptor per CTA, two partial
// (o [NR][D], m [NR], l [NR]) slots per CTA: slot 0 for a row tile that an
// earlier CTA started, slot 1 for one that starts here and ends later.
KIVI_HD inline float* att_part(float* ws, int D, int NR, int cta, int slot)
{
    return ws + kAttHeaderFloats + kAttMaxCTAs * kAttCutInts + ((size_t)cta * 2 + slot) * NR * (D + 2);
}

// The same for the warp kernel: descriptors and slots of every warp, M rows.
constexpr int kAttMaxRanges = kAttMaxCTAs / 2 * 16;
KIVI_HD inline size_t warp_part_floats(int D, int M) { return (size_t)(M * (D + 2) + 3) / 4 * 4; }
KIVI_HD inline float* warp_part(float* ws, int D, int M, long long range, int slot)
{
    return ws + kAttHeaderFloats + kAttMaxRanges * kAttCutInts + ((size_t)range * 2 + slot) * warp_part_floats(D, M);
}

// A CTA has 8 or 16 worker warps, two copy warps (keys, values) and the MMA
// warp.  A tile passes through a chain of steps with a barrier or a wait
// between any two, so where shared memory allows (D <= 128, up to 32 rows) two
// CTAs of 8 worker warps share an SM: one computes while the other waits,
// starts a row or ends one.
template <int D, int NR>
struct AttCfg {
    static constexpr int CTAS = D <= 128 && NR <= 32 ? 2 : 1;  // CTAs per SM
    static constexpr int WORKERS = CTAS == 2 ? 256 : 512;
    static constexpr int THREADS = WORKERS + 96;
    static constexpr int GROUPS = WORKERS / 128;       // row groups
    static constexpr int MH = D == 256 ? 2 : 1;        // 128-channel halves of the output
    static constexpr int NC = NR / GROUPS;             // rows of a worker warp
    static constexpr int CH = NC < 16 ? NC : 16;       // rows of one TMEM read
    static constexpr bool REG_REF = NC <= 16;
    static constexpr bool STACK = NR <= 32;            // both terms of P side by side in one product
    static constexpr int PN = NR <= 64 ? 64 : NR;      // columns of the second product
    static constexpr int PASSES = STACK ? 1 : 2;
    static constexpr int KBYTES = 256 * D;             // 64-token columns of D x 128 bytes
    static constexpr int VATOM = kAttTile * 128;       // 64-channel columns of 128 x 128 bytes
    static constexpr int VBYTES = VATOM * (D == 64 ? 2 : D / 64);  // the M axis has 128 rows at least
    static constexpr int PATOM = kAttTile * 128;       // 64 columns of P
    static constexpr int PTERM = PATOM * PN / 64;      // one term of P
    static constexpr int PBYTES = PTERM * PASSES;
    static constexpr int QBYTES = D / 64 * NR * 128;
    static constexpr int O_K = 0;
    static constexpr int O_V = O_K + KBYTES;
    static constexpr int O_P = O_V + VBYTES;
    static constexpr int O_Q = O_P + PBYTES;
    static constexpr int O_RING = O_Q + QBYTES;
    static constexpr int TM_S = 0;                     // TMEM columns: S of even and odd tiles, O
    static constexpr int TM_O = 2 * NR;
    static constexpr int TM_USED = TM_O + MH * PN;
    static constexpr int TM_COLS = TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;
    // 1024: base alignment; an SM has 228 KB, of which every CTA takes one more
    static constexpr int STATIC = (CTAS == 2 ? 3 : 6) * 1024;  // bound on the kernel's static shared arrays
    static constexpr int RING = (CTAS == 2 ? 113 * 1024 : kAttSmem) - STATIC - 1024 - O_RING;
    static_assert(O_Q % 1024 == 0 && QBYTES % 1024 == 0 && O_P % 1024 == 0, "operand alignment");
    static_assert(D != 256 || NR <= 32, "shared memory");
};

// Sizes the kernel needs besides the descriptor's.
struct AttPlan {
    int lgG, M, RT;       // log2 G, query rows of a KV head, row tiles
    int su;               // 32-token units of a ring stage: a tile's four, or two
    int ns;               // stages of each ring
    int kst, vst;         // bytes of a stage: keys, values
    int kub, vub;         // code bytes of 32 tokens: keys, values
};

template <int D, int NR>
AttPlan att_plan(int G, int bits_k, int bits_v, int M)
{
    using C = AttCfg<D, NR>;
    AttPlan pl;
    pl.lgG = G == 32 ? 5 : G == 64 ? 6 : 7;
    pl.M = M;
    pl.RT = (M + NR - 1) / NR;
    pl.kub = 4 * D * bits_k;
    pl.vub = 4 * D * bits_v;
    for (pl.su = 4;; pl.su = 2) {  // a tile per stage where one fits, else half a tile
        pl.kst = pl.su * (pl.kub + 8 * D);
        pl.vst = pl.su * (pl.vub + 256 * (D / G));
        pl.ns = C::RING / (pl.kst + pl.vst);
        pl.ns = pl.ns < kAttMaxStages ? pl.ns : kAttMaxStages;
        if (pl.ns > 0 || pl.su == 2)
            return pl;
    }
}

template <int D, int NR>
int att_smem_bytes(const AttPlan& pl)
{
    return 1024 + AttCfg<D, NR>::O_RING + pl.ns * (pl.kst + pl.vst);
}

// The warp kernel (attend_warp.cuh).
constexpr int kWarpStatic = 4 * 1024;                      // bound on its static shared arrays

template <int D, int NT>
struct WarpCfg {
    static constexpr int WARPS = NT == 2 ? 12 : D == 256 ? 10 : 16;  // by registers: 168, 200, 128 a thread
    static constexpr int HAT = 64 * D;                     // K_hat or V_hat of a unit
    static_assert(D != 256 || NT == 1, "registers");
};

struct WarpPlan {
    int lgG, M, warps;    // log2 G, query rows of a KV head, warps per CTA
    int kub, vub;         // code bytes of 32 tokens
    int kst, vst;         // with statistics
    int bytes;            // shared memory of a warp
    int by_row;           // records of cut rows by row, not by range
};

template <int D, int NT>
WarpPlan warp_plan(int G, int bits_k, int bits_v, int M)
{
    WarpPlan pl;
    pl.lgG = G == 32 ? 5 : G == 64 ? 6 : 7;
    pl.M = M;
    pl.kub = 4 * D * bits_k;
    pl.vub = 4 * D * bits_v;
    pl.kst = pl.kub + 8 * D;
    pl.vst = pl.vub + 256 * (D / G);
    pl.bytes = WarpCfg<D, NT>::HAT + pl.kst + pl.vst;
    const int fit = (kAttSmem - kWarpStatic) / pl.bytes;
    pl.warps = fit < WarpCfg<D, NT>::WARPS ? fit : WarpCfg<D, NT>::WARPS;
    pl.by_row = 0;
    return pl;
}

}  // namespace kivi
