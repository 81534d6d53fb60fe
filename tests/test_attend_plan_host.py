"""Host checks of the plans of the sparse and tree attention kernels, for
every shape they are instantiated for.

csrc/attend_plan.h sizes the operands, rings and TMEM of the tcgen05 kernel and
the per-warp buffers of the warp kernel.  This test compiles the real header
into a host program and checks what nothing checks at run time: every ring
holds a stage, what a launch asks for fits the shared memory of an SM as many
times as CTAs are meant to share it, bulk copies and operands keep their
alignment, the accumulators fit TMEM, and the workspace holds every piece."""
import json
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kivi_bit_kv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "attend_plan.h"
using namespace kivi;

static bool first = true;
template <int D, int NR> void tensor()
{
    using C = AttCfg<D, NR>;
    for (int G = 32; G <= 128; G *= 2)
        for (int bk = 2; D % G == 0 && bk <= 8; bk *= 2)
            for (int bv = 2; bv <= 8; bv *= 2) {
                const AttPlan p = att_plan<D, NR>(G, bk, bv, NR + 1);
                printf("%s{\"kind\": \"tensor\", \"D\": %d, \"NR\": %d, \"G\": %d, \"bk\": %d, \"bv\": %d, \"ctas\": %d, "
                       "\"threads\": %d, \"static\": %d, \"smem\": %d, \"ns\": %d, \"su\": %d, \"kst\": %d, \"vst\": %d, "
                       "\"kub\": %d, \"vub\": %d, \"lgG\": %d, \"RT\": %d, \"O\": [%d, %d, %d, %d, %d], \"bytes\": [%d, %d, %d, %d], "
                       "\"NC\": %d, \"CH\": %d, \"tm_used\": %d, \"tm_cols\": %d, \"vatom\": %d}",
                       first ? "" : ",\n", D, NR, G, bk, bv, C::CTAS, C::THREADS, C::STATIC, att_smem_bytes<D, NR>(p),
                       p.ns, p.su, p.kst, p.vst, p.kub, p.vub, p.lgG, p.RT, C::O_K, C::O_V, C::O_P, C::O_Q, C::O_RING,
                       C::KBYTES, C::VBYTES, C::PBYTES, C::QBYTES, C::NC, C::CH, C::TM_USED, C::TM_COLS, C::VATOM);
                first = false;
            }
}
template <int D, int NT> void warp()
{
    using C = WarpCfg<D, NT>;
    for (int G = 32; G <= 128; G *= 2)
        for (int bk = 2; D % G == 0 && bk <= 8; bk *= 2)
            for (int bv = 2; bv <= 8; bv *= 2) {
                const WarpPlan p = warp_plan<D, NT>(G, bk, bv, 8 * NT);
                printf(",\n{\"kind\": \"warp\", \"D\": %d, \"NT\": %d, \"G\": %d, \"bk\": %d, \"bv\": %d, \"warps\": %d, \"most\": %d, "
                       "\"bytes\": %d, \"hat\": %d, \"kst\": %d, \"vst\": %d, \"kub\": %d, \"vub\": %d}",
                       D, NT, G, bk, bv, p.warps, C::WARPS, p.bytes, C::HAT, p.kst, p.vst, p.kub, p.vub);
            }
}
int main()
{
    printf("{\"smem\": %d, \"warp_static\": %d, \"max_stages\": %d, \"descs\": %d, \"ranges\": %d, \"max_ctas\": %d, \"rows\": [",
           kAttSmem, kWarpStatic, kAttMaxStages, kAttDescs, kAttMaxRanges, kAttMaxCTAs);
    const int dims[] = {64, 128, 256};
    for (int d = 0; d < 3; ++d)
        for (int M = 1; M <= 200; ++M)
            printf("%s[%d, %d, %d, %d]", d + M > 1 ? ", " : "", dims[d], M, (int)attend_by_warp(dims[d], M), attend_rows(dims[d], M));
    printf("], \"shapes\": [\n");
    tensor<64, 32>(), tensor<64, 64>(), tensor<64, 128>();
    tensor<128, 32>(), tensor<128, 64>(), tensor<128, 128>();
    tensor<256, 32>();
    warp<64, 1>(), warp<64, 2>(), warp<128, 1>(), warp<128, 2>(), warp<256, 1>();
    printf("]}\n");
    return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("attend_plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", f"-I{CSRC}", "-o", str(exe), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return json.loads(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout)


def of_kind(plan, kind):
    return [s for s in plan["shapes"] if s["kind"] == kind]


def test_every_shape_is_planned(plan):
    per = {64: 2 * 9, 128: 3 * 9, 256: 3 * 9}  # group sizes that divide D, times widths
    assert len(of_kind(plan, "tensor")) == 3 * per[64] + 3 * per[128] + per[256]
    assert len(of_kind(plan, "warp")) == 2 * per[64] + 2 * per[128] + per[256]


def test_every_row_count_has_a_kernel(plan):
    for D, M, by_warp, rows in plan["rows"]:
        assert by_warp == (M <= (8 if D == 256 else 16))
        if not by_warp:
            assert rows == 32 if D == 256 else rows in (32, 64, 128)
            assert rows >= M or rows == (32 if D == 256 else 128)


def test_rings_hold_a_stage_and_fit(plan):
    for s in of_kind(plan, "tensor"):
        assert 1 <= s["ns"] <= plan["max_stages"], s
        assert s["su"] in (2, 4)
        assert s["smem"] + s["static"] <= plan["smem"], s
        # an SM has 228 KB, of which every CTA takes one more KB
        assert s["ctas"] * (s["smem"] + s["static"] + 1024) <= 228 * 1024, s
        assert s["ctas"] * s["threads"] <= 2048 and s["threads"] <= 1024
        # the copies are at most a ring ahead of the keys, which are two tiles ahead
        assert 3 + s["ns"] <= plan["descs"], s
        assert s["RT"] == 2
        assert 1 << s["lgG"] == s["G"]


def test_operands_and_copies_are_aligned(plan):
    for s in of_kind(plan, "tensor"):
        ends = [o + n for o, n in zip(s["O"], s["bytes"])]
        assert s["O"][0] == 0 and s["O"][1:] == ends, s  # K, V, P, Q, then the ring
        assert all(o % 1024 == 0 for o in s["O"]), s
        assert s["NC"] % 8 == 0 and s["CH"] % 8 == 0 and s["NC"] % s["CH"] == 0
        assert s["bytes"][1] >= 2 * s["vatom"]
    for s in plan["shapes"]:
        D, G = s["D"], s["G"]
        units = s.get("su", 1)
        assert s["kub"] == 32 * D * s["bk"] // 8 and s["vub"] == 32 * D * s["bv"] // 8
        assert s["kst"] == units * (s["kub"] + 2 * D * 4)
        assert s["vst"] == units * (s["vub"] + 2 * 32 * (D // G) * 4)
        for n in (s["kub"], s["vub"], D * 4, 32 * (D // G) * 4, s["kst"], s["vst"]):
            assert n % 16 == 0, s


def test_accumulators_fit_tmem(plan):
    for s in of_kind(plan, "tensor"):
        assert s["tm_used"] <= s["tm_cols"] <= 512 and s["ctas"] * s["tm_cols"] <= 512, s
        assert s["tm_cols"] & (s["tm_cols"] - 1) == 0


def test_warp_buffers_fit(plan):
    for s in of_kind(plan, "warp"):
        assert 4 <= s["warps"] <= s["most"] <= 16, s
        assert s["bytes"] == s["hat"] + s["kst"] + s["vst"] and s["bytes"] % 16 == 0
        assert s["hat"] == 32 * s["D"] * 2
        assert s["warps"] * s["bytes"] + plan["warp_static"] <= plan["smem"], s
        assert plan["max_ctas"] // 2 * s["warps"] <= plan["ranges"]
