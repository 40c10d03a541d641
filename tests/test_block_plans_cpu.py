"""CPU checks of the block operators' plans (csrc/grkan_plan.h, host code without HIP): a g++-built harness
asks for the plans of a grid of shapes and checks what the kernels and the callers rely on."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gr_kan_rational_amd", "csrc")

COMMON = r"""
#include "grkan_plan.h"
#include <cstdio>
using namespace grkan;
static long checked = 0, bad = 0;
#define CHECK(ok, ...) do { ++checked; if (!(ok) && bad++ < 10) { printf(__VA_ARGS__); printf("\n"); } } while (0)
"""
TAIL = r"""
    printf("checked %ld bad %ld\n", checked, bad);
    return checked == 0 || bad != 0;
}
"""


def run(tmp_path, body):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "plans.cpp", tmp_path / "plans"
    src.write_text(COMMON + "int main() {" + body + TAIL)
    subprocess.run([gxx, "-O2", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_linear_backward_plans_have_kernels_and_workspace(tmp_path):
    """Whatever the alignment of its operands, each product of the backward is planned for a kernel that
    exists, and the workspace asked of the caller, who states none of it, is enough."""
    run(tmp_path, r"""
    const int rows[] = {1, 65, 197, 1003, 4099, 5297, 8449, 12801, 50432, 201728};
    const int act[] = {GRKAN_ACT_NONE, GRKAN_ACT_RATIONAL};
    for (int r : rows)
        for (int i = 49; i < 4100; i += 97)
            for (int o = 51; o < 4100; o += 97)
                for (int a : act) {
                    const size_t most = linear_bwd_bytes(r, i, o, 1, (grkan_act_t)a);
                    for (int al = 0; al < 4; ++al) {
                        LinearBwdPlan p;
                        linear_bwd_plan(r, i, o, 1, (grkan_act_t)a, al & 1, al & 2, &p);
                        CHECK(p.dx.aligned == ((al & 1) != 0) && p.dw.aligned == ((al & 2) != 0), "alignment");
                        CHECK(plan_has_kernel(p.dx) && plan_has_kernel(p.dw), "%d %d %d: no kernel", r, i, o);
                        CHECK(p.total <= most, "%d %d %d: %zu of %zu", r, i, o, p.total, most);
                    }
                }
""")


def test_linear_forward_workspace_is_enough_for_any_alignment(tmp_path):
    """The bytes that the caller is told, who states no alignment, against those of either plan."""
    run(tmp_path, r"""
    const int rows[] = {1, 65, 130, 241, 700, 1003, 1500, 3000, 6789, 9366, 20000, 50432};
    const int act[] = {GRKAN_ACT_NONE, GRKAN_ACT_RATIONAL};
    for (int r : rows)
        for (int i = 48; i < 10000; i += 123)
            for (int o = 60; o < 30000; o += 317)
                for (int a : act) {
                    const size_t said = linear_fwd_bytes(r, i, o, 1, (grkan_act_t)a);
                    for (int al = 0; al < 2; ++al) {
                        const ProductPlan p = plan_product(kFormForward, r, o, i, al, a, act_group(o, 1, (grkan_act_t)a));
                        CHECK(plan_has_kernel(p), "%d %d %d: no kernel", r, i, o);
                        CHECK(p.partials_bytes <= said, "%d %d %d: %zu of %zu", r, i, o, p.partials_bytes, said);
                    }
                }
""")


def test_workspace_queries_follow_the_plans(tmp_path):
    """The library's queries at shapes whose aligned and unaligned plans differ: rows, widths, bytes of the
    plan with more of them."""
    from gr_kan_rational_amd import binding, block

    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    lib = block._library()
    for rows, d_in, d_out, splits in ((130, 2265, 24786, 3), (1003, 6203, 12387, 2), (130, 1688, 24608, 3)):
        got = lib.grkan_linear_act_forward_workspace_size(rows, d_in, d_out, 1, block.GRKAN_ACT_SILU)
        assert got == (splits * rows * d_out * 4 + 255) // 256 * 256


def test_group_norm_plans_fit_a_cus_lds(tmp_path):
    """1 to 8,192 channels with every divisor as groups: no plan asks for more LDS than a CU has, in a launch
    of at most 1,024 threads, and the forward's second pass has room for its statistics."""
    run(tmp_path, r"""
    const int ns[] = {1, 2, 8, 64, 128}, ss[] = {1, 2, 197, 1024, 4097};
    for (int C = 1; C <= 8192; ++C)
        for (int G = 1; G <= C; ++G) {
            if (C % G) continue;
            for (int n : ns)
                for (int s : ss)
                    for (int k = 0; k < 8; ++k) {
                        const int act = k & 1 ? GRKAN_ACT_RATIONAL : GRKAN_ACT_SILU;
                        const int ng = C % 8 ? (C % 3 ? 1 : 3) : 8;
                        NormPlan p;
                        const int st = norm_plan(n, s, C, G, ng, (grkan_act_t)act, k & 2 ? GRKAN_F32 : GRKAN_BF16, k & 4, &p);
                        CHECK(st == GRKAN_OK, "%d x %d x %d / %d: status %d", n, s, C, G, st);
                        CHECK(p.lds <= (160 << 10), "%d x %d x %d / %d: %zu of LDS", n, s, C, G, p.lds);
                        CHECK(p.block >= 1 && p.block <= 1024, "%d x %d x %d / %d: %d threads", n, s, C, G, p.block);
                        CHECK(p.kind != kNormSplit || (size_t)p.groups * 8 <= (160 << 10), "%d groups", p.groups);
                    }
        }
""")
