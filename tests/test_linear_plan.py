"""moe_linear without a GPU: its plan, run on the host over the sizes that a call may have: every pass has a ring of at least two
stages (one is loaded while one is read), fits in shared memory, and together they take all tokens; and the order of a cluster's first steps."""
import os
import subprocess

from bit_moe_decode_02_gb300 import build_ext

SOURCE = r"""
#include "linear_plan.h"
#include <cstdio>
#include <initializer_list>
using namespace moe::linear;

static long long checked = 0;

static bool good(const Plan& p, const Size& a, int clusters)
{
    const int K = p.steps * kCols < a.K ? p.steps * kCols : a.K, nt = p.tokens > 8 ? 2 : 1;
    const int sums = a.fmt == MOE_FMT_INT4 ? p.tokens * (K / a.group) * 4 : 0;
    const int join = p.cs > 1 ? 2 * ((kWarps / p.ks + p.cs - 1) / p.cs) * p.cs * nt * 512 : 0;
    ++checked;
    return p.tokens >= 1 && p.tokens <= 16 && p.tokens <= a.M && (p.cs == 1 || (p.cs == kCluster && clusters > 0)) &&
           p.steps * p.cs * kCols >= a.K && p.ks >= 1 && p.ks <= kWarps && p.stages >= 2 && p.stages <= kMostStages &&
           p.smem() <= kSmem && p.x_pitch >= 2 * K && p.x_pitch % 16 == 0 && p.off_sum >= p.tokens * p.x_pitch &&
           p.off_fac >= p.off_sum + sums && p.off_red >= p.off_fac + 256 && p.off_join >= p.off_red + kWarps * nt * 512 &&
           p.off_ring >= p.off_join + join && p.off_fac % 16 == 0 && p.off_red % 16 == 0 && p.off_join % 16 == 0 &&
           p.off_ring % 128 == 0 && p.stage_bytes % 128 == 0;
}

int main()
{
    const int formats[5][2] = {{MOE_FMT_MXFP4, 32}, {MOE_FMT_INT4, 32}, {MOE_FMT_INT4, 64}, {MOE_FMT_INT4, 128}, {MOE_FMT_INT4, 256}};
    const int rows[] = {1, 17, 512, 2560, 5120, 8192, 9728, 16384, 40000, 65537, 151936, 200000, 1 << 24};
    const int tokens[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17, 27, 33, 40, 64};
    for (const auto& f : formats)
        for (int K = f[1]; K <= 32768; K += f[1])
            for (int N : rows)
                for (int M : tokens)
                    for (int clusters : {0, 32, 35, 38}) {
                        const Size all{N, K, f[0], f[1], M};
                        const Plan first = choose(all, 152, clusters);
                        bool ok = good(first, all, clusters);
                        for (int m0 = 0; ok && m0 < M; m0 += first.tokens) {
                            Size a = all;
                            a.M = M - m0 < first.tokens ? M - m0 : first.tokens;
                            Plan p;
                            plan(p, a, first.cs, first.cs > 1 ? clusters : 152);
                            ok = good(p, a, clusters) && p.tokens == a.M;
                        }
                        if (!ok) {
                            std::printf("bad: %d x %d, format %d, group %d, %d tokens, %d clusters: %d tokens a pass, cs %d, ks %d, "
                                        "%d stages, %d bytes\n", N, K, f[0], f[1], M, clusters, first.tokens, first.cs, first.ks,
                                        first.stages, first.smem());
                            return 1;
                        }
                    }
    std::printf("%lld plans\n", checked);
    return 0;
}
"""


def test_every_size_has_a_plan_that_fits(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", build_ext.CSRC, "-I", os.path.join(build_ext.ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_a_cluster_has_started_before_its_memory_is_written():
    """Every CTA arrives at the cluster's barrier as it starts; the first store to another CTA's shared memory comes after
    the wait for those arrivals.  (The order is invisible in results: starting nearly always takes less than reading x.)"""
    with open(os.path.join(build_ext.CSRC, "moe_linear.cu")) as f:
        kernel = f.read()
    arrive, wait, store = (kernel.index(w) for w in ("barrier.cluster.arrive", "barrier.cluster.wait", "st.shared::cluster"))
    assert arrive < wait < store
