"""Host arithmetic of the attention kernels' geometry over the extents that the entry points
allow: a small program includes the kernels' headers, evaluates their formulas and prints them."""
import os
import subprocess

import pytest

from spatial_transformer_sampling_gb300 import build as gsbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "gs_attn.cuh"
using namespace gs;

static AttnArgs args(int N, int H, int D, int Hq, int Wq, int Hk, int Wk) {
    AttnArgs a = {};
    a.N = N; a.H = H; a.D = D;
    a.Hq = Hq; a.Wq = Wq; a.Hk = Hk; a.Wk = Wk;
    a.Lq = Hq * Wq; a.Lk = Hk * Wk;
    a.P = Wq + Wk - 1;
    a.R = (Hq + Hk - 1) * a.P;
    a.nb = 1;
    return a;
}

// Lines of "what D Hq Wq Hk Wk" on the input, a number for each on the output.
int main() {
    char what[32];
    int D, g[4];
    while (scanf("%31s %d %d %d %d %d", what, &D, g, g + 1, g + 2, g + 3) == 6) {
        const AttnArgs a = args(1, 1, D, g[0], g[1], g[2], g[3]);
        long long v = -1;
        if (!strcmp(what, "stride")) v = rel_stride_of(a);
        if (!strcmp(what, "window")) v = rel_window_of(a);
        const TcBias q = tc_bias_of(a, false), k = tc_bias_of(a, true);
        if (!strcmp(what, "bwd_smem"))
            v = D <= 64 ? tc_bwd_launch_of<64>(k, q, true, rel_window_of(a)).smem
                        : tc_bwd_launch_of<128>(k, q, true, rel_window_of(a)).smem;
        if (!strcmp(what, "bwd_mode"))
            v = D <= 64 ? tc_bwd_launch_of<64>(k, q, true, rel_window_of(a)).mode
                        : tc_bwd_launch_of<128>(k, q, true, rel_window_of(a)).mode;
        if (!strcmp(what, "fwd_smem"))
            v = D <= 64 ? std::max(TcFwdShape<64, kFwdMany>::kSmem, TcFwdShape<64, kFwdSplit>::kSmem) +
                              TcFwdShape<64, kFwdMany>::kStages * q.count * 4
                        : std::max(TcFwdShape<128, kFwdMany>::kSmem, TcFwdShape<128, kFwdSplit>::kSmem) +
                              TcFwdShape<128, kFwdMany>::kStages * q.count * 4;
        if (!strcmp(what, "simt_smem"))
            v = std::max({simt_fwd_smem(D), simt_bwd_smem(D, true, 0), simt_bwd_smem(D, false, rel_window_of(a))});
        if (!strcmp(what, "groups")) v = rel_groups_at_once((int)rel_stride_of(a));
        printf("%lld\n", v);
    }
}
"""


@pytest.fixture(scope="module")
def geometry(tmp_path_factory):
    d = tmp_path_factory.mktemp("geometry")
    src, exe = d / "geometry.cu", d / "geometry"
    src.write_text(PROGRAM)
    r = subprocess.run([gsbuild.nvcc(), *gsbuild.ARCH, "-std=c++17", "--expt-relaxed-constexpr",
                        "-I", gsbuild.CSRC, "-I", gsbuild.INCLUDE, "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert os.path.exists(exe)

    def ask(what, cases):
        text = "".join(f"{what} {D} {q[0]} {q[1]} {k[0]} {k[1]}\n" for D, q, k in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True)
        return [int(x) for x in out.stdout.split()]

    return ask


def test_offsets_of_the_bias_gradients_sums_fit_32_bits(geometry):
    # 512 groups of 32 queries over as many keys as the relative indices allow (2^24): the offset
    # of a group, with the last key's relative index and the entry's own beside it
    cases = [(64, (1, 16384), (1, 4_300_000)), (64, (1, 16384), (1, (1 << 24) - 16383)),
             (64, (2, 8192), (1, 4_190_000)), (64, (1, 9), (4000, 4000)), (64, (32, 32), (32, 32)),
             (64, (1, 1), (1, 1)), (64, (4000, 4000), (1, 1))]
    strides, groups = geometry("stride", cases), geometry("groups", cases)
    assert max(511 * s for s in strides) > 1 << 31 and groups[0] < 512
    for (_, q, k), s, n in zip(cases, strides, groups):
        entries = (q[0] + k[0] - 1) * (q[1] + k[1] - 1)
        assert 1 <= n <= 512 and (n - 1) * s + 2 * entries < 1 << 31
    assert groups[4] == 512


def _widest_use_of_the_window(q, k):
    """Largest number of relative indices that one step of 64 keys adds to, or makes final, for
    any 32 queries."""
    (hq, wq), (hk, wk) = q, k
    P, Lq, Lk = wq + wk - 1, hq * wq, hk * wk
    rel_q = lambda i: (i // wq + hk - 1) * P + i % wq + wk - 1
    rel_k = lambda j: j // wk * P + j % wk
    widest = 0
    for i in range(0, Lq, 32):
        low, high = rel_q(i), rel_q(min(i + 31, Lq - 1))
        top = high
        for j in range(0, Lk, 64):
            bottom = low - rel_k(min(j + 63, Lk - 1))
            final_above = bottom - 1 if j + 64 >= Lk else high - rel_k(j + 64)
            widest = max(widest, high - rel_k(j) - bottom + 1, top - final_above)
            top = final_above
    return widest


WINDOW_GRIDS = [((1, 226), (70, 63)), ((1, 130), (70, 63)), ((1, 34), (64, 63)), ((1, 400), (90, 63)),
                ((1, 500), (9, 21)), ((4, 33), (70, 21)), ((8, 8), (8, 8)), ((32, 32), (32, 32)),
                ((1, 300), (1, 257)), ((3, 100), (5, 70)), ((20, 1), (31, 1)), ((2, 65), (2, 65)),
                ((17, 23), (17, 23)), ((64, 3), (64, 3)), ((20, 8), (4, 130)), ((12, 200), (9, 7)),
                ((7, 9), (65, 9)), ((1, 77), (70, 7))]


def test_window_of_the_bias_gradient_holds_what_a_step_adds_to_and_what_it_leaves(geometry):
    windows = geometry("window", [(64, q, k) for q, k in WINDOW_GRIDS])
    assert any(windows)
    for (q, k), w in zip(WINDOW_GRIDS, windows):
        assert w == 0 or w >= _widest_use_of_the_window(q, k), (q, k, w)


def test_every_launch_fits_into_a_blocks_shared_memory(geometry):
    # grids of one to forty rows, narrow against wide: their windows are the largest
    widths = (1, 2, 4, 8, 12, 16, 20, 31, 32, 48, 64, 96, 128, 130, 200, 208, 224, 256, 300, 466)
    grids = [((hq, wq), (hk, wk)) for hq in (1, 3, 8, 20, 40) for hk in (1, 3, 4, 32, 40)
             for wq in widths for wk in widths]
    for D in (64, 128):
        cases = [(D, q, k) for q, k in grids]
        for what, limit in (("bwd_smem", 223 * 1024), ("fwd_smem", 223 * 1024),
                            ("simt_smem", 227 * 1024 - 256)):
            worst = max(zip(geometry(what, cases), cases))
            assert worst[0] <= limit, (what, worst)


def test_windows_of_the_bias_are_copied_wherever_they_fit(geometry):
    window, through_l1 = 1, 2
    cases = [(64, (32, 32), (32, 32)), (128, (48, 48), (48, 48)), (128, (1, 3000), (1, 3000)),
             (128, (64, 64), (64, 64)), (64, (20, 8), (4, 130))]
    assert geometry("bwd_mode", cases) == [window] * len(cases)
    cases = [(128, (20, 8), (4, 130)), (128, (16, 8), (3, 128)), (128, (40, 16), (40, 208)),
             (128, (1, 32), (32, 1)), (128, (16, 16), (1, 256))]
    assert geometry("bwd_mode", cases) == [through_l1] * len(cases)
