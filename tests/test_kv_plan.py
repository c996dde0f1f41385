"""The attention's plan on the CPU: whatever a batch's plan uses, with any window, lies in the workspace that the query
names, each part in a place of its own."""
from __future__ import annotations

import os
import subprocess
import tempfile

from lora_bgmv_shrink_amd import build as hb

HARNESS = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "kv_internal.hpp"
using namespace lora;

static AttnPlan plan(int hq, int hkv, int d, int eb, const int (&v)[7], int window, int sinks) {
    AttnPlan P;
    std::memset(&P, 0, sizeof P);
    P.a.C.n_kv_heads = hkv;
    P.a.n_q_heads = hq;
    P.a.share = hq / hkv;
    P.a.B.n_seqs = v[0];
    P.a.B.n_rows = v[1];
    P.a.B.n_groups = v[4];
    P.a.window = window;
    P.a.n_sink = sinks;
    plan_attn(P, d, eb, {v[0], v[4]}, {std::min(v[2], v[1]), std::min(v[6], v[1])}, {v[3], v[5]});
    return P;
}

int main() {
    std::mt19937 rng(7);
    auto pick = [&](std::vector<int> v) { return v[rng() % v.size()]; };
    const int heads[][2] = {{32, 8}, {64, 8}, {4, 4}, {20, 1}, {64, 2}, {5, 1}, {512, 256}};
    const int dims[][2] = {{64, 2}, {128, 2}, {256, 2}, {64, 4}, {128, 4}};
    int split = 0, shared = 0, wide = 0;
    for (int n = 0; n < 200000; ++n) {
        const auto& h = heads[rng() % 7];
        const auto& d = dims[rng() % 5];
        const int v[7] = {pick({1, 8, 31, 32, 200, 600, 5000}), pick({1, 32, 100, 900, 4096, 20000}),
                          pick({1, 4, 5, 17, 100, 4096}), pick({0, 1, 512, 513, 2048, 2049, 9000, 60000}),
                          pick({0, 0, 1, 3, 8, 600}), pick({0, 64, 2500, 9000, 70000}), pick({0, 4, 32, 300, 4096})};
        const int window = pick({0, 1, 63, 100, 600, 2048, 8000, 50000}), sinks = pick({0, 4, 200, 3000});
        const size_t bytes = plan(h[0], h[1], d[0], d[1], v, 0, 0).bytes;
        const AttnPlan P = plan(h[0], h[1], d[0], d[1], v, window, sinks);
        struct Part { size_t at, n; };
        std::vector<Part> used;
        for (int k = 0; k < 2; ++k) {
            const AttnPart& W = P.a.part[k];
            const int n_prob = k ? v[4] : v[0];
            if (W.few == 2) {
                ++shared;
                used.push_back({P.off[k][0], (size_t)n_prob * h[1] * sizeof(int2)});
                used.push_back({P.off[k][1], (size_t)2 * W.few_grid * 16 * d[0] * 4});
                used.push_back({P.off[k][2], (size_t)2 * W.few_grid * 16 * sizeof(float2)});
            }
            if (W.slots) {
                ++split;
                wide += P.a.tile_cols == 256;
                used.push_back({P.off[k][3], (size_t)n_prob * sizeof(int4)});
                used.push_back({P.off[k][4], (size_t)W.tile_grid * P.a.tile_cols * d[0] * 4});
                used.push_back({P.off[k][5], (size_t)W.tile_grid * P.a.tile_cols * sizeof(float2)});
            }
            if (P.a.join) used.push_back({P.off[k][6], (size_t)v[1] * h[0] * (d[0] * 4 + sizeof(float2))});
        }
        bool ok = P.bytes == bytes;
        for (size_t i = 0; i < used.size(); ++i) {
            ok = ok && used[i].at % 16 == 0 && used[i].at + used[i].n <= bytes;
            for (size_t j = 0; j < i; ++j)
                ok = ok && (used[i].at + used[i].n <= used[j].at || used[j].at + used[j].n <= used[i].at);
        }
        if (!ok) {
            std::printf("heads %d on %d, d %d (%d bytes), window %d, sinks %d:", h[0], h[1], d[0], d[1], window, sinks);
            for (int x : v) std::printf(" %d", x);
            std::printf("\n");
            return 1;
        }
    }
    std::printf("shared %d split %d wide %d\n", shared, split, wide);
    return shared && split && wide ? 0 : 2;
}
"""


RULE = r"""
int main() {
    // requests of one row and up to so many tokens on 8 key heads: whole heads per workgroup (1) or shares (2)
    const int rows[][3] = {{1, 512, 1}, {1, 1024, 2}, {8, 1024, 1}, {8, 2048, 2}, {16, 2048, 1}, {31, 2048, 1}, {32, 2048, 1},
                           {33, 2048, 1}, {32, 4096, 2}, {512, 8000, 1}};
    for (const auto& r : rows) {
        const int v[7] = {r[0], r[0], 1, r[1], 0, 0, 0};
        const AttnPlan P = plan(32, 8, 128, 2, v, 0, 0);
        std::printf("%d requests of %d tokens: %d\n", r[0], r[1], P.a.part[0].few);
        if (P.a.part[0].few != r[2]) return 1;
    }
    return 0;
}
"""


def run(main):
    code = HARNESS[:HARNESS.index("int main()")] + main
    with tempfile.TemporaryDirectory() as d:
        src, obj, exe = (os.path.join(d, n) for n in ("plan.hip", "plan.o", "plan"))
        with open(src, "w") as f:
            f.write("#include <algorithm>\n#include <cstring>\n" + code)
        lib = ["-Wl,-rpath," + os.path.dirname(hb.LIB_PATH)]
        for cmd in ([hb.HIPCC, *hb.FLAGS, "-I", hb.CSRC, "-c", src, "-o", obj],
                    [hb.HIPCC, obj, hb.LIB_PATH, *lib, "-o", exe]):
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-3000:]
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        print(r.stdout)
        assert r.returncode == 0, r.stdout + r.stderr


def test_plans_fit_their_workspace():
    run(HARNESS[HARNESS.index("int main()"):])


def test_one_request_less_keeps_the_form():
    run(RULE)
