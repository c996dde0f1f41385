"""The attention's plan over a cache in 8 bits, on the CPU: as test_kv_plan.py, with the few-column units of that form."""
from __future__ import annotations

import test_kv_plan


def in_8_bits(code):
    """The harness's batches, planned for a cache in 8 bits (bf16 operands)."""
    code = code.replace("{v[3], v[5]});", "{v[3], v[5]}, true);")
    assert ", true);" in code
    return code.replace("{64, 2}, {128, 2}, {256, 2}, {64, 4}, {128, 4}", "{64, 2}, {128, 2}, {256, 2}, {64, 2}, {128, 2}")


def run(monkeypatch, main):
    monkeypatch.setattr(test_kv_plan, "HARNESS", in_8_bits(test_kv_plan.HARNESS))
    test_kv_plan.run(main)


def test_plans_fit_their_workspace(monkeypatch):
    code = in_8_bits(test_kv_plan.HARNESS)
    run(monkeypatch, code[code.index("int main()"):])


def test_a_smaller_batch_needs_no_more(monkeypatch):
    """A batch none of whose bounds is larger has a workspace that is no larger."""
    run(monkeypatch, r"""
int main() {
    std::mt19937 rng(11);
    auto pick = [&](std::vector<int> v) { return v[rng() % v.size()]; };
    const int heads[][2] = {{32, 8}, {64, 8}, {4, 4}, {20, 1}, {5, 1}, {512, 256}};
    int smaller = 0;
    for (int n = 0; n < 100000; ++n) {
        const auto& h = heads[rng() % 6];
        const int d = pick({64, 128, 256});
        int v[7] = {pick({1, 8, 31, 200, 600, 5000}), pick({1, 32, 900, 20000}), pick({1, 4, 17, 4096}),
                    pick({0, 300, 1500, 2048, 9000, 60000}), pick({0, 1, 8, 600}), pick({0, 64, 2500, 70000}),
                    pick({0, 4, 32, 4096})};
        int w[7];
        for (int i = 0; i < 7; ++i) w[i] = rng() % 2 ? v[i] : (int)(rng() % (v[i] + 1));
        const size_t large = plan(h[0], h[1], d, 2, v, 0, 0).bytes, small = plan(h[0], h[1], d, 2, w, pick({0, 300}), 4).bytes;
        smaller += small < large;
        if (small > large) {
            for (int i = 0; i < 7; ++i) std::printf("%d %d; ", v[i], w[i]);
            std::printf("heads %d on %d of %d: %zu %zu\n", h[0], h[1], d, large, small);
            return 1;
        }
    }
    return smaller ? 0 : 2;
}
""")
