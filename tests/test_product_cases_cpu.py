"""CPU check that the shapes of tests/product_cases.py reach every way in which the 8-bit product is laid out, so that
a change of its plans cannot take one out of the GPU tests unseen."""
import product_cases as cases
import test_block_plans_cpu as plans


def test_cases_cover_every_plan(tmp_path, monkeypatch):
    monkeypatch.setattr(plans, "COMMON", plans.COMMON.replace('"grkan_plan.h"', '"grkan_train_plan.h"')
                        + "#include <set>\n#include <string>\n" + r"""
static std::string one(const Product8Plan &p, long m, long n) {
    if (p.few) return "few" + std::to_string(p.few);
    const long tiles = (m + p.tile - 1) / p.tile * ((n + p.tile - 1) / p.tile) * p.splits, cus = 256;
    const long most = cus * (p.tile == 256 ? 1 : (p.tile == 128 ? 2 : 4));
    return std::to_string(p.tile) + (p.splits > 1 ? " split" : "") + (tiles > most ? " several" : "");
}
static std::string kind(long m, long n, long k, int type, int tile) {
    const bool bf16 = type > 0, cut = type == 2;
    const Product8Plan p = plan_product8(m, n, k, bf16, tile, cut);
    std::string s = std::to_string(type) + (tile ? " tiles " : " columns ") + one(p, p.rows, n);
    if (p.rows < m) s += ", then " + one(plan_product8_whole(m - p.rows, n, k, bf16, tile, cut), m - p.rows, n);
    return s;
}
""")
    rows = lambda c: ",".join("{%d,%d,%d}" % x for x in c)  # noqa: E731
    plans.run(tmp_path, "const long every[][3] = {%s}, cut[][3] = {%s};" % (rows(cases.EVERY), rows(cases.CUT_TILES)) + r"""
    std::set<std::string> have;
    for (auto &c : every)
        for (int type = 0; type < 3; ++type)
            for (int tile = 0; tile < 2; ++tile) have.insert(kind(c[0], c[1], c[2], type, tile));
    for (auto &c : cut) have.insert(kind(c[0], c[1], c[2], 2, 1));
    std::set<std::string> missing;
    for (long m = 1; m < 60000; m = m * 9 / 8 + 1)
        for (long n = 1; n < 10000; n = n * 9 / 8 + 1)
            for (long k = 1; k < 50000; k = k * 8 / 7 + 1)
                for (int type = 0; type < 3; ++type)
                    for (int tile = 0; tile < 2; ++tile) {
                        const std::string s = kind(m, n, k, type, tile);
                        if (!have.count(s) && missing.insert(s).second) CHECK(false, "%s: e.g. %ld x %ld from %ld", s.c_str(), m, n, k);
                        ++checked;
                    }
""")
    for m, n, k in cases.EVERY + cases.CUT_TILES:
        assert n % 16 and k % 16 and (m == 1 or m % 16)
