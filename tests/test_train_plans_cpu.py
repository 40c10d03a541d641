"""CPU checks of the plans of the operators of include/grkan_train.h (csrc/grkan_train_plan.h, host code without
HIP): a g++-built harness asks for the plans of a grid of shapes and checks what the kernels and the callers rely
on."""
import pytest

from test_block_plans_cpu import run as run_block


def run(tmp_path, body):
    run_block(tmp_path, body)


@pytest.fixture(autouse=True)
def header(monkeypatch):
    import test_block_plans_cpu as t

    monkeypatch.setattr(t, "COMMON", t.COMMON.replace('"grkan_plan.h"', '"grkan_train_plan.h"'))


def test_product_plans(tmp_path):
    """A kernel for every plan: rows of 16 for few or small results, a tile of 64, 128 or (bf16 results and a scale for each tile of b)
    256, the rows past its whole rounds by a plan of their own; the splits are whole blocks, cover K and leave none empty; the workspace is enough for every type and layout
    of scales; an XCD's eighth of the tiles and splits fits 31 bits."""
    run(tmp_path, r"""
    const long ms[] = {1, 16, 17, 33, 64, 65, 100, 197, 1003, 4096, 50432, 201728, 2147483391L};
    const long ks[] = {1, 16, 127, 128, 129, 300, 768, 3001, 16384, 50432, 1000000, 1L << 22};
    for (long m : ms)
        for (long n = 1; n <= (1 << 22); n = n * 3 + 5)
            for (long k : ks) {
                if (product8_shape(m, n, k) != GRKAN_OK) continue;
                const size_t most = product8_bytes(m, n, k);
                for (int i = 0; i < 4; ++i) {
                    const bool bf = i & 1, bt = i & 2;
                    const Product8Plan p = plan_product8(m, n, k, bf, bt);
                    CHECK(p.rows >= 1 && p.rows <= m, "%ld %ld %ld: rows %ld", m, n, k, (long)p.rows);
                    if (p.rows < m) {
                        CHECK(p.tile == 256 && p.splits == 1 && p.rows % 256 == 0 && m - p.rows > kFewRows, "rows apart");
                        const Product8Plan r = plan_product8_whole(m - p.rows, n, k, bf, bt);
                        CHECK(r.rows == m - p.rows && r.partials_bytes == p.partials_bytes, "the rest");
                    }
                    CHECK(p.few > 0 || m > kFewRows, "few rows");
                    if (p.few > 0) {
                        CHECK(p.few == 1 || p.few == 2 || p.few == 4, "%ld %ld %ld: few %d", m, n, k, p.few);
                        CHECK(p.splits == 1 && p.partials_bytes == 0, "few rows are not split");
                        CHECK((m + 16 * p.few - 1) / (16 * p.few) < 65536, "grid");
                        continue;
                    }
                    CHECK(p.tile == 64 || p.tile == 128 || (p.tile == 256 && bf && bt), "%ld %ld %ld: tile %d", m, n, k, p.tile);
                    CHECK(p.k_split % kBlock8 == 0 && p.splits >= 1, "%ld %ld %ld: k_split %ld", m, n, k, (long)p.k_split);
                    CHECK((p.splits - 1) * p.k_split < k && p.splits * p.k_split >= k, "%ld %ld %ld: splits", m, n, k);
                    CHECK(p.partials_bytes <= most, "%ld %ld %ld: workspace", m, n, k);
                    CHECK(p.splits == 1 || p.partials_bytes == (size_t)p.splits * m * n * 4, "partials");
                    const double tiles = (double)((m + p.tile - 1) / p.tile) * ((n + p.tile - 1) / p.tile) * p.splits;
                    CHECK(tiles + 16 < 2147483647.0, "%ld %ld %ld: %g tiles", m, n, k, tiles);
                }
            }
""")


def test_residual_plans(tmp_path):
    """Every row of every width has lanes for its channels, with no more accesses a lane than kernels are compiled
    for; every row has a walker; the workspace holds what the walkers leave."""
    run(tmp_path, r"""
    const long rs[] = {1, 2, 3, 5, 64, 197, 2047, 2048, 2049, 50432, 1000003, 2147483647L};
    for (long r : rs)
        for (long c = 1; c <= kMaxChannels; c = c < 40 ? c + 1 : c + 37)
            for (int way = 0; way < 2; ++way)
                for (int post = 0; post < 3; ++post)
                    for (int wide = 0; wide < 3; ++wide) {
                        ResidualPlan p;
                        const long gates = wide ? (r % 2 == 0 ? r / 2 : 1) : 0;
                        residual_plan(r, c, gates, wide == 2 ? c : 1, (grkan_norm_t)post, way, &p);
                        const long lanes = 64L * p.waves, quads = (c + 3) / 4;
                        CHECK(lanes * p.K >= quads && lanes * (p.K - 1) < quads, "%ld channels: %d x %d", c, p.waves, p.K);
                        const int id = p.waves * 8 + p.K;
                        CHECK((p.waves == 1 && p.K <= 4) || id == 18 || id == 19 || id == 34 || id == 35 || id == 66 || id == 67 ||
                              id == 68 || id == 131 || id == 132, "%ld channels: no kernel for %d waves of %d", c, p.waves, p.K);
                        const long walkers = p.blocks * p.per;
                        CHECK(walkers * p.walk >= r && p.walk >= 1 && p.blocks < (1 << 20), "%ld rows: walkers", r);
                        if (!way) continue;
                        size_t need = (size_t)p.blocks * p.sums * c * 4;
                        CHECK(p.off_gate >= need, "%ld %ld: sums", r, c);
                        if (gates > 0 && r > gates) {
                            const size_t g = wide == 2 && c > 1 ? (size_t)walkers * 2 * c * 4 : (size_t)r * 4;
                            CHECK(p.total >= p.off_gate + g, "%ld %ld: gate sums", r, c);
                        }
                    }
""")
