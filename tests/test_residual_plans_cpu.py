"""CPU check of the launch that ends the residual path's backward (csrc/grkan_train_plan.h)."""
import test_block_plans_cpu as plans


def test_sums_fit_a_launch(tmp_path, monkeypatch):
    """A launch of 1,024 threads a workgroup stays below 2^32 threads however many gates there are; every column has
    its workgroups, and every gate a thread, in as many rounds as that takes."""
    monkeypatch.setattr(plans, "COMMON", plans.COMMON.replace('"grkan_plan.h"', '"grkan_train_plan.h"'))
    plans.run(tmp_path, r"""
    const long gates[] = {0, 1, 1023, 1024, 1025, 1L << 20, 1L << 30, (1L << 30) + 1, 1L << 32, 1L << 38};
    for (long g : gates)
        for (long c : {1L, 31L, 32L, 33L, 1024L, 16384L})
            for (int sums = 0; sums < 2; ++sums) {
                const ResidualSums s = residual_sums(c, sums, g);
                CHECK(s.blocks * 1024 < (1L << 32), "%ld gates of %ld channels: %ld workgroups", g, c, (long)s.blocks);
                CHECK(s.columns == (sums ? 3 * ((c + 31) / 32) : 0), "%ld channels", c);
                CHECK(g > 0 ? s.blocks > s.columns : s.blocks == s.columns, "%ld gates", g);
                CHECK(g > (1L << 30) || (s.blocks - s.columns) * 1024 >= g, "%ld gates in one round", g);
            }
""")
