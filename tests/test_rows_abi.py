"""Entry points that state their buffers' rows: exported, and refused without a
plan before anything else is looked at (CPU)."""
import varlen_gqa_split_b200 as vg


def test_rows_entry_points_refuse_unknown_plans():
    from varlen_gqa_split_b200 import build
    build.build()
    L, p = vg.lib(), 0x10000
    for plan in (None, 0x1234):
        assert L.attn_run_rows(plan, p, 4, p, p, 8, 64, 64, p, p, p, p, None) == -5
        assert L.attn_run_paged_rows(plan, p, 4, p, p, 1024, 64, 16, 4, p, 4, p, p, p, p, None) == -5
