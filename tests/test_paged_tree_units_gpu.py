"""Large fp32 trees at d = 128 with 6, 9 and 10 heads to a key/value head, whose units of 32 rows
hold 30 and 27 (test_paged_launches_cpu.py: that they are taken)."""
import pytest

from test_paged_tree_gpu import check_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv", [(6, 1), (9, 1), (20, 2)])
@pytest.mark.parametrize("how", ["tree", "any"])
def test_groups_that_do_not_fill_32_rows(H, Hkv, how):
    for seqs in ([(40, 700), (33, 33), (1, 129), (0, 50), (35, 128)], [(70, 3000), (64, 70)]):
        check_tree(seqs, H, Hkv, 128, "f32", 32, "bshd", how, seed=H, max_pages=200000 // 32, behind=3)
    # keys of few long sequences split over many CTAs, whose sums fill the slots
    check_tree([(64, 9000), (50, 8000)], H, Hkv, 128, "f32", 16, "bhsd", how, seed=H + 1)
