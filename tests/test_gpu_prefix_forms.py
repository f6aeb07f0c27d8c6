"""sdv_prefix_attn: sides of its choices beside those of tests/test_gpu_prefix_attn.py."""
import pytest

import tests.test_gpu_prefix_attn as base
from tests.test_gpu_prefix_attn import BF16, F16

pytestmark = pytest.mark.gpu
sdv = base.sdv

# Wide windows over tables of one tile, joined where the own positions are computed: two or three row groups
# of a kv head, of which some have no row of a window at all (n from 0 to S).
WIDE = [
    (F16, 64, 32, 32, 8, 128, 16, 200, False),
    (BF16, 48, 32, 24, 4, 128, 32, 129, True),
    (F16, 70, 32, 16, 4, 64, 8, 65, True),
    (BF16, 40, 32, 48, 8, 64, 64, 0, False),
    (BF16, 66, 17, 32, 8, 128, 16, 300, False),
]


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_several_row_groups_joined_on_the_spot(sdv, case, monkeypatch):
    monkeypatch.setattr(base, "MANY", WIDE)
    base.test_many_rows_and_short_tables(sdv, case)
