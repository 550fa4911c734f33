"""When a dense product on MXFP4 tokens splits its sums, told from the scratch that
it asks for (none without splits)."""
import pytest

from mxfp4_routed_expert_route_gb300 import _native, build


@pytest.fixture(scope="module")
def scratch():
    build.build()
    return _native.load().mxfp4_linear_workspace_size


@pytest.mark.parametrize("T,I,O", [(16, 2880, 5760), (64, 7168, 4096), (128, 7168, 4096),
                                   (384, 7168, 4096), (512, 4096, 512), (2000, 4096, 512),
                                   (1, 2880, 5760), (8192, 7168, 4096)])
def test_no_split_where_the_join_costs_more_than_it_saves(scratch, T, I, O):
    """Measured in one piece and split: 16 x 2880 x 5760 7.1 and 8.4 us or more, 384 x
    7168 x 4096 13.2 and 22, 512 x 4096 x 512 8.0 and 9.5, the others likewise."""
    assert scratch(T, I, O) == 0


@pytest.mark.parametrize("T,I,O", [(1, 7168, 4096), (16, 7168, 4096), (1, 4096, 512), (48, 4096, 512)])
def test_a_split_where_few_tokens_meet_long_sums(scratch, T, I, O):
    """1 x 7168 x 4096: 10.5 us in one piece, 8.6 in four."""
    assert scratch(T, I, O) > 0
