"""The blocks that a step's list always holds have to fit into it.  CPU only."""
import pytest

from deepseek_v4_sparse_indexer_gb300 import PagedDecodeStep


@pytest.mark.parametrize("blocks,keep", [(2, (2, 1)), (1, (1, 1)), (4, (0, 5)), (4, (5, 0)), (4, (-1, 2)), (4, (2, -1))])
def test_lists_too_short_for_the_kept_blocks(blocks, keep):
    with pytest.raises(ValueError, match="keep_blocks"):
        PagedDecodeStep(2, 8, 16, top_k=0, blocks=blocks, keep_blocks=keep, device="cpu")


@pytest.mark.parametrize("blocks,keep", [(2, (1, 1)), (3, (2, 1)), (4, (0, 4)), (4, (0, 0))])
def test_lists_of_kept_blocks(blocks, keep):
    assert PagedDecodeStep(2, 8, 16, top_k=0, blocks=blocks, keep_blocks=keep, device="cpu").idx.shape == (2, 1, blocks)


def test_no_blocks_to_keep():
    assert PagedDecodeStep(2, 8, 16, top_k=8, keep_blocks=(1, 1), device="cpu").blocks == 0
