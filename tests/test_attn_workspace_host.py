"""Workspace of biloco_attn_paged as a batch's sizes ask for it (no GPU)."""
import pytest

from bit_weight_gemm_amd import binding as B

TILE_ROWS, MOST_ROWS = 128, 64      # rows a workgroup of the tiles kernel takes; above MOST_ROWS a sequence is its


def tile_bytes(tiles, kv_heads, splits, dim):
    return tiles * kv_heads * splits * TILE_ROWS * (dim + 2) * 4


@pytest.mark.parametrize("B_,T,hq,hk,dim,kv", [(32, 32, 64, 8, 128, 131072), (8, 32, 64, 8, 128, 32768),
                                               (64, 64, 40, 8, 128, 32768), (1000, 1000, 16, 2, 64, 100000)])
def test_a_batch_asks_for_the_tiles_it_can_have(B_, T, hq, hk, dim, kv):
    # T new tokens make at most T G / 65 sequences of more than 64 rows, each
    # ending one tile early; their pieces fill 512 workgroups, or exceed them by
    # less than a tile's heads
    rows = T * hq // hk
    seqs = min(B_, rows // (MOST_ROWS + 1))
    tiles = (rows + (TILE_ROWS - 1) * seqs) // TILE_ROWS
    most = tile_bytes(1, 1, 512 + tiles * hk, dim)
    # and the pieces of the sequences of few rows: one a workgroup, 64 rows each
    few = (B_ * hk + 512) * 64 * (dim + 2) * 4 + 8 * (B_ * hk + 1)
    assert B.biloco_attn_workspace_bytes(B_, T, hq, hk, dim, T, kv) <= most + few
