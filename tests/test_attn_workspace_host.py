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


@pytest.mark.parametrize("hq,hk,dim", [(64, 8, 128), (40, 8, 128), (40, 1, 128), (40, 40, 128), (4, 2, 64), (128, 1, 64)])
@pytest.mark.parametrize("kv", [64, 613, 4096, 16384, 32768, 131072])
def test_bytes_cover_every_smaller_call(hq, hk, dim, kv):
    def need(b, t, q, n):
        return B.biloco_attn_workspace_bytes(b, t, hq, hk, dim, q, n)
    tokens = [1, 2, 3, 5, 8, 9, 13, 16, 17, 25, 31, 32, 64, 100, 500, 4096]
    grid = {(b, t, q): need(b, t, q, kv) for b in (1, 2, 3, 8, 31, 32, 33, 200) for t in tokens for q in tokens}
    for (b, t, q), n in grid.items():      # one step down along each axis covers the rest
        for axis, values in ((0, (1, 2, 3, 8, 31, 32, 33, 200)), (1, tokens), (2, tokens)):
            at = values.index((b, t, q)[axis])
            if at:
                less = list((b, t, q))
                less[axis] = values[at - 1]
                assert grid[tuple(less)] <= n, (less, (b, t, q))
        assert need(b, t, q, kv // 2) <= n and need(b, t, q, max(0, kv - 700)) <= n, (b, t, q)


@pytest.mark.parametrize("heads,kv_heads,sequences,kv", [(64, 8, 1, 16384), (64, 8, 1, 32768), (40, 8, 2, 32768),
                                                         (64, 8, 8, 32768), (40, 1, 2, 131072)])
def test_a_block_holds_the_workspace_of_every_step(heads, kv_heads, sequences, kv):
    from bit_weight_gemm_amd.decoder import AttentionBlock, Linear
    dim, width = 128, heads * 128

    def linear(N, K):
        return Linear(None, None, 1.0, None, None, None, N, K, 16)
    block = AttentionBlock(linear((heads + 2 * kv_heads) * dim, width), linear(width, width), heads, kv_heads, dim, None,
                           None, None, None, max_sequences=sequences, max_kv_len=kv, device="cpu")
    for b in range(1, sequences + 1):
        for t in range(1, block.MAX_TOKENS + 1):
            for q in range(1, t + 1):
                assert B.biloco_attn_workspace_bytes(b, t, heads, kv_heads, dim, q, kv) <= block._attn_ws.numel(), (b, t, q)
