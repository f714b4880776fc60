"""The largest row counts of the linear layers, without a GPU: rows that cannot be counted are refused as an
argument, whatever else the call holds, and need no workspace.  (The pointers below are never dereferenced:
each call also has a fault that the next check would report.)"""
import pytest

import self_attention_gb300 as sa
from self_attention_gb300.build import build

X, W, Y, Z = (0x10000000 * (i + 1) for i in range(4))
MOST = (1 << 31) - 256      # the row tiles of 256 end below 2^31


@pytest.fixture(scope="module")
def lib():
    return sa.load_library(build())


@pytest.mark.parametrize("M", [MOST + 1, (1 << 31) - 1])
def test_too_many_rows(lib, M):
    assert sa.attn_linear_bwd_workspace_size(M, 8, 8, 2) == 0
    assert sa.attn_linear_bwd_workspace_size(M, 8, 8, 0) == 0
    assert lib.attn_linear(X + 8, W, 0, 0, Y, 0, M, 8, 8, 0, None) == 1                     # not 3: misaligned
    assert lib.attn_linear_q8(X + 8, Z, W, Z, 0, 0, Y, M, 16, 8, 0, None) == 1
    assert lib.attn_linear_bwd(X, W, Y, Z, 0, 0, 0, 0, 0, M, 8, 8, 2, None) == 1            # not 6: no workspace
    assert lib.attn_out_proj(X + 8, W, 0, 0, Y, 1, 1, M, 64, 8, None) == 1
    assert sa.attn_out_proj_bwd_workspace_size(M, 1, 1, 64, 8) == 0


def test_the_most_rows(lib):
    assert sa.attn_linear_bwd_workspace_size(MOST, 8, 8, 2) >= MOST * 16
    assert sa.attn_linear_bwd_workspace_size(MOST, 8, 8, 0) > 0
    assert lib.attn_linear(X + 8, W, 0, 0, Y, 0, MOST, 8, 8, 0, None) == 3
    assert lib.attn_out_proj(X + 8, W, 0, 0, Y, 1, 1, MOST, 64, 8, None) == 3


@pytest.mark.parametrize("N,padded", [(2, 32), (31, 32), (33, 64)])
def test_short_sequences_count_whole_blocks(lib, N, padded):
    """Sequences of several heads are taken in blocks of 32 rows."""
    most = MOST // padded
    assert sa.attn_out_proj_bwd_workspace_size(most, 2, N, 64, 8) > 0
    assert lib.attn_out_proj(X + 8, W, 0, 0, Y, most, 2, N, 64, 8, None) == 3
    for B in (most + 1, most * 2):
        assert sa.attn_out_proj_bwd_workspace_size(B, 2, N, 64, 8) == 0
        assert lib.attn_out_proj(X + 8, W, 0, 0, Y, B, 2, N, 64, 8, None) == 1
        assert lib.attn_out_proj_bwd(X, W, Y, 0, 0, 0, 0, 0, B, 2, N, 64, 8, None) == 1
    # one token a sequence, or one head, is a plain matrix
    assert sa.attn_out_proj_bwd_workspace_size(most * 2, 2, 1, 64, 8) > 0
    assert (sa.attn_out_proj_bwd_workspace_size(most * 2, 1, N, 64, 8) > 0) == (most * 2 * N <= MOST)
