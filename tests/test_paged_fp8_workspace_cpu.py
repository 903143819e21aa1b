"""Workspace of fa2_paged_fwd_fp8 where the number of CTAs changes: two to each of
152 SMs with up to eight query rows a tile, one with more, and one at head dim
256 and for sequences of several query tiles.  Two fp32 states (O, and m with l)
for each CTA and row of a tile, and 32 bytes for each CTA's merge."""
import ctypes

import pytest

from test_paged_fp8_cpu import _fwd, lib  # noqa: F401 (a fixture)


def need(ctas, rows, d):
    up = lambda x: (x + 255) // 256 * 256
    return up(2 * ctas * rows * d * 4) + up(2 * ctas * rows * 2 * 4) + up(ctas * 32)


@pytest.mark.parametrize("heads,tokens,d,ctas", [
    (1, 1, 64, 304), (7, 1, 64, 304), (8, 1, 64, 304), (4, 2, 128, 304), (8, 1, 256, 152), (9, 1, 64, 152), (3, 3, 128, 152),
    (16, 1, 64, 152), (8, 2, 128, 152), (17, 1, 128, 152), (32, 1, 64, 152), (8, 4, 64, 152)])
def test_rows_of_a_tile(lib, heads, tokens, d, ctas):  # noqa: F811
    size = lib.fa2_paged_fwd_fp8_workspace_bytes(ctypes.byref(_fwd(
        cache_heads=1, heads=heads, cache_head_dim=d, total_q=3 * tokens, max_seqlen_q=tokens)))
    assert size == need(ctas, heads * tokens, d)


@pytest.mark.parametrize("heads,tokens", [(8, 5), (1, 33), (1, 200), (9, 4)])
def test_several_query_tiles_a_sequence(lib, heads, tokens):  # noqa: F811
    size = lib.fa2_paged_fwd_fp8_workspace_bytes(ctypes.byref(_fwd(
        cache_heads=1, heads=heads, cache_head_dim=64, total_q=3 * tokens, max_seqlen_q=tokens)))
    assert size == need(152, 32 // heads * heads, 64)
