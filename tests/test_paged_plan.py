"""Which plan the attention over a paged cache takes, seen in the workspace that it asks for: partials in
the workspace where segments are spread over the grid, none where clusters join them (CPU)."""
import ctypes

import pytest

from tests.test_cache_args import _struct, lib  # noqa: F401


def _bytes(lib, nseq, pages, page_size=64, hq=8, hkv=1, topk=0, **kw):  # noqa: F811
    c = _struct(nseq=nseq, max_pages=pages, num_pages=100, page_size=page_size, Hkv=hkv, **kw)
    return lib.moba_paged_workspace_bytes(ctypes.addressof(c), hq, 1, topk)


@pytest.mark.parametrize("nseq,joined", [(8, True), (14, True), (15, False), (16, False),
                                         (18, False)])
def test_clusters_of_eight_join_only_while_all_run_at_once(lib, nseq, joined):  # noqa: F811
    """4096 tokens in 128 tiles, eight segments or more: a join with eight CTAs to a segment, 4 tiles a
    warp, is within the margin of 3 of the tiles spread, 1.7 or more; with four CTAs, 8 tiles, it is
    not. A B200 runs 15 such clusters at once
    (fewer where its groups of SMs are smaller); a sixteenth would wait for another to end."""
    n = _bytes(lib, nseq, 64)
    assert (n <= 4096) if joined else (n > 1 << 20), n


def test_a_wide_table_is_spread(lib):  # noqa: F811
    assert _bytes(lib, 1, 16) <= 4096 and _bytes(lib, 1, 2048) > 1 << 20
