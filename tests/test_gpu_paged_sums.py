"""The block sums of a paged cache where sequences share pages or are cut back, as include/moba.h says
how: pages, sums and routing as those of sequences that only ever had the rows that stayed."""
import pytest
import torch

from tests.test_gpu_paged import Setup, _check_pages, _check_sums, _cu, _gen, moba  # noqa: F401

pytestmark = pytest.mark.gpu


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("common", [128, 170])  # two whole blocks; ten pages and a block begun
def test_sequences_that_go_on_from_shared_pages(moba, kv, common):  # noqa: F811
    """A common prefix in shared pages, then rows of each sequence in one call. Where the prefix ends
    inside a block, the second sequence has a first page of that block (and its sum), and the page
    that the prefix ends in, of its own: copies."""
    hkv, d, page, block, more = 2, 64, 16, 64, [90, 150]
    lens = [common + m for m in more]
    S = Setup(moba, lens, hkv, d, page, kv, block)
    g = _gen(2)
    pk, pv = _randn(g, common, hkv, d), _randn(g, common, hkv, d)
    S.lens.copy_(_i32([common, 0]))
    moba.moba_cache_append(S.cache, pk, pv, _i32([0, common, common]))
    own = set()
    if common % page:
        own.add(common // page)
    if common % block:
        own.add(common // block * (block // page))
    for x in range(-(-common // page)):
        a, b = int(S.table[0, x]), int(S.table[1, x])
        if x in own:
            for t in (S.k, S.v, S.ks, S.vs, S.sums):
                if t is not None:
                    t.view(torch.uint8)[b].copy_(t.view(torch.uint8)[a])
        else:
            S.table[1, x] = a
    mk, mv = _randn(g, sum(more), hkv, d), _randn(g, sum(more), hkv, d)
    S.lens.copy_(_i32(lens))
    moba.moba_cache_append(S.cache, mk, mv, _i32(_cu(more)))
    k = torch.cat([pk, mk[:more[0]], pk, mk[more[0]:]])
    v = torch.cat([pv, mv[:more[0]], pv, mv[more[0]:]])
    _check_pages(S, lens, k, v)
    _check_sums(S, lens, k)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("start,accepted", [([100, 127, 64], [2, 0, 1]), ([126, 200, 191], [5, 3, 0])])
def test_rejected_draft_rows_taken_back(moba, kv, start, accepted):  # noqa: F811
    """Draft rows over block borders, some of them accepted: the sums of the blocks that the sequences
    ended in are kept before and put back, and the accepted rows written again. Pages, sums and the
    routing have the bits of a cache that only had the accepted rows."""
    hkv, hq, d, page, block, draft, more = 2, 4, 64, 16, 64, 5, 70
    n = len(start)
    top = [x + draft + more for x in start]
    S = Setup(moba, top, hkv, d, page, kv, block, seed=1)
    E = Setup(moba, top, hkv, d, page, kv, block, seed=1)
    g = _gen(4)
    k, v = _randn(g, sum(start), hkv, d), _randn(g, sum(start), hkv, d)
    dk, dv = _randn(g, n * draft, hkv, d), _randn(g, n * draft, hkv, d)
    for X in (S, E):
        X.lens.copy_(_i32(start))
        moba.moba_cache_append(X.cache, k, v, _i32(_cu(start)))
    # the page in which each sequence's last block begins
    home = S.table[torch.arange(n), S.lens.long() // block * (block // page)].long()
    kept = S.sums[home]
    S.lens.add_(draft)
    moba.moba_cache_append(S.cache, dk, dv, _i32([draft * s for s in range(n + 1)]))
    rows = torch.cat([draft * s + torch.arange(a) for s, a in enumerate(accepted)]).cuda()
    final = _i32([a + b for a, b in zip(start, accepted)])
    S.sums[home] = kept
    for X in (S, E):
        X.lens.copy_(final)
        moba.moba_cache_append(X.cache, dk[rows], dv[rows], _i32(_cu(accepted)))
    nk = torch.cat([torch.cat([k[a:b], dk[draft * s:draft * s + x]]) for s, (a, b, x) in enumerate(
        zip(_cu(start), _cu(start)[1:], accepted))])
    nv = torch.cat([torch.cat([v[a:b], dv[draft * s:draft * s + x]]) for s, (a, b, x) in enumerate(
        zip(_cu(start), _cu(start)[1:], accepted))])
    lens = final.tolist()
    _check_pages(S, lens, nk, nv)
    _check_sums(S, lens, nk)
    for s, x in enumerate(lens):
        used = S.table[s, :-(-x // page):block // page].long()
        assert torch.equal(S.sums[used], E.sums[used])
    # and the routing over those blocks, once the sequences are past them
    mk, mv = _randn(g, n * more, hkv, d), _randn(g, n * more, hkv, d)
    q = _randn(g, n, hq, d)
    idx = torch.empty((2, hq, n, 3), dtype=torch.int32, device="cuda")
    got = []
    for X, at in zip((S, E), idx):
        X.lens.add_(more)
        moba.moba_cache_append(X.cache, mk, mv, _i32([more * s for s in range(n + 1)]))
        got.append(moba.moba_paged_decode_fwd(X.cache, q, 3, block_idx_out=at))
    assert torch.equal(idx[0], idx[1])
    assert all(torch.equal(a, b) for a, b in zip(*got))
