"""The block sums of a paged cache where sequences share pages, as include/moba.h says how: pages and
sums as those of sequences on their own."""
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
