"""Attention over a paged cache where a result is easily wrong without looking wrong: queries that
are not finite, values of tiny scales. Tolerances as in test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from oracle import cache_ref as cref
from tests.test_gpu_paged import Setup, _close, _cu, _fill, _gen, _w, moba  # noqa: F401

pytestmark = pytest.mark.gpu

# lens, hq, hkv, d, page: how the rows of a segment come together
CUTS = [
    ([1000, 2], 8, 2, 128, 64),          # a cluster joins each segment
    ([30000, 0, 1], 4, 2, 64, 64),       # many warps share a segment, then the merge
    ([50, 60, 1, 70] * 60, 4, 2, 64, 16),  # mostly one warp per segment
]


def _positive_first(S, lens, seed=1):
    """Appends random rows whose keys have a positive first element; returns nothing."""
    g = _gen(seed)
    k = torch.randn((sum(lens), S.hkv, S.d), generator=g, device="cuda")
    k[..., 0] = k[..., 0].abs() + 0.5
    v = torch.randn((sum(lens), S.hkv, S.d), generator=g, device="cuda")
    S.moba.moba_cache_append(S.cache, k.bfloat16(), v.bfloat16(),
                             torch.tensor(_cu(lens), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("topk", [0, 3])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("cut", CUTS, ids=lambda c: f"{len(c[0])}x{max(c[0])}")
def test_a_query_that_is_not_finite_is_nan_in_its_row_alone(moba, cut, kv, topk):  # noqa: F811
    """A NaN, an infinity, and an infinity that makes every logit -inf: by the formula the row is
    NaN (o and lse), unless it has no position, then it has no keys and is 0, -inf; the other
    rows, of the same kv head too, are right."""
    lens, hq, hkv, d, page = cut
    rows, block = 2, 128
    S = Setup(moba, lens, hkv, d, page, kv, block)
    _positive_first(S, lens)
    n = len(lens) * rows
    q = torch.randn((n, hq, d), generator=_gen(7), device="cuda").bfloat16()
    clean = q.clone()
    bad = np.zeros((n, hq), bool)
    last = n - 1
    for at, h, x in ((1, 0, float("nan")), (1, hq - 1, float("inf")), (0, 1, float("-inf")),
                     (last, 2, float("nan")), (last - 1, 1, float("nan"))):
        q[at, h, 0] = x
        bad[at, h] = True
    if topk:
        o, lse = moba.moba_paged_decode_fwd(S.cache, q, topk, rows_per_seq=rows)
    else:
        o, lse = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=rows)
    kv_rows = [S.rows(s, x) for s, x in enumerate(lens)]
    sums = [cref.f64(S.sums[S.table[s, :-(-x // page):block // page].long()])
            for s, x in enumerate(lens)] if topk else None
    want = list(cref.cached_attention(clean, [x[0] for x in kv_rows], [x[1] for x in kv_rows],
                                      lens, rows, d ** -0.5, sums, block, topk))
    here = np.array([lens[i // rows] - rows + i % rows >= 0 for i in range(n)])
    for i, h in zip(*np.nonzero(bad)):
        if here[i]:
            assert o[i, h].isnan().all() and lse[h, i].isnan(), (i, h)
        else:
            assert not o[i, h].any() and torch.isneginf(lse[h, i]), (i, h)
    keep = torch.from_numpy(~bad).cuda()
    zero = lambda x, m: torch.where(m, x, torch.zeros_like(x))  # noqa: E731
    for x in (want[0], want[3]):
        x[bad] = 0
    want[1][bad.T] = 0
    _close(zero(o, keep[..., None]), zero(lse, keep.T), want, _w(kv))


@pytest.mark.parametrize("n", [40, 700, 20000])  # one warp's tile, a joined segment, a merged one
@pytest.mark.parametrize("exponent", [-121, -115, -100])
def test_values_of_tiny_scales(moba, n, exponent):  # noqa: F811
    """e4m3 values near 2^exponent: scale bytes down to 1. The output is a normal bf16 number."""
    hkv, d = 1, 64
    S = Setup(moba, [n], hkv, d, 16, "e4m3")
    g = _gen(17)
    k = torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16()
    v = (torch.randn((n, hkv, d), generator=g, device="cuda").sign()
         * (1 + torch.rand((n, hkv, d), generator=g, device="cuda"))).double()
    v = (v * 2.0 ** exponent).bfloat16()
    v[..., ::2] = v[..., ::2].abs()  # columns whose mean does not vanish
    moba.moba_cache_append(S.cache, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    q = torch.randn((1, 2, d), generator=g, device="cuda").bfloat16()
    kk, vv = S.rows(0, n)
    o, lse = moba.moba_paged_attn_fwd(S.cache, q)
    assert (o[..., ::2] > 2.0 ** (exponent - 1)).all()
    _close(o, lse, cref.cached_attention(q, [kk], [vv], [n], 1, d ** -0.5), _w("e4m3"))


def test_calls_without_the_native_binding(moba, monkeypatch):  # noqa: F811
    """The same bits where the arguments are marshalled in Python alone."""
    lens = [300, 70]
    g = _gen(5)
    q = torch.randn((2, 4, 64), generator=g, device="cuda").bfloat16()
    k = torch.randn((2, 2, 64), generator=g, device="cuda").bfloat16()
    w = torch.rand(64, generator=g, device="cuda") + 0.5
    rope, pos = moba.rope_table(400, 64), torch.tensor([299, 69], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def run():
        S = Setup(moba, lens, 2, 64, 16, "e4m3", 64)
        S.lens.sub_(1)
        _fill(S, [x - 1 for x in lens])
        S.lens.add_(1)
        y, yk = moba.moba_qk_norm_rope(q, k, w, w, rope, pos)
        grads = moba.moba_qk_norm_rope_bwd(q, k, w, w, rope, pos, y, yk)
        moba.moba_cache_append(S.cache, yk, yk, one)
        cu = _cu(lens)
        rows = moba.moba_cache_read(S.cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), cu)
        return (y, yk, *grads, *rows, *moba.moba_paged_attn_fwd(S.cache, y),
                *moba.moba_paged_decode_fwd(S.cache, y, 3))

    want = run()
    monkeypatch.setattr(moba, "_bind", None)
    assert all(torch.equal(a, b) for a, b in zip(run(), want))


@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_bf16_caches_keep_their_digits(moba, d):  # noqa: F811
    """Values whose weighted sum nearly vanishes, so that a weight's rounding shows: the weights enter
    the value product as two bf16 numbers, the second the first's rounding error (2^-8 of the weight)
    rounded again, which leaves 2^-16 of the weight."""
    lens, h = [2, 3, 5, 9, 17, 40, 700], 4
    S = Setup(moba, lens, h, d, 16, "bf16")
    g = _gen(23)
    T, cu = sum(lens), _cu(lens)
    k = torch.randn((T, h, d), generator=g, device="cuda").bfloat16()
    v = torch.randn((T, h, d), generator=g, device="cuda").bfloat16()
    q = torch.randn((len(lens), h, d), generator=g, device="cuda").bfloat16()
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        z = torch.einsum("uhd,hd->uh", k[a:b].double(), q[s].double()) * d ** -0.5
        p = torch.softmax(z, 0)
        top = p.argmax(0)  # the heaviest key's value cancels the others
        for x in range(h):
            u = a + int(top[x])
            rest = (p[:, x, None] * v[a:b, x].double()).sum(0) - p[top[x], x] * v[u, x].double()
            v[u, x] = (-rest / p[top[x], x]).bfloat16()
    moba.moba_cache_append(S.cache, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    o, lse = moba.moba_paged_attn_fwd(S.cache, q)
    rows = [S.rows(s, n) for s, n in enumerate(lens)]
    want = cref.cached_attention(q, [x[0] for x in rows], [x[1] for x in rows], lens, 1, d ** -0.5)
    _close(o, lse, want, 2.0 ** -16)


@pytest.mark.parametrize("topk", [0, 3])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,rows,width", [([1000], 1, 2048), ([5, 300, 0, 64], 2, 5000),
                                             ([2500] * 9, 1, 600), ([40, 1], 1, 60000)])
def test_page_tables_wider_than_the_sequences(moba, lens, rows, width, kv, topk):  # noqa: F811
    """A table for the longest context that a server allows, short sequences in it: the plan goes by
    the table's width, the results by the lengths."""
    hq, hkv, d, page, block = 8, 2, 64, 16, 64 if width < 30000 else 128
    S = Setup(moba, lens, hkv, d, page, kv, block)
    wide = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    wide[:, :S.table.shape[1]] = S.table
    S.table = wide
    S.cache = moba.PagedCache(S.k, S.v, wide, S.lens, S.ks, S.vs, S.sums, block)
    _fill(S, lens)
    n = len(lens) * rows
    q = torch.randn((n, hq, d), generator=_gen(9), device="cuda").bfloat16()
    idx = None
    if topk:
        idx = torch.empty((hq, n, topk), dtype=torch.int32, device="cuda")
        o, lse = moba.moba_paged_decode_fwd(S.cache, q, topk, rows_per_seq=rows, block_idx_out=idx)
    else:
        o, lse = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=rows)
    kv_rows = [S.rows(s, x) for s, x in enumerate(lens)]
    sums = [cref.f64(S.sums[S.table[s, :-(-x // page):block // page].long()])
            for s, x in enumerate(lens)] if topk else None
    want = cref.cached_attention(q, [x[0] for x in kv_rows], [x[1] for x in kv_rows], lens, rows,
                                 d ** -0.5, sums, block, topk)
    if topk:
        assert np.array_equal(idx.cpu().numpy(), want[2])
    _close(o, lse, want, _w(kv))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [40, 700, 20000])
def test_a_nan_key_is_nan_for_the_rows_that_see_it(moba, n, kv):  # noqa: F811
    """A token whose key is NaN (its position lay outside the rotary table) as the newest of three:
    NaN for its own row, nothing to the rows before it; as an older one: NaN for all of them."""
    hkv, hq, d, rows = 2, 4, 64, 3
    S = Setup(moba, [n, n], hkv, d, 16, kv)
    g = _gen(29)
    k = torch.randn((2 * n, hkv, d), generator=g, device="cuda").bfloat16()
    v = torch.randn((2 * n, hkv, d), generator=g, device="cuda").bfloat16()
    clean = k.clone()
    k[n - 1] = float("nan")          # newest of sequence 0
    k[n + n // 2, 0] = float("nan")  # one kv head of a token in the middle of sequence 1
    q = torch.randn((2 * rows, hq, d), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    moba.moba_cache_append(S.cache, clean, v, cu)
    want = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=rows)
    moba.moba_cache_append(S.cache, k, v, cu)
    o, lse = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=rows)
    bad = torch.zeros((2 * rows, hq), dtype=torch.bool, device="cuda")
    bad[rows - 1] = True
    bad[rows:, :hq // hkv] = True
    assert o[bad].isnan().all() and lse.T[bad].isnan().all()
    assert torch.equal(o[~bad], want[0][~bad]) and torch.equal(lse.T[~bad], want[1].T[~bad])
