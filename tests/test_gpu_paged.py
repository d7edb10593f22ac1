"""The paged cache and the attention over it on the GPU against the fp64 reference.

Tolerances. Codes, scale bytes, page contents and routings are exact. Block sums: fp32 sums of n
bf16 keys, n 2^-24 sum |k|. Attention, per row: the weights enter the value product rounded to
bf16 (2^-8 relative; over an e4m3 cache to f16, 2^-11), the logits are fp32 tensor-core sums of d
exact products (each addition within 2^-22 of the terms' absolute sum, which truncating additions
inside one instruction allow: d 2^-22 sum |q k| scale, `dz` below), the sum of weights and the
join of partials add fp32 roundings (2^-16 together, chains are below 256 long), and o is rounded
once to bf16. So
  |o - ref| <= (w + 2 dz + 2^-15) sum p |v| + 2^-8 |ref|,   |lse - ref| <= dz + 2^-15 (1 + |ref|).
"""
import numpy as np
import pytest
import torch

from oracle import cache_ref as cref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moba():
    from block_sparse_long_moba_b200 import build, moba as m
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.load_library()
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Setup:
    """A pool full of NaN, pages handed out in a random order, -1 in unused table entries."""

    def __init__(self, moba, lens, hkv, d, page, kv, block=None, spare=3, seed=0, room=0):
        self.moba, self.hkv, self.d, self.page, self.block = moba, hkv, d, page, block
        g = _gen(seed)
        need = [-(-x // page) for x in lens]
        self.pool = sum(need) + spare + room * len(lens)
        perm = torch.randperm(self.pool, generator=g, device="cuda").to(torch.int32)
        width = max(1, max(need) + room)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n + room] = perm[at:at + n + room].cpu()
            at += n + room
        self.table = table.cuda()
        kind = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
        shape = (self.pool, hkv, page, d)
        nan = torch.full(shape, float("nan"), device="cuda").to(kind)
        self.k, self.v = nan, nan.clone()
        self.ks = self.vs = None
        if kv != "bf16":
            self.ks = torch.full(shape[:3], 255, dtype=torch.uint8, device="cuda")
            self.vs = self.ks.clone()
        self.sums = torch.full((self.pool, hkv, d), float("nan"), device="cuda") if block else None
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cache = moba.PagedCache(self.k, self.v, self.table, self.lens, self.ks, self.vs,
                                     self.sums, block)

    def rows(self, s, n):
        """Cached (k, v) of the first n tokens of sequence s in fp64 [n, hkv, d]."""
        ids = self.table[s, :-(-n // self.page)].long()
        out = []
        for x, sc in ((self.k, self.ks), (self.v, self.vs)):
            if sc is None:
                y = cref.f64(x[ids])
            else:
                y = cref.dequantise(x.view(torch.uint8)[ids].cpu().numpy(), sc[ids].cpu().numpy())
            out.append(y.transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.d)[:n])
        return out


def _cu(counts):
    return [0] + list(np.cumsum(counts))


def _fill(S, lens, seed=1, scale=1.0, fused=False):
    """Appends whole sequences in one call; returns k, v."""
    g = _gen(seed)
    T = sum(lens)
    x = torch.randn((T, 2 * S.hkv * S.d + (16 if fused else 0)), generator=g, device="cuda") * scale
    x = x.bfloat16()
    w = S.hkv * S.d
    k, v = (x[:, a:a + w].unflatten(1, (S.hkv, S.d)) for a in (0, w))
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    if S.block:  # give the block scores something to find
        k = k.clone()
        at = 0
        for n in lens:
            for j in range(0, n, S.block):
                k[at + j:at + min(n, j + S.block)] += 0.7 * torch.randn(
                    (1, S.hkv, S.d), generator=g, device="cuda").bfloat16()
            at += n
    cu = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
    S.moba.moba_cache_append(S.cache, k, v, cu)
    return k, v


# ------------------------------------------------------------------------------------- append
APPEND = [  # lens, hkv, d, page, kv, block, fused
    ([1], 8, 128, 64, "e4m3", 4096, True),
    ([300, 1, 0, 77, 1000], 8, 128, 64, "e4m3", 128, True),
    ([300, 1, 0, 77, 1000], 2, 64, 16, "bf16", 64, False),
    ([5000, 12000], 3, 64, 32, "e4m3", 4096, False),
    ([4096, 8193], 16, 64, 128, "bf16", 4096, True),
    ([700] * 9, 1, 128, 16, "e4m3", 192, False),
    ([65, 63], 20, 128, 32, "bf16", None, True),
    ([40000], 4, 128, 256, "e4m3", 512, False),
]


def _check_pages(S, lens, k, v):
    cu = _cu(lens)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        ids = S.table[s, :-(-n // S.page)].long()
        for x, cache, sc in ((k, S.k, S.ks), (v, S.v, S.vs)):
            want = x[cu[s]:cu[s + 1]]
            if sc is None:
                got = cache[ids].transpose(1, 2).flatten(0, 1)[:n]
                assert torch.equal(got, want)
            else:
                codes, b = cref.quantise(want)
                got = cache.view(torch.uint8)[ids].transpose(1, 2).flatten(0, 1)[:n]
                assert np.array_equal(got.cpu().numpy(), codes)
                assert np.array_equal(sc[ids].transpose(1, 2).flatten(0, 1)[:n].cpu().numpy(), b)


def _check_sums(S, lens, k):
    if not S.block:
        return
    cu, per = _cu(lens), S.block // S.page
    kk = cref.f64(k)
    for s, n in enumerate(lens):
        for j in range(0, -(-n // S.block)):
            x = kk[cu[s] + j * S.block:cu[s] + min(n, (j + 1) * S.block)]
            got = cref.f64(S.sums[int(S.table[s, j * per])])
            assert (np.abs(got - x.sum(0)) <= (len(x) + 2) * 2.0 ** -24 * np.abs(x).sum(0)).all()


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append_whole_sequences(moba, case):
    lens, hkv, d, page, kv, block, fused = case
    S = Setup(moba, lens, hkv, d, page, kv, block)
    k, v = _fill(S, lens, fused=fused)
    _check_pages(S, lens, k, v)
    _check_sums(S, lens, k)
    # pages of nobody are as they were
    used = set(S.table[S.table >= 0].tolist())
    for p in range(S.pool):
        if p not in used:
            assert S.k[p].float().isnan().all() and S.v[p].float().isnan().all()
    # and so are the slots behind each sequence's last token
    for s, n in enumerate(lens):
        if n % page:
            p = int(S.table[s, n // page])
            assert S.k[p, :, n % page:].float().isnan().all()
    b0 = None if S.sums is None else S.sums.clone()
    _fill(S, lens, fused=fused)  # the same bits every time
    if b0 is not None:
        assert torch.equal(b0.nan_to_num(1.5), S.sums.nan_to_num(1.5))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_in_steps(moba, kv):
    """A prompt, a chunk over a block border, then single tokens: pages and sums as if the rows
    had come at once; a sequence without new rows is left alone."""
    final, hkv, d, page, block = [150, 64, 500], 4, 128, 16, 128
    S = Setup(moba, final, hkv, d, page, kv, block)
    g = _gen(3)
    k = torch.randn((sum(final), hkv, d), generator=g, device="cuda").bfloat16()
    v = torch.randn((sum(final), hkv, d), generator=g, device="cuda").bfloat16()
    cu = _cu(final)
    at = [0, 0, 0]
    for step in ([100, 0, 127], [49, 63, 2], [1, 1, 0], [0, 0, 371]):
        part = [torch.arange(cu[s] + at[s], cu[s] + at[s] + n, device="cuda")
                for s, n in enumerate(step)]
        rows = torch.cat(part)
        at = [a + n for a, n in zip(at, step)]
        S.lens.copy_(torch.tensor(at, dtype=torch.int32))
        moba.moba_cache_append(S.cache, k[rows], v[rows],
                               torch.tensor(_cu(step), dtype=torch.int32, device="cuda"))
    assert at == final
    _check_pages(S, final, k, v)
    _check_sums(S, final, k)


def test_append_extreme_rows(moba):
    """Rows of zeros, of one value at the e4m3 border, of subnormal and of huge values."""
    S = Setup(moba, [8], 1, 64, 16, "e4m3")
    k = torch.zeros((8, 1, 64), device="cuda").bfloat16()
    k[1, 0, 3] = 448.0
    k[2, 0, 3] = -450.0
    k[3] = torch.randn((1, 64), device="cuda").bfloat16() * 2.0 ** -130
    k[4] = torch.randn((1, 64), device="cuda").bfloat16() * 2.0 ** 120
    k[5] = torch.tensor(torch.finfo(torch.bfloat16).max)
    k[6, 0, ::2] = -0.0
    k[7] = torch.exp2(-torch.arange(64, device="cuda").float()).bfloat16()
    moba.moba_cache_append(S.cache, k, -k, torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    _check_pages(S, [8], k, -k)


def test_append_never_leaves_its_pages(moba):
    """Pages outside the pool, positions before zero and behind the table, more rows announced
    than given: those rows are dropped, the others are written."""
    S = Setup(moba, [40, 40], 2, 64, 16, "bf16", 64)
    g = _gen(0)
    k = torch.randn((80, 2, 64), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda")
    bad = S.table.clone()
    bad[0, 1], bad[1, 0] = S.pool, -7
    cache = moba.PagedCache(S.k, S.v, bad, S.lens, block_sums=S.sums, block_size=64)
    moba.moba_cache_append(cache, k, k, cu)
    assert torch.equal(S.k[int(S.table[0, 0])].transpose(0, 1), k[:16])
    assert S.k[int(S.table[0, 1])].isnan().all()
    assert torch.equal(S.k[int(S.table[0, 2])].transpose(0, 1)[:8], k[32:40])
    assert S.k[int(S.table[1, 0])].isnan().all()
    assert torch.equal(S.k[int(S.table[1, 1])].transpose(0, 1), k[56:72])
    assert S.sums[int(S.table[1, 0])].isnan().all()  # no home for that block's sum
    # 40 rows for a sequence of 30 tokens: the first ten have no position
    T = Setup(moba, [30, 40], 2, 64, 16, "bf16", 64)
    moba.moba_cache_append(T.cache, k, k, cu)
    assert torch.equal(T.k[int(T.table[0, 0])].transpose(0, 1), k[10:26])
    # behind the table: a length that its pages cannot hold
    T.lens[0] = 1000
    T.k.fill_(0)
    moba.moba_cache_append(T.cache, k, k, cu)
    assert not T.k[T.table[0, :2].long()].any()
    # offsets that do not fit the rows given
    T.k.fill_(0)
    T.lens[0] = 30
    moba.moba_cache_append(T.cache, k[:50], k[:50], cu)
    assert not T.k[T.table[1][T.table[1] >= 0].long()].any()
    torch.cuda.synchronize()


# --------------------------------------------------------------------------------------- read
@pytest.mark.parametrize("kv,d,hkv,page", [("bf16", 64, 3, 16), ("e4m3", 64, 16, 32),
                                           ("bf16", 128, 8, 128), ("e4m3", 128, 2, 64)])
def test_read_back(moba, kv, d, hkv, page):
    lens = [0, 1, 1000, 0, 63, 2500]
    S = Setup(moba, lens, hkv, d, page, kv)
    k, v = _fill(S, lens, scale=3.0)
    cu = _cu(lens)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = [torch.full((cu[-1] + 5, hkv, d), 9.0, device="cuda").bfloat16() for _ in range(2)]
    gk, gv = moba.moba_cache_read(S.cache, cu_t, cu, k=out[0][:cu[-1]], v=out[1][:cu[-1]])
    for s, n in enumerate(lens):
        wk, wv = S.rows(s, n) if n else (0, 0)
        assert np.array_equal(cref.f64(gk[cu[s]:cu[s + 1]]), wk if n else np.zeros((0, hkv, d)))
        assert np.array_equal(cref.f64(gv[cu[s]:cu[s + 1]]), wv if n else np.zeros((0, hkv, d)))
    assert (out[0][cu[-1]:] == 9.0).all() and (out[1][cu[-1]:] == 9.0).all()
    if kv == "bf16":
        assert torch.equal(gk, k) and torch.equal(gv, v)


def test_read_behind_a_sequence_and_bad_pages(moba):
    S = Setup(moba, [20, 40], 2, 64, 16, "e4m3")
    k, v = _fill(S, [20, 40])
    bad = S.table.clone()
    bad[1, 1] = S.pool + 3
    cache = moba.PagedCache(S.k, S.v, bad, S.lens, S.ks, S.vs)
    cu = [0, 30, 100]
    gk, gv = moba.moba_cache_read(cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), cu)
    for x in (gk, gv):
        assert not x[20:30].any() and not x[70:].any()
        assert x[46:62].isnan().all() and not x[:20].isnan().any() and not x[30:46].isnan().any()


# ---------------------------------------------------------------------------------- attention
def _close(o, lse, want, w):
    o_ref, lse_ref, _, spread, dot = want
    d = o_ref.shape[-1]
    o, lse = cref.f64(o), cref.f64(lse)
    dz = d * 2.0 ** -22 * dot
    gone = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), gone)
    err = np.abs(np.where(gone, 0, lse - np.where(gone, 0, lse_ref)))
    assert (err <= np.where(gone, 1, dz + 2.0 ** -15 * (1 + np.abs(lse_ref)))).all(), err.max()
    bound = (w + 2 * dz.T[..., None] + 2.0 ** -15) * spread + 2.0 ** -8 * np.abs(o_ref)
    assert (np.abs(o - o_ref) <= bound).all(), float((np.abs(o - o_ref) - bound).max())


def _w(kv):
    return 2.0 ** -8 if kv == "bf16" else 2.0 ** -11


DENSE = [  # lens, rows, hq, hkv, d, page, kv
    ([1], 1, 1, 1, 64, 16, "bf16"),
    ([1000], 1, 32, 8, 128, 64, "bf16"),
    ([1000], 1, 32, 8, 128, 64, "e4m3"),
    ([0, 1, 15, 16, 17, 31, 33, 64, 129, 3000], 1, 8, 2, 128, 16, "bf16"),
    ([0, 1, 15, 16, 17, 31, 33, 64, 129, 3000], 1, 8, 2, 128, 16, "e4m3"),
    ([0, 1, 15, 16, 17, 31, 33, 64, 129, 3000], 1, 4, 4, 64, 32, "bf16"),
    ([0, 1, 15, 16, 17, 31, 33, 64, 129, 3000], 1, 4, 4, 64, 16, "e4m3"),
    ([5, 2, 300, 0, 4], 4, 4, 2, 64, 128, "bf16"),    # rows without a position
    ([5, 2, 300, 0, 4], 4, 6, 2, 128, 16, "e4m3"),    # 12 rows a kv head
    ([257, 600], 3, 40, 2, 128, 64, "bf16"),          # 60 rows a kv head: four row tiles
    ([257, 600], 2, 33, 1, 64, 64, "e4m3"),           # 66 rows: five
    ([20000, 3], 1, 4, 1, 128, 256, "bf16"),          # one long sequence over many warps
    ([50, 60, 70] * 70, 1, 4, 2, 64, 16, "bf16"),     # more segments than warps share evenly
    ([500, 7, 470, 512] * 4, 1, 32, 8, 128, 64, "e4m3"),  # a CTA per segment
    ([500, 7, 470, 512] * 4, 1, 32, 8, 128, 32, "bf16"),
    ([9000, 100], 4, 16, 2, 64, 64, "e4m3"),          # 32 rows a kv head over many warps
    ([9000, 100], 4, 8, 2, 128, 64, "bf16"),          # 16 rows a kv head over many warps
    ([17] * 900, 1, 2, 2, 64, 16, "e4m3"),            # many one-tile segments
]


@pytest.mark.parametrize("case", DENSE, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1:]}")
def test_dense_attention(moba, case):
    lens, rows, hq, hkv, d, page, kv = case
    S = Setup(moba, lens, hkv, d, page, kv)
    _fill(S, lens)
    q = torch.randn((len(lens) * rows, hq, d), generator=_gen(7), device="cuda").bfloat16()
    o, lse = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=rows)
    kv_rows = [S.rows(s, n) for s, n in enumerate(lens)]
    want = cref.cached_attention(q, [x[0] for x in kv_rows], [x[1] for x in kv_rows], lens, rows,
                                 d ** -0.5)
    _close(o, lse, want, _w(kv))
    again = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=rows)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_sharp_and_spread_out_logits(moba, kv):
    """Logits from -300 to 300 in an order that keeps raising the maximum, keys and values whose
    scales differ by 2^40 between tokens, and a scale of the logits other than 1 / sqrt(d)."""
    lens, hq, hkv, d = [700, 90], 4, 2, 64
    S = Setup(moba, lens, hkv, d, 32, kv)
    g = _gen(11)
    T = sum(lens)
    k = torch.randn((T, hkv, d), generator=g, device="cuda") * torch.linspace(
        0.01, 8, T, device="cuda")[:, None, None]
    v = torch.randn((T, hkv, d), generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (T, 1, 1), generator=g, device="cuda").float())
    k, v = k.bfloat16(), v.bfloat16()
    moba.moba_cache_append(S.cache, k, v,
                           torch.tensor(_cu(lens), dtype=torch.int32, device="cuda"))
    q = (4 * torch.randn((2, hq, d), generator=g, device="cuda")).bfloat16()
    q[1] *= 2.0 ** -30  # all weights alike
    kv_rows = [S.rows(s, n) for s, n in enumerate(lens)]
    o, lse = moba.moba_paged_attn_fwd(S.cache, q, scale=0.3)
    want = cref.cached_attention(q, [x[0] for x in kv_rows], [x[1] for x in kv_rows], lens, 1, 0.3)
    _close(o, lse, want, _w(kv))


def test_values_of_far_apart_scales(moba):
    """e4m3: values 2^60 apart. A tiny weight on a huge value and a weight near one on small values
    both count: o is the sum of the two, and a row that cannot see the huge value is exact without
    it (the first of two rows)."""
    n, d = 200, 64
    S = Setup(moba, [n], 1, d, 16, "e4m3")
    g = _gen(13)
    k = torch.randn((n, 1, d), generator=g, device="cuda").bfloat16()
    v = torch.randn((n, 1, d), generator=g, device="cuda").bfloat16()
    v[n - 1] *= 2.0 ** 60
    k[n - 1] = 0
    k[n - 1, 0, 0] = -60.0
    q = torch.randn((2, 1, d), generator=g, device="cuda").bfloat16()
    q[:, 0, 0] = 1.0  # logit -60 in units of log e: a weight of about 2^-87 against 200 others
    moba.moba_cache_append(S.cache, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    kk, vv = S.rows(0, n)
    for scale in (0.5, 0.69, 1.0):
        o, lse = moba.moba_paged_attn_fwd(S.cache, q, rows_per_seq=2, scale=scale)
        want = cref.cached_attention(q, [kk], [vv], [n], 2, scale)
        _close(o, lse, want, _w("e4m3"))


def test_sequences_that_share_their_first_pages(moba):
    """Two sequences with the same full pages for a common prefix, read by both at once."""
    hkv, d, page, block, common = 2, 64, 16, 64, 128
    S = Setup(moba, [200, 300], hkv, d, page, "bf16", block)
    k, v = _fill(S, [200, 300])
    shared = S.table.clone()
    shared[0, :common // page] = shared[1, :common // page]
    cache = moba.PagedCache(S.k, S.v, shared, S.lens, block_sums=S.sums, block_size=block)
    S.table = shared
    q = torch.randn((2, 4, d), generator=_gen(3), device="cuda").bfloat16()
    rows = [S.rows(0, 200), S.rows(1, 300)]
    assert np.array_equal(rows[0][0][:common], rows[1][0][:common])
    sums = [cref.f64(S.sums[shared[s, :-(-x // page):4].long()]) for s, x in enumerate((200, 300))]
    ks, vs = [x[0] for x in rows], [x[1] for x in rows]
    o, lse = moba.moba_paged_attn_fwd(cache, q)
    _close(o, lse, cref.cached_attention(q, ks, vs, [200, 300], 1, d ** -0.5), _w("bf16"))
    o, lse = moba.moba_paged_decode_fwd(cache, q, 2)
    _close(o, lse, cref.cached_attention(q, ks, vs, [200, 300], 1, d ** -0.5, sums, block, 2),
           _w("bf16"))


MOBA = [  # lens, rows, hq, hkv, d, page, block, topk, kv
    ([1000], 1, 4, 2, 128, 64, 128, 3, "bf16"),
    ([0, 1, 127, 128, 129, 3000], 1, 8, 2, 128, 16, 128, 4, "e4m3"),
    ([0, 1, 63, 64, 65, 3000], 1, 4, 4, 64, 32, 64, 5, "bf16"),
    ([9000, 4097], 1, 8, 2, 128, 64, 512, 3, "bf16"),
    ([2000, 130], 4, 4, 2, 64, 16, 128, 4, "bf16"),         # rows on both sides of a border
    ([2000, 130, 2], 4, 8, 1, 128, 16, 64, 6, "e4m3"),      # 32 rows: two row tiles
    ([5000], 1, 4, 1, 64, 64, 192, 1, "e4m3"),              # the current block alone
    ([5000, 700], 1, 2, 2, 64, 64, 192, 64, "bf16"),        # more than there are blocks
    ([40000, 33000], 1, 2, 1, 64, 64, 64, 16, "e4m3"),      # 625 blocks: eight CTAs score them
    ([150000], 1, 1, 1, 64, 64, 64, 33, "bf16"),            # 2344 blocks
    ([30000], 3, 48, 2, 128, 128, 128, 7, "bf16"),          # 72 rows: five row tiles
    ([2500] * 40, 1, 8, 8, 64, 16, 128, 5, "e4m3"),
]


@pytest.mark.parametrize("case", MOBA, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1:]}")
def test_moba_attention(moba, case):
    lens, rows, hq, hkv, d, page, block, topk, kv = case
    S = Setup(moba, lens, hkv, d, page, kv, block)
    _fill(S, lens)
    n = len(lens) * rows
    q = torch.randn((n, hq, d), generator=_gen(8), device="cuda").bfloat16()
    idx = torch.full((hq, n, topk), 77, dtype=torch.int32, device="cuda")
    o, lse = moba.moba_paged_decode_fwd(S.cache, q, topk, rows_per_seq=rows, block_idx_out=idx)
    kv_rows = [S.rows(s, x) for s, x in enumerate(lens)]
    per = block // page
    sums = [cref.f64(S.sums[S.table[s, :-(-x // page):per].long()]) for s, x in enumerate(lens)]
    want = cref.cached_attention(q, [x[0] for x in kv_rows], [x[1] for x in kv_rows], lens, rows,
                                 d ** -0.5, sums, block, topk)
    assert np.array_equal(idx.cpu().numpy(), want[2])
    _close(o, lse, want, _w(kv))
    again = moba.moba_paged_decode_fwd(S.cache, q, topk, rows_per_seq=rows)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_equal_scores_go_to_the_lower_block(moba):
    """Blocks of the same keys, a zero query (every score +-0) and NaN sums behind every number."""
    B, n = 64, 640
    S = Setup(moba, [n, n], 1, 64, 64, "bf16", B)
    _fill(S, [n, n])
    S.sums[S.table[0].long()] = torch.randn(64, device="cuda")
    S.sums[S.table[0, 7].long()] = float("nan")
    S.sums[S.table[1].long()] *= -1
    q = torch.randn((2, 2, 64), device="cuda").bfloat16()
    q[1] = 0
    idx = torch.empty((2, 2, 4), dtype=torch.int32, device="cuda")
    moba.moba_paged_decode_fwd(S.cache, q, 4, block_idx_out=idx)
    assert idx.tolist() == [[[0, 1, 2, 9]] * 2] * 2
    S.sums[S.table[0, :6].long()] = float("nan")  # two numbers left for four places
    idx5 = torch.empty((2, 2, 5), dtype=torch.int32, device="cuda")
    moba.moba_paged_decode_fwd(S.cache, q, 5, block_idx_out=idx5)
    assert idx5[:, 0].tolist() == [[0, 1, 6, 8, 9]] * 2


def test_bad_pages_and_lengths_are_that_sequences_nan(moba):
    lens = [300, 300, 300, 300]
    S = Setup(moba, lens, 2, 64, 16, "e4m3", 64)
    _fill(S, lens)
    q = torch.randn((4, 4, 64), device="cuda").bfloat16()
    k0, v0 = S.rows(0, 300)
    sums = cref.f64(S.sums[S.table[0, ::4].long()])
    fine = cref.cached_attention(q[:1], [k0], [v0], [300], 1, 0.125)
    fine_moba = cref.cached_attention(q[:1], [k0], [v0], [300], 1, 0.125, [sums], 64, 3)
    bad = S.table.clone()
    bad[1, 4] = S.pool          # the first page of a past block: its sum and its rows
    bad[2, 18] = -1             # the page that the newest token is in
    lens2 = S.lens.clone()
    lens2[3] = 16 * bad.shape[1] + 1
    cache = moba.PagedCache(S.k, S.v, bad, lens2, S.ks, S.vs, S.sums, 64)
    for got, want in ((moba.moba_paged_attn_fwd(cache, q), fine),
                      (moba.moba_paged_decode_fwd(cache, q, 3), fine_moba)):
        assert got[0][1:].isnan().all() and got[1][:, 1:].isnan().all()
        _close(got[0][:1], got[1][:, :1], want, _w("e4m3"))
    lens2[:] = torch.tensor([-5, 0, 300, 300])
    o, lse = moba.moba_paged_attn_fwd(cache, q)
    assert not o[:2].any() and torch.isneginf(lse[:, :2]).all()


def test_offsets_beyond_32_bits(moba):
    """A pool of more than 2^31 values a tensor, the sequence in its last pages."""
    hkv, d, page, n = 8, 128, 64, 3000
    pages = -(-n // page)
    pool = (1 << 31) // (hkv * page * d) + 200
    k = torch.zeros((pool, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    sums = torch.zeros((pool, hkv, d), device="cuda")
    table = (pool - 1 - torch.arange(pages, device="cuda")).to(torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cache = moba.PagedCache(k, v, table, lens, block_sums=sums, block_size=128)
    g = _gen(1)
    kk = torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16()
    vv = torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    moba.moba_cache_append(cache, kk, vv, cu)
    gk, gv = moba.moba_cache_read(cache, cu, [0, n])
    assert torch.equal(gk, kk) and torch.equal(gv, vv)
    q = torch.randn((1, 16, d), generator=g, device="cuda").bfloat16()
    o, lse = moba.moba_paged_attn_fwd(cache, q)
    want = cref.cached_attention(q, [cref.f64(kk)], [cref.f64(vv)], [n], 1, d ** -0.5)
    _close(o, lse, want, 2.0 ** -8)
    assert not k[0].any()


def test_two_streams_at_once(moba):
    """Two calls with workspaces of their own, in flight at the same time on two streams."""
    lens = [3000, 500, 1200]
    S = Setup(moba, lens, 4, 128, 64, "bf16", 128)
    _fill(S, lens)
    q = torch.randn((2, 3, 8, 128), generator=_gen(5), device="cuda").bfloat16()
    want = [moba.moba_paged_decode_fwd(S.cache, q[i], 4) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(moba.moba_paged_decode_fwd(S.cache, q[i], 4, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_a_captured_step_follows_the_cache(moba):
    """norm + rotary, append and both attentions captured once; replayed while lengths, page
    table and inputs change, each replay against the eager calls on a cache of its own."""
    final, hkv, hq, d, page, block = [400, 150], 2, 8, 64, 16, 64
    S = Setup(moba, final, hkv, d, page, "e4m3", block, seed=2)
    E = Setup(moba, final, hkv, d, page, "e4m3", block, seed=3)
    start = [380, 120]
    for X in (S, E):
        X.lens.copy_(torch.tensor(start, dtype=torch.int32))
        _fill(X, start)
    qkv = torch.randn((2, (hq + 2 * hkv) * d), device="cuda").bfloat16()
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    wq, wk = torch.rand(d, device="cuda") + 0.5, torch.rand(d, device="cuda") + 0.5
    rope = moba.rope_table(1000, d)
    pos = torch.tensor(start, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def step(X):
        X.lens.add_(1)
        yq, yk = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos)
        moba.moba_cache_append(X.cache, yk, v, cu)
        return moba.moba_paged_attn_fwd(X.cache, yq) + moba.moba_paged_decode_fwd(X.cache, yq, 3)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(S)
    for i in range(20):
        qkv.normal_()
        graph.replay()
        want = step(E)
        pos.add_(1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
    assert S.lens.tolist() == [400, 140]


def _near_tie(S, s, q, g, topk):
    """The last selected and the first unselected score of the newest row lie within the rounding
    of the prefill gate's fp32 scores (2^-14 of the sum of the score's absolute terms)."""
    n = int(S.lens[s])
    sums = cref.f64(S.sums[S.table[s, ::S.block // S.page].long()])[:(n - 1) // S.block, g]
    q = cref.f64(q)
    order = np.argsort(-(sums @ q))
    a, b = sums[order[topk - 2]], sums[order[topk - 1]]
    assert a @ q - b @ q <= 2.0 ** -14 * max(np.abs(a) @ np.abs(q), np.abs(b) @ np.abs(q))


def test_two_graphs_at_once(moba):
    """Two captured steps with workspaces of their own, replayed on two streams at the same time."""
    lens = [9000, 400]
    S = Setup(moba, lens, 2, 128, 64, "e4m3", 128)
    _fill(S, lens)
    q = torch.randn((2, 2, 8, 128), generator=_gen(5), device="cuda").bfloat16()
    call = lambda i: (moba.moba_paged_decode_fwd(S.cache, q[i], 6)  # noqa: E731
                      + moba.moba_paged_attn_fwd(S.cache, q[i]))
    want = [call(i) for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


def test_captured_behind_copies_and_a_join_of_streams(moba):
    """A captured step whose first call comes behind a copy, and whose attention comes behind the join
    of two captured streams."""
    lens = [700, 90]
    S = Setup(moba, lens, 2, 64, 16, "bf16", 64)
    _fill(S, lens)
    src = torch.randn((2, 4, 64), generator=_gen(2), device="cuda").bfloat16()
    q = torch.zeros_like(src)
    wq, wk = torch.rand(64, device="cuda") + 0.5, torch.rand(64, device="cuda") + 0.5
    rope, pos = moba.rope_table(100, 64), torch.zeros(2, dtype=torch.int32, device="cuda")
    k = torch.randn((2, 2, 64), generator=_gen(4), device="cuda").bfloat16()
    side = torch.cuda.Stream()

    def step():
        q.copy_(src)
        yq, _ = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos)
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            a = moba.moba_paged_attn_fwd(S.cache, yq)
        b = moba.moba_paged_decode_fwd(S.cache, yq, 3)
        cur.wait_stream(side)
        return a + b + moba.moba_paged_decode_fwd(S.cache, a[0], 2)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(5):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_queries_of_any_size(moba):
    """e4m3: query rows of zeros, of subnormal and of huge values (each row has a scaling of its
    own)."""
    n, d = 300, 64
    S = Setup(moba, [n] * 4, 1, d, 16, "e4m3")
    _fill(S, [n] * 4)
    q = torch.randn((4, 2, d), generator=_gen(6), device="cuda")
    q *= torch.tensor([0.0, 2.0 ** -128, 2.0 ** -60, 2.0 ** 100], device="cuda")[:, None, None]
    q = q.bfloat16()
    rows = [S.rows(s, n) for s in range(4)]
    for scale, use in ((0.125, [0, 1, 2]), (2.0 ** -100, [0, 1, 2, 3])):
        o, lse = moba.moba_paged_attn_fwd(S.cache, q, scale=scale)
        want = cref.cached_attention(q, [r[0] for r in rows], [r[1] for r in rows], [n] * 4, 1,
                                     scale)
        pick = lambda w: (w[0][use], w[1][:, use], None, w[3][use], w[4][:, use])  # noqa: E731
        _close(o[use], lse[:, use], pick(want), _w("e4m3"))


def test_prefill_then_decode(moba):
    """A run of the operators as a model's layer uses them: norm + rotary over the prompt, MoBA
    prefill, the cache written; then tokens one at a time through the paged cache, each against
    the prefill kernels' result for that token over the whole sequence (o within twice the
    prefill's parity tolerance, the routing equal)."""
    hq, hkv, d, page, block, topk = 8, 2, 128, 64, 128, 4
    prompt, steps = [700, 333], 5
    total = [n + steps for n in prompt]
    cu = _cu(total)
    g = _gen(21)
    qkv = torch.randn((cu[-1], (hq + 2 * hkv) * d), generator=g, device="cuda").bfloat16()
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    wq, wk = torch.rand(d, device="cuda") + 0.5, torch.rand(d, device="cuda") + 0.5
    rope = moba.rope_table(2000, d)
    pos = torch.cat([torch.arange(n, device="cuda") for n in total]).to(torch.int32)
    yq, yk = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    idx = torch.empty((hq, cu[-1], topk), dtype=torch.int32, device="cuda")
    o, lse = moba.moba_attn_fwd(yq, yk, v.contiguous(), cu_t, cu, block, topk, block_idx_out=idx)

    S = Setup(moba, total, hkv, d, page, "bf16", block)
    S.lens.copy_(torch.tensor(prompt, dtype=torch.int32))
    first = torch.cat([torch.arange(cu[s], cu[s] + prompt[s], device="cuda") for s in range(2)])
    moba.moba_cache_append(S.cache, yk[first], v[first],
                           torch.tensor(_cu(prompt), dtype=torch.int32, device="cuda"))
    ties = 0
    for i in range(steps):
        at = torch.tensor([cu[s] + prompt[s] + i for s in range(2)], device="cuda")
        S.lens.add_(1)
        nq, nk = moba.moba_qk_norm_rope(q[at], k[at], wq, wk, rope, pos[at])
        assert torch.equal(nq, yq[at])
        moba.moba_cache_append(S.cache, nk, v[at],
                               torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))
        got_idx = torch.empty((hq, 2, topk), dtype=torch.int32, device="cuda")
        po, plse = moba.moba_paged_decode_fwd(S.cache, nq, topk, block_idx_out=got_idx)
        same = (got_idx == idx[:, at]).all(-1)  # [hq, sequence]
        for h, s in (~same).nonzero().tolist():
            _near_tie(S, s, nq[s, h], h // (hq // hkv), topk)
        ok = same.T[..., None]
        err = (po.float() - o[at].float()).abs()
        assert (~ok | (err <= 2e-2 + 2e-2 * o[at].float().abs())).all()
        assert (~same | ((plse - lse[:, at]).abs() <= 2e-3)).all()
        ties += int((~same).sum())
    assert ties <= 2
    # the cached rows packed again are the prefill's inputs
    gk, gv = moba.moba_cache_read(S.cache, cu_t, cu)
    assert torch.equal(gk, yk) and torch.equal(gv, v)
    # the last steps once more as rows of one call (a chunk): the routing and results of the steps
    tail = torch.cat([torch.arange(cu[s + 1] - steps, cu[s + 1], device="cuda") for s in range(2)])
    cidx = torch.empty((hq, 2 * steps, topk), dtype=torch.int32, device="cuda")
    co, clse = moba.moba_paged_decode_fwd(S.cache, yq[tail].contiguous(), topk,
                                          rows_per_seq=steps, block_idx_out=cidx)
    same = (cidx == idx[:, tail]).all(-1)
    assert int((~same).sum()) == ties
    err = (co.float() - o[tail].float()).abs()
    assert (~same.T[..., None] | (err <= 2e-2 + 2e-2 * o[tail].float().abs())).all()
    assert (~same | ((clse - lse[:, tail]).abs() <= 2e-3)).all()
