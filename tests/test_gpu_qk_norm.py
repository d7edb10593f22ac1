"""moba_qk_norm_rope and its gradients on the GPU against the fp64 reference.

Tolerances. Forward: the result is fp32 arithmetic rounded once to bf16, so |y - ref| is at most
half a bf16 step of y (2^-8 |y|) plus the fp32 error of z and the turn: the mean of d squares adds
at most d 2^-24, rsqrtf 2 ulp, four products and a two-term sum one 2^-24 each, relative to the
larger of the pair: below 2^-15 of the row's largest |z|. The same terms bound dx relative to the
size of what it sums. dw: fp32 sums of terms that each carry an error below 2^-15 of the term, the
longest chain c terms: (c 2^-24 + 2^-15) sum |term|.
"""
import numpy as np
import pytest
import torch

from oracle import cache_ref as cref

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
FP = 2.0 ** -15


@pytest.fixture(scope="module")
def moba():
    from block_sparse_long_moba_b200 import build, moba as m
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.load_library()
    return m


def _inputs(moba, T, hq, hkv, d, rot, fused, seed=0, n_pos=5000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:  # slices of one projection, with a tail that belongs to neither
        x = torch.randn((T, (hq + hkv) * d + 24), generator=g, device="cuda").bfloat16()
        q, k = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    else:
        q = torch.randn((T, hq, d), generator=g, device="cuda").bfloat16()
        k = torch.randn((T, hkv, d), generator=g, device="cuda").bfloat16()
    k = k * 37.0 if not fused else k
    wq = torch.randn(d, generator=g, device="cuda")
    wk = torch.randn(d, generator=g, device="cuda")
    pos = torch.randint(0, n_pos, (T,), generator=g, device="cuda").to(torch.int32)
    return q, k, wq, wk, moba.rope_table(n_pos, rot, 500000.0), pos


CASES = [  # T, hq, hkv, d, rot, interleaved, fused
    (1, 32, 8, 128, 128, False, True),
    (1, 1, 1, 64, 64, True, False),
    (37, 32, 8, 128, 128, False, False),
    (301, 16, 16, 64, 32, True, True),
    (300, 5, 3, 64, 64, False, True),
    (129, 7, 1, 128, 16, False, False),
    (64, 4, 2, 128, 96, True, True),
    (2000, 4, 1, 128, 48, False, False),
    (20000, 32, 8, 128, 128, False, True),  # many chunks a warp
    (7000, 20, 20, 64, 48, True, False),
    (16384, 4, 1, 128, 128, False, True),   # few heads, many tokens: rows packed across tokens
    (20001, 1, 3, 128, 64, True, False),
    (4096, 4, 1, 128, 128, False, False),   # the gradients' alone
    (30011, 5, 2, 64, 64, False, True),
    (17000, 16, 2, 128, 32, False, True),   # q by tokens, k by rows
    (16501, 7, 17, 64, 32, True, True),     # and the other way round
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(moba, case):
    T, hq, hkv, d, rot, adj, fused = case
    q, k, wq, wk, rope, pos = _inputs(moba, T, hq, hkv, d, rot, fused)
    yq, yk = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos, eps=1e-5, interleaved=adj)
    assert yq.shape == q.shape and yk.shape == k.shape
    for x, w, y in ((q, wq, yq), (k, wk, yk)):
        want = cref.norm_rope(x, w, cref.f64(rope), pos.cpu().numpy(), 1e-5, adj)
        err = np.abs(cref.f64(y) - want)
        assert (err <= BF * np.abs(want) + FP * np.abs(want).max(-1, keepdims=True)).all()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(moba, case):
    T, hq, hkv, d, rot, adj, fused = case
    q, k, wq, wk, rope, pos = _inputs(moba, T, hq, hkv, d, rot, fused, seed=1)
    g = torch.Generator(device="cuda").manual_seed(9)
    dyq = torch.randn((T, hq, d), generator=g, device="cuda").bfloat16()
    dyk = torch.randn((T, hkv, d), generator=g, device="cuda").bfloat16()
    dq, dk, dwq, dwk = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, eps=1e-5,
                                                  interleaved=adj)
    for x, w, dy, dx, dw in ((q, wq, dyq, dq, dwq), (k, wk, dyk, dk, dwk)):
        wx, ww, size = cref.norm_rope_bwd(x, w, cref.f64(rope), pos.cpu().numpy(), dy, 1e-5, adj)
        err = np.abs(cref.f64(dx) - wx)
        assert (err <= BF * np.abs(wx) + FP * size).all(), float((err / size).max())
        hat = np.abs(cref.norm_rope(x, torch.ones(d), np.concatenate(
            [np.ones((1, rot // 2)), np.zeros((1, rot // 2))], 1), np.zeros(T, int), 1e-5, adj))
        dz = np.abs(cref.rotate(cref.f64(dy), cref.f64(rope), pos.cpu().numpy(), adj, -1.0))
        terms = (hat * dz).sum((0, 1))
        chain = x.shape[0] * x.shape[1]  # no chain is longer than all rows
        assert (np.abs(cref.f64(dw) - ww) <= (chain * 2.0 ** -24 + FP) * terms).all()
    again = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, eps=1e-5,
                                       interleaved=adj)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))


def test_backward_is_the_difference_quotient(moba):
    """The gradients against differences of the fp64 forward along random directions."""
    T, hq, hkv, d = 40, 4, 2, 64
    q, k, wq, wk, rope, pos = _inputs(moba, T, hq, hkv, d, 64, False, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    dyq = torch.randn((T, hq, d), generator=g, device="cuda").bfloat16()
    dyk = torch.randn((T, hkv, d), generator=g, device="cuda").bfloat16()
    dq, _, dwq, _ = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk)
    rng = np.random.default_rng(0)
    ux, uw = rng.standard_normal((T, hq, d)), rng.standard_normal(d)
    f = lambda e: (cref.norm_rope(cref.f64(q) + e * ux, cref.f64(wq) + e * uw, cref.f64(rope),  # noqa: E731
                                  pos.cpu().numpy(), 1e-6, False) * cref.f64(dyq)).sum()
    quotient = (f(1e-5) - f(-1e-5)) / 2e-5
    along = (cref.f64(dq) * ux).sum() + (cref.f64(dwq) * uw).sum()
    # dq is rounded to bf16: at most 2^-8 of each of its products, and the quotient's own 1e-8
    bound = BF * np.abs(cref.f64(dq) * ux).sum() + 1e-6 * abs(quotient) + 1e-3
    assert abs(along - quotient) <= bound


def test_no_rows(moba):
    q, k, wq, wk, rope, pos = _inputs(moba, 0, 4, 2, 64, 64, False)
    yq, yk = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos)
    assert yq.shape == (0, 4, 64) and yk.shape == (0, 2, 64)
    dwq, dwk = torch.full_like(wq, 7.0), torch.full_like(wk, 7.0)
    moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, yq, yk, d_q_weight=dwq, d_k_weight=dwk)
    assert not dwq.any() and not dwk.any()


@pytest.mark.parametrize("T", [6, 17003])
def test_position_outside_the_table_is_nan_in_that_token_only(moba, T):
    q, k, wq, wk, rope, pos = _inputs(moba, T, 4, 2, 128, 64, False, n_pos=50)
    pos[2], pos[4] = 50, -1
    yq, yk = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos)
    for y in (yq, yk):
        bad = y.isnan().flatten(1)
        assert bad[[2, 4]].all() and not bad[[0, 1, 3, 5]].any() and not bad[6:].any()


@pytest.mark.parametrize("T", [9, 16501])
def test_in_place_zero_rows_and_rows_behind_the_call(moba, T):
    """Packed outputs may be the inputs; a row of zeros stays zero; the tokens behind the call's
    are left as they were."""
    q, k, wq, wk, rope, pos = _inputs(moba, T, 4, 2, 64, 64, False, seed=2)
    q[3] = 0
    want = moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos)
    assert not want[0][3].any()
    qq, kk = torch.full((T + 3, 4, 64), 5.0, device="cuda").bfloat16(), k.clone()
    qq[:T] = q
    moba.moba_qk_norm_rope(qq[:T], kk, wq, wk, rope, pos, q_out=qq[:T], k_out=kk)
    assert torch.equal(qq[:T], want[0]) and torch.equal(kk, want[1]) and (qq[T:] == 5.0).all()
    dyq, dyk = torch.randn_like(q), torch.randn_like(k)
    want = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk)
    got = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, dq=dyq, dk=dyk)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_beside_an_eager_stream(moba):
    """A captured forward and backward pass, replayed on new inputs, while the same calls run
    eagerly on a second stream with a workspace of their own."""
    T, hq, hkv, d = 500, 8, 2, 128
    q, k, wq, wk, rope, pos = _inputs(moba, T, hq, hkv, d, 128, False, seed=6)
    dyq, dyk = torch.randn_like(q), torch.randn_like(k)

    def both(stream=None):
        return (moba.moba_qk_norm_rope(q, k, wq, wk, rope, pos, stream=stream)
                + moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, stream=stream))

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    q.normal_()
    dyk.normal_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        eager = both(stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
