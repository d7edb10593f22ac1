"""The weights' gradients of moba_qk_norm_rope_bwd over many rows, within a bound that a missing,
doubled or misplaced part of the sum breaks.

Tolerance. dw[c] is a sum of N = T * heads terms t = dz * (x r). The inputs are independent and of
random sign, so |dw| is about sqrt(N) rms(t). It is summed in parts: a lane adds its rows one after
the other in fp32, the lanes of a warp and the eight warps of a CTA follow, then the CTAs' parts in
fp64. The kernels run at most 148 CTAs of eight warps, a warp takes chunks of 2 KB, and a lane has
four rows of a chunk, so a lane's chain is at most c = 4 (ceil(chunks / 1184) + 1) long, chunks those
of both tensors.
  Additions: each rounds by at most 2^-24 of its running sum, which is below 8 sqrt(c) rms(t)
  (eight standard deviations). The N roundings are independent of each other: their sum is below
  8 sqrt(N) 2^-24 8 sqrt(c) rms(t).
  Terms: each carries an error below 2^-15 of its size (test_gpu_qk_norm.py). The part that is the
  same in every row gives at most 2^-15 |dw|, the part that is not at most 8 sqrt(N) 2^-15 rms(t).
Together about 2^-11.5 of the typical |dw|; the rows of one CTA, where 148 share them, are a
twelfth of it.
"""
import numpy as np
import pytest
import torch

from oracle import cache_ref as cref
from tests.test_gpu_qk_norm import _inputs, moba  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [  # T, hq, hkv, d, rot, interleaved, fused
    (20000, 32, 8, 128, 128, False, True),  # q and k by tokens
    (7000, 20, 20, 64, 48, True, False),
    (16384, 4, 1, 128, 128, False, True),   # both by rows
    (20001, 1, 3, 128, 64, True, False),
    (17000, 16, 2, 128, 32, False, True),   # q by tokens, k by rows
    (16501, 7, 17, 64, 32, True, True),     # and the other way round
    (17003, 4, 5, 128, 128, False, True),   # on both sides of the rule, half a chunk's heads
    (4099, 9, 8, 64, 64, True, False),
    (37, 32, 8, 128, 128, False, False),    # fewer chunks than warps
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_no_part_of_a_weight_gradient_is_lost(moba, case):  # noqa: F811
    T, hq, hkv, d, rot, adj, fused = case
    q, k, wq, wk, rope, pos = _inputs(moba, T, hq, hkv, d, rot, fused, seed=31)
    g = torch.Generator(device="cuda").manual_seed(32)
    dyq = torch.randn((T, hq, d), generator=g, device="cuda").bfloat16()
    dyk = torch.randn((T, hkv, d), generator=g, device="cuda").bfloat16()
    _, _, dwq, dwk = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, eps=1e-5,
                                                interleaved=adj)
    per = 1024 // d  # rows of a chunk
    units = T * (-(-hq // per) + -(-hkv // per))
    c = 4 * (-(-units // (148 * 8)) + 1)
    for x, w, dy, dw in ((q, wq, dyq, dwq), (k, wk, dyk, dwk)):
        _, want, _ = cref.norm_rope_bwd(x, w, cref.f64(rope), pos.cpu().numpy(), dy, 1e-5, adj)
        xx = cref.f64(x)
        hat = xx / np.sqrt((xx * xx).mean(-1, keepdims=True) + 1e-5)
        dz = cref.rotate(cref.f64(dy), cref.f64(rope), pos.cpu().numpy(), adj, -1.0)
        rms = np.sqrt(((dz * hat) ** 2).mean((0, 1)))
        n = T * x.shape[1]
        bound = (2.0 ** -15 * np.abs(want) + 2.0 ** -15 * 8 * np.sqrt(n) * rms
                 + 64 * 2.0 ** -24 * np.sqrt(n * c) * rms)
        # a bound that a gradient of zeros fails in every column, and one that lacks a CTA's rows in
        # nearly every one
        assert bound.max() < np.sqrt(np.mean(want ** 2)) / 100
        part = (dz * hat).reshape(n, d)[:max(1, n // 444)].sum(0)
        assert (np.abs(part) > bound).mean() > 0.9
        assert (np.abs(cref.f64(dw) - want) <= bound).all(), float(
            (np.abs(cref.f64(dw) - want) / bound).max())


@pytest.mark.parametrize("T", [6, 17003])  # by tokens, by rows
def test_gradients_of_a_position_outside_the_table(moba, T):  # noqa: F811
    """NaN in that token's gradients and in the weights', as the forward result was; the other
    tokens' are right."""
    q, k, wq, wk, rope, pos = _inputs(moba, T, 4, 2, 128, 64, False, n_pos=50)
    g = torch.Generator(device="cuda").manual_seed(3)
    dyq = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    dyk = torch.randn(k.shape, generator=g, device="cuda").bfloat16()
    want = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk)
    pos[2], pos[4] = 50, -1
    got = moba.moba_qk_norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[2, 4]] = False
    for a, b in zip(got[:2], want[:2]):
        assert a[[2, 4]].isnan().all() and torch.equal(a[keep], b[keep])
    assert got[2].isnan().all() and got[3].isnan().all()
