"""Pins of the cache operators' fp64 reference (oracle/cache_ref.py) against other statements of
the same formulas: torch autograd, complex rotation, torch's e4m3 conversion, the MoBA oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ref as cref
from oracle import moba_ref as ref


def _table(n, rot, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("d,rot,adj", [(64, 64, False), (64, 32, True), (128, 16, False)])
def test_norm_rope_against_torch_and_complex_numbers(d, rot, adj):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((5, 3, d), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(d, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn((5, 3, d), generator=g, dtype=torch.float64)
    pos = np.array([0, 9, 2, 7, 7])
    rope = _table(10, rot)
    z = torch.nn.functional.rms_norm(x, (d,), w, 1e-6)
    t = torch.from_numpy(rope[pos])
    turn = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
    if adj:
        y = torch.view_as_real(torch.view_as_complex(z[..., :rot].unflatten(-1, (-1, 2))) * turn)
        y = torch.cat([y.flatten(-2), z[..., rot:]], -1)
    else:
        y = torch.complex(z[..., :rot // 2], z[..., rot // 2:rot]) * turn
        y = torch.cat([y.real, y.imag, z[..., rot:]], -1)
    got = cref.norm_rope(x, w, rope, pos, 1e-6, adj)
    assert np.abs(got - y.detach().numpy()).max() < 1e-12
    gx, gw = torch.autograd.grad(y, (x, w), dy)
    dx, dw, size = cref.norm_rope_bwd(x, w, rope, pos, dy, 1e-6, adj)
    assert np.abs(dx - gx.numpy()).max() < 1e-12 and np.abs(dw - gw.numpy()).max() < 1e-12
    assert (np.abs(dx) <= size * 2 * (1 + 1e-9) * math.sqrt(d)).all()


def test_norm_rope_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((2, 1, 64)), rng.standard_normal(64)
    dy, pos, rope = rng.standard_normal((2, 1, 64)), np.array([3, 8]), _table(9, 32)
    dx, dw, _ = cref.norm_rope_bwd(x, w, rope, pos, dy, 1e-6, False)
    f = lambda x, w: (cref.norm_rope(x, w, rope, pos, 1e-6, False) * dy).sum()  # noqa: E731
    for i in (0, 17, 40, 63):
        e = np.zeros(64)
        e[i] = 1e-6
        assert abs((f(x + [[e], [0 * e]], w) - f(x - [[e], [0 * e]], w)) / 2e-6
                   - dx[0, 0, i]) < 1e-7
        assert abs((f(x, w + e) - f(x, w - e)) / 2e-6 - dw[i]) < 1e-7


def test_quantise_against_torch_conversion_and_at_the_border():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((400, 64), generator=g) * torch.exp2(
        torch.randint(-60, 60, (400, 1), generator=g).float())).bfloat16()
    x[0] = 0
    x[1] = 0
    x[1, 5] = 448.0  # exactly representable at scale 1
    x[2] = 0
    x[2, 5] = 450.0  # just above: the next power of two
    x[3] = 1e-38     # below the smallest scale's range
    codes, b = cref.quantise(x)
    assert b[0] == 1 and b[1] == 127 and b[2] == 128 and b[3] == 1
    s = np.exp2(b.astype(np.float64) - 127)
    want = (x.double() / torch.from_numpy(s)[:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(codes, want.view(torch.uint8).numpy())
    back = cref.dequantise(codes, b)
    assert np.array_equal(back, want.double().numpy() * s[:, None])
    # to nearest: within half a step, 2^-4 of the value or 2^-10 of the scale
    assert (np.abs(back - x.double().numpy())
            <= np.maximum(2.0 ** -4 * np.abs(x.double().numpy()), 2.0 ** -10 * s[:, None])).all()


def test_cached_attention_against_the_moba_oracle():
    """The newest rows of cached sequences, MoBA-routed and dense, as moba_ref states them."""
    g = torch.Generator().manual_seed(2)
    cu, B, topk, hq, hkv, d = [0, 700, 1500], 128, 3, 4, 2, 64
    q, k, v = (torch.randn((1500, h, d), generator=g).bfloat16() for h in (hq, hkv, hkv))
    rows = 2
    pos = ref.cache_row_positions(cu, [0, 2, 4])
    cents = ref.centroids(k, cu, B)
    rt = ref.select_blocks(q, cents, cu, B, topk, pos)
    o_ref, lse_ref = ref.attention(q, k, v, cu, B, rt.idx, 0.125, pos)
    ks = [cref.f64(k[a:b]) for a, b in ((0, 700), (700, 1500))]
    vs = [cref.f64(v[a:b]) for a, b in ((0, 700), (700, 1500))]
    sums = [np.stack([x[j:j + B].sum(0) for j in range(0, len(x), B)]) for x in ks]
    o, lse, idx, spread, dot = cref.cached_attention(q[torch.as_tensor(pos)], ks, vs, [700, 800],
                                                     rows, 0.125, sums, B, topk)
    assert np.array_equal(idx, rt.idx)
    assert np.abs(o - o_ref).max() < 1e-12 and np.abs(lse - lse_ref).max() < 1e-12
    full = ref.select_blocks(q, cents, cu, B, 64, pos)
    o_ref, lse_ref = ref.attention(q, k, v, cu, B, full.idx, 0.125, pos)
    o, lse, idx, spread, dot = cref.cached_attention(q[torch.as_tensor(pos)], ks, vs, [700, 800],
                                                     rows, 0.125)
    assert idx is None and np.abs(o - o_ref).max() < 1e-12 and np.abs(lse - lse_ref).max() < 1e-12
    assert (spread >= np.abs(o) - 1e-12).all() and (dot > 0).all()


def test_cached_attention_without_a_position():
    q = np.ones((2, 1, 64))
    o, lse, idx, _, _ = cref.cached_attention(q, [np.ones((1, 1, 64))], [np.ones((1, 1, 64))],
                                              [1], 2, 0.1, [np.ones((1, 1, 64))], 64, 2)
    assert not o[0].any() and lse[0, 0] == -math.inf and (idx[0, 0] == -1).all()
    assert abs(lse[0, 1] - 6.4) < 1e-12 and list(idx[0, 1]) == [0, -1] and o[1].min() == 1
