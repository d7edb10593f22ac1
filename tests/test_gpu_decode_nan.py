"""moba_decode_fwd with queries that are not finite: by the formula that row's o and lse are NaN, as
moba_paged_decode_fwd gives them; the other rows have the bits of a call without it."""
import pytest
import torch

from block_sparse_long_moba_b200 import workloads as wl
from oracle import moba_ref as ref
from tests.test_gpu_decode import moba  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("x", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite(moba, d, x):  # noqa: F811
    cu, cuq, hq, hkv, B, topk = [0, 3000, 3001, 9000], [0, 2, 3, 4], 4, 2, 256, 4
    w = wl.custom(cu, hq, hkv, d, B, topk, "offset")
    q_all, k, v, cu_t = wl.make_inputs(w, seed=0, device="cuda")
    k[..., 0] = k[..., 0].abs() + 0.5  # an infinite q[0] makes all logits +inf, or all -inf
    pos = ref.cache_row_positions(cu, cuq)
    q = q_all[torch.as_tensor(pos, device="cuda")].contiguous()
    cuq_t = torch.tensor(cuq, dtype=torch.int32, device="cuda")
    cents = moba.moba_centroids(k, cu_t, cu, B)

    def run(q):
        return moba.moba_decode_fwd(q, k, v, cents, cu_t, cu, cuq_t, cuq, B, topk, d ** -0.5)

    want = run(q)
    bad = torch.zeros((cuq[-1], hq), dtype=torch.bool, device="cuda")
    for at, h in ((0, 1), (2, 0), (3, 3)):
        bad[at, h] = True
    q[..., 0][bad] = x
    o, lse = run(q)
    assert o[bad].isnan().all() and lse.T[bad].isnan().all()
    assert torch.equal(o[~bad], want[0][~bad]) and torch.equal(lse.T[~bad], want[1].T[~bad])
