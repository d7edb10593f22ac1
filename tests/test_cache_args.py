"""The norm and cache entry points refuse bad arguments on the host (CPU only): the C ABI before it
launches anything, the binding before a pointer reaches the library."""
import ctypes

import pytest
import torch

from block_sparse_long_moba_b200 import moba

FAKE = 0x100000  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_moba_b200 import build
    build.build()
    return moba.load_library()


@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(moba, "_current_device", lambda what, t: t.device)
    monkeypatch.setattr(moba.PagedCache, "_here", lambda self, what: self.device)


def _norm(lib, q=FAKE, q_ld=512, k_ld=256, wq=FAKE, rope=FAKE, n_pos=10, rot=128, T=4, hq=4, hkv=2,
          d=128, eps=1e-6, inter=0, out=FAKE):
    return lib.moba_qk_norm_rope(q, q_ld, FAKE, k_ld, wq, FAKE, rope, n_pos, rot, FAKE, T, hq, hkv,
                                 d, eps, inter, out, out, None)


def test_norm_host_side_errors(lib):
    assert _norm(lib, T=0) == 0                       # nothing to do
    assert _norm(lib, T=-1) == -1
    assert _norm(lib, d=96) == -2
    assert _norm(lib, rot=24) == -2                   # not a multiple of 16
    assert _norm(lib, rot=144) == -2                  # beyond d
    assert _norm(lib, rot=0) == -2
    assert _norm(lib, q_ld=504) == -1                 # tokens overlap
    assert _norm(lib, q_ld=516) == -1                 # rows not 16-byte aligned
    assert _norm(lib, k_ld=128) == -1
    assert _norm(lib, eps=-1.0) == -1
    assert _norm(lib, eps=float("nan")) == -1
    assert _norm(lib, n_pos=0) == -1
    assert _norm(lib, hq=0) == -1
    assert _norm(lib, inter=2) == -1
    assert _norm(lib, q=None) == -1
    assert _norm(lib, q=FAKE + 4) == -1
    assert _norm(lib, wq=None) == -1
    assert _norm(lib, rope=FAKE + 8) == -1
    assert _norm(lib, out=None) == -1
    assert _norm(lib, T=1 << 30, hq=64, q_ld=1 << 14) == -2
    assert lib.moba_qk_norm_rope_bwd_workspace_bytes(4, 2, 128) > 0
    assert lib.moba_qk_norm_rope_bwd_workspace_bytes(4, 2, 96) == 0
    assert lib.moba_qk_norm_rope_bwd_workspace_bytes(0, 2, 128) == 0


def _bwd(lib, T=4, dy=FAKE, dw=FAKE, ws=FAKE, ws_bytes=1 << 30, d=128):
    return lib.moba_qk_norm_rope_bwd(FAKE, 512, FAKE, 256, FAKE, FAKE, FAKE, 10, 64, FAKE, dy, FAKE,
                                     T, 4, 2, d, 1e-6, 0, FAKE, FAKE, dw, FAKE, ws, ws_bytes, None)


def test_norm_bwd_host_side_errors(lib):
    assert _bwd(lib, d=32) == -2
    assert _bwd(lib, dy=None) == -1
    assert _bwd(lib, dw=None) == -1
    assert _bwd(lib, ws=None) == -1
    assert _bwd(lib, ws=FAKE + 16) == -1
    assert _bwd(lib, ws_bytes=256) == -3


def _struct(**kw):
    base = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, block_sums=FAKE, page_table=FAKE,
                seq_lens=FAKE, dtype=0, nseq=2, max_pages=8, num_pages=20, page_size=64, Hkv=2,
                d=128, block_size=128)
    base.update(kw)
    return moba._CacheStruct(**base)


BAD = [
    (dict(k=None), -1), (dict(v=FAKE + 8), -1), (dict(page_table=None), -1),
    (dict(seq_lens=FAKE + 2), -1), (dict(nseq=0), -1), (dict(max_pages=0), -1),
    (dict(num_pages=0), -1), (dict(Hkv=0), -1), (dict(dtype=2), -1), (dict(d=96), -2),
    (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=8192), -2),
    (dict(max_pages=1 << 26), -2), (dict(dtype=1), -1), (dict(k_scale=FAKE, v_scale=FAKE), -1),
    (dict(dtype=1, k_scale=FAKE), -1), (dict(dtype=1, k_scale=FAKE, v_scale=FAKE + 4), -1),
    (dict(block_size=0), -1), (dict(block_size=96), -2), (dict(page_size=128, block_size=192), -2),
    (dict(block_sums=FAKE + 4), -1), (dict(nseq=70000), -1), (dict(Hkv=2000), -2),
]


@pytest.mark.parametrize("change,status", BAD, ids=str)
def test_cache_struct_errors(lib, change, status):
    c = ctypes.addressof(s := _struct(**change))
    ld = 1 << 20
    assert lib.moba_cache_append(c, FAKE, ld, FAKE, ld, FAKE, 4, None) == status
    assert lib.moba_cache_read(c, FAKE, 4, FAKE, FAKE, None) == status
    assert lib.moba_paged_workspace_bytes(c, 4 * s.Hkv, 1, 3) == 0
    assert lib.moba_paged_attn_fwd(c, FAKE, 4 * s.Hkv, 1, 0.1, FAKE, FAKE, FAKE, 1 << 40,
                                   None) == status
    assert lib.moba_paged_decode_fwd(c, FAKE, 4 * s.Hkv, 1, 3, 0.1, None, FAKE, FAKE, FAKE, 1 << 40,
                                     None) == status


def test_append_and_read_errors(lib):
    c = ctypes.addressof(s := _struct())
    ap = lib.moba_cache_append
    assert ap(None, FAKE, 256, FAKE, 256, FAKE, 4, None) == -1
    assert ap(c, FAKE, 256, FAKE, 256, FAKE, 0, None) == 0
    assert ap(c, FAKE, 256, FAKE, 256, FAKE, -1, None) == -1
    assert ap(c, None, 256, FAKE, 256, FAKE, 4, None) == -1
    assert ap(c, FAKE, 128, FAKE, 256, FAKE, 4, None) == -1
    assert ap(c, FAKE, 256, FAKE, 260, FAKE, 4, None) == -1
    assert ap(c, FAKE, 256, FAKE, 256, None, 4, None) == -1
    rd = lib.moba_cache_read
    assert rd(c, FAKE, 0, FAKE, FAKE, None) == 0
    assert rd(c, FAKE, -4, FAKE, FAKE, None) == -1
    assert rd(c, None, 4, FAKE, FAKE, None) == -1
    assert rd(c, FAKE, 4, FAKE + 2, FAKE, None) == -1
    assert s.Hkv == 2


def test_paged_attention_errors(lib):
    c = ctypes.addressof(s := _struct())
    big = 1 << 40

    def dense(q=FAKE, hq=8, rows=1, scale=0.1, o=FAKE, lse=FAKE, ws=FAKE, n=big):
        return lib.moba_paged_attn_fwd(c, q, hq, rows, scale, o, lse, ws, n, None)

    assert dense(hq=7) == -1                    # groups must divide
    assert dense(hq=0) == -1
    assert dense(rows=0) == -1
    assert dense(rows=257) == -2
    assert dense(hq=2 * 257) == -2
    assert dense(scale=0.0) == -1
    assert dense(scale=float("nan")) == -1
    assert dense(q=None) == -1 and dense(o=FAKE + 8) == -1 and dense(lse=None) == -1
    assert dense(ws=None) == -1 and dense(ws=FAKE + 64) == -1
    assert dense(n=128) == -3

    def routed(topk=3, idx=None, n=big):
        return lib.moba_paged_decode_fwd(c, FAKE, 8, 1, topk, 0.1, idx, FAKE, FAKE, FAKE, n, None)

    assert routed(topk=0) == -1 and routed(topk=-1) == -1 and routed(topk=65) == -2
    assert routed(idx=FAKE + 4) == -1 and routed(n=128) == -3
    none = ctypes.addressof(t := _struct(block_sums=None))
    assert lib.moba_paged_decode_fwd(none, FAKE, 8, 1, 3, 0.1, None, FAKE, FAKE, FAKE, big,
                                     None) == -1
    many = ctypes.addressof(u := _struct(max_pages=1 << 17, block_size=64))  # 131072 blocks
    assert lib.moba_paged_decode_fwd(many, FAKE, 8, 1, 3, 0.1, None, FAKE, FAKE, FAKE, big,
                                     None) == -2
    assert lib.moba_paged_workspace_bytes(many, 8, 1, 0) > 0
    assert s.d == t.d == u.d


def _raises(fn, text):
    with pytest.raises(moba.MobaError) as ei:
        fn()
    assert ei.value.status == -1 and text in str(ei.value), str(ei.value)


def _tensors(e4m3=False):
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k = torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16).to(kind)
    return dict(k=k, v=k.clone(), page_table=torch.zeros((2, 3), dtype=torch.int32),
                seq_lens=torch.zeros(2, dtype=torch.int32))


def test_cache_tensors(on_host):
    t = _tensors()
    ok = moba.PagedCache(**t)
    assert ok.nseq == 2 and ok.hkv == 2 and ok.d == 64
    for change, text in (
            (dict(k=t["k"].float()), "bfloat16"), (dict(k=t["k"][0]), "num_pages"),
            (dict(v=t["v"][:5]), "v must have shape"), (dict(v=t["v"].transpose(1, 2)), "v must"),
            (dict(page_table=t["page_table"].long()), "torch.int32"),
            (dict(page_table=t["page_table"][0]), "page_table must be"),
            (dict(seq_lens=t["seq_lens"][:1]), "seq_lens must have shape"),
            (dict(k_scale=torch.zeros((6, 2, 16), dtype=torch.uint8)), "e4m3"),
            (dict(block_sums=torch.zeros((6, 2, 64))), "block_size"),
            (dict(block_sums=torch.zeros((6, 2, 32)), block_size=64), "block_sums must have")):
        _raises(lambda: moba.PagedCache(**{**t, **change}), text)
    _raises(lambda: moba.PagedCache(**_tensors(True)), "k_scale is required")


def test_cache_calls(on_host):
    t = _tensors()
    c = moba.PagedCache(**t)
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32)
    _raises(lambda: moba.moba_cache_append(t, k, k, cu), "PagedCache")
    _raises(lambda: moba.moba_cache_append(c, k[:, :1], k, cu), "k must have shape")
    _raises(lambda: moba.moba_cache_append(c, k, k[:3], cu), "same rows")
    _raises(lambda: moba.moba_cache_append(c, k, k.transpose(0, 1).contiguous().transpose(0, 1),
                                           cu), "packed")
    _raises(lambda: moba.moba_cache_append(c, k, k, cu[:2]), "cu_seqlens_q must have shape")
    _raises(lambda: moba.moba_cache_read(c, cu, [0, 1]), "cu_seqlens_host")
    _raises(lambda: moba.moba_cache_read(c, cu, [0, 1, 4], k=k[:2]), "k must have shape")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    _raises(lambda: moba.moba_paged_attn_fwd(c, q, rows_per_seq=2), "q must have shape")
    _raises(lambda: moba.moba_paged_attn_fwd(c, q.float()), "bfloat16")
    _raises(lambda: moba.moba_paged_attn_fwd(c, q, o=q[:1]), "o must have shape")
    _raises(lambda: moba.moba_paged_decode_fwd(c, q, 3), "block_sums")
    c = moba.PagedCache(**t, block_sums=torch.zeros((6, 2, 64)), block_size=64)
    _raises(lambda: moba.moba_paged_decode_fwd(c, q, 0), "topk")
    bad = torch.zeros((4, 2, 2), dtype=torch.int32)
    _raises(lambda: moba.moba_paged_decode_fwd(c, q, 3, block_idx_out=bad,
                                               workspace=torch.zeros(9, dtype=torch.uint8)),
            "block_idx_out must have shape")


def test_norm_tensors(on_host):
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    k, w = q[:, :2].contiguous(), torch.zeros(64)
    rope, pos = torch.zeros((10, 32)), torch.zeros(4, dtype=torch.int32)
    f = moba.moba_qk_norm_rope
    _raises(lambda: f(q.float(), k, w, w, rope, pos), "bfloat16")
    _raises(lambda: f(q.transpose(0, 1), k, w, w, rope, pos), "packed")
    _raises(lambda: f(q, k[:3], w, w, rope, pos), "tokens")
    _raises(lambda: f(q, k[..., :32].contiguous(), w, w, rope, pos), "k must have shape")
    _raises(lambda: f(q, k, w.bfloat16(), w, rope, pos), "q_weight must be")
    _raises(lambda: f(q, k, w, w[:32], rope, pos), "k_weight must have shape")
    _raises(lambda: f(q, k, w, w, rope[0], pos), "rope must be")
    _raises(lambda: f(q, k, w, w, rope, pos.long()), "positions must be")
    _raises(lambda: f(q, k, w, w, rope, pos, q_out=k), "q_out must have shape")
    b = moba.moba_qk_norm_rope_bwd
    _raises(lambda: b(q, k, w, w, rope, pos, q[:, :2].contiguous(), k), "d_q_out must have shape")
    _raises(lambda: b(q, k, w, w, rope, pos, q, k, d_q_weight=w.double()), "d_q_weight must be")


def test_rope_table_is_exact_at_far_positions():
    t = moba.rope_table(300001, 64, 10000.0, device="cpu")
    import math
    for p, i in ((300000, 0), (299999, 3), (123457, 31)):
        a = p * 10000.0 ** (-2 * i / 64)
        assert abs(float(t[p, i]) - math.cos(a)) < 1e-7
        assert abs(float(t[p, 32 + i]) - math.sin(a)) < 1e-7
