"""Cases that measure the operators around a paged key-value cache: norms and rotary positions of
queries and keys (forward and backward), the cache's write and read, and attention of the newest
tokens over it, dense and block-sparse (MoBA).

`run` computes a case in plain torch operations, or with `own` set through the package's entry
points. Both take what `prepare` made; `exact` states the same results in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
ROPE_BASE = 500000.0  # far positions: the table is computed in 64 bits
DEV = "cuda"


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of one sequence: q and k of a single token, latency only
        dict(name="norm_rope_1_token", op="norm_rope", tokens=1, hq=32, hkv=8, d=128, rot=128,
             pairs="half", fused=True, mix=1),
        # a 128K-token prompt of the Llama-3.1-8B attention shape, q and k read out of the fused
        # projection's rows
        dict(name="norm_rope_128k", op="norm_rope", tokens=131072, hq=32, hkv=8, d=128, rot=128,
             pairs="half", fused=True, mix=2),
        # one training step's backward pass, 16 heads of 64, an odd token count, half of each
        # head rotated in adjacent pairs
        dict(name="norm_rope_bwd_64k", op="norm_rope_bwd", tokens=65521, hq=16, hkv=16, d=64,
             rot=32, pairs="adjacent", fused=False, mix=3),
        # one decode step of a batch: one token a sequence into 8-bit pages
        dict(name="append_64x1_e4m3", op="append", seqs=64, new=1, length=8192, ragged=True,
             hkv=8, d=128, page=64, block=4096, kv="e4m3", fused=True, mix=4),
        # ragged prompts written into 8-bit pages
        dict(name="append_prompts_e4m3", op="append", seqs=4, new=65536, length=65536,
             ragged=True, hkv=8, d=128, page=64, block=4096, kv="e4m3", fused=True, mix=5),
        # the cached keys and values of a ragged batch packed again (chunked prefill, moving a
        # sequence to another card)
        dict(name="read_ragged_e4m3", op="read", seqs=8, length=65536, ragged=True, hkv=8, d=128,
             page=64, block=4096, kv="e4m3", mix=6),
        # dense attention of one short sequence's newest token
        dict(name="attn_1x1000", op="attn", seqs=1, length=1000, ragged=False, rows=1, hq=32,
             hkv=8, d=128, page=64, block=4096, kv="bf16", mix=7),
        # a ragged serving batch, dense layers
        dict(name="attn_32_ragged", op="attn", seqs=32, length=16384, ragged=True, rows=1, hq=32,
             hkv=8, d=128, page=64, block=4096, kv="bf16", mix=8),
        # eight sequences of 128K in 8-bit pages, dense layers
        dict(name="attn_8x128k_e4m3", op="attn", seqs=8, length=131072, ragged=False, rows=1,
             hq=32, hkv=8, d=128, page=64, block=4096, kv="e4m3", mix=9),
        # MoBA decode of one 128K sequence
        dict(name="moba_1x128k", op="moba", seqs=1, length=131071, ragged=False, rows=1, hq=32,
             hkv=8, d=128, page=64, block=4096, topk=12, kv="bf16", mix=10),
        # MoBA decode of eight sequences of 128K
        dict(name="moba_8x128k", op="moba", seqs=8, length=131072, ragged=False, rows=1, hq=32,
             hkv=8, d=128, page=64, block=4096, topk=12, kv="bf16", mix=11),
        # small blocks: thousands of block scores a row, ragged caches in 8-bit pages
        dict(name="moba_small_blocks_e4m3", op="moba", seqs=4, length=229376, ragged=True, rows=1,
             hq=16, hkv=16, d=64, page=64, block=128, topk=32, kv="e4m3", mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "read", "attn", "attn", "moba",
                     "moba"])
    hq, hkv, d = rng.choice([(32, 8, 128), (16, 16, 64), (4, 1, 128), (8, 2, 64), (16, 2, 128)])
    mix = rng.randrange(1 << 20)
    if op.startswith("norm_rope"):
        return dict(op=op, tokens=_log(rng, 1, 65536), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), pairs=rng.choice(["half", "adjacent"]),
                    fused=rng.random() < 0.5, mix=mix)
    seqs = _log(rng, 1, 48)
    # at most 512K cached tokens of 8 heads of 128, so that no case is larger than the listed ones
    most = min(262144, (1 << 29) // (seqs * hkv * d))
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([128, 512, 4096])
    kv = rng.choice(["bf16", "e4m3"])
    # short prompts and fresh sequences, and the long caches that the operators are for
    length = _log(rng, 1, 512) if rng.random() < 0.25 else _log(rng, min(512, most), most)
    case = dict(op=op, seqs=seqs, length=length, ragged=rng.random() < 0.7, hkv=hkv, d=d,
                page=page, block=block, kv=kv, mix=mix)
    if op == "append":
        case["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, case["length"])
        case["fused"] = rng.random() < 0.5
    elif op in ("attn", "moba"):
        case.update(hq=hq, rows=rng.choice([1, 1, 1, 2, 4]))
        if op == "moba":
            case["topk"] = rng.choice([1, 3, 8, 12, 16, 32])
    return case


def _lengths(case):
    """Cached tokens of each sequence (the new ones included) and how many of them are new."""
    rng = random.Random(case["mix"])
    n, top = case["seqs"], case["length"]
    lens = [top] * n
    if case["ragged"] and n > 1:
        lens = [top] + [_log(rng, max(1, top // 16), top) for _ in range(n - 1)]
        rng.shuffle(lens)
    new = [min(x, case.get("new", 1)) for x in lens]
    if case["ragged"] and case.get("new", 1) > 1:
        new = [rng.randint(max(1, x // 2), x) for x in new]
    return lens, new


# ---------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _split(case, tokens, g, hq):
    """q, k, v [tokens, heads, d]: slices of one fused projection's rows, or tensors of their own."""
    hkv, d = case["hkv"], case["d"]
    if case["fused"]:
        qkv = _randn(g, tokens, (hq + 2 * hkv) * d)
        return tuple(x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    return _randn(g, tokens, hq, d), _randn(g, tokens, hkv, d), _randn(g, tokens, hkv, d)


def _scale_bytes(amax):
    """Biased exponent of the smallest power of two s >= 2^-126 with amax / s <= 448."""
    bits = amax.float().view(torch.int32)
    up = ((bits & 0x7FFFFF) > 0x600000).int()  # mantissa above 1.75 = 448 / 256
    return ((bits >> 23) - 8 + up).clamp(min=1)


def _quantise(x):
    """e4m3 codes and scale bytes of x [..., d]: one power of two a row."""
    b = _scale_bytes(x.abs().amax(-1))
    inv = ((254 - b) << 23).view(torch.float32)
    return (x.float() * inv[..., None]).to(torch.float8_e4m3fn), b.to(torch.uint8)


def _dequantise(codes, scale):
    return codes.float() * (scale.int() << 23).view(torch.float32)[..., None]


def _pages(lens, case, g):
    """page_table [seqs, most pages] (-1 behind a sequence's own pages), in an order as a pool that
    has been used for a while gives them out, and the pool's size."""
    need = [-(-x // case["page"]) for x in lens]
    pool = sum(need) + 5
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, pool


def _filled_cache(case, lens, g):
    """A pool whose pages hold keys with a common offset in each block (so that the block scores
    have something to find), values, and each block's key sum at the block's first page."""
    hkv, d, page, block = case["hkv"], case["d"], case["page"], case["block"]
    table, pool = _pages(lens, case, g)
    per = block // page
    k = _randn(g, pool, hkv, page, d)
    v = _randn(g, pool, hkv, page, d)
    seq, col = (table >= 0).nonzero(as_tuple=True)
    ids = table[seq, col].long()
    nblk = -(-table.shape[1] // per)
    off = 0.5 * _randn(g, len(lens), nblk, hkv, d)
    k[ids] += off[seq, col // per][:, :, None, :]
    # sums over the tokens that are there: the last page of a sequence ends inside
    lens_t = torch.tensor(lens, device=DEV)
    left = (lens_t[seq] - col * page).clamp(max=page)
    page_sum = torch.empty((pool, hkv, d), dtype=torch.float32, device=DEV)
    page_sum[:] = k.sum(2, dtype=torch.float32)
    last = (left < page).nonzero()[:, 0]
    keep = torch.arange(page, device=DEV)[None, :] < left[last][:, None]
    page_sum[ids[last]] = (k[ids[last]].float() * keep[:, None, :, None]).sum(2)
    sums = torch.zeros((pool, hkv, d), dtype=torch.float32, device=DEV)
    for j in range(per):
        at = (col % per == j).nonzero()[:, 0]
        sums[table[seq[at], col[at] - j].long()] += page_sum[ids[at]]
    k_scale = v_scale = None
    if case["kv"] == "e4m3":
        k, k_scale = _quantise(k)
        v, v_scale = _quantise(v)
    return dict(k_cache=k, v_cache=v, k_scale=k_scale, v_scale=v_scale, block_sums=sums,
                page_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def _empty_cache(case, lens, g):
    hkv, d, page = case["hkv"], case["d"], case["page"]
    table, pool = _pages(lens, case, g)
    e4m3 = case["kv"] == "e4m3"
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = (torch.zeros((pool, hkv, page, d), dtype=torch.bfloat16, device=DEV).to(kind)
            for _ in range(2))
    ks, vs = ((torch.ones((pool, hkv, page), dtype=torch.uint8, device=DEV) if e4m3 else None)
              for _ in range(2))
    sums = torch.randn((pool, hkv, d), generator=g, device=DEV)
    return dict(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_sums=sums, page_table=table,
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def _offsets(counts):
    out = [0]
    for x in counts:
        out.append(out[-1] + x)
    return out


def _angles(n, rot):
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    state = dict(case=case)
    if op.startswith("norm_rope"):
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        q, k, _ = _split(case, t, g, hq)
        # a packed batch of sequences: positions start again at each
        one = max(1, t // 3 + 1)
        start = 7 if t > 1 else 4095
        state.update(q=q, k=k, rope=_angles(start + one + 1, case["rot"]),
                     positions=(start + torch.arange(t, device=DEV) % one).to(torch.int32),
                     q_weight=1 + 0.2 * torch.randn(d, generator=g, device=DEV),
                     k_weight=1 + 0.2 * torch.randn(d, generator=g, device=DEV))
        if op == "norm_rope_bwd":
            state.update(d_q=_randn(g, t, hq, d), d_k=_randn(g, t, hkv, d))
        return state
    lens, new = _lengths(case)
    state.update(_empty_cache(case, lens, g) if op == "append" else _filled_cache(case, lens, g))
    if op == "append":
        cu = _offsets(new)
        _, state["k"], state["v"] = _split(case, cu[-1], g, 4 * case["hkv"])
        state["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    elif op == "read":
        state["cu_host"] = _offsets(lens)
        state["cu"] = torch.tensor(state["cu_host"], dtype=torch.int32, device=DEV)
    else:
        state["q"] = _randn(g, case["seqs"] * case["rows"], case["hq"], case["d"])
    if own:  # the handle that a serving program keeps for its cache: pointers and sizes
        from block_sparse_long_moba_b200 import moba
        state["cache"] = moba.PagedCache(
            state["k_cache"], state["v_cache"], state["page_table"], state["seq_lens"],
            k_scale=state["k_scale"], v_scale=state["v_scale"], block_sums=state["block_sums"],
            block_size=case["block"])
    return state


# ----------------------------------------------------------------------------------- plain forms
def _rotate(z, state, sign):
    """Pairs of the first rot dimensions turned by sign times the position's angle."""
    rot, pairs = state["case"]["rot"], state["case"]["pairs"]
    row = state["rope"][state["positions"].long()]
    c, s = row[:, None, :rot // 2], sign * row[:, None, rot // 2:]
    head, tail = z[..., :rot], z[..., rot:]
    if pairs == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat([a * c - b * s, b * c + a * s, tail], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), tail], -1)


def _norm_rope(state):
    def one(x, w):
        x = x.float()
        z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        return _rotate(z, state, 1.0).to(torch.bfloat16)
    return {"q": one(state["q"], state["q_weight"]), "k": one(state["k"], state["k_weight"])}


def _norm_rope_bwd(state):
    def one(x, w, dy):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        hat = x * r
        dz = _rotate(dy.float(), state, -1.0)
        dw = (dz * hat).sum((0, 1), dtype=torch.float64).float()
        dhat = dz * w
        dx = r * (dhat - hat * (dhat * hat).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), dw
    dq, dqw = one(state["q"], state["q_weight"], state["d_q"])
    dk, dkw = one(state["k"], state["k_weight"], state["d_k"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _append(state):
    """New rows into their pages; the key sum of each block that they touch."""
    case = state["case"]
    page, block = case["page"], case["block"]
    cu, lens, table = state["cu_q"].long(), state["seq_lens"].long(), state["page_table"].long()
    count = cu[1:] - cu[:-1]
    row = torch.arange(state["k"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = lens[seq] - count[seq] + row - cu[seq]
    pid, slot = table[seq, pos // page], pos % page
    if case["kv"] == "e4m3":
        for x, cache, scale in ((state["k"], "k_cache", "k_scale"),
                                (state["v"], "v_cache", "v_scale")):
            codes, b = _quantise(x)
            state[cache].view(torch.uint8)[pid, :, slot] = codes.view(torch.uint8)
            state[scale][pid, :, slot] = b
    else:
        state["k_cache"][pid, :, slot] = state["k"]
        state["v_cache"][pid, :, slot] = state["v"]
    sums = state["block_sums"]
    home = table[seq, pos // block * (block // page)]  # first page of the row's block
    first = (lens - count)[seq]
    fresh = home[(pos // block) * block >= first]  # the block begins with new rows
    sums[fresh] = 0
    add = torch.zeros_like(sums, dtype=torch.float64)
    add.index_add_(0, home, state["k"].double())  # long sums: in 64 bits
    sums.copy_((sums.double() + add).float())
    return _cache_outputs(state)


def _cache_outputs(state):
    out = {n: state[n] for n in ("k_cache", "v_cache", "block_sums")}
    if state["k_scale"] is not None:
        out.update(k_scale=state["k_scale"], v_scale=state["v_scale"])
    return out


def _read(state):
    page = state["case"]["page"]
    cu, table = state["cu"].long(), state["page_table"].long()
    row = torch.arange(state["cu_host"][-1], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = row - cu[seq]
    pid, slot = table[seq, pos // page], pos % page
    out = {}
    for n in ("k", "v"):
        cache, scale = state[n + "_cache"], state[n + "_scale"]
        if scale is None:
            out[n] = cache[pid, :, slot]
        else:
            codes = cache.view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn)
            out[n] = _dequantise(codes, scale[pid, :, slot]).to(torch.bfloat16)
    return out


def _whole(state, n):
    """Keys or values of all pages of every sequence, in 32 bits: [seqs, hkv, tokens, d]."""
    table = state["page_table"].long().clamp(min=0)
    cache, scale = state[n + "_cache"], state[n + "_scale"]
    if scale is None:
        x = cache[table].float()
    else:
        x = _dequantise(cache.view(torch.uint8)[table].view(torch.float8_e4m3fn), scale[table])
    return x.transpose(1, 2).flatten(2, 3)


def _attend(state, allowed):
    """Softmax over the allowed keys. allowed [seqs, hkv, rows x group or 1, tokens]."""
    case = state["case"]
    n, rows, hq, hkv, d = (case[x] for x in ("seqs", "rows", "hq", "hkv", "d"))
    r = hq // hkv
    q = state["q"].float().view(n, rows, hkv, r, d).transpose(1, 2).flatten(2, 3)
    logits = q @ _whole(state, "k").transpose(-1, -2) * d ** -0.5
    logits = logits.masked_fill(~allowed, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)  # a row with no key: all -inf
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    v = _whole(state, "v").masked_fill_(~allowed.any(2)[..., None], 0)
    o = p @ v / total.clamp(min=1e-38)
    lse = (top + total.log())[..., 0]
    o = o.view(n, hkv, rows, r, d).transpose(1, 2).reshape(n * rows, hq, d).to(torch.bfloat16)
    lse = lse.view(n, hkv, rows, r).permute(1, 3, 0, 2).reshape(hq, n * rows)
    return o, lse


def _places(state):
    """Position of each row [seqs, rows] and of each cached token [tokens]."""
    rows = state["case"]["rows"]
    lens = state["seq_lens"].long()
    at = lens[:, None] - rows + torch.arange(rows, device=DEV)
    return at, torch.arange(state["page_table"].shape[1] * state["case"]["page"], device=DEV)


def _attn(state):
    case = state["case"]
    at, token = _places(state)
    allowed = (token <= at[..., None])  # [seqs, rows, tokens]
    allowed = allowed.repeat_interleave(case["hq"] // case["hkv"], 1)[:, None]
    o, lse = _attend(state, allowed)
    return {"o": o, "lse": lse}


def _moba(state):
    case = state["case"]
    n, rows, hq, hkv, d, k = (case[x] for x in ("seqs", "rows", "hq", "hkv", "d", "topk"))
    r, block, per = hq // hkv, case["block"], case["block"] // case["page"]
    at, token = _places(state)
    here = at.div(block, rounding_mode="floor").repeat_interleave(r, 1)[:, None, :, None]
    home = state["page_table"][:, ::per].long().clamp(min=0)
    nb = home.shape[1]
    # scores in 64 bits: a selection must not hang on rounding. The mean's 1/block is common.
    sums = state["block_sums"][home].double().permute(0, 2, 3, 1)
    q = state["q"].double().view(n, rows, hkv, r, d).transpose(1, 2).flatten(2, 3)
    j = torch.arange(nb, device=DEV)
    score = (q @ sums).masked_fill(j >= here, -math.inf)  # [n, hkv, rows r, nb]
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :k - 1]
    chosen = torch.zeros(score.shape, dtype=torch.bool, device=DEV).scatter_(-1, order, True)
    chosen = (chosen & (j < here)) | (j == here)
    pad = torch.where(chosen, j, nb).sort(-1).values[..., :k]
    if nb < k:
        pad = torch.cat([pad, pad.new_full((*pad.shape[:-1], k - nb), nb)], -1)
    idx = torch.where(pad == nb, -1, pad).to(torch.int32)
    idx = idx.view(n, hkv, rows, r, k).permute(1, 3, 0, 2, 4).reshape(hq, n * rows, k)
    allowed = chosen[..., token // block]
    allowed &= (token <= at[..., None]).repeat_interleave(r, 1)[:, None]
    o, lse = _attend(state, allowed)
    return {"o": o, "lse": lse, "block_idx": idx.contiguous()}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "append": _append,
                "read": _read, "attn": _attn, "moba": _moba}[op](state)
    from block_sparse_long_moba_b200 import moba
    if op == "norm_rope":
        q, k = moba.moba_qk_norm_rope(
            state["q"], state["k"], state["q_weight"], state["k_weight"], state["rope"],
            state["positions"], eps=EPS, interleaved=case["pairs"] == "adjacent")
        return {"q": q, "k": k}
    if op == "norm_rope_bwd":
        dq, dk, dqw, dkw = moba.moba_qk_norm_rope_bwd(
            state["q"], state["k"], state["q_weight"], state["k_weight"], state["rope"],
            state["positions"], state["d_q"], state["d_k"], eps=EPS,
            interleaved=case["pairs"] == "adjacent")
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    cache = state["cache"]
    if op == "append":
        moba.moba_cache_append(cache, state["k"], state["v"], state["cu_q"])
        return _cache_outputs(state)
    if op == "read":
        k, v = moba.moba_cache_read(cache, state["cu"], state["cu_host"])
        return {"k": k, "v": v}
    if op == "attn":
        o, lse = moba.moba_paged_attn_fwd(cache, state["q"], rows_per_seq=case["rows"])
        return {"o": o, "lse": lse}
    idx = torch.empty((case["hq"], state["q"].shape[0], case["topk"]), dtype=torch.int32,
                      device=state["q"].device)
    o, lse = moba.moba_paged_decode_fwd(cache, state["q"], case["topk"],
                                        rows_per_seq=case["rows"], block_idx_out=idx)
    return {"o": o, "lse": lse, "block_idx": idx}


# ------------------------------------------------------------------------------------------ work
def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op.startswith("norm_rope"):
        heads = case["hq"] + hkv
        n = case["tokens"] * heads * d
        # table rows of the positions in use: each once
        table = 4 * case["rot"] * min(case["tokens"], max(1, case["tokens"] // 3 + 1))
        if op == "norm_rope":
            return {"bytes": 4 * n + table + 4 * case["tokens"], "flops": 8 * n}
        return {"bytes": 6 * n + table + 4 * case["tokens"], "flops": 16 * n}
    lens, new = _lengths(case)
    row = 2 * d if case["kv"] == "bf16" else d + 1  # bytes of one cached key or value
    if op == "append":
        n = sum(new) * hkv
        touched = sum((x - 1) // case["block"] - (x - y) // case["block"] + 1
                      for x, y in zip(lens, new))
        return {"bytes": 2 * n * (2 * d + row) + 4 * touched * hkv * d, "flops": 5 * n * d}
    if op == "read":
        n = sum(lens) * hkv
        return {"bytes": 2 * n * (2 * d + row), "flops": 2 * n * d}
    rows, hq = case["rows"], case["hq"]
    io = case["seqs"] * rows * hq * (4 * d + 4)
    if op == "attn":
        n = sum(lens) * hkv
        return {"bytes": 2 * n * row + io, "flops": 4 * rows * (hq // hkv) * n * d}
    total = flops = 0
    for x in lens:
        cur = (x - 1) // case["block"]
        tail = x - cur * case["block"]
        pick = min(case["topk"] - 1, cur)
        # blocks that at least one of the rows of a kv head selects: each head's choice of pick
        # of cur blocks taken as independent and uniform
        union = cur * (1 - (1 - pick / cur) ** (rows * hq // hkv)) if cur else 0
        total += hkv * (2 * row * (union * case["block"] + tail) + 4 * d * cur)
        flops += rows * hq * (4 * d * (pick * case["block"] + tail) + 2 * d * cur)
    return {"bytes": total + io, "flops": flops}


# --------------------------------------------------------------------------- the results, exactly
def _exact_norm(x, w, rope, pos, case):
    x, w, rope = x.double(), w.double(), rope.double()
    z = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    half = case["rot"] // 2
    i = torch.arange(half, device=DEV)
    first, second = (i, i + half) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
    turn = torch.complex(rope[:, :half], rope[:, half:])[pos.long()][:, None]
    y = torch.complex(z[..., first], z[..., second]) * turn
    out = z.clone()
    out[..., first] = y.real
    out[..., second] = y.imag
    return out


def _exact_tokens(state, n, s, count):
    """The first count keys or values of sequence s, [count, hkv, d] in 64 bits."""
    page = state["case"]["page"]
    ids = state["page_table"][s, :-(-count // page)].long()
    x = state[n + "_cache"][ids] if state[n + "_scale"] is None else \
        state[n + "_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    x = x.double()
    if state[n + "_scale"] is not None:
        x = x * torch.pow(2.0, state[n + "_scale"][ids].double() - 127)[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:count]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        rest = (state["rope"], state["positions"], case)
        return {n: _exact_norm(state[n], state[n + "_weight"], *rest) for n in ("q", "k")}
    if op == "norm_rope_bwd":
        out = {}
        for n in ("q", "k"):
            x = state[n].double().requires_grad_(True)
            w = state[n + "_weight"].double().requires_grad_(True)
            y = _exact_norm(x, w, state["rope"], state["positions"], case)
            dx, dw = torch.autograd.grad(y, (x, w), state["d_" + n].double())
            out["d" + n], out["d" + n + "_weight"] = dx, dw
        return out
    lens, new = _lengths(case)
    if op == "append":
        # pages hold what was given (rounded to 8 bits: no 64-bit value); sums in 64 bits
        page, block = case["page"], case["block"]
        sums = state["block_sums"].double()
        cu = _offsets(new)
        k = state["k"].double()
        for s, (x, y) in enumerate(zip(lens, new)):
            for b in range((x - y) // block, (x - 1) // block + 1):
                lo, hi = max(b * block, x - y), min((b + 1) * block, x)
                home = int(state["page_table"][s, b * (block // page)])
                add = k[cu[s] + lo - (x - y):cu[s] + hi - (x - y)].sum(0)
                sums[home] = add + (sums[home] if lo > b * block else 0)
        out = {"k_cache": None, "v_cache": None, "block_sums": sums}
        return {**out, "k_scale": None, "v_scale": None} if case["kv"] == "e4m3" else out
    if op == "read":
        return {n: torch.cat([_exact_tokens(state, n, s, x) for s, x in enumerate(lens)])
                for n in ("k", "v")}
    rows, hq, hkv, d, block = (case[x] for x in ("rows", "hq", "hkv", "d", "block"))
    o = torch.zeros((case["seqs"] * rows, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((hq, case["seqs"] * rows), -math.inf, dtype=torch.float64, device=DEV)
    for s, x in enumerate(lens):
        k, v = (_exact_tokens(state, n, s, x) for n in ("k", "v"))
        for i in range(rows):
            at = x - rows + i
            if at < 0:
                continue
            cur = at // block
            homes = state["page_table"][s, ::block // case["page"]].long()[:cur]
            for h in range(hq):
                g, q = h // (hq // hkv), state["q"][s * rows + i, h].double()
                keys, values = k[:at + 1, g], v[:at + 1, g]
                if op == "moba" and cur > case["topk"] - 1:
                    score = state["block_sums"][homes, g].double() @ q
                    pick = score.sort(dim=0, descending=True, stable=True).indices[:case["topk"] - 1]
                    pick = torch.cat([pick.sort().values, pick.new_tensor([cur])])
                    at_token = (pick[:, None] * block + torch.arange(block, device=DEV)).flatten()
                    at_token = at_token[at_token <= at]
                    keys, values = keys[at_token], values[at_token]
                z = keys @ q / math.sqrt(d)
                lse[h, s * rows + i] = z.logsumexp(0)
                o[s * rows + i, h] = z.softmax(0) @ values
    out = {"o": o, "lse": lse}
    return {**out, "block_idx": None} if op == "moba" else out
