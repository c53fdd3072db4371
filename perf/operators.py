"""Attention over a paged KV cache, the attention mass each cached token
gathers, and the eviction of cached tokens by that mass: cases, inputs, plain
forms and the framework's calls.

A case's request lengths run evenly from its lowest to its highest length (in
an order drawn from the seed), so its work does not depend on the seed.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def _attn(name, **kw):
    c = dict(name=name, op="attention", requests=64, len_lo=512, len_hi=4096, new_lo=1, new_hi=1,
             q_heads=32, kv_heads=8, head_dim=128, block_size=16, layout="NHD", kv="bf16",
             softcap=0.0, window=0)
    c.update(kw)
    return c


def _mass(name, **kw):
    c = _attn(name, **kw)
    c["op"] = "mass"
    c.setdefault("observe", 0)
    return c


def _evict(name, **kw):
    c = dict(name=name, op="evict", layers=8, requests=16, len_lo=512, len_hi=4096, keep=1024,
             sinks=4, recent=64, kv_heads=8, head_dim=128, block_size=16, layout="NHD", kv="bf16",
             in_place=True, words=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a full batch: Llama-3-8B-shaped, one token a request
        _attn("decode_8b"),
        # one chat at its first answer tokens: latency counts
        _attn("decode_one", requests=1, len_lo=709, len_hi=709),
        # fp8 cache of the 70B-shaped workload (64 query heads, 8 to a KV head)
        _attn("decode_70b_fp8", requests=128, len_lo=2048, len_hi=2048, q_heads=64, kv="fp8"),
        # two long documents in large HND blocks, two tokens drafted ahead
        _attn("decode_long_hnd", requests=2, len_lo=99001, len_hi=131072, new_lo=3, new_hi=3,
              block_size=64, layout="HND"),
        # chunked prefill: 2048 new tokens a request over a long cache
        _attn("chunk_8b", requests=4, len_lo=8192, len_hi=8192, new_lo=2048, new_hi=2048),
        # ragged mixed batch (some decode, some prefill), odd sizes, capped scores, sliding window
        _attn("mixed_capped", requests=13, len_lo=33, len_hi=5001, new_lo=1, new_hi=777, q_heads=16,
              kv_heads=2, head_dim=64, kv="fp16", softcap=30.0, window=1024),
        # accumulated attention weight of a decode step
        _mass("mass_decode_8b"),
        # ... of a whole chunk (all its queries are observed)
        _mass("mass_chunk_8b", requests=4, len_lo=8192, len_hi=8192, new_lo=2048, new_hi=2048),
        # ... of the last 32 queries of a ragged prefill, HND
        _mass("mass_window_hnd", requests=7, len_lo=311, len_hi=9000, new_lo=100, new_hi=300,
              observe=32, layout="HND", block_size=32),
        # evict every layer's cache of a batch down to a budget, in place
        _evict("evict_8b"),
        # one short request, one layer: latency counts
        _evict("evict_one", layers=1, requests=1, len_lo=613, len_hi=613, keep=512),
        # into fresh blocks, with the new blocks' checksum words; HND
        _evict("evict_fresh_hnd", layers=4, requests=3, len_lo=6001, len_hi=20011, keep=4096,
               layout="HND", block_size=64, in_place=False, words=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "mass", "mass", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8])
    head_dim = rng.choice([64, 128, 128])
    layout = rng.choice(["NHD", "NHD", "HND", "XSPLIT"])
    block_size = rng.choice([8, 16, 16, 32, 48, 64])
    kv = rng.choice(["bf16", "bf16", "fp16", "fp8"])
    if op == "evict":
        layers = rng.choice([1, 2, 5, 8])
        hi = _log(rng, 70, 16000)
        lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
        cap = max(1, min(32, int(16 * 8 * 8 * 2304 / (layers * kv_heads * hi))))
        return dict(op=op, layers=layers, requests=_log(rng, 1, cap), len_lo=lo, len_hi=hi,
                    keep=max(1, int(hi * rng.uniform(0.05, 0.9))), sinks=rng.choice([0, 1, 4]),
                    recent=rng.choice([0, 16, 33, 64]), kv_heads=kv_heads, head_dim=head_dim,
                    block_size=block_size, layout=rng.choice([layout, "LATENT"]), kv=kv,
                    in_place=rng.random() < 0.6, words=rng.random() < 0.5)
    group = rng.choice([1, 2, 4, 4, 8, 5])
    q_heads = group * kv_heads
    new = 1 if rng.random() < 0.45 else _log(rng, 2, 2048)
    hi = max(new, _log(rng, 65, 60000 if new <= 8 else 12000))
    lo = max(1, min(hi, int(hi * rng.uniform(0.2, 1.0))))
    pairs = 4 * 2048 * 8192 * 32 / 2
    cap = max(1, min(256, int(pairs / (new * hi * q_heads)), int(2 ** 28 / (hi * kv_heads * head_dim))))
    c = dict(op=op, requests=_log(rng, 1, cap), len_lo=lo, len_hi=hi,
             new_lo=rng.choice([1, max(1, new // 2), new]), new_hi=new, q_heads=q_heads,
             kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, layout=layout, kv=kv,
             softcap=rng.choice([0.0, 0.0, 0.0, 25.0]),
             window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
    if op == "mass":
        c["observe"] = rng.choice([0, 0, 16, 32])
    return c


def _spread(lo, hi, n):
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _requests(case):
    """(cached tokens, new tokens) of each request; short chunks fall on long caches and short ones."""
    R = case["requests"]
    lengths = _spread(case["len_lo"], case["len_hi"], R)
    if case["op"] == "evict":
        return [(t, 0) for t in lengths]
    new = _spread(case["new_lo"], case["new_hi"], R)
    return [(t, min(t, new[(r * (R // 2 + 1) + R // 3) % R])) for r, t in enumerate(lengths)]


def _element_bytes(case):
    return 1 if case["kv"] == "fp8" else 2


def _geometry(case):
    """(halves, heads, elements a head holds) of the case's pools."""
    if case["layout"] == "LATENT":
        return 1, 1, 576
    return 2, case["kv_heads"], case["head_dim"]


def _pool_shape(case, nb):
    halves, H, D = _geometry(case)
    bs, x = case["block_size"], 16 // _element_bytes(case)
    return {"NHD": (halves, nb, bs, H, D), "HND": (halves, nb, H, bs, D),
            "XSPLIT": (halves, nb, H, D // x, bs, x),
            "LATENT": (halves, nb, bs, H, D)}[case["layout"]]


def _by_token(pool, layout):
    """A pool of any layout as a view [..., halves, blocks, slots, heads, (elements)]."""
    n = pool.dim()
    if layout == "HND":
        return pool.transpose(n - 3, n - 2)
    if layout == "XSPLIT":
        lead = list(range(n - 5))
        return pool.permute(*lead, n - 5, n - 2, n - 4, n - 3, n - 1)
    return pool


def _fill(shape, dtype, gen):
    if dtype == torch.float8_e4m3fn:
        return torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=gen).to(dtype)
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)


def _tables(case, rng, lengths, spare):
    """Request tables in CSR form over a pool with some blocks to spare."""
    bs = case["block_size"]
    counts = [-(-n // bs) for n in lengths]
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    total = offsets[-1]
    nb = total + spare(total)
    ids = np.random.RandomState(rng.randrange(1 << 31)).permutation(nb).astype(np.int32)
    return offsets, total, nb, ids


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = "cuda"
    R, bs = case["requests"], case["block_size"]
    requests = _requests(case)
    rng.shuffle(requests)
    lengths = [t for t, _ in requests]
    kv = DTYPES[case["kv"]]
    evict = case["op"] == "evict"
    offsets, total, nb, ids = _tables(case, rng, lengths,
                                      lambda t: t + 5 if evict and not case["in_place"] else 5)
    s = dict(case=case, lengths=lengths, num_blocks=nb, total_positions=total,
             max_len=max(lengths), max_positions=max(b - a for a, b in zip(offsets, offsets[1:])),
             pos_offsets=torch.tensor(offsets, dtype=torch.int64, device=dev),
             first_position=torch.zeros(R, dtype=torch.int64, device=dev),
             num_tokens=torch.tensor(lengths, dtype=torch.int64, device=dev),
             block_ids=torch.from_numpy(ids[:total].copy()).to(dev))
    _, H, D = _geometry(case)
    if evict:
        L = case["layers"]
        s["pool"] = _fill((L,) + _pool_shape(case, nb), kv, gen)
        # what attention leaves behind: most tokens gather little, a few much
        s["scores"] = torch.rand((L, nb, H, bs), device=dev, generator=gen).pow_(6).mul_(20)
        s["keep"] = torch.full((R,), case["keep"], dtype=torch.int64, device=dev)
        s["kept"] = [min(case["keep"], n) for n in lengths]
        s["total_kept"] = sum(s["kept"])
        s["new_block_ids"] = (None if case["in_place"]
                              else torch.from_numpy(ids[total:2 * total].copy()).to(dev))
        s["block_sums"] = (torch.zeros(nb, dtype=torch.int64, device=dev)
                           if case["words"] else None)
        return s
    new = [n for _, n in requests]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s.update(new=new, total_new=starts[-1], max_new=max(new),
             new_offsets=torch.tensor(starts, dtype=torch.int64, device=dev),
             pool=_fill(_pool_shape(case, nb), kv, gen),
             scale=1.0 / math.sqrt(D),
             k_scale=0.75 if case["kv"] == "fp8" else 1.0,
             v_scale=1.25 if case["kv"] == "fp8" else 1.0,
             q=torch.randn((starts[-1], case["q_heads"], D),
                           dtype=torch.float16 if case["kv"] == "fp16" else torch.bfloat16,
                           device=dev, generator=gen))
    if case["op"] == "mass":
        # the attention call before this one has left these
        _, s["lse"] = _plain_attention(s)
        s["mass"] = torch.rand((nb, H, bs), device=dev, generator=gen)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _slots(s):
    """Block and slot of every token, [R, max_len], and which tokens exist."""
    bs = s["case"]["block_size"]
    t = torch.arange(s["max_len"], device="cuda")
    at = s["pos_offsets"][:-1, None] + t[None, :] // bs
    blk = s["block_ids"].long()[at.clamp(max=s["total_positions"] - 1)]
    return blk, (t % bs).expand_as(blk), t[None, :] < s["num_tokens"][:, None]


def _queries(s):
    """(request of each new token, its index there), both [total_new]."""
    counts = s["new_offsets"][1:] - s["new_offsets"][:-1]
    R = counts.numel()
    req = torch.repeat_interleave(torch.arange(R, device="cuda"), counts,
                                  output_size=s["total_new"])
    i = torch.arange(s["total_new"], device="cuda") - s["new_offsets"][req]
    return req, i, counts


def _gathered(s, half, blk, slot, exists):
    """[R, heads, max_len, head_dim] in fp32, zeros where no token exists."""
    v = _by_token(s["pool"], s["case"]["layout"])[half]
    if v.dtype == torch.float8_e4m3fn:
        rows = v.view(torch.uint8)[blk, slot].view(torch.float8_e4m3fn)
    else:
        rows = v[blk, slot]
    rows = rows.to(torch.float32).reshape(*blk.shape, s["case"]["kv_heads"], s["case"]["head_dim"])
    return torch.where(exists[:, :, None, None], rows, 0.0).transpose(1, 2)


def _plain_scores(s, blk, slot, exists):
    """Capped scores [R, heads, max_new, group, max_len], -inf where masked."""
    c = s["case"]
    R, H, D = c["requests"], c["kv_heads"], c["head_dim"]
    G = c["q_heads"] // H
    req, i, counts = _queries(s)
    q = torch.zeros((R, s["max_new"], c["q_heads"], D), device="cuda")
    q[req, i] = s["q"].to(torch.float32)
    q = q.view(R, s["max_new"], H, G, D).transpose(1, 2).reshape(R, H, s["max_new"] * G, D)
    k = _gathered(s, 0, blk, slot, exists)
    sc = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] * s["k_scale"])
    if c["softcap"] > 0:
        sc = c["softcap"] * torch.tanh(sc / c["softcap"])
    sc = sc.view(R, H, s["max_new"], G, s["max_len"])
    at = s["num_tokens"][:, None] - counts[:, None] + torch.arange(s["max_new"], device="cuda")
    t = torch.arange(s["max_len"], device="cuda")
    see = exists[:, None, :] & (t <= at[:, :, None])
    if c["window"] > 0:
        see = see & (t > at[:, :, None] - c["window"])
    return sc.masked_fill_(~see[:, None, :, None, :], float("-inf")), req, i, counts


def _plain_attention(s):
    c = s["case"]
    blk, slot, exists = _slots(s)
    sc, req, i, _ = _plain_scores(s, blk, slot, exists)
    R, H, n, G, T = sc.shape
    top = sc.amax(dim=-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = sc.sub_(top).exp_()
    total = p.sum(dim=-1)
    v = _gathered(s, 1, blk, slot, exists)
    o = torch.matmul(p.view(R, H, n * G, T), v).view(R, H, n, G, -1)
    o = o * torch.where(total > 0, s["v_scale"] / total, 0.0)[..., None]
    lse = top[..., 0] + torch.log(total)
    o = o.permute(0, 2, 1, 3, 4).reshape(R, n, c["q_heads"], -1)
    lse = lse.permute(0, 2, 1, 3).reshape(R, n, c["q_heads"])
    return o[req, i].to(s["q"].dtype), lse[req, i]


def _plain_mass(s):
    c = s["case"]
    blk, slot, exists = _slots(s)
    sc, req, i, counts = _plain_scores(s, blk, slot, exists)
    R, H, n, G, T = sc.shape
    lse = torch.full((R, n, c["q_heads"]), float("inf"), device="cuda")
    seen = i >= counts[req] - (c["observe"] if c["observe"] > 0 else s["max_new"])
    lse[req, i] = torch.where(seen[:, None], s["lse"], float("inf"))
    lse = lse.view(R, n, H, G).transpose(1, 2)
    add = sc.sub_(lse[..., None]).exp_().sum(dim=(2, 3))                  # [R, H, T]
    add = torch.where(exists[:, None, :], add, 0.0).transpose(1, 2)       # [R, T, H]
    # tokens that do not exist add nothing, wherever their index points
    s["mass"].transpose(1, 2).index_put_((blk, slot), add, accumulate=True)
    return s["mass"]


def _plain_evict(s):
    c = s["case"]
    bs, R, L = c["block_size"], c["requests"], c["layers"]
    _, H, _ = _geometry(c)
    blk, slot, exists = _slots(s)
    T = s["max_len"]
    t = torch.arange(T, device="cuda")
    N = s["num_tokens"]
    B = torch.minimum(s["keep"], N)
    sinks = B.clamp(max=c["sinks"])
    recent = (B - sinks).clamp(max=c["recent"])
    kind = torch.where((t < sinks[:, None]) | (t >= (N - recent)[:, None]), 2, 1)
    kind = torch.where(exists, kind, 0)                                   # [R, T]
    by_slot = s["scores"].transpose(2, 3)                                 # [L, nb, bs, H]
    score = by_slot[:, blk, slot].permute(0, 1, 3, 2)                     # [L, R, H, T]
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    kinds = torch.gather(kind[None, :, None, :].expand(L, R, H, T), -1, order)
    order = torch.gather(order, -1, torch.sort(kinds, dim=-1, descending=True,
                                               stable=True).indices)
    top = (t < B[:, None])[None, :, None, :].expand(L, R, H, T)
    kept = torch.zeros((L, R, H, T), dtype=torch.bool, device="cuda").scatter_(-1, order, top)
    first = torch.sort(~kept, dim=-1, stable=True).indices                # kept ones first, in order

    r_of = torch.repeat_interleave(torch.arange(R, device="cuda"), B, output_size=s["total_kept"])
    ends = torch.cumsum(B, 0)
    j_of = torch.arange(s["total_kept"], device="cuda") - (ends - B)[r_of]
    src = first[:, r_of, :, j_of].permute(1, 2, 0)                        # [L, H, kept]
    po = s["pos_offsets"][r_of]
    to_ids = s["block_ids"] if s["new_block_ids"] is None else s["new_block_ids"]
    src_blk = s["block_ids"].long()[po + src // bs]
    dst_blk = to_ids.long()[po + j_of // bs].expand_as(src_blk)
    dst_slot = (j_of % bs).expand_as(src_blk)
    li = torch.arange(L, device="cuda")[:, None, None]
    hi = torch.arange(H, device="cuda")[None, :, None]
    raw = s["pool"].view(torch.uint8) if c["kv"] == "fp8" else s["pool"]
    pool = _by_token(raw, c["layout"])
    rows = pool[li, :, src_blk, src % bs, hi]                             # [L, H, kept, halves, ...]
    kept_scores = by_slot[li, src_blk, src % bs, hi]
    pool[li, :, dst_blk, dst_slot, hi] = rows
    by_slot[li, dst_blk, dst_slot, hi] = kept_scores
    out = [s["pool"], s["scores"]]
    if s["block_sums"] is not None:
        x = rows.reshape(L, H, s["total_kept"], -1).view(torch.int64)
        P = x.shape[-1]
        w = 2 * ((s["first_position"][r_of] * bs + j_of)[:, None] * P
                 + torch.arange(P, device="cuda")) + 1
        m = 2 * (li * 65536 + hi) + 1
        per_token = ((x * w).sum(-1) * m).sum(dim=(0, 1))
        if c["in_place"]:
            s["block_sums"][to_ids.long()] = 0
        s["block_sums"][dst_blk[0, 0]] = 0
        s["block_sums"].index_add_(0, dst_blk[0, 0], per_token)
        out.append(s["block_sums"])
    return out


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _cache(s, pool, layer):
    from paged_kv_cache_kvcs_gb300 import workloads as W
    c = s["case"]
    _, H, D = _geometry(c)
    layout = {"NHD": W.LAYOUT_NHD, "HND": W.LAYOUT_HND, "XSPLIT": W.LAYOUT_XSPLIT,
              "LATENT": W.LAYOUT_LATENT}[c["layout"]]
    return W.CacheSpec(pool, s["num_blocks"], layout, layer, 0, H, D * _element_bytes(c))


def _own(s):
    import paged_kv_cache_kvcs_gb300 as K
    c = s["case"]
    table = (s["pos_offsets"], s["first_position"], s["num_tokens"], s["block_ids"])
    if c["op"] == "evict":
        caches = [_cache(s, s["pool"][i], i) for i in range(c["layers"])]
        K.evict(caches, c["block_size"], *table, list(s["scores"].unbind(0)), s["keep"],
                sinks=c["sinks"], recent=c["recent"], new_block_ids=s["new_block_ids"],
                block_sums=s["block_sums"], total_positions=s["total_positions"])
        out = [s["pool"], s["scores"]]
        return out if s["block_sums"] is None else out + [s["block_sums"]]
    common = dict(scale=s["scale"], softcap=c["softcap"], window=c["window"],
                  k_scale=s["k_scale"], kv_dtype=DTYPES[c["kv"]], max_new=s["max_new"],
                  total_positions=s["total_positions"])
    cache = _cache(s, s["pool"], 0)
    if c["op"] == "mass":
        K.attention_mass(cache, c["block_size"], *table, s["q"], s["new_offsets"], s["lse"],
                         s["mass"], observe=c["observe"], **common)
        return s["mass"]
    return K.paged_attention(cache, c["block_size"], *table, s["q"], s["new_offsets"],
                             v_scale=s["v_scale"], **common)


def run(state):
    if own:
        r = _own(state)
    elif state["case"]["op"] == "attention":
        r = _plain_attention(state)
    elif state["case"]["op"] == "mass":
        r = _plain_mass(state)
    else:
        r = _plain_evict(state)
    if state["case"]["kv"] == "fp8" and state["case"]["op"] == "evict":
        r = [r[0].view(torch.uint8)] + list(r[1:])      # moved bytes, compared as they are
    return list(r) if isinstance(r, (list, tuple)) else r


# ---------------------------------------------------------------------------
# Work, and the definition in 64 bits
# ---------------------------------------------------------------------------

def _visible(case):
    """(cached tokens some query sees, (query, token) pairs seen, queries), over the requests."""
    tokens = pairs = queries = 0
    for t, n in _requests(case):
        if case.get("observe", 0) > 0:
            n = min(n, case["observe"])
        w = case["window"] or t
        first = max(0, t - n + 1 - w)
        tokens += t - first
        pairs += sum(min(w, p + 1) for p in range(t - n, t))
        queries += n
    return tokens, pairs, queries


def work(case):
    halves, H, D = _geometry(case)
    es = _element_bytes(case)
    if case["op"] == "evict":
        lengths = [t for t, _ in _requests(case)]
        rows = case["layers"] * H
        kept = sum(min(case["keep"], n) for n in lengths if n > case["keep"] or case["words"]
                   or not case["in_place"])
        read = sum(n for n in lengths if n > case["keep"])
        return {"bytes": rows * (4 * read + kept * (2 * halves * D * es + 4)), "flops": 0}
    tokens, pairs, queries = _visible(case)
    if case["op"] == "mass":
        return {"bytes": tokens * H * (D * es + 8) + queries * case["q_heads"] * (2 * D + 4),
                "flops": 2 * D * case["q_heads"] * pairs}
    return {"bytes": tokens * H * 2 * D * es + queries * case["q_heads"] * (4 * D + 4),
            "flops": 4 * D * case["q_heads"] * pairs}


def _rows64(s, half, r, h):
    """Request r's rows of one head and half, float64 [tokens, elements], read block by block."""
    c, bs, n = s["case"], s["case"]["block_size"], s["lengths"][r]
    lo = int(s["pos_offsets"][r])
    ids = s["block_ids"][lo:lo + -(-n // bs)].long()
    p = s["pool"][half]
    if c["kv"] == "fp8":
        p = p.view(torch.uint8)
    if c["layout"] == "HND":
        rows = p[ids, h].reshape(-1, p.shape[-1])
    elif c["layout"] == "XSPLIT":
        rows = p[ids, h].permute(0, 2, 1, 3).reshape(ids.numel() * bs, -1)
    else:
        rows = p[ids, :, h].reshape(-1, p.shape[-1])
    if c["kv"] == "fp8":
        rows = rows.view(torch.float8_e4m3fn)
    return rows[:n].double()


def _exact_attention(s):
    c = s["case"]
    G = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if c["op"] == "mass" else None
    for r, (n, t) in enumerate(zip(s["new"], s["lengths"])):
        lo = int(s["new_offsets"][r])
        seen = min(n, c.get("observe", 0) or n)
        at = torch.arange(t - n, t, device="cuda")[:, None]
        key = torch.arange(t, device="cuda")[None, :]
        hidden = (key > at) | (key <= at - (c["window"] or t))
        for h in range(c["kv_heads"]):
            k, v = _rows64(s, 0, r, h), _rows64(s, 1, r, h)
            for g in range(h * G, h * G + G):
                z = s["q"][lo:lo + n, g].double() @ k.T * s["scale"] * s["k_scale"]
                if c["softcap"] > 0:
                    z = torch.tanh(z / c["softcap"]) * c["softcap"]
                z[hidden] = float("-inf")
                if mass is not None:
                    e = torch.exp(z - s["lse"][lo:lo + n, g].double()[:, None])[n - seen:].sum(0)
                    ids = s["block_ids"][int(s["pos_offsets"][r]):int(s["pos_offsets"][r + 1])]
                    full = torch.zeros(ids.numel() * c["block_size"], dtype=torch.float64,
                                       device="cuda")
                    full[:t] = e
                    mass[ids.long(), h] += full.view(ids.numel(), -1)
                else:
                    l = torch.logsumexp(z, 1)
                    lse[lo:lo + n, g] = l
                    out[lo:lo + n, g] = torch.exp(z - l[:, None]) @ v * s["v_scale"]
    return [out, lse] if mass is None else mass


def _exact_evict(s):
    c = s["case"]
    bs = c["block_size"]
    halves, H, D = _geometry(c)
    raw = s["pool"].view(torch.uint8).cpu().numpy()
    es = _element_bytes(c)
    scores, ids = s["scores"].cpu().numpy(), s["block_ids"].cpu().numpy()
    to = ids if s["new_block_ids"] is None else s["new_block_ids"].cpu().numpy()
    po = s["pos_offsets"].tolist()
    by, sc = raw.copy(), scores.copy()
    words = None if s["block_sums"] is None else np.zeros(s["num_blocks"], np.uint64)

    def place(blk, slot, h):
        if c["layout"] == "HND":
            return (slice(None), blk, h, slot)
        if c["layout"] == "XSPLIT":
            return (slice(None), blk, h, slice(None), slot)
        return (slice(None), blk, slot, h)

    for r, n in enumerate(s["lengths"]):
        B = min(c["keep"], n)
        a = min(c["sinks"], B)
        w = min(c["recent"], B - a)
        t = np.arange(n)
        blk, slot = ids[po[r] + t // bs], t % bs
        j = np.arange(B)
        dst, dslot = to[po[r] + j // bs], j % bs
        for l in range(c["layers"]):
            for h in range(H):
                mid = np.arange(a, n - w)
                best = mid[np.lexsort((mid, -scores[l][blk[mid], h, slot[mid]]))][:B - a - w]
                keep = np.concatenate([np.arange(a), np.sort(best), np.arange(n - w, n)])
                # the copy is indexed by (half, token); numpy puts sliced axes as they stand
                for half in range(halves):
                    src = place(blk[keep], slot[keep], h)[1:]
                    vals = raw[l, half][src]
                    by[l, half][place(dst, dslot, h)[1:]] = vals
                    if words is not None:
                        x = np.ascontiguousarray(vals.reshape(B, -1)).view(np.uint64)
                        hp = x.shape[1]
                        p = np.arange(hp, dtype=np.uint64) + np.uint64(half * hp)
                        wgt = (j.astype(np.uint64)[:, None] * np.uint64(halves * hp) + p) \
                            * np.uint64(2) + np.uint64(1)
                        tok = (x * wgt).sum(1, dtype=np.uint64) * np.uint64(2 * (l * 65536 + h) + 1)
                        np.add.at(words, dst, tok)
                sc[l, dst, h, dslot] = scores[l, blk[keep], h, slot[keep]]
    moved = torch.from_numpy(by)
    if c["kv"] != "fp8":
        moved = moved.view(DTYPES[c["kv"]])
    out = [moved, torch.from_numpy(sc).double()]
    return out if words is None else out + [torch.from_numpy(words.view(np.int64))]


def exact(case, seed):
    if case["op"] == "evict":
        halves, H, D = _geometry(case)
        if case["layers"] * H * case["requests"] > 4000:
            return None
        return _exact_evict(prepare(case, seed))
    pairs = sum(n * t for t, n in _requests(case))
    if pairs * case["q_heads"] * case["head_dim"] * 4 > 4e12 or \
            case["requests"] * case["q_heads"] > 20000:
        return None
    return _exact_attention(prepare(case, seed))
