"""kvcs_evict, byte for byte against the definition, its words against the
checksum oracle, and a run of the cache's operators together."""

import math

import pytest
import torch

import attention_ref as A
import paged_kv_cache_kvcs_gb300 as K
from helpers import W, OracleCache, OracleRequests, c_form, host_bytes

pytestmark = pytest.mark.gpu
NHD, HND, XS, LAT = W.LAYOUT_NHD, W.LAYOUT_HND, W.LAYOUT_XSPLIT, W.LAYOUT_LATENT


def make(seed=0, layers=2, lengths=(100, 37, 260), spare=60, scores="random", **kw):
    """Caches of several layers sharing one block table, and their scores."""
    cases = [A.Case(seed=seed, layer=l, lengths=lengths, new=[0] * len(lengths), spare=spare,
                    tail=1.5, **kw) for l in range(layers)]
    g = torch.Generator().manual_seed(seed + 99)
    sc = []
    for c in cases:
        x = torch.randn((c.nb, c.heads, c.bs), generator=g)
        if scores == "ties":
            x = torch.randint(0, 3, x.shape, generator=g).float() - 1
            x[torch.rand(x.shape, generator=g) < 0.2] = -0.0
        if scores == "odd":
            u = torch.rand(x.shape, generator=g)
            x[u < 0.1] = float("nan")
            x[(u > 0.1) & (u < 0.2)] = float("inf")
            x[(u > 0.2) & (u < 0.3)] = -float("inf")
        sc.append(x.cuda())
    return cases, sc


def expected(cases, sc, keep, sinks, recent, to_ids=None):
    """Pools and scores after the eviction."""
    pools = [c.pool.cpu().clone() for c in cases]
    scores = [s.cpu().clone() for s in sc]
    for c, pool, s in zip(cases, pools, scores):
        halves = 1 if c.layout == LAT else 2
        src_pool, src_s = pool.clone(), s.clone()
        for r, T in enumerate(c.lengths):
            N = c.values[r].shape[1]
            B = min(keep[r], N)
            ids = c.ids[c.offsets[r]:c.offsets[r + 1]].long()
            to = ids if to_ids is None else to_ids[c.offsets[r]:c.offsets[r + 1]].long()
            t = torch.arange(N)
            for h in range(c.heads):
                row = src_s[ids[t // c.bs], h, t % c.bs].tolist()
                src = torch.tensor(A.kept_tokens(row, N, B, sinks, recent), dtype=torch.long)
                j = torch.arange(B)
                for half in range(halves):
                    a = c.offsets_map[half][ids[src // c.bs], src % c.bs, h]
                    b = c.offsets_map[half][to[j // c.bs], j % c.bs, h]
                    pool[b] = src_pool[a]
                s[to[j // c.bs], h, j % c.bs] = src_s[ids[src // c.bs], h, src % c.bs]
    return pools, scores


def evict(cases, sc, keep, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = cases[0]
    K.evict([x.cache for x in cases], c.bs, *c.table, sc,
            torch.tensor(keep, dtype=torch.int64, device="cuda"), status=status, **kw)
    torch.cuda.synchronize()
    return int(status.item())


def same(cases, sc, want):
    for c, s, p, w in zip(cases, sc, *want):
        assert torch.equal(c.pool.cpu(), p)
        assert torch.equal(s.cpu().view(torch.int32), w.view(torch.int32))


@pytest.mark.parametrize("layout,kw", [
    (NHD, {}), (HND, {}), (HND, dict(kbs=4)), (XS, {}), (LAT, dict(heads=1, dim=576, halves=1)),
    (NHD, dict(interleaved=True)), (NHD, dict(pad=8)), (HND, dict(offset=8)), (XS, dict(offset=8)),
    (NHD, dict(dim=12)), (NHD, dict(dim=256, heads=3, bs=7))], ids=str)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_layouts(layout, kw, kv):
    if kv == "fp8" and kw.get("dim") == 12:
        kw = dict(kw, dim=24)
    cases, sc = make(seed=1, layout=layout, kv=kv, **kw)
    want = expected(cases, sc, [40, 40, 97], 3, 10)
    assert evict(cases, sc, [40, 40, 97], sinks=3, recent=10) == 0
    same(cases, sc, want)


@pytest.mark.parametrize("scores", ["random", "ties", "odd"])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 17), (4, 32), (1000, 5), (5, 1000)])
def test_choice(scores, sinks, recent):
    lengths = (1, 16, 300, 1500, 3001, 50)
    keep = [1, 7, 0, 700, 1024, 80]
    cases, sc = make(seed=2, layers=1, lengths=lengths, scores=scores, dim=8)
    want = expected(cases, sc, keep, sinks, recent)
    assert evict(cases, sc, keep, sinks=sinks, recent=recent) == 0
    same(cases, sc, want)


def test_first_positions_and_nothing_to_do():
    cases, sc = make(seed=3, lengths=(0, 100, 200), first=[0, 2, 40], extra=1)
    want = expected(cases, sc, [5, 20, 5], 2, 2)
    assert evict(cases, sc, [5, 20, 5], sinks=2, recent=2) == 0
    same(cases, sc, want)


def oracle_words(cases, ids, offsets, first, tokens):
    """The oracle's checksums of the blocks in `ids` as they are now."""
    caches = [OracleCache(host_bytes(c.cache.pool), c.nb, c.layout, c.cache.layer, 0, c.heads,
                          c.cache.head_bytes, 8, c.cache.kernel_block_size, c.cache.half_stride,
                          c.cache.block_stride) for c in cases]
    out, status = c_form(caches, cases[0].bs,
                         OracleRequests(offsets, first, tokens, ids.tolist()))
    assert status == 0
    return out


@pytest.mark.parametrize("layout,kw", [
    (NHD, {}), (HND, dict(bs=64)), (XS, {}), (LAT, dict(heads=1, dim=576, halves=1)),
    (NHD, dict(pad=8)), (NHD, dict(dim=12, bs=5)), (HND, dict(dim=256, heads=3, bs=7))], ids=str)
@pytest.mark.parametrize("fresh", [False, True])
def test_words(layout, kw, fresh):
    """The filled blocks' words are their checksums; emptied blocks have 0;
    no other block's word changes."""
    lengths, keep, first = (100, 37, 260), [41, 200, 97], [1, 0, 0]
    cases, sc = make(seed=4, layout=layout, lengths=lengths, first=first, spare=90, **kw)
    c = cases[0]
    to = None
    if fresh:
        free = [b for b in range(c.nb) if b not in set(c.ids.tolist())]
        to = torch.tensor((free * 3)[:c.total], dtype=torch.int32)
        used = 0
        for r in range(3):   # each request its own blocks
            need = -(-min(keep[r], c.values[r].shape[1]) // c.bs)
            to[c.offsets[r]:c.offsets[r] + need] = torch.tensor(free[used:used + need])
            to[c.offsets[r] + need:c.offsets[r + 1]] = -1
            used += need
    want = expected(cases, sc, keep, 2, 9, to)
    words = torch.full((c.nb,), 77, dtype=torch.int64, device="cuda")
    assert evict(cases, sc, keep, sinks=2, recent=9, block_sums=words,
                 new_block_ids=None if to is None else to.cuda()) == 0
    same(cases, sc, want)
    ids = c.ids if to is None else to
    touched = set()
    for r in range(3):
        B = min(keep[r], c.values[r].shape[1])
        need = -(-B // c.bs)
        mine = ids[c.offsets[r]:c.offsets[r] + need]
        got = words[mine.long().cuda()].cpu()
        exp = oracle_words(cases, mine, [0, need], [first[r]], [first[r] * c.bs + B])
        assert [int(x) & (2 ** 64 - 1) for x in got] == exp
        touched |= set(mine.tolist())
        if not fresh:
            rest = c.ids[c.offsets[r] + need:c.offsets[r + 1]]
            assert (words[rest.long().cuda()] == 0).all()
            touched |= set(rest.tolist())
    for b in set(range(c.nb)) - touched:
        assert int(words[b]) == 77


def test_rows_longer_than_shared_memory():
    """More tokens than a CTA holds scores of, beside short requests."""
    lengths = (60000, 20, 700)
    cases, sc = make(seed=9, layers=1, lengths=lengths, heads=1, dim=8, bs=64, spare=3,
                     scores="ties")
    want = expected(cases, sc, [31000, 7, 300], 4, 50)
    assert evict(cases, sc, [31000, 7, 300], sinks=4, recent=50) == 0
    same(cases, sc, want)


def test_shared_source_blocks_into_fresh_ones():
    """Two requests with a common prefix are thinned out into blocks of their own."""
    cases, sc = make(seed=10, layers=2, lengths=(96, 96), spare=40)
    c = cases[0]
    half = c.offsets[1]
    for x in cases:
        x.ids[half:half + 3] = x.ids[:3]
        x.table[3].copy_(x.ids)
        x.values[1] = torch.cat([x.values[0][:, :48], x.values[1][:, 48:]], 1)
    free = [b for b in range(c.nb) if b not in set(c.ids.tolist())]
    to = torch.tensor(free[:c.total], dtype=torch.int32)
    want = expected(cases, sc, [40, 70], 2, 8, to)
    assert evict(cases, sc, [40, 70], sinks=2, recent=8, new_block_ids=to.cuda()) == 0
    same(cases, sc, want)


def test_offsets_past_32_bits():
    cases, sc = make(seed=11, layers=1, lengths=(300, 90), heads=4, dim=128, spare=5)
    c = cases[0]
    nb, n = 70000, c.nb
    if torch.cuda.mem_get_info()[0] < 8 * nb * c.bs * 4 * 128:
        pytest.skip("needs 9 GB")
    big = torch.zeros((2, nb, c.bs, 4, 128), dtype=torch.bfloat16, device="cuda")
    big[:, nb - n:] = c.pool.view(torch.bfloat16).view(2, n, c.bs, 4, 128)
    scores = torch.zeros((nb, 4, c.bs), device="cuda")
    scores[nb - n:] = sc[0]
    keep = torch.tensor([111, 40], dtype=torch.int64, device="cuda")
    words = torch.zeros(nb, dtype=torch.int64, device="cuda")
    want_words = torch.zeros(n, dtype=torch.int64, device="cuda")
    K.evict(W.CacheSpec(big, nb, NHD, 0, 0, 4, 256), c.bs, *c.table[:3], c.table[3] + (nb - n), scores,
            keep, sinks=2, recent=9, block_sums=words)
    K.evict(c.cache, c.bs, *c.table, sc[0], keep, sinks=2, recent=9, block_sums=want_words)
    assert torch.equal(big[:, nb - n:].reshape(-1).view(torch.uint8), c.pool.view(-1))
    assert torch.equal(scores[nb - n:], sc[0]) and torch.equal(words[nb - n:], want_words)
    assert not big[:, :nb - n].any() and not words[:nb - n].any()


def test_bad_requests_are_left_untouched():
    cases, sc = make(seed=5, lengths=(100, 90, 80, 70))
    c = cases[0]
    c.table[3][c.offsets[1] + 2] = c.nb
    c.table[1][3] = -1
    keep = [30, 30, -1, 30]
    want = expected(cases, sc, [30, 90, 80, 70], 0, 0)
    words = torch.full((c.nb,), 5, dtype=torch.int64, device="cuda")
    status = evict(cases, sc, keep, block_sums=words)
    assert status == K.KVCS_STATUS_BAD_BLOCK_ID | K.KVCS_STATUS_BAD_REQUESTS
    same(cases, sc, want)
    for r in (1, 2, 3):
        assert (words[c.ids[c.offsets[r]:c.offsets[r + 1]].long().cuda()] == 5).all()


def test_many_caches():
    """More caches than one launch takes, of different geometry."""
    base = dict(lengths=(60, 25), new=[0, 0], tail=1.0, spare=2)
    cases = [A.Case(seed=6, layer=l, dim=16 if l % 2 else 8, heads=1 + l % 3, layout=l % 2, **base)
             for l in range(140)]
    g = torch.Generator().manual_seed(7)
    sc = [torch.rand((c.nb, c.heads, c.bs), generator=g).cuda() for c in cases]
    want = expected(cases, sc, [20, 20], 1, 4)
    assert evict(cases, sc, [20, 20], sinks=1, recent=4) == 0
    same(cases, sc, want)


def test_captured_and_replayed():
    cases, sc = make(seed=8, layers=1)
    c = cases[0]
    keep = torch.tensor([30, 30, 30], dtype=torch.int64, device="cuda")
    pool0, sc0 = c.pool.clone(), sc[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.evict(c.cache, c.bs, *c.table, sc[0], keep, sinks=1, recent=3, total_positions=c.total)
    for k in (30, 12, 300):
        c.pool.copy_(pool0)
        sc[0].copy_(sc0)
        keep.fill_(k)
        want = expected(cases, sc, [k] * 3, 1, 3)
        g.replay()
        torch.cuda.synchronize()
        same(cases, sc, want)


def test_a_cache_from_write_to_eviction():
    """New tokens are written, attended to and scored, the cache is thinned
    out, and decoding goes on over what is left; the running words follow."""
    torch.manual_seed(0)
    H, G, D, bs, layers, R = 2, 4, 128, 16, 2, 3
    lengths, budget = [75, 130, 40], 48
    per = [-(-(n + 1) // bs) for n in lengths]
    nb = sum(per) + 2
    ids = torch.randperm(nb)[:sum(per)].to(torch.int32).cuda()
    po = torch.tensor([0] + torch.tensor(per).cumsum(0).tolist(), device="cuda")
    fp = torch.zeros(R, dtype=torch.int64, device="cuda")
    nt = torch.tensor(lengths, device="cuda")
    pools = [torch.full((2, nb, bs, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
             for _ in range(layers)]
    caches = [W.CacheSpec(p, nb, NHD, l, 0, H, 2 * D) for l, p in enumerate(pools)]
    sums = torch.zeros(nb, dtype=torch.int64, device="cuda")
    mass = [torch.zeros((nb, H, bs), device="cuda") for _ in range(layers)]
    total = sum(lengths)
    offs = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), device="cuda")
    req = torch.repeat_interleave(torch.arange(R, device="cuda"), nt)
    pos = torch.arange(total, device="cuda") - offs[req]
    slot = ids.long()[po[req] + pos // bs] * bs + pos % bs
    new = lambda n: [torch.randn((n, H, D), device="cuda").bfloat16() for _ in range(layers)]  # noqa: E731
    keys, vals = new(total), new(total)
    K.write_kv(caches, bs, keys, vals, slot, pos, block_sums=sums)
    table = (po, fp, nt, ids)
    for l in range(layers):
        q = torch.randn((total, H * G, D), device="cuda").bfloat16()
        _, lse = K.paged_attention(caches[l], bs, *table, q, offs, max_new=max(lengths))
        K.attention_mass(caches[l], bs, *table, q, offs, lse, mass[l], max_new=max(lengths))
    logical = []
    for l in range(layers):
        kept = {}
        for r in range(R):
            B = min(budget, lengths[r])
            blk = ids.long()[po[r]:po[r + 1]]
            for h in range(H):
                row = mass[l][blk, h].reshape(-1)[:lengths[r]].tolist()
                kept[r, h] = A.kept_tokens(row, lengths[r], B, 2, 8)
        logical.append(kept)
    keep = torch.full((R,), budget, dtype=torch.int64, device="cuda")
    K.evict(caches, bs, *table, mass, keep, sinks=2, recent=8, block_sums=sums)
    nt = torch.minimum(nt, keep)
    # one more token: written behind the kept ones, then attended to
    k2, v2 = new(R), new(R)
    slot2 = ids.long()[po[:-1] + nt // bs] * bs + nt % bs
    K.write_kv(caches, bs, k2, v2, slot2, nt, block_sums=sums)
    nt = nt + 1
    table = (po, fp, nt, ids)
    q2 = torch.randn((R, H * G, D), device="cuda").bfloat16()
    words = K.block_checksums(caches, bs, *table)
    torch.cuda.synchronize()
    for r in range(R):
        used = -(-int(nt[r]) // bs)
        blk = ids.long()[int(po[r]):int(po[r]) + used]
        assert torch.equal(sums[blk], words[int(po[r]):int(po[r]) + used])
    for l in range(layers):
        out, _ = K.paged_attention(caches[l], bs, *table, q2,
                                   torch.arange(R + 1, device="cuda"), max_new=1)
        for r in range(R):
            for h in range(H * G):
                src = torch.tensor(logical[l][r, h // G], device="cuda") + offs[r]
                k = torch.cat([keys[l][src, h // G], k2[l][r:r + 1, h // G]]).double()
                v = torch.cat([vals[l][src, h // G], v2[l][r:r + 1, h // G]]).double()
                w = torch.softmax(k @ q2[r, h].double() * D ** -0.5, 0)
                want = w @ v
                # two roundings to bf16 (weights, output) and the sums' 2^-15
                tol = (w @ v.abs()) * (2 ** -8 + 2 ** -13) + want.abs() * 2 ** -8 + 1e-6
                assert ((out[r, h].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fresh", [False, True])
def test_requests_that_share_positions_move_only_their_blocks(fresh):
    """Positions that decrease somewhere let requests share them, and the
    space of their lists: flagged, and only bytes of their blocks change."""
    cases, sc = make(seed=41, layers=1, lengths=(160, 160, 400), spare=60)
    c = cases[0]
    c.table[0].copy_(torch.tensor([0, 10, 4, 10]))
    used = [int(b) for b in c.ids[:10]]
    kw = {}
    if fresh:
        spare = sorted(set(range(c.nb)) - set(c.ids.tolist()))
        to = torch.tensor((spare * 2)[:c.total], dtype=torch.int32)
        kw["new_block_ids"] = to.cuda()
        used = to[:10].tolist()
    before = c.pool.clone()
    assert evict(cases, sc, [150, 150, 90], **kw) == K.KVCS_STATUS_BAD_REQUESTS
    keep = torch.ones(before.numel(), dtype=torch.bool)
    keep[c.offsets_map[:, used].flatten()] = False
    assert torch.equal(c.pool.cpu()[keep], before.cpu()[keep])


@pytest.mark.parametrize("scores", ["random", "odd"])
@pytest.mark.parametrize("keep", [1, 1000, 8192, 8193, 16000, 20011])
@pytest.mark.parametrize("fresh", [False, True])
def test_one_long_request_among_short_ones(scores, keep, fresh):
    """A row with more scores than the launch's shared memory holds (sized by
    the average): part of them is read again, and they move in steps."""
    lengths = [20011] + [5] * 40
    cases, sc = make(seed=43, layers=1, lengths=lengths, heads=2, dim=8, bs=16, spare=1400,
                     scores=scores)
    c = cases[0]
    kw, to = {}, None
    if fresh:
        spare = sorted(set(range(c.nb)) - set(c.ids.tolist()))
        to = torch.tensor(spare[:c.total], dtype=torch.int32)
        kw["new_block_ids"] = to.cuda()
    keeps = [keep] + [3] * 40
    want = expected(cases, sc, keeps, 7, 99, to)
    assert evict(cases, sc, keeps, sinks=7, recent=99, **kw) == 0
    same(cases, sc, want)
