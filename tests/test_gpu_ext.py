"""Attention with first tokens kept past a window, of drafted trees, and over
caches with scales, against the 64-bit forms in ext_ref, whose error bounds are
derived there."""

import pytest
import torch

import attention_ref as A
import ext_ref as X
import paged_kv_cache_kvcs_gb300 as K
from paged_kv_cache_kvcs_gb300 import workloads as W

pytestmark = pytest.mark.gpu
NHD, HND, XS = W.LAYOUT_NHD, W.LAYOUT_HND, W.LAYOUT_XSPLIT


def make(kv, **kw):
    if kv in ("int8s", "fp8s"):
        return X.ScaledCase(kv[:-1], **kw)
    return A.Case(kv=kv, **kw)


def parents_of(trees):
    return torch.tensor([u for t in trees for u in t], dtype=torch.int32, device="cuda")


def run(case, trees=None, q=None, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if isinstance(case, X.ScaledCase):
        kw.update(k_scales=case.k_scales, v_scales=case.v_scales)
    args = (case.cache, case.bs, *case.table, case.q if q is None else q, case.new_offsets)
    if trees is None:
        out, lse = K.paged_attention(*args, kv_dtype=case.kv, status=status, **kw)
    else:
        out, lse = K.tree_attention(*args, parents_of(trees), kv_dtype=case.kv, status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def check(case, trees=None, blocked=None, want_status=0, max_new="known", **kw):
    m = {"max_new": max(case.new)} if max_new == "known" else {}
    out, lse, status = run(case, trees, **kw, **m)
    ref = X.attention(case, trees=trees, blocked=blocked, **kw)
    assert status == want_status
    A.close(out, ref[0], ref[2])
    A.close(lse, ref[1], ref[3])
    return out, lse


def trees_of(new, seed=0, chain=0.4):
    g = torch.Generator().manual_seed(seed)
    return [X.random_tree(n, g, chain) for n in new]


GEOMETRIES = [
    dict(dim=128, heads=2, group=4, bs=16),
    dict(dim=64, heads=3, group=1, bs=16),
    dict(dim=128, heads=1, group=8, bs=64),
    dict(dim=80, heads=2, group=5, bs=48),
    dict(dim=256, heads=1, group=2, bs=32),
    dict(dim=8, heads=2, group=3, bs=7),
    dict(dim=64, heads=1, group=24, bs=24),
]
GEO = pytest.mark.parametrize("geo", GEOMETRIES, ids=lambda g: "-".join(map(str, g.values())))
KINDS = ["bf16", "fp16", "fp8", "int8s", "fp8s"]
LENGTHS = [1, 2, 15, 17, 63, 65, 128, 400, 1025]


# ---------------------------------------------------------------------------
# windows with first tokens kept
# ---------------------------------------------------------------------------

@GEO
@pytest.mark.parametrize("kv", KINDS)
def test_sinks_decode(kv, geo):
    case = make(kv, lengths=LENGTHS, new=[1] * 9, seed=3, **geo)
    check(case, window=50, sinks=5)
    check(case, window=130, sinks=100, softcap=12.0)


@GEO
@pytest.mark.parametrize("kv", KINDS)
def test_sinks_chunks(kv, geo):
    case = make(kv, lengths=[5, 33, 700, 77, 500, 260], new=[5, 33, 17, 0, 129, 200], seed=4, **geo)
    check(case, window=40, sinks=3)


@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (100, 64), (100, 129), (300, 1), (64, 10 ** 12),
                                          (10 ** 12, 7), (0, 9), (33, 0)])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [150, 3, 61, 300]], ids=["one", "many"])
@pytest.mark.parametrize("kv", ["bf16", "int8s"])
def test_windows_and_sinks(window, sinks, new, kv):
    """Sinks below, inside and above the window's start; none; no window."""
    case = make(kv, lengths=[900, 90, 61, 333], new=new, seed=5, dim=128)
    check(case, window=window, sinks=sinks, scale=0.3)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 170, 1]], ids=["one", "many"])
@pytest.mark.parametrize("dim", [64, 128])
def test_sinks_count_request_positions(new, dim):
    """A request's listed blocks may start behind some or all of the sinks."""
    case = A.Case(lengths=[600, 400, 200], new=new, first=[1, 3, 0], seed=6, dim=dim)
    check(case, window=60, sinks=20)
    check(case, window=60, sinks=40)
    check(case, window=60, sinks=70)


@pytest.mark.parametrize("new", [[1, 1], [90, 260], [5, 17]], ids=str)
@pytest.mark.parametrize("kv", ["bf16", "int8s"])
@pytest.mark.parametrize("rubbish", [-1, 2 ** 31 - 1])
def test_blocks_between_are_not_looked_up(new, kv, rubbish):
    """Ids of the blocks between the sinks' and the windows' may be anything."""
    case = make(kv, lengths=[1500, 2000], new=new, seed=7, dim=128, group=2)
    want = run(case, window=100, sinks=20, max_new=max(new))
    for r, n in enumerate(new):
        first = case.lengths[r] - n - 100 + 1
        case.table[3][case.offsets[r] + 2:case.offsets[r] + first // 16] = rubbish
    got = run(case, window=100, sinks=20, max_new=max(new))
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("new", [[1, 1], [70, 200]], ids=str)
def test_bad_blocks_of_sinks_and_windows_are_left_out(new):
    case = A.Case(dim=128, lengths=[1000, 700], new=new, seed=8)
    last = [(n - 1) // 16 for n in case.lengths]
    case.table[3][case.offsets[0]] = -1
    case.table[3][case.offsets[1] + last[1] - 1] = case.nb
    check(case, window=100, sinks=20, blocked={0: (0,), 1: (last[1] - 1,)},
          want_status=K.KVCS_STATUS_BAD_BLOCK_ID)


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("fp16", 64), ("fp8", 64), ("fp8", 128), ("int8s", 128),
                                    ("fp8s", 64)])
@pytest.mark.parametrize("new", [[2, 1, 3], [20, 33, 70]], ids=["few", "many"])
def test_bad_blocks_of_sinks_beside_the_window(new, kv, dim):
    """A bad block of the sinks is left out and flagged where the window starts
    in the sinks' last tile of 128 tokens: the first one, or a later one."""
    case = make(kv, dim=dim, lengths=[300, 420, 330], new=new, seed=34)
    case.table[3][case.offsets[0]] = -1
    case.table[3][case.offsets[1] + 8] = case.nb
    case.table[3][case.offsets[2] + 1] = -7
    # windows that start at 81 to 99, 188 to 220 and 61 to 128; the bad blocks are
    # tokens 0 to 15, 128 to 143 and 16 to 31
    check(case, window=200, sinks=140, blocked={0: (0,), 1: (8,), 2: (1,)},
          want_status=K.KVCS_STATUS_BAD_BLOCK_ID)


@pytest.mark.parametrize("kv", ["bf16", "int8s"])
@pytest.mark.parametrize("bad", [0, 119, 120, 122], ids=str)
def test_bad_blocks_of_sinks_in_split_calls(bad, kv):
    """One request, its tokens split into parts of some tiles: a part may begin
    where the sinks end and the window starts."""
    case = make(kv, dim=128, heads=1, lengths=[4000], new=[20], seed=35)
    case.table[3][case.offsets[0] + bad] = -1
    check(case, window=2000, sinks=1960, blocked={0: (bad,)}, want_status=K.KVCS_STATUS_BAD_BLOCK_ID)


def list_only(case, counts):
    """Has the table list each request's first blocks alone."""
    ids = [case.ids[o:o + n] for o, n in zip(case.offsets, counts)]
    case.values = [v[:, :n * case.bs] for v, n in zip(case.values, counts)]
    case.ids = torch.cat(ids)
    case.offsets = [sum(counts[:r]) for r in range(len(counts) + 1)]
    case.total = case.offsets[-1]
    case.table[0] = torch.tensor(case.offsets, dtype=torch.int64, device="cuda")
    case.table[3] = case.ids.to("cuda")


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("fp16", 64), ("fp8", 128), ("int8s", 64), ("fp8s", 128)])
@pytest.mark.parametrize("new", [[1, 3, 2, 1], [20, 20, 33, 70]], ids=["few", "many"])
def test_sinks_of_tables_that_end_before_the_window(new, kv, dim):
    """Where the listed blocks end before the windows start, rows still see the
    sinks among them: in the first tile of 128 tokens, in the window's own, in
    whole ones before."""
    case = make(kv, dim=dim, lengths=[200, 569, 1100, 900], new=new, seed=36)
    list_only(case, [2, 25, 19, 57])
    # listed tokens: 32, 400, 304 and 900; the windows start at 81 (100), 450 (468),
    # 968 (998) and 731 (800) and later
    for sinks in (8, 130, 400):
        check(case, window=100, sinks=sinks)
    check(case, trees_of(new, 17), window=100, sinks=140)


@pytest.mark.parametrize("new", [[1, 2], [40, 90]], ids=["few", "many"])
@pytest.mark.parametrize("kv", ["bf16", "int8s"])
def test_sinks_past_2_to_the_30(new, kv):
    """Request positions and sinks beyond 2^30 (tables that list the last blocks)."""
    case = make(kv, dim=128, lengths=[2 ** 31 + 300, 2 ** 30 + 210], new=new,
                first=[2 ** 27, 2 ** 26], seed=39)
    check(case, window=40, sinks=2 ** 30 + 20)
    check(case, window=40, sinks=2 ** 31 + 30)
    check(case, window=40, sinks=2 ** 62)
    check(case, trees_of(new, 18, 0.9), window=20, sinks=2 ** 31 + 270)


# ---------------------------------------------------------------------------
# drafted trees
# ---------------------------------------------------------------------------

@GEO
@pytest.mark.parametrize("kv", KINDS)
def test_trees(kv, geo):
    new = [1, 2, 3, 16, 17, 0, 33, 70]
    lengths = [1, 40, 3, 200, 17, 9, 500, 333]
    case = make(kv, lengths=lengths, new=new, seed=9, **geo)
    check(case, trees_of(new, 1))


@pytest.mark.parametrize("new", [[300, 129, 257], [1024, 40, 5], [64, 64, 64], [3, 2, 4]], ids=str)
@pytest.mark.parametrize("shape", ["random", "chain", "star", "deep"])
@pytest.mark.parametrize("kv,group", [("bf16", 1), ("fp16", 4), ("int8s", 2)])
def test_tree_shapes(new, shape, kv, group):
    case = make(kv, dim=64, heads=1, group=group, lengths=[n + 333 for n in new], new=new, seed=10)
    trees = {"random": lambda: trees_of(new, 2), "chain": lambda: [list(range(-1, n - 1)) for n in new],
             "star": lambda: [[-1] * n for n in new], "deep": lambda: trees_of(new, 3, 0.97)}[shape]()
    out, lse = check(case, trees)
    if shape == "chain":     # a text
        plain = run(case, max_new=max(new))
        ref = X.attention(case)
        A.close(out, plain[0].cpu().double(), 2 * ref[2])
        A.close(lse, plain[1].cpu().double(), 2 * ref[3])


@pytest.mark.parametrize("window,sinks", [(1, 0), (4, 0), (40, 0), (4, 30), (40, 350), (600, 5)])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("new", [[4, 3, 1], [150, 33, 61]], ids=["few", "many"])
@pytest.mark.parametrize("kv", ["bf16", "fp8s"])
def test_tree_windows(window, sinks, softcap, new, kv):
    """Windows go by positions: depths, not places in the cache; some are
    shorter than the tree is deep."""
    case = make(kv, lengths=[n + 300 for n in new], new=new, seed=11, dim=128, group=4, first=[0, 1, 0])
    check(case, trees_of(new, 4, 0.9), window=window, sinks=sinks, softcap=softcap, scale=0.4)


@pytest.mark.parametrize("layout,kw", [
    (HND, {}), (HND, dict(kbs=4)), (XS, {}), (NHD, dict(interleaved=True)),
    (NHD, dict(pad=16)), (NHD, dict(pad=8)), (HND, dict(offset=8)), (XS, dict(offset=8)),
    (HND, dict(interleaved=True, pad=48))], ids=str)
@pytest.mark.parametrize("kv", ["bf16", "int8s", "fp8s"])
@pytest.mark.parametrize("dim", [64, 128])
def test_layouts(layout, kw, kv, dim):
    new = [1, 1, 80, 40]
    case = make(kv, layout=layout, dim=dim, lengths=[70, 1, 259, 90], new=new, seed=12, **kw)
    check(case, trees_of(new, 5))
    check(case, window=30, sinks=6)


@pytest.mark.parametrize("new", [[5, 4, 6], [90, 60, 200], [5, 90, 1]], ids=str)
@pytest.mark.parametrize("bad", [2, -2, 2 ** 31 - 1, -2 ** 31])
def test_bad_parents_are_flagged(new, bad):
    """A tree with a parent at or behind its child, or below -1: its request's
    rows see nothing, the others' are as they were.  (Non-finite values reach
    nobody.)"""
    case = A.Case(dim=128, lengths=[n + 100 for n in new], new=new, seed=13)
    case.put(1, 1, 3, torch.full((1, 128), float("nan")))
    trees = trees_of(new, 6)
    trees[1][2] = bad
    out, lse = check(case, trees, want_status=K.KVCS_STATUS_BAD_REQUESTS)
    lo, hi = case.starts[1], case.starts[2]
    assert (out[lo:hi] == 0).all() and torch.isneginf(lse[lo:hi]).all()


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8", "fp8s"])
@pytest.mark.parametrize("dim,new", [(64, [4, 3]), (128, [70, 200]), (64, [12, 40])])
def test_nonfinite_values_of_other_branches(kv, dim, new):
    """What a branch's tokens hold never reaches the other branches."""
    case = make(kv, dim=dim, lengths=[n + 200 for n in new], new=new, seed=14)
    trees = [[-1] + [0 if i % 2 else max(i - 2, 0) for i in range(1, n)] for n in new]
    for r, n in enumerate(new):
        t = case.lengths[r] - n + 1
        for half in (0, 1):
            if kv == "fp8s":
                case.set_scale(r, half, t, float("nan"))
            else:
                case.put(r, half, t, torch.full((1, dim), float("nan")))
    out, lse, status = run(case, trees, max_new=max(new))
    ref = X.attention(case, trees=trees)
    hit = torch.cat([X.sees(case, r, tree=trees[r])[:, case.lengths[r] - n + 1]
                     for r, n in enumerate(new)])
    assert status == 0 and hit.any() and not hit.all()
    A.close(out[~hit.cuda()], ref[0][~hit], ref[2][~hit])
    A.close(lse[~hit.cuda()], ref[1][~hit], ref[3][~hit])
    assert torch.isnan(out[hit.cuda()]).all()


@pytest.mark.parametrize("new", [[6, 6], [300, 200]], ids=str)
def test_nonfinite_values_past_windows_and_sinks(new):
    """What lies between the sinks and the windows never reaches a row."""
    case = A.Case(dim=128, lengths=[1000, 900], new=new, seed=15)
    for r in (0, 1):
        for t in (9, 15, 16, 100, case.lengths[r] - new[r] - 60):
            for half in (0, 1):
                case.put(r, half, t, torch.full((1, 128), float("inf") if t % 2 else float("nan")))
    check(case, trees_of(new, 7), window=50, sinks=9)
    check(case, window=50, sinks=9)


def test_mixed_batches_of_trees():
    """Requests on both sides of the row limits, max_new known or not; requests
    of more than the limit are flagged and left."""
    new = [1, 300, 2, 0, 5, 90, 1, 1]
    case = A.Case(dim=64, group=4, lengths=[n + 50 * i for i, n in enumerate(new)], new=new, seed=16)
    check(case, trees_of(new, 8))
    check(case, trees_of(new, 8), max_new="unknown")
    new = [1100, 3]
    case = A.Case(dim=64, heads=1, group=1, lengths=[1200, 60], new=new, seed=17)
    trees = trees_of(new, 9)
    out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
    _, _, status = run(case, trees, out=out)
    ref = X.attention(case, trees=trees)
    assert status == K.KVCS_STATUS_BAD_REQUESTS and (out[:1100] == 7).all()
    A.close(out[1100:], ref[0][1100:], ref[2][1100:])
    with pytest.raises(K.KvcsError):
        run(case, trees, max_new=1100)


@pytest.mark.parametrize("new", [1, 4, 100])
@pytest.mark.parametrize("kv", ["bf16", "int8s"])
def test_long_and_split(new, kv):
    """One request over the whole GPU: groups split between CTAs and joined."""
    case = make(kv, heads=1, group=4, dim=128, lengths=[30011], new=[new], bs=32, seed=18)
    check(case, trees_of([new], 10))
    check(case, window=9000, sinks=700)


def test_more_units_than_the_gpu_holds():
    g = torch.Generator().manual_seed(19)
    lengths = torch.randint(20, 700, (24,), generator=g).tolist()
    new = [min(n, 17 + (7 * i) % 200) for i, n in enumerate(lengths)]
    case = A.Case(dim=128, heads=4, group=4, lengths=lengths, new=new, seed=19)
    check(case, trees_of(new, 11))
    check(case, window=150, sinks=30)


# ---------------------------------------------------------------------------
# caches with scales
# ---------------------------------------------------------------------------

@GEO
@pytest.mark.parametrize("kv", ["int8s", "fp8s"])
@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float16])
def test_scaled(kv, geo, q_dtype):
    case = make(kv, lengths=LENGTHS, new=[1, 1, 3, 17, 2, 40, 1, 33, 1], seed=20, q_dtype=q_dtype, **geo)
    check(case, k_scale=0.5, v_scale=2.0)


@pytest.mark.parametrize("kv", ["int8s", "fp8s"])
@pytest.mark.parametrize("spread", [8.0, 20.0])
@pytest.mark.parametrize("new", [[1, 1], [20, 40]], ids=["one", "many"])
def test_scales_far_apart(kv, spread, new):
    """Tokens' V scales up to 2^100 apart: each row's output keeps the precision
    of the tokens that make it."""
    case = make(kv, dim=128, lengths=[300, 700], new=new, seed=21, spread=spread)
    # scores of ordinary size: K's scales alike again
    fine = make(kv, dim=128, lengths=[300, 700], new=new, seed=21, spread=0.0)
    case.k_scales = fine.k_scales
    for a, b in zip(case.values, fine.values):
        a[0] = b[0]
    check(case)


@pytest.mark.parametrize("new", [[1, 1], [70, 200]], ids=["one", "many"])
@pytest.mark.parametrize("rubbish", [float("nan"), float("inf"), 3e38, 0.0, -1.0])
def test_scales_out_of_sight_reach_nobody(new, rubbish):
    """Scales of later tokens, of those before the window, of empty slots."""
    case = make("int8s", dim=128, lengths=[150, 300], new=new, seed=22)
    want = run(case, window=20, sinks=2, max_new=max(new))
    for r in (0, 1):
        blk = case.ids[case.offsets[r]:].long()
        for t in range(2, case.lengths[r] - new[r] - 20 + 1):
            b = int(blk[t // 16])
            case.k_scales[b, :, t % 16] = rubbish
            case.v_scales[b, :, t % 16] = rubbish
    case.k_scales[torch.isnan(case.k_scales)] = rubbish
    got = run(case, window=20, sinks=2, max_new=max(new))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the last token's: only the last row sees it
    if new[0] > 1:
        case.v_scales[int(case.ids[case.offsets[0] + 149 // 16]), :, 149 % 16] = rubbish
        got = run(case, window=20, sinks=2, max_new=max(new))
        assert torch.equal(got[0][:new[0] - 1], want[0][:new[0] - 1])


def test_scales_of_either_sign_and_small():
    case = make("fp8s", dim=64, lengths=[200, 90], new=[1, 30], seed=23)
    for r in (0, 1):
        for t in range(0, case.lengths[r], 3):
            case.set_scale(r, 1, t, -0.7)
            case.set_scale(r, 0, t, -0.2)
        for t in range(1, case.lengths[r], 5):
            case.set_scale(r, 1, t, 1e-30)
    check(case)


@pytest.mark.parametrize("kv,dim", [("int8s", 128), ("fp8s", 64), ("int8s", 80)])
@pytest.mark.parametrize("new", [[4, 3], [70, 33]], ids=["few", "many"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("half", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("softcap", [0.0, 12.0])
def test_scales_not_finite_in_sight(softcap, half, value, new, kv, dim):
    """One makes the rows that see it NaN, whatever the products' signs: here the
    last tokens' but two, and a cached one of the second request."""
    case = make(kv, dim=dim, lengths=[150, 300], new=new, seed=37)
    case.set_scale(0, half, 147, value)
    case.set_scale(1, half, 40, value)
    out, lse, status = run(case, max_new=max(new), softcap=softcap)
    ref = X.attention(case, softcap=softcap)
    hit = torch.cat([X.sees(case, r)[:, t] for r, t in ((0, 147), (1, 40))])
    assert status == 0 and hit.any() and not hit.all()
    assert torch.isnan(out[hit.cuda()]).all()
    if half == 0:
        assert torch.isnan(lse[hit.cuda()]).all()
    A.close(out[~hit.cuda()], ref[0][~hit], ref[2][~hit])
    A.close(lse[~hit.cuda()], ref[1][~hit], ref[3][~hit])


@pytest.mark.parametrize("kv", ["int8s", "fp8s"])
@pytest.mark.parametrize("new", [[1, 1], [20, 90]], ids=["one", "many"])
def test_large_values(kv, new):
    """V values of some 2^116, as bfloat16 holds them, under scores alike: weights
    near 1, whose products of random signs add up to some 2^122 before the division
    by their sum.  (Relative to a weight of 2^-13, as fp16 products are made, that
    would be past the largest 32-bit number.)"""
    case = make(kv, dim=128, lengths=[300, 3000], new=new, seed=38, spread=0.5)
    case.v_scales *= 2.0 ** 116
    for v in case.values:
        v[1] *= 2.0 ** 116
    check(case, scale=0.01)


# ---------------------------------------------------------------------------
# many rows over 8-bit caches
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bs", [7, 16, 24, 64])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv", ["fp8", "int8s", "fp8s"])
def test_many_rows_over_bytes(kv, dim, bs):
    new = [300, 33, 9, 1, 0, 129]
    case = make(kv, dim=dim, bs=bs, heads=2, group=3, lengths=[n + 413 for n in new], new=new, seed=30)
    scales = dict(k_scale=0.5, v_scale=2.0) if kv == "fp8" else {}
    check(case, trees_of(new, 8), **scales)
    check(case, trees_of(new, 9), window=70, sinks=20, softcap=12.0, **scales)
    check(case, window=150, sinks=5, **scales)
    check(case, window=260, sinks=140, max_new="unknown", scale=-0.3, **scales)


@pytest.mark.parametrize("dim", [64, 128])
def test_every_e4m3_value(dim):
    """All finite values, subnormal ones and both zeros among them, as K and V."""
    case = A.Case(kv="fp8", q_dtype=torch.bfloat16, dim=dim, lengths=[256, 131], new=[70, 100], seed=31)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[torch.isfinite(every)]
    for t in range(0, 100, 3):
        for half in (0, 1):
            case.put(0, half, t, every.roll(-dim * (t % 4) - t)[:dim][None].expand(case.heads, dim))
    check(case, trees_of([70, 100], 10), scale=0.01)


@pytest.mark.parametrize("new", [[300, 200], [40, 90]], ids=str)
@pytest.mark.parametrize("kv", ["fp8", "fp8s", "int8s"])
def test_nonfinite_bytes_past_windows_and_sinks(kv, new):
    """NaN bytes and scales between the sinks and the windows never reach a row."""
    case = make(kv, dim=128, lengths=[1000, 900], new=new, seed=32)
    plain = make(kv, dim=128, lengths=[1000, 900], new=new, seed=32)
    for r in (0, 1):
        for t in (9, 15, 16, 100, case.lengths[r] - new[r] - 60):
            for half in (0, 1):
                if kv == "fp8":
                    case.put(r, half, t, torch.full((1, 128), float("nan")))
                else:
                    case.set_scale(r, half, t, float("nan") if t % 2 else float("inf"))
    for trees in (trees_of(new, 7), None):
        kw = dict(window=50, sinks=9, max_new=max(new))
        got, want = run(case, trees, **kw), run(plain, trees, **kw)
        assert got[2] == want[2] == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_blocks_under_many_rows_of_bytes():
    new = [70, 200]
    case = make("fp8s", dim=128, lengths=[900, 700], new=new, seed=33)
    case.table[3][case.offsets[0] + 3] = -1
    case.table[3][case.offsets[1] + 11] = case.nb
    check(case, trees_of(new, 11), blocked={0: (3,), 1: (11,)}, want_status=K.KVCS_STATUS_BAD_BLOCK_ID)


# ---------------------------------------------------------------------------
# the calls
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv,new", [("bf16", [4] * 9), ("bf16", [200, 90, 1]), ("int8s", [4, 30, 9])], ids=str)
def test_graph_replay_streams_and_determinism(kv, new):
    """Captured and replayed over refilled trees, two graphs with workspaces of
    their own, on another stream, and twice: the same bits."""
    case = make(kv, dim=128, lengths=[1000 + 137 * i for i in range(len(new))], new=new, seed=24)
    m = max(new)
    kw = dict(max_new=m, window=700, sinks=10)
    trees = [trees_of(new, s) for s in (1, 2)]
    want = [run(case, t, **kw) for t in trees]
    assert not torch.equal(want[0][0], want[1][0])
    assert torch.equal(want[0][0], run(case, trees[0], **kw)[0])
    if kv == "int8s":
        kw.update(k_scales=case.k_scales, v_scales=case.v_scales)
    kw.update(total_positions=case.total, kv_dtype=case.kv)
    args = (case.cache, case.bs, *case.table, case.q, case.new_offsets)
    side = torch.cuda.Stream()
    ups = [parents_of(t) for t in trees]
    up = ups[0].clone()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = K.tree_attention(*args, up, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(K.tree_attention(*args, up, **kw))
    for k in (0, 1, 0):
        up.copy_(ups[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o[0], want[k][0]) and torch.equal(o[1], want[k][1])


def test_given_workspace_strided_queries_and_left_rows():
    new = [3, 100]
    case = A.Case(dim=64, lengths=[50, 400], new=new, seed=25)
    trees = trees_of(new, 12)
    n, hq, d = case.q.shape
    fused = torch.zeros((n + 3, hq * d + 2 * 2 * d), device="cuda", dtype=case.q.dtype)
    fused[1:n + 1, :hq * d] = case.q.reshape(n, -1)
    q = fused[:, :hq * d].view(n + 3, hq, d)
    out = torch.full((n + 3, hq, d), 7.0, dtype=case.q.dtype, device="cuda")
    lse = torch.full((n + 3, hq), 7.0, device="cuda")
    size = K.attention_workspace_bytes(case.cache, case.bs, 2, case.total, q, max_new=100, window=60,
                                       sinks=4, tree=True)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    up = torch.full((n + 3,), 99, dtype=torch.int32, device="cuda")
    up[1:n + 1] = parents_of(trees)
    K.tree_attention(case.cache, case.bs, *case.table, q, case.new_offsets + 1, up, out=out, lse=lse,
                     workspace=ws, max_new=100, window=60, sinks=4)
    ref = X.attention(case, trees=trees, window=60, sinks=4)
    A.close(out[1:n + 1], ref[0], ref[2])
    A.close(lse[1:n + 1], ref[1], ref[3])
    for x in (out, lse):
        assert (x[:1] == 7).all() and (x[n + 1:] == 7).all()
    with pytest.raises(ValueError):
        K.tree_attention(case.cache, case.bs, *case.table, q, case.new_offsets + 1, up,
                         workspace=ws[:size - 1], max_new=100, window=60, sinks=4)


def test_two_calls_at_once():
    cases = [make(kv, dim=128, lengths=[3000 + 500 * i, 900], new=new, seed=26 + i)
             for i, (kv, new) in enumerate((("bf16", [4, 4]), ("int8s", [3, 20]), ("bf16", [120, 300]),
                                            ("fp8s", [1, 1])))]
    trees = [trees_of(c.new, i) for i, c in enumerate(cases)]
    alone = [run(c, t, max_new=max(c.new)) for c, t in zip(cases, trees)]
    ups = [parents_of(t) for t in trees]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, up, s in zip(cases, ups, streams):
            more = dict(k_scales=c.k_scales, v_scales=c.v_scales) if isinstance(c, X.ScaledCase) else {}
            got.append(K.tree_attention(c.cache, c.bs, *c.table, c.q, c.new_offsets, up, kv_dtype=c.kv,
                                        max_new=max(c.new), stream=s, total_positions=c.total, **more))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("new", [[0, 0], [0, 3]], ids=str)
def test_little_to_do(new):
    """No new tokens; no cached tokens but the new ones, or none listed."""
    case = A.Case(dim=64, lengths=[0, 3], new=new, seed=27)
    check(case, trees_of(new, 13))
    case = A.Case(dim=64, lengths=[0, 2], new=[3, 4], seed=28)
    check(case, trees_of([3, 4], 14))
    case = A.Case(dim=128, lengths=[100, 40], new=[60, 40], first=[9, 3], seed=29)
    check(case, trees_of([60, 40], 15), window=20, sinks=4)


def test_offsets_past_32_bits():
    """Blocks, and their scales, beyond 4 GiB from the arrays' bases."""
    nb, H, bs, D = 1100000, 4, 16, 64
    if torch.cuda.mem_get_info()[0] < 4 * nb * bs * H * D:
        pytest.skip("needs 18 GB")
    case = make("int8s", dim=D, heads=H, group=4, lengths=[200, 77], new=[9, 3], seed=30)
    n = case.nb
    big = torch.zeros((2, nb, bs, H, D), dtype=torch.int8, device="cuda")
    big[:, nb - n:] = case.pool.view(torch.int8).view(2, n, bs, H, D)
    far = [torch.zeros((nb, H, bs), device="cuda") for _ in range(2)]
    far[0][nb - n:], far[1][nb - n:] = case.k_scales, case.v_scales
    trees = trees_of(case.new, 16)
    want = run(case, trees, max_new=9)
    got = K.tree_attention(W.CacheSpec(big, nb, NHD, 0, 0, H, D), bs, *case.table[:3],
                           case.table[3] + (nb - n), case.q, case.new_offsets, parents_of(trees),
                           max_new=9, k_scales=far[0], v_scales=far[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_torch_refusals():
    case = make("int8s", dim=64, lengths=[40], new=[2], seed=31)
    args = (case.cache, case.bs, *case.table, case.q, case.new_offsets)
    s = dict(k_scales=case.k_scales, v_scales=case.v_scales, kv_dtype=torch.int8)
    up = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    for bad in (dict(s, v_scales=None), dict(s, k_scales=case.k_scales.half()),
                dict(s, k_scales=case.k_scales[:-1]), dict(s, v_scales=case.v_scales.cpu()),
                dict(s, k_scales=case.k_scales.transpose(1, 2)), dict(kv_dtype=torch.int8)):
        with pytest.raises(ValueError):
            K.paged_attention(*args, **bad)
    for tree in (None, up.long(), up[:1], up.cpu()):
        with pytest.raises(ValueError):
            K.tree_attention(*args, tree, **s)
    with pytest.raises(K.KvcsError):
        K.paged_attention(*args, sinks=-1, window=5, **s)
    K.tree_attention(*args, up, **s)
