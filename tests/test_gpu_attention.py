"""kvcs_paged_attention and kvcs_attention_mass against the 64-bit forms in
attention_ref, whose error bounds are derived there."""

import math

import pytest
import torch

import attention_ref as A
import paged_kv_cache_kvcs_gb300 as K
from paged_kv_cache_kvcs_gb300 import workloads as W

pytestmark = pytest.mark.gpu
NHD, HND, XS = W.LAYOUT_NHD, W.LAYOUT_HND, W.LAYOUT_XSPLIT


def run(case, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = K.paged_attention(case.cache, case.bs, *case.table, case.q, case.new_offsets,
                                 kv_dtype=case.kv, status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def check(case, max_new="known", blocked=None, want_status=0, **kw):
    m = {"max_new": max(case.new)} if max_new == "known" else {}
    out, lse, status = run(case, **kw, **m)
    ref = A.attention(case, blocked=blocked, **kw)
    assert status == want_status
    A.close(out, ref[0], ref[2])
    A.close(lse, ref[1], ref[3])
    return out, lse


GEOMETRIES = [
    dict(dim=128, heads=2, group=4, bs=16),
    dict(dim=64, heads=3, group=1, bs=16),
    dict(dim=128, heads=1, group=8, bs=64),
    dict(dim=80, heads=2, group=5, bs=48),
    dict(dim=256, heads=1, group=2, bs=32),
    dict(dim=8, heads=2, group=3, bs=7),
    dict(dim=96, heads=1, group=16, bs=1),
    dict(dim=128, heads=1, group=24, bs=16),
]


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("geo", GEOMETRIES, ids=lambda g: "-".join(map(str, g.values())))
def test_decode(kv, geo):
    """One new token a request, lengths around tile and block borders."""
    check(A.Case(kv=kv, lengths=[1, 2, 15, 16, 17, 63, 64, 65, 127, 400, 1025],
                 new=[1] * 11, seed=3, **geo), k_scale=0.5, v_scale=2.0)


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("geo", GEOMETRIES, ids=lambda g: "-".join(map(str, g.values())))
def test_chunks(kv, geo):
    """Chunks of new tokens, with and without earlier tokens; none at all."""
    check(A.Case(kv=kv, lengths=[5, 33, 200, 77, 300, 130], new=[5, 33, 17, 0, 129, 70], seed=4,
                 **geo))


@pytest.mark.parametrize("layout,kw", [
    (HND, {}), (HND, dict(kbs=4)), (XS, {}), (NHD, dict(interleaved=True)),
    (NHD, dict(pad=16)), (NHD, dict(pad=8)), (HND, dict(offset=8)), (XS, dict(offset=8)),
    (HND, dict(interleaved=True, pad=48))], ids=str)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_layouts(layout, kw, kv, dim):
    check(A.Case(kv=kv, layout=layout, dim=dim, lengths=[70, 1, 259, 90], new=[1, 1, 80, 40],
                 seed=5, **kw))


@pytest.mark.parametrize("window", [0, 1, 16, 100])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("new", [[1, 1, 1], [150, 3, 61]])
@pytest.mark.parametrize("dim", [64, 128])
def test_window_and_softcap(window, softcap, new, dim):
    check(A.Case(lengths=[600, 90, 61], new=new, seed=6, dim=dim, scale=2.0),
          window=window, softcap=softcap, scale=0.3)


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [40, 1, 170, 64]])
@pytest.mark.parametrize("dim", [64, 128])
def test_empty_rows(new, dim):
    """Requests with no cached tokens, fewer cached than new ones, or whose
    listed blocks start past what a row may see."""
    check(A.Case(lengths=[0, 0, 30, 100], new=new, first=[0, 3, 0, 2], seed=7, dim=dim), window=33)


def test_first_position_and_extra_positions():
    case = A.Case(lengths=[200, 64, 130], new=[3, 1, 66], first=[5, 1, 0], extra=2, seed=8, dim=128)
    check(case)
    check(case, max_new="unknown")


@pytest.mark.parametrize("new", [1, 4, 100])
def test_long_and_split(new):
    """One request over the whole GPU: groups split between CTAs and joined."""
    check(A.Case(heads=1, group=4, dim=128, lengths=[30011], new=[new], bs=32, seed=9))


@pytest.mark.parametrize("new,group", [([1] * 40, 4), ([1, 300, 2, 0, 5, 90, 1, 1], 4),
                                       ([16, 17, 4, 5], 2), ([8, 8, 8], 8)])
def test_mixed_batches(new, group):
    """max_new known or not, and batches on both sides of the row limits."""
    g = torch.Generator().manual_seed(10)
    lengths = [n + int(torch.randint(0, 700, (1,), generator=g)) for n in new]
    case = A.Case(dim=64, group=group, lengths=lengths, new=new, seed=10)
    a = check(case)
    b = check(case, max_new="unknown")


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("dim,new", [(64, [1, 1]), (128, [1, 1]), (128, [70, 200]), (64, [5, 12])])
def test_nonfinite_values_in_masked_places(kv, dim, new):
    """Values that a row does not see never reach it: later tokens' NaN and
    infinite K and V, and those before the window."""
    case = A.Case(kv=kv, dim=dim, lengths=[150, 300], new=new, seed=11)
    bad = [float("nan")] if kv == "fp8" else [float("nan"), float("inf"), -float("inf")]
    for i, b in enumerate(bad):
        for r in (0, 1):
            T = case.lengths[r]
            case.put(r, 1, 3 + i, torch.full((1, dim), b))          # before every window
            case.put(r, 0, 7 + i, torch.full((1, dim), b))
    # the last token's V: only the last row sees it
    if new[0] > 1:
        case.put(0, 1, 149, torch.full((1, dim), float("nan")))
        case.put(1, 1, 290, torch.full((1, dim), float("nan")))
    out, lse, _ = run(case, window=20, max_new=max(new))
    ref = A.attention(case, window=20)
    keep = torch.isfinite(ref[0]).all(-1).all(-1)
    seen_k = torch.ones(len(keep), dtype=torch.bool)
    for r in (0, 1):      # rows that see a bad K are NaN: leave them out here
        see = A.visible(case, r, 20)
        lo = case.starts[r]
        seen_k[lo:lo + new[r]] = ~see[:, 7:7 + len(bad)].any(1)
    assert (keep & seen_k).sum() > 0
    sel = keep & seen_k
    A.close(out[sel.cuda()], ref[0][sel], ref[2][sel])
    A.close(lse[sel.cuda()], ref[1][sel], ref[3][sel])
    # and the rows that see a NaN value have it
    assert torch.isnan(out.cpu()[~keep & seen_k]).any(-1).all()


def test_scores_of_equal_and_extreme_size():
    """Scores far apart (one token takes all weight) and all equal."""
    case = A.Case(dim=128, lengths=[200, 200], new=[1, 90], seed=12, scale=30.0)
    check(case, scale=1.0)
    check(case, scale=0.0)
    check(case, scale=-1.0)


def test_strided_queries_and_given_outputs():
    case = A.Case(dim=64, lengths=[50, 400], new=[3, 100], seed=13)
    n, hq, d = case.q.shape
    fused = torch.randn((n, hq * d + 2 * 2 * d), device="cuda").to(case.q.dtype)
    fused[:, :hq * d] = case.q.reshape(n, -1)
    q = fused[:, :hq * d].view(n, hq, d)
    assert q.stride(0) != hq * d
    out = torch.empty_like(case.q)
    lse = torch.empty((n, hq), device="cuda")
    ws = torch.full((K.attention_workspace_bytes(case.cache, case.bs, 2, case.total, q, max_new=100),), 255,
                    dtype=torch.uint8, device="cuda")
    got = K.paged_attention(case.cache, case.bs, *case.table, q, case.new_offsets, out=out, lse=lse,
                            workspace=ws, max_new=100)
    assert got[0] is out and got[1] is lse
    ref = A.attention(case)
    A.close(out, ref[0], ref[2])
    A.close(lse, ref[1], ref[3])


def test_rows_no_request_owns_are_left():
    case = A.Case(dim=128, lengths=[50, 90], new=[2, 70], seed=14)
    n = case.q.shape[0]
    q = torch.cat([case.q[:1], case.q, case.q[:2]])
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    K.paged_attention(case.cache, case.bs, *case.table, q, case.new_offsets + 1, out=out, lse=lse,
                      max_new=70)
    ref = A.attention(case)
    A.close(out[1:1 + n], ref[0], ref[2])
    for x in (out, lse):
        assert (x[:1] == 7).all() and (x[1 + n:] == 7).all()


@pytest.mark.parametrize("new", [[1, 1], [33, 100]])
def test_bad_block_ids_are_left_out(new):
    case = A.Case(dim=128, lengths=[100, 300], new=new, seed=15)
    case.table[3][case.offsets[0] + 2] = -1
    case.table[3][case.offsets[1] + 5] = case.nb
    case.table[3][case.offsets[1] + 6] = 2 ** 31 - 1
    check(case, blocked={0: (2,), 1: (5, 6)}, want_status=K.KVCS_STATUS_BAD_BLOCK_ID)


def test_bad_tables_are_flagged():
    """Rows of requests with inconsistent tables see nothing; a request of
    more than max_new new tokens is left as it was."""
    base = dict(dim=64, lengths=[100, 60, 80], new=[1, 1, 1], seed=16)

    def outcome(change, **kw):
        case = A.Case(**base)
        change(case)
        out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
        _, lse, status = run(case, out=out, **kw)
        ref = A.attention(A.Case(**base))
        return case, out, lse, status, ref

    def negative_first(c):
        c.table[1][1] = -4

    def decreasing(c):
        c.table[0][1] = c.total + 9

    for change, hit in ((negative_first, [1]), (decreasing, [0, 1])):
        case, out, lse, status, ref = outcome(change, max_new=1)
        assert status == K.KVCS_STATUS_BAD_REQUESTS
        for r in range(3):
            if r in hit:
                assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
            else:
                A.close(out[r:r + 1], ref[0][r:r + 1], ref[2][r:r + 1])

    def too_many(c):
        c.new_offsets.copy_(torch.tensor([0, 0, 2, 3]))
    case, out, lse, status, ref = outcome(too_many, max_new=1)
    assert status == K.KVCS_STATUS_BAD_REQUESTS and (out[:2] == 7).all()
    A.close(out[2:], ref[0][2:], ref[2][2:])


def test_shared_prefix_blocks():
    """Two requests listing the same blocks read the same tokens."""
    case = A.Case(dim=128, lengths=[96, 96], new=[2, 40], seed=17)
    lo, hi = case.offsets[1], case.offsets[2]
    case.table[3][lo:hi] = case.table[3][:hi - lo].clone()
    case.values[1] = case.values[0]
    check(case)


@pytest.mark.parametrize("new", [[1] * 9, [200, 90, 1]])
def test_graph_replay_streams_and_determinism(new):
    """Captured and replayed over refilled inputs, on another stream, and
    twice: the same bits."""
    lengths = [1000 + 137 * i for i in range(len(new))]
    case = A.Case(dim=128, lengths=lengths, new=new, seed=18)
    m = max(new)
    first = run(case, max_new=m)
    assert torch.equal(first[0], run(case, max_new=m)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = K.paged_attention(case.cache, case.bs, *case.table, case.q, case.new_offsets,
                                 max_new=m, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    g = torch.cuda.CUDAGraph()
    q = case.q.clone()
    with torch.cuda.graph(g):
        out, lse = K.paged_attention(case.cache, case.bs, *case.table, q, case.new_offsets,
                                     max_new=m, total_positions=case.total)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        out2, _ = K.paged_attention(case.cache, case.bs, *case.table, q, case.new_offsets,
                                    max_new=m, total_positions=case.total)
    for s in (1.0, 0.5, 1.0):
        q.copy_(case.q * s)
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out2)
        if s == 1.0:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


PAGES = [dict(bs=8), dict(bs=24), dict(bs=40), dict(bs=128), dict(bs=256),
         dict(bs=32, kbs=8, layout=HND), dict(bs=48, kbs=16, layout=HND), dict(bs=4)]


@pytest.mark.parametrize("pages", PAGES, ids=str)
@pytest.mark.parametrize("group,dim", [(1, 128), (3, 64), (5, 128), (7, 64)])
def test_chunks_of_any_page_and_group(pages, group, dim):
    """Pages that end inside a tile, and query groups that do not divide one."""
    case = A.Case(dim=dim, group=group, lengths=[333, 150, 129], new=[140, 150, 30], seed=30, **pages)
    check(case)
    check_mass(case)


def test_more_units_than_the_gpu_holds():
    """Every CTA goes through several units, some of them short."""
    g = torch.Generator().manual_seed(31)
    lengths = torch.randint(20, 420, (24,), generator=g).tolist()
    new = [min(n, 17 + (7 * i) % 200) for i, n in enumerate(lengths)]
    case = A.Case(dim=128, heads=4, group=4, lengths=lengths, new=new, seed=31)
    check(case)
    check(case, window=40)
    check_mass(case, observe=100)
    check_mass(case, window=40)


def test_offsets_past_32_bits():
    """Blocks beyond 4 GiB from the pool's base, and pools whose V lies further."""
    nb, H, bs, D = 70000, 4, 16, 128
    if torch.cuda.mem_get_info()[0] < 2 * nb * bs * H * D * 2 * 2:
        pytest.skip("needs 5 GB")
    big = torch.zeros((2, nb, bs, H, D), dtype=torch.bfloat16, device="cuda")
    small = A.Case(dim=D, heads=H, group=4, lengths=[200, 77], new=[1, 1], seed=32, tail=0.0)
    chunk = A.Case(dim=D, heads=H, group=4, lengths=[200, 77], new=[90, 77], seed=32, tail=0.0)
    n = small.nb
    big[:, nb - n:] = small.pool.view(torch.bfloat16).view(2, n, bs, H, D)
    for case in (small, chunk):
        assert torch.equal(case.pool, small.pool)
        want = run(case, max_new=max(case.new))
        mass = torch.zeros((n, H, bs), device="cuda")
        K.attention_mass(case.cache, bs, *case.table, case.q, case.new_offsets, want[1], mass)
        cache = W.CacheSpec(big, nb, NHD, 0, 0, H, 2 * D)
        table = case.table[:3] + [case.table[3] + (nb - n)]
        got = K.paged_attention(cache, bs, *table, case.q, case.new_offsets, max_new=max(case.new))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        far = torch.zeros((nb, H, bs), device="cuda")
        K.attention_mass(cache, bs, *table, case.q, case.new_offsets, want[1], far)
        assert torch.equal(far[nb - n:], mass) and not far[:nb - n].any()


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace."""
    cases = [A.Case(dim=128, lengths=[3000 + 500 * i, 900], new=new, seed=33 + i)
             for i, new in enumerate(([1, 1], [120, 300], [1, 1], [64, 1]))]
    alone = [run(c, max_new=max(c.new)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [K.paged_attention(c.cache, c.bs, *c.table, c.q, c.new_offsets, max_new=max(c.new),
                                 stream=s, total_positions=c.total) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_nothing_to_do():
    case = A.Case(dim=64, lengths=[0, 30], new=[0, 0], seed=34)
    out, lse, status = run(case)
    assert out.numel() == 0 and lse.numel() == 0 and status == 0
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    q = torch.full((3, 8, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    K.paged_attention(case.cache, case.bs, zero, none, none, none.int(), q, zero, out=out)
    torch.cuda.synchronize()
    assert (out == 7).all()


# ---------------------------------------------------------------------------
# attention mass
# ---------------------------------------------------------------------------

def check_mass(case, blocked=None, want_status=0, observe=0, max_new=True, **kw):
    lse = A.attention(case, blocked=blocked, **kw)[1].float().cuda()
    before = torch.rand((case.nb, case.heads, case.bs), device="cuda")
    got = before.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = {"max_new": max(case.new)} if max_new else {}
    K.attention_mass(case.cache, case.bs, *case.table, case.q, case.new_offsets, lse, got,
                     observe=observe, kv_dtype=case.kv, status=status, **kw, **m)
    torch.cuda.synchronize()
    want, tol = A.mass(case, lse, before, observe=observe, blocked=blocked, **kw)
    assert int(status.item()) == want_status
    A.close(got, want, tol)
    return got


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("geo", GEOMETRIES, ids=lambda g: "-".join(map(str, g.values())))
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1, 1], [5, 33, 17, 0, 129, 70]], ids=["one", "many"])
def test_mass(kv, geo, new):
    check_mass(A.Case(kv=kv, lengths=[5, 33, 200, 77, 300, 130], new=new, seed=20, **geo),
               k_scale=0.5)


@pytest.mark.parametrize("layout,kw", [
    (HND, {}), (HND, dict(kbs=4)), (XS, {}), (NHD, dict(interleaved=True)),
    (NHD, dict(pad=8)), (HND, dict(offset=8)), (XS, dict(offset=8))], ids=str)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [1, 1, 80, 40]], ids=["one", "many"])
def test_mass_layouts(layout, kw, kv, new):
    check_mass(A.Case(kv=kv, layout=layout, dim=128, lengths=[70, 1, 259, 90], new=new, seed=21,
                      **kw))


@pytest.mark.parametrize("observe", [0, 1, 16, 500])
@pytest.mark.parametrize("window,softcap", [(0, 0.0), (33, 0.0), (33, 15.0)])
@pytest.mark.parametrize("new", [[1, 1, 1], [150, 3, 61]], ids=["one", "many"])
def test_mass_observed_window_softcap(observe, window, softcap, new):
    check_mass(A.Case(lengths=[600, 90, 61], new=new, seed=22, dim=128), observe=observe,
               window=window, softcap=softcap)


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [40, 1, 170, 64]], ids=["one", "many"])
def test_mass_empty_rows_and_first_positions(new):
    check_mass(A.Case(lengths=[0, 0, 30, 100], new=new, first=[0, 3, 0, 2], seed=23, dim=64),
               window=33, max_new=False)


@pytest.mark.parametrize("new", [[1, 1], [33, 100]])
def test_mass_bad_block_ids(new):
    case = A.Case(dim=128, lengths=[100, 300], new=new, seed=24)
    case.table[3][case.offsets[0] + 2] = -1
    case.table[3][case.offsets[1] + 5] = case.nb
    case.ids[case.offsets[0] + 2] = 0
    check_mass(case, blocked={0: (2,), 1: (5,)}, want_status=K.KVCS_STATUS_BAD_BLOCK_ID)


def test_mass_sums_to_the_observed_weight():
    """Every row's weights sum to 1, so a head's mass grows by rows seen."""
    case = A.Case(dim=128, lengths=[500, 90], new=[100, 1], seed=25)
    _, lse, _ = run(case, max_new=100)
    mass = torch.zeros((case.nb, case.heads, case.bs), device="cuda")
    K.attention_mass(case.cache, case.bs, *case.table, case.q, case.new_offsets, lse, mass,
                     max_new=100)
    total = mass.double().sum((0, 2)).cpu()
    assert torch.allclose(total, torch.full((case.heads,), 101.0 * case.group, dtype=torch.float64),
                          rtol=1e-4)


@pytest.mark.parametrize("new", [[1] * 9, [200, 90, 1]])
def test_mass_repeats_bit_for_bit(new):
    case = A.Case(dim=128, lengths=[1000 + 137 * i for i in range(len(new))], new=new, seed=26)
    _, lse, _ = run(case, max_new=max(new))
    got = []
    for _ in range(2):
        mass = torch.zeros((case.nb, case.heads, case.bs), device="cuda")
        K.attention_mass(case.cache, case.bs, *case.table, case.q, case.new_offsets, lse, mass,
                         max_new=max(new))
        got.append(mass)
    assert torch.equal(*got)


@pytest.mark.parametrize("R", [4, 12, 40])
def test_requests_that_share_rows_stay_within_the_workspace(R):
    """Offsets that decrease somewhere let requests share rows: more units
    than sound tables have.  They are flagged, and nothing is written behind
    the workspace that sound tables need, or in rows that no request owns."""
    case = A.Case(dim=64, lengths=[2048] * R, new=[0] * (R - 1) + [264], seed=31)
    case.new_offsets.copy_(torch.tensor([(r % 2) * 256 for r in range(R)] + [256]))
    n = K.attention_workspace_bytes(case.cache, case.bs, R, case.total, case.q)
    space = torch.full((n + (8 << 20),), 171, dtype=torch.uint8, device="cuda")
    out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
    _, _, status = run(case, workspace=space, out=out)
    assert status == K.KVCS_STATUS_BAD_REQUESTS
    assert (space[n:] == 171).all() and (out[256:] == 7).all()


@pytest.mark.parametrize("softcap", [0.5, 7.0, 40.0, 1e4])
@pytest.mark.parametrize("kv", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_capped_scores_on_either_side_of_the_cap(softcap, kv, dim):
    """Scores that all lie far above the cap, on both sides of it (within a
    tile too), and far below it."""
    case = A.Case(kv=kv, lengths=[700, 300], new=[130, 20], seed=33, dim=dim, scale=2.0)
    check(case, softcap=softcap, scale=4.0 / dim)
    check_mass(case, softcap=softcap, scale=4.0 / dim)
    check(case, softcap=softcap, scale=-4.0 / dim)


@pytest.mark.parametrize("kw", [{}, dict(window=700), dict(softcap=9.0, scale=-0.1)], ids=str)
@pytest.mark.parametrize("new,lengths", [([5, 1, 64, 130, 2], [9000, 30, 4100, 2000, 3]),
                                         ([17], [5000]), ([40] + [1] * 40, [12000] + [500] * 40),
                                         ([100, 20], [60, 7000])])
@pytest.mark.parametrize("dim", [64, 128])
def test_split_chunks_among_others(kw, new, lengths, dim):
    """Chunks whose token ranges are split and joined, beside decode steps,
    rows that see nothing, and parts that a window leaves empty."""
    case = A.Case(dim=dim, heads=2, group=4, lengths=lengths, new=new, seed=44)
    check(case, **kw)
    check(case, max_new="unknown", **kw)
    check_mass(case, **kw)


@pytest.mark.parametrize("kv", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 0), (128, 1500)])
def test_nonfinite_values_in_split_chunks(kv, dim, window):
    """NaN and infinite V that only the later rows of a split chunk see, in
    another part than most of their tokens, and NaN before the window."""
    case = A.Case(kv=kv, dim=dim, lengths=[6000], new=[64], seed=45)
    case.put(0, 1, 5990, torch.full((1, dim), float("nan")))
    case.put(0, 1, 5970, torch.full((1, dim), float("inf")))
    if window:
        case.put(0, 1, 100, torch.full((1, dim), float("nan")))
    out, lse, _ = run(case, window=window, max_new=64)
    ref = A.attention(case, window=window)
    A.close(lse, ref[1], ref[3])
    A.close(out, ref[0], ref[2])
    assert torch.isfinite(ref[0][:34]).all() and torch.isnan(ref[0][54:]).all()


def bits(case, poison=None, **kw):
    """Attention and mass of a case, after another call has left shared memory
    full of `poison`'s numbers."""
    m = max(case.new)
    if poison is not None:
        run(poison, max_new=max(poison.new))
    out, lse, _ = run(case, max_new=m, **kw)
    mass = torch.zeros((case.nb, case.heads, case.bs), device="cuda")
    if poison is not None:
        run(poison, max_new=max(poison.new))
    K.attention_mass(case.cache, case.bs, *case.table, case.q, case.new_offsets, lse, mass,
                     max_new=m, kv_dtype=case.kv, **kw)
    torch.cuda.synchronize()
    return out, lse, mass


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[1, 1], [40, 70]], ids=["one", "many"])
def test_capped_scores_hang_on_nothing_unseen(kv, dim, new):
    """What a row does not see never changes its bits: large finite values in
    slots past the last token, in later tokens and before the window, other
    requests' queries, and what another call has left in shared memory."""
    kw = dict(kv=kv, dim=dim, lengths=[300, 190], new=new, seed=50, bs=16)
    cap = dict(softcap=12.0, scale=dim ** -0.5, window=150)
    plain = A.Case(tail=0.0, **kw)
    out, lse, mass = bits(plain, **cap)
    ref = A.attention(plain, **cap)
    A.close(lse, ref[1], ref[3])
    big = 448.0 if kv == "fp8" else 6e4
    poison = A.Case(kv=kv, dim=dim, lengths=[2000] * 8, new=[64] * 8, seed=51,
                    scale=100.0 if kv == "fp8" else 3000.0)
    other = A.Case(tail=big, **kw)
    for r, n in enumerate(new):
        first = other.lengths[r] - n
        for t in range(max(0, first - 160), max(0, first - 150)):      # before every window
            other.put(r, 0, t, torch.full((1, dim), big))
        if n > 1:                                                      # seen by the last row alone
            other.put(r, 0, other.lengths[r] - 1, torch.full((1, dim), big))
    got = bits(other, poison=poison, **cap)
    same = torch.ones(plain.starts[-1], dtype=torch.bool)
    for r, n in enumerate(new):
        if n > 1:
            same[plain.starts[r + 1] - 1] = False
    assert torch.equal(out[same.cuda()], got[0][same.cuda()])
    assert torch.equal(lse[same.cuda()], got[1][same.cuda()])
    if max(new) == 1:
        for h in range(plain.heads):
            assert torch.equal(mass[:, h], got[2][:, h])
    # the second request's queries do not change the first one's mass
    other = A.Case(tail=big, **kw)
    other.q[other.starts[1]:] *= 100.0
    got = bits(other, poison=poison, **cap)
    ids = plain.ids[:plain.offsets[1]].long()
    assert torch.equal(mass[ids], got[2][ids])
    n = plain.starts[1]
    assert torch.equal(out[:n], got[0][:n]) and torch.equal(lse[:n], got[1][:n])


@pytest.mark.parametrize("softcap", [1e4, 1e6, 1e9])
@pytest.mark.parametrize("kv,new", [("bf16", [1, 1]), ("fp16", [130, 20]), ("fp8", [1, 1]),
                                    ("fp8", [130, 20])])
def test_caps_far_above_the_scores(softcap, kv, new):
    """A cap that scores never come near changes them by no more than their
    own rounding: tanh is right relative to the score, not to the cap.

    Bound: that of uncapped scores, and 2^-20 of a score for the capping: 2^-21
    for tanh and five roundings of 2^-24 (the two constants, the product with
    one, and the two products that join cap, x and tanh(x) / x)."""
    case = A.Case(kv=kv, lengths=[700, 300], new=new, seed=55, dim=128)
    want, bound = A.attention(case, softcap=softcap), A.attention(case)
    out, lse, _ = run(case, softcap=softcap, max_new=max(new))
    top = max(float(A.scores(case, r, h, 128 ** -0.5, 1.0, 0.0)[0].abs().max())
              for r in (0, 1) for h in range(case.heads * case.group))
    more = top * 2.0 ** -20
    widest = max(float(v[1].double().abs().max()) for v in case.values)
    A.close(out, want[0], bound[2] + 2 * more * widest)
    A.close(lse, want[1], bound[3] + more)
    before = torch.zeros((case.nb, case.heads, case.bs))
    exact = want[1].float().cuda()
    mass = before.cuda()
    K.attention_mass(case.cache, case.bs, *case.table, case.q, case.new_offsets, exact, mass,
                     max_new=max(new), kv_dtype=case.kv, softcap=softcap)
    A.close(mass, A.mass(case, exact, before, softcap=softcap)[0],
            A.mass(case, exact, before)[1] * (1 + 2 * more) + 2 * more *
            A.mass(case, exact, before, softcap=softcap)[0])


@pytest.mark.parametrize("spread", [0.1, 1.0])
@pytest.mark.parametrize("length", [1000, 65536])
@pytest.mark.parametrize("kv,dim,new", [("fp16", 64, 1), ("fp16", 128, 33), ("fp16", 64, 300),
                                        ("fp16", 80, 20), ("fp8", 128, 1), ("fp8", 64, 20),
                                        ("bf16", 128, 33)])
def test_small_weights_beside_a_large_one(kv, dim, new, length, spread):
    """One token takes nearly all weight and has a V of 0, as sinks have: the
    output is made of the many others' weights, about 2^-24 each.

    Bound: beyond attention_ref's, what a weight is off by where it is too
    small for fp16's full precision, half its smallest step: 2^-25 of 2^-14
    (chunk kernel: 2^-7) of the row's largest weight."""
    if length > 1000 and new > 100:
        pytest.skip("a long reference")
    case = A.Case(kv=kv, heads=1, group=2, dim=dim, lengths=[length], new=[new], seed=60,
                  scale=spread, tail=0.0)
    v = (case.values[0][1].float() + 1).to(case.kv)
    case.values[0][1] = v
    whole, raw = length // case.bs, v.view(torch.uint8).cuda()
    pool = case.pool.view(2, case.nb, case.bs, -1)
    ids = case.ids.long().cuda()
    pool[1, ids[:whole]] = raw[:whole * case.bs].view(whole, case.bs, -1)
    if length % case.bs:
        pool[1, ids[whole], :length % case.bs] = raw[whole * case.bs:].view(length % case.bs, -1)
    case.q[:, :, 0] = 8.0
    sink = torch.zeros((1, dim))
    sink[0, 0] = 17.0 * dim ** 0.5 / 8
    case.put(0, 0, 0, sink)
    case.put(0, 1, 0, torch.zeros((1, dim)))
    out, lse, status = run(case, v_scale=1024.0, max_new=new)
    ref = A.attention(case, v_scale=1024.0)
    assert status == 0 and float(ref[0].abs().max()) > 1e-3
    step = 2.0 ** -32 if kv == "fp16" and dim in (64, 128) and new * 2 > 16 else 2.0 ** -39
    lost = case.values[0][1].double().abs().sum(0)[0] * (step if kv != "bf16" else 0.0) * 1024.0
    A.close(out, ref[0], ref[2] + lost)
    A.close(lse, ref[1], ref[3])


@pytest.mark.parametrize("new", [[1, 1], [3, 40]], ids=["one", "many"])
def test_queries_and_scales_that_underflow_together(new):
    """Queries so small that a row's factor is 0 in 32 bits: all scores are 0,
    and masked ones stay masked."""
    case = A.Case(kv="fp8", lengths=[37, 100], new=new, seed=61, dim=64)
    case.q.fill_(1e-38)
    check(case, k_scale=1e-8)
    check_mass(case, k_scale=1e-8)


def test_outputs_belong_to_the_default_stream_given_by_its_handle():
    """A call on stream 0, by number, from within another stream: what it
    allocates belongs to stream 0, and to no other that the allocator would
    let it be used again on."""
    case = A.Case(dim=64, lengths=[400, 90], new=[1, 30], seed=62)
    want = run(case, max_new=30)
    with torch.cuda.stream(torch.cuda.Stream()):
        out, lse = K.paged_attention(case.cache, case.bs, *case.table, case.q, case.new_offsets,
                                     max_new=30, stream=0, total_positions=case.total)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for t in (out, lse):
        owner = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert owner == [0]


@pytest.mark.parametrize("dim", [64, 128])
def test_bad_blocks_among_many_units(dim):
    """Units of one and of two query tiles that follow one another on a CTA,
    some slowed down by the look-up of bad blocks in their last tokens."""
    g = torch.Generator().manual_seed(63)
    lengths = torch.randint(40, 500, (40,), generator=g).tolist()
    new = [min(n, 5 + (37 * i) % 120) for i, n in enumerate(lengths)]
    case = A.Case(dim=dim, heads=8, group=4, lengths=lengths, new=new, seed=63, tail=0.0)
    blocked = {}
    for r in range(0, 40, 3):
        last = case.counts[r] - 1
        blocked[r] = (last, max(0, last - 4))
        for b in blocked[r]:
            case.table[3][case.offsets[r] + b] = -1 if r % 2 else case.nb + r
    out, lse = check(case, blocked=blocked, want_status=K.KVCS_STATUS_BAD_BLOCK_ID)
    for _ in range(3):
        again = run(case, max_new=max(new))
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    check_mass(case, blocked=blocked, want_status=K.KVCS_STATUS_BAD_BLOCK_ID)
