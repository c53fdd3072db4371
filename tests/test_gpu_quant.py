"""kvcs_write_kv_quantised and kvcs_read_kv: stored values bit for bit against
the definition computed on the host, scales and values read back within half a
step of their types, and the cache as a whole: written, attended to, read back."""

import pytest
import torch

import attention_ref as A
import ext_ref as X
import paged_kv_cache_kvcs_gb300 as K
from paged_kv_cache_kvcs_gb300 import workloads as W

pytestmark = pytest.mark.gpu
NHD, HND, XS, LATENT = W.LAYOUT_NHD, W.LAYOUT_HND, W.LAYOUT_XSPLIT, W.LAYOUT_LATENT
DEV = "cuda"
INT8, FP8 = torch.int8, torch.float8_e4m3fn


class Cache:
    """One cache of bytes with its scales, and request tables over it."""

    def __init__(self, lengths, layout=NHD, heads=2, dim=64, bs=16, kbs=0, offset=0, pad=0, layer=0,
                 element=1, seed=0, first=None):
        g = torch.Generator().manual_seed(seed)
        self.layout, self.heads, self.dim, self.bs, self.lengths = layout, heads, dim, bs, lengths
        self.halves = 1 if layout == LATENT else 2
        self.element = element
        hb = dim * element
        self.first = first or [0] * len(lengths)
        counts = [max(0, -(-n // bs) - f) for n, f in zip(lengths, self.first)]
        self.offsets = [sum(counts[:i]) for i in range(len(counts) + 1)]
        self.nb = self.offsets[-1] + 3
        self.ids = torch.randperm(self.nb, generator=g)[:self.offsets[-1]].to(torch.int32)
        page = bs * heads * hb
        bstride = page + pad if pad else 0
        hstride = self.nb * bstride
        self.at = A.token_bytes(layout, self.halves, self.nb, bs, heads, hb, hstride, bstride, kbs)
        size = (int(self.at.max()) + 8) // 8 * 8
        buf = torch.full((size + 16,), 0x55, dtype=torch.uint8, device=DEV)
        skip = (offset - buf.data_ptr()) % 16
        self.pool = buf[skip:skip + size]
        self.spec = W.CacheSpec(self.pool, self.nb, layout, layer, 0, heads, hb, half_stride=hstride,
                                block_stride=bstride, kernel_block_size=kbs)
        self.scales = [torch.full((self.nb, heads, bs), 7.0, device=DEV) for _ in range(self.halves)]
        dev = lambda x, t: torch.tensor(x, dtype=t, device=DEV)  # noqa: E731
        self.table = [dev(self.offsets, torch.int64), dev(self.first, torch.int64),
                      dev(lengths, torch.int64), self.ids.to(DEV)]

    def slots(self, tokens):
        """Slots of (request, token) pairs."""
        return torch.tensor([int(self.ids[self.offsets[r] + t // self.bs - self.first[r]]) * self.bs
                             + t % self.bs for r, t in tokens], dtype=torch.int64)

    def bytes_of(self, half, slots):
        """[n, heads, head bytes] of the pool."""
        at = self.at[half, slots // self.bs, slots % self.bs]
        return self.pool.cpu()[at]

    def put(self, half, slots, stored):
        at = self.at[half, slots // self.bs, slots % self.bs]
        self.pool[at.to(DEV)] = stored.contiguous().view(torch.uint8).view(at.shape).to(DEV)

    def scale_kw(self):
        return dict(k_scales=self.scales[0], v_scales=self.scales[1] if self.halves == 2 else None)


def rows(n, heads, dim, dtype, seed, spread=4.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, dim), generator=g) * torch.exp2(torch.randn((n, heads, 1), generator=g) * spread)
    return x.to(dtype).to(DEV)


def check_write(c, tokens, keys, values, dtype, words=True, k_scale=None, v_scale=None, pad=0):
    """Writes the tokens, and compares all of the pool, the scales and the words."""
    slots = c.slots(tokens)
    pos = torch.tensor([t for _, t in tokens], dtype=torch.int64)
    sent = torch.cat([slots, torch.tensor([-1, -7, -2 ** 40][:pad], dtype=torch.int64)])
    sums = torch.zeros(c.nb, dtype=torch.int64, device=DEV) if words else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = c.pool.cpu().clone()
    scales_before = [s.cpu().clone() for s in c.scales]
    kw = c.scale_kw() if k_scale is None else dict(k_scale=k_scale, v_scale=v_scale)
    K.write_kv_quantised(c.spec, c.bs, keys, values, sent.to(DEV),
                         torch.cat([pos, torch.zeros(pad, dtype=torch.int64)]).to(DEV), kv_dtype=dtype,
                         block_sums=sums, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    n = len(tokens)
    for half, x in enumerate([keys, values][:c.halves]):
        stored, scales = X.quantised(x[:n].reshape(n, c.heads, c.dim), dtype,
                                     None if k_scale is None else (k_scale, v_scale)[half])
        at = c.at[half, slots // c.bs, slots % c.bs]
        want[at] = stored.view(torch.uint8).view(at.shape)
        if k_scale is None:
            ws = scales_before[half]
            ws[slots // c.bs, :, slots % c.bs] = scales
            got = c.scales[half].cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(ws))
            assert torch.equal(got.nan_to_num(), ws.nan_to_num())
    assert torch.equal(c.pool.cpu(), want)
    if words:      # the running words are the checksums of what is there, token by token
        held = torch.zeros(c.nb, dtype=torch.int64)
        for half in range(c.halves):
            P = c.dim // 8
            x = c.bytes_of(half, slots).contiguous().view(torch.int64)           # [n, heads, P]
            w = 2 * (pos[:, None, None] * (P * c.halves) + half * P + torch.arange(P)) + 1
            m = 2 * (c.spec.layer * 65536 + torch.arange(c.heads)) + 1
            held.index_add_(0, slots // c.bs, ((x * w).sum(-1) * m).sum(-1))
        assert torch.equal(sums.cpu(), held)


LAYOUTS = [(NHD, {}), (HND, {}), (HND, dict(kbs=4)), (XS, {}), (NHD, dict(pad=16)), (NHD, dict(pad=8)),
           (HND, dict(offset=8)), (XS, dict(offset=8))]


@pytest.mark.parametrize("layout,kw", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", [INT8, FP8])
@pytest.mark.parametrize("wide", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,dim", [(2, 64), (8, 128), (3, 80)])
def test_write(layout, kw, dtype, wide, heads, dim):
    c = Cache([37, 5, 18], layout, heads, dim, layer=3, **kw)
    tokens = [(r, t) for r, n in enumerate(c.lengths) for t in range(n)]
    order = torch.randperm(len(tokens), generator=torch.Generator().manual_seed(1)).tolist()
    tokens = [tokens[i] for i in order[:51]]
    k, v = (rows(54, heads, dim, wide, s) for s in (2, 3))
    check_write(c, tokens, k, v, dtype, pad=3)


@pytest.mark.parametrize("layout,heads,dim,bs", [
    (NHD, 1, 8, 7), (NHD, 5, 24, 16), (HND, 2, 8, 16), (NHD, 2, 512, 16), (NHD, 2, 520, 8), (HND, 1, 2048, 4),
    (XS, 1, 1040, 8), (LATENT, 1, 576, 16), (LATENT, 1, 40, 16), (LATENT, 1, 1000, 16), (NHD, 40, 128, 1)])
@pytest.mark.parametrize("dtype", [INT8, FP8])
def test_write_of_any_width(layout, heads, dim, bs, dtype):
    c = Cache([11, 1, 20], layout, heads, dim, bs)
    tokens = [(r, t) for r, n in enumerate(c.lengths) for t in range(n)]
    k = rows(len(tokens), heads, dim, torch.bfloat16, 4)
    v = None if layout == LATENT else rows(len(tokens), heads, dim, torch.bfloat16, 5)
    check_write(c, tokens, k, v, dtype)
    check_write(c, tokens[3:4], k[:1], None if v is None else v[:1], dtype, words=False)


@pytest.mark.parametrize("dtype", [INT8, FP8])
@pytest.mark.parametrize("wide", [torch.bfloat16, torch.float16])
def test_rows_of_special_values(dtype, wide):
    """Zeros, ones of equal magnitude, subnormal and largest values; a NaN or an
    infinity makes its row's scale NaN and its bytes 0."""
    c = Cache([16], heads=2, dim=64)
    big = torch.finfo(wide).max
    tiny = torch.finfo(wide).smallest_normal
    x = rows(16, 2, 64, wide, 6)
    x[0] = 0
    x[1] = -1.5
    x[2] = 0
    x[2, :, 5] = tiny / 2
    x[3, 0] = big
    x[3, 1, 7] = -big
    x[4] = tiny
    x[5, 0, 3] = float("nan")
    x[6, 1, 63] = float("inf")
    x[7, 0, 0] = -float("inf")
    x[8] = -0.0
    x[9, :, 1:] = 0
    # halfway between two integers of the stored type
    x[10] = (torch.arange(64, device=DEV) - 31.5).to(wide)
    x[10, :, 0] = 127
    check_write(c, [(0, t) for t in range(16)], x, x.flip(0).contiguous(), dtype)
    assert torch.isnan(c.scales[0]).sum() == 3


def test_one_scale_for_all():
    """float8 caches without scale arrays: values past the type's largest stop
    there, NaN stays."""
    c = Cache([40, 9], heads=2, dim=64)
    tokens = [(r, t) for r, n in enumerate(c.lengths) for t in range(n)]
    k, v = (rows(49, 2, 64, torch.bfloat16, s) for s in (7, 8))
    k[3, 0, 0], k[3, 1, 1], k[4, 0, 5] = float("inf"), -float("inf"), float("nan")
    check_write(c, tokens, k, v, FP8, k_scale=0.05, v_scale=0.3)
    assert all((s == 7).all() for s in c.scales)


def test_strided_rows_many_caches_and_kinds():
    """Several caches of different layouts and widths in one call, keys and
    values of a fused projection."""
    specs = [(NHD, 2, 64), (HND, 2, 64), (XS, 4, 32), (NHD, 1, 128)]
    n = 33
    caches = [Cache([n], layout, h, d, layer=i, seed=9) for i, (layout, h, d) in enumerate(specs)]
    fused = rows(n, 1, 4 * 384, torch.bfloat16, 10).view(n, 4 * 384)
    keys = [fused[:, 384 * i:384 * i + 128].view(n, h, d) for i, (_, h, d) in enumerate(specs)]
    values = [fused[:, 384 * i + 128:384 * i + 256].view(n, h, d) for i, (_, h, d) in enumerate(specs)]
    slots = caches[0].slots([(0, t) for t in range(n)])
    pos = torch.arange(n, device=DEV)
    sums = torch.zeros(caches[0].nb, dtype=torch.int64, device=DEV)
    scales = dict(k_scales=[c.scales[0] for c in caches], v_scales=[c.scales[1] for c in caches])
    K.write_kv_quantised([c.spec for c in caches], 16, keys, values, slots.to(DEV), pos, kv_dtype=INT8,
                         block_sums=sums, **scales)
    for c, k, v in zip(caches, keys, values):
        for half, x in enumerate((k, v)):
            stored, s = X.quantised(x, INT8)
            assert torch.equal(c.bytes_of(half, slots), stored.view(torch.uint8))
            assert torch.equal(c.scales[half].cpu()[slots // 16, :, slots % 16], s)
    words = K.block_checksums([c.spec for c in caches], 16, *caches[0].table)
    assert torch.equal(words, sums[caches[0].ids.to(DEV).long()])
    # all of them read back, into rows of a wider buffer
    wide = torch.full((n + 2, 4 * 384), 9.0, dtype=torch.float16, device=DEV)
    ko = [wide[:, 384 * i:384 * i + 128].view(n + 2, h, d) for i, (_, h, d) in enumerate(specs)]
    vo = [wide[:, 384 * i + 128:384 * i + 256].view(n + 2, h, d) for i, (_, h, d) in enumerate(specs)]
    K.read_kv([c.spec for c in caches], 16, *caches[0].table, torch.tensor([1, n + 1], device=DEV),
              keys=ko, values=vo, kv_dtype=INT8, **scales)
    for x, y in zip(keys + values, ko + vo):
        stored, s = X.quantised(x, INT8)
        want = (stored.float() * s[..., None]).half()
        assert torch.equal(y[1:-1].cpu(), want)
    assert (wide[0] == 9).all() and (wide[-1] == 9).all()
    assert (wide.view(n + 2, 4, 384)[:, :, 256:] == 9).all()


def test_more_caches_than_a_launch_holds():
    n, L = 3, 70
    c = Cache([n], heads=1, dim=16)
    pools = torch.zeros((L, c.pool.numel()), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((L, 2, c.nb, 1, 16), device=DEV)
    specs = [W.CacheSpec(pools[i], c.nb, NHD, i, 0, 1, 16) for i in range(L)]
    x = rows(n, L, 16, torch.bfloat16, 11).transpose(0, 1).contiguous().view(L, n, 1, 16)
    slots = c.slots([(0, t) for t in range(n)]).to(DEV)
    ks, vs = list(scales[:, 0].unbind(0)), list(scales[:, 1].unbind(0))
    sums = torch.zeros(c.nb, dtype=torch.int64, device=DEV)
    before = K.launch_count()
    K.write_kv_quantised(specs, 16, list(x.unbind(0)), list(x.flip(1).contiguous().unbind(0)), slots,
                         torch.arange(n, device=DEV), kv_dtype=FP8, k_scales=ks, v_scales=vs,
                         block_sums=sums)
    assert K.launch_count() == before + 2
    assert torch.equal(K.block_checksums(specs, 16, *c.table), sums[c.ids.to(DEV).long()])
    k, v = K.read_kv(specs, 16, *c.table, torch.tensor([0, n], device=DEV), kv_dtype=FP8, k_scales=ks,
                     v_scales=vs)
    for i in range(L):
        for y, z in ((k[i], x[i]), (v[i], x[i].flip(0))):
            stored, s = X.quantised(z, FP8)
            assert torch.equal(y.cpu(), (stored.float() * s[..., None]).to(torch.bfloat16))


def test_write_flags_bad_slots_and_positions():
    c = Cache([20], heads=2, dim=32, bs=8)
    k = rows(4, 2, 32, torch.bfloat16, 12)
    sums = torch.zeros(c.nb, dtype=torch.int64, device=DEV)
    for slots, positions, want in (([c.nb * 8, 2 ** 50, 3, -1], [0, 1, 2, 3], K.KVCS_STATUS_BAD_BLOCK_ID),
                                   ([4, 5, -1, -1], [-3, 1, 0, 0], K.KVCS_STATUS_BAD_REQUESTS)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        K.write_kv_quantised(c.spec, 8, k, k, torch.tensor(slots, device=DEV),
                             torch.tensor(positions, device=DEV), kv_dtype=INT8, block_sums=sums,
                             status=status, **c.scale_kw())
        assert int(status.item()) == want
    stored, scales = X.quantised(k, INT8)
    assert torch.equal(c.bytes_of(0, torch.tensor([3, 4, 5])), stored[[2, 0, 1]].view(torch.uint8))
    assert torch.equal(c.scales[1].cpu()[0, :, 3:6].T, scales[[2, 0, 1]])
    assert (c.scales[0] != 7).sum() == 3 * 2      # no scale of a token that was not written


# ---------------------------------------------------------------------------
# reading
# ---------------------------------------------------------------------------

def check_read(c, kv_dtype, out, count, scaled, k_scale=1.0, v_scale=1.0, **kw):
    """Reads the last count[r] tokens of every request."""
    g = torch.Generator().manual_seed(13)
    tokens = [(r, t) for r, n in enumerate(c.lengths) for t in range(c.first[r] * c.bs, n)]
    slots = c.slots(tokens)
    held = []
    for half in range(c.halves):
        x = torch.randn((len(tokens), c.heads, c.dim), generator=g) * 20
        x = x.clamp(-127, 127).round().to(INT8) if kv_dtype == INT8 else x.to(kv_dtype)
        c.put(half, slots, x)
        x = x.double()
        if scaled:
            s = torch.rand((len(tokens), c.heads), generator=g) + 0.01
            c.scales[half].fill_(float("nan"))
            c.scales[half][(slots // c.bs).to(DEV), :, (slots % c.bs).to(DEV)] = s.to(DEV)
            x = x * s[..., None].double()
        held.append(x * (v_scale if half else k_scale))
    starts = [2]
    for n in count:
        starts.append(starts[-1] + n)
    total = starts[-1] + 3
    shape = (total, c.heads, c.dim)
    ko, vo = (torch.full(shape, 5.0, dtype=out, device=DEV) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.read_kv(c.spec, c.bs, *c.table, torch.tensor(starts, device=DEV), keys=ko,
              values=vo if c.halves == 2 else None, kv_dtype=kv_dtype, k_scale=k_scale, v_scale=v_scale,
              status=status, **(c.scale_kw() if scaled else {}), **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    index = {t: i for i, t in enumerate(tokens)}
    for half, y in enumerate([ko, vo][:c.halves]):
        y = y.cpu()
        assert (y[:2] == 5).all() and (y[-3:] == 5).all()
        at = [index[(r, c.lengths[r] - n + i)] for r, n in enumerate(count) for i in range(n)]
        want = held[half][at]
        # a scale's product and the value's in 32 bits, and the output's rounding
        tol = want.abs() * (A.HALF_STEP[out] + 2.0 ** -22) + torch.finfo(out).smallest_normal * A.HALF_STEP[out]
        A.close(y[2:-3], want, tol)


@pytest.mark.parametrize("layout,kw", LAYOUTS, ids=str)
@pytest.mark.parametrize("kv", ["int8s", "fp8s", "fp8", "bf16", "fp16"])
@pytest.mark.parametrize("heads,dim", [(2, 64), (8, 128), (3, 80)])
def test_read(layout, kw, kv, heads, dim):
    dtype = {"int8s": INT8, "fp8s": FP8, "fp8": FP8, "bf16": torch.bfloat16, "fp16": torch.float16}[kv]
    c = Cache([37, 5, 180], layout, heads, dim, element=dtype.itemsize, **kw)
    for out in (torch.bfloat16, torch.float16):
        check_read(c, dtype, out, [37, 2, 101], kv[-1] == "s", k_scale=0.5, v_scale=3.0)


@pytest.mark.parametrize("layout,heads,dim,bs", [
    (NHD, 1, 8, 7), (NHD, 5, 24, 16), (HND, 2, 8, 16), (NHD, 2, 520, 8), (HND, 1, 2048, 4), (XS, 1, 1040, 8),
    (LATENT, 1, 576, 16), (LATENT, 1, 40, 16), (LATENT, 1, 1000, 16), (NHD, 40, 128, 1)])
def test_read_of_any_width(layout, heads, dim, bs):
    c = Cache([11, 0, 1, 20, 40], layout, heads, dim, bs, first=[0, 0, 0, 0, 1])
    for count in ([11, 0, 1, 20, 40 - bs], [0, 0, 1, 0, 0], [3, 0, 0, 9, 1]):
        check_read(c, INT8, torch.bfloat16, count, True)


def test_read_many_tokens():
    c = Cache([3000, 1, 1777, 4000], heads=4, dim=64)
    check_read(c, INT8, torch.float16, [3000, 1, 1700, 4000], True)


def test_read_flags():
    """Bad blocks read as zeros; rows before a request's first listed token too;
    rows of bad offsets, and of no request, stay."""
    c = Cache([40, 40, 40, 40], heads=2, dim=32, first=[0, 0, 1, 0])
    c.pool.fill_(1)
    c.table[3][c.offsets[0] + 1] = -1
    c.table[3][c.offsets[1] + 2] = c.nb
    c.table[1][3] = -5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def read(offsets, total):
        out = [torch.full((total, 2, 32), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        status.zero_()
        K.read_kv(c.spec, 16, *c.table, torch.tensor(offsets, device=DEV), keys=out[0], values=out[1],
                  kv_dtype=INT8, k_scales=torch.ones_like(c.scales[0]),
                  v_scales=torch.ones_like(c.scales[0]), status=status)
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1])
        return out[0][:, 0, 0].cpu().float()
    y = read([0, 40, 80, 120, 160], 165)
    want = torch.ones(165)
    want[16:32] = 0
    want[40 + 32:80] = 0
    want[80:96] = 0                # the third lists its blocks from position 1 on
    want[120:160] = 0              # no tokens known of a request with bad tables
    want[160:] = 5
    assert int(status.item()) == K.KVCS_STATUS_BAD_BLOCK_ID | K.KVCS_STATUS_BAD_REQUESTS
    assert torch.equal(y, want), (y - want).nonzero()
    c.table[1][3] = 0
    y = read([0, 3, 3, 9, 7], 12)     # offsets that decrease: the last request's rows
    assert int(status.item()) & K.KVCS_STATUS_BAD_REQUESTS
    y = read([0, 3, 6, 9, 50], 12)    # or that leave the rows
    assert int(status.item()) & K.KVCS_STATUS_BAD_REQUESTS
    assert torch.equal(y[:9], torch.tensor([1.0] * 3 + [0.0] * 3 + [1.0] * 3)) and (y[9:] == 5).all()


# ---------------------------------------------------------------------------
# the calls, and the operators together
# ---------------------------------------------------------------------------

def test_graphs_streams_and_determinism():
    n = 70
    c = Cache([n], heads=2, dim=128)
    slots, pos = c.slots([(0, t) for t in range(n)]).to(DEV), torch.arange(n, device=DEV)
    k, v = (rows(n, 2, 128, torch.bfloat16, s) for s in (14, 15))
    ends = torch.tensor([0, n], device=DEV)
    ko, vo = (torch.zeros((n, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def both(stream=None):
        K.write_kv_quantised(c.spec, 16, k, v, slots, pos, kv_dtype=INT8, stream=stream, **c.scale_kw())
        K.read_kv(c.spec, 16, *c.table, ends, keys=ko, values=vo, kv_dtype=INT8, total_positions=c.offsets[-1],
                  stream=stream, **c.scale_kw())

    def want(x):
        stored, s = X.quantised(x, INT8)
        return (stored.float() * s[..., None]).to(torch.bfloat16).to(DEV)
    both()
    assert torch.equal(ko, want(k)) and torch.equal(vo, want(v))
    ko.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    torch.cuda.synchronize()
    assert torch.equal(ko, want(k))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for s in (2.0, -0.3):
        k.mul_(s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ko, want(k)) and torch.equal(vo, want(v))


@pytest.mark.parametrize("dtype", [INT8, FP8])
@pytest.mark.parametrize("layout", [NHD, HND, XS])
def test_a_cache_from_prompt_to_tree(dtype, layout):
    """A prompt is quantised as it is written, a drafted tree behind it; the tree
    attends to the cache under a window with first tokens kept; the cache reads
    back as what attention took it for, and its words are its checksums."""
    heads, group, dim, prompt, tree_n = 2, 4, 128, 700, 9
    n = prompt + tree_n
    c = Cache([n, 50], layout, heads, dim, seed=16)
    k, v = (rows(n + 50, heads, dim, torch.bfloat16, s, spread=0.5) for s in (17, 18))
    tokens = [(0, t) for t in range(n)] + [(1, t) for t in range(50)]
    slots = c.slots(tokens).to(DEV)
    pos = torch.tensor([t for _, t in tokens], device=DEV)
    sums = torch.zeros(c.nb, dtype=torch.int64, device=DEV)
    for part in (slice(0, prompt), slice(prompt, n), slice(n, n + 50)):
        K.write_kv_quantised(c.spec, 16, k[part], v[part], slots[part], pos[part], kv_dtype=dtype,
                             block_sums=sums, **c.scale_kw())
    new = [tree_n, 1]
    trees = [X.random_tree(tree_n, torch.Generator().manual_seed(19)), [-1]]
    up = torch.tensor(sum(trees, []), dtype=torch.int32, device=DEV)
    q = rows(tree_n + 1, heads * group, dim, torch.bfloat16, 20, spread=0.0)
    offsets = torch.tensor([0, tree_n, tree_n + 1], device=DEV)
    out, lse = K.tree_attention(c.spec, 16, *c.table, q, offsets, up, kv_dtype=dtype, window=200, sinks=4,
                                max_new=tree_n, **c.scale_kw())
    ko, vo = K.read_kv(c.spec, 16, *c.table, torch.tensor([0, n, n + 50], device=DEV), kv_dtype=dtype,
                       **c.scale_kw())
    words = K.block_checksums([c.spec], 16, *c.table)
    torch.cuda.synchronize()

    class Held(X.ScaledCase):       # the reference's view of the same cache
        def __init__(self):
            self.lengths, self.new, self.first, self.bs = [n, 50], new, [0, 0], 16
            self.heads, self.group, self.dim, self.q_dtype = heads, group, dim, torch.bfloat16
            self.starts, self.q, self.values = [0, tree_n, tree_n + 1], q, []
            for part in (slice(0, n), slice(n, n + 50)):
                both = []
                for x in (k, v):
                    stored, s = X.quantised(x[part], dtype)
                    both.append(stored.double() * s[..., None].double())
                self.values.append(torch.stack(both))
    held = Held()
    ref = X.attention(held, trees=trees, window=200, sinks=4)
    A.close(out, ref[0], ref[2])
    A.close(lse, ref[1], ref[3])
    for half, (y, x) in enumerate(((ko, k), (vo, v))):
        want = torch.cat([t[half] for t in held.values])
        A.close(y, want, want.abs() * (2.0 ** -8 + 2.0 ** -22))
        # and half a step of the stored type from what was written (a quotient of up to 127 is
        # off by 2^-23 of itself, an eighth of 2^-13 of the half step; the scale by less)
        top = x.cpu().double().abs().amax(-1, keepdim=True)
        step = top / 127 / 2 if dtype == INT8 else x.cpu().double().abs() * 2.0 ** -4 + top * 2.0 ** -10 / 448
        assert ((want - x.cpu().double()).abs() <= step * (1 + 2.0 ** -13)).all()
    assert torch.equal(words, sums[c.ids.to(DEV).long()])


def test_little_to_do():
    c = Cache([0, 30], heads=2, dim=64)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    before = c.pool.clone()
    K.write_kv_quantised(c.spec, 16, k, k, none, none, kv_dtype=INT8, **c.scale_kw())
    ko, vo = K.read_kv(c.spec, 16, *c.table, torch.zeros(3, dtype=torch.int64, device=DEV), kv_dtype=INT8,
                       **c.scale_kw())
    torch.cuda.synchronize()
    assert ko.shape == vo.shape == (0, 2, 64) and torch.equal(c.pool, before)


def test_torch_refusals():
    c = Cache([30], heads=2, dim=64)
    k = rows(30, 2, 64, torch.bfloat16, 21)
    slots, pos = c.slots([(0, t) for t in range(30)]).to(DEV), torch.arange(30, device=DEV)
    ok = dict(kv_dtype=INT8, **c.scale_kw())

    def write(keys=k, values=k, slots=slots, pos=pos, **kw):
        K.write_kv_quantised(c.spec, 16, keys, values, slots, pos, **{**ok, **kw})
    write()
    for bad in (dict(keys=k.float()), dict(keys=k[:29]), dict(values=k.half()), dict(values=k.cpu()),
                dict(keys=k[:, :, :32]), dict(keys=k.transpose(1, 2)), dict(keys=k[:, :, ::2]),
                dict(slots=slots.int()), dict(pos=pos[:-1]), dict(kv_dtype=torch.uint8),
                dict(k_scales=c.scales[0].double()), dict(v_scales=c.scales[0][:-1]),
                dict(block_sums=slots[:2])):
        with pytest.raises(ValueError):
            write(**bad)
    for bad in (dict(kv_dtype=torch.bfloat16), dict(k_scales=None, v_scales=None), dict(k_scale=2.0)):
        with pytest.raises((ValueError, K.KvcsError)):
            write(**bad)
    ends = torch.tensor([0, 30], device=DEV)

    def read(ends=ends, **kw):
        return K.read_kv(c.spec, 16, *c.table, ends, **{**ok, **kw})
    read()
    for bad in (dict(ends=ends.int()), dict(ends=ends[:1]), dict(keys=k.float()), dict(keys=k, values=k[:20]),
                dict(dtype=torch.float32), dict(kv_dtype=torch.uint8), dict(total_tokens=31, keys=k)):
        with pytest.raises(ValueError):
            read(**bad)


def test_scales_with_the_heads_last_are_refused():
    """As many scales in another order, contiguous: each call says so.  A flat
    tensor, and one of more blocks, are taken."""
    case = X.ScaledCase("int8", dim=64, heads=2, bs=16, lengths=[40], new=[2], seed=44)
    n = case.lengths[0]
    k = torch.randn(n, 2, 64, device=DEV).bfloat16()
    slots = case.table[3].long().repeat_interleave(16)[:n] * 16 + torch.arange(n, device=DEV) % 16
    ends = torch.tensor([0, n], device=DEV)

    def calls(ks, vs):
        s = dict(kv_dtype=torch.int8, k_scales=ks, v_scales=vs)
        return (lambda: K.paged_attention(case.cache, 16, *case.table, case.q, case.new_offsets, **s),
                lambda: K.tree_attention(case.cache, 16, *case.table, case.q, case.new_offsets,
                                         torch.full((2,), -1, dtype=torch.int32, device=DEV), **s),
                lambda: K.write_kv_quantised(case.cache, 16, k, k, slots, torch.arange(n, device=DEV), **s),
                lambda: K.read_kv(case.cache, 16, *case.table, ends, **s))
    ks, vs = case.k_scales, case.v_scales
    last = ks.transpose(1, 2).contiguous()
    for bad in ((last, last), (ks, last), (last, vs)):
        for call in calls(*bad):
            with pytest.raises(ValueError, match="heads before slots"):
                call()
    for call in calls(ks.reshape(-1), torch.cat([vs, vs])):
        call()
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Blocks beyond 4 GiB from the pool's base."""
    nb, H, bs, D = 1100000, 4, 16, 64
    if torch.cuda.mem_get_info()[0] < 4 * nb * bs * H * D:
        pytest.skip("needs 18 GB")
    big = torch.zeros((2, nb, bs, H, D), dtype=INT8, device=DEV)
    scales = [torch.zeros((nb, H, bs), device=DEV) for _ in range(2)]
    spec = W.CacheSpec(big, nb, NHD, 0, 0, H, D)
    k = rows(40, H, D, torch.bfloat16, 22)
    ids = torch.tensor([nb - 1, 3, nb - 7], dtype=torch.int32, device=DEV)
    t = torch.arange(40, device=DEV)
    slots = ids[t // bs].long() * bs + t % bs
    K.write_kv_quantised(spec, bs, k, k.flip(0).contiguous(), slots, t, kv_dtype=INT8, k_scales=scales[0],
                         v_scales=scales[1])
    one = lambda x: torch.tensor(x, device=DEV)  # noqa: E731
    ko, vo = K.read_kv(spec, bs, one([0, 3]), one([0]), one([40]), ids, one([0, 40]), k_scales=scales[0],
                       v_scales=scales[1])
    stored, s = X.quantised(k, INT8)
    want = (stored.float() * s[..., None]).to(torch.bfloat16)
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want.flip(0))
    assert int(torch.count_nonzero(big[:, [3, nb - 7, nb - 1]])) == 2 * int((stored != 0).sum())
