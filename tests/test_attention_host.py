"""The attention, attention-mass and eviction entry points without a GPU:
bad arguments are refused on the host, before any CUDA call (a call that
passes its checks returns KVCS_ECUDA here, where there is no GPU)."""

import ctypes
import math

import pytest
import torch

import paged_kv_cache_kvcs_gb300 as K
from paged_kv_cache_kvcs_gb300 import _binding as B
from test_abi_host import FakeCache
from test_binding_host import FakeTensor

NO_GPU = not torch.cuda.is_available()
pytestmark = pytest.mark.skipif(not NO_GPU, reason="fake addresses: only where nothing can run")


def attention(**kw):
    a = B.kvcs_attention(q=1 << 20, q_stride=0, new_offsets=1 << 21, total_new=4, max_new=0,
                         q_heads=32, q_dtype=0, kv_dtype=0, scale=0.1, softcap=0.0, k_scale=1.0,
                         v_scale=1.0, window=0, out=1 << 22, lse=1 << 23, workspace=1 << 24,
                         workspace_bytes=1 << 30, observe=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


REQS = dict(num_requests=2, pos_offsets=1 << 12, first_position=1 << 13, num_tokens=1 << 14,
            block_ids=1 << 15)


def attend(cache=None, bs=16, positions=10, reqs=None, mass=False, **kw):
    arr = K.cache_array([cache or FakeCache()])
    r = B.kvcs_requests(**{**REQS, **(reqs or {})})
    a = attention(**kw)
    lib = K.load_library()
    if mass:
        return lib.kvcs_attention_mass(arr, bs, ctypes.byref(r), positions, ctypes.byref(a),
                                       1 << 25 if mass is True else mass, None, None)
    return lib.kvcs_paged_attention(arr, bs, ctypes.byref(r), positions, ctypes.byref(a), None,
                                    None)


@pytest.mark.parametrize("mass", [False, True])
def test_attention_refusals(mass):
    def code(*a, **kw):
        return attend(*a, mass=mass, **kw)
    assert code() == K.KVCS_ECUDA
    assert code(FakeCache(layout=1, kernel_block_size=4)) == K.KVCS_ECUDA
    assert code(FakeCache(layout=3), kv_dtype=1, q_dtype=1) == K.KVCS_ECUDA
    assert code(FakeCache(head_bytes=128), kv_dtype=2, q_dtype=1) == K.KVCS_ECUDA
    # types
    for bad in (dict(kv_dtype=3), dict(kv_dtype=-1), dict(q_dtype=2), dict(q_dtype=1),
                dict(kv_dtype=1)):
        assert code(**bad) == K.KVCS_EINVAL, bad
    # sizes
    for bad in (dict(q_heads=30), dict(q_heads=0), dict(total_new=-1), dict(max_new=5),
                dict(max_new=-1), dict(window=-1), dict(observe=-1), dict(q_stride=-8),
                dict(q_stride=32 * 128 - 8), dict(q_stride=32 * 128 + 4)):
        assert code(**bad) == K.KVCS_EINVAL, bad
    # numbers
    for name in ("scale", "k_scale", "v_scale", "softcap"):
        for v in (math.nan, math.inf):
            assert code(**{name: v}) == K.KVCS_EINVAL, name
    assert code(softcap=-1.0) == K.KVCS_EINVAL
    # pointers
    for bad in (dict(q=None), dict(q=(1 << 20) + 8), dict(new_offsets=None),
                dict(lse=(1 << 23) + 2)):
        assert code(**bad) == K.KVCS_EINVAL, bad
    for bad in (dict(pos_offsets=None), dict(first_position=None), dict(num_tokens=None),
                dict(block_ids=None), dict(num_requests=-1)):
        assert code(reqs=bad) == K.KVCS_EINVAL, bad
    assert code(positions=-1) == K.KVCS_EINVAL
    # caches
    assert code(FakeCache(layout=4, piece_bytes=4)) == K.KVCS_EINVAL
    assert code(FakeCache(base=(1 << 20) + 4)) == K.KVCS_EINVAL
    assert code(bs=0) == K.KVCS_EINVAL
    assert code(FakeCache(layout=2, num_heads=1, head_bytes=1152)) == K.KVCS_EUNSUPPORTED
    assert code(FakeCache(head_bytes=1024)) == K.KVCS_EUNSUPPORTED         # 512 elements
    assert code(FakeCache(head_bytes=24)) == K.KVCS_EUNSUPPORTED           # 12
    assert code(FakeCache(head_offset=65530, num_heads=8)) == K.KVCS_EUNSUPPORTED
    assert code(bs=1 << 20) == K.KVCS_EUNSUPPORTED                          # a 2 GiB page
    assert code(total_new=1 << 26) == K.KVCS_EUNSUPPORTED                   # 2^31 rows
    # nothing to do
    assert code(total_new=0, q=None, new_offsets=None) == K.KVCS_OK
    assert code(reqs=dict(num_requests=0, pos_offsets=None)) == K.KVCS_OK


def test_attention_alone():
    for bad in (dict(out=None), dict(out=(1 << 22) + 8), dict(workspace=None),
                dict(workspace=(1 << 24) + 8)):
        assert attend(**bad) == K.KVCS_EINVAL, bad
    assert attend(lse=None) == K.KVCS_ECUDA            # lse is optional here ...
    assert attend(lse=None, mass=True) == K.KVCS_EINVAL   # ... and an input there
    assert attend(mass=(1 << 25) + 2) == K.KVCS_EINVAL


def test_workspace_sizes():
    fn = K.load_library().kvcs_attention_workspace

    def size(cache=None, requests=2, sms=152, positions=100, **kw):
        n = ctypes.c_int64(-1)
        a = attention(q=None, out=None, workspace=None, **kw)
        rc = fn(K.cache_array([cache or FakeCache()]), 16, requests, positions, ctypes.byref(a), sms,
                ctypes.byref(n))
        return n.value if rc == K.KVCS_OK else rc
    one = size(total_new=2, max_new=1)
    many = size(FakeCache(layout=3), total_new=400, max_new=200)
    assert 0 < one < many
    # few long rows: their token range is split, which takes room
    split = size(requests=1, positions=4000, total_new=64, max_new=64)
    assert size(requests=64, positions=4000, total_new=64 * 64, max_new=64) < split
    assert size(total_new=2, max_new=1, sms=76) < one
    assert size(q_heads=3) == K.KVCS_EINVAL
    assert size(requests=-1) == K.KVCS_EINVAL
    assert size(positions=-1) == K.KVCS_EINVAL
    assert fn(K.cache_array([FakeCache()]), 16, 2, 10, ctypes.byref(attention()), 152, None) == \
        K.KVCS_EINVAL


def evict(caches=None, positions=10, reqs=None, scores=None, n=None, **kw):
    caches = caches or [FakeCache()]
    ptrs = (ctypes.c_void_p * len(caches))(*(scores or [1 << 20] * len(caches)))
    ev = B.kvcs_eviction(ptrs, 1 << 16, 0, 0, None, None, 1 << 17, 1 << 30)
    for k, v in kw.items():
        setattr(ev, k, v)
    r = B.kvcs_requests(**{**REQS, **(reqs or {})})
    return K.load_library().kvcs_evict(K.cache_array(caches), len(caches) if n is None else n, 16,
                                       ctypes.byref(r), positions, ctypes.byref(ev), None, None)


def test_evict_refusals():
    assert evict() == K.KVCS_ECUDA
    assert evict([FakeCache(layout=2, num_heads=1, head_bytes=1152)]) == K.KVCS_ECUDA
    assert evict([FakeCache(layer=i) for i in range(300)]) == K.KVCS_ECUDA
    assert evict([FakeCache(layout=4, piece_bytes=4)]) == K.KVCS_EINVAL
    assert evict([FakeCache(), FakeCache()]) == K.KVCS_EINVAL       # the same heads twice
    assert evict(n=0) == K.KVCS_EINVAL
    assert evict(scores=[None]) == K.KVCS_EINVAL
    assert evict(scores=[(1 << 20) + 2]) == K.KVCS_EINVAL
    for bad in (dict(sinks=-1), dict(recent=-1), dict(keep=None), dict(keep=(1 << 16) + 4),
                dict(new_block_ids=(1 << 16) + 2), dict(block_sums=(1 << 16) + 4),
                dict(workspace=None), dict(workspace=(1 << 17) + 8), dict(workspace_bytes=8)):
        assert evict(**bad) == K.KVCS_EINVAL, bad
    assert evict(positions=-1) == K.KVCS_EINVAL
    assert evict(reqs=dict(block_ids=None)) == K.KVCS_EINVAL
    assert evict(reqs=dict(num_requests=0)) == K.KVCS_OK
    assert evict(positions=0, reqs=dict(block_ids=None)) == K.KVCS_OK
    assert evict(positions=1 << 27) == K.KVCS_EUNSUPPORTED        # 2^31 tokens
    n = K.eviction_workspace_bytes([FakeCache()], 16, 2, 10)
    assert n > 0 and evict(workspace_bytes=n) == K.KVCS_ECUDA
    assert evict(workspace_bytes=n - 1) == K.KVCS_EINVAL
    with pytest.raises(K.KvcsError):
        K.eviction_workspace_bytes([FakeCache(head_bytes=12)], 16, 2, 10)


class FakeQ(FakeTensor):
    """A CUDA tensor [tokens, heads, dim] as far as the checks look."""

    def __init__(self, shape, dtype, dev=0, strides=None):
        super().__init__(shape[0] * shape[1] * shape[2], dtype, dev)
        self.shape = torch.Size(shape)
        self.strides = strides or (shape[1] * shape[2], shape[2], 1)

    def dim(self):
        return 3

    def stride(self, i):
        return self.strides[i]


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: torch.device("cuda", 0))
    R, P = 2, 10

    def call(q=None, cache=None, new=None, kv=None, fn=None, **kw):
        i64 = torch.int64
        table = (FakeTensor(R + 1, i64), FakeTensor(R, i64), FakeTensor(R, i64),
                 FakeTensor(P, torch.int32))
        fn = fn or K.paged_attention
        return fn(cache or FakeCache(), 16, *table,
                  FakeQ((4, 32, 128), torch.bfloat16) if q is None else q,
                  new or FakeTensor(R + 1, i64), total_positions=P, kv_dtype=kv, **kw)

    cpu = torch.zeros((4, 32, 128), dtype=torch.bfloat16)
    for bad, what in ((dict(q=cpu), "CUDA"),
                      (dict(q=FakeQ((4, 32, 128), torch.float32)), "bfloat16"),
                      (dict(q=FakeQ((4, 32, 128), torch.bfloat16, dev=1)), "runs on"),
                      (dict(q=FakeQ((4, 32, 64), torch.bfloat16)), "elements"),
                      (dict(q=FakeQ((4, 32, 128), torch.bfloat16, strides=(4096, 1, 32))), "packed"),
                      (dict(q=FakeQ((4, 32, 128), torch.bfloat16, strides=(128, 512, 1))), "packed"),
                      (dict(kv=torch.float32), "kv_dtype"),
                      (dict(new=FakeTensor(R, torch.int64)), "new_offsets"),
                      (dict(new=FakeTensor(R + 1, torch.int32)), "new_offsets"),
                      (dict(out=FakeTensor(10, torch.bfloat16)), "out"),
                      (dict(out=FakeTensor(1 << 20, torch.float16)), "out"),
                      (dict(out=FakeTensor(1 << 20, torch.bfloat16),
                            lse=FakeTensor(3, torch.float32)), "lse")):
        with pytest.raises(ValueError, match=what):
            call(**bad)
    with pytest.raises(K.KvcsError):     # the library's own refusal
        call(q=FakeQ((4, 30, 128), torch.bfloat16), out=FakeTensor(1 << 20, torch.bfloat16),
             lse=FakeTensor(1 << 20, torch.float32))

    def mass(*a, **kw):
        lse = kw.pop("lse", FakeTensor(128, torch.float32))
        m = kw.pop("m", FakeTensor(100 * 8 * 16, torch.float32))
        return K.attention_mass(*a, lse, m, **kw)
    for bad, what in ((dict(lse=FakeTensor(127, torch.float32)), "lse"),
                      (dict(m=FakeTensor(100 * 8 * 16 - 1, torch.float32)), "mass"),
                      (dict(m=FakeTensor(100 * 8 * 16, torch.float16)), "mass")):
        with pytest.raises(ValueError, match=what):
            call(fn=mass, **bad)

    def ev(*a, **kw):
        table = a[2:6]
        kw.pop("kv_dtype")
        sc = kw.pop("sc", [FakeTensor(100 * 8 * 16, torch.float32)])
        keep = kw.pop("keep", FakeTensor(R, torch.int64))
        return K.evict([a[0]], 16, *table, sc, keep, **kw)
    for bad, what in ((dict(sc=[]), "one tensor per cache"),
                      (dict(sc=[FakeTensor(99, torch.float32)]), "scores"),
                      (dict(keep=FakeTensor(1, torch.int64)), "keep"),
                      (dict(new_block_ids=FakeTensor(P - 1, torch.int32)), "new_block_ids"),
                      (dict(block_sums=FakeTensor(99, torch.int64)), "block_sums"),
                      (dict(status=FakeTensor(1, torch.float32)), "status")):
        with pytest.raises(ValueError, match=what):
            call(fn=ev, **bad)


def test_evictions_too_large_are_refused_before_any_work():
    """More rows than a launch can number, or more tokens, in the call and in
    its workspace's size alike; a refusal leaves words and caches as they
    were (here, without a GPU, any work at all would be KVCS_ECUDA)."""
    def size(caches, requests, positions):
        n = ctypes.c_int64(-1)
        rc = K.load_library().kvcs_eviction_workspace(
            K.cache_array(caches), len(caches), 16, requests, positions, ctypes.byref(n))
        return n.value if rc == K.KVCS_OK else rc
    small, large = FakeCache(layer=0, num_heads=1), FakeCache(layer=1, num_heads=8)
    many = dict(num_requests=1 << 24)                  # 2^27 rows of the large cache
    for caches in ([large], [small, large]):
        assert evict(caches, reqs=many, block_sums=1 << 26, workspace_bytes=1 << 62) == \
            K.KVCS_EUNSUPPORTED
        assert size(caches, 1 << 24, 10) == K.KVCS_EUNSUPPORTED
    fewer = dict(num_requests=(1 << 24) - 1)
    assert evict([small, large], reqs=fewer, workspace_bytes=1 << 62) == K.KVCS_ECUDA
    assert size([small, large], (1 << 24) - 1, 10) > 0
    assert size([large], 2, 1 << 27) == K.KVCS_EUNSUPPORTED         # 2^31 tokens
    assert size([large], 2, (1 << 27) - 1) > 0
    assert size([large], 2, 1 << 60) == K.KVCS_EUNSUPPORTED


@pytest.mark.parametrize("mass", [False, True])
def test_scales_that_32_bits_do_not_hold_are_refused(mass):
    """Each number may be finite and what the kernels make of them not: an
    infinite scale turns a product of 0 into NaN."""
    for bad in (dict(scale=1e30, k_scale=1e30), dict(scale=3e38), dict(softcap=3e38),
                dict(softcap=1e-30, scale=1e30), dict(softcap=1e38, scale=0.1),
                dict(scale=-1e30, k_scale=1e30)):
        assert attend(mass=mass, **bad) == K.KVCS_EINVAL, bad
    for good in (dict(scale=1e-30, k_scale=1e-30), dict(softcap=50.0, scale=1e-37),
                 dict(softcap=1e30), dict(scale=0.0, softcap=50.0),
                 dict(scale=-1.0, softcap=1e-3), dict(scale=1e38)):
        assert attend(mass=mass, **good) == K.KVCS_ECUDA, good


@pytest.mark.parametrize("mass", [False, True])
def test_requests_of_2_30_new_tokens_are_refused(mass):
    """Positions of new tokens are 31-bit numbers too."""
    one = FakeCache(num_heads=1, head_bytes=16)
    n = 1 << 30
    assert attend(one, mass=mass, q_heads=1, total_new=n) == K.KVCS_EUNSUPPORTED
    assert attend(one, mass=mass, q_heads=1, total_new=n + 5, max_new=n) == K.KVCS_EUNSUPPORTED
    space = dict(workspace_bytes=1 << 50)
    assert attend(one, mass=mass, q_heads=1, total_new=n - 1, **space) == K.KVCS_ECUDA
    assert attend(one, mass=mass, q_heads=1, total_new=n + 5, max_new=n - 1, **space) == K.KVCS_ECUDA


def test_misaligned_tables_are_refused():
    """Tables that the kernels could not read without a fault."""
    for name, at in REQS.items():
        if name == "num_requests":
            continue
        off = {name: at + (2 if name == "block_ids" else 4)}
        for code in (attend(reqs=off), attend(reqs=off, mass=True), evict(reqs=off)):
            assert code == K.KVCS_EINVAL, name
    for mass in (False, True):
        assert attend(new_offsets=(1 << 21) + 4, mass=mass) == K.KVCS_EINVAL
    lib, arr, r, a = K.load_library(), K.cache_array([FakeCache()]), B.kvcs_requests(**REQS), attention()
    ev = B.kvcs_eviction((ctypes.c_void_p * 1)(1 << 20), 1 << 16, 0, 0, None, None, 1 << 17, 1 << 30)
    head = (arr, 16, ctypes.byref(r), 10)
    for status, code in (((1 << 26) + 2, K.KVCS_EINVAL), (1 << 26, K.KVCS_ECUDA)):
        assert lib.kvcs_paged_attention(*head, ctypes.byref(a), status, None) == code
        assert lib.kvcs_attention_mass(*head, ctypes.byref(a), 1 << 25, status, None) == code
        assert lib.kvcs_evict(arr, 1, *head[1:], ctypes.byref(ev), status, None) == code


def test_evictions_of_very_long_rows_are_refused_before_any_work():
    """The move takes more CTAs a row where a head's row is past 32 KiB; that
    many have to fit a grid too, which was only seen between the launches."""
    wide = FakeCache(num_heads=1, head_bytes=1 << 20)      # 256 column groups, in 2 halves
    def code(requests):
        return evict([wide], reqs=dict(num_requests=requests), block_sums=1 << 26,
                     workspace_bytes=1 << 62)
    def size(requests):
        n = ctypes.c_int64()
        return K.load_library().kvcs_eviction_workspace(K.cache_array([wide]), 1, 16, requests, 10,
                                                        ctypes.byref(n))
    assert code(1 << 22) == size(1 << 22) == K.KVCS_EUNSUPPORTED
    assert code((1 << 22) - 1) == K.KVCS_ECUDA and size((1 << 22) - 1) == K.KVCS_OK
