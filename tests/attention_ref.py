"""Plain 64-bit forms of the paged-cache operators, for the tests.

Inputs are built token by token on the host (`Batch`): logical K and V per
request, placed in a pool of any layout by byte offsets computed here.  The
references read the logical values, never the pool.
"""

from __future__ import annotations

import math
from dataclasses import dataclass, field

import numpy as np
import torch

from paged_kv_cache_kvcs_gb300 import workloads as W

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # of the output types


def token_bytes(layout, halves, nb, bs, H, hb, half_stride=0, block_stride=0, kbs=0):
    """Byte offset of every (half, block, slot, head, byte) of a pool."""
    page = bs * H * hb
    hs = half_stride or nb * page
    bst = block_stride or page
    half = torch.arange(halves).view(-1, 1, 1, 1, 1) * hs
    blk = torch.arange(nb).view(1, -1, 1, 1, 1) * bst
    s = torch.arange(bs).view(1, 1, -1, 1, 1)
    h = torch.arange(H).view(1, 1, 1, -1, 1)
    b = torch.arange(hb).view(1, 1, 1, 1, -1)
    if layout in (W.LAYOUT_NHD, W.LAYOUT_LATENT):
        inner = (s * H + h) * hb + b
    elif layout == W.LAYOUT_HND:
        k = kbs or bs
        inner = (s // k) * (H * k * hb) + (h * k + s % k) * hb + b
    else:   # x-split
        inner = ((h * (hb // 16) + b // 16) * bs + s) * 16 + b % 16
    return half + blk + inner


@dataclass
class Batch:
    """Requests over one cache, with logical K/V on the host."""
    lengths: list
    new: list
    first: list
    kv: list = field(default_factory=list)      # per request [halves, T, H, D], the stored type

    def __post_init__(self):
        pass


def fill(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


class Case:
    """One cache, its pool on `device`, request tables, and queries."""

    def __init__(self, *, kv="bf16", q_dtype=None, layout=W.LAYOUT_NHD, heads=2, group=4, dim=64,
                 bs=16, lengths=(37,), new=(1,), first=None, kbs=0, interleaved=False, offset=0,
                 pad=0, seed=0, layer=0, spare=3, tail=float("nan"), scale=1.0, halves=2,
                 device="cuda", extra=0):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.layout, self.heads, self.group, self.dim, self.bs = \
            TYPES[kv], layout, heads, group, dim, bs
        self.q_dtype = q_dtype or (torch.bfloat16 if kv == "fp8" else self.kv)
        self.es = 1 if kv == "fp8" else 2
        hb = dim * self.es
        self.lengths, self.new = list(lengths), list(new)
        R = len(self.lengths)
        self.first = list(first) if first is not None else [0] * R
        counts = [max(0, -(-n // bs) - f) + extra for n, f in zip(self.lengths, self.first)]
        offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
        total = offsets[-1]
        nb = total + spare
        ids = torch.randperm(nb, generator=gen)[:total].to(torch.int32)
        # the whole pool starts as what masked places may hold
        page = bs * heads * hb
        half_stride = block_stride = 0
        if interleaved:
            half_stride, block_stride = page, 2 * page + pad
        elif pad:
            block_stride = page + pad
            half_stride = nb * block_stride
        at = token_bytes(layout, halves, nb, bs, heads, hb, half_stride, block_stride, kbs)
        size = int(at.max()) + 1
        size = (size + 7) // 8 * 8
        junk = torch.full((size // self.es + 1,), tail, dtype=torch.float32).to(self.kv)
        raw = junk.view(torch.uint8)[:size].clone()
        self.values = []
        for r in range(R):
            T = max(0, min(self.lengths[r], (self.first[r] + counts[r]) * bs) - self.first[r] * bs)
            v = fill((halves, T, heads, dim), self.kv, gen, scale)
            t = torch.arange(T)
            blk = ids[offsets[r] + t // bs].long()
            for half in range(halves):
                raw[at[half, blk, t % bs]] = v[half].view(torch.uint8).view(T, heads, hb)
            self.values.append(v)
        buf = torch.zeros(size + 16, dtype=torch.uint8, device=device)
        skip = (offset - buf.data_ptr()) % 16 if offset else (-buf.data_ptr()) % 16
        self.pool = buf[skip:skip + size]
        self.pool.copy_(raw.to(device))
        self.offsets_map = at
        self.counts, self.offsets, self.total, self.nb, self.ids = counts, offsets, total, nb, ids
        self.cache = W.CacheSpec(self.pool, nb, layout, layer, 0, heads, hb,
                                 half_stride=half_stride, block_stride=block_stride,
                                 kernel_block_size=kbs)
        dev = lambda x, t: torch.tensor(x, dtype=t, device=device)  # noqa: E731
        self.table = [dev(offsets, torch.int64), dev(self.first, torch.int64),
                      dev(self.lengths, torch.int64), ids.to(device)]
        starts = np.concatenate([[0], np.cumsum(self.new)]).tolist()
        self.starts = starts
        self.new_offsets = dev(starts, torch.int64)
        self.q = fill((starts[-1], heads * group, dim), self.q_dtype, gen).to(device)
        self.device = device

    def put(self, r, half, token, values):
        """Overwrites one token's values (all heads), logically and in the pool."""
        v = values.to(self.kv).expand(self.heads, self.dim).contiguous()
        self.values[r][half, token] = v
        blk = int(self.ids[self.offsets[r] + token // self.bs])
        at = self.offsets_map[half, blk, token % self.bs].to(self.device)
        self.pool[at] = v.view(torch.uint8).view(self.heads, -1).to(self.device)


def visible(case, r, window, blocked=()):
    """[n, T] truth values: which of request r's tokens its new tokens see."""
    T, n = case.values[r].shape[1], case.new[r]
    base = case.first[r] * case.bs
    pos = case.lengths[r] - n + torch.arange(n)[:, None] - base
    t = torch.arange(T)[None, :]
    see = t <= pos
    if window:
        see &= t > pos - window
    for b in blocked:
        see &= (t // case.bs) != b
    return see


def scores(case, r, h, scale, k_scale, softcap):
    """Query head h of request r: scores [n, T] in 64 bits, and the sums of
    absolute products that their rounding errors are relative to."""
    lo = case.starts[r]
    q = case.q[lo:lo + case.new[r], h].cpu().double()
    k = case.values[r][0, :, h // case.group].double()
    k = torch.where(torch.isfinite(k), k, 0.0) if not torch.isfinite(k).all() else k
    s = q @ k.T * (scale * k_scale)
    size = q.abs() @ k.abs().T * abs(scale * k_scale)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    return s, size


def score_error(dim, size, softcap=0.0):
    """Bound on a score's error: dim products summed in 32 bits by the tensor
    cores, which may truncate at two bits below the largest term (2^-22 of it
    per step of 16, taken at the sum of magnitudes), a scaling, and for capped
    scores tanh's 2^-21 of the cap."""
    return (dim / 16 + 4) * 2.0 ** -22 * size + 2.0 ** -21 * softcap


def attention(case, *, scale=None, k_scale=1.0, v_scale=1.0, softcap=0.0, window=0, blocked=None):
    """(out, lse, bound on out, bound on lse) in 64 bits, [total_new, q_heads, ...]."""
    scale = case.dim ** -0.5 if scale is None else scale
    n_all, Hq = case.starts[-1], case.heads * case.group
    out = torch.zeros((n_all, Hq, case.dim), dtype=torch.float64)
    lse = torch.full((n_all, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = HALF_STEP[case.q_dtype]
    for r in range(len(case.lengths)):
        n = case.new[r]
        if n == 0:
            continue
        see = visible(case, r, window, (blocked or {}).get(r, ()))
        lo = case.starts[r]
        T = see.shape[1]
        for h in range(Hq):
            if T == 0:
                continue
            s, size = scores(case, r, h, scale, k_scale, softcap)
            s = torch.where(see, s, -math.inf)
            z = torch.logsumexp(s, 1)
            some = see.any(1)
            w = torch.where(some[:, None], torch.exp(s - z[:, None]), 0.0)
            v = case.values[r][1, :, h // case.group].double()
            # a row's value comes from the tokens it sees alone
            fine = torch.where(torch.isfinite(v), v, 0.0)
            o = w @ fine * v_scale
            if not torch.isfinite(v).all():
                for i in range(n):
                    o[i] = (w[i, see[i], None] * v[see[i]]).sum(0) * v_scale
            ds = torch.where(see, score_error(case.dim, size, softcap), 0.0).amax(1)
            # each weight: its score's error, 2^-22 for 2^x, one rounding to
            # 16 bits; sums in 32 bits over T terms; then the output's rounding
            mag = w @ fine.abs() * abs(v_scale)
            per = (2 * ds + 2.0 ** -21 + T * 2.0 ** -23 + u)[:, None]
            out[lo:lo + n, h] = o
            tol[lo:lo + n, h] = o.abs().nan_to_num(0, 0, 0) * u + mag * per + 1e-7 * u
            lse[lo:lo + n, h] = torch.where(some, z, -math.inf)
            tol_lse[lo:lo + n, h] = ds + 2.0 ** -21 + T * 2.0 ** -23 + \
                torch.where(some, z, 0.0).abs() * 2.0 ** -22
    return out, lse, tol, tol_lse


def mass(case, lse, before, *, scale=None, k_scale=1.0, softcap=0.0, window=0, observe=0,
         blocked=None):
    """(mass, bound) in 64 bits, [num_blocks, heads, block_size]."""
    scale = case.dim ** -0.5 if scale is None else scale
    out = before.cpu().double().clone()
    tol = out.abs() * 2.0 ** -24
    for r in range(len(case.lengths)):
        n = case.new[r]
        see = visible(case, r, window, (blocked or {}).get(r, ()))
        T = see.shape[1]
        if n == 0 or T == 0:
            continue
        if observe:
            see[:max(0, n - observe)] = False
        lo = case.starts[r]
        t = torch.arange(T)
        ids = case.ids[case.offsets[r] + t // case.bs].long()
        for h in range(case.heads * case.group):
            s, size = scores(case, r, h, scale, k_scale, softcap)
            z = lse[lo:lo + n, h].cpu().double()
            w = torch.where(see, torch.exp(s - z[:, None]), 0.0)
            err = score_error(case.dim, size, softcap) + z.abs().nan_to_num(0, 0, 0)[:, None] * \
                2.0 ** -22 + 2.0 ** -21 + n * case.group * 2.0 ** -24
            kh = h // case.group
            out[ids, kh, t % case.bs] += w.sum(0)
            tol[ids, kh, t % case.bs] += (w * err).sum(0) + w.sum(0) * 2.0 ** -23
    return out, tol


def close(got, want, tol):
    """Within the bound, and equal where the value is not finite."""
    got = got.detach().cpu().double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    off = (got - want).abs()[fine]
    bad = off > tol[fine]
    assert not bad.any(), (float(off.max()), float((off / tol[fine].clamp(min=1e-300)).max()),
                           int(bad.sum()))


def kept_tokens(score, N, B, sinks, recent):
    """Tokens one row keeps, by the definition (score: N floats)."""
    a = min(sinks, B)
    w = min(recent, B - a)
    order = sorted(range(a, N - w), key=lambda j: (
        -math.inf if math.isnan(score[j]) else -score[j] if not math.isinf(score[j])
        else (-1e39 if score[j] > 0 else 1e39), j))
    return list(range(a)) + sorted(order[:B - a - w]) + list(range(N - w, N))
