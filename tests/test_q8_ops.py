"""KV pools held in 8 bits: rows quantised and read back, decode and extend attention over codes, against plain
64-bit definitions.

The pages have no 8-bit cache; these stand beside kv_pool_write and the attention entry points.
"""
import ctypes
import math
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

from prefix_cached_kv_radix_gb300 import api

api.load()
gpu = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
INT8, E4M3 = api.RX_Q8_INT8, api.RX_Q8_E4M3
TYPE = {INT8: torch.int8, E4M3: torch.float8_e4m3fn}
TOP = {INT8: 127.0, E4M3: 448.0}
A = 0x1000        # stands for an aligned device address in calls that are refused before any launch


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def desc_of(dt, hq, hkv, d, slots=64, scale=None):
    return api.make_desc(api.RX_F32 if dt == F else api.RX_BF16, hq, hkv, d, slots, 1 / math.sqrt(d) if scale is None else scale)


def i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def i64(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int64, device=dev)


def indptr(lens, dev, start=0):
    return i64(np.concatenate([[0], np.cumsum(lens)]) + start, dev)


# ============================================================================ definitions, in 64 bits
def scales_of(x, fmt):
    """The write's scales of rows x [..., d]."""
    a = x.double().abs().amax(-1)
    if fmt == INT8:
        s = (a / 127.0).float().double().clamp(min=2.0 ** -126)
    else:
        s = torch.full_like(a, 2.0 ** -126)
        for e in range(-126, 121):                # the first power of two that is large enough
            s = torch.where(448.0 * s < a, torch.full_like(a, 2.0 ** (e + 1)), s)
    return torch.where(a.isfinite(), s, torch.full_like(a, math.nan))


def codes_of(x, s, fmt):
    y = x.double() / s.double()[..., None]
    if fmt == INT8:
        return torch.where(y.isnan(), torch.zeros_like(y), y).clamp(-127, 127).round()
    y = torch.where(s.isnan()[..., None], torch.zeros_like(y), y).clamp(-448, 448)
    power = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).long() - 3
    step = ((power + 1023) << 52).view(torch.float64)        # 2 ** power, exactly
    return (y / step).round() * step


def as_codes(values, fmt):
    return values.to(torch.int8) if fmt == INT8 else values.float().to(torch.float8_e4m3fn)


def bytes_of(t):
    return t.view(torch.uint8)


class Cache:
    """Pools of codes with every slot filled, made here and not by the write."""

    def __init__(self, dev, fmt, slots, hkv, d, block=1, seed=0, size=1.0):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.q8, self.fmt, self.block = api.q8_desc(fmt, block, block > 1), fmt, block
        x = torch.randn(2, slots, hkv, d, generator=g, device=dev) * size
        x *= torch.randn(2, slots, 1, 1, generator=g, device=dev).exp()
        blocks = -(-slots // block)
        if block == 1:
            self.scales = scales_of(x, fmt).permute(1, 2, 0).float().contiguous()
        else:
            self.scales = (1 + torch.rand(blocks, hkv, 2, generator=g, device=dev)) * (4 * size / TOP[fmt])
        per_slot = self.scales[torch.arange(slots, device=dev) // block]
        self.k, self.v = (as_codes(codes_of(x[j], per_slot[:, :, j], fmt), fmt) for j in range(2))

    def values(self, slots):
        s = self.scales[slots.long() // self.block].double()
        k, v = (bytes_of(p)[slots.long()].view(p.dtype).double() for p in (self.k, self.v))
        return k * s[..., :1], v * s[..., 1:]


def attend(q, k, v, scale, first):
    """Rows q [n, hq, d], row i over keys 0 .. first + i of k, v [len, hkv, d], in 64 bits.  Returns the rows, their
    log-sum-exp, sum_j p_j |v_j|, a bound of the 32-bit sums' error of a score, the largest p_j |v_ji| of a row times its
    keys, and the largest |v_ji| times its keys."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    q = q.double().view(n, hkv, hq // hkv, d)
    seen = torch.arange(k.shape[0], device=q.device)[None, :] <= first + torch.arange(n, device=q.device)[:, None]
    if k.shape[0] == 0 or n == 0:
        z = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
        return z, torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device), z, z[..., 0], z[..., 0], z[..., 0]
    s = torch.einsum("nhgd,khd->nhgk", q, k) * scale
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    mag = torch.einsum("nhgd,khd->nhgk", q.abs(), k.abs()) * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.clamp(min=-1e300)[..., None])
    o, a = torch.einsum("nhgk,khd->nhgd", p, v), torch.einsum("nhgk,khd->nhgd", p, v.abs())
    # d products summed in 32 bits with a few roundings of the scaled score after them
    err = (d + 8) * 2.0 ** -23 * mag.masked_fill(~seen[:, None, None, :], 0).amax(-1)
    top = v.abs().amax(-1).t()[None, :, None, :]
    weighed = (p * top).masked_fill(~seen[:, None, None, :], 0).amax(-1) * k.shape[0]
    largest = top.expand(p.shape).masked_fill(~seen[:, None, None, :], 0).amax(-1) * k.shape[0]
    return tuple(t.reshape(n, hq, *t.shape[3:]) for t in (o, lse, a, err, weighed, largest))


def agree(out, lse, want, dt):
    """out is off by its own rounding, the rounding of the weighted probabilities (bf16 rows: 2^-8 of each at most) and
    the scores' 32-bit errors, which change a probability by that much of itself, twice (its own and the sum's).  A weighted
    probability p_j vs_j held in 16 bits with 5 of exponent next to the row's largest has steps of 2^-24 of that at least,
    half of one times a code at most (two such parts, the second 2^-11 as large: 2^-35); the largest code of a
    row here is at least half the largest there is.  And p_j below 2^-126 is zero in 32 bits."""
    o, z, a, err, weighed, largest = want
    half, part, step = (2.0 ** -8, 2.0 ** -8, 2.0 ** -24) if dt == BF else (2.0 ** -24, 2.0 ** -20, 2.0 ** -35)
    tol = half * o.abs() + (part + 2 * err[..., None] + 2.0 ** -19) * a * (1 + half)
    tol += (weighed * step + largest * 2.0 ** -126)[..., None] + 1e-30
    bad = (out.double() - o).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((out.double() - o).abs() / tol).max()))
    if lse is not None:
        empty = z.isinf()
        assert torch.equal(lse.double()[empty], z[empty])
        gap = (lse.double() - z).abs()[~empty]
        assert (gap <= err[~empty] + 2.0 ** -18 * (1 + z.abs()[~empty])).all(), float(gap.max())


# ============================================================================ refusals (CPU)
def refused(fn, *args):
    rc = getattr(api.load(), fn)(*args)
    assert rc == api.RX_EINVAL, (fn, rc)
    assert fn in api.load().rx_last_error().decode()


BAD_CACHES = (api.rx_q8_desc(2, 1, 0), api.rx_q8_desc(-1, 1, 0), api.rx_q8_desc(0, 0, 1), api.rx_q8_desc(0, 3, 1),
              api.rx_q8_desc(0, 2, 0), api.rx_q8_desc(0, -4, 1), api.rx_q8_desc(0, 1, 2), api.rx_q8_desc(0, -(1 << 31), 1))
BAD_SHAPES = (desc_of(BF, 4, 0, 64), desc_of(BF, 4, 2, 96), desc_of(BF, 4, 2, 64, slots=0), desc_of(BF, 4, 2, 64, slots=1 << 31),
              api.make_desc(7, 4, 2, 64, 4, 1.0))
BAD_HEADS = (desc_of(BF, 4, 3, 64), desc_of(BF, 0, 2, 64), desc_of(BF, -4, 2, 64))


def test_write_q8_refuses():
    def call(desc=None, q8=None, batch=1, ind=A, pi=A, ns=A, k=A, ks=128, v=A, vs=128, kp=A, vp=A, sc=A, r2t=A, stride=8, total=4):
        refused("kv_pool_write_q8", ctypes.byref(desc or desc_of(BF, 4, 2, 64)), ctypes.byref(q8 or api.q8_desc(INT8)), batch, A, pi,
                ns, ind, k, ks, v, vs, kp, vp, sc, r2t, stride, total, None, None)
    for bad in BAD_CACHES:
        call(q8=bad)
    for bad in BAD_SHAPES:
        call(desc=bad)
    for kw in (dict(batch=-1), dict(total=-1), dict(total=1 << 31), dict(stride=-1), dict(ind=None), dict(pi=None), dict(ns=None),
               dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(sc=None), dict(k=A + 8), dict(v=A + 2), dict(ks=120),
               dict(vs=130), dict(kp=A + 8), dict(vp=A + 1), dict(sc=A + 4)):
        call(**kw)


def test_read_q8_refuses():
    def call(desc=None, q8=None, n=4, sl=A, kp=A, vp=A, sc=A, k=A, ks=128, v=A, vs=128):
        refused("kv_pool_read_q8", ctypes.byref(desc or desc_of(BF, 4, 2, 64)), ctypes.byref(q8 or api.q8_desc(INT8)), n, sl, kp, vp, sc,
                k, ks, v, vs, None, None)
    for bad in BAD_CACHES:
        call(q8=bad)
    for bad in BAD_SHAPES:
        call(desc=bad)
    for kw in (dict(n=-1), dict(n=1 << 31), dict(sl=None), dict(kp=None), dict(vp=None), dict(sc=None), dict(k=A + 8), dict(v=A + 2),
               dict(ks=120), dict(vs=130), dict(kp=A + 8), dict(sc=A + 4)):
        call(**kw)


def test_decode_q8_refuses():
    def call(desc=None, q8=None, batch=1, q=A, r2t=A, stride=8, lens=A, kp=A, vp=A, sc=A, out=A, longest=8, ws=A, nbytes=1 << 40):
        refused("decode_attention_q8", ctypes.byref(desc or desc_of(BF, 4, 2, 64)), ctypes.byref(q8 or api.q8_desc(INT8)), batch, q, r2t,
                stride, lens, None, kp, vp, sc, out, None, longest, ws, nbytes, None, None)
    for bad in BAD_CACHES:
        call(q8=bad)
    for bad in BAD_SHAPES + BAD_HEADS:
        call(desc=bad)
    for kw in (dict(batch=-1), dict(stride=-1), dict(longest=-1), dict(q=None), dict(r2t=None), dict(lens=None), dict(kp=None),
               dict(vp=None), dict(sc=None), dict(out=None), dict(q=A + 8), dict(out=A + 4), dict(kp=A + 8), dict(sc=A + 4)):
        call(**kw)


def test_extend_q8_refuses():
    def call(desc=None, q8=None, batch=1, q=A, ind=A, pre=A, r2t=A, stride=8, kp=A, vp=A, sc=A, out=A, rows=4, longest=8, ws=A,
             nbytes=1 << 40):
        refused("prefix_extend_attention_q8", ctypes.byref(desc or desc_of(BF, 4, 2, 64)), ctypes.byref(q8 or api.q8_desc(INT8)), batch,
                q, ind, pre, r2t, stride, kp, vp, sc, out, None, rows, longest, ws, nbytes, None, None)
    for bad in BAD_CACHES:
        call(q8=bad)
    for bad in BAD_SHAPES + BAD_HEADS:
        call(desc=bad)
    for kw in (dict(batch=-1), dict(stride=-1), dict(longest=-1), dict(rows=-1), dict(q=None), dict(ind=None), dict(pre=None),
               dict(r2t=None), dict(kp=None), dict(vp=None), dict(sc=None), dict(out=None), dict(q=A + 8), dict(out=A + 4),
               dict(vp=A + 8), dict(sc=A + 4)):
        call(**kw)


def test_attention_q8_scales_and_sizes_refused():
    """Scales that are not finite, or not once in base 2; more rows than a launch has blocks; workspaces of shapes that no call takes."""
    c = ctypes.byref(api.q8_desc(INT8))
    for scale in (math.inf, -math.inf, math.nan, 3e38):
        d = desc_of(BF, 4, 2, 64)
        d.scale = scale
        refused("decode_attention_q8", ctypes.byref(d), c, 1, A, A, 8, A, None, A, A, A, A, None, 8, A, 1 << 40, None, None)
        refused("prefix_extend_attention_q8", ctypes.byref(d), c, 1, A, A, A, A, 8, A, A, A, A, None, 4, 8, A, 1 << 40, None, None)
    most = 2 ** 31 - 1
    for hq, hkv in ((4096, 4096), (4096, 1)):
        refused("prefix_extend_attention_q8", ctypes.byref(desc_of(F, hq, hkv, 64)), c, most, A, A, A, A, most, A, A, A, A, None, most,
                most, A, 1 << 60, None, None)
    for d in (desc_of(BF, 4, 2, 256), desc_of(F, 4, 2, 0, scale=1.0), desc_of(BF, 4, 3, 64), desc_of(BF, 4, 0, 64)):
        assert api.decode_q8_workspace_bytes(d, 4, 100) == 0 and api.extend_q8_workspace_bytes(d, 4, 5, 100) == 0


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d", [(12, 12, 64), (32, 8, 128), (64, 1, 128), (16, 4, 64)])
def test_attention_q8_workspaces_grow(dt, hq, hkv, d):
    """A workspace made for the greatest call is enough for every smaller one."""
    desc = desc_of(dt, hq, hkv, d, 10 ** 6)
    decode_most = api.decode_q8_workspace_bytes(desc, 300, 9000)
    extend_most = api.extend_q8_workspace_bytes(desc, 300, 200, 9000)
    for batch in (1, 4, 16, 64, 300):
        for longest in (1, 300, 3000, 9000):
            assert api.decode_q8_workspace_bytes(desc, batch, longest) <= decode_most
            for rows in (1, 2, 9, 16, 17, 200):
                assert api.extend_q8_workspace_bytes(desc, batch, rows, longest) <= extend_most


def test_nothing_to_do_is_no_error():
    """No requests, no rows, no slots: fine, without a device."""
    d, c = desc_of(BF, 4, 2, 64), api.q8_desc(E4M3)
    lib, by = api.load(), ctypes.byref
    assert lib.kv_pool_write_q8(by(d), by(c), 0, *[None] * 5, 0, None, 0, None, None, None, None, 0, 0, None, None) == api.RX_OK
    assert lib.kv_pool_read_q8(by(d), by(c), 0, None, None, None, None, None, 0, None, 0, None, None) == api.RX_OK
    assert lib.decode_attention_q8(by(d), by(c), 0, None, None, 0, None, None, None, None, None, None, None, 0, None, 0, None,
                                   None) == api.RX_OK
    assert lib.prefix_extend_attention_q8(by(d), by(c), 1, None, None, None, None, 0, None, None, None, None, None, 0, 0, None, 0,
                                          None, None) == api.RX_OK


# ============================================================================ writing
def special_rows(x, fmt):
    """Rows whose scales and codes are on a border: zeros, the smallest and largest numbers, halves between codes,
    largest values that a power of two times 448 just holds or just does not."""
    n = x.shape[0]
    big = 3e38
    rows = [torch.zeros_like(x[0, 0]), torch.full_like(x[0, 0], big), torch.full_like(x[0, 0], -big)]
    d = x.shape[-1]
    ramp = torch.arange(d, device=x.device, dtype=torch.float32)
    rows.append((ramp - d // 2 + 0.5).clamp(-126.5, 126.5).index_fill(0, i64([0], x.device), 127.0).to(x.dtype))  # scale 1: halves
    rows.append((ramp * 2.0 ** -9).index_fill(0, i64([1], x.device), 448.0).to(x.dtype))      # e4m3's smallest steps
    rows.append((ramp * 2.0 ** -10).index_fill(0, i64([1], x.device), 448.0).to(x.dtype))     # and halves of them
    for top in (448.0 * 2 ** 5, 450.0, 1.75 * 2 ** -20, 1.7578125 * 2 ** -20, 1e-37, 2.0 ** -126, 2.0 ** -133):
        rows.append((torch.randn(d, device=x.device).clamp(-1, 1) * top).index_fill(0, i64([3], x.device), top).to(x.dtype))
    for j, r in enumerate(rows[:n]):
        x[j, 0] = r
    return x


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hkv,d,block,strided", [(1, 64, 1, False), (3, 128, 1, True), (12, 64, 1, True), (8, 128, 1, False),
                                                 (2, 64, 4, True), (5, 128, 64, False), (2, 128, 1 << 30, False)])
def test_write_q8(dev, fmt, dt, hkv, d, block, strided):
    torch.manual_seed(hkv * d + block)
    lens, pre = [1, 0, 37, 5, 200], [0, 3, 17, 0, 900]
    n, slots, lead = sum(lens), 2600, 2
    total = n + lead + 3                         # two rows before the batch, three behind it
    wide = special_rows(torch.randn(total, 3 * hkv if strided else hkv, d, device=dev).to(dt), fmt)
    x = special_rows(torch.randn(total, hkv, d, device=dev).to(dt), fmt)
    k, v = (wide[:, hkv:2 * hkv], wide[:, :hkv]) if strided else (x, wide)
    ids = torch.randperm(slots, device=dev).to(torch.int32)
    new, old = ids[:total].contiguous(), ids[total:total + sum(pre)].contiguous()
    c = api.q8_desc(fmt, block, block > 1)
    kp, vp = (torch.full((slots, hkv, d), 0x55, dtype=torch.uint8, device=dev) for _ in range(2))
    blocks = -(-slots // block)
    if block > 1:
        scales = (0.25 + torch.rand(blocks, hkv, 2, device=dev)) * (3.0 / TOP[fmt])
        scales[0, 0] = 1.0                       # halves between codes
    else:
        scales = torch.full((blocks, hkv, 2), 7.0, device=dev)
    was = scales.clone()
    r2t = torch.full((len(lens), 1104), 99, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    desc = desc_of(dt, hkv, hkv, d, slots)
    api.kv_pool_write_q8(desc, c, len(lens), old, indptr(pre, dev), new, indptr(lens, dev, lead), k, v, kp.view(TYPE[fmt]),
                         vp.view(TYPE[fmt]), scales, r2t, total, st)
    assert int(st) == 0
    rows = slice(lead, lead + n)
    at = new[rows].long()
    for j, (name, y, pool) in enumerate((("k", k, kp), ("v", v, vp))):
        s = was[at // block, :, j].double() if block > 1 else scales_of(y[rows], fmt)
        if block == 1:
            assert torch.equal(scales[at, :, j].double().nan_to_num(-1), s.nan_to_num(-1)), name
        want = bytes_of(as_codes(codes_of(y[rows], s, fmt), fmt))
        got = pool[at]
        zero = (want & 0x7f) == 0                # a code of -0 is a zero as well
        assert torch.equal(torch.where(zero, want & 0x7f, want), torch.where(zero, got & 0x7f, got)), name
        rest = torch.ones(slots, dtype=torch.bool, device=dev)
        rest[at] = False
        assert (pool[rest] == 0x55).all()
    if block > 1:
        assert torch.equal(scales, was)
    else:
        assert (scales[rest] == 7.0).all()
    qo, po = np.concatenate([[0], np.cumsum(lens)]) + lead, np.concatenate([[0], np.cumsum(pre)])
    for b in range(len(lens)):
        want = torch.cat([old[po[b]:po[b + 1]], new[qo[b]:qo[b + 1]]])
        assert torch.equal(r2t[b, :len(want)], want) and (r2t[b, len(want):] == -1).all()


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
def test_write_q8_not_finite(dev, fmt, dt):
    """An infinity or a NaN: that token, head and pool reads as NaN; its neighbours are what they are."""
    x = torch.randn(4, 3, 64, device=dev).to(dt)
    y = x.clone()
    y[1, 2, 63], y[2, 0, 5], y[3, 1, 0] = math.inf, math.nan, -math.inf
    c, desc = api.q8_desc(fmt), desc_of(dt, 3, 3, 64, 8)
    pools = [torch.zeros(8, 3, 64, dtype=torch.int8, device=dev).view(TYPE[fmt]) for _ in range(2)]
    scales, st = torch.zeros(8, 3, 2, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    new = i32([6, 1, 3, 0], dev)
    api.kv_pool_write_q8(desc, c, 1, None, i64([0, 0], dev), new, i64([0, 4], dev), y, x, *pools, scales, None, 4, st)
    out = [torch.empty_like(x) for _ in range(2)]
    api.kv_pool_read_q8(desc, c, new, *pools, scales, *out, st)
    assert int(st) == 0
    bad = torch.zeros(4, 3, dtype=torch.bool, device=dev)
    bad[1, 2] = bad[2, 0] = bad[3, 1] = True
    assert out[0][bad].isnan().all() and out[0][~bad].isfinite().all() and out[1].isfinite().all()
    assert (bytes_of(pools[0])[new.long()][bad] == 0).all()
    if fmt == E4M3:                              # a step is at most an eighth of the value, or 2^-9 of the scale
        gap = (out[1].double() - x.double()).abs()
        assert (gap <= x.double().abs() / 16 + scales[new.long(), :, 1:].double() * 2.0 ** -10).all()


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_write_q8_fixed_takes_any_value(dev, fmt):
    """Given scales: values past the largest code are cut to it; a NaN is a zero."""
    x = torch.tensor([math.inf, -math.inf, math.nan, 1e38, -1e38, 1.0, -1.0, 0.0] * 8, device=dev).view(1, 1, 64)
    c, desc = api.q8_desc(fmt, 2, True), desc_of(F, 1, 1, 64, 2)
    pools = [torch.zeros(2, 1, 64, dtype=torch.int8, device=dev).view(TYPE[fmt]) for _ in range(2)]
    scales, st = torch.full((1, 1, 2), 0.5, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    api.kv_pool_write_q8(desc, c, 1, None, None, i32([1], dev), i64([0, 1], dev), x, x, *pools, scales, None, 1, st)
    t = TOP[fmt]
    want = torch.tensor([t, -t, 0.0, t, -t, 2.0, -2.0, 0.0] * 8, device=dev)
    for p in pools:
        assert torch.equal(p[1, 0].float(), want)
        assert (bytes_of(p)[0] == 0).all()


@gpu
def test_write_q8_bad_slots_and_lengths(dev):
    """A bad slot leaves its row out and the others in; a batch longer than its rows is reported."""
    x = torch.randn(4, 2, 64, device=dev)
    c, desc = api.q8_desc(INT8), desc_of(F, 2, 2, 64, 8)
    for new, qo, code, written in (([1, 8, 2, -1], [0, 4], api.RX_DEV_BAD_SLOT, [1, 2]),
                                   ([1, 4, 2, 3], [0, 9], api.RX_DEV_BAD_LENGTH, [1, 4, 2, 3]),
                                   ([1, 4, 2, 3], [-2, 2], api.RX_DEV_BAD_LENGTH, [1, 4]),
                                   ([1, 4, 2, 3], [3, 1], api.RX_DEV_BAD_LENGTH, [])):
        pools = [torch.zeros(8, 2, 64, dtype=torch.int8, device=dev) for _ in range(2)]
        scales, st = torch.zeros(8, 2, 2, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
        api.kv_pool_write_q8(desc, c, 1, None, i64([0, 0], dev), i32(new, dev), i64(qo, dev), x, x, *pools, scales, None, 4, st)
        assert int(st) == code
        touched = (scales != 0).flatten(1).any(1).nonzero().flatten().tolist()
        assert sorted(touched) == sorted(written)


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt,hkv,d,block", [(BF, 8, 128, 1), (F, 8, 128, 16), (BF, 3, 64, 1), (F, 5, 64, 1)])
def test_write_q8_many_rows(dev, fmt, dt, hkv, d, block):
    """Calls of a size where several rows are in flight at once, with odd numbers of rows and heads."""
    n = 20011 if d == 128 else 70001 // hkv * 2
    x = torch.randn(n, 2 * hkv, d, device=dev).to(dt)
    k, v = x[:, :hkv], x[:, hkv:]
    slots = n + 5
    new = torch.randperm(slots, device=dev)[:n].to(torch.int32)
    c = api.q8_desc(fmt, block, block > 1)
    pools = [torch.zeros(slots, hkv, d, dtype=torch.int8, device=dev).view(TYPE[fmt]) for _ in range(2)]
    scales = (1 + torch.rand(-(-slots // block), hkv, 2, device=dev)) * (3.0 / TOP[fmt]) if block > 1 else torch.zeros(slots, hkv, 2, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    desc = desc_of(dt, hkv, hkv, d, slots)
    api.kv_pool_write_q8(desc, c, 1, None, None, new, i64([1, n - 1], dev), k, v, *pools, scales, None, n, st)
    out = [torch.full((n, hkv, d), 7.0, dtype=dt, device=dev) for _ in range(2)]
    api.kv_pool_read_q8(desc, c, new, *pools, scales, *out, st)
    assert int(st) == 0
    at = new[1:n - 1].long()
    for j, y in enumerate((k, v)):
        s = scales[at // block, :, j].double()
        if block == 1:
            assert torch.equal(s, scales_of(y[1:n - 1], fmt))
        want = codes_of(y[1:n - 1], s, fmt)
        got = bytes_of(pools[j])[at].view(TYPE[fmt]).double()
        assert torch.equal(got, want)
        assert torch.equal(out[j][1:n - 1], (got.float() * s.float()[..., None]).to(dt))
        assert (bytes_of(pools[j])[new[[0, n - 1]].long()] == 0).all()


# ============================================================================ reading
@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hkv,d,block,n", [(1, 64, 1, 1), (3, 128, 1, 77), (12, 64, 16, 700), (8, 128, 1, 1025), (2, 64, 1 << 30, 9)])
def test_read_q8(dev, fmt, dt, hkv, d, block, n):
    slots = n + 13
    cache = Cache(dev, fmt, slots, hkv, d, block, seed=n)
    if fmt == INT8:
        cache.k[0, 0, 0] = -128                  # a code that the write does not make
    else:
        bytes_of(cache.k)[0, 0, 0] = 0x7f        # e4m3's NaN
    at = torch.randint(0, slots, (n,), device=dev, dtype=torch.int32)
    at[0] = 0
    wide = torch.full((n, 2 * hkv + 1, d), 3.0, dtype=dt, device=dev)
    k, v = wide[:, :hkv], wide[:, hkv + 1:]
    desc, st = desc_of(dt, hkv, hkv, d, slots), torch.zeros(1, dtype=torch.int32, device=dev)
    api.kv_pool_read_q8(desc, cache.q8, at, cache.k, cache.v, cache.scales, k, v, st)
    assert int(st) == 0
    s = cache.scales[at.long() // block]
    for j, (got, pool) in enumerate(((k, cache.k), (v, cache.v))):
        want = (bytes_of(pool)[at.long()].view(pool.dtype).float() * s[:, :, j:j + 1]).to(dt)
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert (wide[:, hkv] == 3.0).all()
    only = torch.empty(n, hkv, d, dtype=dt, device=dev)
    api.kv_pool_read_q8(desc, cache.q8, at, None, cache.v, cache.scales, None, only, st)
    assert torch.equal(only, v)
    at[n // 2] = slots
    only.fill_(5.0)
    api.kv_pool_read_q8(desc, cache.q8, at, cache.k, None, cache.scales, only, None, st)
    assert int(st) == api.RX_DEV_BAD_SLOT
    keep = torch.arange(n, device=dev) != n // 2
    assert (only[~keep] == 5.0).all() and torch.equal(only[keep].nan_to_num(7.0), k[keep].nan_to_num(7.0))


# ============================================================================ decode
def groups_of(dev, indptr_, members, lens, size, longest):
    """The struct holds addresses: the arrays stay with it."""
    arrays = i32(indptr_, dev), i32(members, dev), i32(lens, dev)
    g = api.shared_groups_struct(len(indptr_) - 1, size, *arrays, longest)
    g._keep = arrays
    return g


def table_of(lens, stride, slots, dev, seed=0):
    """Slot tables of requests that share nothing; unused entries -1.  Returns it and the slots in use."""
    ids = torch.randperm(slots, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    t, at = torch.full((max(len(lens), 1), stride), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        t[b, :n] = ids[at:at + n]
        at += n
    return t.to(dev), ids[:at].long().to(dev)


def decode(dev, cache, dt, hq, hkv, d, lens, r2t, groups=None, scale=None, q=None, longest=None, ws=None):
    b = len(lens)
    desc = desc_of(dt, hq, hkv, d, cache.k.shape[0], scale)
    if q is None:
        q = torch.randn(b, hq, d, generator=torch.Generator(device=dev).manual_seed(b + hq), device=dev).to(dt)
    out, lse = torch.full_like(q, 9.0), torch.full((b, hq), 9.0, device=dev)
    longest = max(max(lens), 1) if longest is None else longest
    nbytes = api.decode_q8_workspace_bytes(desc, b, longest, groups)
    if ws is None and nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    api.decode_attention_q8(desc, cache.q8, b, q, r2t, i32(lens, dev), cache.k, cache.v, cache.scales, out, lse, longest, ws, st,
                            groups=groups)
    return q, out, lse, int(st)


def poison(cache, used):
    """Every slot that is not in use holds NaN: a scale of NaN (block 1)."""
    if cache.block == 1:
        rest = torch.ones(cache.k.shape[0], dtype=torch.bool, device=used.device)
        rest[used] = False
        cache.scales[rest] = math.nan


HEADS = [(4, 4, 64), (12, 12, 64), (8, 2, 128), (6, 2, 64), (16, 2, 128), (7, 1, 128), (12, 1, 64), (32, 2, 128)]


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_decode_q8(dev, fmt, dt, hq, hkv, d):
    lens = [1, 0, 2, 15, 16, 17, 63, 64, 65, 129, 300, 1, 777]
    slots = sum(lens) + 40
    r2t, used = table_of(lens, 784, slots, dev)
    cache = Cache(dev, fmt, slots, hkv, d, seed=hq)
    poison(cache, used)
    q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, lens, r2t)
    assert st == 0
    for b, n in enumerate(lens):
        k, v = cache.values(r2t[b, :n])
        agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), n - 1), dt)


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("lens,block", [([5000], 1), ([20011, 3], 64), ([1025, 1024, 1023, 2049], 16), ([70001], 1 << 30)])
def test_decode_q8_long(dev, fmt, dt, lens, block):
    hq, hkv, d = 8, 2, 128
    slots = sum(lens) + 5
    r2t, used = table_of(lens, (max(lens) + 7) // 8 * 8, slots, dev)
    cache = Cache(dev, fmt, slots, hkv, d, block, seed=1)
    poison(cache, used)
    q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, lens, r2t)
    assert st == 0
    for b, n in enumerate(lens):
        k, v = cache.values(r2t[b, :n])
        agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), n - 1), dt)


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
def test_decode_q8_scales_far_apart(dev, fmt, dt):
    """Value rows of very different sizes, zeros among them, keys that say much and nothing: the sums keep what
    is attended, whatever the sizes of the rest."""
    hq, hkv, d, n = 8, 2, 64, 200
    cache = Cache(dev, fmt, n, hkv, d, seed=3)
    r2t = torch.arange(n, dtype=torch.int32, device=dev)[None]
    cache.scales[:, :, 1] *= (torch.randn(n, hkv, device=dev) * 12).exp2()
    cache.scales[3, :, 1], cache.scales[5, :, 1] = 1e30, 2.0 ** -126
    bytes_of(cache.v)[7] = 0
    cache.scales[7, :, 1] = 2.0 ** -126
    cache.scales[9, :, 0], cache.scales[7, :, 0] = 0.0, 4.0
    for size in (0.1, 1.0, 30.0):
        q = (torch.randn(1, hq, d, device=dev) * size).to(dt)
        q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, [n], r2t, q=q)
        k, v = cache.values(r2t[0])
        agree(out, lse, attend(q, k, v, 1 / math.sqrt(d), n - 1), dt)
        far = cache.scales.clone()               # all but an unattended huge row
        cache.scales[3, :, 1] = 1.0
        q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, [n], r2t, q=q)
        k, v = cache.values(r2t[0])
        agree(out, lse, attend(q, k, v, 1 / math.sqrt(d), n - 1), dt)
        cache.scales.copy_(far)


@gpu
@pytest.mark.parametrize("dt", [BF, F])
def test_decode_q8_queries_far_apart(dev, dt):
    """Queries from far below to far above one in a batch, zeros among them."""
    hq, hkv, d = 4, 2, 128
    lens = [33] * 8
    r2t, _ = table_of(lens, 40, 300, dev)
    cache = Cache(dev, INT8, 300, hkv, d, seed=5)
    q = torch.randn(8, hq, d, device=dev)
    q *= torch.tensor([1e-38, 1e-20, 1e-6, 1.0, 100.0, 1e4, 0.0, 1.0], device=dev)[:, None, None]
    q[7, 0, 1:] = 0.0
    q[7, 1, ::2] *= 1e-5
    q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, lens, r2t, q=q.to(dt))
    assert st == 0
    for b in range(8):
        k, v = cache.values(r2t[b, :33])
        agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), 32), dt)


@gpu
@pytest.mark.parametrize("dt", [BF, F])
def test_decode_q8_bad_slots_and_lengths(dev, dt):
    """Keys at bad slots are left out; requests with bad lengths are left as they were."""
    hq, hkv, d = 8, 2, 64
    lens = [40, 3, 70, 20, 5, 9]
    r2t, _ = table_of(lens, 72, 200, dev)
    cache = Cache(dev, E4M3, 200, hkv, d, seed=2)
    r2t[0, 7], r2t[0, 39], r2t[1, :3] = -1, 200, -5
    q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, lens, r2t)
    assert st == api.RX_DEV_BAD_SLOT
    for b, n in enumerate(lens):
        ok = r2t[b, :n]
        ok = ok[(ok >= 0) & (ok < 200)]
        k, v = cache.values(ok)
        agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), len(ok) - 1), dt)
    for wrong, longest in ((-1, 70), (73, 100), (71, 70)):
        q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, [40, wrong, 5], r2t[[0, 1, 4]].contiguous(), longest=longest)
        assert st in (api.RX_DEV_BAD_LENGTH, api.RX_DEV_BAD_SLOT)
        assert (out[1] == 9.0).all() and (lse[1] == 9.0).all() and (out[2] != 9.0).any()


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
def test_decode_q8_groups(dev, fmt, dt):
    """Requests that share leading slots give what they give alone."""
    hq, hkv, d = 8, 2, 128
    lens = [300, 411, 301, 90, 640, 300, 17]
    slots = 3000
    r2t, _ = table_of(lens, 648, slots, dev)
    r2t[[1, 2, 5], :300] = r2t[0, :300].clone()
    r2t[4, :77] = r2t[3, :77].clone()
    cache = Cache(dev, fmt, slots, hkv, d, seed=4)
    g = groups_of(dev, [0, 4, 6], [0, 1, 2, 5, 4, 3], [300, 77], 4, 300)
    q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, lens, r2t, groups=g)
    assert st == 0
    for b, n in enumerate(lens):
        k, v = cache.values(r2t[b, :n])
        agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), n - 1), dt)


@gpu
@pytest.mark.parametrize("fmt,block,hq,hkv,d,members,shared", [(E4M3, 1, 32, 8, 128, 70, 4001), (INT8, 64, 12, 12, 64, 300, 129),
                                                             (INT8, 1, 8, 1, 128, 5, 20000), (E4M3, 1, 6, 2, 64, 200, 1)])
def test_decode_q8_large_groups(dev, fmt, block, hq, hkv, d, members, shared):
    """Groups whose rows fill several tiles, runs that several SMs share; members that have nothing of their own; others
    between them."""
    b = members + 6
    lens = [shared + 3 * (i % 4) for i in range(members)] + [0, 1, 40, shared, 2, 7]
    slots = shared + sum(n - shared for n in lens[:members]) + sum(lens[members:]) + 9
    ids = torch.randperm(slots, device=dev).to(torch.int32)
    stride = (max(lens) + 7) // 8 * 8
    r2t = torch.full((b, stride), -1, dtype=torch.int32, device=dev)
    at = shared
    for i, n in enumerate(lens):
        k = shared if i < members else 0
        r2t[i, :k] = ids[:k]
        r2t[i, k:n] = ids[at:at + n - k]
        at += n - k
    cache = Cache(dev, fmt, slots, hkv, d, block, seed=8)
    g = groups_of(dev, [0, members], np.random.default_rng(0).permutation(members), [shared], members, shared)
    q, out, lse, st = decode(dev, cache, BF, hq, hkv, d, lens, r2t, groups=g)
    assert st == 0
    for i in [0, 1, 2, members - 1] + list(range(members, b)):
        k, v = cache.values(r2t[i, :lens[i]])
        agree(out[i:i + 1], lse[i:i + 1], attend(q[i:i + 1], k, v, 1 / math.sqrt(d), lens[i] - 1), BF)
    alone = decode(dev, cache, BF, hq, hkv, d, lens, r2t)
    # the same sums in another order: each within the bound above, so twice its rounding apart
    assert ((out - alone[1]).float().abs().max() <= 2.0 ** -6 * out.float().abs().max())
    assert torch.equal(lse.isinf(), alone[2].isinf()) and (lse - alone[2]).nan_to_num(0.0).abs().max() < 1e-3


@gpu
def test_decode_q8_bad_groups(dev):
    """Members that are no request, runs longer than a member or than the table, boundaries that decrease: reported or left out,
    and every request gets its row."""
    hq, hkv, d = 8, 2, 128
    lens = [90, 80, 50, 90]
    r2t, _ = table_of(lens, 96, 400, dev)
    r2t[1, :80] = r2t[0, :80]
    r2t[3, :90] = r2t[0, :90]
    cache = Cache(dev, INT8, 400, hkv, d, seed=4)
    for ind, mem, length, code in (([0, 3], [0, 7, 1], [80], api.RX_DEV_BAD_LENGTH), ([0, 2], [0, -1], [60], api.RX_DEV_BAD_LENGTH),
                                   ([0, 3], [0, 1, 3], [85], 0), ([0, 2], [0, 1], [97], api.RX_DEV_BAD_LENGTH),
                                   ([0, 2, 1], [0, 1], [80, 5], api.RX_DEV_BAD_LENGTH), ([0, 9], [0, 1], [80], api.RX_DEV_BAD_LENGTH),
                                   ([0, 0], [0], [80], 0), ([0, 2], [0, 1], [0], api.RX_DEV_BAD_LENGTH)):
        mem = mem + [0] * 8
        g = groups_of(dev, ind, mem, length, 3, 90)
        q, out, lse, st = decode(dev, cache, BF, hq, hkv, d, lens, r2t, groups=g)
        assert st == code, (ind, mem, length)
        for b, n in enumerate(lens):
            k, v = cache.values(r2t[b, :n])
            agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), n - 1), BF)


@gpu
def test_decode_q8_one_workspace_for_all(dev):
    """The workspace of the greatest call, for calls that share contexts out and calls that do not."""
    hq, hkv, d = 12, 12, 64
    desc = desc_of(BF, hq, hkv, d, 40000)
    ws = torch.empty(api.decode_q8_workspace_bytes(desc, 16, 3000), dtype=torch.uint8, device=dev)
    for lens in ([3000], [2500, 3000], [3000, 1] * 8, [30] * 16, [2000] * 9):
        r2t, _ = table_of(lens, 3000, 40000, dev)
        cache = Cache(dev, E4M3, 40000, hkv, d, seed=6)
        q, out, lse, st = decode(dev, cache, BF, hq, hkv, d, lens, r2t, ws=ws)
        assert st == 0
        for b, n in enumerate(lens):
            k, v = cache.values(r2t[b, :n])
            agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), n - 1), BF)


@gpu
def test_decode_q8_requests_named_twice(dev):
    """A request that is named twice, in a group or in two of different lengths, is reported and has its row all the same."""
    hq, hkv, d = 8, 2, 128
    lens = [90, 80, 50, 90, 64]
    r2t, _ = table_of(lens, 96, 600, dev)
    for b in (1, 2, 3, 4):
        r2t[b, :50] = r2t[0, :50]
    cache = Cache(dev, E4M3, 600, hkv, d, seed=6)
    for ind, mem, length in (([0, 3], [0, 1, 0], [50]), ([0, 2, 4], [0, 1, 1, 3], [50, 20]), ([0, 40], [4] * 40, [50]),
                             ([0, 3, 6], [0, 1, 2, 2, 1, 0], [40, 40])):
        g = groups_of(dev, ind, mem, length, 40, 50)
        q, out, lse, st = decode(dev, cache, BF, hq, hkv, d, lens * 8, r2t.repeat(8, 1), groups=g)
        assert st == api.RX_DEV_BAD_LENGTH
        for b, n in enumerate(lens * 8):
            k, v = cache.values(r2t[b % 5, :n])
            agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), n - 1), BF)


# ============================================================================ extend
def extend(dev, cache, dt, hq, hkv, d, lens, pre, r2t, scale=None, lead=0, longest=None, q=None):
    n = sum(lens)
    desc = desc_of(dt, hq, hkv, d, cache.k.shape[0], scale)
    if q is None:
        q = torch.randn(lead + n + 2, hq, d, generator=torch.Generator(device=dev).manual_seed(n + hq), device=dev).to(dt)
    out, lse = torch.full_like(q, 9.0), torch.full((q.shape[0], hq), 9.0, device=dev)
    longest = r2t.shape[1] if longest is None else longest
    nbytes = api.extend_q8_workspace_bytes(desc, len(lens), max(lens), longest)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    api.prefix_extend_attention_q8(desc, cache.q8, len(lens), q, indptr(lens, dev, lead), i32(pre, dev), r2t, cache.k, cache.v,
                                   cache.scales, out, lse, max(lens), ws, st, max_kv_len=longest)
    assert (out[:lead] == 9.0).all() and (out[lead + n:] == 9.0).all() and (lse[lead + n:] == 9.0).all()
    return q, out, lse, int(st)


def extend_agrees(cache, dt, d, lens, pre, r2t, q, out, lse, lead=0):
    at = lead
    for b, (n, p) in enumerate(zip(lens, pre)):
        k, v = cache.values(r2t[b, :n + p])
        agree(out[at:at + n], lse[at:at + n], attend(q[at:at + n], k, v, 1 / math.sqrt(d), p), dt)
        at += n


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_extend_q8(dev, fmt, dt, hq, hkv, d):
    lens, pre = [1, 3, 0, 17, 64, 129, 5, 2], [0, 0, 50, 100, 31, 127, 700, 128]
    total = [a + b for a, b in zip(lens, pre)]
    slots = sum(total) + 33
    r2t, used = table_of(total, 712, slots, dev)
    cache = Cache(dev, fmt, slots, hkv, d, seed=hq)
    poison(cache, used)
    q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, lens, pre, r2t, lead=3)
    assert st == 0
    extend_agrees(cache, dt, d, lens, pre, r2t, q, out, lse, lead=3)


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("lens,pre,block", [([1], [9000], 1), ([7], [20000], 16), ([300], [1500], 1), ([2, 33], [4000, 130], 64),
                                            ([513], [0], 1 << 30)])
def test_extend_q8_long(dev, fmt, dt, lens, pre, block):
    hq, hkv, d = 8, 2, 128
    total = [a + b for a, b in zip(lens, pre)]
    slots = sum(total) + 33
    r2t, used = table_of(total, (max(total) + 7) // 8 * 8, slots, dev)
    cache = Cache(dev, fmt, slots, hkv, d, block, seed=7)
    poison(cache, used)
    q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, lens, pre, r2t)
    assert st == 0
    extend_agrees(cache, dt, d, lens, pre, r2t, q, out, lse)


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
def test_extend_q8_later_rows_do_not_reach_earlier_ones(dev, fmt, dt):
    """A new token whose key or value is not finite: the rows before it are what they are without it."""
    hq, hkv, d = 8, 2, 64
    r2t, _ = table_of([200], 200, 210, dev)
    cache = Cache(dev, fmt, 210, hkv, d, seed=9)
    cache.scales[r2t[0, 150].long()] = math.nan
    cache.scales[r2t[0, 180].long()] = math.inf
    q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, [150], [50], r2t)
    assert st == 0 and out[:100].isfinite().all() and out[100:150].isnan().all()
    k, v = cache.values(r2t[0, :150])
    agree(out[:100], lse[:100], attend(q[:100], k, v, 1 / math.sqrt(d), 50), dt)


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
def test_extend_q8_scales_far_apart(dev, fmt, dt):
    hq, hkv, d, n = 4, 2, 64, 140
    cache = Cache(dev, fmt, 300, hkv, d, seed=3)
    r2t, _ = table_of([290], 296, 300, dev)
    cache.scales[:, :, 1] *= (torch.randn(300, hkv, device=dev) * 12).exp2()
    cache.scales[r2t[0, 3].long(), :, 1] = 1e30
    bytes_of(cache.v)[r2t[0, 7].long()] = 0
    cache.scales[r2t[0, 7].long(), :, 1] = 2.0 ** -126
    cache.scales[r2t[0, 200].long(), :, 0] = 0.0
    q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, [n], [150], r2t)
    assert st == 0
    extend_agrees(cache, dt, d, [n], [150], r2t, q, out, lse)


@gpu
@pytest.mark.parametrize("dt", [BF, F])
def test_extend_q8_bad_slots_and_lengths(dev, dt):
    hq, hkv, d = 8, 2, 64
    lens, pre = [20, 3, 40], [30, 0, 130]
    r2t, _ = table_of([50, 3, 170], 176, 300, dev)
    cache = Cache(dev, INT8, 300, hkv, d, seed=2)
    r2t[0, 7], r2t[0, 49], r2t[1, 0], r2t[2, 131] = -1, 300, 1 << 30, -7
    q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, lens, pre, r2t)
    assert st == api.RX_DEV_BAD_SLOT
    at = 0
    for b, (n, p) in enumerate(zip(lens, pre)):
        for i in range(n):
            ok = r2t[b, :p + i + 1]
            ok = ok[(ok >= 0) & (ok < 300)]
            k, v = cache.values(ok)
            agree(out[at:at + 1], lse[at:at + 1], attend(q[at:at + 1], k, v, 1 / math.sqrt(d), len(ok) - 1), dt)
            at += 1
    good, _ = table_of([50, 3, 170], 176, 300, dev)
    for pre, longest in (([30, -1, 130], 176), ([30, 175, 130], 176), ([30, 100, 130], 102)):
        q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, lens, pre, good, longest=longest)
        assert st == api.RX_DEV_BAD_LENGTH
        assert (out[20:23] == 9.0).all()
        extend_agrees(cache, dt, d, [20], [30], good, q, out, lse)


@gpu
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows", [1, 8, 40, 5000])
def test_attention_q8_bounds_far_above(dev, dt, rows):
    """The host's bounds may be far above the lengths; batches without any new token or key."""
    hq, hkv, d, most = 4, 2, 64, 2 ** 31 - 1
    desc = desc_of(dt, hq, hkv, d, 300)
    cache = Cache(dev, E4M3, 300, hkv, d, seed=3)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for lens, pre in (([0, 0, 0], [5, 0, 70]), ([0, 1, 0, 0, 1], [0, 0, 9, 3, 90])):
        r2t, _ = table_of([n + p for n, p in zip(lens, pre)], 96, 300, dev)
        q = torch.randn(sum(lens) + 1, hq, d, device=dev).to(dt)
        out = torch.full_like(q, 9.0)
        lse = torch.full((len(q), hq), 9.0, device=dev)
        ws = torch.empty(max(api.extend_q8_workspace_bytes(desc, len(lens), rows, most), 1), dtype=torch.uint8, device=dev)
        api.prefix_extend_attention_q8(desc, cache.q8, len(lens), q, indptr(lens, dev), i32(pre, dev), r2t, cache.k, cache.v,
                                       cache.scales, out, lse, rows, ws, st, max_kv_len=most)
        assert int(st) == 0 and (out[-1] == 9.0).all() and (lse[-1] == 9.0).all()
        extend_agrees(cache, dt, d, lens, pre, r2t, q, out, lse)
    r2t, _ = table_of([0, 7, 0], 8, 300, dev)
    q, out, lse, code = decode(dev, cache, dt, hq, hkv, d, [0, 7, 0], r2t, longest=most)
    k, v = cache.values(r2t[1, :7])
    assert code == 0 and (out[[0, 2]] == 0).all() and lse[[0, 2]].isneginf().all()
    agree(out[1:2], lse[1:2], attend(q[1:2], k, v, 1 / math.sqrt(d), 6), dt)


# ============================================================================ together
@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_q8(dev, fmt, dt, captured):
    """Prompts written and extended, then tokens decoded one by one, as a serving loop runs them; eager and as a
    captured graph whose inputs change between replays; on a stream of its own."""
    hq, hkv, d, slots, b = 8, 2, 64, 600, 3
    torch.manual_seed(11)
    cache = Cache(dev, fmt, slots, hkv, d, seed=1)
    ids = torch.randperm(slots, device=dev).to(torch.int32)
    lens = [60, 1, 130]
    stride = 144
    desc, c = desc_of(dt, hq, hkv, d, slots), cache.q8
    r2t = torch.full((b, stride), -1, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    n = sum(lens)
    x = torch.randn(n, hq + 2 * hkv, d, device=dev).to(dt)
    q, k, v = x[:, :hq].contiguous(), x[:, hq:hq + hkv], x[:, hq + hkv:]
    out, lse = torch.empty_like(q), torch.empty(n, hq, device=dev)
    ew = torch.empty(max(api.extend_q8_workspace_bytes(desc, b, 130, stride), 1), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.kv_pool_write_q8(desc, c, b, None, i64([0] * 4, dev), ids[:n].contiguous(), indptr(lens, dev), k, v, cache.k, cache.v,
                             cache.scales, r2t, n, st)
        api.prefix_extend_attention_q8(desc, c, b, q, indptr(lens, dev), i32([0] * 3, dev), r2t, cache.k, cache.v, cache.scales, out,
                                       lse, 130, ew, st)
    side.synchronize()
    extend_agrees(cache, dt, d, lens, [0] * 3, r2t, q, out, lse)
    # the prompts' values are what was written
    at = ids[:n].long()
    want = codes_of(v, scales_of(v, fmt), fmt) * scales_of(v, fmt)[..., None]
    assert torch.equal(cache.values(at)[1], want)

    steps = 4
    kv_lens, qd = i32(lens, dev), torch.empty(b, hq, d, dtype=dt, device=dev)
    kn, vn = (torch.empty(b, hkv, d, dtype=dt, device=dev) for _ in range(2))
    new, old, oi = (torch.zeros(b, dtype=torch.int32, device=dev), torch.zeros(stride * b, dtype=torch.int32, device=dev),
                    torch.zeros(b + 1, dtype=torch.int64, device=dev))
    od, ld = torch.empty_like(qd), torch.empty(b, hq, device=dev)
    longest = max(lens) + steps
    dw = torch.empty(max(api.decode_q8_workspace_bytes(desc, b, longest), 1), dtype=torch.uint8, device=dev)
    qi = indptr([1] * b, dev)

    def step():
        api.kv_pool_write_q8(desc, c, b, old, oi, new, qi, kn, vn, cache.k, cache.v, cache.scales, r2t, b, st)
        api.decode_attention_q8(desc, c, b, qd, r2t, kv_lens, cache.k, cache.v, cache.scales, od, ld, longest, dw, st)

    graph = None
    tables = [r2t[i, :m].clone() for i, m in enumerate(lens)]
    for t in range(steps):
        fresh = ids[n + t * b:n + (t + 1) * b]
        oi.copy_(indptr([len(x) for x in tables], dev))
        old[:int(oi[-1])] = torch.cat(tables)
        tables = [torch.cat([x, fresh[i:i + 1]]) for i, x in enumerate(tables)]
        new.copy_(fresh)
        for y in (qd, kn, vn):
            y.copy_(torch.randn(y.shape, device=dev).to(dt))
        kv_lens.copy_(i32([len(x) for x in tables], dev))
        if captured:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        else:
            step()
        assert int(st) == 0
        for i, x in enumerate(tables):
            kk, vv = cache.values(x)
            agree(od[i:i + 1], ld[i:i + 1], attend(qd[i:i + 1], kk, vv, 1 / math.sqrt(d), len(x) - 1), dt)


@gpu
@pytest.mark.parametrize("dt", [BF, F])
def test_q8_calls_at_once(dev, dt):
    """Calls on three streams, and two captured graphs replayed side by side, with workspaces of their own, give what each gives
    alone."""
    hq, hkv, d, slots = 16, 4, 128, 9000
    cache = Cache(dev, E4M3, slots, hkv, d, seed=12)
    desc = desc_of(dt, hq, hkv, d, slots)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    jobs = []
    for i, (lens, pre) in enumerate((([40, 300], [3000, 0]), ([1] * 9, [900] * 9), ([700], [1200]))):
        total = [a + b for a, b in zip(lens, pre)]
        stride = (max(total) + 7) // 8 * 8
        r2t, _ = table_of(total, stride, slots, dev, seed=i)
        q = torch.randn(sum(lens), hq, d, device=dev).to(dt)
        ws = [torch.empty(max(n, 256), dtype=torch.uint8, device=dev) for n in
              (api.extend_q8_workspace_bytes(desc, len(lens), max(lens), stride), api.decode_q8_workspace_bytes(desc, len(lens), stride))]
        jobs.append(dict(r2t=r2t, lens=lens, ind=indptr(lens, dev), pre=i32(pre, dev), kv=i32(total, dev), q=q, ws=ws, stride=stride,
                         out=torch.zeros_like(q), dec=torch.zeros(len(lens), hq, d, dtype=dt, device=dev), dq=q[:len(lens)].contiguous()))

    def run(j):
        api.prefix_extend_attention_q8(desc, cache.q8, len(j["lens"]), j["q"], j["ind"], j["pre"], j["r2t"], cache.k, cache.v, cache.scales,
                                       j["out"], None, max(j["lens"]), j["ws"][0], st)
        api.decode_attention_q8(desc, cache.q8, len(j["lens"]), j["dq"], j["r2t"], j["kv"], cache.k, cache.v, cache.scales, j["dec"], None,
                                j["stride"], j["ws"][1], st)
    want = []
    for j in jobs:
        run(j)
        torch.cuda.synchronize()
        want.append((j["out"].clone(), j["dec"].clone()))
    streams = [torch.cuda.Stream() for _ in jobs]
    graphs = []
    for j, s in zip(jobs[:2], streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            run(j)
    for captured in (False, True):
        for j in jobs:
            j["out"].zero_(), j["dec"].zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i, (j, s) in enumerate(zip(jobs, streams)):
                with torch.cuda.stream(s):
                    graphs[i].replay() if captured and i < 2 else run(j)
        torch.cuda.synchronize()
        assert int(st) == 0
        for j, w in zip(jobs, want):
            assert torch.equal(j["out"], w[0]) and torch.equal(j["dec"], w[1])


@gpu
def test_q8_slots_past_32_bits(dev):
    """Pools of more than 2^31 bytes, slots at their ends."""
    hq, hkv, d = 32, 16, 128
    slots = (1 << 31) // (hkv * d) + 5000
    q8 = api.q8_desc(E4M3)
    pools = [torch.zeros(slots, hkv, d, dtype=torch.int8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = torch.zeros(slots, hkv, 2, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    desc = desc_of(BF, hq, hkv, d, slots)
    n = 400
    new = (slots - 1 - torch.randperm(4000, device=dev)[:n]).to(torch.int32)
    k, v = (torch.randn(n, hkv, d, device=dev).to(BF) for _ in range(2))
    r2t = torch.empty(1, n, dtype=torch.int32, device=dev)
    api.kv_pool_write_q8(desc, q8, 1, None, i64([0, 0], dev), new, i64([0, n], dev), k, v, *pools, scales, r2t, n, st)
    out = [torch.empty_like(k) for _ in range(2)]
    api.kv_pool_read_q8(desc, q8, new, *pools, scales, *out, st)
    for y, o in zip((k, v), out):
        assert torch.equal(o.double(), codes_of(y, scales_of(y, E4M3), E4M3) * scales_of(y, E4M3)[..., None])
    q = torch.randn(60, hq, d, device=dev).to(BF)
    got, lse = torch.empty_like(q), torch.empty(60, hq, device=dev)
    ws = torch.empty(max(api.extend_q8_workspace_bytes(desc, 1, 60, n), api.decode_q8_workspace_bytes(desc, 1, n), 256),
                     dtype=torch.uint8, device=dev)
    api.prefix_extend_attention_q8(desc, q8, 1, q, i64([0, 60], dev), i32([n - 60], dev), r2t, *pools, scales, got, lse, 60, ws, st)
    values = [o.double() for o in out]
    agree(got, lse, attend(q, *values, 1 / math.sqrt(d), n - 60), BF)
    api.decode_attention_q8(desc, q8, 1, q[:1], r2t, i32([n], dev), *pools, scales, got[:1], lse[:1], n, ws, st)
    agree(got[:1], lse[:1], attend(q[:1], *values, 1 / math.sqrt(d), n - 1), BF)
    assert int(st) == 0


@gpu
def test_binding_refuses(dev):
    """Wrong types, sizes and devices are refused by the extension and by the Python code alike."""
    hq, hkv, d, slots = 4, 2, 64, 32
    cache = Cache(dev, INT8, slots, hkv, d)
    desc, st = desc_of(BF, hq, hkv, d, slots), torch.zeros(1, dtype=torch.int32, device=dev)
    r2t, _ = table_of([5, 9], 16, slots, dev)
    q = torch.zeros(2, hq, d, dtype=BF, device=dev)
    good = dict(q=q, r2t=r2t, lens=i32([5, 9], dev), k=cache.k, v=cache.v, s=cache.scales, out=q.clone(), st=st)
    ext = api.ops_ext()
    assert ext is not None
    try:
        for use in (ext, False):
            api._ops_ext = use
            for name, wrong in (("q", q.float()), ("q", q[:1]), ("q", q.cpu()), ("q", q.transpose(1, 2)), ("r2t", r2t.long()),
                                ("lens", i64([5, 9], dev)), ("k", cache.k.view(torch.float8_e4m3fn)), ("v", cache.v[:5]),
                                ("s", cache.scales[:5]), ("s", cache.scales.double()), ("out", q[:1]), ("st", st.long())):
                a = dict(good, **{name: wrong})
                with pytest.raises(ValueError):
                    api.decode_attention_q8(desc, cache.q8, 2, a["q"], a["r2t"], a["lens"], a["k"], a["v"], a["s"], a["out"], None, 9,
                                            torch.empty(1 << 20, dtype=torch.uint8, device=dev), a["st"])
            rows = torch.zeros(3, hkv, d, dtype=BF, device=dev)
            for name, wrong in (("k", rows.float()), ("k", rows[:2]), ("k", rows.cpu()), ("s", cache.scales[1:])):
                a = dict(dict(k=rows, s=cache.scales), **{name: wrong})
                with pytest.raises(ValueError):
                    api.kv_pool_write_q8(desc, cache.q8, 1, None, i64([0, 0], dev), i32([1, 2, 3], dev), i64([0, 3], dev), a["k"], rows,
                                         cache.k, cache.v, a["s"], None, 3, st)
                with pytest.raises(ValueError):
                    api.kv_pool_read_q8(desc, cache.q8, i32([1, 2, 3], dev), cache.k, cache.v, a["s"], a["k"], rows, st)
    finally:
        api._ops_ext = ext


# ============================================================================ what the table may hold, any value of it
@gpu
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("d,block", [(64, 1), (128, 16)])
@pytest.mark.parametrize("bad", [-2, -1, -3, -2 ** 31, 2 ** 31 - 1])
def test_extend_q8_any_bad_slot(dev, dt, d, block, bad):
    """Whatever a bad entry's value: reported and left out, by calls of few rows and of many, beside the others and alone."""
    hq, hkv, slots = 8, 2, 800
    for lens, pre in (([30, 5, 40], [200, 9, 0]), ([1, 2, 2], [200, 9, 0])):
        total = [n + p for n, p in zip(lens, pre)]
        for places in ([(0, 7)], [(0, 7), (0, 130), (0, total[0] - 1), (1, 0), (1, 9)], [(2, 0), (2, 1)]):
            r2t, _ = table_of(total, 240, slots, dev)
            cache = Cache(dev, INT8, slots, hkv, d, block, seed=2)
            for b, i in places:
                r2t[b, i] = bad
            q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, lens, pre, r2t)
            assert st == api.RX_DEV_BAD_SLOT
            at = 0
            for b, (n, p) in enumerate(zip(lens, pre)):
                for i in range(n):
                    ok = r2t[b, :p + i + 1]
                    ok = ok[(ok >= 0) & (ok < slots)]
                    agree(out[at:at + 1], lse[at:at + 1], attend(q[at:at + 1], *cache.values(ok), 1 / math.sqrt(d), len(ok) - 1), dt)
                    at += 1


@gpu
@pytest.mark.parametrize("bad", [-2, -1, -2 ** 31, 2 ** 31 - 1])
def test_decode_q8_any_bad_slot_in_a_shared_run(dev, bad):
    """A bad entry in a group's run, or behind it, is reported and left out."""
    hq, hkv, d, slots = 8, 2, 128, 3000
    lens = [300, 411, 301, 90, 640, 300]
    for place in (0, 131, 299, 300):
        r2t, _ = table_of(lens, 648, slots, dev)
        r2t[[1, 2, 5], :300] = r2t[0, :300].clone()
        if place < 300:
            r2t[[0, 1, 2, 5], place] = bad
        else:
            r2t[1, place] = bad
        cache = Cache(dev, E4M3, slots, hkv, d, seed=4)
        g = groups_of(dev, [0, 4], [0, 1, 2, 5], [300], 4, 300)
        q, out, lse, st = decode(dev, cache, BF, hq, hkv, d, lens, r2t, groups=g)
        assert st == api.RX_DEV_BAD_SLOT
        for b, n in enumerate(lens):
            ok = r2t[b, :n]
            ok = ok[(ok >= 0) & (ok < slots)]
            agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], *cache.values(ok), 1 / math.sqrt(d), len(ok) - 1), BF)


# ============================================================================ value scales of any size, f32 rows
def one_product(dev, fmt, n, hq, hkv, d, rows, power, seed=0):
    """Queries and a cache whose scores are one product each, at most 1, so that little of the score is rounded: channel 5
    alone, of 24 bits.  V's scales are 1 to 2 times 2^power."""
    g = torch.Generator(device=dev).manual_seed(seed + n + hq + rows)
    cache = Cache(dev, fmt, n, hkv, d, seed=seed)
    cache.scales[..., 0] = math.sqrt(d) / TOP[fmt]
    cache.scales[..., 1] = (1 + torch.rand(n, hkv, generator=g, device=dev)) * 2.0 ** power
    q = torch.zeros(rows, hq, d, device=dev)
    q[..., 5] = 0.5 + 0.5 * torch.rand(rows, hq, generator=g, device=dev)
    r2t = torch.randperm(n, generator=g, device=dev).to(torch.int32)[None].contiguous()
    return cache, q, r2t


def agree_f32(out, want, keys):
    """f32 rows of scores of one product, |score| <= 1.  A score is off by 2.5 * 2^-22 of itself (two f16 parts of a query, the sum
    of their products, five roundings of the factors) and a rounding of its distance from the reference, an exponential by
    2^-22, a weight by its two parts' 2^-22 and its product's 2^-24: below 2^-19.2 of each p_j, and again of their sum.  The tensor
    core adds 16 products to a sum, each cut off at 2^-23 of the largest: 17 * 2^-23 of sum p |v| an instruction, two of them a
    16 keys of a warp."""
    o, _, a, _, _, _ = want
    tol = a * (2 ** -18.2 + 2 * math.ceil(keys / 16) * 17 * 2.0 ** -23 + 2.0 ** -23)
    assert (out.double() - o).abs().le(tol).all(), float(((out.double() - o).abs() / tol).max())


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (8, 8, 64), (2, 1, 128), (16, 8, 128), (12, 4, 64)])
@pytest.mark.parametrize("power", [0, -10, -60, -110, -120, -126, 100])
def test_q8_value_scales_of_any_size(dev, fmt, hq, hkv, d, power):
    """f32 rows are as exact with values near the smallest and largest numbers as with others."""
    n = 16
    cache, q, r2t = one_product(dev, fmt, n, hq, hkv, d, 1, power)
    q, out, lse, st = decode(dev, cache, F, hq, hkv, d, [n], r2t, q=q)
    assert st == 0
    agree_f32(out, attend(q, *cache.values(r2t[0]), 1 / math.sqrt(d), n - 1), n)
    rows = 12
    cache, q, r2t = one_product(dev, fmt, n, hq, hkv, d, rows, power)
    q, out, lse, st = extend(dev, cache, F, hq, hkv, d, [rows], [n - rows], r2t, q=torch.cat([q, q[:2]]))
    assert st == 0
    agree_f32(out[:rows], attend(q[:rows], *cache.values(r2t[0]), 1 / math.sqrt(d), n - rows), n)


@gpu
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (8, 8, 64), (2, 1, 128), (16, 8, 128)])
def test_decode_q8_many_keys_of_tiny_values(dev, dt, hq, hkv, d):
    """A thousand keys that count alike, with the smallest scale that the write makes: their mean, a normal number.  (Weights of
    one are exact in any type; a sum of 1000 / 16 instructions, cut off 17 * 2^-23 each at most, and the output's rounding.)"""
    n = 1000
    cache = Cache(dev, INT8, n, hkv, d, seed=1)
    cache.scales[..., 1] = 2.0 ** -126
    cache.k.zero_()
    r2t = torch.randperm(n, device=dev).to(torch.int32)[None].contiguous()
    q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, [n], r2t)
    assert st == 0
    o, _, a, _, _, _ = attend(q, *cache.values(r2t[0]), 1 / math.sqrt(d), n - 1)
    tol = a * (64 * 2 * 17 * 2.0 ** -23) + (o.abs() * 2.0 ** -8 + 2.0 ** -133 if dt == BF else 0)
    assert (out.double() - o).abs().le(tol).all(), float(((out.double() - o).abs() / a).max())


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("s", [2.0 ** -126, 1.5 * 2.0 ** -100, 2.0 ** 120, 1.25 * 2.0 ** 121, 1.75 * 2.0 ** 126, 2.0 ** 127])
def test_write_q8_given_scales_of_any_size(dev, fmt, dt, s):
    """Given scales from the smallest to the largest normal numbers, with rows of any size: codes of the real quotient, cut."""
    x = torch.tensor([math.inf, -math.inf, 3.3e38, -3.3e38, 1e38, -1e38, 1.0, 2.0 ** -120, -(2.0 ** -126), 2.0 ** -133, s, -s, 3 * s, 2.5 * s, 1.5 * s,
                      0.0] * 4, device=dev, dtype=torch.float64).float().to(dt).view(1, 1, 64)
    c, desc = api.q8_desc(fmt, 1, True), desc_of(dt, 1, 1, 64, 1)
    pools = [torch.zeros(1, 1, 64, dtype=torch.int8, device=dev).view(TYPE[fmt]) for _ in range(2)]
    scales, st = torch.full((1, 1, 2), s, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    api.kv_pool_write_q8(desc, c, 1, None, None, i32([0], dev), i64([0, 1], dev), x, x, *pools, scales, None, 1, st)
    want = codes_of(x[0], scales[0, :, 0], fmt)
    for p in pools:
        assert torch.equal(p[0].double(), want), (p[0].double() - want).nonzero()


def test_q8_errors_name_the_call():
    """Without a device, calls that pass all checks fail under their own names, decode with groups too.  (In a process that sees
    no GPU, wherever it runs: the addresses are none.)"""
    code = textwrap.dedent("""
        import ctypes
        from prefix_cached_kv_radix_gb300 import api
        lib, by, A = api.load(), ctypes.byref, 0x1000
        d, c = api.make_desc(api.RX_BF16, 8, 2, 128, 64, 0.1), api.q8_desc(api.RX_Q8_INT8)
        g = api.rx_shared_groups()
        g.num_groups, g.max_group_size, g.max_group_len = 1, 2, 8
        g.d_group_indptr, g.d_group_members, g.d_group_len = A, A, A
        def failed(fn, *args):
            rc = getattr(lib, fn)(*args)
            text = lib.rx_last_error().decode()
            assert rc not in (api.RX_OK, api.RX_EINVAL) and text.startswith(fn + ":"), (fn, rc, text)
        failed("decode_attention_q8", by(d), by(c), 2, A, A, 8, A, by(g), A, A, A, A, None, 8, A, 1 << 40, None, None)
        failed("decode_attention_q8", by(d), by(c), 2, A, A, 8, A, None, A, A, A, A, None, 8, A, 1 << 40, None, None)
        for rows in (1, 5):
            failed("prefix_extend_attention_q8", by(d), by(c), 1, A, A, A, A, 8, A, A, A, A, None, rows, 8, A, 1 << 40, None, None)
        failed("kv_pool_write_q8", by(d), by(c), 1, A, A, A, A, A, 256, A, 256, A, A, A, A, 8, 4, None, None)
        failed("kv_pool_read_q8", by(d), by(c), 4, A, A, A, A, A, 256, A, 256, None, None)
    """)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), capture_output=True, text=True)
    assert got.returncode == 0, got.stderr


@gpu
@pytest.mark.parametrize("dt", [BF, F])
def test_attention_q8_lengths_near_the_32_bit_limit(dev, dt):
    """Requests of more than 2^31 - 2^16 keys are refused on the device, before any of their slots is read: the table here holds the
    first of its entries only."""
    hq, hkv, d, most = 8, 2, 64, 2 ** 31 - 1
    desc, cache = desc_of(dt, hq, hkv, d, 64), Cache(dev, INT8, 64, hkv, d, seed=1)
    table = torch.zeros(4096, dtype=torch.int32, device=dev)
    lib, by = api.load(), ctypes.byref
    for length in (most, most - 1000, most - 65534):
        st, out = torch.zeros(1, dtype=torch.int32, device=dev), torch.full((40, hq, d), 9.0, device=dev, dtype=dt)
        q, lse = torch.zeros_like(out), torch.full((40, hq), 9.0, device=dev)
        ws = torch.empty(api.decode_q8_workspace_bytes(desc, 1, most), dtype=torch.uint8, device=dev)
        lens = i32([length], dev)
        assert lib.decode_attention_q8(by(desc), by(cache.q8), 1, q.data_ptr(), table.data_ptr(), most, lens.data_ptr(), None,
                                       cache.k.data_ptr(), cache.v.data_ptr(), cache.scales.data_ptr(), out.data_ptr(), lse.data_ptr(), most,
                                       ws.data_ptr(), ws.numel(), st.data_ptr(), torch.cuda.current_stream().cuda_stream) == api.RX_OK
        assert int(st) == api.RX_DEV_BAD_LENGTH and (out == 9.0).all() and (lse == 9.0).all()
        for rows in (2, 40):
            st.zero_()
            ws = torch.empty(api.extend_q8_workspace_bytes(desc, 1, rows, most), dtype=torch.uint8, device=dev)
            ind, pre = i64([0, rows], dev), i32([length - rows], dev)
            assert lib.prefix_extend_attention_q8(by(desc), by(cache.q8), 1, q.data_ptr(), ind.data_ptr(), pre.data_ptr(), table.data_ptr(),
                                                  most, cache.k.data_ptr(), cache.v.data_ptr(), cache.scales.data_ptr(), out.data_ptr(),
                                                  lse.data_ptr(), rows, most, ws.data_ptr(), ws.numel(), st.data_ptr(),
                                                  torch.cuda.current_stream().cuda_stream) == api.RX_OK
            assert int(st) == api.RX_DEV_BAD_LENGTH and (out == 9.0).all() and (lse == 9.0).all()


# ============================================================================ what the tolerances and sizes above leave out
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (16, 8, 128)])
def test_agree_f32_notices_a_part_left_out(hq, hkv, d):
    """Queries or weights of one f16 part instead of two, here in the oracle: agree_f32 refuses either."""
    cpu, n = torch.device("cpu"), 16
    cache, q, r2t = one_product(cpu, INT8, n, hq, hkv, d, 1, 0)
    k, v = cache.values(r2t[0])
    want = attend(q, k, v, 1 / math.sqrt(d), n - 1)
    agree_f32(want[0].float(), want, n)
    with pytest.raises(AssertionError):
        agree_f32(attend(q.half(), k, v, 1 / math.sqrt(d), n - 1)[0], want, n)
    s = torch.einsum("hgd,khd->hgk", q[0].double().view(hkv, hq // hkv, d), k) / math.sqrt(d)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    vs, codes = cache.scales[r2t[0].long(), :, 1].double(), v / cache.scales[r2t[0].long(), :, 1:].double()
    w = p * vs.t()[:, None, :]
    w = (w * (2.0 ** 14 / w.amax(-1, keepdim=True))).half().double() / (2.0 ** 14 / w.amax(-1, keepdim=True))
    with pytest.raises(AssertionError):
        agree_f32((torch.einsum("hgk,khd->hgd", w, codes) / p.sum(-1, keepdim=True)).reshape(1, hq, d), want, n)


EIGHTS = [(8, 8, 64), (32, 8, 128), (24, 8, 64), (16, 16, 128)]


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d", EIGHTS)
def test_attention_q8_kv_heads_by_eights(dev, fmt, dt, hq, hkv, d):
    """Eight kv heads a CTA, a warp each: whole contexts of many requests, and a few long ones shared out."""
    for lens in ([1, 0, 2, 15, 16, 17, 33, 40] * 30, [5000, 3, 2047]):
        slots = sum(lens) + 9
        r2t, used = table_of(lens, (max(lens) + 7) // 8 * 8, slots, dev)
        cache = Cache(dev, fmt, slots, hkv, d, seed=hq)
        poison(cache, used)
        q, out, lse, st = decode(dev, cache, dt, hq, hkv, d, lens, r2t)
        assert st == 0
        for b in list(range(min(len(lens), 16))) + [len(lens) - 1]:
            k, v = cache.values(r2t[b, :lens[b]])
            agree(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], k, v, 1 / math.sqrt(d), lens[b] - 1), dt)
    most = 16 * hkv // hq                        # as many tokens as make 16 rows
    for lens, pre in (([most, 1, 0, most, 2] * 40, [0, 30, 5, 11, 1] * 40), ([most, 1], [4100, 700])):
        total = [a + b for a, b in zip(lens, pre)]
        slots = sum(total) + 9
        r2t, used = table_of(total, (max(total) + 7) // 8 * 8, slots, dev)
        cache = Cache(dev, fmt, slots, hkv, d, seed=hq)
        poison(cache, used)
        q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, lens, pre, r2t)
        assert st == 0
        few = min(len(lens), 10)
        extend_agrees(cache, dt, d, lens[:few], pre[:few], r2t, q, out, lse)


def cut_off(x):
    """f32 numbers with the last bits of their float64 values cut off."""
    y = x.float()
    return torch.where(y.double().abs() > x.abs(), torch.nextafter(y, torch.zeros_like(y)), y)


def long_sum_tolerance(stages):
    """Of a sum of positive terms in 32 bits, relative: a stage's own sum is four instructions, each cut off at 17 * 2^-23; the
    stages are added with rounding, independent and 2^-24 of the sum so far at most, which grows evenly: beyond 6 times the
    square root of their squares' sum, stages / 3, with a probability below 2 e^-18; weights are off by 2^-21."""
    return 4 * 17 * 2.0 ** -23 + 6 * math.sqrt(stages / 3) * 2.0 ** -24 + 2.0 ** -21


def test_long_sums_tolerance_notices_sums_cut_off():
    g, stages = torch.Generator().manual_seed(0), 1600
    terms = torch.rand(stages, 64, generator=g, dtype=torch.float64) + 0.5
    exact, rounded, cut = terms.sum(0), torch.zeros(64), torch.zeros(64)
    for t in terms:
        rounded = (rounded.double() + t).float()
        cut = cut_off(cut.double() + t)
    assert ((rounded.double() - exact).abs() / exact).max() < long_sum_tolerance(stages)
    assert ((cut.double() - exact).abs() / exact).max() > long_sum_tolerance(stages)


@gpu
def test_decode_q8_f32_long_sums(dev):
    """51200 keys that count alike: 1600 stages one after another, added with rounding and not cut off as the tensor core does."""
    hq, hkv, d, n, b = 8, 8, 64, 51200, 300
    cache = Cache(dev, INT8, n, hkv, d, seed=1)
    bytes_of(cache.v).copy_(torch.randint(1, 128, cache.v.shape, device=dev, dtype=torch.uint8))
    cache.scales[..., 1] = 1 + torch.rand(n, hkv, device=dev)
    r2t = torch.randperm(n, device=dev).to(torch.int32)[None].repeat(b, 1)
    q, out, lse, st = decode(dev, cache, F, hq, hkv, d, [n] * b, r2t, q=torch.zeros(b, hq, d, device=dev))
    assert st == 0
    want = cache.values(torch.arange(n, device=dev))[1].mean(0)
    assert ((out.double() - want).abs() / want).max() < long_sum_tolerance(1600)
    assert (lse.double() - math.log(n)).abs().max() < 2.0 ** -18 * (1 + math.log(n))


@gpu
def test_extend_q8_items_of_seconds(dev):
    """Items that take longer than any wait between a block's warps for a single tile may (2 s): two of 110 million keys a block, with a
    bad slot in every tile.  One key outweighs the others by e^100, so every row is that key's value."""
    hkv, d, rows, keys = 304, 64, 17, 110_000_000
    desc, q8, slots = desc_of(BF, hkv, hkv, d, 4, scale=1.0), api.q8_desc(INT8), 4
    k, v = (torch.zeros(slots, hkv, d, dtype=torch.int8, device=dev) for _ in range(2))
    k[0, :, 0], k[1:, :, 0] = 100, -100
    v[0] = torch.randint(-127, 128, (hkv, d), device=dev)
    v[1:] = 127
    scales = torch.full((slots, hkv, 2), 0.5, device=dev)
    table = torch.ones(1, keys, dtype=torch.int32, device=dev)
    table[0, ::128] = -1
    table[0, keys - rows - 1] = 0
    q = torch.zeros(rows, hkv, d, dtype=BF, device=dev)
    q[..., 0] = 1.0
    out, lse = torch.full_like(q, 9.0), torch.full((rows, hkv), 9.0, device=dev)
    ws = torch.empty(api.extend_q8_workspace_bytes(desc, 1, rows, keys), dtype=torch.uint8, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    api.prefix_extend_attention_q8(desc, q8, 1, q, i64([0, rows], dev), i32([keys - rows], dev), table, k, v, scales, out, lse, rows, ws, st)
    assert int(st) == api.RX_DEV_BAD_SLOT
    assert torch.equal(out.float(), (v[0].float() * 0.5).expand(rows, hkv, d))
    assert (lse - 50.0).abs().max() < 1e-3


@gpu
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d,n", [(4, 4, 64, 2), (4, 2, 128, 4), (8, 8, 128, 3), (8, 2, 64, 4)])
@pytest.mark.parametrize("which", [0, 1])
def test_extend_q8_few_rows_do_not_see_later_scales(dev, fmt, dt, hq, hkv, d, n, which):
    """Calls of few rows: a later token's key or value scale, whatever it is, leaves the rows before it as they are."""
    for pre in (0, 15, 131):
        r2t, _ = table_of([n + pre], 144, 150, dev)
        cache = Cache(dev, fmt, 150, hkv, d, seed=9)
        for scale in (math.nan, math.inf, 2.0 ** 127):
            last = r2t[0, pre + n - 1].long()
            kept = cache.scales[last].clone()
            cache.scales[last, :, which] = scale
            q, out, lse, st = extend(dev, cache, dt, hq, hkv, d, [n], [pre], r2t)
            cache.scales[last] = kept
            k, v = cache.values(r2t[0, :n + pre - 1])
            agree(out[:n - 1], lse[:n - 1], attend(q[:n - 1], k, v, 1 / math.sqrt(d), pre), dt)
            assert st == 0 and (not math.isnan(scale) or out[n - 1].isnan().all())
