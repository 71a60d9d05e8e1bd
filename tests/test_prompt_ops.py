"""Whole-prompt attention, rotary pool writes, and pool-row moves: host checks on CPU, and the
kernels against plain 64-bit definitions on the GPU.

No configuration of the pages names these; they stand beside kv_pool_write and the attention
entry points and share their conventions.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from prefix_cached_kv_radix_gb300 import api
from tests.prompt_cases import attention, close, rotate

api.load()
gpu = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
A = 0x1000        # stands for an aligned device address in calls that are refused before any launch


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def desc_of(dt, hq, hkv, d, slots=64, scale=None):
    return api.make_desc(api.RX_F32 if dt == F else api.RX_BF16, hq, hkv, d, slots, 1 / math.sqrt(d) if scale is None else scale)


def indptr(lens, dev, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + start, dtype=torch.int64, device=dev)


def i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


# ============================================================================ refusals (CPU)
def refused(fn, *args):
    rc = getattr(api.load(), fn)(*args)
    assert rc == api.RX_EINVAL, (fn, rc)
    assert fn in api.load().rx_last_error().decode()


def test_prompt_attention_refuses():
    def call(desc=None, batch=1, q=A, qs=256, k=A, ks=128, v=A, vs=128, ind=A, out=A, os_=256, total=4):
        refused("prompt_attention", ctypes.byref(desc or desc_of(BF, 4, 2, 64)), batch, q, qs, k, ks, v, vs, ind, out, os_,
                None, total, None, None)
    for kw in (dict(batch=-1), dict(total=-1), dict(total=1 << 31), dict(q=None), dict(k=None), dict(v=None), dict(ind=None),
               dict(out=None), dict(q=A + 8), dict(k=A + 2), dict(qs=255), dict(ks=127), dict(ks=64), dict(os_=248),
               dict(vs=132), dict(desc=desc_of(BF, 4, 3, 64)), dict(desc=desc_of(BF, 4, 0, 64)), dict(desc=desc_of(BF, 4, 2, 96)),
               dict(desc=desc_of(BF, 4, 2, 64, scale=-1.0)), dict(desc=desc_of(BF, 4, 2, 64, scale=math.inf)),
               dict(desc=desc_of(BF, 4, 2, 64, scale=math.nan)), dict(desc=desc_of(BF, 4, 2, 64, scale=3e38)), dict(desc=api.make_desc(7, 4, 2, 64, 4, 1.0))):
        call(**kw)


def test_kv_pool_write_rope_refuses():
    base = dict(desc=desc_of(BF, 4, 2, 64), rope=api.rope_desc(32), batch=1, ps=A, pi=A, ns=A, qi=A, pos=A, pstr=4, q=A, qs=256,
                k=A, ks=128, v=A, vs=128, qo=2 * A, qos=256, ko=None, kos=0, kp=A, vp=A, r2t=A, stride=8, total=4)

    def call(**kw):
        c = dict(base, **kw)
        refused("kv_pool_write_rope", ctypes.byref(c["desc"]), ctypes.byref(c["rope"]), *[c[x] for x in list(base)[2:]], None, None)

    def rope(**kw):
        r = api.rope_desc(kw.pop("sections", 32))
        for x, y in kw.items():
            setattr(r, x, y)
        return r
    for kw in (dict(batch=-1), dict(total=-1), dict(stride=-1), dict(qi=None), dict(pos=None), dict(pstr=3), dict(k=None),
               dict(v=None), dict(kp=None), dict(vp=None), dict(pi=None), dict(ns=None), dict(q=None), dict(qo=None),
               dict(ns=None, r2t=None), dict(q=A + 4), dict(ks=120), dict(vs=129), dict(qo=A, qos=264), dict(ko=A, kos=136),
               dict(kp=A + 8), dict(desc=desc_of(BF, 4, 2, 80)), dict(desc=api.make_desc(3, 4, 2, 64, 4, 1.0)),
               dict(rope=rope(n_axes=0)), dict(rope=rope(n_axes=5)), dict(rope=rope(rot_dim=24)), dict(rope=rope(rot_dim=128)),
               dict(rope=rope(rot_dim=0)), dict(rope=rope(rot_dim=32)), dict(rope=rope(base=0.0)), dict(rope=rope(base=math.nan)),
               dict(rope=rope(sections=[40, -8], rot_dim=64)), dict(rope=api.rope_desc(32, inv_freq=[math.inf] * 32))):
        call(**kw)
    with pytest.raises(ValueError):
        api.rope_desc([8] * 5)
    with pytest.raises(ValueError):
        api.rope_desc(32, inv_freq=[1.0] * 31)


def test_kv_pool_copy_and_fork_refuse():
    d = desc_of(BF, 4, 2, 64)

    def pools(*a):
        return (ctypes.c_void_p * max(len(a), 1))(*a)
    for kw in (dict(n=-1), dict(page=0), dict(page=65), dict(np_=-1), dict(pl=None), dict(pl=pools(A, None)), dict(pl=pools(A, A + 8)),
               dict(pl=pools(A, A)), dict(src=None), dict(dst=None), dict(desc=desc_of(BF, 4, 1, 4)), dict(desc=desc_of(BF, 4, 2, 64, 0))):
        c = dict(dict(desc=d, np_=2, pl=pools(A, 2 * A), page=1, n=3, src=A, dst=A), **kw)
        refused("kv_pool_copy", ctypes.byref(c["desc"]), c["np_"], c["pl"], c["page"], c["n"], c["src"], c["dst"], None, None)
    base = dict(np_=2, pl=pools(A, 2 * A), rows=2, par=A, keep=A, lens=A, ti=A, ts=A, rin=A, inr=2, ins=8, rout=2 * A, outs=8, tail=3)
    for kw in (dict(rows=-1), dict(inr=-1), dict(ins=-1), dict(outs=-1), dict(tail=-1), dict(par=None), dict(keep=None),
               dict(lens=None), dict(ti=None), dict(ts=None), dict(rin=None), dict(rout=None), dict(pl=pools(A, A)),
               dict(rout=A), dict(rout=A + 60), dict(rin=2 * A + 60)):
        c = dict(base, **kw)
        refused("kv_pool_fork", ctypes.byref(d), *[c[x] for x in base], None, None)


def test_empty_calls_need_no_gpu():
    d, L = desc_of(BF, 4, 2, 64), api.load()
    r = api.rope_desc([16, 8, 8])
    assert L.prompt_attention(ctypes.byref(d), 0, None, 0, None, 0, None, 0, None, None, 0, None, 5, None, None) == api.RX_OK
    assert L.prompt_attention(ctypes.byref(d), 3, None, 0, None, 0, None, 0, A, None, 0, None, 0, None, None) == api.RX_OK
    assert L.kv_pool_write_rope(ctypes.byref(d), ctypes.byref(r), 0, *[None] * 5, 0, None, 0, None, 0, None, 0, None, 0, None, 0,
                                None, None, None, 0, 0, None, None) == api.RX_OK
    assert L.kv_pool_copy(ctypes.byref(d), 0, None, 1, 5, A, A, None, None) == api.RX_OK
    assert L.kv_pool_copy(ctypes.byref(d), 1, (ctypes.c_void_p * 1)(A), 1, 0, None, None, None, None) == api.RX_OK
    assert L.kv_pool_fork(ctypes.byref(d), 0, None, 0, *[None] * 6, 0, 0, None, 0, 0, None, None) == api.RX_OK


# ============================================================================ radix_resize (CPU)
def filled(num_slots, seed, seqs):
    t = api.RadixTree(num_slots, seed)
    for toks in seqs:
        sl, m, _ = t.match_prefix(toks)
        t.insert(toks, np.concatenate([sl, t.alloc_slots(len(toks) - m)]))
    return t


def free_order(t):
    n = t.stats()["free_slots"]
    sl = t.alloc_slots(n)
    t.free_slots(sl)
    return sl.tolist()


@pytest.mark.parametrize("seed,num,new", [(1, 64, 40), (2, 64, 27), (3, 200, 30), (4, 31, 31), (5, 40, 90), (6, 40, 41)])
def test_resize_against_model(seed, num, new):
    rng = np.random.default_rng(seed)
    seqs = [np.concatenate([[7, 7, 7], rng.integers(0, 3, rng.integers(1, 6))]).astype(np.int32) for _ in range(5)]
    t = filled(num, seed, seqs)
    before = {i: t.match_prefix(s)[0].tolist() for i, s in enumerate(seqs)}
    free = free_order(t)
    used = sorted({x for v in before.values() for x in v})
    src, dst = t.resize(new)
    # the model: used slots from `new` on, ascending, take the usable free slots in their order
    want_src = [x for x in used if x >= new]
    left = [x for x in free if x < new]
    assert src.tolist() == want_src and dst.tolist() == left[:len(want_src)]
    moved = dict(zip(want_src, dst.tolist()))
    for i, s in enumerate(seqs):
        assert t.match_prefix(s)[0].tolist() == [moved.get(x, x) for x in before[i]]
    t.check()
    assert t.stats()["num_slots"] == t.num_slots == new
    assert free_order(t) == left[len(want_src):] + list(range(num, new))
    assert not set(src.tolist()) & set(dst.tolist())


def test_resize_refuses_and_leaves_the_tree():
    t = filled(64, 9, [np.arange(20, dtype=np.int32)])
    held, n = t.alloc_slots(3), ctypes.c_int64()
    free, cached = t.stats()["free_slots"], t.match_prefix(np.arange(20, dtype=np.int32))[0].tolist()

    def code(new):
        with pytest.raises(api.RxError) as e:
            t.resize(new)
        t.check()
        assert t.stats()["num_slots"] == 64 and t.stats()["free_slots"] == free
        assert t.match_prefix(np.arange(20, dtype=np.int32))[0].tolist() == cached
        return e.value.code
    assert code(0) == code(-1) == code(1 << 31) == api.RX_EINVAL
    assert code(int(held.max())) == api.RX_EINVAL          # held by the caller
    t.free_slots(held)
    free = t.stats()["free_slots"]
    assert code(19) == api.RX_ENOMEM                       # 20 tokens are cached
    _, m, node = t.match_prefix(np.arange(20, dtype=np.int32))
    t.lock(node)
    assert code(max(cached)) == api.RX_ELOCKED
    t.unlock(node)
    need = sum(x >= 30 for x in cached)
    assert need > 1
    buf = np.empty(64, np.int32)
    args = (t.h, 30, api._addr(buf), api._addr(buf[32:]))
    assert api.load().radix_resize(*args, need - 1, ctypes.byref(n)) == api.RX_EINVAL and n.value == need
    assert api.load().radix_resize(t.h, 30, None, None, 0, ctypes.byref(n)) == api.RX_EINVAL and n.value == need
    assert api.load().radix_resize(*args, need, ctypes.byref(n)) == api.RX_OK and n.value == need
    t.check()


def test_resize_then_serve():
    """A shrunk pool fills, evicts, and grows again."""
    t = filled(50, 3, [np.arange(i, i + 10, dtype=np.int32) for i in (0, 100, 200)])
    t.resize(30)
    assert t.stats()["free_slots"] == 0
    freed = t.evict(10)
    assert len(freed) == 10 and freed.max() < 30
    assert t.resize(33)[0].size == 0
    sl = t.alloc_slots(13)
    assert sorted(sl.tolist()) == sorted(freed.tolist() + [30, 31, 32])
    t.insert(np.arange(300, 313, dtype=np.int32), sl)
    t.check()


# ============================================================================ kv_pool_copy, kv_pool_fork
def some_pools(gen, n, num, hkv, d, dt):
    x = torch.randn(n, num, hkv, d, generator=gen, device="cuda").to(dt)
    return x, [x[i] for i in range(n)]


@gpu
@pytest.mark.parametrize("dt,hkv,d", [(BF, 1, 64), (BF, 3, 64), (BF, 8, 128), (F, 1, 64), (F, 5, 128), (BF, 12, 64)])
@pytest.mark.parametrize("page,pages,n", [(1, 50, 1), (1, 4000, 1999), (16, 37, 18), (64, 9, 4), (7, 20, 6)])
@pytest.mark.parametrize("pools", [1, 2, 6])
def test_copy(dev, dt, hkv, d, page, pages, n, pools):
    gen = torch.Generator("cuda").manual_seed(n + d)
    num = pages * page + (page - 1)                       # a last page that is not whole
    x, lst = some_pools(gen, pools, num, hkv, d, dt)
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    src, dst, st = ids[:n].clone(), ids[n:2 * n].clone(), i32([0], "cuda")
    if n > 2:
        src[1] = src[0]                                   # one source, two destinations
        dst[2] = src[2]                                   # left where it is
    want = x.clone()
    w = want[:, :pages * page].unflatten(1, (pages, page))      # a view
    w[:, dst.long()] = w[:, src.long()].clone()
    api.kv_pool_copy(desc_of(dt, hkv, hkv, d, num), lst, src, dst, page, st)
    assert int(st.item()) == 0 and torch.equal(x, want)


@gpu
def test_copy_many_pools_and_bad_pages(dev):
    gen = torch.Generator("cuda").manual_seed(1)
    x, lst = some_pools(gen, 300, 40, 1, 64, BF)
    src, dst, st = i32([5, 40, 3, -1, 9], "cuda"), i32([20, 21, 40, 22, 23], "cuda"), i32([0], "cuda")
    want = x.clone()
    want[:, 20], want[:, 23] = x[:, 5], x[:, 9]
    api.kv_pool_copy(desc_of(BF, 1, 1, 64, 40), lst, src, dst, 1, st)
    assert int(st.item()) == api.RX_DEV_BAD_SLOT and torch.equal(x, want)


@gpu
def test_copy_far_rows(dev):
    """Byte offsets past 2^32 in one pool."""
    num = (5 << 30) // 2048
    pool = torch.empty(num, 8, 128, dtype=BF, device="cuda")
    pool[num - 1] = 3.0
    pool[num // 2] = 4.0
    src, dst, st = i32([num - 1, num // 2], "cuda"), i32([0, num - 2], "cuda"), i32([0], "cuda")
    api.kv_pool_copy(desc_of(BF, 8, 8, 128, num), [pool], src, dst, 1, st)
    assert (pool[0] == 3).all() and (pool[num - 2] == 4).all() and int(st.item()) == 0


def fork_case(gen, parents, children, ctx, page, extra=11):
    rng = np.random.default_rng(parents * 7 + children)
    lens = rng.integers(0, ctx + 1, parents)
    rows = [(p, int(lens[p])) for p in range(parents) for _ in range(children)]
    rng.shuffle(rows)
    rows = [(int(p), int(n)) for p, n in rows]
    keep = [n - n % page if rng.random() < 0.7 else int(rng.integers(0, n + 1)) for _, n in rows]
    tails = [n - k for (_, n), k in zip(rows, keep)]
    num = int(lens.sum() + sum(tails) + extra)
    ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((parents, ctx + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for p, n in enumerate(lens):
        table[p, :n] = ids[at:at + n]
        at += n
    return rows, keep, tails, num, table, ids[at:at + max(sum(tails), 1)].contiguous()


@gpu
@pytest.mark.parametrize("dt,hkv,d,pools", [(BF, 2, 64, 2), (BF, 8, 128, 4), (F, 3, 128, 1), (BF, 1, 64, 0)])
@pytest.mark.parametrize("parents,children,ctx,page", [(1, 1, 5, 4), (3, 4, 70, 16), (40, 3, 50, 16), (2, 600, 20, 8), (2, 2, 2600, 64)])
def test_fork(dev, dt, hkv, d, pools, parents, children, ctx, page):
    gen = torch.Generator("cuda").manual_seed(ctx)
    rows, keep, tails, num, table, tail_slots = fork_case(gen, parents, children, ctx, page)
    x, lst = some_pools(gen, pools, num, hkv, d, dt) if pools else (torch.zeros(1), [])
    want = x.clone()
    out, st = torch.full((len(rows), ctx + 5), 99, dtype=torch.int32, device="cuda"), i32([0], "cuda")
    api.kv_pool_fork(desc_of(dt, hkv, hkv, d, num), lst, i32([p for p, _ in rows], "cuda"), i32(keep, "cuda"),
                     i32([n for _, n in rows], "cuda"), indptr(tails, "cuda"), tail_slots, table, out, sum(tails), st)
    at, T, tl, got = 0, table.tolist(), tail_slots.tolist(), out.tolist()
    src, dst = [], []
    for f, (p, n) in enumerate(rows):
        tail = tl[at:at + tails[f]]
        assert got[f] == T[p][:keep[f]] + tail + [-1] * (ctx + 5 - n)
        src += T[p][keep[f]:n]
        dst += tail
        at += tails[f]
    if pools:
        want[:, dst] = want[:, src].clone()
        assert torch.equal(x, want)
    assert int(st.item()) == 0


@gpu
def test_fork_bad_rows(dev):
    gen = torch.Generator("cuda").manual_seed(2)
    x, lst = some_pools(gen, 2, 64, 2, 64, BF)
    table = torch.arange(20, dtype=torch.int32, device="cuda").reshape(2, 10)
    tails = torch.arange(40, 60, dtype=torch.int32, device="cuda")
    # rows: a good one, a parent too high, keep past the length, a length past the table, a tail list too long, a good one
    par, keep, lens = [1, 2, 0, 0, 0, 0], [7, 1, 6, 4, 8, 9], [9, 3, 5, 11, 10, 10]
    ti = torch.tensor([0, 2, 4, 4, 11, 12, 13], device="cuda")
    out, st, want = torch.empty(6, 12, dtype=torch.int32, device="cuda"), i32([0], "cuda"), x.clone()
    api.kv_pool_fork(desc_of(BF, 2, 2, 64, 64), lst, i32(par, "cuda"), i32(keep, "cuda"), i32(lens, "cuda"), ti, tails, table, out, 13, st)
    assert int(st.item()) == api.RX_DEV_BAD_LENGTH
    assert out[0].tolist() == list(range(10, 17)) + [40, 41] + [-1] * 3
    assert (out[1:5] == -1).all()
    assert out[5].tolist() == list(range(9)) + [52] + [-1] * 2
    want[:, [40, 41, 52]] = x[:, [17, 18, 9]]
    assert torch.equal(x, want)
    # a slot outside the pool, in the parent's row and in the tail
    st.zero_()
    table[0, 9], tails[0] = 64, -1
    want = x.clone()
    api.kv_pool_fork(desc_of(BF, 2, 2, 64, 64), lst, i32([0, 1], "cuda"), i32([9, 9], "cuda"), i32([10, 10], "cuda"),
                     torch.tensor([0, 1, 2], device="cuda"), tails, table, out[:2].contiguous(), 2, st)
    want[:, 41] = x[:, 19]
    assert int(st.item()) == api.RX_DEV_BAD_SLOT and torch.equal(x, want)


@gpu
@pytest.mark.parametrize("rows", [5, 70, 2000])
def test_fork_offsets_that_decrease(dev, rows):
    """Offsets that fall back at bad rows: every good row has its table and its copies all the same, and tail
    tokens of bad rows and behind the last are left alone."""
    gen = torch.Generator("cuda").manual_seed(rows)
    rng = np.random.default_rng(rows)
    tail_of = [int(x) for x in rng.integers(0, 4, rows)]
    bad = sorted({3, *(int(x) for x in rng.integers(1, rows - 1, rows // 20))})
    ti, at = [0], 0
    for f in range(rows):                                  # a bad row's end is anywhere, the next good one goes on behind it
        ti.append(at + tail_of[f])
        at = ti[-1]
    for f in bad:
        ti[f + 1] = int(rng.integers(-3, ti[f] + 1)) if f != 3 else 0
    # the row after a bad one starts at the offset that is out of place: it is bad too unless that happens to fit
    keep = [int(x) for x in rng.integers(0, 5, rows)]
    lens = [k + t for k, t in zip(keep, tail_of)]
    par = [f % 2 for f in range(rows)]
    total, num = at + 7, at + 7 + 40
    good = [ti[f] >= 0 and ti[f + 1] <= total and ti[f + 1] - ti[f] == tail_of[f] for f in range(rows)]
    owner = {}
    for f in range(rows):
        for i in range(ti[f], ti[f + 1]) if good[f] else ():
            assert i not in owner                          # the case names each slot once
            owner[i] = f
    assert not all(good) and any(a > b for a, b in zip(ti, ti[1:]))
    x, lst = some_pools(gen, 3, num, 2, 64, BF)
    table = torch.arange(20, dtype=torch.int32, device="cuda").reshape(2, 10)
    tails = torch.arange(40, 40 + total, dtype=torch.int32, device="cuda")
    out, st, want = torch.full((rows, 11), 99, dtype=torch.int32, device="cuda"), i32([0], "cuda"), x.clone()
    api.kv_pool_fork(desc_of(BF, 2, 2, 64, num), lst, i32(par, "cuda"), i32(keep, "cuda"), i32(lens, "cuda"), torch.tensor(ti, device="cuda"), tails,
                     table, out, total, st)
    assert int(st.item()) == api.RX_DEV_BAD_LENGTH
    for f, row in enumerate(out.tolist()):
        mine = [10 * par[f] + j for j in range(keep[f])] + [40 + i for i in range(ti[f], ti[f + 1])] if good[f] else []
        assert row == mine + [-1] * (11 - len(mine)), f
    for i, f in owner.items():
        want[:, 40 + i] = x[:, 10 * par[f] + keep[f] + i - ti[f]]
    assert torch.equal(x, want)


# ============================================================================ kv_pool_write_rope
def rope_case(gen, dt, hq, hkv, d, new, pre, axes_pos, slots_extra=9, wide=1):
    T, P = sum(new), sum(pre)
    ids = torch.randperm(T + P + slots_extra, generator=gen, device="cuda").to(torch.int32)
    x = torch.randn(T, hq + 2 * hkv + wide, d, generator=gen, device="cuda").to(dt)
    return dict(q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:hq + 2 * hkv], x=x, num=T + P + slots_extra,
                ps=ids[:P].contiguous(), ns=ids[P:P + T].contiguous(), pi=indptr(pre, "cuda"), qi=indptr(new, "cuda"),
                pos=axes_pos.to(torch.int32).contiguous())


@gpu
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("hq,hkv,d,sections,cyclic,inter", [
    (4, 4, 64, [32], False, False), (4, 4, 64, [32], False, True), (8, 2, 128, [16, 24, 24], False, False),
    (8, 2, 128, [24, 20, 20], True, False), (7, 1, 128, [12, 11, 5, 4], True, True), (3, 1, 64, [3, 0, 5], False, False),
    (5, 5, 128, [32], False, False), (1, 1, 64, [0, 8], True, True)])
@pytest.mark.parametrize("new,pre", [([1], [0]), ([1] * 70, [3] * 70), ([0, 5, 1, 0, 33], [2, 0, 1100, 7, 0]), ([1300], [9])])
def test_rope_write(dev, dt, hq, hkv, d, sections, cyclic, inter, new, pre):
    gen = torch.Generator("cuda").manual_seed(len(new) + d)
    T = sum(new)
    far = torch.tensor([0, 5, -100000, 2 ** 31 - 3000])[:len(sections), None].cuda()
    pos = torch.randint(0, 3000, (len(sections), T + 5), generator=gen, device="cuda") + far
    c = rope_case(gen, dt, hq, hkv, d, new, pre, pos)
    desc = desc_of(dt, hq, hkv, d, c["num"])
    rope = api.rope_desc(sections, 10000.0, cyclic=cyclic, interleaved=inter)
    kp, vp = (torch.full((c["num"], hkv, d), 7.5, dtype=dt, device="cuda") for _ in range(2))
    qo, ko = torch.empty(T, hq, d, dtype=dt, device="cuda"), torch.empty(T, hkv, d, dtype=dt, device="cuda")
    stride = max(a + b for a, b in zip(new, pre)) + 3
    r2t, st = torch.full((len(new), stride), 99, dtype=torch.int32, device="cuda"), i32([0], "cuda")
    keep = c["x"].clone()
    api.kv_pool_write_rope(desc, rope, len(new), c["ps"], c["pi"], c["ns"], c["qi"], c["pos"], c["q"], c["k"], c["v"], qo, ko, kp,
                           vp, r2t, T, st)
    assert int(st.item()) == 0 and torch.equal(c["x"], keep)
    half = sum(sections)
    freq = 10000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / (2 * half))
    for got, src in ((qo, c["q"]), (ko, c["k"])):
        want, tol = rotate(src, c["pos"][:, :T], sections, freq, cyclic, inter)
        close(got, want, tol)
    at = c["ns"].long()
    assert torch.equal(kp[at], ko) and torch.equal(vp[at], c["v"])
    other = torch.ones(c["num"], dtype=torch.bool, device="cuda")
    other[at] = False
    assert (kp[other] == 7.5).all() and (vp[other] == 7.5).all()
    p0, q0 = np.cumsum([0] + pre), np.cumsum([0] + new)
    for b in range(len(new)):
        row = torch.cat([c["ps"][p0[b]:p0[b + 1]], c["ns"][q0[b]:q0[b + 1]]]).tolist()
        assert r2t[b].tolist() == row + [-1] * (stride - len(row))
    # the table and values are kv_pool_write's
    k2, v2, t2 = torch.empty_like(kp), torch.empty_like(vp), torch.empty_like(r2t)
    api.kv_pool_write(desc, len(new), c["ps"] if c["ps"].numel() else None, c["pi"], c["ns"], c["qi"], ko, c["v"].contiguous(), k2,
                      v2, t2, T, st)
    assert torch.equal(t2, r2t) and torch.equal(k2[at], kp[at]) and torch.equal(v2[at], vp[at]) and int(st.item()) == 0


@gpu
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("T", [5, 2000])
def test_rope_in_place_alone_and_padded(dev, dt, T):
    """In place in the projection's rows, without pool and table; rows outside the batch stay; own
    frequencies."""
    gen = torch.Generator("cuda").manual_seed(T)
    hq, hkv, d, a, z = 6, 2, 64, 2, 1
    pos = torch.randint(0, 1 << 20, (1, T), generator=gen, device="cuda")
    c = rope_case(gen, dt, hq, hkv, d, [T], [0], pos)
    freq = torch.rand(16, generator=gen, device="cuda", dtype=torch.float64) * 40 - 20
    rope = api.rope_desc(16, inv_freq=freq.cpu().numpy())
    desc, st, before = desc_of(dt, hq, hkv, d, c["num"]), i32([0], "cuda"), c["x"].clone()
    qi = torch.tensor([a, a, T - z], device="cuda")
    args = (desc, rope, 2, None, None, None, qi, c["pos"])
    api.kv_pool_write_rope(*args, c["q"], c["k"], None, c["q"], c["k"], None, None, None, T, st)
    for name, lo, h in (("q", 0, hq), ("k", hq, hkv)):
        src = before[:, lo:lo + h]
        want, tol = rotate(src, c["pos"], [16], freq)
        close(c[name][a:T - z], want[a:T - z], tol[a:T - z], name)
        assert torch.equal(c[name][:a], src[:a]) and torch.equal(c[name][T - z:], src[T - z:])
    assert torch.equal(c["x"][:, hq + hkv:], before[:, hq + hkv:]) and int(st.item()) == 0
    # keys only, into the pool; the queries left to someone else
    kp, vp = (torch.zeros(c["num"], hkv, d, dtype=dt, device="cuda") for _ in range(2))
    api.kv_pool_write_rope(desc, rope, 2, None, None, c["ns"], qi, c["pos"], None, before[:, hq:hq + hkv], c["v"], None, None, kp, vp,
                           None, T, st)
    at = c["ns"][a:T - z].long()
    assert torch.equal(kp[at], c["k"][a:T - z]) and torch.equal(vp[at], c["v"][a:T - z]) and int(st.item()) == 0
    assert kp.abs().sum(dim=(1, 2)).ne(0).sum() == T - z - a


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("scale", [2.0 ** -54, 2.0 ** -40, 1e-6, 0.3, 50.0])
def test_rope_negative_frequencies(dev, dt, scale):
    """Each frequency and its negative at positions next to both ends of 32 bits: the angle's stated error,
    2^-52 of it and 2^-25 turn, in either sign.  Rows of ones and zeros show cosine and sine alone: to the
    angle's error come the sine's or cosine's own (2 EPS32 of a value up to 1, and the rounding to the type)."""
    freq = np.array([-0.99, 0.99, -0.5, 0.5, -1.51, 1.51, -1.0, 1.0]) * 2 * math.pi * scale
    pos = torch.tensor([[2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, -2 ** 31 + 1, 1 << 30, 12345, -1, 0]], dtype=torch.int32, device="cuda")
    n = pos.shape[1]
    k = torch.zeros(n, 1, 64, dtype=dt, device="cuda")
    k[:, :, :8] = 1
    out, st = torch.empty_like(k), i32([0], "cuda")
    api.kv_pool_write_rope(desc_of(dt, 1, 1, 64), api.rope_desc(8, inv_freq=freq), 1, None, None, None, torch.tensor([0, n], device="cuda"),
                           pos, None, k, None, None, out, None, None, None, n, st)
    ang = pos[0].double()[:, None] * torch.tensor(freq, device="cuda")
    half = 2.0 ** -8 if dt == BF else 2.0 ** -24
    tol = 2 * math.pi * 2.0 ** -25 + ang.abs() * 2.0 ** -50        # 2^-52 here, and the product's and the frequency's there
    for got, want in ((out[:, 0, :8].double(), ang.cos()), (out[:, 0, 8:16].double(), ang.sin())):
        assert ((got - want).abs() <= tol + want.abs() * (half + 2 * 2.0 ** -24) + 1e-40).all()
    assert int(st.item()) == 0


@gpu
def test_rope_bad_slots_and_lengths(dev):
    gen = torch.Generator("cuda").manual_seed(8)
    c = rope_case(gen, BF, 2, 2, 64, [40], [0], torch.arange(40, device="cuda")[None])
    desc, rope = desc_of(BF, 2, 2, 64, c["num"]), api.rope_desc(32)
    kp, vp = (torch.full((c["num"], 2, 64), 7.5, dtype=BF, device="cuda") for _ in range(2))
    ns = c["ns"].clone()
    ns[3], ns[17] = -1, c["num"]
    qo, st = torch.empty(40, 2, 64, dtype=BF, device="cuda"), i32([0], "cuda")
    r2t = torch.empty(1, 40, dtype=torch.int32, device="cuda")
    api.kv_pool_write_rope(desc, rope, 1, None, c["pi"], ns, c["qi"], c["pos"], c["q"], c["k"], c["v"], qo, None, kp, vp, r2t, 40, st)
    assert int(st.item()) == api.RX_DEV_BAD_SLOT
    assert r2t[0, 3] == r2t[0, 17] == -1
    assert (kp != 7.5).any(dim=2).any(dim=1).sum() == 38
    st.zero_()
    for table in (r2t, None):
        api.kv_pool_write_rope(desc, rope, 1, None, c["pi"], c["ns"], torch.tensor([0, 41], device="cuda"), c["pos"], c["q"], c["k"],
                               c["v"], qo, None, kp, vp, table, 40, st)
        assert int(st.item()) == api.RX_DEV_BAD_LENGTH
        st.zero_()


@gpu
@pytest.mark.parametrize("table", [True, False])
@pytest.mark.parametrize("ends", [(0, -1), (0, -2 ** 32 + 1000), (5, -2 ** 32 + 2 ** 20), (0, -2 ** 62), (20, 3), (-2 ** 40, -2 ** 32 + 30),
                                  (2 ** 63 - 2, -2 ** 63 + 1)])
def test_rope_boundaries_far_below_zero(dev, table, ends):
    """Boundaries that 32 bits would take for others, or whose sums wrap: reported, and no row, slot or table
    entry of the bad request is touched."""
    gen = torch.Generator("cuda").manual_seed(14)
    c = rope_case(gen, BF, 2, 2, 64, [40], [0], torch.arange(40, device="cuda")[None])
    kp, vp = (torch.full((c["num"], 2, 64), 7.5, dtype=BF, device="cuda") for _ in range(2))
    qo, ko = (torch.full((40, 2, 64), 7.5, dtype=BF, device="cuda") for _ in range(2))
    r2t, st = torch.full((1, 48), 99, dtype=torch.int32, device="cuda"), i32([0], "cuda")
    api.kv_pool_write_rope(desc_of(BF, 2, 2, 64, c["num"]), api.rope_desc(32), 1, c["ps"], c["pi"], c["ns"],
                           torch.tensor(ends, dtype=torch.int64, device="cuda"), c["pos"], c["q"], c["k"], c["v"], qo, ko, kp, vp,
                           r2t if table else None, 40, st)
    assert int(st.item()) == api.RX_DEV_BAD_LENGTH
    for x in (kp, vp, qo, ko):
        assert (x == 7.5).all()
    assert (r2t == (-1 if table else 99)).all()


@gpu
def test_rope_without_a_prefix_list(dev):
    """No list of matched slots: fine for requests without any, a bad length for the others."""
    gen = torch.Generator("cuda").manual_seed(12)
    c = rope_case(gen, BF, 2, 2, 64, [4, 3, 5], [0, 0, 0], torch.arange(12, device="cuda")[None])
    kp, vp = (torch.zeros(c["num"], 2, 64, dtype=BF, device="cuda") for _ in range(2))
    for pi, want in (([0, 0, 0, 0], api.RX_DEV_OK), ([0, 0, 2, 2], api.RX_DEV_BAD_LENGTH)):
        r2t, st = torch.empty(3, 9, dtype=torch.int32, device="cuda"), i32([0], "cuda")
        api.kv_pool_write_rope(desc_of(BF, 2, 2, 64, c["num"]), api.rope_desc(32), 3, None, torch.tensor(pi, device="cuda"), c["ns"],
                               c["qi"], c["pos"], None, c["k"], c["v"], None, None, kp, vp, r2t, 12, st)
        ns = c["ns"].tolist()
        mid = ns[4:7] + [-1] * 6 if want == api.RX_DEV_OK else [-1] * 9
        assert int(st.item()) == want and r2t.tolist() == [ns[:4] + [-1] * 5, mid, ns[7:] + [-1] * 4]


@gpu
@pytest.mark.parametrize("native", [True, False])
def test_binding_refuses(dev, native, monkeypatch):
    """The same refusals from the extension and from the Python code that stands in for it."""
    if not native:
        monkeypatch.setattr(api, "_ops_ext", False)
    d, st = desc_of(BF, 4, 2, 64, 10), i32([0], "cuda")
    q, k = torch.zeros(8, 4, 64, dtype=BF, device="cuda"), torch.zeros(8, 2, 64, dtype=BF, device="cuda")
    ip = torch.tensor([0, 8], device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:7]), dict(k=q), dict(out=q.transpose(0, 1)), dict(ip=ip.int()), dict(ip=ip[:1]),
                dict(lse=torch.zeros(7, 4, device="cuda")), dict(q=q.cpu()), dict(st=st.long())):
        a = dict(dict(q=q, k=k, out=torch.empty_like(q), ip=ip, lse=None, st=st), **bad)
        with pytest.raises(ValueError):
            api.prompt_attention(d, 1, a["q"], a["k"], k, a["ip"], a["out"], a["lse"], 8, a["st"])
    with pytest.raises(ValueError):
        api.kv_pool_copy(d, [k], i32([1], "cuda"), i32([2], "cuda"), 1, st)      # not num_slots rows
    pool = torch.zeros(10, 2, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        api.kv_pool_copy(d, [pool], i32([1, 2], "cuda"), i32([2], "cuda"), 1, st)
    with pytest.raises(ValueError):
        api.kv_pool_write_rope(d, api.rope_desc(32), 1, None, None, None, ip, torch.zeros(2, 8, dtype=torch.int32, device="cuda"), q, k,
                               None, q, k, None, None, None, 8, st)


@gpu
@pytest.mark.parametrize("native", [True, False])
def test_binding_refuses_other_types_and_places(dev, native, monkeypatch):
    """Types of the same size as the right ones, and buffers on the host."""
    if not native:
        monkeypatch.setattr(api, "_ops_ext", False)
    d, st, ip = desc_of(BF, 4, 2, 64, 10), i32([0], "cuda"), torch.tensor([0, 8], device="cuda")
    q, k = torch.zeros(8, 4, 64, dtype=BF, device="cuda"), torch.zeros(8, 2, 64, dtype=BF, device="cuda")
    lse = torch.zeros(8, 4, device="cuda")
    for bad in (dict(q=q.half()), dict(out=q.half()), dict(lse=lse.cpu()), dict(lse=lse.int()), dict(ip=ip.double()), dict(st=st.float())):
        a = dict(dict(q=q, out=torch.empty_like(q), ip=ip, lse=lse, st=st), **bad)
        with pytest.raises(ValueError):
            api.prompt_attention(d, 1, a["q"], k, k, a["ip"], a["out"], a["lse"], 8, a["st"])
    pool, one = torch.zeros(10, 2, 64, dtype=BF, device="cuda"), i32([1], "cuda")
    for bad in (pool.half(), pool.cpu(), pool.short(), pool.transpose(0, 1)):
        with pytest.raises(ValueError):
            api.kv_pool_copy(d, [pool, bad], one, one, 1, st)
    for bad in (one, one.cpu()[None], one.float()[None]):
        with pytest.raises(ValueError):
            api.kv_pool_fork(d, [pool], one, one, one, ip, one, one[None], bad, 0, st)


@gpu
@pytest.mark.parametrize("native", [True, False])
def test_binding_refuses_pools_of_another_size(dev, native, monkeypatch):
    """A rotary write's pools have the descriptor's slots, no fewer and no more, as those of the row movers."""
    if not native:
        monkeypatch.setattr(api, "_ops_ext", False)
    d, st, ip = desc_of(BF, 4, 2, 64, 10), i32([0], "cuda"), torch.tensor([0, 1], device="cuda")
    k, pos, slot = torch.ones(1, 2, 64, dtype=BF, device="cuda"), i32([[0]], "cuda"), i32([4], "cuda")
    pool = [torch.zeros(n, 2, 64, dtype=BF, device="cuda") for n in (10, 9, 11)]

    def write(kp, vp, slots=slot):
        api.kv_pool_write_rope(d, api.rope_desc(32), 1, None, None, slots, ip, pos, None, k, k, None, None if slots is not None else k.clone(),
                               kp, vp, None, 1, st)
    for kp, vp in ((pool[1], pool[0]), (pool[2], pool[0]), (pool[0], pool[2]), (pool[0], None), (pool[0].float(), pool[0])):
        with pytest.raises(ValueError):
            write(kp, vp)
    write(pool[1], None, slots=None)                       # no pool is written: none is looked at
    write(pool[0], pool[0].clone())
    assert int(st.item()) == 0 and pool[0].ne(0).any(dim=2).any(dim=1).nonzero().flatten().tolist() == [4]


@gpu
def test_binding_in_python_makes_the_same_calls(dev, monkeypatch):
    """Every operator through the extension and through the Python code: the same results."""
    gen = torch.Generator("cuda").manual_seed(11)
    c = rope_case(gen, BF, 4, 2, 64, [30, 50], [3, 0], torch.arange(80, device="cuda")[None])
    desc, rope, st = desc_of(BF, 4, 2, 64, c["num"]), api.rope_desc(32), i32([0], "cuda")
    stream, results = torch.cuda.Stream(), []
    for ext in (None, False):
        monkeypatch.setattr(api, "_ops_ext", ext)
        x, lst = some_pools(torch.Generator("cuda").manual_seed(12), 2, c["num"], 2, 64, BF)
        qo, ko, r2t = torch.empty(80, 4, 64, dtype=BF, device="cuda"), torch.empty(80, 2, 64, dtype=BF, device="cuda"), i32([[0] * 56] * 2, "cuda")
        out, lse, fork = torch.empty_like(qo), torch.empty(80, 4, device="cuda"), i32([[0] * 60] * 2, "cuda")
        torch.cuda.synchronize()
        for s in (None, stream, stream.cuda_stream):
            api.kv_pool_write_rope(desc, rope, 2, c["ps"], c["pi"], c["ns"], c["qi"], c["pos"], c["q"], c["k"], c["v"], qo, ko, *lst, r2t, 80,
                                   st, stream=s)
            api.kv_pool_write_rope(desc, rope, 2, c["ps"].data_ptr(), c["pi"].data_ptr(), c["ns"], c["qi"], c["pos"], c["q"], c["k"], c["v"],
                                   qo, ko, *lst, r2t.data_ptr(), 80, st, stream=s, r2t_stride=56)
            api.prompt_attention(desc, 2, qo, ko, c["v"], c["qi"], out, lse, 80, st, stream=s)
            api.kv_pool_copy(desc, lst, c["ps"], c["ns"][:3].contiguous(), 1, st, stream=s)
            api.kv_pool_fork(desc, lst, i32([1, 0], "cuda"), i32([40, 33], "cuda"), i32([50, 33], "cuda"), indptr([10, 0], "cuda"), c["ns"][:10].contiguous(),
                             r2t, fork, 10, st, stream=s)
            torch.cuda.synchronize()
        results.append((x, qo, ko, r2t, out, lse, fork))
    assert int(st.item()) == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ============================================================================ prompt_attention
def rows_of(gen, T, hq, hkv, d, dt, wide=0):
    """q, k, v as parts of one projection's rows (wide more columns than needed between them)."""
    x = torch.randn(T, hq + 2 * hkv + wide, d, generator=gen, device="cuda").to(dt)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]


def run_prompt(q, k, v, lens, desc, start=0, total=None, lse=True):
    total = q.shape[0] if total is None else total
    out = torch.full((q.shape[0], desc.hq, desc.head_dim), 7.5, dtype=q.dtype, device="cuda")
    L = torch.full((q.shape[0], desc.hq), 7.5, device="cuda") if lse else None
    st = i32([0], "cuda")
    api.prompt_attention(desc, len(lens), q, k, v, indptr(lens, "cuda", start), out, L, total, st)
    torch.cuda.synchronize()
    return out, L, int(st.item())


def check_prompt(q, k, v, lens, desc, start=0):
    out, lse, st = run_prompt(q, k, v, lens, desc, start)
    assert st == 0
    want, wl, to, tl = attention(q, k, v, lens, desc.scale, start)
    a, b = start, start + sum(lens)
    close(out[a:b], want[a:b], to[a:b], "out")
    close(lse[a:b], wl[a:b], tl[a:b], "lse")
    assert (out[:a] == 7.5).all() and (out[b:] == 7.5).all() and (lse[:a] == 7.5).all() and (lse[b:] == 7.5).all()
    return out, lse


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 1, 128), (6, 2, 128), (14, 2, 64), (1, 1, 128), (16, 2, 128)])
def test_prompt_lengths(dev, dt, hq, hkv, d):
    gen = torch.Generator("cuda").manual_seed(hq * 100 + d)
    for lens in ([1], [0, 1, 2, 0], [127, 128, 129], [255, 1, 256, 257], [33, 0, 300, 64, 65], [700]):
        q, k, v = rows_of(gen, sum(lens), hq, hkv, d, dt, wide=3)
        check_prompt(q, k, v, lens, desc_of(dt, hq, hkv, d))


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("hq,hkv", [(71, 1), (128, 1), (150, 1), (130, 2), (260, 2)])
def test_prompt_many_heads_per_kv_head(dev, dt, hq, hkv):
    """Up to and past the 128 rows of a tile."""
    gen = torch.Generator("cuda").manual_seed(hq)
    lens = [3, 130, 1]
    q, k, v = rows_of(gen, sum(lens), hq, hkv, 64, dt)
    check_prompt(q, k, v, lens, desc_of(dt, hq, hkv, 64))


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_many_sequences(dev, dt):
    """Enough items that a block takes several, and more sequences than a warp looks at at once."""
    gen = torch.Generator("cuda").manual_seed(5)
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 60, 400)] + [513] + [int(x) for x in rng.integers(0, 3, 800)]
    q, k, v = rows_of(gen, sum(lens), 4, 2, 64, dt)
    check_prompt(q, k, v, lens, desc_of(dt, 4, 2, 64))


@gpu
@pytest.mark.parametrize("dt,hq,hkv,d,n", [(F, 4, 4, 128, 2500), (BF, 8, 2, 128, 6000), (BF, 12, 12, 64, 3001), (BF, 64, 8, 128, 2100)])
def test_prompt_long(dev, dt, hq, hkv, d, n):
    gen = torch.Generator("cuda").manual_seed(n)
    q, k, v = rows_of(gen, n, hq, hkv, d, dt)
    check_prompt(q, k, v, [n], desc_of(dt, hq, hkv, d))


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("lens", [[2100, 1, 0, 1437, 640, 900], [700] * 9, [5120]])
@pytest.mark.parametrize("bad", [0.0, math.inf, math.nan])
def test_prompt_many_long_items(dev, dt, lens, bad):
    """Calls of more items than run at once, whose sequences are long (f32 then takes larger register tiles),
    with values that are not finite here and there, rows in front and behind, and one scale of zero."""
    gen = torch.Generator("cuda").manual_seed(len(lens))
    n = sum(lens)
    q, k, v = rows_of(gen, n + 70, 16, 4, 64, dt, wide=1)
    for x in (q, k, v):
        x[:30] = math.nan
        x[30 + n:] = math.nan
    if bad:
        for at in (0, 63, 64, 699, 701, n // 2, n - 1):
            v[30 + at, at % 4, at % 64] = bad
    check_prompt(q, k, v, lens, desc_of(dt, 16, 4, 64, scale=None if bad or len(lens) > 1 else 0.0), start=30)


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("hq,hkv,d,lens", [(12, 12, 64, [2500]), (16, 2, 128, [1300, 1, 0, 850]), (14, 2, 64, [640, 1700, 129]),
                                           (4, 4, 128, [5000]), (8, 8, 128, [1025, 2047])])
@pytest.mark.parametrize("bad", [0.0, math.inf, math.nan])
def test_prompt_one_or_two_items_an_sm(dev, dt, hq, hkv, d, lens, bad):
    """Calls of a few items an SM, long ones and short ones among them, whose blocks take more than one."""
    gen = torch.Generator("cuda").manual_seed(hq)
    n = sum(lens)
    q, k, v = rows_of(gen, n + 5, hq, hkv, d, dt)
    for x in (q, k, v):
        x[n:] = math.nan
    if bad:
        for at in (0, 127, 128, n // 3, n - 1):
            v[at, at % hkv, at % d] = bad
    check_prompt(q, k, v, lens, desc_of(dt, hq, hkv, d))


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_leaves_other_rows(dev, dt):
    """Rows before the first and behind the last sequence, NaN inside: neither read nor written."""
    gen = torch.Generator("cuda").manual_seed(1)
    lens = [200, 57]
    q, k, v = rows_of(gen, 400, 4, 2, 128, dt)
    for x in (q, k, v):
        x[:70] = math.nan
        x[70 + 257:] = math.nan
    check_prompt(q, k, v, lens, desc_of(dt, 4, 2, 128), start=70)


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (8, 2, 64), (6, 2, 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prompt_non_finite_values_stay_in_their_place(dev, dt, hq, hkv, d, bad):
    """A non-finite value reaches the rows of its sequence from its own on; a non-finite key's row is
    hidden from earlier rows and other sequences as well."""
    gen = torch.Generator("cuda").manual_seed(2)
    lens = [150, 301, 90]
    q, k, v = rows_of(gen, sum(lens), hq, hkv, d, dt)
    for at in (40, 149, 150 + 200, 150 + 255, 150 + 300, 451):
        v[at, (at % hkv), at % d] = bad
    v[451, 0, 3] = math.nan
    check_prompt(q, k, v, lens, desc_of(dt, hq, hkv, d))
    k[150 + 280:150 + 301] = math.nan             # the tail of the second sequence: those rows are NaN
    out, lse, st = run_prompt(q, k, v, lens, desc_of(dt, hq, hkv, d))
    want, wl, to, tl = attention(q, k, v, lens, desc_of(dt, hq, hkv, d).scale)
    rows = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    rows[150 + 280:150 + 301] = False
    close(out[rows], want[rows], to[rows], "out")
    close(lse[rows], wl[rows], tl[rows], "lse")
    assert torch.isnan(out[~rows].float()).all() and torch.isnan(lse[~rows]).all()


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_prompt_non_finite_values_of_vanishing_weight(dev, dt, d, bad):
    """A value that is not finite under a score so low that its probability is 0 in 32 bits, in tiles that the
    mask cuts for some rows and not for others: that channel of the rows that attend it is not finite
    (which of infinity and NaN is left open), and everything else is as if the value were finite."""
    gen = torch.Generator("cuda").manual_seed(15)
    n = 600
    for at in (3, 200, 300, 599):
        q, k, v = (x.contiguous() for x in rows_of(gen, n, 2, 1, d, dt))
        q = q.abs() + 0.5
        k[at] = -1000.0                                     # scores of -500 sqrt(d) and below, beside others of a few
        desc = desc_of(dt, 2, 1, d)
        clean, _, st = run_prompt(q, k, v, [n], desc)
        want, wl, to, tl = attention(q, k, v, [n], desc.scale)
        assert st == 0
        close(clean, want, to, "clean")
        v[at, 0, 5] = bad
        out, lse, st = run_prompt(q, k, v, [n], desc)
        close(lse, wl, tl, "lse")
        rest = torch.ones_like(out, dtype=torch.bool)
        rest[at:, :, 5] = False
        assert st == 0 and torch.equal(out[rest], clean[rest])
        assert not torch.isfinite(out[at:, :, 5].float()).any()


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_growing_and_extreme_scores(dev, dt):
    """Scores whose maximum keeps growing (the running maximum moves at every tile), one that falls,
    the type's lowest values as keys, and a scale of zero."""
    gen = torch.Generator("cuda").manual_seed(3)
    n, d = 700, 64
    q, k, v = (x.contiguous() for x in rows_of(gen, n, 2, 1, d, dt))
    ramp = torch.linspace(0.1, 6, n, device="cuda")[:, None, None]
    q0 = q[:1].expand_as(q).contiguous()
    for kk in (q0[:, :1] * ramp, q0[:, :1] * ramp.flip(0)):
        check_prompt(q0, kk.to(dt).contiguous(), v, [n], desc_of(dt, 2, 1, d))
    check_prompt(q, k, v, [n], desc_of(dt, 2, 1, d, scale=0.0))
    low = torch.full_like(k, torch.finfo(dt).min)
    low[0] = 0
    pos = q.abs() + 0.1
    out, lse, st = run_prompt(pos, low, v, [n], desc_of(dt, 2, 1, d))
    assert torch.equal(out, v[:1].expand(n, 2, d))        # every later key underflows: row 0's value exactly
    assert (lse == 0).all()


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("hq,hkv,d,lens", [(2, 2, 64, [300]), (4, 1, 128, [1, 70, 0, 2, 129]), (16, 4, 64, [700] * 9)])
@pytest.mark.parametrize("scale", [0.0, 1e-39, 2.0 ** -126])
def test_prompt_scale_of_nearly_nothing(dev, dt, hq, hkv, d, lens, scale):
    """Products of up to 1e37 by a scale of zero are zero: each row is the mean of the values up to it; and
    scales near and below the least normal number."""
    gen = torch.Generator("cuda").manual_seed(d)
    q, k, v = rows_of(gen, sum(lens), hq, hkv, d, F)
    if scale == 0:
        flushes = torch.set_flush_denormal(True)           # the host's setting does not matter, nor does zero's sign
        try:
            runs = [run_prompt(q.to(dt), k.to(dt), v.to(dt), lens, desc_of(dt, hq, hkv, d, scale=z))[0] for z in (0.0, -0.0)]
        finally:
            torch.set_flush_denormal(False)
        assert torch.isfinite(runs[0].float()).all() and torch.equal(*runs), flushes
    check_prompt((q * 1e18).to(dt), (k * 1e18).to(dt), v.to(dt), lens, desc_of(dt, hq, hkv, d, scale=scale))


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_far_rows(dev, dt):
    """Element offsets past 2^32: 5000 rows, a million elements apart."""
    n, gap = 5000, 1 << 20
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    big = torch.empty(n * gap, dtype=dt, device="cuda")
    gen = torch.Generator("cuda").manual_seed(4)
    rows = big.as_strided((n, 4, 64), (gap, 64, 1))
    rows[-300:] = torch.randn(300, 4, 64, generator=gen, device="cuda").to(dt)
    q, k, v = rows[:, :2], rows[:, 2:3], rows[:, 3:4]
    out = torch.full((n, 2, 64), 7.5, dtype=dt, device="cuda")
    st = i32([0], "cuda")
    desc = desc_of(dt, 2, 1, 64)
    api.prompt_attention(desc, 2, q, k, v, indptr([100, 200], "cuda", n - 300), out, None, n, st)
    want, _, to, _ = attention(q[-300:], k[-300:], v[-300:], [100, 200], desc.scale)
    close(out[-300:], want, to)
    wide = big.as_strided((n, 2, 64), (gap, 64, 1), 1024)   # and written that far apart
    api.prompt_attention(desc, 2, q, k, v, indptr([100, 200], "cuda", n - 300), wide, None, n, st)
    assert torch.equal(wide[-300:], out[-300:]) and int(st.item()) == 0


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_bad_boundaries_are_reported_and_skipped(dev, dt):
    gen = torch.Generator("cuda").manual_seed(6)
    q, k, v = rows_of(gen, 300, 4, 2, 64, dt)
    desc = desc_of(dt, 4, 2, 64)
    for ind in ([0, 100, 301], [0, 100, 1 << 40], [-5, 100, 300]):
        out = torch.full((300, 4, 64), 7.5, dtype=dt, device="cuda")
        st = i32([0], "cuda")
        api.prompt_attention(desc, 2, q, k, v, torch.tensor(ind, device="cuda"), out, None, 300, st)
        assert int(st.item()) == api.RX_DEV_BAD_LENGTH
        good = slice(0, 100) if ind[0] == 0 else slice(100, 300)
        want, _, to, _ = attention(q[good], k[good], v[good], [good.stop - good.start], desc.scale)
        close(out[good], want, to)
        rest = torch.ones(300, dtype=torch.bool, device="cuda")
        rest[good] = False
        assert (out[rest] == 7.5).all()


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("hq,ind,total", [(4, [0, 50, 30, 80], 80), (64, [0, 50, 30, 80], 80), (128, [0, 60, 10, 80], 80),
                                          (64, [0, 900, 30, 1000], 1000), (16, [0] * 70 + [90, 80, 100], 100), (128, [0, 300, 250, 300, 300], 300)])
def test_prompt_decreasing_boundaries_are_reported(dev, dt, hq, ind, total):
    """However few tokens a tile holds, and in either order of the items; rows outside every sequence stay."""
    gen = torch.Generator("cuda").manual_seed(9)
    q, k, v = rows_of(gen, total + 40, hq, 1, 64, dt)
    for at in (0, 20):
        out = torch.full((total + 40, hq, 64), 7.5, dtype=dt, device="cuda")
        st = i32([0], "cuda")
        api.prompt_attention(desc_of(dt, hq, 1, 64), len(ind) - 1, q, k, v, torch.tensor(ind, device="cuda") + at, out, None, total + 40, st)
        assert int(st.item()) == api.RX_DEV_BAD_LENGTH
        assert (out[:at] == 7.5).all() and (out[at + total:] == 7.5).all()


@gpu
def test_prompt_too_long_a_sequence_is_reported(dev):
    """One row more than 2^26 (one head, the same rows as q, k and v: 8.6 GB, and as much for the output)."""
    n = (1 << 26) + 1
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    x, out = torch.empty(n + 3, 1, 64, dtype=BF, device="cuda"), torch.empty(n + 3, 1, 64, dtype=BF, device="cuda")
    x[n:] = 1.0
    out[:100], out[n - 100:] = 7.5, 7.5
    st = i32([0], "cuda")
    api.prompt_attention(desc_of(BF, 1, 1, 64), 2, x, x, x, torch.tensor([0, n, n + 3], device="cuda"), out, None, n + 3, st)
    assert int(st.item()) == api.RX_DEV_BAD_LENGTH
    assert (out[:100] == 7.5).all() and (out[n - 100:n] == 7.5).all() and (out[n:] == 1.0).all()


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_small_calls_beside_a_long_one(dev, dt):
    """Small calls on other streams while a long one holds every SM, and as it leaves them one by one: blocks
    take the work of those that have not begun, so that one may have several items of a small call."""
    gen = torch.Generator("cuda").manual_seed(8)
    desc, st = desc_of(dt, 4, 2, 64), i32([0], "cuda")
    small = [rows_of(gen, sum(lens), 4, 2, 64, dt) + (lens, indptr(lens, "cuda")) for lens in ([513], [1, 200, 0, 64, 300], [30] * 20)]
    want = [run_prompt(q, k, v, lens, desc)[0] for q, k, v, lens, _ in small]
    n = 12000 if dt == BF else 5000
    lq, lk, lv = rows_of(gen, n, 16, 2, 64, dt)
    ldesc, lip = desc_of(dt, 16, 2, 64), indptr([n], "cuda")
    long_out = torch.empty(n, 16, 64, dtype=dt, device="cuda")
    streams, outs = [torch.cuda.Stream() for _ in range(5)], []
    torch.cuda.synchronize()
    for r in range(6):
        with torch.cuda.stream(streams[0]):
            api.prompt_attention(ldesc, 1, lq, lk, lv, lip, long_out, None, n, st)
        for i in range(12):
            q, k, v, lens, ip = small[i % 3]
            with torch.cuda.stream(streams[1 + i % 4]):
                o = torch.full((q.shape[0], 4, 64), 7.5, dtype=dt, device="cuda")
                api.prompt_attention(desc, len(lens), q, k, v, ip, o, None, q.shape[0], st)
                outs.append((i % 3, o))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for i, o in outs:
        assert torch.equal(o, want[i])


@gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("n", [90, 2500])
def test_chain_of_calls_without_waits(dev, dt, n):
    """Each operator reads what the one before it wrote, in eager order, and twice as a captured graph:
    turned in place, attended, the pool's rows moved, forked, attended again through the forked table."""
    gen = torch.Generator("cuda").manual_seed(n)
    hq, hkv, d = 4, 2, 64
    c = rope_case(gen, dt, hq, hkv, d, [n], [0], torch.arange(n, device="cuda")[None], slots_extra=2 * n)
    num, T = c["num"], n
    desc, rope, st = desc_of(dt, hq, hkv, d, num), api.rope_desc(32), i32([0], "cuda")
    free = torch.tensor(sorted(set(range(num)) - set(c["ns"].tolist())), dtype=torch.int32, device="cuda")
    dst, tail = free[:n].contiguous(), free[n:2 * n].contiguous()
    x0, x = c["x"], torch.empty_like(c["x"])
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    pools = [torch.empty(num, hkv, d, dtype=dt, device="cuda") for _ in range(2)]
    r2t, moved = torch.empty(1, n, dtype=torch.int32, device="cuda"), dst[None].contiguous()
    fork, out, dec = torch.empty(1, n, dtype=torch.int32, device="cuda"), torch.empty(n, hq, d, dtype=dt, device="cuda"), torch.empty(1, hq, d, dtype=dt, device="cuda")
    zero, kvl, ti = i32([0], "cuda"), i32([n], "cuda"), indptr([n], "cuda")
    ws = torch.empty(max(api.decode_workspace_bytes(desc, 1, n), 256), dtype=torch.uint8, device="cuda")

    def run():
        x.copy_(x0)
        api.kv_pool_write_rope(desc, rope, 1, None, c["pi"], c["ns"], c["qi"], c["pos"], q, k, v, q, k, *pools, r2t, T, st)
        api.prompt_attention(desc, 1, q, k, v, c["qi"], out, None, T, st)
        api.kv_pool_copy(desc, pools, c["ns"], dst, 1, st)
        api.kv_pool_fork(desc, pools, zero, zero, kvl, ti, tail, moved, fork, n, st)
        api.decode_attention(desc, 1, out[n - 1:], fork, kvl, *pools, dec, None, n, ws, st)
        api.kv_pool_write_rope(desc, rope, 1, None, None, None, c["qi"], c["pos"], q, k, None, q, k, None, None, None, T, st)

    def wipe():
        for t in (x, *pools, out, dec):
            t.fill_(math.nan)
        r2t.fill_(-7), fork.fill_(-7)

    def take():
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return [t.clone() for t in (q, k, out, dec, fork, r2t)] + [p[i.long()] for p in pools for i in (c["ns"], dst, tail)]
    wipe()
    run()
    got = take()
    assert torch.equal(got[6], got[7]) and torch.equal(got[6], got[8]) and torch.equal(got[4][0], tail)
    turned = [torch.empty(n, h, d, dtype=dt, device="cuda") for h in (hq, hkv)]
    api.kv_pool_write_rope(desc, rope, 1, None, None, None, c["qi"], c["pos"], x0[:, :hq], x0[:, hq:hq + hkv], None, *turned, None, None,
                           None, T, st)
    torch.cuda.synchronize()
    want, _, to, _ = attention(*turned, v, [n], desc.scale)
    close(out, want, to, "out")
    for r in range(3):
        wipe()
        run()
        for a, b in zip(got, take()):
            assert torch.equal(a, b)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
        run()
    for r in range(3):
        wipe()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
        for a, b in zip(got, take()):
            assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_prompt_streams_and_graphs(dev, dt):
    """Calls on several streams at once, and two graphs captured on one stream and replayed on two,
    give the first call's bits."""
    gen = torch.Generator("cuda").manual_seed(7)
    desc = desc_of(dt, 8, 2, 128)
    sets = []
    for lens in ([900, 300, 77], [64] * 40 + [1500]):
        q, k, v = rows_of(gen, sum(lens), 8, 2, 128, dt)
        out, lse, st = run_prompt(q, k, v, lens, desc)
        assert st == 0
        sets.append((q, k, v, lens, out, indptr(lens, "cuda")))
    st = i32([0], "cuda")
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    torch.cuda.synchronize()
    for r in range(3):
        for i, s in enumerate(streams):
            q, k, v, lens, _, ip = sets[i % 2]
            with torch.cuda.stream(s):
                o = torch.empty_like(sets[i % 2][4])
                api.prompt_attention(desc, len(lens), q, k, v, ip, o, None, q.shape[0], st)
                outs.append((i % 2, o))
    torch.cuda.synchronize()
    for i, o in outs:
        assert torch.equal(o, sets[i][4])
    graphs = []
    for q, k, v, lens, want, ip in sets:
        g, o = torch.cuda.CUDAGraph(), torch.zeros_like(want)
        with torch.cuda.graph(g, stream=streams[0]):
            api.prompt_attention(desc, len(lens), q, k, v, ip, o, None, q.shape[0], st)
        graphs.append((g, o, want))
    for r in range(5):
        for (g, o, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, o, want in graphs:
        assert torch.equal(o, want)
    assert int(st.item()) == 0


@gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_branches_that_fork_and_join(dev, dt):
    """Two streams joined by events, eager and as a graph of two branches: a call that depends on kernels of
    both waits for both, though each call's set-up may begin before the one in front of it has ended."""
    gen = torch.Generator("cuda").manual_seed(13)
    hq, hkv, d, n = 8, 2, 128, 3000
    c = rope_case(gen, dt, hq, hkv, d, [n], [0], torch.arange(n, device="cuda")[None], slots_extra=2 * n)
    desc, rope, st = desc_of(dt, hq, hkv, d, c["num"]), api.rope_desc(64), i32([0], "cuda")
    free = torch.tensor(sorted(set(range(c["num"])) - set(c["ns"].tolist())), dtype=torch.int32, device="cuda")
    one, two = free[:n].contiguous(), free[n:2 * n].contiguous()
    pools = [torch.empty(c["num"], hkv, d, dtype=dt, device="cuda") for _ in range(2)]
    q, k = torch.empty(n, hq, d, dtype=dt, device="cuda"), torch.empty(n, hkv, d, dtype=dt, device="cuda")
    out = torch.empty_like(q)
    fork, zero, kvl, ti = torch.empty(1, n, dtype=torch.int32, device="cuda"), i32([0], "cuda"), i32([n], "cuda"), indptr([n], "cuda")
    moved = one[None].contiguous()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def run():                                              # on stream a
        api.kv_pool_write_rope(desc, rope, 1, None, c["pi"], c["ns"], c["qi"], c["pos"], c["q"], c["k"], c["v"], q, k, *pools, None, n, st)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            api.prompt_attention(desc, 1, q, k, c["v"], c["qi"], out, None, n, st)
        api.kv_pool_copy(desc, pools, c["ns"], one, 1, st)
        a.wait_stream(b)
        # reads what the copy moved, overwrites (in place) what the other branch read
        api.kv_pool_fork(desc, pools, zero, zero, kvl, ti, two, moved, fork, n, st)
        api.kv_pool_write_rope(desc, rope, 1, None, None, None, c["qi"], c["pos"], q, k, None, q, k, None, None, None, n, st)

    def wipe():
        for t in (*pools, q, k, out):
            t.fill_(math.nan)
        torch.cuda.synchronize()

    def take():
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return [t.clone() for t in (q, k, out, fork)] + [p[i.long()] for p in pools for i in (c["ns"], one, two)]
    wipe()
    with torch.cuda.stream(a):
        run()
    got = take()
    turned = [torch.empty_like(q), torch.empty_like(k)]
    api.kv_pool_write_rope(desc, rope, 1, None, None, None, c["qi"], c["pos"], c["q"], c["k"], None, *turned, None, None, None, n, st)
    torch.cuda.synchronize()
    want, _, to, _ = attention(*turned, c["v"], [n], desc.scale)
    close(got[2], want, to, "out")
    assert torch.equal(got[4], got[5]) and torch.equal(got[4], got[6]) and torch.equal(got[4], turned[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=a):
        run()
    for r in range(6):
        wipe()
        with torch.cuda.stream(a):
            g.replay() if r % 2 else run()
        for x, y in zip(got, take()):
            assert torch.equal(x, y)
