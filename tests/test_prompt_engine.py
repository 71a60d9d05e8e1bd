"""The rotary write, whole-prompt attention, forks and resizing as a serving loop uses them
together, through the engine, against plain 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

from prefix_cached_kv_radix_gb300 import api
from tests.prompt_cases import HALF, close, rotate

api.load()
pytestmark = pytest.mark.gpu
BASE = 10000.0


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Layer:
    """Random rows of one layer for every token of some sequences, and what attention over them is:
    queries and keys turned in 64 bits, rounded as the kernels round them."""

    def __init__(self, seed, dt, hq, hkv, d, sections, cyclic):
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.dt, self.hq, self.hkv, self.d, self.sections, self.cyclic = dt, hq, hkv, d, sections, cyclic
        self.freq = BASE ** (-2.0 * torch.arange(sum(sections), dtype=torch.float64, device="cuda") / (2 * sum(sections)))
        self.q, self.k, self.v, self.pos = {}, {}, {}, {}

    def add(self, name, n):
        """n more tokens of sequence `name`: their fused rows and positions."""
        x = torch.randn(n, self.hq + 2 * self.hkv, self.d, generator=self.gen, device="cuda").to(self.dt)
        p = torch.randint(0, 5000, (len(self.sections), n), generator=self.gen, device="cuda")
        for store, part, dim in ((self.q, x[:, :self.hq], 0), (self.k, x[:, self.hq:self.hq + self.hkv], 0),
                                 (self.v, x[:, self.hq + self.hkv:], 0), (self.pos, p, 1)):
            store[name] = part if name not in store else torch.cat([store[name], part], dim)
        return x, p

    def want(self, name):
        """out, its bound: attention over the turned rows of the whole sequence.  The kernels' turned rows
        differ from these by their bounds, `a` of them relative per score, which moves a probability by
        twice that; they are added to the attention's own bound."""
        q, tq = rotate(self.q[name], self.pos[name], self.sections, self.freq, self.cyclic)
        k, tk = rotate(self.k[name], self.pos[name], self.sections, self.freq, self.cyclic)
        n, scale = q.shape[0], 1 / math.sqrt(self.d)
        rep = self.hq // self.hkv
        outs, tols = [], []
        for h in range(self.hq):
            Q, K, V, eq, ek = q[:, h], k[:, h // rep], self.v[name][:, h // rep].double(), tq[:, h], tk[:, h // rep]
            hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            P = torch.softmax((Q @ K.t() * scale).masked_fill(hidden, -math.inf), 1)
            ds = ((eq @ K.abs().t() + Q.abs() @ ek.t() + eq @ ek.t() + (self.d + 8) * 2.0 ** -24 * (Q.abs() @ K.abs().t())) * scale)
            ds = ds.masked_fill(hidden, 0).amax(1, keepdim=True)
            o = P @ V
            rounded = HALF[self.dt] if self.dt != torch.float32 else 0.0
            outs.append(o)
            tols.append((P @ V.abs()) * (torch.expm1(2 * ds) + rounded + (n + 30) * 2.0 ** -23) * 1.01 + o.abs() * (HALF[self.dt] + 2.0 ** -22))
        return torch.stack(outs, 1), torch.stack(tols, 1)


@pytest.mark.parametrize("dtype,hq,hkv,d,sections,cyclic", [("bf16", 8, 2, 128, [24, 20, 20], True), ("f32", 4, 4, 64, [32], False)])
def test_prompts_then_decode_after_resize_and_fork(dtype, hq, hkv, d, sections, cyclic):
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [200, 1, 333]
    layers = [Layer(s, dt, hq, hkv, d, sections, cyclic) for s in (1, 2)]
    eng = PrefixCacheEngine(dtype, hq, hkv, d, 4096, 7, num_layers=2)
    rope = api.rope_desc(sections, BASE, cyclic=cyclic)
    rng = np.random.default_rng(3)
    prompts = [rng.integers(b * 1000, b * 1000 + 900, n).astype(np.int32) for b, n in enumerate(lens)]

    # cold prompts: one rotary write and one attention per layer
    plan = eng.plan(prompts, lens)
    dev = eng.upload(plan)
    for i, lay in enumerate(layers):
        parts = [lay.add(b, n) for b, n in enumerate(lens)]
        x, pos = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1).to(torch.int32).contiguous()
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        eng.write_rope(plan, dev, rope, pos, q, k, v, q, k_out=k, layer=i)          # in place
        out = torch.empty(sum(lens), hq, d, dtype=dt, device="cuda")
        eng.prompt(plan, dev, q, k, v, out)
        at = 0
        for b, n in enumerate(lens):
            want, tol = lay.want(b)
            close(out[at:at + n], want, tol, f"layer {i} prompt {b}")
            at += n
        # the same through the pools
        again = torch.empty_like(out)
        eng.extend(plan, dev, q.contiguous(), again, layer=i)
        at = 0
        for b, n in enumerate(lens):
            want, tol = lay.want(b)
            close(again[at:at + n], want, tol, f"layer {i} extend {b}")
            at += n
    eng.finish(plan)

    # the pools shrink to a little more than what is cached
    assert eng.resize(600) > 0
    eng.tree.check()
    assert eng.k_pools.shape[1] == 600 and eng.tree.stats()["num_slots"] == 600

    # a decode step: one more token each, through the moved rows
    for b in range(3):
        prompts[b] = np.append(prompts[b], np.int32(5000 + b))
    plan = eng.plan(prompts, [1, 1, 1])
    assert plan.layout.total_prefix == sum(lens)
    with pytest.raises(ValueError):
        eng.prompt(plan, {}, None, None, None, None)
    dev = eng.upload(plan)
    outs, queries = [], []
    for i, lay in enumerate(layers):
        parts = [lay.add(b, 1) for b in range(3)]
        x, pos = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1).to(torch.int32).contiguous()
        q = torch.empty(3, hq, d, dtype=dt, device="cuda")
        eng.write_rope(plan, dev, rope, pos, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q, layer=i)
        out = torch.empty_like(q)
        eng.decode(plan, dev, q, out, layer=i)
        for b in range(3):
            want, tol = lay.want(b)
            close(out[b], want[-1], tol[-1], f"layer {i} decode {b}")
        outs.append(out)
        queries.append(q)
    assert eng.device_status() == 0

    # forks: children of the three that keep whole pages of 16 and copy the rest, grown pools first
    assert eng.resize(5000) == 0 and eng.k_pools.shape[1] == 5000
    rows = [2, 0, 2, 1, 0]
    L = np.array([lens[p] + 1 for p in rows], np.int32)
    r2t = dev["r2t"][:3].contiguous()
    table, tail = eng.fork(r2t, rows, L - L % 16, L)
    assert len(tail) == int((L % 16).sum())
    for f, p in enumerate(rows):
        keep = L[f] - L[f] % 16
        assert torch.equal(table[f, :keep], r2t[p, :keep]) and not torch.equal(table[f, keep:L[f]], r2t[p, keep:L[f]])
    old = r2t[torch.tensor(rows, device="cuda")]
    for f in range(5):                                     # the parents' own tails are gone: only the copies are left
        keep = int(L[f] - L[f] % 16)
        for pool in (eng.k_pools, eng.v_pools):
            pool[:, old[f, keep:L[f]].long()] = math.nan
    kv = torch.tensor(L, device="cuda")
    for i in range(2):
        q = queries[i][torch.tensor(rows, device="cuda")].contiguous()
        out = torch.empty_like(q)
        ws = torch.empty(max(api.decode_workspace_bytes(eng.desc, 5, int(L.max())), 256), dtype=torch.uint8, device="cuda")
        api.decode_attention(eng.desc, 5, q, table, kv, eng.k_pools[i], eng.v_pools[i], out, None, int(L.max()), ws, eng.status)
        for f, p in enumerate(rows):
            want, tol = layers[i].want(p)
            close(out[f], want[-1], tol[-1], f"layer {i} fork {f}")
    eng.tree.free_slots(tail)
    eng.commit(plan)
    eng.tree.unlock_batch(plan.last_nodes)
    eng.tree.check()
    assert eng.device_status() == 0


def test_one_call_step_after_resize():
    """The one-call path binds the pools' addresses and size once; a resize makes it do so again."""
    import workloads as W
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine, _dev_from_host
    from tests.gpu_cases import compare, oracle_rows
    spec = W.spec_branching("resize-step", "bf16", 8, 2, 128, 4096, W.QWEN_VOCAB, 5, root=96, n_children=2, child_len=40,
                            leaves_per_child=2, n_new=33)
    w = W.generate(spec)
    eng = PrefixCacheEngine("bf16", 8, 2, 128, 4096, 5)
    for i in range(len(spec.histories)):
        k, v = w.history_kv(i)
        eng.populate(w.history_tokens(i), k, v)
    q, k, v = (_dev_from_host(x, "bf16", eng.device) for x in w.stacked_new())
    qo = w.qo_indptr()
    for i, slots in enumerate((4096, 900, 9000)):
        if slots != eng.num_slots:
            eng.resize(slots)
        # the same rows under new token ids: a new step on the same cached prefixes
        toks = [np.concatenate([w.request_prefix_tokens(b), 200000 + 10000 * i + 100 * b + np.arange(n)]).astype(np.int32)
                for b, n in enumerate(spec.req_new)]
        ind = np.concatenate([[0], np.cumsum([len(t) for t in toks])]).astype(np.int64)
        out = torch.empty_like(q)
        eng.step(np.concatenate(toks), ind, spec.req_new, q, k, v, out)
        torch.cuda.synchronize()
        assert eng.device_status() == 0
        for b in range(w.batch):
            want, _ = oracle_rows(w, b)
            compare(out[qo[b]:qo[b + 1]].float().cpu().numpy(), want, f"{slots} slots, request {b}")
        eng.tree.check()


def test_resize_on_another_stream_is_in_order():
    """What the engine's stream has written is moved, and what comes there next sees it moved, also where
    the memory of the old pools is used again at once."""
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    n, slots = 3000, 20000
    eng = PrefixCacheEngine("bf16", 8, 8, 128, slots, 3)
    toks = np.arange(n, dtype=np.int32)
    k, v = (torch.randn(n, 8, 128, device="cuda").bfloat16() for _ in range(2))
    eng.populate(toks, k, v)
    a, b = torch.randn(8192, 8192, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for size in (40000, 6000, 70000):
        with torch.cuda.stream(b):
            for _ in range(4):
                a @ a                                  # a busy stream
        eng.resize(size, stream=b)
        junk = [torch.full((slots, 8, 128), 9.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
        sl, m, _ = eng.tree.match_prefix(toks)
        at = torch.tensor(sl, device="cuda").long()
        assert m == n and torch.equal(eng.k_pool[at], k) and torch.equal(eng.v_pool[at], v)
        del junk
    assert eng.device_status() == 0


@pytest.mark.parametrize("own", [False, True])
def test_fork_on_another_stream_is_in_order(own):
    """Rows and table that the engine's stream is still writing are forked whole, and what comes on the engine's
    stream next (the table read, the parents' rows overwritten, the given-back slots written again) comes after
    the fork; `own`: on the engine's stream itself.  The stream is given as such and as an address."""
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    n, keep = 2000, 16
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        eng = PrefixCacheEngine("bf16", 8, 8, 128, 3 * n, 3, num_layers=2)
        a = torch.randn(8192, 8192, device="cuda")
        rows = torch.randn(2, 2, n, 8, 128, device="cuda").bfloat16()
    other = s if own else torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (other, other.cuda_stream):
        at = eng.tree.alloc_slots(n)
        idx = torch.tensor(at, device="cuda").long()
        with torch.cuda.stream(s):
            table = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
            rows.neg_()
            for _ in range(6):
                a @ a                                      # a busy stream, then the parent's rows and table on it
            eng.k_pools[:, idx], eng.v_pools[:, idx] = rows[0], rows[1]
            table[0] = idx.int()
        got, tail = eng.fork(table, [0], [keep], [n], stream=handle)
        with torch.cuda.stream(s):
            del table
            junk = torch.full((1, n), -5, dtype=torch.int32, device="cuda")
            eng.k_pools[:, idx[keep:]], eng.v_pools[:, idx[keep:]] = math.nan, math.nan
            seen = got.clone()
            copies = torch.stack([eng.k_pools[:, seen[0].long()], eng.v_pools[:, seen[0].long()]])
            eng.k_pools[:, torch.tensor(tail, device="cuda").long()] = math.nan
            eng.tree.free_slots(tail)
            eng.tree.free_slots(at)
        torch.cuda.synchronize()
        assert seen[0].tolist() == at[:keep].tolist() + tail.tolist()
        assert torch.equal(copies, rows) and (junk == -5).all()
    assert eng.device_status() == 0


@pytest.mark.parametrize("failing", ["memory", "first copy", "second copy", "growing", "slots held"])
def test_failed_resize_is_consistent(failing, monkeypatch):
    """A resize that fails leaves tree, pools and descriptor of one size, and every match names rows that are
    there: nothing has changed, or, where the copy of the moved rows itself fails, they are no longer cached."""
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    eng = PrefixCacheEngine("bf16", 2, 2, 64, 256, 3, num_layers=2)
    toks, n = np.arange(90, dtype=np.int32), 90
    kv = [[torch.randn(n, 2, 64, device="cuda").bfloat16() for _ in range(2)] for _ in range(2)]
    eng.populate(toks, *kv)
    before, stats = eng.tree.match_prefix(toks)[0].tolist(), eng.tree.stats()
    assert max(before) >= 120
    calls, copy, held = [], api.kv_pool_copy, None

    def fails(*a):
        calls.append(a)
        if len(calls) == (2 if failing == "second copy" else 1):
            raise api.RxError("kv_pool_copy", api.RX_ECUDA, "planted")
        return copy(*a)

    def none_left(*a, **kw):
        raise torch.OutOfMemoryError("planted")
    with monkeypatch.context() as m:
        if failing == "slots held":
            held = eng.tree.alloc_slots(eng.tree.stats()["free_slots"])
            stats = eng.tree.stats()
        elif failing in ("memory", "growing"):
            for f in ("empty", "zeros", "from_numpy"):
                m.setattr(torch, f, none_left)
        else:
            m.setattr(api, "kv_pool_copy", fails)
        with pytest.raises((api.RxError, torch.OutOfMemoryError)):
            eng.resize(300 if failing == "growing" else 120)
    if held is not None:
        eng.tree.free_slots(held)
        stats = eng.tree.stats()
    size = 120 if failing == "second copy" else 256
    assert eng.num_slots == eng.desc.num_slots == eng.k_pools.shape[1] == eng.v_pools.shape[1] == eng.tree.stats()["num_slots"] == size
    eng.tree.check()
    slots, m, _ = eng.tree.match_prefix(toks)
    if failing == "second copy":
        assert m == 0 and eng.tree.stats()["free_slots"] == 120
        eng.populate(toks, *kv)                            # and it serves on
        slots = eng.tree.match_prefix(toks)[0]
    else:
        assert slots.tolist() == before
        for key in ("cached_tokens", "free_slots"):
            assert eng.tree.stats()[key] == stats[key]
        assert eng.resize(120) > 0
        slots = eng.tree.match_prefix(toks)[0]
    at = torch.tensor(slots, device="cuda").long()
    for i in range(2):
        assert torch.equal(eng.k_pools[i][at], kv[0][i]) and torch.equal(eng.v_pools[i][at], kv[1][i])
    assert eng.device_status() == 0


def test_refused_fork_gives_its_slots_back():
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    eng = PrefixCacheEngine("f32", 2, 2, 64, 64, 3)
    free = eng.tree.stats()["free_slots"]
    with pytest.raises(ValueError):
        eng.fork(torch.zeros(1, 8, device="cuda"), [0], [2], [5])          # not a table of slots
    assert eng.tree.stats()["free_slots"] == free
    with pytest.raises(ValueError):
        eng.fork(torch.zeros(1, 8, dtype=torch.int32, device="cuda"), [0], [6], [5])
    assert eng.tree.stats()["free_slots"] == free
    eng.tree.check()


@pytest.mark.parametrize("op", ["resize", "fork"])
def test_interrupted_move_is_consistent(op, monkeypatch):
    """Ctrl-C in the midst of a resize or a fork: no match names rows that were not moved, no slot is lost."""
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    eng = PrefixCacheEngine("f32", 2, 2, 64, 256, 3)
    toks = np.arange(90, dtype=np.int32)
    eng.populate(toks, *(torch.randn(90, 2, 64, device="cuda") for _ in range(2)))
    assert max(eng.tree.match_prefix(toks)[0]) >= 120
    free, left, copy = eng.tree.stats()["free_slots"], [1], api.kv_pool_copy

    def interrupted(*a):
        if op == "fork" or not left:
            raise KeyboardInterrupt
        left.pop()
        return copy(*a)
    with monkeypatch.context() as m:
        m.setattr(api, "kv_pool_copy", interrupted)
        m.setattr(api, "kv_pool_fork", interrupted)
        with pytest.raises(KeyboardInterrupt):
            if op == "resize":
                eng.resize(120)
            else:
                eng.fork(torch.zeros(1, 8, dtype=torch.int32, device="cuda"), [0], [2], [5])
    eng.tree.check()
    size = 120 if op == "resize" else 256
    assert eng.num_slots == eng.desc.num_slots == eng.k_pools.shape[1] == eng.tree.stats()["num_slots"] == size
    assert eng.tree.match_prefix(toks)[1] == (0 if op == "resize" else 90)
    assert eng.tree.stats()["free_slots"] == (120 if op == "resize" else free)


@pytest.mark.parametrize("stream", ["no stream", 1 << 70])
def test_moves_on_what_is_no_stream_change_nothing(stream):
    from prefix_cached_kv_radix_gb300.engine import PrefixCacheEngine
    eng = PrefixCacheEngine("f32", 2, 2, 64, 64, 3)
    eng.populate(np.arange(20, dtype=np.int32), *(torch.randn(20, 2, 64, device="cuda") for _ in range(2)))
    before = eng.tree.stats()
    for call in (lambda: eng.fork(torch.zeros(1, 8, dtype=torch.int32, device="cuda"), [0], [2], [5], stream=stream),
                 lambda: eng.resize(30, stream=stream), lambda: eng.resize(90, stream=stream)):
        with pytest.raises(Exception):
            call()
        after = eng.tree.stats()
        assert all(after[k] == before[k] for k in ("free_slots", "num_slots", "cached_tokens"))
        assert eng.num_slots == eng.desc.num_slots == eng.k_pools.shape[1] == 64
        eng.tree.check()
