"""Cases of the operators around the attention kernels: rotary positions written into the KV
pools, attention over whole prompts, and moving rows of the pools.

Each case is one call as a serving loop makes it.  `own` false computes it with elementary torch
operations in 32 bits (64 for rotary angles); `own` true calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

#: (query heads, kv heads, head_dim) of the workloads this repository is measured on, and a small one
SHAPES = {"gpt2": (12, 12, 64), "gqa4": (32, 8, 128), "gqa8": (64, 8, 128), "small": (16, 4, 64), "tiny": (4, 4, 64)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # kv_pool_write_rope: one decode token for each of 64 chats on a shared system prompt
        dict(name="rope, 64 decode tokens", op="rope", dtype="bf16", shape="gpt2", seqs=64, new=1, prefix=409, rot=64,
             axes=1, cyclic=False, interleaved=False, far=0, lens=1),
        # one decode token each for a large batch with long tables, positions far into the context, neighbouring pairs
        dict(name="rope, 256 far decode tokens", op="rope", dtype="bf16", shape="gqa4", seqs=256, new=1, prefix=8191,
             rot=128, axes=1, cyclic=False, interleaved=True, far=900001, lens=2),
        # prompts with images: time, height and width positions, the axes' frequencies taken in turn
        dict(name="rope, 24 image prompts", op="rope", dtype="bf16", shape="gqa8", seqs=24, new=2049, prefix=0, rot=128,
             axes=3, cyclic=True, interleaved=False, far=0, lens=3),
        # full precision rows of which half the head turns, the axes' frequencies in blocks
        dict(name="rope, f32 half heads", op="rope", dtype="f32", shape="gqa4", seqs=7, new=1500, prefix=77, rot=64,
             axes=3, cyclic=False, interleaved=False, far=31, lens=4),
        # prompt_attention: one cold question
        dict(name="prompt, one of 409", op="prompt", dtype="bf16", shape="gpt2", seqs=1, new=409, even=True, lens=5),
        # a packed batch of cold prompts of very different lengths
        dict(name="prompt, 48 ragged", op="prompt", dtype="bf16", shape="gqa4", seqs=48, new=2113, even=False, lens=6),
        # a long document
        dict(name="prompt, one of 32768", op="prompt", dtype="bf16", shape="gqa4", seqs=1, new=32768, even=True, lens=7),
        # full precision prompts
        dict(name="prompt, 8 f32 ragged", op="prompt", dtype="f32", shape="small", seqs=8, new=2001, even=False, lens=8),
        # kv_pool_copy: slots moved down before a small pool shrinks
        dict(name="copy, 700 slots", op="copy", dtype="bf16", shape="gpt2", pages=700, page=1, layers=2, lens=9),
        # pages of 16 tokens of several layers, as a large pool is compacted
        dict(name="copy, 3001 pages of 16", op="copy", dtype="bf16", shape="gqa4", pages=3001, page=16, layers=4, lens=10),
        # kv_pool_fork: 8 answers sampled from each of 12 prompts, the last partial page copied
        dict(name="fork, 96 answers", op="fork", dtype="bf16", shape="gpt2", parents=12, children=8, ctx=523, tail=15,
             layers=2, lens=11),
        # beams over long contexts that part with their whole answers so far, in full precision
        dict(name="fork, 64 beams", op="fork", dtype="f32", shape="gqa4", parents=16, children=4, ctx=4099, tail=401,
             layers=2, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "copy", "fork"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    lens = rng.randrange(1 << 30)
    if op == "rope":
        shape = rng.choice(list(SHAPES))
        d = SHAPES[shape][2]
        new = rng.choice([1, _log(rng, 2, 2048)])
        seqs = _log(rng, 1, 256 if new == 1 else max(1, 24576 // new))
        return dict(op=op, dtype=dtype, shape=shape, seqs=min(seqs, 256), new=new, prefix=rng.choice([0, _log(rng, 1, 8191)]),
                    rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 2, 3, 4]), cyclic=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, far=rng.choice([0, _log(rng, 1, 1000000)]), lens=lens)
    if op == "prompt":
        if dtype == "f32":
            shape, new = rng.choice(["small", "tiny", "gpt2"]), _log(rng, 1, 2048)
            seqs = min(16, _log(rng, 1, max(1, 12288 // new)))
        else:
            shape, new = rng.choice(["gpt2", "gqa4", "gqa4", "small"]), _log(rng, 1, 16384)
            seqs = min(64, _log(rng, 1, max(1, 32768 // new)))
        return dict(op=op, dtype=dtype, shape=shape, seqs=seqs, new=new, even=rng.random() < 0.3, lens=lens)
    if op == "copy":
        page = rng.choice([1, 1, 16, 64])
        layers = rng.randint(1, 4)
        shape = rng.choice(["gpt2", "gqa4", "small"])
        return dict(op=op, dtype=dtype, shape=shape, pages=max(1, _log(rng, 8, 32768) // page), page=page, layers=layers, lens=lens)
    parents = _log(rng, 1, 24)
    return dict(op="fork", dtype=dtype, shape=rng.choice(["gpt2", "gqa4", "small"]), parents=parents,
                children=rng.randint(1, 8), ctx=_log(rng, 8, 4099), tail=_log(rng, 1, 256), layers=rng.randint(1, 3),
                lens=lens)


def _prompt_lens(case):
    """Tokens of each sequence: all alike, or spread over the logarithm up to the longest (and one of them is it)."""
    n, top = case["seqs"], case["new"]
    if case.get("even") or top == 1:
        return [top] * n
    r = random.Random(case["lens"])
    out = [_log(r, 1, top) for _ in range(n)]
    out[r.randrange(n)] = top
    return out


def _prefix_lens(case):
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, case["prefix"]) for _ in range(case["seqs"])]


def _fork_plan(case):
    """Per output row: parent, tokens kept in the parent's slots, and tokens in all."""
    r = random.Random(case["lens"] + 2)
    rows = []
    for p in range(case["parents"]):
        n = r.randint(max(1, case["ctx"] // 2), case["ctx"])
        for c in range(case["children"]):
            tail = 0 if c == 0 else r.randint(0, min(n, case["tail"]))   # the first child stays where the parent is
            rows.append((p, n - tail, n))
    return rows


def _sections(case):
    """Frequency pairs of each axis: as even as whole numbers allow, the first axis takes what is left over."""
    half, a = case["rot"] // 2, case["axes"]
    s = [half // a] * a
    s[0] += half - sum(s)
    return s


def _axis_of_pair(case):
    s, out = _sections(case), []
    if not case["cyclic"]:
        for a, n in enumerate(s):
            out += [a] * n
        return out
    left, a = list(s), 0
    for _ in range(case["rot"] // 2):     # the axes in turn; one that has its share drops out
        while not left[a]:
            a = (a + 1) % len(s)
        out.append(a)
        left[a] -= 1
        a = (a + 1) % len(s)
    return out


BASE = 1000000.0


def _stride(n):
    return (n + 7) // 8 * 8


# --------------------------------------------------------------------------- states
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _fused(g, T, hq, hkv, d, dt):
    """Rows of one projection's output: a token's queries, keys and values side by side."""
    x = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda", dtype=torch.float32).to(dt)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv, d = SHAPES[case["shape"]]
    dt = TYPES[case["dtype"]]
    st = dict(case=case, hq=hq, hkv=hkv, d=d, dt=dt, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "rope":
        lens = _prompt_lens(dict(case, even=case["new"] == 1))
        pre = _prefix_lens(case)
        T, P = sum(lens), sum(pre)
        slots = torch.randperm(2 * T + P + 16, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        st["num_slots"] = slots.numel()
        st["q"], st["k"], st["v"] = _fused(g, T, hq, hkv, d, dt)
        st["batch"], st["total"] = case["seqs"], T
        st["prefix_slots"], st["new_slots"] = slots[:P].contiguous() if P else slots[:1].contiguous(), slots[P:P + T].contiguous()
        st["prefix_indptr"], st["qo_indptr"] = _ints(_indptr(pre), torch.int64), _ints(_indptr(lens), torch.int64)
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), _ints(lens, torch.int64))
        first = torch.arange(T, device="cuda") - st["qo_indptr"][seq] + _ints(pre, torch.int64)[seq] + case["far"]
        pos = [first] + [torch.randint(0, 120, (T,), generator=g, device="cuda") + first // 4 for _ in range(case["axes"] - 1)]
        st["positions"] = torch.stack(pos).to(torch.int32).contiguous()
        st["stride"] = _stride(max(p + n for p, n in zip(pre, lens)))
        st["r2t"] = torch.empty(case["seqs"], st["stride"], dtype=torch.int32, device="cuda")
        st["k_pool"] = torch.zeros(st["num_slots"], hkv, d, dtype=dt, device="cuda")
        st["v_pool"] = torch.zeros_like(st["k_pool"])
        st["q_out"] = torch.empty(T, hq, d, dtype=dt, device="cuda")
    elif case["op"] == "prompt":
        lens = _prompt_lens(case)
        T = sum(lens)
        st["lens"], st["batch"], st["total"] = lens, len(lens), T
        st["num_slots"] = T
        st["q"], st["k"], st["v"] = _fused(g, T, hq, hkv, d, dt)
        st["indptr"] = _ints(_indptr(lens), torch.int64)
        st["out"] = torch.empty(T, hq, d, dtype=dt, device="cuda")
        st["lse"] = torch.empty(T, hq, dtype=torch.float32, device="cuda")
    elif case["op"] == "copy":
        n, page = case["pages"], case["page"]
        total = 2 * n + n // 2 + 2
        ids = torch.randperm(total, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        st["src"], st["dst"] = ids[:n].contiguous(), ids[n:2 * n].contiguous()
        st["num_slots"] = total * page
        st["pools"] = torch.randn(case["layers"], 2, st["num_slots"], hkv, d, generator=g, device="cuda").to(dt)
        st["list"] = [st["pools"][i, j] for i in range(case["layers"]) for j in range(2)]
    else:
        rows = _fork_plan(case)
        own_len = {}
        for p, _, n in rows:
            own_len[p] = n
        lens = [own_len[p] for p in range(case["parents"])]
        tails = [n - keep for _, keep, n in rows]
        L, X = sum(lens), sum(tails)
        slots = torch.randperm(L + X + 64, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        st["num_slots"] = slots.numel()
        st["stride"] = _stride(max(lens))
        table = torch.full((case["parents"], st["stride"]), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(st["stride"], device="cuda")
        table[col[None, :] < _ints(lens, torch.int64)[:, None]] = slots[:L]
        st["r2t_in"], st["r2t_out"] = table, torch.empty(len(rows), st["stride"], dtype=torch.int32, device="cuda")
        st["tail_slots"] = slots[L:L + max(X, 1)].contiguous()
        st["total_tail"] = X
        st["parents"], st["keep"], st["kv_lens"] = (_ints([r[i] for r in rows]) for i in range(3))
        st["tail_indptr"] = _ints(_indptr(tails), torch.int64)
        st["pools"] = torch.randn(case["layers"], 2, st["num_slots"], hkv, d, generator=g, device="cuda").to(dt)
        st["list"] = [st["pools"][i, j] for i in range(case["layers"]) for j in range(2)]
    return st


# --------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, interleaved):
    """Rows x [T, h, d] with the pairs of their first `rot` channels turned by the angles of cos, sin [T, rot / 2]."""
    x = x.float()
    c, s = cos[:, None, :], sin[:, None, :]
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return out


def _plain_rope(st):
    case, dt, rot = st["case"], st["dt"], st["case"]["rot"]
    freq = BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = st["positions"].double()[torch.tensor(_axis_of_pair(case), device="cuda")].t() * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    st["q_out"].copy_(_turn(st["q"], cos, sin, rot, case["interleaved"]).to(dt))
    at = st["new_slots"].long()
    st["k_pool"][at] = _turn(st["k"], cos, sin, rot, case["interleaved"]).to(dt)
    st["v_pool"][at] = st["v"]
    pre, new = st["prefix_indptr"].diff()[:, None], st["qo_indptr"].diff()[:, None]
    col = torch.arange(st["stride"], device="cuda")[None, :]
    was, fresh = st["prefix_indptr"][:-1, None] + col, st["qo_indptr"][:-1, None] + col - pre
    old = st["prefix_slots"][was.clamp(max=st["prefix_slots"].numel() - 1)]
    got = st["new_slots"][fresh.clamp(0, st["new_slots"].numel() - 1)]
    st["r2t"].copy_(torch.where(col < pre, old, torch.where(col < pre + new, got, -1)))
    return st["q_out"], st["k_pool"], st["v_pool"], st["r2t"]


def _plain_prompt(st):
    hq, hkv, d = st["hq"], st["hkv"], st["d"]
    start = 0
    for n in st["lens"]:
        q = st["q"][start:start + n].float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)
        k = st["k"][start:start + n].float().permute(1, 2, 0)[:, None]
        v = st["v"][start:start + n].float().permute(1, 0, 2)[:, None]
        step = max(1, min(n, (1 << 31) // (hq * n)))
        for a in range(0, n, step):           # a block of queries at a time: their scores fit the memory
            b = min(n, a + step)
            s = (q[:, :, a:b] @ k[..., :b]) * (1.0 / math.sqrt(d))
            hidden = torch.arange(b, device="cuda")[None, :] > torch.arange(a, b, device="cuda")[:, None]
            s.masked_fill_(hidden, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = (s - m).exp_()
            z = p.sum(-1, keepdim=True)
            o = (p @ v[:, :, :b]) / z
            st["out"][start + a:start + b] = o.permute(2, 0, 1, 3).reshape(b - a, hq, d).to(st["dt"])
            st["lse"][start + a:start + b] = (m + z.log())[..., 0].permute(2, 0, 1).reshape(b - a, hq)
        start += n
    return st["out"], st["lse"]


def _plain_copy(st):
    page, pools = st["case"]["page"], st["pools"]
    paged = pools.view(pools.shape[0], 2, -1, page, st["hkv"], st["d"])
    paged[:, :, st["dst"].long()] = paged[:, :, st["src"].long()]
    return st["pools"]


def _plain_fork(st):
    col = torch.arange(st["stride"], device="cuda")[None, :]
    keep, n = st["keep"].long()[:, None], st["kv_lens"].long()[:, None]
    parent = st["parents"].long()
    at = (st["tail_indptr"][:-1, None] + col - keep).clamp(0, st["tail_slots"].numel() - 1)
    tail = (col >= keep) & (col < n)
    rows = st["r2t_in"][parent]
    st["r2t_out"].copy_(torch.where(col < keep, rows, torch.where(tail, st["tail_slots"][at], -1)))
    if st["total_tail"]:
        st["pools"][:, :, st["r2t_out"][tail].long()] = st["pools"][:, :, rows[tail].long()]
    return st["r2t_out"], st["pools"]


# --------------------------------------------------------------------------- the library's calls
def _handles(st):
    """What a program makes once for a layer: the shape descriptor and the rotary descriptor."""
    if "desc" not in st:
        from prefix_cached_kv_radix_gb300 import api
        case = st["case"]
        st["desc"] = api.make_desc(api.RX_F32 if case["dtype"] == "f32" else api.RX_BF16, st["hq"], st["hkv"], st["d"],
                                   st["num_slots"], 1.0 / math.sqrt(st["d"]))
        if case["op"] == "rope":
            st["rope"] = api.rope_desc(_sections(case), BASE, cyclic=case["cyclic"], interleaved=case["interleaved"])
        st["api"] = api
    return st["api"]


def _own_run(st):
    api, op = _handles(st), st["case"]["op"]
    if op == "rope":
        api.kv_pool_write_rope(st["desc"], st["rope"], st["batch"], st["prefix_slots"], st["prefix_indptr"], st["new_slots"],
                               st["qo_indptr"], st["positions"], st["q"], st["k"], st["v"], st["q_out"], None, st["k_pool"],
                               st["v_pool"], st["r2t"], st["total"], st["status"])
        return st["q_out"], st["k_pool"], st["v_pool"], st["r2t"]
    if op == "prompt":
        api.prompt_attention(st["desc"], st["batch"], st["q"], st["k"], st["v"], st["indptr"], st["out"], st["lse"],
                             st["total"], st["status"])
        return st["out"], st["lse"]
    if op == "copy":
        api.kv_pool_copy(st["desc"], st["list"], st["src"], st["dst"], st["case"]["page"], st["status"])
        return st["pools"]
    api.kv_pool_fork(st["desc"], st["list"], st["parents"], st["keep"], st["kv_lens"], st["tail_indptr"], st["tail_slots"],
                     st["r2t_in"], st["r2t_out"], st["total_tail"], st["status"])
    return st["r2t_out"], st["pools"]


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "prompt": _plain_prompt, "copy": _plain_copy, "fork": _plain_fork}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the least there is to do
def work(case):
    hq, hkv, d = SHAPES[case["shape"]]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        lens, pre = _prompt_lens(dict(case, even=case["new"] == 1)), _prefix_lens(case)
        T = sum(lens)
        stride = _stride(max(p + n for p, n in zip(pre, lens)))
        index = 4 * sum(pre) + 4 * T + 4 * case["axes"] * T + 4 * len(lens) * stride + 16 * len(lens)
        return {"bytes": 2 * T * (hq + 2 * hkv) * d * size + index, "flops": T * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "prompt":
        lens = _prompt_lens(case)
        T = sum(lens)
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": T * (2 * hq + 2 * hkv) * d * size + 4 * T * hq + 8 * len(lens), "flops": 4 * d * hq * pairs}
    if case["op"] == "copy":
        return {"bytes": case["pages"] * (8 + 2 * 2 * case["layers"] * case["page"] * hkv * d * size), "flops": 0}
    rows = _fork_plan(case)
    tail, stride = sum(n - keep for _, keep, n in rows), _stride(max(n for _, _, n in rows))
    table = 4 * len(rows) * stride + 4 * sum({p: n for p, _, n in rows}.values()) + 4 * tail
    return {"bytes": table + 20 * len(rows) + 2 * tail * 2 * case["layers"] * hkv * d * size, "flops": 0}


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] in ("copy", "fork"):
        return None                          # moved values: nothing is computed
    st = prepare(case, seed)
    if case["op"] == "rope":
        rot, half = case["rot"], case["rot"] // 2
        pairs = torch.arange(half, dtype=torch.float64, device="cuda")
        axis = torch.tensor(_axis_of_pair(case), device="cuda")
        angle = st["positions"].double().index_select(0, axis).t() * torch.exp(pairs * (-2.0 * math.log(BASE) / rot))
        z = torch.polar(torch.ones_like(angle), angle)[:, None, :]

        def turned(x):
            x = x.double()
            body = x[..., :rot].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
            body = body if case["interleaved"] else body.transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(body.contiguous()) * z)
            y = (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)
            return torch.cat([y, x[..., rot:]], -1)

        k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
        k_pool.index_copy_(0, st["new_slots"].long(), turned(st["k"]))
        v_pool.index_copy_(0, st["new_slots"].long(), st["v"].double())
        return turned(st["q"]), k_pool, v_pool, None
    hq, hkv, d = st["hq"], st["hkv"], st["d"]
    out = torch.empty(st["total"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["total"], hq, dtype=torch.float64, device="cuda")
    at = 0
    for n in st["lens"]:
        for h in range(hq):
            key, val = (st[x][at:at + n, h // (hq // hkv)].double() for x in ("k", "v"))
            ask = st["q"][at:at + n, h].double() / math.sqrt(d)
            for a in range(0, n, 4096):
                b = min(n, a + 4096)
                s = torch.einsum("id,jd->ij", ask[a:b], key[:b])
                s[torch.ones(b - a, b, dtype=torch.bool, device="cuda").triu(a + 1)] = -math.inf
                z = torch.logsumexp(s, 1)
                lse[at + a:at + b, h] = z
                out[at + a:at + b, h] = torch.exp(s - z[:, None]) @ val[:b]
        at += n
    return out, lse
