"""Cases of the 8-bit KV cache: rows quantised as they are written into the pools, rows read back, and
decode and extend attention over pools held in 8 bits.

A pool holds codes, int8 or e4m3; a value is its code times the scale of its block of slots and kv head.
Each case is one call as a serving loop makes it.  `own` false computes it with elementary torch operations
in 32 bits (64 for the quotients that are rounded to whole codes); `own` true calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

#: (query heads, kv heads, head_dim) of the workloads this repository is measured on, and small ones
SHAPES = {"gpt2": (12, 12, 64), "gqa4": (32, 8, 128), "gqa8": (64, 8, 128), "small": (16, 4, 64), "tiny": (4, 4, 64)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST = {"int8": 127.0, "e4m3": 448.0}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # kv_pool_write_q8: one decode token for each of 64 chats on a shared system prompt
        dict(name="write, 64 decode tokens", op="write", dtype="bf16", code="int8", shape="gpt2", block=1, fixed=False, seqs=64,
             new=1, prefix=409, lens=1),
        # the prompts of a large batch, parts of one projection's output
        dict(name="write, 24 ragged prompts", op="write", dtype="bf16", code="e4m3", shape="gqa4", block=1, fixed=False, seqs=24,
             new=2049, prefix=0, lens=2),
        # full precision rows into a pool whose pages of 16 slots have calibrated scales
        dict(name="write, f32 into fixed scales", op="write", dtype="f32", code="int8", shape="gqa4", block=16, fixed=True, seqs=7,
             new=1500, prefix=77, lens=3),
        # kv_pool_read_q8: one cached prompt for a layer that wants its rows
        dict(name="read, 700 slots", op="read", dtype="bf16", code="e4m3", shape="gpt2", block=1, fixed=False, slots=700, lens=4),
        # the prefixes of a batch, for a pool in 16 bits
        dict(name="read, 40001 slots", op="read", dtype="bf16", code="int8", shape="gqa4", block=1, fixed=False, slots=40001, lens=5),
        # decode_attention_q8: 64 chats on a shared system prompt
        dict(name="decode, 64 chats", op="decode", dtype="bf16", code="int8", shape="gpt2", block=1, fixed=False, seqs=64, ctx=441,
             least=411, shared=0, lens=6),
        # a large batch with contexts of 1024 to 8192 tokens
        dict(name="decode, 256 long", op="decode", dtype="bf16", code="e4m3", shape="gqa4", block=1, fixed=False, seqs=256, ctx=8192,
             least=1024, shared=0, lens=7),
        # two questions on very long documents
        dict(name="decode, 2 documents", op="decode", dtype="bf16", code="int8", shape="gqa8", block=1, fixed=False, seqs=2,
             ctx=131071, least=100001, shared=0, lens=8),
        # full precision rows over pages of 16 slots with calibrated scales
        dict(name="decode, 33 in f32", op="decode", dtype="f32", code="e4m3", shape="small", block=16, fixed=True, seqs=33, ctx=3001,
             least=1, shared=0, lens=9),
        # prefix_extend_attention_q8: 64 short questions on a system prompt
        dict(name="extend, 64 questions", op="extend", dtype="bf16", code="int8", shape="gpt2", block=1, fixed=False, seqs=64, new=8,
             prefix=409, even=True, lens=10),
        # long chats that go on
        dict(name="extend, 4 long chats", op="extend", dtype="bf16", code="e4m3", shape="gqa8", block=1, fixed=False, seqs=4, new=512,
             prefix=16384, even=False, lens=11),
        # full precision rows over ragged prefixes
        dict(name="extend, 9 in f32", op="extend", dtype="f32", code="int8", shape="small", block=1, fixed=False, seqs=9, new=101,
             prefix=1201, even=False, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "extend", "extend"])
    fixed = rng.random() < 0.3
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), code=rng.choice(["int8", "e4m3"]), fixed=fixed,
                block=rng.choice([1, 16, 64]) if fixed else 1, lens=rng.randrange(1 << 30))
    f32 = case["dtype"] == "f32"
    if op == "write":
        new = rng.choice([1, _log(rng, 2, 2048)])
        return dict(case, shape=rng.choice(["gpt2", "gqa4", "gqa8", "small"]), new=new,
                    seqs=min(256, _log(rng, 1, 256 if new == 1 else max(1, 24576 // new))), prefix=rng.choice([0, _log(rng, 1, 4096)]))
    if op == "read":
        return dict(case, shape=rng.choice(["gpt2", "gqa4", "small", "tiny"]), slots=_log(rng, 1, 32768))
    if op == "decode":
        ctx = _log(rng, 1, 8192 if f32 else 131071)
        seqs = min(256, _log(rng, 1, max(1, (65536 if f32 else 524288) // ctx)))
        shared = rng.randint(1, ctx) if not f32 and seqs > 1 and rng.random() < 0.3 else 0
        return dict(case, shape=rng.choice(["small", "tiny", "gqa4"] if f32 else ["gpt2", "gqa4", "gqa4", "gqa8", "small"]), seqs=seqs,
                    ctx=ctx, least=max(1, shared, ctx // rng.choice([1, 2, 100])), shared=shared)
    new = _log(rng, 1, 128 if f32 else 1024)
    prefix = rng.choice([0, _log(rng, 1, 1024 if f32 else 16384)])
    most = (1 << 18 if f32 else 1 << 24) // (new * (prefix + new))
    return dict(case, shape=rng.choice(["small", "tiny"] if f32 else ["gpt2", "gqa4", "gqa8", "small"]), new=new, prefix=prefix,
                seqs=min(64, _log(rng, 1, max(1, most))), even=rng.random() < 0.3)


def _spread(case, n, least, top):
    """n lengths of least .. top, one of them the longest."""
    r = random.Random(case["lens"])
    out = [r.randint(least, top) for _ in range(n)]
    out[r.randrange(n)] = top
    return out


def _new_lens(case):
    if case["new"] == 1 or case.get("even"):
        return [case["new"]] * case["seqs"]
    return _spread(case, case["seqs"], 1, case["new"])


def _prefix_lens(case):
    if case.get("even"):
        return [case["prefix"]] * case["seqs"]
    r = random.Random(case["lens"] + 1)
    return [r.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["seqs"])]


def _group_of(case):
    """The requests of the decode batch that share their first tokens: the first two thirds."""
    return max(2, case["seqs"] * 2 // 3) if case["shared"] else 0


def _stride(n):
    return (n + 7) // 8 * 8


# --------------------------------------------------------------------------- codes and scales
def _scales_of(x, code):
    """The scale of each row of x [rows, heads, d] that has no fixed one: the smallest that its largest value
    fits, for e4m3 a power of two (so that neither the quotients nor the values read back are rounded)."""
    top = x.float().abs().amax(-1)
    if code == "int8":
        s = (top.double() / 127.0).float().clamp(min=2.0 ** -126)
    else:
        part, power = torch.frexp(top.double() / torch.full_like(top, 448.0))      # a number 448 would be taken as its reciprocal
        power = torch.where(top > 0, power - (part == 0.5).to(power.dtype), -126).clamp(-126, 127)
        s = ((power + 127) << 23).view(torch.float32)        # 2 ** power
    return torch.where(torch.isfinite(top), s, math.nan)


def _codes_of(x, s, code):
    """x / s, rounded to the nearest code; rows whose scale is NaN have zeros."""
    y = x.double() / s.double()[..., None]
    y = torch.where(torch.isnan(s)[..., None], 0.0, y).clamp(-LARGEST[code], LARGEST[code])
    return (y.round() if code == "int8" else y.float()).to(CODES[code])


def _take(pool, at):
    """Rows of a pool, by slot."""
    return pool.view(torch.uint8)[at].view(pool.dtype)


def _put(pool, at, rows):
    pool.view(torch.uint8)[at] = rows.view(torch.uint8)


# --------------------------------------------------------------------------- states
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _rows(g, n, heads, d):
    """Rows as projections give them: some channels larger than others, and tokens that differ in size."""
    channel = torch.randn(heads, d, generator=g, device="cuda").mul(0.5).exp()
    return torch.randn(n, heads, d, generator=g, device="cuda") * channel * torch.randn(n, 1, 1, generator=g, device="cuda").mul(0.3).exp()


def _fixed_scales(g, blocks, hkv, code):
    """Calibrated scales: about four standard deviations of the block's values fit."""
    spread = 1.0 + 0.5 * torch.rand(blocks, hkv, 2, generator=g, device="cuda")
    return spread * (6.0 / LARGEST[code])


def _pools(st, g, filled):
    """Empty pools, or pools that hold cached tokens in every slot."""
    n, hkv, d, code, block = st["num_slots"], st["hkv"], st["d"], st["case"]["code"], st["case"]["block"]
    blocks = -(-n // block)
    st["scales"] = _fixed_scales(g, blocks, hkv, code) if st["case"]["fixed"] else torch.zeros(blocks, hkv, 2, device="cuda")
    st["k_pool"] = torch.zeros(n, hkv, d, device="cuda", dtype=torch.int8).view(CODES[code])
    st["v_pool"] = torch.zeros(n, hkv, d, device="cuda", dtype=torch.int8).view(CODES[code])
    if not filled:
        return
    for j, name in enumerate(("k_pool", "v_pool")):
        for a in range(0, n, 65536):
            b = min(n, a + 65536)
            x = _rows(g, b - a, hkv, d)
            if st["case"]["fixed"]:
                s = st["scales"][torch.arange(a, b, device="cuda") // block, :, j]
            else:
                s = _scales_of(x, code)
                st["scales"][a:b, :, j] = s
            _put(st[name], slice(a, b), _codes_of(x, s, code))


def _table(lens, slots):
    """A slot table: row b lists lens[b] slots, one after another of `slots`, then -1."""
    stride = _stride(max(lens))
    table = torch.full((len(lens), stride), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(stride, device="cuda")[None, :] < _ints(lens, torch.int64)[:, None]] = slots
    return table


def _shuffled(g, n):
    return torch.randperm(n, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv, d = SHAPES[case["shape"]]
    dt = TYPES[case["dtype"]]
    st = dict(case=case, hq=hq, hkv=hkv, d=d, dt=dt, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "write":
        lens, pre = _new_lens(case), _prefix_lens(case)
        T, P = sum(lens), sum(pre)
        slots = _shuffled(g, 2 * T + P + 16)
        st["num_slots"], st["batch"], st["total"] = slots.numel(), len(lens), T
        x = _rows(g, T, hq + 2 * hkv, d).to(dt)              # a token's queries, keys and values side by side
        st["k"], st["v"] = x[:, hq:hq + hkv], x[:, hq + hkv:]
        st["prefix_slots"], st["new_slots"] = slots[:max(P, 1)].contiguous(), slots[P:P + T].contiguous()
        st["prefix_indptr"], st["qo_indptr"] = _ints(_indptr(pre), torch.int64), _ints(_indptr(lens), torch.int64)
        st["stride"] = _stride(max(p + n for p, n in zip(pre, lens)))
        st["r2t"] = torch.empty(len(lens), st["stride"], dtype=torch.int32, device="cuda")
        _pools(st, g, False)
    elif case["op"] == "read":
        n = case["slots"]
        st["num_slots"] = n + n // 4 + 3
        st["slots"] = _shuffled(g, st["num_slots"])[:n].contiguous()
        _pools(st, g, True)
        st["k_out"], st["v_out"] = (torch.empty(n, hkv, d, dtype=dt, device="cuda") for _ in range(2))
    elif case["op"] == "decode":
        lens = _spread(case, case["seqs"], case["least"], case["ctx"])
        n, m = case["shared"], _group_of(case)
        slots = _shuffled(g, sum(lens) + 64)
        st["num_slots"], st["batch"], st["lens"] = slots.numel(), len(lens), lens
        st["r2t"] = _table(lens, slots[:sum(lens)])
        if m:                                                # the members' first tokens are the first member's
            st["r2t"][1:m, :n] = st["r2t"][:1, :n]
            st["grp_indptr"], st["grp_members"], st["grp_len"] = _ints([0, m]), _ints(list(range(m))), _ints([n])
        st["kv_lens"] = _ints(lens)
        st["q"] = torch.randn(len(lens), hq, d, generator=g, device="cuda").to(dt)
        _pools(st, g, True)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(len(lens), hq, dtype=torch.float32, device="cuda")
    else:
        lens, pre = _new_lens(case), _prefix_lens(case)
        T, total = sum(lens), [p + n for p, n in zip(pre, lens)]
        slots = _shuffled(g, sum(total) + 64)
        st["num_slots"], st["batch"], st["lens"], st["pre"] = slots.numel(), len(lens), lens, pre
        st["r2t"] = _table(total, slots[:sum(total)])
        st["qo_indptr"], st["prefix_lens"] = _ints(_indptr(lens), torch.int64), _ints(pre)
        st["q"] = torch.randn(T, hq, d, generator=g, device="cuda").to(dt)
        _pools(st, g, True)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(T, hq, dtype=torch.float32, device="cuda")
    return st


# --------------------------------------------------------------------------- plain forms
def _values(st, name, at):
    """The cached rows at these slots, in 32 bits."""
    s = st["scales"][at // st["case"]["block"], :, 0 if name == "k_pool" else 1]
    return _take(st[name], at).float() * s[..., None]


def _plain_write(st):
    code, at = st["case"]["code"], st["new_slots"].long()
    for j, (name, x) in enumerate((("k_pool", st["k"]), ("v_pool", st["v"]))):
        if st["case"]["fixed"]:
            s = st["scales"][at // st["case"]["block"], :, j]
        else:
            s = _scales_of(x, code)
            st["scales"][at, :, j] = s
        _put(st[name], at, _codes_of(x, s, code))
    pre, new = st["prefix_indptr"].diff()[:, None], st["qo_indptr"].diff()[:, None]
    col = torch.arange(st["stride"], device="cuda")[None, :]
    was, fresh = st["prefix_indptr"][:-1, None] + col, st["qo_indptr"][:-1, None] + col - pre
    old = st["prefix_slots"][was.clamp(max=st["prefix_slots"].numel() - 1)]
    got = st["new_slots"][fresh.clamp(0, st["new_slots"].numel() - 1)]
    st["r2t"].copy_(torch.where(col < pre, old, torch.where(col < pre + new, got, -1)))
    return st["k_pool"], st["v_pool"], st["scales"], st["r2t"]


def _plain_read(st):
    at = st["slots"].long()
    st["k_out"].copy_(_values(st, "k_pool", at).to(st["dt"]))
    st["v_out"].copy_(_values(st, "v_pool", at).to(st["dt"]))
    return st["k_out"], st["v_out"]


def _attend(q, k, v, seen):
    """Softmax attention: q [b, h, n, g, d], k and v [b, l, h, d], seen [b, n, l].  Returns the rows and their
    log-sum-exp."""
    b, h, n, g, d = q.shape
    s = (q.reshape(b, h, n * g, d) @ k.permute(0, 2, 3, 1)).view(b, h, n, g, -1) * (1.0 / math.sqrt(d))
    s = s.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp()
    z = p.sum(-1, keepdim=True)
    o = (p.view(b, h, n * g, -1) @ v.permute(0, 2, 1, 3)).view(b, h, n, g, d) / z
    return o, (m + z.log())[..., 0]


def _plain_decode(st):
    b, hq, hkv, d = st["batch"], st["hq"], st["hkv"], st["d"]
    at = st["r2t"].clamp(min=0).long()
    seen = torch.arange(at.shape[1], device="cuda")[None, None, :] < st["kv_lens"][:, None, None]
    o, lse = _attend(st["q"].float().view(b, hkv, 1, hq // hkv, d), _values(st, "k_pool", at), _values(st, "v_pool", at), seen)
    st["out"].copy_(o.reshape(b, hq, d).to(st["dt"]))
    st["lse"].copy_(lse.reshape(b, hq))
    return st["out"], st["lse"]


def _plain_extend(st):
    b, hq, hkv, d, n = st["batch"], st["hq"], st["hkv"], st["d"], max(st["lens"])
    at = st["r2t"].clamp(min=0).long()
    row = torch.arange(n, device="cuda")[None, :]
    real = row < st["qo_indptr"].diff()[:, None]
    src = (st["qo_indptr"][:-1, None] + row).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][src].float().view(b, n, hkv, hq // hkv, d).transpose(1, 2)
    last = st["prefix_lens"].long()[:, None] + row
    seen = torch.arange(at.shape[1], device="cuda")[None, None, :] <= last[:, :, None]
    o, lse = _attend(q, _values(st, "k_pool", at), _values(st, "v_pool", at), seen)
    st["out"].copy_(o.transpose(1, 2).reshape(b, n, hq, d)[real].to(st["dt"]))
    st["lse"].copy_(lse.transpose(1, 2).reshape(b, n, hq)[real])
    return st["out"], st["lse"]


# --------------------------------------------------------------------------- the library's calls
def _handles(st):
    """What a program makes once: the shape and the cache format, a workspace, the batch's shared prefixes."""
    if "desc" not in st:
        from prefix_cached_kv_radix_gb300 import api
        case = st["case"]
        st["desc"] = api.make_desc(api.RX_F32 if case["dtype"] == "f32" else api.RX_BF16, st["hq"], st["hkv"], st["d"],
                                   st["num_slots"], 1.0 / math.sqrt(st["d"]))
        st["q8"] = api.q8_desc(api.RX_Q8_INT8 if case["code"] == "int8" else api.RX_Q8_E4M3, case["block"], case["fixed"])
        st["groups"], nbytes = None, 0
        if case["op"] == "decode":
            if case["shared"]:
                st["groups"] = api.shared_groups_struct(1, _group_of(case), st["grp_indptr"], st["grp_members"], st["grp_len"],
                                                        case["shared"])
            nbytes = api.decode_q8_workspace_bytes(st["desc"], st["batch"], max(st["lens"]), st["groups"])
        elif case["op"] == "extend":
            nbytes = api.extend_q8_workspace_bytes(st["desc"], st["batch"], max(st["lens"]), st["r2t"].shape[1])
        st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
        st["api"] = api
    return st["api"]


def _own_run(st):
    api, op = _handles(st), st["case"]["op"]
    if op == "write":
        api.kv_pool_write_q8(st["desc"], st["q8"], st["batch"], st["prefix_slots"], st["prefix_indptr"], st["new_slots"],
                             st["qo_indptr"], st["k"], st["v"], st["k_pool"], st["v_pool"], st["scales"], st["r2t"], st["total"],
                             st["status"])
        return st["k_pool"], st["v_pool"], st["scales"], st["r2t"]
    if op == "read":
        api.kv_pool_read_q8(st["desc"], st["q8"], st["slots"], st["k_pool"], st["v_pool"], st["scales"], st["k_out"], st["v_out"],
                            st["status"])
        return st["k_out"], st["v_out"]
    if op == "decode":
        api.decode_attention_q8(st["desc"], st["q8"], st["batch"], st["q"], st["r2t"], st["kv_lens"], st["k_pool"], st["v_pool"],
                                st["scales"], st["out"], st["lse"], max(st["lens"]), st["ws"], st["status"], groups=st["groups"])
    else:
        api.prefix_extend_attention_q8(st["desc"], st["q8"], st["batch"], st["q"], st["qo_indptr"], st["prefix_lens"], st["r2t"],
                                       st["k_pool"], st["v_pool"], st["scales"], st["out"], st["lse"], max(st["lens"]), st["ws"],
                                       st["status"])
    return st["out"], st["lse"]


def run(state):
    if own:
        return _own_run(state)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "extend": _plain_extend}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the least there is to do
def work(case):
    hq, hkv, d = SHAPES[case["shape"]]
    size = 4 if case["dtype"] == "f32" else 2
    cached = 2 * hkv * d                                     # a slot's codes

    def scales(slots):                                       # one for each block, or each slot where blocks are not dense
        return 8 * hkv * slots

    if case["op"] == "write":
        lens, pre = _new_lens(case), _prefix_lens(case)
        T = sum(lens)
        stride = _stride(max(p + n for p, n in zip(pre, lens)))
        index = 4 * sum(pre) + 4 * T + 4 * len(lens) * stride + 16 * len(lens)
        return {"bytes": T * cached * (size + 1) + scales(T) + index, "flops": 2 * T * cached}
    if case["op"] == "read":
        return {"bytes": case["slots"] * (cached * (size + 1) + 4) + scales(case["slots"]), "flops": case["slots"] * cached}
    if case["op"] == "decode":
        lens, m = _spread(case, case["seqs"], case["least"], case["ctx"]), _group_of(case)
        keys = sum(lens) - (m - 1) * case["shared"] if m else sum(lens)
        return {"bytes": keys * cached + scales(keys) + 4 * sum(lens) + len(lens) * hq * (2 * d * size + 4),
                "flops": 4 * d * hq * sum(lens)}
    lens, pre = _new_lens(case), _prefix_lens(case)
    keys = sum(lens) + sum(pre)
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(pre, lens))
    return {"bytes": keys * (cached + 4) + scales(keys) + sum(lens) * hq * (2 * d * size + 4), "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------- in 64 bits
def _power_of_two(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def exact(case, seed):
    st = prepare(case, seed)
    code, block, hq, hkv, d = case["code"], case["block"], st["hq"], st["hkv"], st["d"]
    if case["op"] == "write":
        out, slots = [], st["new_slots"].long()
        scales = st["scales"].double()
        for j, (name, x) in enumerate((("k_pool", st["k"]), ("v_pool", st["v"]))):
            x = x.double()
            if case["fixed"]:
                s = scales[:, :, j].index_select(0, torch.div(slots, block, rounding_mode="floor"))
            else:
                top = torch.linalg.vector_norm(x, math.inf, dim=-1)
                if code == "int8":
                    s = torch.maximum(top / 127.0, torch.full_like(top, 2.0 ** -126)).to(torch.float32).double()
                else:
                    top = torch.maximum(top, torch.full_like(top, 448.0 * 2.0 ** -126))
                    s = _power_of_two(torch.floor(torch.log2(top / 448.0)) - 1)
                    for _ in range(2):                       # a power of two at most as large, to the first that is large enough
                        s = torch.where(s * 448.0 < top, s * 2.0, s)
                scales[:, :, j].index_copy_(0, slots, s)
            y = torch.clamp(x / s.unsqueeze(-1), -LARGEST[code], LARGEST[code])
            if code == "int8":
                pool = st[name].clone()
                pool.index_copy_(0, slots, torch.round(y).to(torch.int8))
            else:                                            # eight steps in each power of two down to 2^-6, and those of 2^-6 below
                step = _power_of_two(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                pool = st[name].double()
                pool.index_copy_(0, slots, torch.round(y / step) * step)
            out.append(pool)
        return out[0], out[1], scales, None
    if case["op"] == "read":
        got, slots = [], st["slots"].long()
        for j, name in enumerate(("k_pool", "v_pool")):
            s = st["scales"][:, :, j].double().index_select(0, torch.div(slots, block, rounding_mode="floor"))
            got.append(st[name].double().index_select(0, slots) * s.unsqueeze(-1))
        return tuple(got)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b in range(st["batch"]):
        new, old = (1, st["lens"][b] - 1) if case["op"] == "decode" else (st["lens"][b], st["pre"][b])
        slots = st["r2t"][b, :old + new].long()
        where = torch.div(slots, block, rounding_mode="floor")
        key, val = (st[name].view(torch.uint8).index_select(0, slots).view(CODES[code]).double()
                    * st["scales"][:, :, j].index_select(0, where).double().unsqueeze(-1) for j, name in enumerate(("k_pool", "v_pool")))
        ask = st["q"][at:at + new].double() / math.sqrt(d)
        for h in range(hkv):
            rows = ask[:, h * (hq // hkv):(h + 1) * (hq // hkv)]
            s = torch.einsum("igd,jd->gij", rows, key[:, h])
            if new > 1:
                s.masked_fill_(torch.ones(new, old + new, dtype=torch.bool, device="cuda").triu(old + 1), -math.inf)
            z = torch.logsumexp(s, -1)
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            lse[at:at + new, heads] = z.t()
            out[at:at + new, heads] = torch.einsum("gij,jd->igd", torch.exp(s - z[..., None]), val[:, h])
        at += new
    return out, lse
