"""The operators of a generation step that surround attention and the experts,
as cases that can be measured: the norms around a block with its gate and
residual, the layout of a batch over the paged cache, beam search's selection
over beams and vocabulary, and the reordering of the cache's rows after it.

`run` computes a case in its plain form (elementary torch operations, 32 bits,
64 where scores of different beams are compared) or, where `own` is true, by
the calls a user makes of the library.

Layout of the cache (the library's definition, include/ft_kv.h): a page is one
complete record [L][2][Hkv][page][D] of 16-bit values; row r of the table lists
the pages of sequence r in order, -1 beyond them; lens[r] is the number of its
tokens; refs[p] counts the rows that hold page p.  The three arrays are one
int32 buffer here, so that a pass can start from the same control state each
time with one copy.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # ---- norms around a block
        # one token of a decode step, after attention's output projection: latency
        {"name": "norm_one", "op": "norm", "T": 1, "H": 2048, "block": "bf16", "resid": "f32", "out": "bf16", "post": False,
         "gate": "none"},
        # a decode batch with a norm on both sides of the block and a gate for each channel
        {"name": "norm_decode", "op": "norm", "T": 67, "H": 4096, "block": "bf16", "resid": "f32", "out": "bf16",
         "post": True, "gate": "channel"},
        # a prompt chunk of odd length whose residual stream is kept in 16 bits, gated value by value
        {"name": "norm_prompt_16", "op": "norm", "T": 4001, "H": 2048, "block": "f16", "resid": "f16", "out": "f16",
         "post": True, "gate": "full"},
        # a prompt chunk after the experts, whose sum is fp32: bandwidth
        {"name": "norm_prompt", "op": "norm", "T": 8192, "H": 4096, "block": "f32", "resid": "f32", "out": "bf16",
         "post": False, "gate": "none"},
        # ---- layout of a batch
        # a decode step of 64 requests, one token each: latency
        {"name": "batch_decode", "op": "batch", "B": 64, "n": 1, "tokens": 2000, "page": 64, "pad": 0},
        # as many requests as a plan takes, drafts of up to four tokens, padded to a fixed size
        {"name": "batch_drafts", "op": "batch", "B": 1024, "n": 4, "tokens": 700, "page": 16, "pad": 300},
        # prompts of a prefill step
        {"name": "batch_prompts", "op": "batch", "B": 9, "n": 9000, "tokens": 4000, "page": 64, "pad": 7},
        # ---- beam search's selection
        # one request of four beams over a small vocabulary: latency
        {"name": "select_one", "op": "select", "B": 1, "K": 4, "N": 4, "V": 32000, "type": "f32", "ended": False},
        # a batch whose rows start anywhere, twice as many candidates as beams, some beams ended, some tokens forbidden
        {"name": "select_batch", "op": "select", "B": 16, "K": 4, "N": 8, "V": 100003, "type": "bf16", "ended": True},
        # a large batch: bandwidth
        {"name": "select_large", "op": "select", "B": 128, "K": 8, "N": 8, "V": 131072, "type": "bf16", "ended": False},
        # ---- reordering of the cache's rows
        # one request of four beams in a cache of eight layers
        {"name": "reorder_4", "op": "reorder", "B": 1, "K": 4, "tokens": 1000, "L": 8, "Hkv": 4, "D": 128, "page": 64,
         "type": "bf16"},
        # 32 requests of eight beams
        {"name": "reorder_256", "op": "reorder", "B": 32, "K": 8, "tokens": 2000, "L": 4, "Hkv": 4, "D": 64, "page": 32,
         "type": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "batch", "select", "select", "reorder"])
    if op == "norm":
        dt = rng.choice(["bf16", "f16"])
        c = {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 8, 1024), "block": rng.choice([dt, dt, "f32"]),
             "resid": rng.choice([dt, "f32"]), "out": rng.choice([dt, dt, "f32"]), "post": rng.choice([False, True]),
             "gate": rng.choice(["none", "none", "channel", "token", "full"])}
        while c["T"] * c["H"] > 1 << 24:
            c["T"] = max(1, c["T"] // 2)
        return c
    if op == "batch":
        B = _log(rng, 1, 1024)
        n = rng.choice([1, 1, 5, _log(rng, 1, max(1, 40000 // B))])
        return {"op": op, "B": B, "n": n, "tokens": _log(rng, 1, 4000), "page": rng.choice([16, 32, 64, 128]),
                "pad": rng.choice([0, rng.randint(1, 500)])}
    if op == "select":
        K = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c = {"op": op, "B": _log(rng, 1, 64), "K": K, "N": rng.choice([K, K, 2 * K, rng.randint(1, 32)]),
             "V": _log(rng, 1000, 200000), "type": rng.choice(["bf16", "f16", "f32"]), "ended": rng.choice([False, True])}
        while c["B"] * K * c["V"] > 1 << 26:
            c["B"] = max(1, c["B"] // 2)
            if c["B"] == 1:
                break
        return c
    c = {"op": op, "B": _log(rng, 1, 32), "K": rng.choice([2, 3, 4, 8, 16]), "tokens": _log(rng, 2, 2000), "L": rng.randint(1, 8),
         "Hkv": rng.choice([1, 2, 4]), "D": rng.choice([64, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
         "type": rng.choice(["bf16", "f16"])}
    while _pages(c) * _page_values(c) > 1 << 29:
        if c["L"] > 1:
            c["L"] //= 2
        elif c["B"] > 1:
            c["B"] //= 2
        else:
            c["tokens"] //= 2
    return c


# ------------------------------------------------------------------ what a case fixes

def _rnd(case):
    """The case's own random stream: its lengths and lists are part of the case, not of the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _batch_lengths(case):
    """(tokens held, tokens added) of each request; rows that are new or add nothing among them."""
    r = _rnd(case)
    held = [r.randint(0, case["tokens"]) for _ in range(case["B"])]
    add = [case["n"] if b == 0 or case["n"] == 1 else r.randint(0, case["n"]) for b in range(case["B"])]
    return held, add


def _ceil(a, b):
    return -(-a // b)


def _batch_pages(case):
    """Pages that the requests hold before and after."""
    held, add = _batch_lengths(case)
    return sum(_ceil(h, case["page"]) for h in held), sum(_ceil(h + a, case["page"]) for h, a in zip(held, add))


def _lineage(case):
    """(length of each request, how much of it all its beams share, each row's parent): the beams of a request
    have one length; after a step about half of them go on and the rest start anew from those."""
    r = _rnd(case)
    B, K = case["B"], case["K"]
    lens = [r.randint(max(1, case["tokens"] // 2), case["tokens"]) for _ in range(B)]
    shared = [n // 2 // case["page"] * case["page"] for n in lens]
    parents = [b * K + min(K - 1, int(r.random() ** 2 * K)) for b in range(B) for _ in range(K)]
    return lens, shared, parents


def _copies(case):
    """Tokens copied: of each parent's last page, one child keeps the place and the others get a copy."""
    lens, _, parents = _lineage(case)
    return sum(lens[p // case["K"]] % case["page"] for p in parents) - \
        sum(lens[p // case["K"]] % case["page"] for p in set(parents))


def _pages(case):
    """Pages of a reorder case: a child's last page may need a place while its old row's is still held by nobody else."""
    lens, shared, _ = _lineage(case)
    P, K = case["page"], case["K"]
    return sum(s // P + K * (_ceil(n, P) - s // P) for n, s in zip(lens, shared)) + case["B"] * K + 5


def _page_values(case):
    return case["L"] * 2 * case["Hkv"] * case["page"] * case["D"]


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        size = {k: _DT[case[k]].itemsize for k in ("block", "resid", "out")}
        gate = {"none": 0, "channel": H * 2, "token": T * 4, "full": T * H * size["block"]}[case["gate"]]
        per = size["block"] + 2 * size["resid"] + size["out"]
        return {"bytes": T * H * per + gate + (2 if case["post"] else 1) * H * 2, "flops": T * H * (12 if case["post"] else 7)}
    if case["op"] == "batch":
        held, add = _batch_lengths(case)
        before, after = _batch_pages(case)
        T, B = sum(add) + case["pad"], case["B"]
        # list, lengths read and written, prefix sums; three arrays of the tokens; table entries and counts of new pages
        return {"bytes": B * 20 + T * 16 + (after - before) * 12, "flops": 0}
    if case["op"] == "select":
        R, V = case["B"] * case["K"], case["V"]
        return {"bytes": R * V * _DT[case["type"]].itemsize + R * 8 + case["B"] * case["N"] * 16, "flops": R * V * 4}
    lens, _, parents = _lineage(case)
    K = case["K"]
    # copied tokens read and written; the entries of the rows that change, read and written
    moved = sum(_ceil(lens[p // K], case["page"]) for i, p in enumerate(parents) if p != i)
    return {"bytes": _copies(case) * (_page_values(case) // case["page"]) * 4 + moved * 8 + len(parents) * 12, "flops": 0}


# ------------------------------------------------------------------ inputs

class _State:
    pass


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(gen, shape, dt, scale=1.0):
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda") * scale)
    return out


def _cache(s, L, Hkv, D, page, n_pages, row_pages, table, lens, dt):
    """Control arrays from Python lists and, where the library is asked for, its handle on them."""
    rows = len(table)
    s.rows, s.row_pages, s.n_pages, s.page = rows, row_pages, n_pages, page
    refs, full = [0] * n_pages, []
    for r in table:
        full.append(list(r) + [-1] * (row_pages - len(r)))
        for p in r:
            refs[p] += 1
    s.ctl0 = _ints([p for r in full for p in r] + list(lens) + refs)
    s.ctl = s.ctl0.clone()
    a, b = rows * row_pages, rows * row_pages + rows
    s.table, s.lens, s.refs = s.ctl[:a].view(rows, row_pages), s.ctl[a:b], s.ctl[b:]
    s.pv = s.pool.view(n_pages, L, 2, Hkv, page, D)
    if own:
        import moe_expert_cache_gb300 as ft
        s.kv = ft.KvCache(L, Hkv, Hkv, D, page, n_pages, rows, row_pages, s.pool, s.table, s.lens, s.refs,
                          dtype=ft.FT_KV_BF16 if dt == torch.bfloat16 else ft.FT_KV_F16, T_max=1, B_max=1)


def prepare(case, seed):
    s = _State()
    s.case = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = random.Random(seed)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # weights in 16 bits, of the type that the call's other 16-bit values have
        w = _DT[next((case[k] for k in ("block", "resid", "out") if case[k] != "f32"), "bf16")]
        s.block = _normal(gen, (T, H), _DT[case["block"]], 1.5)
        s.resid = _normal(gen, (T, H), _DT[case["resid"]], 4.0)
        # a few channels of the residual stream are much larger than the rest, as in trained models
        s.resid[:, torch.randint(0, H, (max(1, H // 500),), generator=gen, device="cuda")] *= 30
        s.post = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(w) if case["post"] else None
        s.pre = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(w)
        s.gate = {"none": lambda: None, "channel": lambda: _normal(gen, (H,), w, 0.5),
                  "token": lambda: torch.rand(T, generator=gen, device="cuda"),
                  "full": lambda: _normal(gen, (T, H), _DT[case["block"]], 0.5)}[case["gate"]]()
        s.h = torch.empty_like(s.resid)
        s.y = torch.empty(T, H, dtype=_DT[case["out"]], device="cuda")
        s.eps, s.rs, s.bs = 1e-6, 1.0, 0.7
        if own:
            import moe_expert_cache_gb300 as ft
            t = {torch.bfloat16: ft.FT_T_BF16, torch.float16: ft.FT_T_F16, torch.float32: ft.FT_T_F32}
            s.norm = ft.BlockNorm(H, pre=s.pre, post=s.post, w_type=t[w], block_type=t[s.block.dtype], resid_type=t[s.resid.dtype],
                                  out_type=t[s.y.dtype], eps=s.eps, resid_scale=s.rs, block_scale=s.bs,
                                  gate={"none": ft.FT_GATE_NONE, "channel": ft.FT_GATE_CHANNEL, "token": ft.FT_GATE_TOKEN,
                                        "full": ft.FT_GATE_FULL}[case["gate"]],
                                  gate_type=ft.FT_T_F32 if s.gate is None else t[s.gate.dtype])
    elif case["op"] == "batch":
        held, add = _batch_lengths(case)
        page = case["page"]
        before, after = _batch_pages(case)
        n_pages = after + 11
        ids = list(range(n_pages))
        rnd.shuffle(ids)
        table, at = [], 0
        for h in held:
            table.append(ids[at:at + _ceil(h, page)])
            at += _ceil(h, page)
        # the rows that the requests use are some of the table's, in any order
        spare = 3
        where = rnd.sample(range(case["B"] + spare), case["B"])
        rows, lens = [[] for _ in range(case["B"] + spare)], [0] * (case["B"] + spare)
        for b, r in enumerate(where):
            rows[r], lens[r] = table[b], held[b]
        s.pool = torch.zeros(n_pages * 2 * page * 64, dtype=torch.bfloat16, device="cuda")
        _cache(s, 1, 1, 64, page, n_pages, max(_ceil(h + a, page) for h, a in zip(held, add)) + 1, rows, lens, torch.bfloat16)
        s.where, s.add = _ints(where), _ints(add)
        s.T = sum(add) + case["pad"]
        s.cu = torch.empty(case["B"] + 1, dtype=torch.int32, device="cuda")
        s.row_of, s.pos = (torch.empty(s.T, dtype=torch.int32, device="cuda") for _ in range(2))
        s.slots = torch.empty(s.T, dtype=torch.int64, device="cuda")
    elif case["op"] == "select":
        B, K, N, V = case["B"], case["K"], case["N"], case["V"]
        R = B * K
        dt = _DT[case["type"]]
        s.logits = _normal(gen, (R, V), dt, 2.5)
        # a few likely tokens a row, as a trained model has
        hot = torch.randperm(V, generator=gen, device="cuda")[:20]
        s.logits[:, hot] += (6 + 3 * torch.randn(R, 20, generator=gen, device="cuda")).to(dt)
        s.scores = -20 * torch.rand(R, generator=gen, device="cuda") / (1 + K)
        s.eos, s.done = -1, None
        if case["ended"]:
            s.eos = V // 3
            s.done = (torch.rand(R, generator=gen, device="cuda") < 0.2).int()
            # a grammar forbids a third of the tokens of every other row
            for i in range(0, R, 2):
                s.logits[i, torch.rand(V, generator=gen, device="cuda") < 0.33] = -math.inf
        s.out = [torch.empty(B, N, dtype=torch.float32, device="cuda")] + \
            [torch.empty(B, N, dtype=torch.int32, device="cuda") for _ in range(3 if case["ended"] else 2)]
        if own:
            import moe_expert_cache_gb300 as ft
            s.beams = ft.Beams(V, R, N, dtype={"bf16": ft.FT_T_BF16, "f16": ft.FT_T_F16, "f32": ft.FT_T_F32}[case["type"]])
    else:
        lens, shared, parents = _lineage(case)
        page, K, dt = case["page"], case["K"], _DT[case["type"]]
        n_pages = _pages(case)
        s.pool = _normal(gen, n_pages * _page_values(case), dt)
        ids = list(range(n_pages))
        rnd.shuffle(ids)
        table, at = [], 0
        for n, sh in zip(lens, shared):
            common = ids[at:at + sh // page]
            at += sh // page
            for _ in range(K):
                mine = _ceil(n, page) - sh // page
                table.append(common + ids[at:at + mine])
                at += mine
        _cache(s, case["L"], case["Hkv"], case["D"], page, n_pages, max(map(len, table)) + 1, table,
               [n for n in lens for _ in range(K)], dt)
        s.parents = _ints(parents)
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c = s.case
    if c["op"] == "norm":
        H = c["H"]
        s.norm.forward(c["T"], s.resid, H, block=s.block, ld_b=H, gate=s.gate, ld_g=H, resid_out=s.h, ld_ro=H, out=s.y, ld_o=H)
        return [s.h, s.y]
    if c["op"] == "select":
        s.beams.select(c["B"], c["K"], c["N"], s.logits, c["V"], s.scores, s.out[0], s.out[1], s.out[2], done=s.done,
                       eos=s.eos, out_done=s.out[3] if c["ended"] else None)
        return s.out
    s.ctl.copy_(s.ctl0)
    if c["op"] == "batch":
        s.kv.batch(c["B"], s.add, s.T, s.cu, s.row_of, s.pos, rows=s.where, slots=s.slots)
        return [s.table, s.lens, s.refs, s.cu, s.row_of, s.pos, s.slots]
    s.kv.reorder(c["B"] * c["K"], s.parents)
    return [s.table, s.lens, s.refs, s.pool]


def _run_plain(s):
    c = s.case
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "select":
        return _plain_select(s, c)
    s.ctl.copy_(s.ctl0)
    if c["op"] == "batch":
        return _plain_batch(s)
    return _plain_reorder(s)


def _plain_norm(s):
    z = s.block.float()
    if s.post is not None:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + s.eps) * s.post.float()
    if s.gate is not None:
        g = s.gate.float()
        z = z * (g[:, None] if s.case["gate"] == "token" else g)
    h = s.rs * s.resid.float() + s.bs * z
    s.h.copy_(h)
    s.y.copy_(h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s.eps) * s.pre.float())
    return [s.h, s.y]


def _plain_batch(s):
    page, rows = s.page, s.where.long()
    old, add = s.lens[rows].long(), s.add.long()
    have, want = (old + page - 1) // page, (old + add + page - 1) // page
    free = (s.refs == 0).nonzero().flatten()
    col = torch.arange(s.row_pages, device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = fresh.flatten().long().cumsum(0).view_as(fresh) - 1
    new = free[at.clamp(min=0, max=len(free) - 1)].int()
    s.table[rows] = torch.where(fresh, new, s.table[rows])
    s.refs[new[fresh].long()] = 1
    s.lens[rows] = (old + add).int()
    end = add.cumsum(0)
    s.cu[0] = 0
    s.cu[1:] = end
    t = torch.arange(s.T, device="cuda")
    b = (t[:, None] >= end[None, :]).sum(1)
    there = b < len(end)
    b = b.clamp(max=len(end) - 1)
    p = torch.where(there, old[b] + t - (end[b] - add[b]), 0)
    r = torch.where(there, rows[b], -1)
    pg = s.table[r.clamp(min=0), p // page].long()
    s.row_of.copy_(r)
    s.pos.copy_(p)
    s.slots.copy_(torch.where(there, pg * page + p % page, -1))
    return [s.table, s.lens, s.refs, s.cu, s.row_of, s.pos, s.slots]


def _plain_select(s, c):
    B, K, N, V = c["B"], c["K"], c["N"], c["V"]
    x = s.logits.double()
    m = x.amax(-1, keepdim=True)
    x -= m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    x += s.scores.double()[:, None]
    if s.done is not None:
        ended = s.done != 0
        x[ended] = -math.inf
        x[ended, s.eos] = s.scores.double()[ended]
    best, at = torch.sort(x.view(B, K * V), dim=-1, descending=True, stable=True)  # equal scores stay in order
    best, at = best[:, :N], at[:, :N]
    there = best > -math.inf
    beam = at // V + K * torch.arange(B, device="cuda")[:, None]
    s.out[0].copy_(best)
    s.out[1].copy_(torch.where(there, beam, -1))
    s.out[2].copy_(torch.where(there, at % V, -1))
    if s.done is not None:
        s.out[3].copy_(there & ((s.done[beam] != 0) | (at % V == s.eos)))
    return s.out


def _plain_reorder(s):
    page, n = s.page, s.rows
    me, parent = torch.arange(n, device="cuda"), s.parents.long()
    length = s.lens[parent].long()
    full, part = length // page, length % page
    # the child that keeps its parent's last page: the parent's own row if it goes on, else the first in the list
    keeper = torch.full((n,), n, device="cuda").scatter_reduce(0, parent, torch.where(parent == me, -1, me), "amin")
    keeps = (keeper[parent] == me) | (parent == me)
    need = (part > 0) & ~keeps
    old, new = s.table.clone(), s.table[parent]
    col = torch.arange(s.row_pages, device="cuda")[None, :]
    new = torch.where(col < (full + ((part > 0) & keeps).long())[:, None], new, -1)
    s.refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    s.refs.index_add_(0, new.clamp(min=0).flatten().long(), (new >= 0).flatten().int())
    free = (s.refs == 0).nonzero().flatten()
    page_of = free[(need.long().cumsum(0) - 1).clamp(min=0)]
    src = old[parent[need], full[need]].long()
    new[me[need], full[need]] = page_of[need].int()
    s.refs[page_of[need]] = 1
    s.table.copy_(new)
    s.lens.copy_(length)
    tok = torch.arange(page, device="cuda")[None, None, None, None, :, None] < part[need][:, None, None, None, None, None]
    s.pv[page_of[need]] = torch.where(tok, s.pv[src], s.pv[page_of[need]])
    return [s.table, s.lens, s.refs, s.pool]


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """What the definition gives in 64 bits; tables, counts and maps are whole numbers and have no other value."""
    if case["op"] == "batch":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        def unit(v):  # a row over its root mean square
            return v / torch.sqrt(torch.einsum("th,th->t", v, v) / v.shape[1] + s.eps)[:, None]

        h, y = [], []
        for t in range(0, case["T"], 1024):
            e = slice(t, t + 1024)
            a = s.block[e].double()
            if s.post is not None:
                a = torch.einsum("th,h->th", unit(a), s.post.double())
            if case["gate"] == "channel":
                a = torch.einsum("th,h->th", a, s.gate.double())
            elif case["gate"] == "token":
                a = torch.einsum("th,t->th", a, s.gate[e].double())
            elif case["gate"] == "full":
                a = a * s.gate[e].double()
            h.append(torch.add(s.resid[e].double() * s.rs, a, alpha=s.bs))
            y.append(torch.einsum("th,h->th", unit(h[-1]), s.pre.double()))
        return [torch.cat(h), torch.cat(y)]
    if case["op"] == "reorder":
        # row by row from lists of pages
        table, lens, parents = s.table.tolist(), s.lens.tolist(), s.parents.tolist()
        held = [[p for p in r if p >= 0] for r in table]
        pool = s.pv.double()
        took, rows, wanting = set(), [], []
        order = [i for i in range(len(held)) if parents[i] == i] + [i for i in range(len(held)) if parents[i] != i]
        keeps = {i for i in order if parents[i] not in took and not took.add(parents[i])}
        for i, p in enumerate(parents):
            whole, rest = divmod(lens[p], s.page)
            rows.append(held[p] if i in keeps else held[p][:whole])
            if rest and i not in keeps:
                wanting.append((held[p][whole], rest))
        used = {p for r in rows for p in r}
        free = (p for p in range(s.n_pages) if p not in used)
        for src, rest in wanting:
            pool[next(free), ..., :rest, :] = s.pv[src, ..., :rest, :].double()
        return [None, None, None, pool.view(-1)]
    B, K, N, V = (case[k] for k in "BKNV")
    rows = []
    for b in range(B):
        # the N best of each beam by their logits, then the N best of those; equal ones by beam, then by token
        found = []
        for i in range(b * K, (b + 1) * K):
            base = float(s.scores[i].double())
            if case["ended"] and bool(s.done[i]):
                found.append((-base, i, s.eos, 1))
                continue
            x = s.logits[i].double()
            at = ((x >= torch.topk(x, min(N, V)).values[-1]) & (x > -math.inf)).nonzero().flatten()
            base -= float(torch.logsumexp(x, 0))
            found += [(-(base + u), i, v, int(v == s.eos)) for u, v in zip(x[at].tolist(), at.tolist())]
        found = sorted(found)[:N]
        rows.append(found + [(math.inf, -1, -1, 0)] * (N - len(found)))
    out = [torch.tensor([[-f[0] for f in r] for r in rows], dtype=torch.float64, device="cuda")]
    out += [torch.tensor([[f[j] for f in r] for r in rows], dtype=torch.int32, device="cuda") for j in (1, 2, 3)]
    return out if case["ended"] else out[:3]
