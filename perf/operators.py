"""The paged key/value cache's operators as cases that can be measured: the
norm-rotate-store pass, attention over a page table with a shared prefix, and
the page operations (extend, fork, free, compact).

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, where `own` is true, by the calls a user makes of the library.

Layout of the cache (the library's definition, include/ft.h): a page is one
complete record [L][2][Hkv][page][D] of 16-bit values (K then V of every
layer); row r of the table lists the pages of sequence r in order, -1 beyond
them; lens[r] is the number of its tokens; refs[p] counts the rows that hold
page p.  The three arrays are one int32 buffer here, so that a pass can start
from the same control state each time with one copy.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # ---- norm, rotation and store
        # one token of one request in a decode step: pure latency
        {"name": "rope_one", "op": "rope", "T": 1, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "rot": 128, "form": "half",
         "type": "bf16"},
        # a decode batch with wide heads of which a quarter is rotated
        {"name": "rope_batch_d256", "op": "rope", "T": 129, "Hq": 16, "Hkv": 2, "D": 256, "page": 32, "rot": 64,
         "form": "half", "type": "f16"},
        # a prompt chunk of odd length: bandwidth
        {"name": "rope_prompt", "op": "rope", "T": 8191, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "rot": 128,
         "form": "half", "type": "bf16"},
        # ---- attention
        # one request, one token, about a thousand keys: the smallest call, latency
        {"name": "attn_one", "op": "attn", "B": 1, "n": 1, "prefix": 0, "tail": 1023, "Hq": 32, "Hkv": 4, "D": 128, "page": 64,
         "type": "bf16"},
        # decode of 64 requests behind one 8192-token system prompt, own parts of 1..512 tokens
        {"name": "attn_decode_64", "op": "attn", "B": 64, "n": 1, "prefix": 8192, "tail": 512, "Hq": 32, "Hkv": 4, "D": 128,
         "page": 64, "type": "bf16"},
        # checking drafts of up to 5 tokens, small heads in threes, small pages
        {"name": "attn_draft_d64", "op": "attn", "B": 23, "n": 5, "prefix": 4000, "tail": 700, "Hq": 24, "Hkv": 8, "D": 64,
         "page": 16, "type": "f16"},
        # a few agents over one very long document
        {"name": "attn_long", "op": "attn", "B": 6, "n": 1, "prefix": 131072, "tail": 2500, "Hq": 32, "Hkv": 4, "D": 128,
         "page": 128, "type": "bf16"},
        # a large decode batch with wide heads
        {"name": "attn_decode_d256", "op": "attn", "B": 130, "n": 1, "prefix": 16384, "tail": 1000, "Hq": 16, "Hkv": 2,
         "D": 256, "page": 32, "type": "bf16"},
        # prompts of up to 4000 tokens behind a shared prefix: compute
        {"name": "attn_prompt", "op": "attn", "B": 3, "n": 4000, "prefix": 8192, "tail": 4000, "Hq": 32, "Hkv": 4, "D": 128,
         "page": 64, "type": "bf16"},
        # ---- pages
        # a request splits into four samples: three forks of one partial page each
        {"name": "pages_fork_4", "op": "fork", "n": 3, "tokens": 1000, "L": 8, "Hkv": 4, "D": 128, "page": 64, "pages": 512,
         "type": "bf16"},
        # a beam step over 64 rows: half the rows are dropped, forked anew from the others, and every row grows by a token
        {"name": "pages_beam_64", "op": "beam", "n": 64, "tokens": 2000, "L": 24, "Hkv": 4, "D": 64, "page": 32, "pages": 4099,
         "type": "f16"},
        # the pool is compacted so that its upper part can be given back: a third of the live pages moves
        {"name": "pages_compact", "op": "compact", "n": 100, "live": 1733, "moved": 601, "L": 8, "Hkv": 4, "D": 128, "page": 64,
         "pages": 2999, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "fork", "beam", "compact"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "f16"])}
    if op == "rope":
        c.update(T=_log(rng, 1, 8191), Hq=Hkv * rng.randint(1, 8), rot=16 * rng.randint(1, D // 16),
                 form=rng.choice(["half", "pair"]))
    elif op == "attn":
        c.update(Hq=Hkv * rng.randint(1, 8))
        if rng.random() < 0.25:  # prompts
            n = _log(rng, 16, 3000)
            c.update(B=rng.randint(1, 3), n=n, tail=n + rng.randint(0, 500))
        else:
            n = rng.choice([1, 1, 1, 2, 3, 8])
            c.update(B=_log(rng, 1, 128), n=n, tail=max(n, _log(rng, 1, 2500)))
        c["prefix"] = rng.choice([0, 1, 1, 1]) * c["page"] * (_log(rng, 16, 32768) // c["page"])
        while work(c)["flops"] > 4e11 or c["B"] * c["tail"] * Hkv * D > 1 << 28:
            c["B"] = max(1, c["B"] // 2)
            c["prefix"] = c["prefix"] // 2 // c["page"] * c["page"]
    else:
        c["L"] = rng.randint(1, 8)
        if op == "compact":
            live = _log(rng, 2, 1000)
            moved = rng.randint(1, max(1, live // 2))
            c.update(n=rng.randint(1, 64), live=live, moved=moved, pages=live + moved + rng.randint(0, 300))
        elif op == "fork":
            c.update(n=_log(rng, 1, 64), tokens=_log(rng, 1, 4000))
            c["pages"] = -(-c["tokens"] // c["page"]) + c["n"] + rng.randint(0, 200)
        else:
            c.update(n=rng.randint(2, 64), tokens=_log(rng, 2, 1000))
            c["pages"] = c["n"] * (c["tokens"] // c["page"] + 3) + rng.randint(0, 100)
        while c["L"] > 1 and c["pages"] * _page_values(c) > 1 << 30:
            c["L"] -= 1
        while c["pages"] * _page_values(c) > 1 << 30:
            c["D"] //= 2
            c["page"] = max(16, c["page"] // 2) if op == "compact" else c["page"]
            if c["D"] < 64:
                c["D"], c["Hkv"] = 64, max(1, c["Hkv"] // 2)
    return c


# ------------------------------------------------------------------ what a case fixes

def _rnd(case):
    """The case's own random stream: its lengths are part of the case, not of the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _attn_lengths(case):
    """(queries, total length) of each request; the first has the case's largest ones."""
    r = _rnd(case)
    q, lens = [], []
    for b in range(case["B"]):
        n = case["n"] if b == 0 else r.randint(max(1, case["n"] // 2), case["n"])
        own_part = case["tail"] if b == 0 else r.randint(n, max(n, case["tail"]))
        q.append(n)
        lens.append(case["prefix"] + own_part)
    return q, lens


def _beam_rows(case):
    """(lengths of all rows, dropped rows, the row each of them is forked from anew)."""
    r = _rnd(case)
    n = case["n"]
    lens = [r.randint(max(1, case["tokens"] // 2), case["tokens"]) for _ in range(n)]
    drop = r.sample(range(n), n // 2)
    keep = [i for i in range(n) if i not in set(drop)]
    return lens, drop, [r.choice(keep) for _ in drop]


def _page_values(case):
    return case["L"] * 2 * case["Hkv"] * case["page"] * case["D"]


def work(case):
    D, page = case["D"], case["page"]
    if case["op"] == "rope":
        T, heads = case["T"], case["Hq"] + 2 * case["Hkv"]
        return {"bytes": T * heads * D * 4 + T * case["rot"] * 4 + T * 8, "flops": T * (case["Hq"] + case["Hkv"]) * (3 * D + 3 * case["rot"])}
    if case["op"] == "attn":
        q, lens = _attn_lengths(case)
        keys = case["prefix"] + sum(x - case["prefix"] for x in lens)  # distinct ones
        seen = sum(n * (x - n) + n * (n + 1) // 2 for n, x in zip(q, lens))
        return {"bytes": keys * 2 * case["Hkv"] * D * 2 + 2 * sum(q) * case["Hq"] * D * 2, "flops": 4 * D * case["Hq"] * seen}
    pv, n = _page_values(case), case["n"]
    if case["op"] == "fork":
        return {"bytes": n * (case["tokens"] % page) * (pv // page) * 4 + n * (-(-case["tokens"] // page)) * 8, "flops": 0}
    if case["op"] == "beam":
        lens, drop, src = _beam_rows(case)
        return {"bytes": sum(lens[s] % page for s in src) * (pv // page) * 4 + sum(-(-lens[s] // page) for s in src) * 16, "flops": 0}
    return {"bytes": case["moved"] * pv * 4 + case["pages"] * 8 + case["live"] * 8, "flops": 0}


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dt, scale=1.0):
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda") * scale)
    return out


class _State:
    pass


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(s, case, L, Hq, n_pages, rows, row_pages, table, lens, T_max):
    """Control arrays from Python lists and, where the library is asked for, its handle on them."""
    s.rows, s.row_pages, s.n_pages, s.page = rows, row_pages, n_pages, case["page"]
    refs = [0] * n_pages
    full = []
    for r in table:
        full.append(list(r) + [-1] * (row_pages - len(r)))
        for p in r:
            refs[p] += 1
    s.ctl0 = _ints([p for r in full for p in r] + list(lens) + refs)
    s.ctl = s.ctl0.clone()
    a, b = rows * row_pages, rows * row_pages + rows
    s.table, s.lens, s.refs = s.ctl[:a].view(rows, row_pages), s.ctl[a:b], s.ctl[b:]
    s.pv = s.pool.view(n_pages, L, 2, case["Hkv"], case["page"], case["D"])
    if own:
        import moe_expert_cache_gb300 as ft
        s.kv = ft.KvCache(L, Hq, case["Hkv"], case["D"], case["page"], n_pages, rows, row_pages, s.pool, s.table, s.lens,
                          s.refs, dtype=ft.FT_KV_BF16 if case["type"] == "bf16" else ft.FT_KV_F16, T_max=T_max, B_max=rows)


def prepare(case, seed):
    s = _State()
    s.case = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = random.Random(seed)
    dt, page, D, Hkv = _DT[case["type"]], case["page"], case["D"], case["Hkv"]
    if case["op"] == "rope":
        # the tokens of a batch: a few requests, each with a run of new positions in a cache of two layers
        T, Hq = case["T"], case["Hq"]
        B = min(T, 3) if T > 256 else T
        per = [T // B + (1 if b < T % B else 0) for b in range(B)]
        own_rnd = _rnd(case)
        start = [own_rnd.randint(0, 500) for _ in range(B)]
        npg = [-(-(a + n) // page) for a, n in zip(start, per)]
        ids = list(range(sum(npg) + 3))
        rnd.shuffle(ids)
        table, at = [], 0
        for n in npg:
            table.append(ids[at:at + n])
            at += n
        s.pool = _normal(gen, len(ids) * 2 * 2 * Hkv * page * D, dt)
        _cache(s, case, 2, Hq, len(ids), B, max(npg), table, [a + n for a, n in zip(start, per)], T)
        s.layer = 1
        # 16 more columns than the heads need: the projection's output is one wider buffer
        s.ld = (Hq + 2 * Hkv) * D + 16
        s.qkv = _normal(gen, (T, s.ld), dt, 2.0)
        s.wq = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        s.wk = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        s.row_of = _ints([b for b, n in enumerate(per) for _ in range(n)])
        s.pos = _ints([a + i for a, n in zip(start, per) for i in range(n)])
        s.max_pos = max(a + n for a, n in zip(start, per))
        f = 1e6 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        ang = torch.arange(s.max_pos, device="cuda", dtype=torch.float64)[:, None] * f
        s.cs = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s.out = torch.empty(T, Hq * D, dtype=dt, device="cuda")
        s.eps = 1e-6
    elif case["op"] == "attn":
        Hq, P = case["Hq"], case["prefix"] // page
        s.q_lens, s.kv_lens = _attn_lengths(case)
        tails = [-(-x // page) - P for x in s.kv_lens]
        ids = list(range(P + sum(tails) + 2))
        rnd.shuffle(ids)
        table, at = [], P
        for n in tails:
            table.append(ids[:P] + ids[at:at + n])
            at += n
        T, B = sum(s.q_lens), case["B"]
        s.pool = _normal(gen, len(ids) * 2 * Hkv * page * D, dt)
        _cache(s, case, 1, Hq, len(ids), B, P + max(tails), table, s.kv_lens, T)
        s.layer = 0
        # keys have channels of their own size and mean, as cached keys do
        s.pv[:, 0, 0] *= (0.5 + torch.rand(D, generator=gen, device="cuda")).to(dt)
        s.pv[:, 0, 0] += torch.randn(D, generator=gen, device="cuda").to(dt)
        s.q = _normal(gen, (T, Hq * D), dt, 1.5)
        s.out = torch.empty(T, Hq * D, dtype=dt, device="cuda")
        s.scale = 1 / math.sqrt(D)
        cu = [0]
        for n in s.q_lens:
            cu.append(cu[-1] + n)
        s.cu, s.cu_q = cu, _ints(cu)
        s.group_start, s.group_tokens = _ints([0, B]), _ints([case["prefix"]])
        if own:  # a program plans once a step and calls each of its layers with that plan
            s.kv.attn_plan(B, T, s.cu_q, rows=None, n_groups=1, group_start=s.group_start, group_tokens=s.group_tokens)
    elif case["op"] in ("fork", "beam"):
        n_pages, L = case["pages"], case["L"]
        s.pool = _normal(gen, n_pages * _page_values(case), dt)
        ids = list(range(n_pages))
        rnd.shuffle(ids)
        if case["op"] == "fork":
            lens = [case["tokens"]] + [0] * case["n"]
            s.parents, s.children = _ints([0] * case["n"]), _ints(list(range(1, case["n"] + 1)))
        else:
            lens, drop, src = _beam_rows(case)
            s.children, s.parents = _ints(drop), _ints(src)
            s.grow, s.by = _ints(list(range(case["n"]))), _ints([1] * case["n"])
        npg = [-(-x // page) for x in lens]
        table, at = [], 0
        for n in npg:
            table.append(ids[at:at + n])
            at += n
        _cache(s, case, L, Hkv, n_pages, len(lens), max(npg) + 1, table, lens, 1)
    else:
        n_pages, L, live, moved = case["pages"], case["L"], case["live"], case["moved"]
        s.pool = _normal(gen, n_pages * _page_values(case), dt)
        ids = rnd.sample(range(live), live - moved) + rnd.sample(range(live, n_pages), moved)
        rnd.shuffle(ids)
        own_rnd = _rnd(case)
        cut = sorted(own_rnd.randint(0, live) for _ in range(case["n"] - 1))
        table = [ids[a:b] for a, b in zip([0] + cut, cut + [live])]
        # every fourth row shares the first pages of the one before it
        for i in range(3, len(table), 4):
            table[i] = table[i - 1][:len(table[i - 1]) // 2] + table[i]
        _cache(s, case, L, Hkv, n_pages, len(table), max(len(r) for r in table) or 1, table, [len(r) * page for r in table], 1)
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c = s.case
    if c["op"] == "rope":
        s.kv.qk_rope_store(s.layer, c["T"], s.qkv, s.ld, s.row_of, s.pos, s.out, c["Hq"] * c["D"], q_norm=s.wq, k_norm=s.wk,
                           eps=s.eps, cos_sin=s.cs, max_pos=s.max_pos, rot=c["rot"], pair=c["form"] == "pair")
        return [s.out, s.pool]
    if c["op"] == "attn":
        s.kv.attn_forward(s.layer, s.q, c["Hq"] * c["D"], s.out, c["Hq"] * c["D"], s.scale)
        return s.out
    s.ctl.copy_(s.ctl0)
    if c["op"] == "compact":
        s.kv.compact()
    else:
        if c["op"] == "beam":
            s.kv.free(len(s.children), s.children)
        s.kv.fork(len(s.children), s.parents, s.children)
        if c["op"] == "beam":
            s.kv.extend(c["n"], s.grow, s.by)
    return [s.table, s.lens, s.refs, s.pool]


def _run_plain(s):
    c = s.case
    if c["op"] == "rope":
        return _plain_rope(s, c)
    if c["op"] == "attn":
        return _plain_attn(s, c)
    s.ctl.copy_(s.ctl0)
    if c["op"] == "compact":
        _plain_compact(s)
    else:
        if c["op"] == "beam":
            _plain_free(s, s.children.long())
        _plain_fork(s, s.parents.long(), s.children.long())
        if c["op"] == "beam":
            _plain_extend(s, s.grow.long(), s.by.long())
    return [s.table, s.lens, s.refs, s.pool]


def _rotate(x, cs, rot, pair):
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if pair else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if pair else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s, c):
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    x = s.qkv[:, :(Hq + 2 * Hkv) * D].float().view(T, Hq + 2 * Hkv, D)
    cs = s.cs[s.pos.long()]

    def normed(h, w):
        return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s.eps) * w.float()

    pair = c["form"] == "pair"
    q = _rotate(normed(x[:, :Hq], s.wq), cs, c["rot"], pair)
    k = _rotate(normed(x[:, Hq:Hq + Hkv], s.wk), cs, c["rot"], pair)
    pos = s.pos.long()
    pg = s.table[s.row_of.long(), pos // s.page].long()
    s.pv[pg, s.layer, 0, :, pos % s.page] = k.to(s.pool.dtype)
    s.pv[pg, s.layer, 1, :, pos % s.page] = x[:, Hq + Hkv:].to(s.pool.dtype)
    s.out.copy_(q.reshape(T, Hq * D))
    return [s.out, s.pool]


def _plain_attn(s, c):
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    for b, (n, length) in enumerate(zip(s.q_lens, s.kv_lens)):
        pg = s.table[b, :-(-length // s.page)].long()
        k = s.pv[pg, s.layer, 0].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :length].float()
        v = s.pv[pg, s.layer, 1].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :length].float()
        step = max(1, (1 << 28) // (Hq * length))
        for i in range(0, n, step):
            m = min(step, n - i)
            t0 = s.cu[b] + i
            q = s.q[t0:t0 + m].float().view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D)
            x = (torch.bmm(q, k.transpose(1, 2)) * s.scale).view(Hkv, G, m, length)
            if n > 1:
                last = length - n + i + torch.arange(m, device="cuda")
                x = x.masked_fill(torch.arange(length, device="cuda")[None, :] > last[:, None], -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            x = x / x.sum(-1, keepdim=True)
            o = torch.bmm(x.view(Hkv, G * m, length), v)
            s.out[t0:t0 + m] = o.view(Hkv, G, m, D).permute(2, 0, 1, 3).reshape(m, Hq * D).to(s.out.dtype)
    return s.out


def _plain_free(s, rows):
    pg = s.table[rows]
    s.refs.index_add_(0, pg.clamp(min=0).flatten().long(), -(pg >= 0).flatten().int())
    s.table[rows] = -1
    s.lens[rows] = 0


def _plain_fork(s, parents, children):
    page = s.page
    length = s.lens[parents].long()
    part = length % page
    free = (s.refs == 0).nonzero().flatten()
    need = part > 0
    at = need.long().cumsum(0) - 1
    new = free[at.clamp(min=0)]
    pg = s.table[parents]
    shared = torch.arange(s.row_pages, device="cuda")[None, :] < (length // page)[:, None]
    s.refs.index_add_(0, pg.clamp(min=0).flatten().long(), shared.flatten().int())
    last = (length // page).clamp(max=s.row_pages - 1)
    src = pg[torch.arange(len(parents), device="cuda"), last].long()
    child = torch.where(shared, pg, -1)
    child[torch.arange(len(parents), device="cuda")[need], last[need]] = new[need].int()
    s.table[children] = child
    s.lens[children] = length.int()
    s.refs[new[need]] = 1
    tok = torch.arange(page, device="cuda")[None, None, None, None, :, None] < part[need][:, None, None, None, None, None]
    s.pv[new[need]] = torch.where(tok, s.pv[src[need]], s.pv[new[need]])


def _plain_extend(s, rows, by):
    page = s.page
    old = s.lens[rows].long()
    have, want = (old + page - 1) // page, (old + by + page - 1) // page
    free = (s.refs == 0).nonzero().flatten()
    col = torch.arange(s.row_pages, device="cuda")[None, :]
    add = (col >= have[:, None]) & (col < want[:, None])
    at = add.flatten().long().cumsum(0).view_as(add) - 1
    new = free[at.clamp(min=0, max=len(free) - 1)].int()
    s.table[rows] = torch.where(add, new, s.table[rows])
    s.refs[new[add].long()] = 1
    s.lens[rows] = (old + by).int()


def _plain_compact(s):
    used = s.refs > 0
    live = used.sum()
    at = torch.arange(s.n_pages, device="cuda")
    src, dst = (used & (at >= live)).nonzero().flatten(), (~used & (at < live)).nonzero().flatten()
    s.pv[dst] = s.pv[src]
    to = at.int()
    to[src] = dst.int()
    s.table.copy_(torch.where(s.table >= 0, to[s.table.clamp(min=0).long()], -1))
    s.refs[dst] = s.refs[src]
    s.refs[src] = 0


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """What the definition gives in 64 bits; pages and counts are whole numbers or copies and have no other value."""
    if case["op"] not in ("rope", "attn"):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        # every head as complex numbers turned by the angle whose cosine and sine the table holds
        T, rot = case["T"], case["rot"]
        x = s.qkv[:, :(Hq + 2 * Hkv) * D].double().reshape(T, Hq + 2 * Hkv, D)
        w = torch.cat([s.wq.double().expand(Hq, D), s.wk.double().expand(Hkv, D)])
        h = x[:, :Hq + Hkv]
        h = w * h / torch.sqrt(h.square().sum(-1, keepdim=True) / D + s.eps)
        t = s.cs.double()[s.pos.long()]
        turn = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
        if case["form"] == "pair":
            z = torch.view_as_complex(h[..., :rot].reshape(T, Hq + Hkv, rot // 2, 2).contiguous()) * turn
            h[..., :rot] = torch.view_as_real(z).reshape(T, Hq + Hkv, rot)
        else:
            z = torch.complex(h[..., :rot // 2].contiguous(), h[..., rot // 2:rot].contiguous()) * turn
            h[..., :rot // 2], h[..., rot // 2:rot] = z.real, z.imag
        pool = s.pv.double()
        pg = s.table[s.row_of.long(), s.pos.long() // s.page].long()
        at = s.pos.long() % s.page
        for t0 in range(0, T, 1024):
            e = slice(t0, min(T, t0 + 1024))
            pool[pg[e], s.layer, 0, :, at[e]] = h[e, Hq:]
            pool[pg[e], s.layer, 1, :, at[e]] = x[e, Hq + Hkv:]
        return [h[:, :Hq].reshape(T, Hq * D), pool.view(-1)]
    if work(case)["flops"] > 8e12:
        return None
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda").view(-1, Hq, D)
    q = s.q.double().view(-1, Hq, D)
    for b, (n, length) in enumerate(zip(s.q_lens, s.kv_lens)):
        at = torch.arange(length, device="cuda")
        pg = s.table[b].long()[at // s.page]
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            k = s.pv[pg, s.layer, 0, h, at % s.page].double()
            v = s.pv[pg, s.layer, 1, h, at % s.page].double()
            for i in range(0, n, 512):
                m = min(512, n - i)
                x = s.scale * (q[s.cu[b] + i:s.cu[b] + i + m, hq] @ k.T)
                hidden = at[None, :] > (length - n + i + torch.arange(m, device="cuda"))[:, None]
                x[hidden] = -math.inf
                out[s.cu[b] + i:s.cu[b] + i + m, hq] = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) @ v
    return out.view(-1, Hq * D)
