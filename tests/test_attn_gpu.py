"""Attention over the page table against the fp64 oracle: head sizes, types,
pages, lengths around the tile and page sizes, shared prefixes, empty rows,
whatever lies in unused places, strides, streams, graphs, refusals."""
import numpy as np
import pytest

from tests.kv_harness import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_lengths(D, page, kind):
    # one query each; lengths around the 64-key tile and the page
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500]
    c = Cache(lens, D=D, page=page, kind=kind, Hq=6, Hkv=2, T_max=16, seed=D + page)
    c.poison(float("nan"))
    c.check_attend([1] * len(lens))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (5, 1), (24, 3), (128, 1)])
def test_head_layouts(Hq, Hkv):
    c = Cache([200, 70, 1], D=64, page=32, Hq=Hq, Hkv=Hkv, T_max=40, L=3, seed=Hq)
    c.poison(float("inf"))
    c.check_attend([1, 3, 1], layer=2, ld_extra=8)


@pytest.mark.parametrize("D,G", [(64, 3), (128, 8), (256, 5)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_prompts_are_causal(D, G, kind):
    # prompts that cover several row tiles, some of them ending inside one; earlier context or none
    lens, ns = [333, 130, 65, 700], [333, 100, 1, 65]
    c = Cache(lens, D=D, page=16, kind=kind, Hq=2 * G, Hkv=2, T_max=sum(ns) + 3, seed=G)
    c.poison(float("nan"))
    c.check_attend(ns)


def test_rows_that_see_nothing():
    # more queries than tokens: the first ones see no key; an empty row; a request without queries
    c = Cache([3, 0, 40, 64], D=128, page=16, Hq=8, Hkv=2, T_max=200)
    c.poison(float("nan"))
    out, _ = c.attend([5, 2, 0, 130])
    got = out.float().cpu().numpy()
    assert np.all(got[:2, :8 * 128] == 0) and np.all(got[5:7, :8 * 128] == 0) and np.all(got[7:73, :8 * 128] == 0)
    c.check_attend([5, 2, 0, 130])


@pytest.mark.parametrize("D,page,kind,G", [(64, 16, "f16", 3), (128, 64, "bf16", 8), (128, 128, "f16", 1), (256, 32, "bf16", 8)])
@pytest.mark.parametrize("n", [1, 5])
def test_shared_prefix(D, page, kind, G, n):
    shared = 5 * 128 if page == 128 else 13 * page + (0 if page > 16 else 16 * 20)
    lens = [shared + n + x for x in (0, 1, 17, 64, 300, 7, 129)]
    c = Cache(lens, D=D, page=page, kind=kind, Hq=2 * G, Hkv=2, shared=shared, T_max=64, seed=D + n)
    c.poison(float("nan"))
    c.check_attend([n] * len(lens), groups=([0, len(lens)], [shared]))


def test_groups_and_claims():
    # two groups and ungrouped requests around them; claims that are too large, not whole pages, or zero
    import torch
    page, shared = 32, 320
    lens = [50] + [shared + x for x in (33, 1, 64, 90)] + [10] + [shared + x for x in (5, 200)] + [77]
    c = Cache(lens, D=64, page=page, Hq=32, Hkv=2, T_max=64, shared=0, seed=5)
    # rows 1-4 share one prefix and rows 6-7 another: make their first pages the same
    for rows in ([1, 2, 3, 4], [6, 7]):
        for r in rows[1:]:
            for i in range(shared // page):
                old, new = c.model.rows[r][i], c.model.rows[rows[0]][i]
                c.model.refs[old] -= 1
                c.model.refs[new] += 1
                c.model.rows[r][i] = new
    c.table.copy_(torch.from_numpy(c.model.table()))
    c.poison(float("nan"))
    ns = [1, 1, 2, 1, 1, 1, 1, 3, 1]
    for toks in ([shared, shared], [10 ** 6, 300], [0, 31], [321, 64]):
        # group 0 covers requests 1-4; group 1 covers 6-7 (5 and 8 in groups of their own)
        c.check_attend(ns, groups=([1, 5, 6, 8], [toks[0], 0, toks[1]]))
    c.check_attend(ns)


def test_rows_in_any_order_and_many_requests():
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(1, 90, 150)]
    c = Cache(lens, D=64, page=16, Hq=2, Hkv=1, T_max=200)
    rows = [int(x) for x in rng.permutation(150)[:97]]
    ns = [int(min(x, lens[r])) for x, r in zip(rng.integers(0, 3, 97), rows)]
    c.check_attend(ns, rows=rows)


def test_as_many_requests_as_a_plan_takes():
    rng = np.random.default_rng(8)
    lens = [32 + int(x) for x in rng.integers(1, 30, 1024)]
    c = Cache(lens, D=64, page=16, Hq=2, Hkv=1, T_max=1024, shared=32, seed=8)
    c.poison(float("nan"))
    c.check_attend([1] * 1024, groups=([0, 400, 1024], [32, 32]))
    c.check_attend([1] * 1024)


@pytest.mark.parametrize("D,page,kind,Hq,Hkv", [(128, 64, "bf16", 8, 2), (128, 16, "f16", 9, 3), (256, 32, "bf16", 16, 1),
                                                (256, 128, "f16", 4, 4)])
def test_requests_of_few_rows_and_some_of_many(D, page, kind, Hq, Hkv):
    # ungrouped requests of one token or a few, several tokens' causal edge inside a tile, rows without a key, and
    # now and then one of many rows between them
    rng = np.random.default_rng(D + page)
    B = 400 // Hkv
    lens = [int(x) for x in rng.integers(0, 400, B)]
    ns = [int(x) for x in rng.integers(0, 3, B)]
    most = 16 * Hkv // Hq
    for i in range(0, B, 9):
        ns[i], lens[i] = most + 1, lens[i] + most  # just too many rows
    for i in range(5, B, 37):
        ns[i], lens[i] = 100 * Hkv // Hq, lens[i] + 60
    while sum(ns) * (Hq // Hkv) > 16 * B:
        ns[int(rng.integers(0, B))] = 0
    c = Cache(lens, D=D, page=page, Hq=Hq, Hkv=Hkv, kind=kind, T_max=sum(ns), seed=D)
    c.poison(float("nan"))
    c.check_attend(ns)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 9])
def test_keys_of_minus_infinity_and_growing_scores(D, n):
    # the first key, or all of the first tile's, score -inf; after them scores that grow from tile to tile
    for dead in (1, 130):
        c = Cache([700], D=D, page=64, Hq=4, Hkv=1, T_max=16)
        t = c.torch.arange(700, device="cuda")
        pg = c.table[0].long()[t // 64]
        up = c.torch.linspace(0.05, 4.0, 700, device="cuda")[:, None]
        c.pool[pg, 0, 0, 0, t % 64] = (c.pool[pg, 0, 0, 0, t % 64].float() * up).to(c.dt)
        c.pool[pg[:dead], 0, 0, 0, t[:dead] % 64, 0] = float("-inf")
        q = c.randn(n, 4 * D, scale=1.5)
        q.view(n, 4, D)[:, :, 0] = 1.0
        c.check_attend([n], q=q)


def test_long_axis_split():
    # one request over many CTAs: the join of dozens of pieces, with the largest scores last and first
    for flip in (False, True):
        c = Cache([9000], D=128, page=64, Hq=4, Hkv=1, T_max=4)
        up = c.torch.linspace(0.2, 3.0, 9000, device="cuda")
        up = up.flip(0) if flip else up
        t = c.torch.arange(9000, device="cuda")
        pg = c.table[0].long()[t // 64]
        c.pool[pg, 0, 0, 0, t % 64] = (c.pool[pg, 0, 0, 0, t % 64].float() * up[:, None]).to(c.dt)
        c.check_attend([2])


def test_scores_that_grow_and_scales():
    # every tile's maximum exceeds the last by far more than the lag: O is rescaled each time
    c = Cache([640], D=64, page=64, Hq=2, Hkv=1, T_max=4)
    t = c.torch.arange(640, device="cuda")
    pg = c.table[0].long()[t // 64]
    k = c.torch.zeros(640, 64, device="cuda")
    k[:, 0] = (t // 64).float() * 16
    c.pool[pg, 0, 0, 0, t % 64] = k.to(c.dt)
    q = c.randn(2, 128, scale=0.1)
    q[:, 0] = 4.0
    q[:, 64] = -4.0
    c.check_attend([2], q=q, scale=0.5)
    c.check_attend([2], q=q, scale=1e-6)


def test_repeats_are_equal_and_ungrouped_agrees():
    shared = 256
    lens = [shared + x for x in (100, 50, 60, 8)]
    c = Cache(lens, D=128, page=64, Hq=16, Hkv=2, shared=shared, T_max=16)
    a, q = c.attend([1] * 4, groups=([0, 4], [shared]))
    b, _ = c.attend([1] * 4, groups=([0, 4], [shared]), q=q)
    assert c.torch.equal(a, b)
    d, _ = c.attend([1] * 4, q=q)
    # both sides are within their own roundings of the same value
    assert float((a.double() - d.double()).abs().max()) <= 4 * 2.0 ** -8 * float(c.pool.abs().max())


def test_pool_past_32_bits():
    # element offsets over 2^32 in the pool: the pages in use are the first and the last ones
    import torch
    D, page, Hkv, L = 128, 128, 8, 4
    per = L * 2 * Hkv * page * D
    n_pages = (1 << 32) // per + 3
    assert n_pages * per > 1 << 32
    import moe_expert_cache_gb300 as ft
    pool = torch.zeros(n_pages, L, 2, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, n_pages - 1, n_pages - 2], [n_pages - 3, -1, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300, 100], dtype=torch.int32, device="cuda")
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    g = torch.Generator(device="cuda").manual_seed(0)
    for p in table[table >= 0].tolist():
        pool[p] = torch.randn(pool.shape[1:], generator=g, device="cuda").to(pool.dtype)
    kv = ft.KvCache(L, Hkv, Hkv, D, page, n_pages, 2, 3, pool, table, lens, refs, T_max=4, B_max=2)
    q = torch.randn(2, Hkv * D, generator=g, device="cuda").to(pool.dtype)
    out = torch.empty_like(q)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    kv.attn_plan(2, 2, cu)
    kv.attn_forward(3, q, Hkv * D, out, Hkv * D, D ** -0.5)
    assert kv.status() == ft.FT_OK
    for b, n in ((0, 300), (1, 100)):
        pg = table[b].long()
        k = pool[pg, 3, 0].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n].double()
        v = pool[pg, 3, 1].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n].double()
        s = torch.einsum("hd,hnd->hn", q[b].double().view(Hkv, D), k) * D ** -0.5
        w = s.softmax(-1)
        ref, mass = torch.einsum("hn,hnd->hd", w, v), torch.einsum("hn,hnd->hd", w, v.abs())
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * mass + 1e-6
        assert bool(((out[b].double().view(Hkv, D) - ref).abs() <= tol).all())
    kv.close()


def test_other_stream_and_graph():
    import torch
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Cache([100, 65, 30], D=128, page=64, Hq=8, Hkv=2, T_max=8, stream=s.cuda_stream, row_pages=8)
        q, out = c.randn(3, 8 * 128), c.torch.zeros(3, 8 * 128, dtype=c.dt, device="cuda")
        cu = c.ints([0, 1, 2, 3])

        def step():
            c.kv.attn_plan(3, 3, cu)
            c.kv.attn_forward(0, q, 8 * 128, out, 8 * 128, 0.1)

        step()
        s.synchronize()
        first = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        out.zero_()
        graph.replay()
        s.synchronize()
        assert torch.equal(out, first)
        # the plan follows the lengths on the device
        c.lens.copy_(c.ints([33, 65, 1]))
        graph.replay()
        s.synchronize()
        c.model.lens = [33, 65, 1]
        want, _ = c.attend([1, 1, 1], q=q, scale=0.1)
        s.synchronize()
        assert torch.equal(out, want) and not torch.equal(out, first)
    assert c.kv.status() == c.ft.FT_OK


def test_refusals():
    c = Cache([40, 20], D=64, page=16, Hq=4, Hkv=2, T_max=8, B_max=2)
    ft, kv = c.ft, c.kv.h
    q, out, cu = c.randn(8, 256), c.randn(8, 256), c.ints([0, 1, 2])
    p = lambda t: t.data_ptr()  # noqa: E731
    assert ft.attn_forward(kv, 0, p(q), 256, p(out), 256, 1.0) == ft.FT_ERR_STATE
    for bad in ((3, 2), (-1, 2), (2, 9), (2, -1)):
        assert ft.attn_plan(kv, bad[0], bad[1], p(cu), None, 0, None, None) == ft.FT_ERR_ARG
    assert ft.attn_plan(kv, 2, 2, None, None, 0, None, None) == ft.FT_ERR_ARG
    assert ft.attn_plan(kv, 2, 2, p(cu), None, 1, None, None) == ft.FT_ERR_ARG
    assert ft.attn_plan(kv, 2, 2, p(cu), None, 3, p(cu), p(cu)) == ft.FT_ERR_ARG
    assert ft.attn_plan(kv, 2, 2, p(cu), None, 0, None, None) == ft.FT_OK
    for args in ((1, p(q), 256, p(out), 256, 1.0), (-1, p(q), 256, p(out), 256, 1.0), (0, None, 256, p(out), 256, 1.0),
                 (0, p(q), 248, p(out), 256, 1.0), (0, p(q), 256, p(out), 260, 1.0), (0, p(q) + 2, 256, p(out), 256, 1.0),
                 (0, p(q), 256, p(q), 256, 1.0), (0, p(q), 256, p(q) + 512, 256, 1.0), (0, p(q), 256, p(out), 256, 0.0),
                 (0, p(q), 256, p(out), 256, float("nan")), (0, p(q), 256, p(out), 256, float("inf"))):
        assert ft.attn_forward(kv, *args) == ft.FT_ERR_ARG, args
    assert c.kv.status() == ft.FT_OK
    # what the device finds: offsets that descend or pass T, a row or a length out of range, groups out of order
    out.fill_(7)
    bad = [dict(cu=[0, 2, 1]), dict(cu=[1, 1, 2]), dict(cu=[0, 1, 3]), dict(rows=[0, 2]), dict(rows=[-1, 0]),
           dict(lens=[-1, 5]), dict(lens=[40, 49]), dict(groups=([0, 3], [16])), dict(groups=([1, 0], [16])),
           dict(groups=([0, 2], [-1]))]
    for b in bad:
        c.lens.copy_(c.ints(b.get("lens", [40, 20])))
        g = b.get("groups")
        keep = [c.ints(b.get("cu", [0, 1, 2])), c.ints(b.get("rows", [0, 1]))] + [c.ints(x) for x in g or ()]
        c.kv.attn_plan(2, 2, keep[0], rows=keep[1], n_groups=1 if g else 0, group_start=keep[2] if g else None,
                       group_tokens=keep[3] if g else None)
        c.kv.attn_forward(0, q, 256, out, 256, 1.0)
        assert c.kv.status() == ft.FT_ERR_DEVICE, b
        assert bool((out == 7).all()), b
    # a page index out of range within a row's length
    c.lens.copy_(c.ints([40, 20]))
    c.table[0, 1] = c.n_pages
    c.kv.attn_plan(2, 2, cu)
    c.kv.attn_forward(0, q, 256, out, 256, 1.0)
    assert c.kv.status() == ft.FT_ERR_DEVICE
    assert c.kv.status() == ft.FT_OK
    # nothing to do is not an error
    c.kv.attn_plan(0, 0, None)
    c.kv.attn_forward(0, q, 256, out, 256, 1.0)
    assert c.kv.status() == ft.FT_OK
