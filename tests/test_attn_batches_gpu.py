"""Attention of large batches: more work items on a CTA than it keeps in shared memory, more segments than the plan
keeps there and than it has threads, steps that a graph replays with other lengths, two caches at a time."""
import numpy as np
import pytest

from tests.kv_dense import check_dense
from tests.kv_harness import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("D,page,kind,Hq", [(64, 16, "f16", 8), (128, 64, "bf16", 16), (256, 32, "bf16", 8)])
def test_1024_requests_of_eight_heads(D, page, kind, Hq, grouped):
    # 8192 segments, 27 and more items a CTA
    rng = np.random.default_rng(D)
    shared = 64
    lens = [int(x) for x in shared + rng.integers(1, 140, 1024)]
    lens[77], lens[900] = 1100, shared + 1
    c = Cache(lens, D=D, page=page, kind=kind, Hq=Hq, Hkv=8, shared=shared, T_max=1024, seed=D)
    c.poison(float("nan"))
    out, q = c.attend([1] * 1024, groups=([0, 500, 1024], [shared, shared]) if grouped else None)
    assert c.kv.status() == c.ft.FT_OK
    check_dense(c, [1] * 1024, out, q)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_a_prompt_of_2500_row_tiles(kind):
    # 128 query heads on one key/value head: a row tile a token
    c = Cache([2600], D=64, page=64, kind=kind, Hq=128, Hkv=1, T_max=2500)
    c.poison(float("nan"))
    out, q = c.attend([2500])
    assert c.kv.status() == c.ft.FT_OK
    check_dense(c, [2500], out, q)


@pytest.mark.parametrize("D", [64, 128])
def test_more_segments_than_the_plan_keeps_behind_a_shared_prefix(D):
    # 160 rows of a request are a row tile and a quarter: the rows of all take three fifths of the tiles over the prefix
    rng = np.random.default_rng(D)
    ns = [int(x) for x in rng.choice([2, 2, 2, 5], 1024)]
    lens = [64 + n + int(x) for n, x in zip(ns, rng.integers(0, 60, 1024))]
    c = Cache(lens, D=D, page=16, Hq=80, Hkv=1, shared=64, T_max=sum(ns) + 5, seed=D)
    assert sum(-(-n * 80 // 128) for n in ns) > 2048
    c.poison(float("nan"))
    for groups in (([0, 1024], [64]), None):
        out, q = c.attend(ns, groups=groups)
        assert c.kv.status() == c.ft.FT_OK
        check_dense(c, ns, out, q)


@pytest.mark.parametrize("D,kind", [(64, "f16"), (128, "bf16"), (256, "bf16")])
def test_graph_replays_other_lengths_behind_a_prefix(D, kind):
    # the buffers of a captured step have room for 12 tokens; each replay has fewer, on rows of other lengths
    import torch
    B, T, shared, Hq, Hkv = 6, 12, 320, 8, 2
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Cache([shared + 200] * B, D=D, page=32, kind=kind, Hq=Hq, Hkv=Hkv, shared=shared, T_max=T, stream=s.cuda_stream)
        q = c.randn(T, Hq * D, scale=1.5)
        out = torch.empty_like(q)
        cu, start, tokens = c.ints([0] * (B + 1)), c.ints([0, B]), c.ints([shared])

        def step():
            c.kv.attn_plan(B, T, cu, n_groups=1, group_start=start, group_tokens=tokens)
            c.kv.attn_forward(0, q, Hq * D, out, Hq * D, D ** -0.5)

        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for ns, own, claim in (([1] * 6, [1, 30, 200, 64, 65, 7], shared), ([2] * 6, [100, 2, 64, 199, 3, 128], shared),
                               ([0, 3, 1, 0, 5, 1], [1, 9, 130, 4, 5, 77], 10 ** 6), ([1, 0, 0, 0, 0, 1], [50, 1, 1, 1, 1, 80], 0)):
            lens = [shared + x for x in own]
            c.lens.copy_(c.ints(lens))
            cu.copy_(c.ints(np.concatenate([[0], np.cumsum(ns)]).tolist()))
            tokens.fill_(claim)
            for _ in range(2):
                out.fill_(7)
                graph.replay()
                s.synchronize()
                check_dense(c, ns, out, q, lens=lens)
                assert bool((out[sum(ns):] == 7).all())
                again = out.clone()
            assert torch.equal(out, again)
    assert c.kv.status() == c.ft.FT_OK


def test_two_caches_on_two_streams():
    # different head sizes and plans, launched in turn without waiting
    import torch
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for s, (D, B, Hq, Hkv) in zip(streams, ((128, 40, 8, 2), (256, 21, 4, 1))):
        with torch.cuda.stream(s):
            lens = [100 + 37 * (i % 9) for i in range(B)]
            c = Cache(lens, D=D, page=64, Hq=Hq, Hkv=Hkv, T_max=B, stream=s.cuda_stream, seed=D)
            q = c.randn(B, Hq * D, scale=1.5)
            outs = [torch.zeros_like(q) for _ in range(8)]
            cu = c.ints(range(B + 1))
            work.append((s, c, q, outs, cu, B))
    torch.cuda.synchronize()
    for i in range(8):
        for s, c, q, outs, cu, B in work:
            with torch.cuda.stream(s):
                c.kv.attn_plan(B, B, cu)
                c.kv.attn_forward(0, q, c.Hq * c.D, outs[i], c.Hq * c.D, c.D ** -0.5)
    for s, c, q, outs, cu, B in work:
        assert c.kv.status() == c.ft.FT_OK
        with torch.cuda.stream(s):
            check_dense(c, [1] * B, outs[0], q)
            assert all(torch.equal(o, outs[0]) for o in outs[1:])
        s.synchronize()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_grouped_and_ungrouped_results_within_the_bound(D):
    shared = 256
    lens = [shared + x for x in (100, 50, 60, 8)]
    c = Cache(lens, D=D, page=64, Hq=16, Hkv=2, shared=shared, T_max=16)
    a, q = c.attend([1] * 4, groups=([0, 4], [shared]))
    b, _ = c.attend([1] * 4, q=q)
    for out in (a, b):
        check_dense(c, [1] * 4, out, q)


@pytest.mark.parametrize("D,Hq,n", [(64, 4, 1), (128, 4, 1), (128, 32, 60), (256, 4, 3)])
def test_what_a_bad_number_reaches(D, Hq, n):
    # keys that a query does not see may hold anything; a bad value makes bad numbers of what sees it, in its column
    import torch
    for bad in (float("nan"), float("inf"), float("-inf")):
        c = Cache([300, 290], D=D, page=16, Hq=Hq, Hkv=2, T_max=2 * n)
        p, o = divmod(299, 16)
        if n > 1:  # the last key of row 0 is seen by its last query alone
            c.pool[c.model.rows[0][p], 0, 0, :, o] = bad
        q = c.randn(2 * n, Hq * D)
        out, _ = c.attend([n, n], q=q)
        if n > 1:
            keep = torch.ones(2 * n, dtype=torch.bool)
            keep[n - 1] = False
            assert bool(torch.isfinite(out.float().cpu()[keep]).all())
            c.pool[c.model.rows[0][p], 0, 0, :, o] = 0
            same, _ = c.attend([n, n], q=q)
            assert torch.equal(out.cpu()[keep], same.cpu()[keep])
        # a bad value at a token that every query sees
        c.pool[c.model.rows[0][2], 0, 1, 1, 5, 3] = bad
        out = c.attend([n, n], q=q)[0].float().cpu().view(2 * n, Hq, D)
        fine = torch.isfinite(out)
        assert bool(fine[n:].all()) and bool(fine[:n, :Hq // 2].all())
        assert not bool(fine[:n, Hq // 2:, 3].any())
        fine[:n, Hq // 2:, 3] = True
        assert bool(fine.all())
        assert c.kv.status() == c.ft.FT_OK


@pytest.mark.parametrize("D,page,Hq", [(64, 16, 16), (128, 64, 32), (256, 32, 16)])
def test_claims_that_the_pages_do_not_bear_out(D, page, Hq):
    # rows that share fewer pages than is claimed, down to none: the pages that they do share are taken
    import torch
    shared, own = 40 * page, 5 * page
    for differs in ({3: 39}, {1: 17, 6: 30}, {7: 0}, {0: 25}, {i: 9 for i in range(1, 8)}):
        c = Cache([shared + own + i for i in range(8)], D=D, page=page, Hq=Hq, Hkv=2, shared=shared, T_max=16,
                  spare=8 * len(differs), seed=page)
        free = [p for p in range(c.n_pages) if c.model.refs[p] == 0]
        for i, (r, j) in enumerate(differs.items()):
            c.model.refs[c.model.rows[r][j]] -= 1
            c.model.rows[r][j] = free[i]
            c.model.refs[free[i]] = 1
        c.table.copy_(torch.from_numpy(c.model.table()))
        for ns in ([1] * 8, [1, 0, 2, 3, 1, 2, 1, 0]):
            for groups in (([0, 8], [shared]), ([0, 8], [10 ** 6]), ([0, 4, 8], [shared, shared - 1]), ([1, 7], [shared])):
                out, q = c.attend(ns, groups=groups)
                assert c.kv.status() == c.ft.FT_OK
                check_dense(c, ns, out, q)


def test_claims_over_long_prefixes_and_many_requests():
    # more pages than a warp compares at a time, more requests than there are warps; one page in the middle differs
    import torch
    shared, page, B = 700 * 16, 16, 50
    for row, j in ((49, 699), (13, 300), (30, 256), (7, 255)):
        c = Cache([shared + 1 + 3 * i for i in range(B)], D=64, page=page, Hq=16, Hkv=1, shared=shared, T_max=B, spare=3, seed=j)
        c.model.rows[row][j] = next(p for p in range(c.n_pages) if c.model.refs[p] == 0)
        c.table.copy_(torch.from_numpy(c.model.table()))
        out, q = c.attend([1] * B, groups=([0, B], [shared]))
        assert c.kv.status() == c.ft.FT_OK
        check_dense(c, [1] * B, out, q)
