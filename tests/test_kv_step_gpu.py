"""Row reordering and batch layout of the key/value cache against the oracle: control state, lists and page contents
bit for bit."""
import numpy as np
import pytest

from oracle import kv as okv
from tests.kv_harness import Cache

pytestmark = pytest.mark.gpu

STATUS = {None: "FT_OK", "device": "FT_ERR_DEVICE", "capacity": "FT_ERR_CAPACITY"}


def _reorder(c, rows, parents, plain_rows=False):
    before, want = c.pool.clone(), None
    try:
        copies = c.model.reorder(rows, parents)
    except okv.Refused as e:
        copies, want = [], str(e)
    c.kv.reorder(len(rows), c.ints(parents), rows=None if plain_rows else c.ints(rows))
    assert c.kv.status() == getattr(c.ft, STATUS[want])
    c.check_control()
    ref = before.view(c.torch.int16).cpu().numpy().copy()
    okv.copy_pages(ref, copies)
    assert np.array_equal(c.pool.view(c.torch.int16).cpu().numpy(), ref)
    if want is None:
        assert c.kv.last() == {"allocated": len(copies), "copied": len(copies), "live": -1}
    return want


def _batch(c, rows, add, T, plain_rows=False, slots=True):
    want = None
    try:
        ref = c.model.batch(rows, add, T)
    except okv.Refused as e:
        want, ref = str(e), ([0] * (len(rows) + 1), [-1] * T, [0] * T, [-1] * T)
    torch = c.torch
    cu, row_of, pos = (torch.full((n + 4,), 77, dtype=torch.int32, device="cuda") for n in (len(rows) + 1, T, T))
    sl = torch.full((T + 4,), 77, dtype=torch.int64, device="cuda")
    c.kv.batch(len(rows), c.ints(add), T, cu, row_of, pos, rows=None if plain_rows else c.ints(rows), slots=sl if slots else None)
    assert c.kv.status() == getattr(c.ft, STATUS[want])
    c.check_control()
    for got, w in zip((cu, row_of, pos, sl), ref):
        if got is sl and not slots:
            w = []
        assert got.tolist() == list(w) + [77] * (got.numel() - len(w))
    return want


@pytest.mark.parametrize("D,page,L,Hkv,kind", [(64, 16, 3, 1, "bf16"), (128, 64, 2, 4, "f16"), (256, 128, 1, 2, "bf16"), (64, 32, 5, 3, "f16")])
def test_random_life(D, page, L, Hkv, kind):
    rng = np.random.default_rng(D + page)
    c = Cache([0] * 12, D=D, page=page, L=L, Hkv=Hkv, Hq=Hkv, n_pages=40, row_pages=9, kind=kind)
    for step in range(70):
        rows = [int(x) for x in rng.permutation(12)[:rng.integers(0, 13)]]
        if step % 2:
            whole = step % 10 == 1
            rows = list(range(len(rows))) if whole else rows
            _reorder(c, rows, [int(rng.integers(-1, 12)) for _ in rows], plain_rows=whole)
        else:
            add = [int(rng.integers(0, page + 3)) for _ in rows]
            _batch(c, rows, add, sum(add) + int(rng.integers(-1, 5)) if sum(add) else 3, slots=step % 4 == 0)


def test_beams_of_many_requests():
    # 512 rows of up to 30 pages: more entries than one step of the stage; then 1024 rows
    rng = np.random.default_rng(1)
    for B, K, pages in ((64, 8, 30), (256, 4, 5), (1, 1024, 41)):
        n = B * K
        lens = [int(x) for x in rng.integers(1, 16 * pages, n)]
        c = Cache(lens, D=64, page=16, Hq=1, Hkv=1, row_pages=pages + 3, spare=n // 2, B_max=1)
        _reorder(c, list(range(n)), [b * K + int(rng.integers(0, K)) for b in range(B) for _ in range(K)], plain_rows=True)
        _batch(c, list(range(n)), [1] * n, n)
        _reorder(c, [int(x) for x in rng.permutation(n)[:n // 2]], [int(x) for x in rng.integers(0, n, n // 2)])


def test_long_rows():
    # more columns than the stage holds for these rows
    rng = np.random.default_rng(2)
    lens = [16 * 3000 + 5, 16 * 2999, 16 * 700 + 1, 7] + [16 * 40 + 3] * 28
    c = Cache(lens, D=64, page=16, Hq=1, Hkv=1, row_pages=3100, spare=40, B_max=1)
    _reorder(c, list(range(32)), [3, 0, 0, 1] + [int(x) for x in rng.integers(0, 32, 28)], plain_rows=True)
    _batch(c, list(range(32)), [int(x) for x in rng.integers(0, 900, 32)], 20000)


def test_more_than_is_staged_at_once():
    # 1024 rows of up to 300 pages, of which up to 256 are common: the columns are moved in several passes
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(16 * 90, 16 * 300, 1024)]
    c = Cache(lens, D=64, page=16, Hq=1, Hkv=1, row_pages=301, shared=16 * 256, spare=1100, B_max=1)
    for _ in range(2):
        _reorder(c, [int(x) for x in rng.permutation(1024)], [int(x) for x in rng.integers(-1, 1024, 1024)])
    # 1000 empty rows become copies of one of 291 pages: with too few free pages all is taken back
    for spare in (999, 1000):
        c = Cache([0] * 1000 + [16 * 290 + 3], D=64, page=16, Hq=1, Hkv=1, row_pages=301, spare=spare, B_max=1)
        assert _reorder(c, list(range(1000)), [1000] * 1000, plain_rows=True) == ("capacity" if spare < 1000 else None)


def test_reorder_refusals_change_nothing():
    c = Cache([40, 24, 16, 0], D=64, page=16, Hq=1, Hkv=1, row_pages=4, spare=0)
    ft = c.ft
    for rows, parents in (([0, 0], [1, 1]), ([4], [0]), ([-1], [0]), ([0], [4]), ([0], [-2]), ([3], [0])):
        state = (list(map(list, c.model.rows)), list(c.model.lens), list(c.model.refs))
        assert _reorder(c, rows, parents) == ("capacity" if rows == [3] else "device")
        assert (c.model.rows, c.model.lens, c.model.refs) == state
    # a row that ends gives its pages to a copy of the same call
    assert _reorder(c, [1, 3], [0, -1]) is None
    for n in (-1, 5):
        assert ft.kv_reorder(c.kv.h, n, None, c.lens.data_ptr()) == ft.FT_ERR_ARG
    assert ft.kv_reorder(c.kv.h, 1, None, None) == ft.FT_ERR_ARG
    assert ft.kv_reorder(c.kv.h, 0, None, None) == ft.FT_OK
    # pages outside the pool, counts that do not hold: found before anything moves
    keep = c.table.clone()
    c.table[0, 0] = 99
    c.kv.reorder(1, c.ints([0]), rows=c.ints([2]))
    assert c.kv.status() == ft.FT_ERR_DEVICE
    c.table.copy_(keep)
    c.refs[c.model.rows[2][0]] = 0
    refs = c.refs.clone()
    c.kv.reorder(1, c.ints([0]), rows=c.ints([2]))
    assert c.kv.status() == ft.FT_ERR_DEVICE
    assert c.torch.equal(c.refs, refs) and c.torch.equal(c.table, keep) and c.lens.tolist() == c.model.lens


def test_more_rows_than_a_call_takes():
    c = Cache([1] * 1100, D=64, page=16, Hq=1, Hkv=1, B_max=1)
    assert c.ft.kv_reorder(c.kv.h, 1025, None, c.ints([0] * 1025).data_ptr()) == c.ft.FT_ERR_ARG
    _reorder(c, list(range(1024)), [1050] * 1024, plain_rows=True)


@pytest.mark.parametrize("B", [0, 1, 5, 1024, 1025, 2048, 2049, 5000])
def test_batches(B):
    rng = np.random.default_rng(B)
    rows = [int(x) for x in rng.permutation(B + 2)[:B]]
    lens = [int(x) for x in rng.integers(0, 70, B + 2)]
    c = Cache(lens, D=64, page=16, Hq=1, Hkv=1, row_pages=9, spare=3 * B + 3, B_max=1)
    _batch(c, rows, [1] * B, B)
    add = [int(x) for x in rng.integers(0, 4, B)]
    _batch(c, rows, add, sum(add) + 9)
    if B:
        _batch(c, list(range(B)), add, sum(add), plain_rows=True)
        _batch(c, rows, add[:-1] + [70], 70 * B + 100)


@pytest.mark.parametrize("T", [4095, 4096, 4097, 30000])
def test_prompts(T):
    for adds in ([T], [0, T - 3, 0, 3, 0], [T // 3] * 3 + [0] * 5, [T // 7 + 1] * 6):
        c = Cache([33, 0, 16, 5, 64, 1, 0, 40], D=64, page=64, Hq=1, Hkv=1, row_pages=T // 64 + 4, spare=T // 64 + 20, B_max=1)
        _batch(c, list(range(7, 7 - len(adds), -1)), adds, T + 1)


def test_batch_refusals():
    c = Cache([40, 0, 16, 0], D=64, page=16, Hq=1, Hkv=1, row_pages=4, spare=1)
    ft, torch = c.ft, c.torch
    big = 2 ** 31 - 1
    for rows, add, T in (([0, 0], [1, 1], 5), ([4], [1], 5), ([-1], [1], 5), ([0], [-1], 5), ([0], [25], 30), ([0, 1], [3, 3], 5),
                         ([1], [17], 20), ([0, 1, 2, 3], [big] * 4, 5), ([1, 0], [2, 1], 0), ([0, 0], [1, 1], 5005), ([4], [1], 5005),
                         ([0], [-1], 5005), ([0], [25], 5005), ([1], [17], 5005), ([0, 1], [2500, 2500], 4999)):
        state = (list(map(list, c.model.rows)), list(c.model.lens), list(c.model.refs))
        assert _batch(c, rows, add, T) is not None
        assert (c.model.rows, c.model.lens, c.model.refs) == state
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    l = torch.zeros(16, dtype=torch.int64, device="cuda")
    P, Q = i.data_ptr(), l.data_ptr()
    ok = [c.kv.h, 2, P, P + 16, 4, P + 32, P + 64, P + 96, Q]
    c.table.fill_(-1), c.lens.zero_(), c.refs.zero_()
    i[1] = 1
    assert ft.kv_batch(*ok) == ft.FT_OK and c.kv.status() == ft.FT_OK
    for at, v in ((1, -1), (1, 5), (3, None), (4, -1), (5, None), (6, None), (7, None), (5, P + 2), (8, Q + 4), (6, P + 2),
                  (7, P + 76), (6, P + 40), (5, P + 4), (5, P + 20), (8, P + 64), (2, P + 1), (3, P + 3), (2, P + 100)):
        bad = list(ok)
        bad[at] = v
        assert ft.kv_batch(*bad) == ft.FT_ERR_ARG, (at, v)


def test_graph_of_a_beam_step():
    """select's lists go straight into reorder and batch; the captured step is replayed."""
    import torch

    import moe_expert_cache_gb300 as ft
    s = torch.cuda.Stream()
    B, K, V, steps = 3, 4, 3001, 9
    n = B * K
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn(steps, n, V, generator=g, device="cuda") * 3
    x = logits[0].clone()
    runs = []
    for captured in (False, True):
        c = Cache([21] * n, D=64, page=16, Hq=1, Hkv=1, row_pages=4, spare=30, stream=s.cuda_stream)
        bm = ft.Beams(V, n, K, stream=s.cuda_stream)
        sc = torch.zeros(n, device="cuda")
        par, tok = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
        cu, row_of, pos, add = (torch.ones(n + 1, dtype=torch.int32, device="cuda") for _ in range(4))
        slots = torch.empty(n, dtype=torch.int64, device="cuda")

        def step():
            bm.select(B, K, K, x, V, sc, sc, par, tok)
            c.kv.reorder(n, par)
            c.kv.batch(n, add, n, cu, row_of, pos, slots=slots)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph, stream=s):
                step()
        for i in range(steps):
            x.copy_(logits[i])
            torch.cuda.synchronize()
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            c.model.reorder(list(range(n)), par.tolist())
            want = c.model.batch(list(range(n)), [1] * n, n)
            assert [cu.tolist(), row_of.tolist()[:n], pos.tolist()[:n], slots.tolist()] == [list(w) for w in want]
            c.check_control()
        assert bm.status() == ft.FT_OK and c.kv.status() == ft.FT_OK
        runs.append([t.clone() for t in (sc, par, tok, c.table, c.pool)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
