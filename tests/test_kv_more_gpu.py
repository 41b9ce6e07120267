"""More of the key/value cache on the GPU: buffers that overlap, control state that does not hold together, a pool that
is made smaller."""
import pytest

from tests.kv_harness import Cache

pytestmark = pytest.mark.gpu


def test_rope_output_that_overlaps_its_input():
    import torch
    T, Hq, Hkv, D = 5, 4, 2, 64
    w, wq = (Hq + 2 * Hkv) * D, Hq * D
    c = Cache([T], D=D, page=16, Hq=Hq, Hkv=Hkv, T_max=T)
    ft = c.ft
    ld = w + wq + 8
    buf = c.randn(3 * T, ld, scale=2.0)
    cs = torch.randn(T, D, generator=c.gen, device="cuda")
    row_of, pos = c.ints([0] * T), c.ints(range(T))
    base = buf.data_ptr() + T * ld * 2  # rows T..2T-1 are the input

    def call(q_out, ld_q, T=T):
        return ft.qk_rope_store(c.kv.h, 0, T, base, ld, row_of.data_ptr(), pos.data_ptr(), q_out, ld_q, None, None, 1e-6,
                                cs.data_ptr(), T, D, 0)

    # into the input's heads from a shifted start, across the end of its rows, with another stride, by a row up or down
    for off, ld_q in ((16, ld), (-16, ld), (2 * wq, ld), (2 * (w - 8), ld), (2 * (ld - wq + 8), ld), (2 * ld, ld), (-2 * ld, ld),
                      (0, ld + 8), (2 * w, ld - 8), (2 * w, ld + 8), (2 * ((T - 1) * ld + w - 8), wq),
                      (-2 * ((T - 1) * wq + 8), wq)):
        assert call(base + off, ld_q) == ft.FT_ERR_ARG, (off, ld_q)
    # the same rows elsewhere give what they give in columns beside the input, in a row of another stride, in place
    want = torch.empty(T, wq, dtype=c.dt, device="cuda")
    keep = buf.clone()
    assert call(want.data_ptr(), wq) == ft.FT_OK
    for off, ld_q in ((2 * w, ld), (2 * (w + 8), ld), (2 * T * ld, ld), (-2 * T * ld, ld), (2 * ((T - 1) * ld + w), wq),
                      (-2 * T * wq, wq), (2 * (w - 3 * ld), ld), (0, ld)):
        buf.copy_(keep)
        assert call(base + off, ld_q) == ft.FT_OK, (off, ld_q)
        at = T * ld + off // 2
        got = torch.as_strided(buf, (T, wq), (ld_q, 1), at)
        assert torch.equal(got, want), (off, ld_q)
    # one token: only its own values count
    buf.copy_(keep)
    assert call(base + 2 * (w - 8), ld, T=1) == ft.FT_ERR_ARG
    assert call(base + 2 * w, wq, T=1) == ft.FT_OK
    assert torch.equal(torch.as_strided(buf, (1, wq), (wq, 1), T * ld + w), want[:1])
    assert c.kv.status() == ft.FT_OK


def _control(c):
    return c.table.cpu().tolist(), c.lens.cpu().tolist(), c.refs.cpu().tolist()


def test_pages_out_of_range_change_nothing():
    import torch
    c = Cache([40, 0, 16, 0], D=64, page=16, Hq=1, Hkv=1, row_pages=4, spare=2)
    for page in (-1, c.n_pages, 2 ** 31 - 1):
        for at in (0, 2):  # a page that a fork shares, and the last, of which it copies the tokens
            good = int(c.table[0, at])
            c.table[0, at] = page
            before, pool = _control(c), c.pool.clone()
            c.kv.free(2, c.ints([2, 0]))
            assert c.kv.status() == c.ft.FT_ERR_DEVICE
            c.kv.fork(2, c.ints([2, 0]), c.ints([1, 3]))
            assert c.kv.status() == c.ft.FT_ERR_DEVICE
            assert c.kv.last() == {"allocated": 0, "copied": 0, "live": -1}
            assert _control(c) == before and torch.equal(c.pool, pool)
            c.table[0, at] = good
    c.kv.fork(2, c.ints([2, 0]), c.ints([1, 3]))
    assert c.kv.status() == c.ft.FT_OK


def test_a_count_that_is_0_is_reported_and_stays():
    # rows 0 and 1 hold the same two pages, whose counts say otherwise
    for first, second, status in (([0], [1], "both"), ([0, 1], [], "one call")):
        c = Cache([32, 32, 0], D=64, page=16, Hq=1, Hkv=1, shared=32, row_pages=4)
        a, b = c.model.rows[0]
        c.refs[a] = 1                  # one too few
        c.refs[b] = 2
        c.kv.free(len(first), c.ints(first))
        if second:
            assert c.kv.status() == c.ft.FT_OK
            assert int(c.refs[a]) == 0 and int(c.refs[b]) == 1
            c.kv.free(len(second), c.ints(second))
        assert c.kv.status() == c.ft.FT_ERR_DEVICE, status
        table, lens, refs = _control(c)
        assert lens == [0, 0, 0] and table == [[-1] * 4] * 3 and not any(refs)
        # the pages can be taken again
        c.kv.extend(1, c.ints([0]), c.ints([20]))
        assert c.kv.status() == c.ft.FT_OK


def test_a_smaller_cache_goes_on_where_a_compacted_one_stopped():
    # what ft_kv_compact is for: the control state is the caller's, so a new handle on the first pages goes on with it
    import torch
    page, D, Hq, Hkv = 16, 64, 4, 2
    c = Cache([70, 33, 0, 100], D=D, page=page, Hq=Hq, Hkv=Hkv, n_pages=40, row_pages=12, T_max=8)
    ft = c.ft
    c.model.compact()
    before, q = c.attend([1, 1, 0, 1])
    c.kv.compact()
    live = c.kv.last()["live"]
    assert c.kv.status() == ft.FT_OK and live == 5 + 3 + 7
    c.check_control()
    c.kv.close()
    c.pool[live + 4:] = float("nan")   # the caller's own again
    c.kv = ft.KvCache(1, Hq, Hkv, D, page, live + 4, 4, 12, c.pool[:live + 4], c.table, c.lens, c.refs[:live + 4], T_max=8,
                      B_max=4)
    after, _ = c.attend([1, 1, 0, 1], q=q)
    assert torch.equal(before, after)
    c.model.n_pages, c.model.refs = live + 4, c.model.refs[:live + 4]
    c.model.extend([2], [4 * page])
    c.kv.extend(1, c.ints([2]), c.ints([4 * page]))
    assert c.kv.status() == ft.FT_OK
    assert c.table.cpu().tolist() == c.model.table().tolist()
    c.kv.extend(1, c.ints([2]), c.ints([1]))
    assert c.kv.status() == ft.FT_ERR_CAPACITY
    c.kv.close()
