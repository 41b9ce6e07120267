"""Page operations and the norm-rotate-store pass against the oracle: control
state and page contents bit for bit, heads within one rounding."""
import numpy as np
import pytest

from oracle import kv as okv
from tests.kv_harness import U, Cache

pytestmark = pytest.mark.gpu


def _apply(c, name, *lists):
    """One call on the device and on the oracle; the pool is compared bit for bit."""
    before = c.pool.clone()
    want = None
    try:
        copies = getattr(c.model, name)(*lists)
    except okv.Refused as e:
        copies, want = [], str(e)
    args = [c.ints(x) for x in lists]
    if name == "compact":
        c.kv.compact()
    else:
        getattr(c.kv, name)(len(lists[0]), *args)
    assert c.kv.status() == {None: c.ft.FT_OK, "device": c.ft.FT_ERR_DEVICE, "capacity": c.ft.FT_ERR_CAPACITY}[want]
    c.check_control()
    ref = before.view(c.torch.int16).cpu().numpy().copy()
    okv.copy_pages(ref, copies)
    assert np.array_equal(c.pool.view(c.torch.int16).cpu().numpy(), ref)
    return copies


@pytest.mark.parametrize("D,page,L,Hkv", [(64, 16, 3, 1), (128, 64, 2, 4), (256, 128, 1, 2), (64, 32, 5, 3)])
def test_random_life_of_a_cache(D, page, L, Hkv):
    rng = np.random.default_rng(D + page)
    c = Cache([0] * 12, D=D, page=page, L=L, Hkv=Hkv, Hq=Hkv, n_pages=40, row_pages=9)
    for step in range(60):
        m = c.model
        op = rng.choice(["extend", "fork", "free", "compact"], p=[0.45, 0.25, 0.2, 0.1])
        if op == "extend":
            rows = [int(x) for x in rng.permutation(12)[:rng.integers(0, 6)]]
            _apply(c, op, rows, [int(rng.integers(0, 2 * page + 2)) for _ in rows])
        elif op == "fork":
            empty = [r for r in range(12) if m.lens[r] == 0]
            rng.shuffle(empty)
            ch = empty[:rng.integers(0, 5)]
            _apply(c, op, [int(rng.integers(0, 12)) for _ in ch], ch)
        elif op == "free":
            _apply(c, op, [int(x) for x in rng.permutation(12)[:rng.integers(0, 4)]])
        else:
            copies = _apply(c, op)
            live = sum(1 for x in m.refs if x)
            assert c.kv.last() == {"allocated": 0, "copied": len(copies), "live": live}
            assert all(x > 0 for x in m.refs[:live]) and not any(m.refs[live:])


def test_large_pool_takes_the_lowest_free_pages():
    # more pages than one step of the scans; every third one is free
    n = 13001
    c = Cache([0, 0, 0], D=64, page=16, Hq=1, Hkv=1, n_pages=n, row_pages=5000)
    held = [p for p in range(n) if p % 3]
    c.model.rows[0], c.model.lens[0] = held[:5000], 80000
    c.model.rows[1], c.model.lens[1] = held[5000:8667], 3667 * 16
    for p in held[:8667]:
        c.model.refs[p] = 1
    c.table.copy_(c.torch.from_numpy(c.model.table()))
    c.lens.copy_(c.ints(c.model.lens))
    c.refs.copy_(c.ints(c.model.refs))
    _apply(c, "extend", [2], [4300 * 16 + 3])
    _apply(c, "free", [0])
    _apply(c, "compact")


def test_long_lists():
    # lists of more rows than a step of the scans; forks of whole and of partial pages, one parent many times
    rng = np.random.default_rng(4)
    n = 2600
    c = Cache([0] * n, D=64, page=16, Hq=1, Hkv=1, n_pages=9000, row_pages=6, B_max=1)
    a = [int(x) for x in rng.permutation(n)[:1301]]
    _apply(c, "extend", a, [int(x) for x in rng.integers(0, 60, len(a))])
    empty = [r for r in range(n) if c.model.lens[r] == 0]
    held = [r for r in a[:60] if c.model.lens[r]]
    _apply(c, "fork", [int(rng.choice(held)) if i % 2 else held[7] for i in range(len(empty) - 1)], empty[1:])
    _apply(c, "extend", list(range(n)), [int(x) for x in rng.integers(0, 20, n)])
    assert sum(1 for x in c.model.lens if x) > 2400
    _apply(c, "free", [int(x) for x in rng.permutation(n)[:2001]])
    _apply(c, "compact")


def test_page_refusals_change_nothing():
    c = Cache([40, 0, 16, 0], D=64, page=16, Hq=1, Hkv=1, row_pages=4, spare=1)
    bad = [("extend", [0, 0], [1, 1]), ("extend", [4], [1]), ("extend", [-1], [1]), ("extend", [0], [-1]),
           ("extend", [0], [25]), ("extend", [1], [65]), ("fork", [0], [2]), ("fork", [4], [1]), ("fork", [-1], [1]),
           ("fork", [0, 0], [1, 1]), ("fork", [0], [9]), ("fork", [0, 1], [1, 3]), ("fork", [1], [1]), ("free", [0, 2, 0]), ("free", [4]),
           ("extend", [1], [17]), ("fork", [0, 0], [1, 3])]
    for name, *lists in bad:
        before = (list(map(list, c.model.rows)), list(c.model.lens), list(c.model.refs))
        _apply(c, name, *lists)
        assert (c.model.rows, c.model.lens, c.model.refs) == before
    _apply(c, "fork", [0], [1])  # one page is left
    _apply(c, "extend", [0], [8])  # the last page has room
    ft = c.ft
    for n in (-1, 5):
        assert ft.kv_free(c.kv.h, n, c.lens.data_ptr()) == ft.FT_ERR_ARG
        assert ft.kv_extend(c.kv.h, n, c.lens.data_ptr(), c.lens.data_ptr()) == ft.FT_ERR_ARG
        assert ft.kv_fork(c.kv.h, n, c.lens.data_ptr(), c.lens.data_ptr()) == ft.FT_ERR_ARG
    assert ft.kv_extend(c.kv.h, 1, c.lens.data_ptr(), None) == ft.FT_ERR_ARG
    assert ft.kv_fork(c.kv.h, 1, None, c.lens.data_ptr()) == ft.FT_ERR_ARG
    assert ft.kv_free(c.kv.h, 1, None) == ft.FT_ERR_ARG
    # a table that names pages outside the pool, or pages that nobody holds, is found before anything moves
    c.table[0, 0] = 99
    c.kv.free(1, c.ints([0]))
    assert c.kv.status() == ft.FT_ERR_DEVICE
    assert c.lens.cpu().tolist() == c.model.lens


# ------------------------------------------------------------- norm, rotation, store

def _rope_case(D, page, kind, rot, pair, T, *, Hq=6, Hkv=2, ld_extra=0, norm="qk", in_place=False, seed=0, L=2):
    lens = [37, 0, 300, 5]
    c = Cache(lens, D=D, page=page, kind=kind, L=L, Hq=Hq, Hkv=Hkv, T_max=max(1, T), seed=seed)
    torch = c.torch
    rng = np.random.default_rng(seed)
    places = [(r, i) for r, n in enumerate(lens) for i in range(n)]
    pick = [places[i] for i in rng.permutation(len(places))[:T]]
    row_of, pos = [a for a, _ in pick], [b for _, b in pick]
    for i in range(0, T, 7):
        if T > 1:
            row_of[i] = -1  # padding
    max_pos = 301
    ld = (Hq + 2 * Hkv) * D + ld_extra
    qkv = c.randn(T, ld, scale=2.0)
    cs = torch.randn(max_pos, max(1, rot), generator=c.gen, device="cuda")
    wq = c.randn(D) if "q" in norm else None
    wk = c.randn(D) if "k" in norm else None
    q_out = qkv if in_place else torch.full((T, Hq * D + 8), 7.0, dtype=c.dt, device="cuda")
    x, before = qkv.double().cpu().numpy(), c.pool.clone()
    raw = qkv.clone()
    ro, po = c.ints(row_of), c.ints(pos)
    c.kv.qk_rope_store(L - 1, T, qkv, ld, ro, po, q_out, ld if in_place else Hq * D + 8, q_norm=wq, k_norm=wk, eps=1e-5,
                       cos_sin=cs, max_pos=max_pos, rot=rot, pair=pair)
    assert c.kv.status() == c.ft.FT_OK
    got_q, got = q_out.double().cpu().numpy(), c.pool.double().cpu().numpy()
    csh = cs.double().cpu().numpy()
    wqh, wkh = (None if w is None else w.double().cpu().numpy() for w in (wq, wk))
    want = before.double().cpu().numpy()
    # one rounding of the result; the fp32 steps before it (mean of D squares, root, two products and a
    # sum) are off by less than 2^-18 of the pair's magnitude
    u = U[kind]

    def close(a, b, size):
        return np.all(np.abs(a - b) <= u * np.abs(b) + 2.0 ** -18 * size + 1e-7)

    for t in range(T):
        for h in range(Hq + Hkv):
            v = x[t, h * D:(h + 1) * D]
            w = wqh if h < Hq else wkh
            y = okv.normed(v, w, 1e-5)
            cos, sin = csh[pos[t], :rot // 2], csh[pos[t], rot // 2:rot]
            z = okv.rotated(y, cos, sin, pair) if rot else y
            size = np.abs(y).max() * max(1.0, np.abs(csh[pos[t]]).max()) * 2
            if h < Hq:
                g = got_q[t, h * D:(h + 1) * D]
                assert (np.all(g == 0) if row_of[t] < 0 else close(g, z, size)), (t, h)
            elif row_of[t] >= 0:
                p = c.model.rows[row_of[t]][pos[t] // page]
                o = pos[t] % page
                assert close(got[p, L - 1, 0, h - Hq, o], z, size), (t, h)
                want[p, L - 1, 0, h - Hq, o] = got[p, L - 1, 0, h - Hq, o]
        if row_of[t] >= 0:
            p, o = c.model.rows[row_of[t]][pos[t] // page], pos[t] % page
            want[p, L - 1, 1, :, o] = x[t, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].reshape(Hkv, D)
    assert np.array_equal(got, want)  # values bit for bit, nothing else in the pool touched
    if in_place:
        assert torch.equal(q_out[:, Hq * D:], raw[:, Hq * D:])
    else:
        assert bool((q_out[:, Hq * D:] == 7).all())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("D,page,rot", [(64, 16, 64), (64, 32, 16), (128, 64, 128), (128, 16, 48), (256, 128, 64), (256, 32, 256),
                                        (256, 64, 0)])
def test_rope_store(D, page, rot, pair, kind):
    _rope_case(D, page, kind, rot, pair, 40, seed=rot)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (32, 4), (24, 3)])
@pytest.mark.parametrize("T", [1, 3, 200])
def test_rope_heads_and_strides(Hq, Hkv, T):
    _rope_case(128, 64, "bf16", 128, False, T, Hq=Hq, Hkv=Hkv, ld_extra=24, seed=T)


@pytest.mark.parametrize("norm", ["", "q", "k"])
def test_rope_without_norms_and_in_place(norm):
    _rope_case(64, 16, "bf16", 64, False, 30, norm=norm)
    _rope_case(128, 16, "f16", 32, True, 30, norm=norm, in_place=True)


def test_rope_many_tokens():
    # enough tokens that a warp keeps a token over several steps of heads
    import torch
    T, Hq, Hkv, D, page = 4096, 32, 4, 64, 16
    c = Cache([T], D=D, page=page, Hq=Hq, Hkv=Hkv, T_max=T)
    qkv = c.randn(T, (Hq + 2 * Hkv) * D)
    cs = torch.randn(T, D, generator=c.gen, device="cuda")
    out = torch.empty(T, Hq * D, dtype=c.dt, device="cuda")
    c.kv.qk_rope_store(0, T, qkv, qkv.shape[1], c.ints([0] * T), c.ints(range(T)), out, Hq * D, cos_sin=cs, max_pos=T, rot=D)
    assert c.kv.status() == c.ft.FT_OK
    x = qkv.double().view(T, -1, D)
    a, b, co, si = x[..., :32], x[..., 32:], cs.double()[:, None, :32], cs.double()[:, None, 32:]
    y = torch.cat([a * co - b * si, b * co + a * si], -1)
    size = 2 * x.abs().max() * cs.abs().max()
    assert bool(((out.double().view(T, Hq, D) - y[:, :Hq]).abs() <= 2.0 ** -8 * y[:, :Hq].abs() + 2.0 ** -18 * size).all())
    pg = c.table[0].long()
    k = c.pool[pg, 0, 0].permute(0, 2, 1, 3).reshape(T, Hkv, D).double()
    v = c.pool[pg, 0, 1].permute(0, 2, 1, 3).reshape(T, Hkv, D)
    assert bool(((k - y[:, Hq:Hq + Hkv]).abs() <= 2.0 ** -8 * y[:, Hq:Hq + Hkv].abs() + 2.0 ** -18 * size).all())
    assert torch.equal(v, qkv.view(T, -1, D)[:, Hq + Hkv:])


def test_rope_refusals():
    c = Cache([20, 0], D=64, page=16, L=2, Hq=4, Hkv=2, T_max=8, row_pages=3)
    ft, torch = c.ft, c.torch
    qkv, q, cs = c.randn(4, 512), c.randn(4, 256), torch.ones(64, 64, device="cuda")
    ro, po = c.ints([0, 0, 0, 0]), c.ints([0, 1, 2, 3])
    p = lambda t: t.data_ptr()  # noqa: E731

    def call(layer=0, T=4, qkv_=None, ld=512, ro_=None, q_=None, ldq=256, wq=None, eps=1e-6, cs_=None, mp=64, rot=64, pair=0):
        return ft.qk_rope_store(c.kv.h, layer, T, p(qkv) if qkv_ is None else qkv_, ld, p(ro) if ro_ is None else ro_, p(po),
                                p(q) if q_ is None else q_, ldq, wq, None, eps, p(cs) if cs_ is None else cs_, mp, rot, pair)

    assert call() == ft.FT_OK and call(T=0) == ft.FT_OK
    for kw in (dict(layer=2), dict(layer=-1), dict(T=-1), dict(qkv_=0), dict(ld=504), dict(ld=516), dict(ro_=0), dict(q_=0),
               dict(ldq=248), dict(ldq=258), dict(qkv_=p(qkv) + 2), dict(wq=p(qkv) + 2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(cs_=0), dict(cs_=p(cs) + 4), dict(mp=0), dict(rot=8), dict(rot=80), dict(rot=-16),
               dict(pair=2), dict(q_=p(qkv))):
        assert call(**kw) == ft.FT_ERR_ARG, kw
    assert c.kv.status() == ft.FT_OK
    # places that are not there: treated as padding and reported
    for r, x in ((2, 0), (-2, 0), (0, -1), (0, 32), (0, 48), (0, 64), (1, 0), (0, 2 ** 31 - 1)):
        pool = c.pool.clone()
        ro.fill_(-1)
        ro[1], po[1] = r, x
        q.fill_(7)
        c.kv.qk_rope_store(0, 4, qkv, 512, ro, po, q, 256, cos_sin=cs, max_pos=64, rot=64)
        assert c.kv.status() == ft.FT_ERR_DEVICE, (r, x)
        assert torch.equal(pool, c.pool) and bool((q == 0).all())


def test_init_refusals():
    c = Cache([20], D=64, page=16, Hq=4, Hkv=2)
    ft = c.ft
    p = [t.data_ptr() for t in (c.pool, c.table, c.lens, c.refs)]
    good = [1, 4, 2, 64, 16, c.n_pages, 1, c.row_pages, 0, 4, 1] + p + [None]
    st, h = ft.kv_init(*good)
    assert st == ft.FT_OK
    ft.kv_destroy(h)
    for i, v in ((0, 0), (1, 3), (1, 0), (1, 516), (2, 0), (3, 96), (3, 32), (4, 8), (4, 256), (5, 0), (6, 0), (7, 0), (8, 2),
                 (9, 0), (10, 0), (10, 1025), (11, 0), (11, p[0] + 64), (12, 0), (13, p[2] + 2), (14, 0), (7, 1 << 27),
                 (6, 65537)):
        bad = list(good)
        bad[i] = v
        st, h = ft.kv_init(*bad)
        assert st == ft.FT_ERR_ARG and h is None, (i, v)
    assert ft.kv_scratch_bytes(32, 4, 128, 100, 8, 64, 8) > 0
    ft.kv_destroy(None)
