"""Pins of the key/value cache's oracle: hand-worked tables, invariants on
random lives, closed forms and a dense brute force; and the host-side argument
checks of the entry points, which need no GPU."""
import math
import random

import numpy as np
import pytest

from oracle import kv as okv


def test_hand_worked_pages():
    m = okv.Pages(6, 4, 3, 4)
    assert m.extend([2, 0], [5, 4]) == []
    assert (m.rows, m.lens, m.refs) == ([[2], [], [0, 1], []], [4, 0, 5, 0], [1, 1, 1, 0, 0, 0])
    # row 2 has one full page and one token: the child shares page 0 and gets a copy of one token
    assert m.fork([2, 0], [1, 3]) == [(1, 3, 1)]
    assert m.rows == [[2], [0, 3], [0, 1], [2]] and m.refs == [2, 1, 2, 1, 0, 0]
    m.free([2])
    assert m.refs == [1, 0, 2, 1, 0, 0] and m.rows[2] == []
    # pages in use: 0, 2, 3; page 3 moves to 1
    assert m.compact() == [(3, 1, 4)]
    assert m.rows == [[2], [0, 1], [], [2]] and m.refs == [1, 1, 2, 0, 0, 0]
    with pytest.raises(okv.Refused, match="capacity"):
        m.extend([0, 1, 2], [8, 4, 12])
    with pytest.raises(okv.Refused, match="device"):
        m.fork([0], [1])
    assert m.table().tolist() == [[2, -1, -1], [0, 1, -1], [-1, -1, -1], [2, -1, -1]]


def test_random_lives_keep_the_invariants():
    rnd = random.Random(2)
    for _ in range(30):
        page = rnd.choice([1, 3, 4])
        m = okv.Pages(25, 8, 6, page)
        words = [[] for _ in range(8)]       # what each row says, token by token
        store = [[None] * page for _ in range(25)]
        for step in range(60):
            op = rnd.choice(["extend", "fork", "free", "compact"])
            try:
                if op == "extend":
                    rows = rnd.sample(range(8), rnd.randint(0, 3))
                    add = [rnd.randint(0, 7) for _ in rows]
                    m.extend(rows, add)
                    for r, a in zip(rows, add):
                        for j in range(a):
                            at = len(words[r])
                            words[r].append((step, r, j))
                            store[m.rows[r][at // page]][at % page] = (step, r, j)
                else:
                    if op == "fork":
                        empty = [r for r in range(8) if not m.lens[r]]
                        ch = rnd.sample(empty, rnd.randint(0, min(2, len(empty))))
                        pa = [rnd.randrange(8) for _ in ch]
                        copies = m.fork(pa, ch)
                        for p, c in zip(pa, ch):
                            words[c] = list(words[p])
                    elif op == "free":
                        rows = rnd.sample(range(8), rnd.randint(0, 2))
                        copies = m.free(rows)
                        for r in rows:
                            words[r] = []
                    else:
                        copies = m.compact()
                    for s, d, tok in copies:
                        store[d][:tok] = store[s][:tok]
            except okv.Refused:
                pass
            # every row still reads its own words; counts are the number of holders; rows have the pages they need
            held = [0] * 25
            for r in range(8):
                assert len(m.rows[r]) == -(-m.lens[r] // page) and m.lens[r] == len(words[r])
                assert [store[m.rows[r][i // page]][i % page] for i in range(m.lens[r])] == words[r]
                for p in m.rows[r]:
                    held[p] += 1
            assert held == m.refs


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(5, 4))
    # equal scores: the mean of what is seen; the last query sees all, the first of two one token less
    out, mass = okv.attention(np.zeros((2, 4)), rng.normal(size=(5, 4)), v, 2, 1.0)
    assert np.allclose(out[1], v.mean(0)) and np.allclose(out[0], v[:4].mean(0))
    assert np.allclose(mass[1], np.abs(v).mean(0))
    # one dominating key; queries before the first token
    k = np.zeros((3, 4))
    k[1, 0] = 1
    out, _ = okv.attention(np.array([[800.0, 0, 0, 0]] * 5), k, v[:3], 5, 1.0)
    assert np.allclose(out[4], v[1]) and np.all(out[:2] == 0) and np.allclose(out[2], v[0])
    # against an independent scalar computation
    q, k = rng.normal(size=(1, 4)), rng.normal(size=(5, 4))
    w = [math.exp(0.3 * sum(a * b for a, b in zip(q[0], k[j]))) for j in range(5)]
    want = [sum(w[j] * v[j][i] for j in range(5)) / sum(w) for i in range(4)]
    assert np.allclose(okv.attention(q, k, v, 1, 0.3)[0][0], want)


def test_rotation_and_norm():
    x = np.array([3.0, 4.0, 1.0, 2.0])
    assert np.allclose(okv.normed(x, None, 0), x)
    assert np.allclose(okv.normed([3.0, 4.0], [1.0, 2.0], 0.0), np.array([3.0, 8.0]) / math.sqrt(12.5))
    # a quarter turn of each pair: half form pairs (0,2), (1,3); pair form (0,1), (2,3)
    c, s = np.zeros(2), np.ones(2)
    assert np.allclose(okv.rotated(x, c, s, False), [-1, -2, 3, 4])
    assert np.allclose(okv.rotated(x, c, s, True), [-4, 3, -2, 1])
    # rotations keep lengths and differences of angles decide products
    a, b = 0.7, 1.9
    q = okv.rotated(x, np.cos([a, 2 * a]), np.sin([a, 2 * a]), False)
    k = okv.rotated(x[::-1], np.cos([b, 2 * b]), np.sin([b, 2 * b]), False)
    q2 = okv.rotated(x, np.cos([a + 1, 2 * a + 2]), np.sin([a + 1, 2 * a + 2]), False)
    k2 = okv.rotated(x[::-1], np.cos([b + 1, 2 * b + 2]), np.sin([b + 1, 2 * b + 2]), False)
    assert np.isclose(q @ k, q2 @ k2) and np.isclose(q @ q, x @ x)
    assert np.allclose(okv.rotated(x, np.ones(1), np.zeros(1), False), x)  # values past the rotated ones stay


def test_copy_pages_touches_only_the_tokens():
    pool = np.arange(4 * 1 * 2 * 1 * 3 * 2).reshape(4, 1, 2, 1, 3, 2)
    ref = pool.copy()
    okv.copy_pages(pool, [(0, 2, 2)])
    assert np.array_equal(pool[2, :, :, :, :2], ref[0, :, :, :, :2]) and np.array_equal(pool[2, :, :, :, 2], ref[2, :, :, :, 2])
    assert np.array_equal(pool[[0, 1, 3]], ref[[0, 1, 3]])


def test_host_checks_need_no_gpu():
    import moe_expert_cache_gb300 as ft
    assert ft.kv_page_bytes(48, 4, 128, 64) == 48 * 2 * 4 * 64 * 128 * 2
    for bad in ((0, 4, 128, 64), (1, 0, 128, 64), (1, 1, 96, 64), (1, 1, 64, 8), (1, 1, 64, 256)):
        assert ft.kv_page_bytes(*bad) == 0
    assert ft.kv_init(1, 4, 2, 64, 16, 8, 1, 4, 0, 4, 1, None, None, None, None, None) == (ft.FT_ERR_ARG, None)
    assert ft.kv_init(1, 4, 3, 64, 16, 8, 1, 4, 0, 4, 1, 1024, 1024, 1024, 1024, None) == (ft.FT_ERR_ARG, None)
    assert ft.kv_extend(None, 0, None, None) == ft.FT_ERR_ARG
    assert ft.kv_fork(None, 0, None, None) == ft.FT_ERR_ARG
    assert ft.kv_free(None, 0, None) == ft.FT_ERR_ARG
    assert ft.kv_compact(None) == ft.FT_ERR_ARG
    assert ft.qk_rope_store(None, 0, 1, None, 0, None, None, None, 0, None, None, 0.0, None, 0, 0, 0) == ft.FT_ERR_ARG
    assert ft.attn_plan(None, 0, 0, None, None, 0, None, None) == ft.FT_ERR_ARG
    assert ft.attn_forward(None, 0, None, 0, None, 0, 1.0) == ft.FT_ERR_ARG
    assert ft.kv_last(None, None) == ft.FT_ERR_ARG
    assert ft.kv_status(None) == ft.FT_ERR_ARG
    ft.kv_destroy(None)
