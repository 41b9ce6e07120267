"""ft_beam_select against the oracle: which continuations, in which order, and their scores."""
import math

import numpy as np
import pytest

from oracle import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# A score is off by its own rounding (U of it) and by what the sum over the vocabulary is, in roundings of 2^-24: 4 for
# ex2 (2 ulp), 13 for its arguments (a term of weight w has an argument of -log2 w, and the sum of w log2(1/w) is at most
# log2 V < 18.. 24, times log 2), 21 additions in a thread and a warp, 8 in a CTA, 70 over a row's chunks and lanes, 3 for
# the constant that stands for log2(e), 8 for the two exponentials that join sums, 1 for the logarithm.
LSE = 132 * U


def _dt(kind):
    import torch

    import moe_expert_cache_gb300 as ft
    return {"bf16": (torch.bfloat16, ft.FT_T_BF16), "f16": (torch.float16, ft.FT_T_F16), "f32": (torch.float32, ft.FT_T_F32)}[kind]


def _logits(R, V, kind, seed=0, extra=0, offset=0, scale=3.0):
    """[R, V] view of rows of V + extra values that start `offset` values into a buffer; NaN around them."""
    import torch
    dt, _ = _dt(kind)
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = V + extra
    buf = torch.full((offset + R * ld + 16,), float("nan"), dtype=dt, device="cuda")
    x = torch.as_strided(buf, (R, V), (ld, 1), offset)
    x.copy_((torch.randn(R, V, generator=g, device="cuda") * scale).to(dt))
    return x, ld


def _check(B, K, N, x, ld, scores, *, done=None, eos=-1, rows=None, beams=None, kind="f32", R_max=None, N_max=None,
           status=None, out=None):
    import torch

    import moe_expert_cache_gb300 as ft
    V = x.shape[1]
    bm = beams or ft.Beams(V, R_max or max(1, B * K), N_max or N, dtype=_dt(kind)[1])
    sc = torch.tensor(scores, dtype=torch.float32, device="cuda") if isinstance(scores, (list, np.ndarray)) else scores
    dn = None if done is None else torch.tensor(done, dtype=torch.int32, device="cuda")
    rw = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    s0 = sc.cpu().numpy().astype(np.float64)
    o = out or (torch.full((B, N), 7.0, device="cuda"),) + tuple(torch.full((B, N), -7, dtype=torch.int32, device="cuda") for _ in range(3))
    bm.select(B, K, N, x, ld, sc, o[0], o[1], o[2], rows=rw, done=dn, eos=eos, out_done=o[3])
    assert bm.status() == (ft.FT_OK if status is None else status)
    got = [t.cpu().numpy() for t in o]
    xs = x.double().cpu().numpy()
    for b in range(B):
        e = slice(b * K, (b + 1) * K)
        want = gen.beam_select(xs[e], s0[e], N, done=None if done is None else done[e], eos=eos)
        n = sum(1 for w in want if w[1] >= 0)
        back = {} if rows is None else {rows[b * K + k]: k for k in range(K)}
        lse = {}
        for i in range(N):
            score, parent, token, ended = (g[b, i] for g in got)
            if i >= n:
                assert (score, parent, token, ended) == (-math.inf, -1, -1, 0)
                continue
            k = parent - b * K if rows is None else back[parent]
            assert 0 <= k < K and 0 <= token < V and ended == int(token == eos)
            if done is not None and done[b * K + k]:
                assert token == eos and score == s0[b * K + k]
                true = s0[b * K + k]
            else:
                if k not in lse:
                    row = xs[b * K + k]
                    lse[k] = row.max(), math.log(math.fsum(np.exp(row - row.max())))
                true = s0[b * K + k] + ((xs[b * K + k, token] - lse[k][0]) - lse[k][1])
            tol = LSE + U * abs(true)
            assert abs(score - true) <= tol, (b, i, score, true)
            # in its place: beams whose scores are this near may be told apart by their sums' errors
            assert abs(true - want[i][0]) <= 2 * tol, (b, i, true, want[i])
            if (k, token) != want[i][1:3]:
                assert any(abs(want[j][0] - want[i][0]) <= 2 * tol and want[j][1] != want[i][1]
                           for j in (i - 1, i + 1) if 0 <= j < n) or i == n - 1
        # of each beam exactly its best, equal logits by token
        for k in range(K):
            mine = [int(v) for p, v in zip(got[1][b, :n], got[2][b, :n]) if (p - b * K if rows is None else back[p]) == k]
            if done is not None and done[b * K + k]:
                assert len(mine) <= 1
                continue
            order = np.argsort(-xs[b * K + k], kind="stable")[:len(mine)]
            assert mine == order.tolist()
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 2047, 2049, 8191, 8193, 32000, 100003])
def test_vocabularies(V, kind):
    x, ld = _logits(6, V, kind, seed=V, extra=3, offset=1)
    _check(2, 3, 5, x, ld, -np.arange(6.0) / 4, kind=kind)


@pytest.mark.parametrize("B,K,N", [(1, 1, 1), (1, 1, 64), (1, 64, 64), (3, 5, 10), (70, 4, 4), (2, 16, 33), (130, 8, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_beams(B, K, N, kind):
    x, ld = _logits(B * K, 9001, kind, seed=B + K, extra=7)
    r = np.random.default_rng(K)
    _check(B, K, N, x, ld, (-3 * r.random(B * K)).astype(np.float32), kind=kind, R_max=B * K + 3, N_max=64,
           rows=[int(v) for v in r.permutation(2000)[:B * K]])


def test_every_alignment_of_a_row():
    for kind, n in (("f32", 4), ("bf16", 8)):
        for offset in range(n):
            x, ld = _logits(3, 4099, kind, seed=offset, extra=1, offset=offset)
            _check(1, 3, 6, x, ld, [0.0, -0.5, -1.0], kind=kind)


def test_many_candidates_to_join():
    # 16 beams of 13 chunks of 64 candidates: more than the list of the joining CTA holds
    x, ld = _logits(16, 100003, "bf16", seed=5)
    _check(1, 16, 64, x, ld, [0.0] * 16, kind="bf16")
    # ... all of them equal
    x.zero_()
    got = _check(1, 16, 64, x, ld, [0.0] * 16, kind="bf16")
    assert got[1][0].tolist() == [0] * 64 and got[2][0].tolist() == list(range(64))


def test_more_candidates_than_the_threads_hold():
    # 32 beams of more than 128 chunks of 64 candidates
    x, ld = _logits(32, 600003, "f32", seed=11)
    _check(1, 32, 64, x, ld, (-np.arange(32) / 64).astype(np.float32))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5000, 40000])
def test_order_of_the_logits(V, kind):
    import torch
    x, ld = _logits(4, V, kind)
    x[0] = torch.arange(V, device="cuda") / 1000
    x[1] = -torch.arange(V, device="cuda") / 1000
    x[2] = 1.0                                  # all equal
    x[3] = (torch.arange(V, device="cuda") % 3 == 1).to(x.dtype)
    x[2, ::2] = 0.0
    x[2, 1::2] = -0.0                           # ... in value
    for N in (1, 4, 64):
        for r in range(4):
            _check(1, 1, N, x[r:r + 1], ld, [0.0], kind=kind)
        _check(1, 4, N, x, ld, [0.0, -0.1, -0.2, -0.3], kind=kind)


def test_forbidden_tokens():
    import torch
    inf = math.inf
    for kind in ("f32", "bf16", "f16"):
        x, ld = _logits(5, 20000, kind, seed=2)
        lowest = torch.finfo(x.dtype).min
        keep = x[0, 17777].clone()
        x[0] = -inf
        x[0, 17777] = keep                      # one token
        x[1] = -inf                             # none
        x[2, ::2] = -inf
        x[3, 3:] = lowest                       # the type's lowest value is a logit
        x[4] = lowest
        for N in (1, 3, 8):
            for r in range(5):
                _check(1, 1, N, x[r:r + 1], ld, [-1.0], kind=kind)
            _check(1, 5, N, x, ld, [0.0, -1.0, -2.0, -3.0, -4.0], kind=kind)
    # fewer tokens than candidates, in all beams
    x, ld = _logits(3, 3000, "f32")
    x[:] = -inf
    x[0, 5], x[2, 2999], x[2, 0] = 1.0, 2.0, 2.0
    got = _check(1, 3, 8, x, ld, [0.0, 0.0, -5.0])
    assert got[2][0].tolist() == [5, 0, 2999] + [-1] * 5


def test_tokens_of_one_group():
    # nearly all that may be chosen lies with few threads: more than the list holds
    x, ld = _logits(1, 8192, "f32", seed=3)
    keep = x.clone()
    x[:] = -math.inf
    for lane in range(0, 31 * 4):  # 124 threads' vectors of four, in every step of 1024
        for j in range(8):
            a = j * 1024 + lane * 4
            x[:, a:a + 4] = keep[:, a:a + 4]
    _check(1, 1, 64, x, ld, [0.0], R_max=700)


def test_large_logits():
    for v in (1e4, 1e6, 3e7, 1e30, 3.4e38):
        x, ld = _logits(2, 5000, "f32", seed=1, scale=1.0)
        x[0] *= v / 100 if v < 1e38 else 1.0
        x[1] = v
        x[1, 7] = -v
        import torch
        import moe_expert_cache_gb300 as ft
        bm = ft.Beams(5000, 2, 4)
        s = torch.zeros(2, device="cuda")
        o = torch.empty(2, 4, device="cuda"), *(torch.empty(2, 4, dtype=torch.int32, device="cuda") for _ in range(2))
        bm.select(2, 1, 4, x, ld, s, *o)
        assert bm.status() == ft.FT_OK
        want = [gen.beam_select(x[r:r + 1].double().cpu().numpy(), [0.0], 4) for r in range(2)]
        for r in range(2):
            assert o[2][r].tolist() == [w[2] for w in want[r]]
            for got, w in zip(o[0][r].tolist(), want[r]):
                # the constant that stands for log2(e) is off by 2^-25: so is a difference of logits, where a sum is of
                # terms apart; here those within a few of the largest count
                assert abs(got - w[0]) <= LSE + U * abs(w[0]), (v, got, w)


def test_bad_rows_and_scores():
    import moe_expert_cache_gb300 as ft
    x, ld = _logits(6, 30000, "f32", seed=9)
    x[1, 29999] = math.nan
    x[3, 0] = math.inf
    _check(2, 3, 5, x, ld, [0.0] * 6, status=ft.FT_ERR_DEVICE)
    x, ld = _logits(6, 300, "f32", seed=9)
    _check(2, 3, 5, x, ld, [0.0, math.nan, -1.0, math.inf, -0.5, -2.0], status=ft.FT_ERR_DEVICE)
    _check(2, 3, 5, x, ld, [0.0, -math.inf, -math.inf, -math.inf, -math.inf, -math.inf])


def test_ended_beams():
    x, ld = _logits(8, 7001, "bf16", seed=4)
    x[1] = math.nan  # the row of an ended beam, of a beam without a score: not read
    x[6] = math.nan
    s = [-1.0, -1.2, -0.3, -9.0, -1.0, -1.0, -math.inf, -1e30]
    for N in (4, 8):
        _check(2, 4, N, x, ld, s, done=[0, 1, 0, 5, 0, 0, 0, 1], eos=33, kind="bf16")
    _check(2, 4, 3, x, ld, s, done=[1] * 8, eos=0, kind="bf16")
    x[1], x[6] = 0.0, 1.0
    _check(2, 4, 4, x, ld, s, eos=33, kind="bf16")  # no beam has ended yet
    # among the best: the beam ends now
    x[:, 33] = 30
    got = _check(2, 4, 4, x, ld, s, done=[0] * 8, eos=33, kind="bf16")
    assert got[3].sum() >= 2


def test_in_place_and_again():
    import torch

    import moe_expert_cache_gb300 as ft
    B, K, V = 3, 4, 5003
    x, ld = _logits(B * K, V, "f32", seed=6)
    bm = ft.Beams(V, 50, 8)
    done = [0, 1, 0, 0] * B
    a = _check(B, K, K, x, ld, [0.0, -1.0, -2.0, -3.0] * B, done=done, eos=9, beams=bm)
    sc = torch.tensor([0.0, -1.0, -2.0, -3.0] * B, device="cuda")
    dn = torch.tensor(done, dtype=torch.int32, device="cuda")
    par, tok = (torch.empty(B * K, dtype=torch.int32, device="cuda") for _ in range(2))
    bm.select(B, K, K, x, ld, sc, sc, par, tok, done=dn, eos=9, out_done=dn)
    assert bm.status() == ft.FT_OK
    for got, want in zip((sc, par, tok, dn), a):
        assert np.array_equal(got.cpu().numpy().reshape(B, K), want)
    # the same handle with other sizes in between
    _check(1, 1, 8, x[:1], ld, [0.0], beams=bm)
    _check(12, 1, 2, x, ld, [0.0] * 12, beams=bm)
    _check(B, K, K, x, ld, [0.0, -1.0, -2.0, -3.0] * B, done=done, eos=9, beams=bm)
    bm.select(0, 4, 4, None, 0, None, None, None, None)
    bm.close()


def test_graph_and_stream():
    import torch

    import moe_expert_cache_gb300 as ft
    s = torch.cuda.Stream()
    B, K, V = 4, 4, 33333
    x, ld = _logits(B * K, V, "bf16", seed=7)
    bm = ft.Beams(V, B * K, K, dtype=ft.FT_T_BF16, stream=s.cuda_stream)
    sc = torch.zeros(B * K, device="cuda")
    par, tok = (torch.empty(B * K, dtype=torch.int32, device="cuda") for _ in range(2))

    def steps():
        for _ in range(3):  # (each takes the scores that the one before it left)
            bm.select(B, K, K, x, ld, sc, sc, par, tok)
    torch.cuda.synchronize()
    steps()
    torch.cuda.synchronize()
    want = [t.clone() for t in (sc, par, tok)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        steps()
    for _ in range(2):
        sc.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((sc, par, tok), want))
    assert bm.status() == ft.FT_OK


def test_rows_far_apart():
    # offsets past 32 bits
    import torch

    import moe_expert_cache_gb300 as ft
    V, ld = 1000, 1 << 29
    buf = torch.zeros(9 * ld + V, dtype=torch.bfloat16, device="cuda")  # 9.7 GB, 4.8e9 values
    x = torch.as_strided(buf, (10, V), (ld, 1))
    g = torch.Generator(device="cuda").manual_seed(0)
    x.copy_(torch.randn(10, V, generator=g, device="cuda"))
    _check(2, 5, 5, x, ld, [0.0] * 10, kind="bf16")


def test_many_requests():
    # more rows than warps run at once
    x, ld = _logits(6000, 61, "f16", seed=8, extra=2)
    r = np.random.default_rng(0)
    _check(3000, 2, 3, x, ld, (-r.random(6000)).astype(np.float32), kind="f16")


def test_what_lies_around_the_outputs():
    import torch

    import moe_expert_cache_gb300 as ft
    B, K, N, V = 5, 3, 7, 2500
    x, ld = _logits(B * K, V, "bf16", seed=1)
    x[:, 3:] = -math.inf  # few candidates
    bm = ft.Beams(V, B * K, N, dtype=ft.FT_T_BF16)
    sc = torch.zeros(B * K, device="cuda")
    buf = torch.full((4, 4 + B * N + 4), 99, dtype=torch.int32, device="cuda")
    f = buf[0].view(torch.float32)
    bm.select(B, K, N, x, ld, sc, f[4:], buf[1, 4:], buf[2, 4:], eos=2, out_done=buf[3, 4:])
    assert bm.status() == ft.FT_OK
    assert (buf[:, :4] == 99).all() and (buf[:, 4 + B * N:] == 99).all()
    mid = slice(4, 4 + B * N)
    assert bool(((buf[2, mid] >= 0) & (buf[2, mid] < 3)).all()) and torch.equal(buf[3, mid] == 1, buf[2, mid] == 2)


def test_handles_at_once():
    # two handles on two streams, calls of both in flight
    import torch

    import moe_expert_cache_gb300 as ft
    B, K, V = 16, 4, 50003
    x, ld = _logits(B * K, V, "f32", seed=3)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sc = torch.zeros(B * K, device="cuda")
    hs = [ft.Beams(V, B * K, K, stream=s.cuda_stream) for s in streams]
    outs = [[[torch.empty(B * K, device="cuda")] + [torch.empty(B * K, dtype=torch.int32, device="cuda") for _ in range(2)]
             for _ in range(8)] for _ in hs]
    torch.cuda.synchronize()
    for i in range(8):
        for h, o in zip(hs, outs):
            h.select(B, K, K, x, ld, sc, *o[i])
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            assert all(torch.equal(a, b) for a, b in zip(t, outs[0][0]))


def test_refusals():
    import torch

    import moe_expert_cache_gb300 as ft
    B, K, N, V = 2, 3, 4, 100
    x, ld = _logits(B * K, V, "bf16")
    bm = ft.Beams(V, 6, 4, dtype=ft.FT_T_BF16)
    i = torch.zeros(400, dtype=torch.int32, device="cuda")
    f = torch.zeros(100, device="cuda")
    P, F, X = i.data_ptr(), f.data_ptr(), x.data_ptr()
    ok = dict(B=B, K=K, N=N, logits=X, ld=V, scores=F, rows=P, done=P + 128, eos=5, os=F + 128, op=P + 256, ot=P + 384, od=P + 512)

    def call(**kw):
        return ft.beam_select(bm.h, *{**ok, **kw}.values())
    assert call() == ft.FT_OK and bm.status() == ft.FT_OK
    for bad in (dict(B=-1), dict(B=3), dict(K=0), dict(K=65), dict(N=0), dict(N=5), dict(logits=None), dict(logits=X + 1), dict(ld=99),
                dict(ld=1 << 41), dict(scores=None), dict(scores=F + 2), dict(eos=-2), dict(eos=100), dict(eos=-1), dict(os=None),
                dict(op=None), dict(ot=None), dict(rows=P + 1), dict(done=P + 130), dict(od=P + 514), dict(os=F), dict(os=F + 4),
                dict(op=P), dict(op=P + 20), dict(ot=P + 256), dict(ot=P + 280), dict(od=P + 128), dict(od=P + 384), dict(os=X), dict(os=X + 64),
                dict(op=F + 20), dict(N=3, os=F + 4), dict(N=3, od=P + 132), dict(N=3, op=F), dict(N=3, od=P)):
        assert call(**bad) == ft.FT_ERR_ARG, bad
    assert call(N=3, os=F, od=P + 128) == ft.FT_OK  # in place
    assert call(rows=None, done=None, eos=-1, od=None) == ft.FT_OK
    assert bm.status() == ft.FT_OK
    assert ft.beam_scratch_bytes(V, 0, 6, 4) > 0
