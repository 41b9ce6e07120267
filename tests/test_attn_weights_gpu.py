"""Weights far below a row's largest one, in f16, whose smallest number is 2^-24: many of them together are a part of
the result that does not round away."""
import numpy as np
import pytest

from tests.kv_harness import U, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv,n,groups", [
    (64, 8, 8, 1, False),
    (64, 24, 8, 3, True),
    (128, 8, 8, 1, False),    # few rows that share nothing: the transposed form
    (128, 32, 8, 2, False),
    (128, 8, 8, 1, True),     # the same rows under a claim of no shared token: the form of many rows
    (128, 128, 8, 9, False),  # 144 rows: two row tiles
    (256, 8, 8, 1, False),
    (256, 16, 8, 2, True),
])
def test_many_weak_keys_behind_a_strong_one(D, Hq, Hkv, n, groups):
    # all requests read the same pages.  With 64 * 8 of them a CTA has whole requests, so that the first key, whose
    # score is 18 to 21 above the others' (weights of 2^-26 to 2^-30.3 of its own), is the reference of all that follow
    B, N, page = 64, 4096, 64
    c = Cache([N] * B, D=D, page=page, kind="f16", Hq=Hq, Hkv=Hkv, shared=N, T_max=B * n, seed=D + n)
    torch = c.torch
    kv = c.pool[c.table[0].long(), 0]                          # [pages, 2, Hkv, page, D]
    K = kv[:, 0].permute(1, 0, 2, 3).reshape(Hkv, N, D).clone() * 0.01
    V = kv[:, 1].permute(1, 0, 2, 3).reshape(Hkv, N, D).clone()
    K[:, :, 0] = -(18 + 3 * torch.rand(Hkv, N, generator=c.gen, device="cuda")).half()
    K[:, 0] = 0
    V[:] = V * 0.25 + 1
    V[:, 0] = 0
    c.pool[c.table[0].long(), 0, 0] = K.view(Hkv, -1, page, D).permute(1, 0, 2, 3)
    c.pool[c.table[0].long(), 0, 1] = V.view(Hkv, -1, page, D).permute(1, 0, 2, 3)
    q = c.randn(B * n, Hq * D, scale=0.01)
    q.view(B * n, Hq, D)[:, :, 0] = 1
    out, _ = c.attend([n] * B, q=q, scale=1.0, groups=([0, B], [0]) if groups else None)
    assert c.kv.status() == c.ft.FT_OK
    G, worst = Hq // Hkv, 0.0
    qd = q.double().view(B, n, Hkv, G, D)
    got = out.double().view(B, n, Hkv, G, D)
    for h in range(Hkv):
        s = torch.einsum("bngd,kd->bngk", qd[:, :, h], K[h].double())
        hidden = torch.arange(N, device="cuda")[None, :] > (N - n + torch.arange(n, device="cuda"))[:, None]
        w = s.masked_fill(hidden[None, :, None, :], -np.inf).softmax(-1)
        ref, mass = w @ V[h].double(), w @ V[h].double().abs()
        # the bound of every other test, with weights that lose up to 2^-33 of the largest one each (2^-25, the half of
        # f16's smallest number, on a reference that is 2^8 lower)
        tol = U["f16"] * ref.abs() + (U["f16"] + 2.0 ** -13) * mass + N * 2.0 ** -33 * float(V.abs().max()) + 1e-6
        err = (got[:, :, h] - ref).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        worst = max(worst, float((err / tol).max()))
    assert worst < 1
