"""The norm-rotate-store pass over prompts: enough tokens that a warp keeps a token's factors over several steps of
heads and over the change from queries to keys, with norms, in every form and head size."""
import numpy as np
import pytest

from tests.kv_harness import U, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,Hq,Hkv,rot,pair,kind,T", [
    (64, 16, 32, 8, 64, True, "bf16", 3001),
    (64, 32, 31, 1, 32, False, "f16", 5000),
    (128, 64, 32, 4, 128, False, "bf16", 2500),
    (128, 128, 24, 3, 48, True, "f16", 1999),
    (256, 32, 16, 2, 64, False, "f16", 1001),
    (256, 64, 10, 10, 256, True, "bf16", 2047),
    (128, 16, 16, 2, 0, False, "bf16", 4001),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompt_with_norms(D, page, Hq, Hkv, rot, pair, kind, T, in_place):
    import torch
    c = Cache([T + 9], D=D, page=page, Hq=Hq, Hkv=Hkv, kind=kind, L=2, T_max=T, seed=T)
    ld = (Hq + 2 * Hkv) * D + 8
    qkv = c.randn(T, ld, scale=2.0)
    cs = torch.randn(T + 9, max(rot, 16), generator=c.gen, device="cuda")[:, :max(rot, 1)].contiguous()
    wq, wk = c.randn(D), c.randn(D)
    rng = np.random.default_rng(T)
    where = rng.permutation(T + 9)[:T]
    row = np.zeros(T, dtype=int)
    row[::11] = -1
    x = qkv.double()[:, :(Hq + 2 * Hkv) * D].reshape(T, -1, D)
    raw, before = qkv.clone(), c.pool.clone()
    out = qkv if in_place else torch.empty(T, Hq * D, dtype=c.dt, device="cuda")
    c.kv.qk_rope_store(1, T, qkv, ld, c.ints(row), c.ints(where), out, ld if in_place else Hq * D, q_norm=wq, k_norm=wk, eps=1e-5,
                       cos_sin=cs, max_pos=T + 9, rot=rot, pair=pair)
    assert c.kv.status() == c.ft.FT_OK
    y = x[:, :Hq + Hkv] / (x[:, :Hq + Hkv].square().mean(-1, keepdim=True) + 1e-5).sqrt()
    y = torch.cat([y[:, :Hq] * wq.double(), y[:, Hq:] * wk.double()], 1)
    z, pos = y.clone(), torch.from_numpy(where).cuda()
    if rot:
        co, si = (t[:, None] for t in cs.double()[pos].split(rot // 2, -1))
        i = torch.arange(rot // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if pair else (i, i + rot // 2)
        z[..., a], z[..., b] = y[..., a] * co - y[..., b] * si, y[..., b] * co + y[..., a] * si
    # one rounding of the result; the fp32 steps before it are off by less than 2^-18 of the pair's magnitude
    size = 2 * y.abs().amax(-1, keepdim=True) * max(1.0, float(cs.abs().max()))
    tol = U[kind] * z.abs() + 2.0 ** -18 * size + 1e-7
    live = torch.from_numpy(row >= 0).cuda()
    got = out[:, :Hq * D].double().view(T, Hq, D)
    assert bool(((got - z[:, :Hq]).abs() <= tol[:, :Hq])[live].all()) and bool((got[~live] == 0).all())
    pg, o = c.table[0].long()[pos // page][live], (pos % page)[live]
    k = c.pool[pg, 1, 0, :, o].double()
    assert bool(((k - z[live, Hq:]).abs() <= tol[live, Hq:]).all())
    assert torch.equal(c.pool[pg, 1, 1, :, o].double(), x[live, Hq + Hkv:])
    c.pool[pg, 1, :, :, o] = before[pg, 1, :, :, o]
    assert torch.equal(c.pool, before)  # nothing else in the pool is touched
    if in_place:
        assert torch.equal(qkv[:, Hq * D:], raw[:, Hq * D:])
