"""Shared helpers of the key/value cache's GPU tests: a cache with a random
page layout, its host copy, and the comparison with the fp64 oracle."""
from __future__ import annotations

import numpy as np

from oracle import kv as okv

# Unit roundoffs of the two types.
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def attn_tolerance(kind, ref, mass, n_keys, vmax):
    """Elementwise bound on the kernel's error, from its roundings: the output's (u |ref|), the
    weights' (each off by u of itself: u * sum w|v|; f16 weights under 2^-14 of the largest lose up
    to 2^-25 each), and 2^-13 of sum w|v| for the fp32 scores (D products of magnitude up to a few
    tens, 2^-24 each, doubled by the exponential) and sums."""
    u = U[kind]
    sub = n_keys * 2.0 ** -25 * vmax if kind == "f16" else 0.0
    return u * np.abs(ref) + (u + 2.0 ** -13) * mass + sub + 1e-6


class Cache:
    """A pool, control arrays and handle; rows laid out over shuffled pages."""

    def __init__(self, lens, *, L=1, Hq=4, Hkv=2, D=64, page=16, kind="bf16", shared=0, seed=0, spare=2, row_pages=None,
                 T_max=64, B_max=None, stream=0, fill=1.0, n_pages=None):
        import torch

        import moe_expert_cache_gb300 as ft
        self.ft, self.torch = ft, torch
        self.L, self.Hq, self.Hkv, self.D, self.page, self.kind = L, Hq, Hkv, D, page, kind
        self.dt = torch.bfloat16 if kind == "bf16" else torch.float16
        rng = np.random.default_rng(seed)
        np_of = [-(-x // page) for x in lens]
        P = shared // page
        need = P + sum(max(0, n - P) for n in np_of)
        self.n_pages = n_pages or need + spare
        ids = list(rng.permutation(self.n_pages))
        common, at = [int(i) for i in ids[:P]], P
        self.row_pages = row_pages or max(np_of + [1])
        self.model = okv.Pages(self.n_pages, len(lens), self.row_pages, page)
        for r, (n, x) in enumerate(zip(np_of, lens)):
            own = max(0, n - P)
            self.model.rows[r] = common[:n] + [int(i) for i in ids[at:at + own]]
            self.model.lens[r] = x
            at += own
            for p in self.model.rows[r]:
                self.model.refs[p] += 1
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (self.n_pages, L, 2, Hkv, page, D)
        self.pool = (torch.randn(shape, generator=g, device="cuda") * fill).to(self.dt)
        self.table = torch.from_numpy(self.model.table()).cuda()
        self.lens = torch.tensor(self.model.lens, dtype=torch.int32, device="cuda")
        self.refs = torch.tensor(self.model.refs, dtype=torch.int32, device="cuda")
        self.gen = g
        self.kv = ft.KvCache(L, Hq, Hkv, D, page, self.n_pages, len(lens), self.row_pages, self.pool, self.table, self.lens,
                             self.refs, dtype=ft.FT_KV_BF16 if kind == "bf16" else ft.FT_KV_F16, T_max=T_max,
                             B_max=B_max or max(1, len(lens)), stream=stream)

    def ints(self, v):
        return self.torch.tensor(list(v), dtype=self.torch.int32, device="cuda")

    def randn(self, *shape, scale=1.0):
        return (self.torch.randn(*shape, generator=self.gen, device="cuda") * scale).to(self.dt)

    def poison(self, value):
        """Put `value` wherever no row keeps a token."""
        used = np.zeros((self.n_pages, self.page), dtype=bool)
        for r, pages in enumerate(self.model.rows):
            for i, p in enumerate(pages):
                used[p, :max(0, min(self.page, self.model.lens[r] - i * self.page))] = True
        m = self.torch.from_numpy(~used).cuda()[:, None, None, None, :, None]
        self.pool.masked_fill_(m, value)

    def host_pool(self):
        return self.pool.double().cpu().numpy()

    def keys_values(self, pool, row, layer, h):
        n = self.model.lens[row]
        t = [(self.model.rows[row][i // self.page], i % self.page) for i in range(n)]
        k = np.array([pool[p, layer, 0, h, o] for p, o in t]).reshape(n, self.D)
        v = np.array([pool[p, layer, 1, h, o] for p, o in t]).reshape(n, self.D)
        return k, v

    def check_control(self):
        m = self.model
        assert np.array_equal(self.table.cpu().numpy(), m.table())
        assert self.lens.cpu().tolist() == m.lens
        assert self.refs.cpu().tolist() == m.refs

    def attend(self, ns, *, layer=0, rows=None, groups=None, q_scale=1.5, scale=None, ld_extra=0, q=None):
        """Plan and run attention of ns[b] queries per request; returns (out, q), the padded buffers."""
        T = sum(ns)
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(int).tolist()
        ld = self.Hq * self.D + ld_extra
        q = self.randn(max(1, T), ld, scale=q_scale) if q is None else q
        out = self.torch.full((max(1, T), ld), 7.0, dtype=self.dt, device="cuda")
        kw = {}
        if groups is not None:
            starts, toks = groups
            self._g = (self.ints(starts), self.ints(toks))
            kw = dict(n_groups=len(toks), group_start=self._g[0], group_tokens=self._g[1])
        self._a = (self.ints(cu), None if rows is None else self.ints(rows))
        self.kv.attn_plan(len(ns), T, self._a[0], rows=self._a[1], **kw)
        self.kv.attn_forward(layer, q, ld, out, ld, scale or self.D ** -0.5)
        return out, q

    def check_attend(self, ns, *, layer=0, rows=None, scale=None, **kw):
        out, q = self.attend(ns, layer=layer, rows=rows, scale=scale, **kw)
        assert self.kv.status() == self.ft.FT_OK
        pool, got, qh = self.host_pool(), out.double().cpu().numpy(), q.double().cpu().numpy()
        G, D, t0 = self.Hq // self.Hkv, self.D, 0
        worst = 0.0
        for b, n in enumerate(ns):
            row = b if rows is None else rows[b]
            for h in range(self.Hkv):
                if n == 0:
                    continue
                k, v = self.keys_values(pool, row, layer, h)
                for hq in range(h * G, (h + 1) * G):
                    ref, mass = okv.attention(qh[t0:t0 + n, hq * D:(hq + 1) * D], k, v, n, scale or D ** -0.5)
                    tol = attn_tolerance(self.kind, ref, mass, len(k), np.abs(v).max() if len(v) else 0.0)
                    err = np.abs(got[t0:t0 + n, hq * D:(hq + 1) * D] - ref)
                    assert np.all(err <= tol), (b, hq, float((err / tol).max()))  # a NaN fails too
                    worst = max(worst, float((err / tol).max()))
            t0 += n
        assert np.all(got[:sum(ns), self.Hq * D:] == 7.0), "columns past the heads were written"
        return worst
