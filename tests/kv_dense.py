"""Attention of a whole batch in fp64 on the GPU, for batches that are too large for the oracle's loops."""
from __future__ import annotations

import torch

from tests.kv_harness import U


def check_dense(c, ns, out, q, *, lens=None, rows=None, layer=0, scale=None, budget=1 << 27):
    """Compare out with softmax(scale q K^T) V over each row's pages, within the bound of kv_harness.attn_tolerance.
    Requests are taken together, padded to the longest; `budget` bounds the fp64 values of a step."""
    D, G, scale = c.D, c.Hq // c.Hkv, scale or c.D ** -0.5
    lens = c.model.lens if lens is None else lens
    rows = list(range(len(ns))) if rows is None else rows
    t0, starts = 0, []
    for n in ns:
        starts.append(t0)
        t0 += n
    u, worst = U[c.kind], 0.0
    todo = sorted((b for b in range(len(ns)) if ns[b]), key=lambda b: (ns[b], lens[rows[b]]))
    at = 0
    while at < len(todo):
        n = ns[todo[at]]
        m = 1
        while at + m < len(todo) and ns[todo[at + m]] == n:
            longest = max(1, lens[rows[todo[at + m]]])
            if (m + 1) * longest * max(2 * D, G * n) > budget:
                break
            m += 1
        part = todo[at:at + m]
        at += m
        ln = torch.tensor([lens[rows[b]] for b in part], device="cuda")
        N = max(1, int(ln.max()))
        pos = torch.arange(N, device="cuda")
        pages = c.table[torch.tensor([rows[b] for b in part], device="cuda")].long()[:, :-(-N // c.page)].clamp(min=0)
        st = torch.tensor([starts[b] for b in part], device="cuda")
        step = max(1, min(n, budget // (m * N * G)))
        for h in range(c.Hkv):
            kv = c.pool[pages, layer, :, h]                                     # [m, pages, 2, page, D]
            kv = kv.permute(2, 0, 1, 3, 4).reshape(2, m, -1, D)[:, :, :N]
            kv = kv.masked_fill((pos[None, :] >= ln[:, None])[None, :, :, None], 0).double()
            vmax = kv[1].abs().amax()
            for i in range(0, n, step):
                e = torch.arange(i, min(n, i + step), device="cuda")
                tok = (st[:, None] + e[None, :])                                # [m, tokens]
                x = q[tok, :c.Hq * D].view(m, len(e), c.Hq, D)[:, :, h * G:(h + 1) * G].double()
                s = torch.einsum("mtgd,mkd->mtgk", x, kv[0]) * scale
                seen = pos[None, None, :] <= (ln[:, None] - n + e[None, :])[:, :, None]
                s = s.masked_fill(~seen[:, :, None, :], -torch.inf)
                w = torch.nan_to_num(s.softmax(-1))                            # a query that sees no key: zeros
                ref, mass = w @ kv[1][:, None], w @ kv[1].abs()[:, None]
                got = out[tok, :c.Hq * D].view(m, len(e), c.Hq, D)[:, :, h * G:(h + 1) * G].double()
                sub = N * 2.0 ** -25 * vmax if c.kind == "f16" else 0.0
                tol = u * ref.abs() + (u + 2.0 ** -13) * mass + sub + 1e-6
                err = (got - ref).abs()
                assert bool((err <= tol).all()), (h, float((err / tol).max()))  # a NaN fails too
                worst = max(worst, float((err / tol).max()))
    return worst
