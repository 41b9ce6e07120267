"""A small MoE model that answers with the paged key/value cache: one prompt is
read, the sequence is forked into several, they decode together behind their
shared prefix, some end, and the pool is compacted so that its memory can go to
the expert cache.

    python examples/decode_with_cache.py

Every layer of a step is: norm, projection, ft_qk_rope_store, ft_attn_forward,
output projection, norm, router, ft_route_ctl, ft_moe_forward.  Weights are
random; the projections, the residual sums and the choice of the next token
are plain torch.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_cache_gb300 as ft  # noqa: E402
import synth  # noqa: E402

BF16 = torch.bfloat16


def rms(x, eps=1e-6):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


class Model:
    """L layers of attention and experts over one pool of pages and one expert cache."""

    def __init__(self, L=2, H=256, Hq=8, Hkv=2, D=64, E=8, k=2, F=128, vocab=97, page=16, n_pages=64, rows=8, row_pages=24,
                 T_max=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.L, self.H, self.Hq, self.Hkv, self.D, self.E, self.k, self.F = L, H, Hq, Hkv, D, E, k, F
        self.page, self.T_max, self.max_pos = page, T_max, row_pages * page

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).to(BF16)

        self.embed = torch.randn(vocab, H, generator=g, device="cuda")
        self.head = torch.randn(H, vocab, generator=g, device="cuda")
        self.qkv = [w(H, (Hq + 2 * Hkv) * D) for _ in range(L)]
        self.q_norm = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF16) for _ in range(L)]
        self.k_norm = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF16) for _ in range(L)]
        self.out = [w(Hq * D, H) for _ in range(L)]
        self.router = [torch.randn(H, E, generator=g, device="cuda") * H ** -0.5 for _ in range(L)]
        angles = torch.arange(self.max_pos, device="cuda")[:, None] * 1e4 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos_sin = torch.cat([angles.cos(), angles.sin()], 1).float().contiguous()

        # the experts: one record each in page-locked host memory, all of them resident once used
        self.experts = [[synth.expert_weights_bf16(seed, l, e, H, F) for e in range(E)] for l in range(L)]
        nb = ft.record_bytes(H, F)
        host = torch.empty(L * E * nb, dtype=torch.uint8, pin_memory=True)
        for l in range(L):
            for e in range(E):
                at = (l * E + e) * nb
                host[at:at + nb] = torch.from_numpy(synth.pack_record_bf16(*self.experts[l][e]).view(np.uint8))
        self.moe = ft.Context(L, E, k, H, F, L * E, host, T_max=T_max)
        # the cache: the pool and its control arrays are the program's own
        self.pool = torch.zeros(n_pages * ft.kv_page_bytes(L, Hkv, D, page), dtype=torch.uint8, device="cuda")
        self.table = torch.full((rows, row_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.kv = ft.KvCache(L, Hq, Hkv, D, page, n_pages, rows, row_pages, self.pool, self.table, self.lens, self.refs,
                             T_max=T_max, B_max=rows)

    def ints(self, v):
        return torch.tensor(list(v), dtype=torch.int32, device="cuda")

    def step(self, rows, tokens, starts, shared=0):
        """tokens[i] (a list) go on row rows[i] from position starts[i] on; the rows' first `shared` tokens are on
        the same pages.  Returns the hidden states of all tokens, in order."""
        n = [len(t) for t in tokens]
        T, w = sum(n), self.Hq * self.D
        ids = torch.tensor([t for ts in tokens for t in ts], device="cuda")
        row_ids = self.ints(rows)
        row_of = self.ints(r for r, c in zip(rows, n) for _ in range(c))
        pos = self.ints(s + i for s, c in zip(starts, n) for i in range(c))
        cu = self.ints(np.concatenate([[0], np.cumsum(n)]).tolist())
        self.kv.extend(len(rows), row_ids, self.ints(n))
        group = {}
        if shared and len(rows) > 1:  # (without a claim requests of few tokens run the faster form)
            group = dict(n_groups=1, group_start=self.ints([0, len(rows)]), group_tokens=self.ints([shared]))
        self.kv.attn_plan(len(rows), T, cu, rows=row_ids, **group)
        h = self.embed[ids].clone()
        q = torch.empty(T, w, dtype=BF16, device="cuda")
        o = torch.empty_like(q)
        y = torch.empty(T, self.H, device="cuda")
        for l in range(self.L):
            qkv = rms(h).to(BF16) @ self.qkv[l]
            self.kv.qk_rope_store(l, T, qkv, qkv.shape[1], row_of, pos, q, w, q_norm=self.q_norm[l], k_norm=self.k_norm[l],
                                  cos_sin=self.cos_sin, max_pos=self.max_pos, rot=self.D)
            self.kv.attn_forward(l, q, w, o, w, self.D ** -0.5)
            h += (o @ self.out[l]).float()
            x = rms(h).to(BF16)
            logits = x.float() @ self.router[l]
            # B_P = B_H: every expert that is missing is fetched, none is left to the host
            self.moe.route_ctl(l, T, logits=logits, B_P=1.0, B_H=1.0)
            self.moe.moe_forward(x, None, y)
            h += y
        return h

    def next_tokens(self, h):
        return (rms(h) @ self.head).argmax(-1).tolist()


def run(prompt_len=150, forks=4, new=12, seed=0, verbose=True, **sizes):
    """Returns (model, the tokens of each surviving row, what compaction did)."""
    m = Model(seed=seed, **sizes)
    rng = np.random.default_rng(seed)
    prompt = [int(t) for t in rng.integers(0, m.embed.shape[0], prompt_len)]
    for at in range(0, prompt_len, m.T_max):  # the prompt in chunks
        h = m.step([0], [prompt[at:at + m.T_max]], [at])
    first = torch.topk(rms(h[-1:]) @ m.head, forks).indices[0].tolist()
    rows = list(range(1, forks + 1))
    m.kv.fork(forks, m.ints([0] * forks), m.ints(rows))  # complete pages are shared, the last one is copied
    shared = prompt_len // m.page * m.page
    answers = [[t] for t in first]
    for i in range(new):
        h = m.step(rows, [[a[-1]] for a in answers], [prompt_len + i] * forks, shared)
        for a, t in zip(answers, m.next_tokens(h)):
            a.append(t)
    # the prompt's own row and every second answer end; the others' pages move together
    gone = [0] + rows[1::2]
    m.kv.free(len(gone), m.ints(gone))
    m.kv.compact()
    info = m.kv.last()
    rows, answers = rows[::2], answers[::2]
    h = m.step(rows, [[a[-1]] for a in answers], [prompt_len + new] * len(rows), shared)
    assert m.kv.status() == ft.FT_OK and m.moe.status() == ft.FT_OK
    if verbose:
        print("answers:", answers)
        print(f"pages in use after compaction: 0..{info['live'] - 1} of {len(m.refs)} ({info['copied']} moved)")
    return m, prompt, answers, h, info


if __name__ == "__main__":
    run()
