"""Beam search over the small MoE model of decode_with_cache.py, all of it on the
device: the host only keeps what each step chose, to read the texts back.

    python examples/beam_search.py

A step is: ft_beam_select (the best continuations of each request's beams),
ft_kv_reorder (the cache's rows follow), ft_kv_batch (rows of beams that have not
ended grow by a token), then the layers.  Row b*K + k of the cache is beam k of
request b.
"""
from __future__ import annotations

import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_cache_gb300 as ft  # noqa: E402
from examples.decode_with_cache import Model  # noqa: E402


def run(prompt_lens=(37, 50), K=4, new=10, eos=5, seed=0, verbose=True, **sizes):
    """Returns (model, prompts, the texts and scores of each request's beams, best first, a trace of all steps)."""
    B, n = len(prompt_lens), len(prompt_lens) * K
    m = Model(seed=seed, rows=n, n_pages=n * 8, **sizes)
    V = m.embed.shape[0]
    rng = np.random.default_rng(seed)
    prompts = [[int(t) for t in rng.integers(0, V, p)] for p in prompt_lens]

    def zeros(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    beams = ft.Beams(V, n, K)
    logits = zeros(n + 1, V, dtype=torch.float32)  # a row for each beam, and one for padding
    # before the first step each request has one beam, its prompt
    scores = torch.full((n,), -math.inf, device="cuda")
    scores[::K] = 0
    done, parents, tokens = zeros(n), zeros(n), zeros(n)
    for b, prompt in enumerate(prompts):
        for at in range(0, len(prompt), m.T_max):
            _, last = m.step([b * K], [prompt[at:at + m.T_max]])
        logits[b * K] = last[-1] @ m.head
    trace = []
    for i in range(new):
        before = (logits[:n].clone(), scores.clone(), done.clone())
        beams.select(B, K, K, logits, V, scores, scores, parents, tokens, done=done, eos=eos, out_done=done)
        m.kv.reorder(n, parents)
        trace.append(before + (scores.clone(), parents.clone(), tokens.clone(), done.clone()))
        # beams that have ended add nothing: the step is padded to n tokens
        m.lay_out(n, 1 - done, n)
        there = m.row_of >= 0
        row = torch.where(there, m.row_of, n).long()
        h, last = m.forward(torch.where(there, tokens[row.clamp(max=n - 1)], 0).long(), n, n)
        logits[row] = last @ m.head
    assert beams.status() == ft.FT_OK and m.kv.status() == ft.FT_OK and m.moe.status() == ft.FT_OK
    # the texts, read back through the parents
    texts = []
    for b in range(B):
        for k in range(K):
            text, at = [], b * K + k
            for *_, parent, token, end in reversed(trace):
                t, p = int(token[at]), int(parent[at])
                text.append(t)
                at = p
            text.reverse()
            if eos in text:  # (an ended beam repeats it)
                text = text[:text.index(eos) + 1]
            texts.append(text)
    if verbose:
        for b in range(B):
            for k in range(K):
                print(f"request {b}: {float(scores[b * K + k]):8.3f}  {texts[b * K + k]}")
    return m, prompts, texts, scores, trace, (h, m.row_of)


if __name__ == "__main__":
    run()
