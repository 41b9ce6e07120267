"""The example's model against the same model computed densely in fp32 from all
tokens of each sequence, without a cache, a page or a fork."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _dense(m, tokens):
    """Hidden states of a sequence, every layer over the whole of it; operands rounded where the model rounds."""
    import torch
    T = len(tokens)

    def b(x):
        return x.to(torch.bfloat16).float()

    def rms(x, eps=1e-6):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)

    def turn(x, w):
        x = rms(x) * w.float()
        c, s = m.cos_sin[:T, None, :m.D // 2], m.cos_sin[:T, None, m.D // 2:]
        a, z = x[..., :m.D // 2], x[..., m.D // 2:]
        return b(torch.cat([a * c - z * s, z * c + a * s], -1))

    h = m.embed[torch.tensor(tokens, device="cuda")].clone()
    for l in range(m.L):
        x = b(b(rms(h)) @ m.qkv[l].float()).view(T, m.Hq + 2 * m.Hkv, m.D)
        q, k, v = turn(x[:, :m.Hq], m.q_norm[l]), turn(x[:, m.Hq:m.Hq + m.Hkv], m.k_norm[l]), x[:, m.Hq + m.Hkv:]
        k, v = (t.repeat_interleave(m.Hq // m.Hkv, 1) for t in (k, v))
        s = torch.einsum("thd,uhd->htu", q, k) * m.D ** -0.5
        s = s.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), float("-inf"))
        o = b(torch.einsum("htu,uhd->thd", s.softmax(-1), v).reshape(T, -1))
        h = h + b(o @ m.out[l].float())
        x = b(rms(h))
        gates = (x @ m.router[l]).softmax(-1)  # all experts are chosen
        for e in range(m.E):
            wg, wu, wd = (torch.from_numpy((w.astype(np.uint32) << 16).view(np.float32)).cuda() for w in m.experts[l][e])
            h = h + gates[:, e:e + 1] * ((torch.nn.functional.silu(x @ wg.T) * (x @ wu.T)) @ wd.T)
    return h


def test_example_matches_the_dense_model():
    sys.path.insert(0, ROOT)
    from examples.decode_with_cache import run
    # all experts are chosen, so no rounding can change which; the answers are the library's own
    m, prompt, answers, h, info = run(prompt_len=150, forks=4, new=10, E=4, k=4, verbose=False)
    for a, got in zip(answers, h):
        want = _dense(m, prompt + a)[-1]
        # bf16 roundings (2^-8 each) at a dozen places of two layers, summed as if all were independent and
        # of the size of the hidden state: sqrt(24) * 2^-8 = 0.019
        assert float((got - want).norm() / want.norm()) <= 0.019
    # rows 1 and 3 are left: 9 shared pages and one own each for positions 144..160
    live = 9 + 2 * (-(-(150 + 10) // 16) - 9)
    assert info["live"] == live
    assert int((m.refs > 0).sum()) == 9 + 2 * (-(-161 // 16) - 9) and int(m.refs.max()) == 2
