"""Selection, reordering, batch layout and norms together, as the example runs them: every choice against the oracle on
the logits that the step had, and the hidden state of every beam against the dense model over that beam's text."""
import os
import sys

import pytest

from oracle import gen
from tests.test_example_gpu import _dense

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("ends", [False, True])
def test_beam_search_matches_the_dense_model(ends):
    sys.path.insert(0, ROOT)
    from examples.beam_search import run
    K, new, eos = 4, 8, 96
    if ends:  # a token of the best text, so that beams end at it
        eos = run(prompt_lens=(37, 50), K=K, new=new, eos=eos, E=4, k=4, verbose=False)[2][0][4]
    m, prompts, texts, scores, trace, (h, row_of) = run(prompt_lens=(37, 50), K=K, new=new, eos=eos, E=4, k=4, verbose=False)
    for logits, before, done, after, parents, tokens, ended in trace:
        x, s, d = logits.double().cpu().numpy(), before.cpu().numpy(), done.tolist()
        for b in range(2):
            e = slice(b * K, (b + 1) * K)
            want = gen.beam_select(x[e], s[e], K, done=d[e], eos=eos, first_row=b * K)
            assert [w[1:] for w in want] == list(zip(parents[e].tolist(), tokens[e].tolist(), ended[e].tolist()))
            for got, w in zip(after[e].tolist(), want):
                assert abs(got - w[0]) <= 2.0 ** -24 * (132 + abs(w[0]))  # as in test_beam_gpu
    rows = row_of.tolist()
    last = trace[-1]
    live = 0
    for i, text in enumerate(texts):
        full = prompts[i // K] + text
        # the cache holds the prompt and every token that a beam went on from (not the eos that ends it)
        assert int(m.lens[i]) == len(full) - (text[-1] == eos)
        if int(last[6][i]):
            assert text[-1] == eos and i not in rows
            continue
        live += 1
        want = _dense(m, full)[-1]
        got = h[rows.index(i)]
        # as in test_example_gpu
        assert float((got - want).norm() / want.norm()) <= 0.019
    assert rows.count(-1) == len(rows) - live
    assert not ends or live < len(rows)
    # each row's pages are its own but for those that it shares complete
    refs = [0] * len(m.refs)
    for r in m.table.tolist():
        for p in r:
            if p >= 0:
                refs[p] += 1
    assert refs == m.refs.tolist()
