"""More of the key/value cache on the GPU: buffers that overlap."""
import pytest

from tests.kv_harness import Cache

pytestmark = pytest.mark.gpu


def test_rope_output_that_overlaps_its_input():
    import torch
    T, Hq, Hkv, D = 5, 4, 2, 64
    w, wq = (Hq + 2 * Hkv) * D, Hq * D
    c = Cache([T], D=D, page=16, Hq=Hq, Hkv=Hkv, T_max=T)
    ft = c.ft
    ld = w + wq + 8
    buf = c.randn(3 * T, ld, scale=2.0)
    cs = torch.randn(T, D, generator=c.gen, device="cuda")
    row_of, pos = c.ints([0] * T), c.ints(range(T))
    base = buf.data_ptr() + T * ld * 2  # rows T..2T-1 are the input

    def call(q_out, ld_q, T=T):
        return ft.qk_rope_store(c.kv.h, 0, T, base, ld, row_of.data_ptr(), pos.data_ptr(), q_out, ld_q, None, None, 1e-6,
                                cs.data_ptr(), T, D, 0)

    # into the input's heads from a shifted start, across the end of its rows, with another stride, by a row up or down
    for off, ld_q in ((16, ld), (-16, ld), (2 * wq, ld), (2 * (w - 8), ld), (2 * (ld - wq + 8), ld), (2 * ld, ld), (-2 * ld, ld),
                      (0, ld + 8), (2 * w, ld - 8), (2 * w, ld + 8), (2 * ((T - 1) * ld + w - 8), wq),
                      (-2 * ((T - 1) * wq + 8), wq)):
        assert call(base + off, ld_q) == ft.FT_ERR_ARG, (off, ld_q)
    # the same rows elsewhere give what they give in columns beside the input, in a row of another stride, in place
    want = torch.empty(T, wq, dtype=c.dt, device="cuda")
    keep = buf.clone()
    assert call(want.data_ptr(), wq) == ft.FT_OK
    for off, ld_q in ((2 * w, ld), (2 * (w + 8), ld), (2 * T * ld, ld), (-2 * T * ld, ld), (2 * ((T - 1) * ld + w), wq),
                      (-2 * T * wq, wq), (2 * (w - 3 * ld), ld), (0, ld)):
        buf.copy_(keep)
        assert call(base + off, ld_q) == ft.FT_OK, (off, ld_q)
        at = T * ld + off // 2
        got = torch.as_strided(buf, (T, wq), (ld_q, 1), at)
        assert torch.equal(got, want), (off, ld_q)
    # one token: only its own values count
    buf.copy_(keep)
    assert call(base + 2 * (w - 8), ld, T=1) == ft.FT_ERR_ARG
    assert call(base + 2 * w, wq, T=1) == ft.FT_OK
    assert torch.equal(torch.as_strided(buf, (1, wq), (wq, 1), T * ld + w), want[:1])
    assert c.kv.status() == ft.FT_OK
