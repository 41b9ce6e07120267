"""Sizes and arguments that the norms and the beam selection refuse before they touch a device."""
import moe_expert_cache_gb300 as ft

P = 1 << 20  # an address; none of these calls gets as far as using it


def _norm(T=4, H=64, block=P, ld_b=64, gp=None, ld_g=0, resid=2 * P, ld_r=64, resid_out=3 * P, ld_ro=64, out=4 * P, ld_o=64, **d):
    f = dict(block_type=0, resid_type=2, out_type=0, w_type=0, gate_type=0, gate=0, post_norm=0, post=None, pre=None, eps=1e-6,
             resid_scale=1.0, block_scale=1.0)
    f.update(d)
    desc = ft.NormDesc(H, *[f[n] for n, _ in ft.NormDesc._fields_[1:]])
    return ft.block_norm(desc, T, block, ld_b, gp, ld_g, resid, ld_r, resid_out, ld_ro, out, ld_o)


def test_norm_arguments():
    nan, inf = float("nan"), float("inf")
    bad = [dict(T=-1), dict(H=0), dict(H=4), dict(H=68), dict(H=16392, ld_b=16392, ld_r=16392, ld_ro=16392, ld_o=16392), dict(eps=-1e-6),
           dict(eps=nan), dict(eps=inf), dict(resid_scale=inf), dict(block_scale=nan), dict(block_type=3), dict(resid_type=-1),
           dict(out_type=1), dict(w_type=1, pre=6 * P), dict(gate_type=1, gate=2, gp=5 * P), dict(gate=4), dict(gate=-1), dict(post_norm=2), dict(gate=1),
           dict(block=None, post_norm=1), dict(block=None, gate=1, gate_type=0), dict(resid=None),
           dict(resid_out=None, out=None), dict(ld_b=56), dict(ld_r=68), dict(ld_ro=0), dict(ld_o=-64), dict(block=P + 8), dict(out=P + 2),
           dict(pre=P + 8), dict(post=P + 2, post_norm=1),
           dict(gate=1, gp=5 * P + 8), dict(gate=3, gp=5 * P), dict(gate=2, gp=5 * P + 1), dict(gate=3, gp=5 * P, ld_g=60),
           dict(gate=2, gate_type=2, gp=5 * P + 2), dict(ld_b=1 << 62), dict(ld_o=1 << 58, T=5), dict(ld_r=(1 << 60) + 8, T=1)]
    for b in bad:
        assert _norm(**b) == ft.FT_ERR_ARG, b
    assert _norm(T=0) == ft.FT_OK
    desc = ft.NormDesc()
    assert ft.load().ft_block_norm(None, 1, P, 64, None, 0, P, 64, P, 64, P, 64, None) == ft.FT_ERR_ARG
    assert ft.block_norm(desc, 1, P, 64, None, 0, P, 64, P, 64, P, 64) == ft.FT_ERR_ARG


def test_norm_overlaps():
    row = 64 * 2
    for b in (dict(out=P + 16), dict(out=P - 16), dict(out=P, out_type=2), dict(out=P, ld_o=72), dict(out=P + 3 * row), dict(resid_out=2 * P + 32),
              dict(resid_out=2 * P, ld_ro=128), dict(out=3 * P), dict(out=3 * P + 1008), dict(resid_out=2 * P, out=2 * P, out_type=2),
              dict(pre=4 * P), dict(pre=3 * P + 512), dict(out=P + row, ld_b=128, ld_o=136),
              dict(ld_b=128, ld_o=128, out=P + 112), dict(resid_out=2 * P, out=2 * P + 16)):
        assert _norm(**b) == ft.FT_ERR_ARG, b
    for b in (dict(gate=3, gp=4 * P, ld_g=64), dict(gate=3, gp=3 * P, ld_g=128), dict(gate=1, gp=4 * P + 256), dict(gate=2, gp=4 * P + 2),
              dict(gate=2, gp=4 * P - 6)):
        assert _norm(**b) == ft.FT_ERR_ARG, b


def test_beam_sizes():
    for V, dt, R, N in ((0, 0, 1, 1), ((1 << 24) + 1, 0, 1, 1), (10, 3, 1, 1), (10, -1, 1, 1), (10, 0, 0, 1), (10, 0, 65537, 1),
                        (10, 0, 1, 0), (10, 0, 1, 65)):
        assert ft.beam_init(V, dt, R, N, None) == (ft.FT_ERR_ARG, None), (V, dt, R, N)
        assert ft.beam_scratch_bytes(V, dt, R, N) == 0
    assert ft.beam_select(None, 1, 1, 1, P, 10, P, None, None, -1, P, P, P, None) == ft.FT_ERR_ARG
    assert ft.beam_status(None) == ft.FT_ERR_ARG
    ft.beam_destroy(None)
    assert ft.kv_reorder(None, 1, None, P) == ft.FT_ERR_ARG
    assert ft.kv_batch(None, 1, None, P, 1, P, P, P, None) == ft.FT_ERR_ARG
