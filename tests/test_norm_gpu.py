"""ft_block_norm against the formula in 64 bits, element by element."""
import itertools

import numpy as np
import pytest

from oracle import gen

pytestmark = pytest.mark.gpu

UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}
U = 2.0 ** -24


def _types():
    import torch

    import moe_expert_cache_gb300 as ft
    return ({"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32},
            {"bf16": ft.FT_T_BF16, "f16": ft.FT_T_F16, "f32": ft.FT_T_F32})


def _rows(g, T, H, dt, scale, extra):
    """A buffer whose rows are longer than H; what lies beyond is NaN."""
    import torch
    buf = torch.full((max(1, T), H + extra), float("nan"), dtype=dt, device="cuda")
    buf[:, :H] = (torch.randn(max(1, T), H, generator=g, device="cuda") * scale).to(dt)
    return buf


def _bounds(block, resid, gate, post_norm, post, pre, eps, rs, bs, n_out, n_res):
    """(h, its bound, out, its bound) of one token.

    Roundings of 2^-24 each: a sum of H squares takes at most 32 additions in a thread, 5 among the lanes and 16 among
    the warps, and a rounding of each square, so 54; half of it in the root, with 6 for the quotient, eps and rsqrtf
    (2 ulp): r is off by 33, a product with weight, gate and scale by 4 more: 37 of |bs g z|; 1 of |rs r|; the sum 1 of
    |h|.  out: the same 33 and 3 products, 36 of |out|, and what h is off by, in the element and through the root (off by
    at most the root mean square of h's own errors over that of h)."""
    h, y = gen.block_norm(block, resid, gate=gate, post_norm=post_norm, post=post, pre=pre, eps=eps, resid_scale=rs,
                          block_scale=bs)
    z = 0 if block is None else h - rs * np.asarray(resid, dtype=np.float64)
    dh = U * (37 * np.abs(z) + np.abs(rs * resid) + np.abs(h)) + 2.0 ** -140
    root = np.sqrt(np.mean(h * h) + eps)
    w = 1.0 if pre is None else np.abs(pre)
    dy = (dh + np.abs(h) * np.sqrt(np.mean(dh * dh)) / root) / root * w + 36 * U * np.abs(y)
    return h, dh + UNIT[n_res] * (np.abs(h) + dh) + TINY[n_res], y, dy + UNIT[n_out] * (np.abs(y) + dy) + TINY[n_out]


def _run(T, H, block="bf16", resid="f32", out="bf16", gate="none", gate_type=None, w=None, post_norm=False, weights=True,
         eps=1e-6, rs=1.0, bs=1.0, extra=0, stored=("h", "y"), in_place=(), stream=None, seed=0, edit=None):
    import torch

    import moe_expert_cache_gb300 as ft
    dts, ids = _types()
    g = torch.Generator(device="cuda").manual_seed(seed)
    small = next((t for t in (block, resid, out) if t not in (None, "f32")), "bf16")
    w = w or small
    gate_type = gate_type or (block or small)
    b = None if block is None else _rows(g, T, H, dts[block], 1.5, extra)
    r = _rows(g, T, H, dts[resid], 4.0, 2 * extra)
    if edit:
        edit(b, r)
    gt = {"none": lambda: None, "channel": lambda: torch.randn(H, generator=g, device="cuda").to(dts[gate_type]),
          "token": lambda: torch.randn(max(1, T), generator=g, device="cuda").to(dts[gate_type]),
          "full": lambda: _rows(g, T, H, dts[gate_type], 1.0, extra)}[gate]()
    pre, post = ((1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dts[w]) if weights else None for _ in range(2))
    b0, r0 = None if b is None else b.clone(), r.clone()
    h = (r if "h" in in_place else torch.full((max(1, T), H + extra), 7.0, dtype=dts[resid], device="cuda")) if "h" in stored else None
    y = (b if "y" in in_place else torch.full((max(1, T), H + 3 * extra), 7.0, dtype=dts[out], device="cuda")) if "y" in stored else None
    n = ft.BlockNorm(H, pre=pre, post=post if post_norm else None, post_norm=post_norm,
                     block_type=ids[block or "f32"], resid_type=ids[resid], out_type=ids[out], w_type=ids[w],
                     gate={"none": 0, "channel": 1, "token": 2, "full": 3}[gate], gate_type=ids[gate_type], eps=eps, resid_scale=rs,
                     block_scale=bs, stream=stream.cuda_stream if stream else 0)
    if stream:
        stream.wait_stream(torch.cuda.current_stream())
    n.forward(T, r, r.shape[1], block=b, ld_b=0 if b is None else b.shape[1], gate=gt, ld_g=gt.shape[-1] if gate == "full" else 0,
              resid_out=h, ld_ro=0 if h is None else h.shape[1], out=y, ld_o=0 if y is None else y.shape[1])
    torch.cuda.synchronize()
    f = lambda t: None if t is None else t.double().cpu().numpy()
    bh, rh, gh, preh, posth, hh, yh = f(b0), f(r0), f(gt), f(pre), f(post), f(h), f(y)
    worst = 0.0
    for t in range(T):
        gg = None if gate == "none" else gh if gate == "channel" else gh[t] if gate == "token" else gh[t, :H]
        want_h, dh, want_y, dy = _bounds(None if bh is None else bh[t, :H], rh[t, :H], gg, post_norm, posth if post_norm else None, preh,
                                         eps, rs, bs, out, resid)
        for got, want, tol in ((hh, want_h, dh), (yh, want_y, dy)):
            if got is None:
                continue
            err = np.abs(got[t, :H] - want)
            assert np.all(err <= tol), (t, float(np.nanmax(err / tol)))  # a NaN fails too
            worst = max(worst, float((err / tol).max()))
    for got, buf in ((h, r0 if "h" in in_place else None), (y, b0 if "y" in in_place else None)):
        if got is None:
            continue
        rest = got[:, H:] if T else got
        assert bool((rest.isnan() if buf is not None else rest == 7.0).all()), "columns past H were written"
    return worst


@pytest.mark.parametrize("H", [8, 64, 200, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2880, 4096, 4104, 7176, 8192, 8200, 16384])
def test_channels(H):
    _run(5, H, post_norm=True, gate="channel", extra=8, rs=0.5, bs=-0.75, seed=H)


@pytest.mark.parametrize("small", ["bf16", "f16"])
def test_types(small):
    for i, (b, r, o) in enumerate(itertools.product((small, "f32", None), (small, "f32"), (small, "f32"))):
        for H in (256, 1536, 6000, 9008):  # a warp's row, and one, two and four vectors a thread
            _run(3, H, block=b, resid=r, out=o, w=small if i % 2 else "f32", post_norm=b is not None and i % 3 == 0,
                 gate="none" if b is None else ("none", "channel", "token", "full")[i % 4],
                 gate_type=None if b is None else ("f32" if i % 2 else small), seed=i, extra=16)


@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 5, 127, 611])
def test_tokens(T):
    _run(T, 320, gate="token", gate_type="f32", post_norm=True, extra=8)
    _run(T, 1288, gate="full", block="f32", resid="f32", extra=8)


def test_parts_that_are_absent():
    for H in (512, 2048):
        _run(3, H, block=None)
        _run(3, H, block=None, stored=("y",))
        _run(3, H, stored=("h",))
        _run(3, H, stored=("y",), gate="channel")
        _run(3, H, weights=False, post_norm=True)
        _run(3, H, eps=0.0, bs=0.0, rs=-1.0)


def test_in_place():
    for H in (512, 4096):
        _run(9, H, in_place=("h",), post_norm=True, extra=8)
        _run(9, H, in_place=("h", "y"), post_norm=True, gate="full", extra=8)
        _run(9, H, in_place=("h", "y"), block="f32", out="f32", extra=8)


def test_rows_of_zeros_and_extremes():
    def zeros(b, r):
        b[1], r[1] = 0, 0
        r[2] = -b[2].float()  # the sum is zero, the parts are not
        b[3] = 0
    for H in (512, 2048):
        _run(4, H, edit=zeros, post_norm=False)
        _run(4, H, edit=zeros, post_norm=True)

    def large(b, r):
        r[0, :8] = 1e15  # squares of 1e30
        b[1] *= 1e-20    # squares under fp32's smallest: eps is what is left
        r[1] = 0
    _run(2, 2048, block="f32", edit=large)
    _run(2, 2048, block="f32", edit=large, post_norm=True)


def test_nan_stays_in_its_row():
    import torch

    def bad(b, r):
        b[1, 5] = float("nan")
        r[3, 7] = float("inf")
    import moe_expert_cache_gb300 as ft
    for H in (512, 2048):
        g = torch.Generator(device="cuda").manual_seed(0)
        b, r = _rows(g, 5, H, torch.bfloat16, 1.0, 0), _rows(g, 5, H, torch.float32, 1.0, 0)
        bad(b, r)
        h, y = torch.empty_like(r), torch.empty_like(b)
        ft.BlockNorm(H).forward(5, r, H, block=b, ld_b=H, resid_out=h, ld_ro=H, out=y, ld_o=H)
        assert bool(y[[0, 2, 4]].isfinite().all()) and bool(h[[0, 2, 4]].isfinite().all())
        assert bool(y[1].isnan().all()) and int(h[1].isnan().sum()) == 1
        assert bool(y[3, 7].isnan()) and bool((y[3, :7] == 0).all())  # 1 / inf


def test_other_stream_and_graph():
    import torch

    import moe_expert_cache_gb300 as ft
    s = torch.cuda.Stream()
    _run(33, 2048, stream=s, post_norm=True)
    H, T = 1024, 7
    g = torch.Generator(device="cuda").manual_seed(0)
    b, r = _rows(g, T, H, torch.bfloat16, 1.0, 0), _rows(g, T, H, torch.float32, 1.0, 0)
    y = torch.empty_like(b)
    r0 = r.clone()
    n = ft.BlockNorm(H, stream=s.cuda_stream)
    call = lambda: n.forward(T, r, H, block=b, ld_b=H, resid_out=r, ld_ro=H, out=y, ld_o=H)
    torch.cuda.synchronize()
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    want_r, want_y = r.clone(), y.clone()
    r.copy_(r0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            call()
    r.copy_(r0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, want_r) and torch.equal(y, want_y)


def test_a_large_batch():
    # more rows than CTAs run at once, offsets of rows past 32 bits
    import torch

    import moe_expert_cache_gb300 as ft
    T, H = 70001, 512
    ld = 65536
    big = torch.empty((T - 1) * ld + H, dtype=torch.bfloat16, device="cuda")  # 9 GB, 4.6e9 elements
    b = torch.as_strided(big, (T, H), (ld, 1))
    g = torch.Generator(device="cuda").manual_seed(0)
    b.copy_(torch.randn(T, H, generator=g, device="cuda"))
    r = torch.randn(T, H, generator=g, device="cuda")
    h, y = torch.empty_like(r), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ft.BlockNorm(H).forward(T, r, H, block=big, ld_b=ld, resid_out=h, ld_ro=H, out=y, ld_o=H)
    want = r.double() + b.double()
    assert bool(((h - want).abs() <= 3 * U * (r.abs() + b.abs().float())).all())
    want = want / torch.sqrt((want * want).mean(-1, keepdim=True) + 1e-6)
    assert bool(((y - want).abs() <= (UNIT["bf16"] + 100 * U) * want.abs() + 100 * U).all())
