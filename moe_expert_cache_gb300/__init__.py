"""Python binding of libft (the C ABI in include/ft.h, ft_kv.h and ft_gen.h): argument marshalling only.

Every function here has the name of the C entry point without its ``ft_``
prefix and takes plain integers for pointers (device or host addresses, e.g.
``tensor.data_ptr()``) and streams (``torch.cuda.Stream.cuda_stream``).  Every
step of the hot path runs in the CUDA library; there is no Python or CPU
fallback: if libft.so is missing this module raises on first use.

``Context``, ``KvCache`` and ``Beams`` are small convenience owners of an
``ft_ctx*``, an ``ft_kv*`` and an ``ft_beam*``, ``BlockNorm`` holds an
``ft_norm_desc``; they raise ``FtError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libft.so")

FT_OK = 0
FT_ERR_ARG = -1
FT_ERR_CUDA = -2
FT_ERR_OOM = -3
FT_ERR_CAPACITY = -4
FT_ERR_TIMEOUT = -5
FT_ERR_STATE = -6
FT_ERR_DEVICE = -7
FT_FMT_BF16 = 0
FT_FMT_NVFP4 = 1
FT_FMT_MXFP4 = 2
FT_FMT_FP8 = 3
FT_KV_BF16 = 0
FT_KV_F16 = 1
FT_T_BF16 = 0
FT_T_F16 = 1
FT_T_F32 = 2
FT_GATE_NONE = 0
FT_GATE_CHANNEL = 1
FT_GATE_TOKEN = 2
FT_GATE_FULL = 3

_c_int = ctypes.c_int32
_c_i64 = ctypes.c_int64
_c_f = ctypes.c_float
_c_p = ctypes.c_void_p


class CtlInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("layer", "T", "u", "h", "m", "q0", "q1", "q", "nC", "u_gpu", "n_assign")] + \
               [("clock", ctypes.c_uint32)]


class KvInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("allocated", "copied", "live")]


class NormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("H", "block_type", "resid_type", "out_type", "w_type", "gate_type", "gate", "post_norm")] + \
               [(n, ctypes.c_void_p) for n in ("post", "pre")] + \
               [(n, ctypes.c_float) for n in ("eps", "resid_scale", "block_scale")]


class Counters(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("calls", "unique", "hits", "misses", "fills", "cpu", "assign")]


FT_K_COUNT = 16


class Profile(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * FT_K_COUNT), ("launches", ctypes.c_uint64 * FT_K_COUNT)]


# name -> (restype, argtypes)
_SIGS = {
    "ft_abi_version": (_c_int, []),
    "ft_status_str": (ctypes.c_char_p, [_c_int]),
    "ft_record_bytes": (ctypes.c_size_t, [_c_int, _c_int, _c_int]),
    "ft_layer_init": (_c_int, [ctypes.POINTER(_c_p), _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                               _c_int, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "ft_route_ctl": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_p, _c_p, ctypes.c_double, ctypes.c_double]),
    "ft_moe_forward": (_c_int, [_c_p, _c_p, _c_p, _c_p]),
    "ft_prefill_begin": (_c_int, [_c_p, _c_int]),
    "ft_prefill_layer": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_p]),
    "ft_cache_resize": (_c_int, [_c_p, _c_int]),
    "ft_measure_link": (_c_int, [_c_p, _c_int, _c_int, ctypes.POINTER(ctypes.c_double)]),
    "ft_get_ctl_state": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p]),
    "ft_set_ctl_state": (_c_int, [_c_p, _c_p, _c_p, _c_p, ctypes.c_uint32]),
    "ft_get_last_ctl": (_c_int, [_c_p, ctypes.POINTER(CtlInfo), _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "ft_read_slot": (_c_int, [_c_p, _c_int, _c_p]),
    "ft_get_counters": (_c_int, [_c_p, ctypes.POINTER(Counters)]),
    "ft_profile_enable": (_c_int, [_c_p, _c_int]),
    "ft_profile_read": (_c_int, [_c_p, ctypes.POINTER(Profile)]),
    "ft_profile_pause": (_c_int, [_c_p, _c_int]),
    "ft_kernel_name": (ctypes.c_char_p, [_c_int]),
    "ft_num_slots": (_c_int, [_c_p]),
    "ft_expert_ffn_noalloc": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int,
                                       _c_p]),
    "ft_noalloc_status": (_c_int, [_c_p]),
    "ft_set_wait_limit": (_c_int, [_c_p, ctypes.c_uint64]),
    "ft_get_status": (_c_int, [_c_p]),
    "ft_destroy": (None, [_c_p]),
    "ft_kv_page_bytes": (ctypes.c_size_t, [_c_int] * 4),
    "ft_kv_scratch_bytes": (ctypes.c_size_t, [_c_int] * 7),
    "ft_kv_init": (_c_int, [ctypes.POINTER(_c_p)] + [_c_int] * 11 + [_c_p] * 5),
    "ft_kv_extend": (_c_int, [_c_p, _c_int, _c_p, _c_p]),
    "ft_kv_fork": (_c_int, [_c_p, _c_int, _c_p, _c_p]),
    "ft_kv_free": (_c_int, [_c_p, _c_int, _c_p]),
    "ft_kv_compact": (_c_int, [_c_p]),
    "ft_qk_rope_store": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p, _c_f, _c_p,
                                  _c_int, _c_int, _c_int]),
    "ft_attn_plan": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_p, _c_int, _c_p, _c_p]),
    "ft_attn_forward": (_c_int, [_c_p, _c_int, _c_p, _c_i64, _c_p, _c_i64, _c_f]),
    "ft_kv_last": (_c_int, [_c_p, ctypes.POINTER(KvInfo)]),
    "ft_kv_status": (_c_int, [_c_p]),
    "ft_kv_destroy": (None, [_c_p]),
    "ft_kv_reorder": (_c_int, [_c_p, _c_int, _c_p, _c_p]),
    "ft_kv_batch": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "ft_block_norm": (_c_int, [_c_p, _c_int] + [_c_p, _c_i64] * 5 + [_c_p]),
    "ft_beam_scratch_bytes": (ctypes.c_size_t, [_c_int] * 4),
    "ft_beam_init": (_c_int, [ctypes.POINTER(_c_p)] + [_c_int] * 4 + [_c_p]),
    "ft_beam_select": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_int] + [_c_p] * 4),
    "ft_beam_status": (_c_int, [_c_p]),
    "ft_beam_destroy": (None, [_c_p]),
}

_lib = None


def load() -> ctypes.CDLL:
    """Load libft.so (built by __graft_entry__.build / build.py); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libft.so is not built ({LIB_PATH}); run moe_expert_cache_gb300/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


class FtError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)} ({status})")
        self.status = status


def _check(st: int, what: str) -> None:
    if st != FT_OK:
        raise FtError(st, what)


# ---------------------------------------------------------------- raw calls

def abi_version() -> int:
    return load().ft_abi_version()


def status_str(s: int) -> str:
    return load().ft_status_str(s).decode()


def record_bytes(H: int, F: int, fmt: int = FT_FMT_BF16) -> int:
    return load().ft_record_bytes(H, F, fmt)


def layer_init(L, E, k, H, F, S, fmt, T_max, T_prefill_max, host_pool, nvfp4_global, compute_stream,
               transfer_stream):
    h = _c_p()
    st = load().ft_layer_init(ctypes.byref(h), L, E, k, H, F, S, fmt, T_max, T_prefill_max, host_pool,
                              nvfp4_global, compute_stream, transfer_stream)
    return st, h.value


def route_ctl(ctx, layer, T, logits, topk_ids, topk_w, B_P, B_H) -> int:
    return load().ft_route_ctl(ctx, layer, T, logits, topk_ids, topk_w, B_P, B_H)


def moe_forward(ctx, x, partial_C, y) -> int:
    return load().ft_moe_forward(ctx, x, partial_C, y)


def prefill_begin(ctx, layer) -> int:
    return load().ft_prefill_begin(ctx, layer)


def prefill_layer(ctx, buffer, layer, next_layer, T, x, logits, y) -> int:
    return load().ft_prefill_layer(ctx, buffer, layer, next_layer, T, x, logits, y)


def cache_resize(ctx, S_new) -> int:
    return load().ft_cache_resize(ctx, S_new)


def measure_link(ctx, n_records, reps, gbps) -> int:
    return load().ft_measure_link(ctx, n_records, reps, gbps)


def get_ctl_state(ctx, slot_for_id, id_for_slot, stamps, clock) -> int:
    return load().ft_get_ctl_state(ctx, slot_for_id, id_for_slot, stamps, clock)


def set_ctl_state(ctx, slot_for_id, id_for_slot, stamps, clock) -> int:
    return load().ft_set_ctl_state(ctx, slot_for_id, id_for_slot, stamps, clock)


def get_last_ctl(ctx, info, F, C, victims, topk_ids, gates, slots_topk) -> int:
    return load().ft_get_last_ctl(ctx, info, F, C, victims, topk_ids, gates, slots_topk)


def read_slot(ctx, slot, host_dst) -> int:
    return load().ft_read_slot(ctx, slot, host_dst)


def get_counters(ctx, out) -> int:
    return load().ft_get_counters(ctx, out)


def profile_enable(ctx, enable) -> int:
    return load().ft_profile_enable(ctx, enable)


def profile_pause(ctx, paused) -> int:
    return load().ft_profile_pause(ctx, paused)


def profile_read(ctx, out) -> int:
    return load().ft_profile_read(ctx, out)


def kernel_name(kid: int):
    n = load().ft_kernel_name(kid)
    return n.decode() if n else None


def expert_ffn_noalloc(records, n_records, route_records, gates, x, partial_C, y, T, k, H, F, stream=None) -> int:
    """Context-free decode expert FFN that allocates nothing (see include/ft.h)."""
    return load().ft_expert_ffn_noalloc(records, n_records, route_records, gates, x, partial_C, y, T, k, H, F,
                                        stream)


def noalloc_status(stream=None) -> int:
    """Sync `stream`; return and clear the allocation-free path's error word."""
    return load().ft_noalloc_status(stream)


def num_slots(ctx) -> int:
    return load().ft_num_slots(ctx)


def set_wait_limit(ctx, ns) -> int:
    return load().ft_set_wait_limit(ctx, ns)


def get_status(ctx) -> int:
    return load().ft_get_status(ctx)


def destroy(ctx) -> None:
    load().ft_destroy(ctx)


def kv_page_bytes(L, Hkv, D, page) -> int:
    return load().ft_kv_page_bytes(L, Hkv, D, page)


def kv_scratch_bytes(Hq, Hkv, D, n_pages, n_rows, T_max, B_max) -> int:
    return load().ft_kv_scratch_bytes(Hq, Hkv, D, n_pages, n_rows, T_max, B_max)


def kv_init(L, Hq, Hkv, D, page, n_pages, n_rows, row_pages, dtype, T_max, B_max, pool, table, lens, refs, stream):
    h = _c_p()
    st = load().ft_kv_init(ctypes.byref(h), L, Hq, Hkv, D, page, n_pages, n_rows, row_pages, dtype, T_max, B_max, pool,
                           table, lens, refs, stream)
    return st, h.value


def kv_extend(kv, n, rows, add) -> int:
    return load().ft_kv_extend(kv, n, rows, add)


def kv_fork(kv, n, parents, children) -> int:
    return load().ft_kv_fork(kv, n, parents, children)


def kv_free(kv, n, rows) -> int:
    return load().ft_kv_free(kv, n, rows)


def kv_compact(kv) -> int:
    return load().ft_kv_compact(kv)


def kv_reorder(kv, n, rows, parents) -> int:
    return load().ft_kv_reorder(kv, n, rows, parents)


def kv_batch(kv, B, rows, add, T, cu_q, row_of, pos, slots) -> int:
    return load().ft_kv_batch(kv, B, rows, add, T, cu_q, row_of, pos, slots)


def qk_rope_store(kv, layer, T, qkv, ld, row_of, pos, q_out, ld_q, q_norm, k_norm, eps, cos_sin, max_pos, rot,
                  pair) -> int:
    return load().ft_qk_rope_store(kv, layer, T, qkv, ld, row_of, pos, q_out, ld_q, q_norm, k_norm, eps, cos_sin,
                                   max_pos, rot, pair)


def attn_plan(kv, B, T, cu_q, rows, n_groups, group_start, group_tokens) -> int:
    return load().ft_attn_plan(kv, B, T, cu_q, rows, n_groups, group_start, group_tokens)


def attn_forward(kv, layer, q, ld_q, out, ld_o, scale) -> int:
    return load().ft_attn_forward(kv, layer, q, ld_q, out, ld_o, scale)


def kv_last(kv, info) -> int:
    return load().ft_kv_last(kv, info)


def kv_status(kv) -> int:
    return load().ft_kv_status(kv)


def kv_destroy(kv) -> None:
    load().ft_kv_destroy(kv)


def block_norm(desc, T, block, ld_b, gate, ld_g, resid, ld_r, resid_out, ld_ro, out, ld_o, stream=None) -> int:
    """``desc`` is a NormDesc; the norms, gate and residual sum between two blocks (see include/ft_gen.h)."""
    return load().ft_block_norm(ctypes.addressof(desc), T, block, ld_b, gate, ld_g, resid, ld_r, resid_out, ld_ro, out, ld_o,
                                stream)


def beam_scratch_bytes(V, dtype, R_max, N_max) -> int:
    return load().ft_beam_scratch_bytes(V, dtype, R_max, N_max)


def beam_init(V, dtype, R_max, N_max, stream):
    h = _c_p()
    st = load().ft_beam_init(ctypes.byref(h), V, dtype, R_max, N_max, stream)
    return st, h.value


def beam_select(bm, B, K, N, logits, ld, scores, rows, done, eos, out_scores, out_parents, out_tokens, out_done) -> int:
    return load().ft_beam_select(bm, B, K, N, logits, ld, scores, rows, done, eos, out_scores, out_parents, out_tokens,
                                 out_done)


def beam_status(bm) -> int:
    return load().ft_beam_status(bm)


def beam_destroy(bm) -> None:
    load().ft_beam_destroy(bm)


# ------------------------------------------------------------ convenience

def _ptr(a) -> int | None:
    """Address of a numpy array / torch tensor / int; None for None."""
    try:
        return a.data_ptr()
    except AttributeError:
        pass
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "ctypes"):
        return a.ctypes.data
    raise TypeError(type(a))


class Context:
    """Owner of one ft_ctx*; every method raises FtError on a non-zero status.

    ``host_pool`` is a page-locked host tensor (or address) holding L*E
    records of ``record_bytes(H, F, fmt)`` bytes.  ``fmt`` is FT_FMT_BF16,
    FT_FMT_NVFP4 (then ``nvfp4_global`` is a fp32 array of L*E per-record
    globals), FT_FMT_MXFP4 or FT_FMT_FP8 (block-FP8); the record layouts are
    in include/ft.h.  Streams are ``torch.cuda.Stream.cuda_stream`` handles
    (0: the legacy default stream).
    """

    def __init__(self, L, E, k, H, F, S, host_pool, *, fmt=FT_FMT_BF16, T_max=16, T_prefill_max=0,
                 nvfp4_global=None, compute_stream=0, transfer_stream=0):
        st, h = layer_init(L, E, k, H, F, S, fmt, T_max, T_prefill_max, _ptr(host_pool), _ptr(nvfp4_global),
                           compute_stream or None, transfer_stream or None)
        _check(st, "ft_layer_init")
        self.h = h
        self.L, self.E, self.k, self.H, self.F, self.fmt = L, E, k, H, F, fmt
        self._keep = (host_pool, nvfp4_global)

    def close(self):
        if self.h:
            destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def S(self) -> int:
        return num_slots(self.h)

    def route_ctl(self, layer, T, logits=None, topk_ids=None, topk_w=None, B_P=1.0, B_H=1.0):
        _check(route_ctl(self.h, layer, T, _ptr(logits), _ptr(topk_ids), _ptr(topk_w), B_P, B_H), "ft_route_ctl")

    def moe_forward(self, x, partial_C, y):
        _check(moe_forward(self.h, _ptr(x), _ptr(partial_C), _ptr(y)), "ft_moe_forward")

    def prefill_begin(self, layer):
        _check(prefill_begin(self.h, layer), "ft_prefill_begin")

    def prefill_layer(self, buffer, layer, next_layer, T, x, logits, y):
        _check(prefill_layer(self.h, buffer, layer, next_layer, T, _ptr(x), _ptr(logits), _ptr(y)),
               "ft_prefill_layer")

    def cache_resize(self, S_new):
        _check(cache_resize(self.h, S_new), "ft_cache_resize")

    def measure_link(self, n_records, reps=3):
        """B_P: record-copy GB/s over the host link, measured with the fill path."""
        g = ctypes.c_double(0.0)
        _check(measure_link(self.h, n_records, reps, ctypes.byref(g)), "ft_measure_link")
        return g.value

    def ctl_state(self):
        import numpy as np
        S = self.S
        sfi = np.empty(self.L * self.E, dtype=np.int32)
        ifs = np.empty(S, dtype=np.int32)
        stp = np.empty(S, dtype=np.uint32)
        clk = np.empty(1, dtype=np.uint32)
        _check(get_ctl_state(self.h, _ptr(sfi), _ptr(ifs), _ptr(stp), _ptr(clk)), "ft_get_ctl_state")
        return sfi, ifs, stp, int(clk[0])

    def set_ctl_state(self, slot_for_id, id_for_slot, stamps, clock):
        import numpy as np
        a = np.ascontiguousarray(slot_for_id, dtype=np.int32)
        b = np.ascontiguousarray(id_for_slot, dtype=np.int32)
        c = np.ascontiguousarray(stamps, dtype=np.uint32)
        _check(set_ctl_state(self.h, _ptr(a), _ptr(b), _ptr(c), int(clock)), "ft_set_ctl_state")

    def last_ctl(self, T):
        import numpy as np
        info = CtlInfo()
        E, k = self.E, self.k
        F = np.empty(E, dtype=np.int32)
        C = np.empty(E, dtype=np.int32)
        V = np.empty(E, dtype=np.int32)
        ids = np.empty(T * k, dtype=np.int32)
        g = np.empty(T * k, dtype=np.float32)
        sl = np.empty(T * k, dtype=np.int32)
        _check(get_last_ctl(self.h, ctypes.byref(info), _ptr(F), _ptr(C), _ptr(V), _ptr(ids), _ptr(g), _ptr(sl)),
               "ft_get_last_ctl")
        return {"info": info, "F": F[:info.q].tolist(), "C": C[:info.nC].tolist(), "victims": V[:info.q].tolist(),
                "ids": ids.reshape(T, k), "gates": g.reshape(T, k), "slots_topk": sl.reshape(T, k)}

    def read_slot(self, slot):
        import numpy as np
        out = np.empty(record_bytes(self.H, self.F, self.fmt), dtype=np.uint8)
        _check(read_slot(self.h, slot, _ptr(out)), "ft_read_slot")
        return out

    def counters(self) -> dict:
        c = Counters()
        _check(get_counters(self.h, ctypes.byref(c)), "ft_get_counters")
        return {n: getattr(c, n) for n, _ in Counters._fields_}

    def status(self) -> int:
        return get_status(self.h)

    def set_wait_limit(self, ns: int):
        """Limit of the BF16 decode kernel's progress waits (0: the 2 s default)."""
        _check(set_wait_limit(self.h, ns), "ft_set_wait_limit")

    def profile_enable(self, on: bool = True):
        _check(profile_enable(self.h, 1 if on else 0), "ft_profile_enable")

    def profile_pause(self, paused: bool):
        _check(profile_pause(self.h, 1 if paused else 0), "ft_profile_pause")

    def profile_read(self) -> dict:
        pr = Profile()
        _check(profile_read(self.h, ctypes.byref(pr)), "ft_profile_read")
        out = {}
        for i in range(FT_K_COUNT):
            if pr.launches[i]:
                out[kernel_name(i)] = {"ms": pr.ms[i], "launches": int(pr.launches[i])}
        return out


class KvCache:
    """Owner of one ft_kv*; every method raises FtError on a non-zero status.

    ``pool`` is a device tensor (or address) of n_pages page records of
    ``kv_page_bytes(L, Hkv, D, page)`` bytes; ``table`` [n_rows, row_pages],
    ``lens`` [n_rows] and ``refs`` [n_pages] are int32 device tensors.  They
    stay the caller's; an empty cache has table -1, lens 0 and refs 0.  All
    calls run on ``stream`` (a ``torch.cuda.Stream.cuda_stream`` handle, 0: the
    legacy default stream).  Layouts and meanings are in include/ft_kv.h.
    """

    def __init__(self, L, Hq, Hkv, D, page, n_pages, n_rows, row_pages, pool, table, lens, refs, *, dtype=FT_KV_BF16,
                 T_max=16, B_max=16, stream=0):
        self.h = None
        st, h = kv_init(L, Hq, Hkv, D, page, n_pages, n_rows, row_pages, dtype, T_max, B_max, _ptr(pool), _ptr(table),
                        _ptr(lens), _ptr(refs), stream or None)
        _check(st, "ft_kv_init")
        self.h, self._lib = h, load()
        self._keep = (pool, table, lens, refs)

    def close(self):
        if self.h:
            kv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def extend(self, n, rows, add):
        st = self._lib.ft_kv_extend(self.h, n, _ptr(rows), _ptr(add))
        if st:
            _check(st, "ft_kv_extend")

    def fork(self, n, parents, children):
        st = self._lib.ft_kv_fork(self.h, n, _ptr(parents), _ptr(children))
        if st:
            _check(st, "ft_kv_fork")

    def free(self, n, rows):
        st = self._lib.ft_kv_free(self.h, n, _ptr(rows))
        if st:
            _check(st, "ft_kv_free")

    def reorder(self, n, parents, *, rows=None):
        """Row rows[i] (None: row i) becomes what row parents[i] was, all at once; -1 empties it."""
        st = self._lib.ft_kv_reorder(self.h, n, _ptr(rows), _ptr(parents))
        if st:
            _check(st, "ft_kv_reorder")

    def batch(self, B, add, T, cu_q, row_of, pos, *, rows=None, slots=None):
        """Grow the rows by add[b] tokens and list the new tokens for attn_plan and qk_rope_store, padded to T."""
        st = self._lib.ft_kv_batch(self.h, B, _ptr(rows), _ptr(add), T, _ptr(cu_q), _ptr(row_of), _ptr(pos), _ptr(slots))
        if st:
            _check(st, "ft_kv_batch")

    def compact(self):
        st = self._lib.ft_kv_compact(self.h)
        if st:
            _check(st, "ft_kv_compact")

    def qk_rope_store(self, layer, T, qkv, ld, row_of, pos, q_out, ld_q, *, q_norm=None, k_norm=None, eps=1e-6,
                      cos_sin=None, max_pos=0, rot=0, pair=False):
        st = self._lib.ft_qk_rope_store(self.h, layer, T, _ptr(qkv), ld, _ptr(row_of), _ptr(pos), _ptr(q_out), ld_q,
                                        _ptr(q_norm), _ptr(k_norm), eps, _ptr(cos_sin), max_pos, rot, 1 if pair else 0)
        if st:
            _check(st, "ft_qk_rope_store")

    def attn_plan(self, B, T, cu_q, *, rows=None, n_groups=0, group_start=None, group_tokens=None):
        """Lay out the work of a step from the lengths on the stream now; every layer's attn_forward uses it."""
        st = self._lib.ft_attn_plan(self.h, B, T, _ptr(cu_q), _ptr(rows), n_groups, _ptr(group_start), _ptr(group_tokens))
        if st:
            _check(st, "ft_attn_plan")

    def attn_forward(self, layer, q, ld_q, out, ld_o, scale):
        st = self._lib.ft_attn_forward(self.h, layer, _ptr(q), ld_q, _ptr(out), ld_o, scale)
        if st:
            _check(st, "ft_attn_forward")

    def last(self) -> dict:
        """What the last page operation did (syncs)."""
        i = KvInfo()
        _check(kv_last(self.h, ctypes.byref(i)), "ft_kv_last")
        return {n: getattr(i, n) for n, _ in KvInfo._fields_}

    def status(self) -> int:
        return kv_status(self.h)


class BlockNorm:
    """The norms around a block at one place of a model, with its gate and residual sum (include/ft_gen.h).

    ``pre`` and ``post`` are weight tensors [H] (or addresses) of type ``w_type``; None: all one.
    ``post_norm`` says whether the block's output is normalised (None: where ``post`` is given).
    Types are FT_T_*, ``gate`` is FT_GATE_*.  Calls run on ``stream``.
    """

    def __init__(self, H, *, pre=None, post=None, post_norm=None, block_type=FT_T_BF16, resid_type=FT_T_F32,
                 out_type=FT_T_BF16, w_type=FT_T_BF16, gate=FT_GATE_NONE, gate_type=FT_T_BF16, eps=1e-6, resid_scale=1.0,
                 block_scale=1.0, stream=0):
        norm = post is not None if post_norm is None else bool(post_norm)
        self.desc = NormDesc(H, block_type, resid_type, out_type, w_type, gate_type, gate, 1 if norm else 0, _ptr(post),
                             _ptr(pre), eps, resid_scale, block_scale)
        self.stream = stream or None
        self._at, self._lib = ctypes.addressof(self.desc), load()
        self._keep = (pre, post)

    def forward(self, T, resid, ld_r, *, block=None, ld_b=0, gate=None, ld_g=0, resid_out=None, ld_ro=0, out=None, ld_o=0):
        st = self._lib.ft_block_norm(self._at, T, _ptr(block), ld_b, _ptr(gate), ld_g, _ptr(resid), ld_r, _ptr(resid_out),
                                     ld_ro, _ptr(out), ld_o, self.stream)
        if st:
            _check(st, "ft_block_norm")


class Beams:
    """Owner of one ft_beam*: the choice of the next tokens of beams over a vocabulary of V (include/ft_gen.h).

    All calls run on ``stream``; every method raises FtError on a non-zero status.
    """

    def __init__(self, V, R_max, N_max, *, dtype=FT_T_F32, stream=0):
        self.h = None
        st, h = beam_init(V, dtype, R_max, N_max, stream or None)
        _check(st, "ft_beam_init")
        self.h, self._lib = h, load()

    def close(self):
        if self.h:
            beam_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def select(self, B, K, N, logits, ld, scores, out_scores, out_parents, out_tokens, *, rows=None, done=None, eos=-1,
               out_done=None):
        """The N best continuations of each of B requests of K beams, best first."""
        st = self._lib.ft_beam_select(self.h, B, K, N, _ptr(logits), ld, _ptr(scores), _ptr(rows), _ptr(done), eos,
                                      _ptr(out_scores), _ptr(out_parents), _ptr(out_tokens), _ptr(out_done))
        if st:
            _check(st, "ft_beam_select")

    def status(self) -> int:
        return beam_status(self.h)
