"""Thin Python binding over libhq.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: tensors are passed as device pointers, the status code
is checked, and a non-zero status raises :class:`HqError`.  PyTorch is used for
device memory and streams only.  If ``libhq.so`` is missing, importing this
module raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhq.so")

HQ_HEAD_DIM = 128
HQ_STAGE = 64
HQ_QBUF = 64
PAGE_POSITIONS = 64
PAGE_BYTES = 10304
PAGE_KCODES, PAGE_VCODES, PAGE_KSZ, PAGE_VSZ, PAGE_VLMASK = 0, 4096, 8192, 9216, 10240
STATE_T, STATE_NPACKED, STATE_NVL, STATE_NQ, STATE_KSEL, STATE_ERR = range(6)
STATE_WORDS = 8
OP_SELECT, OP_MERGE, OP_DECODE = 0, 1, 2
DEVERR_STAGING_FULL, DEVERR_CAPACITY, DEVERR_VL_CAPACITY, DEVERR_TIMEOUT, DEVERR_PAGE = 1, 2, 4, 8, 16
DEVERR_ROWS = 32
F16, BF16, F32 = 0, 1, 2
_DTYPE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = range(5)
KV8_E4M3, KV8_INT8 = 0, 1
KV8_PAGE_BYTES, KV8_TAIL, KV8_WS_ZERO = 16448, 128, 4096


class HqError(RuntimeError):
    pass


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -m hybrid_precision_attention_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)


class HqCacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "D", "W", "rho_bp", "cap", "vl_cap")] + [
        (n, ctypes.c_void_p)
        for n in ("pages", "kf", "vf", "vl_pos", "kr", "vr", "qbuf", "vl_sel", "state", "page_table", "score_acc",
                  "qlse")
    ] + [("n_pages", ctypes.c_int32), ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def page_layout(k_bits: int = 4, v_bits: int = 4) -> dict:
    """Page geometry of a code width pair (include/hq.h, HQ_PAGE_SUBPOS and friends)."""
    pr = 32 if k_bits + v_bits > 8 else 64
    sub = pr * (16 * k_bits + 16 * v_bits + 32)
    mask = (64 // pr) * sub
    return {"pr": pr, "sub": sub, "mask": mask, "bytes": (mask + 16 + 63) // 64 * 64,
            "kcodes": 0, "vcodes": pr * 16 * k_bits, "ksz": pr * 16 * (k_bits + v_bits),
            "vsz": pr * 16 * (k_bits + v_bits) + pr * 16}


_P = ctypes.c_void_p
_I = ctypes.c_int32
_S = ctypes.c_size_t
_CP = ctypes.POINTER(HqCacheStruct)

_lib.hq_abi_version.restype = _I
_lib.hq_status_str.restype = ctypes.c_char_p
_lib.hq_status_str.argtypes = [_I]
_lib.hq_last_error.restype = ctypes.c_char_p
_lib.hq_last_error.argtypes = []
_lib.hq_cache_validate.restype = _I
_lib.hq_cache_validate.argtypes = [_CP]
_lib.hq_workspace_bytes.restype = _S
_lib.hq_workspace_bytes.argtypes = [_CP, _I, _I]
_lib.hq_cache_reset.restype = _I
_lib.hq_cache_reset.argtypes = [_CP, _P]
_lib.hq_select_vlines.restype = _I
_lib.hq_select_vlines.argtypes = [_CP, _P, _I, _P, _I, _P, _P, _S, _P]
_lib.hq_pack_merge.restype = _I
_lib.hq_pack_merge.argtypes = [_CP, _P, _P, _I, _P, _S, _P]
_lib.hq_decode_attn.restype = _I
_lib.hq_decode_attn.argtypes = [_CP, _P, _P, _P, _P, ctypes.c_float, _P, _S, _P]
_lib.hq_decode_attn_noalloc.restype = _I
_lib.hq_decode_attn_noalloc.argtypes = [_CP, _P, _P, _P, _P, ctypes.c_float, _P]
_lib.hq_prefill_workspace_bytes.restype = _S
_lib.hq_prefill_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
_lib.hq_prefill_attn.restype = _I
_lib.hq_prefill_attn.argtypes = [_I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _S, _P]
PREFILL_E4M3, PREFILL_INT8_QK = 0, 1

_lib.hq_diag_stream_read.restype = _I
_lib.hq_diag_stream_read.argtypes = [_P, _S, _P, _I, _P]



class HqRopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("x_batch", "x_tok", "x_head", "y_batch", "y_tok", "y_head")
    ] + [("H", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class HqKv8CacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hkv", "D", "cap", "fmt", "n_pages")] + [
        (n, ctypes.c_void_p) for n in ("pages", "page_table", "tail_k", "tail_v", "tail_scale", "err")]


_L = ctypes.c_int64
_F = ctypes.c_float
_DBL = ctypes.c_double
_KP = ctypes.POINTER(HqKv8CacheStruct)
_RP = ctypes.POINTER(HqRopeTensor)
_lib.hq_rope_freqs.restype = _I
_lib.hq_rope_freqs.argtypes = [_I, _DBL, _I, _DBL, _DBL, _DBL, _DBL, _P, ctypes.POINTER(_F)]
_lib.hq_rope.restype = _I
_lib.hq_rope.argtypes = [_I, _I, _I, _I, _I, _I, _I, _RP, _RP, _P, _P, _F, _P]
_lib.hq_kv8_validate.restype = _I
_lib.hq_kv8_validate.argtypes = [_KP]
_lib.hq_kv8_append.restype = _I
_lib.hq_kv8_append.argtypes = [_KP, _I, _P, _L, _L, _P, _L, _L, _I, _P, _P, _P]
_lib.hq_kv8_read.restype = _I
_lib.hq_kv8_read.argtypes = [_KP, _I, _P, _I, _I, _P, _P, _L, _L, _L, _I, _P]
_lib.hq_kv8_attn_workspace_bytes.restype = _S
_lib.hq_kv8_attn_workspace_bytes.argtypes = [_KP, _I, _I]
_lib.hq_kv8_attn.restype = _I
_lib.hq_kv8_attn.argtypes = [_KP, _I, _P, _L, _L, _I, _I, _P, _P, _I, _I, _F, _P, _L, _L, _P, _P, _S, _P]

EXPORTED = ("hq_abi_version", "hq_status_str", "hq_last_error", "hq_cache_validate", "hq_workspace_bytes", "hq_cache_reset",
            "hq_select_vlines", "hq_pack_merge", "hq_decode_attn", "hq_decode_attn_noalloc",
            "hq_prefill_workspace_bytes", "hq_prefill_attn", "hq_rope_freqs", "hq_rope", "hq_kv8_validate", "hq_kv8_append",
            "hq_kv8_read", "hq_kv8_attn_workspace_bytes", "hq_kv8_attn", "hq_diag_stream_read")


def _check(st: int, what: str):
    if st != 0:
        detail = f" [{_lib.hq_last_error().decode()}]" if st == 5 else ""
        raise HqError(f"{what}: {_lib.hq_status_str(st).decode()} (status {st}){detail}")


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise HqError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def k_of(n: int, rho_bp: int) -> int:
    """ceil(rho * n) in integer basis points (same rule as the kernels)."""
    if n <= 0 or rho_bp <= 0:
        return 0
    return min(n, (n * rho_bp + 9999) // 10000)


def abi_version() -> int:
    return int(_lib.hq_abi_version())


class HybridCache:
    """Device buffers of one layer's hybrid cache (layout: include/hq.h, struct hq_cache).

    ``paged=True`` keeps the K4V4 store as a pool of ``n_pages`` pages (default:
    exactly the pages the batch can use) with a page table ``[B, Hkv, cap/64]``;
    ``page_order`` (optional, a permutation of the pool indices) fills the table,
    else page j of (b, h) is pool page (b*Hkv + h)*(cap/64) + j."""

    def __init__(self, B: int, Hq: int, Hkv: int, cap: int, W: int = 128, rho_bp: int = 500, vl_cap: int = None,
                 device="cuda", D: int = HQ_HEAD_DIM, paged: bool = False, n_pages: int = None, page_order=None,
                 running_scores: bool = False, decode_lse: bool = True, k_bits: int = 4, v_bits: int = 4):
        cap = ((cap + 127) // 128) * 128
        if vl_cap is None:
            vl_cap = max(16, ((k_of(max(cap - W, 0), rho_bp) + 15) // 16) * 16)
        self.B, self.Hq, self.Hkv, self.D, self.W, self.rho_bp, self.cap, self.vl_cap = B, Hq, Hkv, D, W, rho_bp, cap, vl_cap
        self.R = ((W + HQ_STAGE + 15) // 16) * 16   # HQ_RING_LEN(W)
        self.npg = cap // PAGE_POSITIONS
        self.k_bits, self.v_bits = k_bits, v_bits
        self.layout = page_layout(k_bits, v_bits)
        PB = self.layout["bytes"]
        dev = torch.device(device)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)
        self.paged = paged
        if paged:
            self.n_pages = n_pages if n_pages is not None else B * Hkv * self.npg
            self.pages = z((self.n_pages, PB), torch.uint8)
            order = torch.arange(B * Hkv * self.npg, dtype=torch.int32) if page_order is None else \
                torch.as_tensor(page_order, dtype=torch.int32)
            self.page_table = order.reshape(B, Hkv, self.npg).to(dev).contiguous()
        else:
            self.n_pages = 0
            self.pages = z((B, Hkv, self.npg, PB), torch.uint8)
            self.page_table = None
        self.kf = z((B, Hkv, vl_cap, D), torch.float16)
        self.vf = z((B, Hkv, vl_cap, D), torch.float16)
        self.vl_pos = z((B, Hkv, vl_cap), torch.int32)
        self.kr = z((B, Hkv, self.R, D), torch.float16)
        self.vr = z((B, Hkv, self.R, D), torch.float16)
        self.qbuf = z((B, Hq, HQ_QBUF, D), torch.float16)
        self.vl_sel = z((B, Hkv, vl_cap), torch.int32)
        self.state_t = z((B, STATE_WORDS), torch.int32)
        self.score_acc = z((B, Hkv, cap), torch.float32) if running_scores else None
        self.qlse = torch.full((B, Hq, HQ_QBUF), float("nan"), dtype=torch.float32, device=dev) if decode_lse else None
        self.c = HqCacheStruct(B, Hq, Hkv, D, W, rho_bp, cap, vl_cap, *[t.data_ptr() for t in (
            self.pages, self.kf, self.vf, self.vl_pos, self.kr, self.vr, self.qbuf, self.vl_sel, self.state_t)],
            self.page_table.data_ptr() if paged else None,
            self.score_acc.data_ptr() if running_scores else None,
            self.qlse.data_ptr() if decode_lse else None, self.n_pages, k_bits, v_bits, 0)
        _check(_lib.hq_cache_validate(ctypes.byref(self.c)), "hq_cache_validate")
        self._ws = {}

    def slot(self, b: int) -> "CacheSlot":
        """Single-sequence view of batch row b (a B = 1 descriptor into the same buffers)."""
        return CacheSlot(self, b)

    def workspace(self, op: int, L: int = 0) -> torch.Tensor:
        n = int(_lib.hq_workspace_bytes(ctypes.byref(self.c), op, L))
        if n == 0:
            raise HqError("hq_workspace_bytes returned 0")
        w = self._ws.get(op)
        if w is None or w.numel() < n:
            w = torch.zeros(n, dtype=torch.uint8, device=self.pages.device)
            self._ws[op] = w
        return w

    def states(self) -> list:
        """Every sequence's state row as a dict."""
        rows = self.state_t.cpu().tolist()
        return [{"T": s[STATE_T], "n_packed": s[STATE_NPACKED], "n_vl": s[STATE_NVL], "n_q": s[STATE_NQ],
                 "k_sel": s[STATE_KSEL], "err": s[STATE_ERR]} for s in rows]

    def state(self, b: int = None) -> dict:
        """State row b; with b omitted, the rows must agree (a uniform batch) and
        the common row is returned, with the error bits of all rows OR-ed."""
        rows = self.states()
        if b is not None:
            return rows[b]
        out = dict(rows[0])
        err = 0
        for r in rows:
            err |= r["err"]
            for k in ("T", "n_packed", "n_vl", "n_q", "k_sel"):
                if r[k] != out[k]:
                    raise HqError(f"state rows differ ({k}): use state(b) or states() for a ragged batch")
        out["err"] = err
        return out

    def nbytes(self) -> int:
        ts = [self.pages, self.kf, self.vf, self.vl_pos, self.kr, self.vr, self.qbuf, self.vl_sel, self.state_t]
        for t in (self.page_table, self.score_acc, self.qlse):
            if t is not None:
                ts.append(t)
        return sum(t.numel() * t.element_size() for t in ts)

    def page_bytes(self) -> np.ndarray:
        """The K4V4 pages of every (b, h) in position order: uint8 [B, Hkv, cap/64, PAGE_BYTES] (host copy)."""
        pg = self.pages.cpu().numpy()
        if not self.paged:
            return pg
        tab = self.page_table.cpu().numpy().astype(np.int64)
        return pg[np.clip(tab, 0, self.n_pages - 1)]

    def packed(self) -> dict:
        """The packed store by position (host copies): codes kq/vq uint8 [B,Hkv,cap,16*bits],
        scale/zero words ksz/vsz uint32 [B,Hkv,cap,D/32], VL bitmap vl_bits bool [B,Hkv,cap]."""
        pg = self.page_bytes()
        B, H, npg, _ = pg.shape
        ly = self.layout
        pr, nsub = ly["pr"], 64 // ly["pr"]

        def take(off, width):
            parts = [pg[..., s * ly["sub"] + off:s * ly["sub"] + off + pr * width].reshape(B, H, npg, pr, width)
                     for s in range(nsub)]
            return np.concatenate(parts, axis=3).reshape(B, H, npg * 64, width)
        m = pg[..., ly["mask"]:ly["mask"] + 8].copy()
        bits = np.unpackbits(m, axis=-1, bitorder="little").reshape(B, H, npg * 64).astype(bool)
        return {"kq": take(ly["kcodes"], 16 * self.k_bits), "vq": take(ly["vcodes"], 16 * self.v_bits),
                "ksz": take(ly["ksz"], 16).copy().view(np.uint32), "vsz": take(ly["vsz"], 16).copy().view(np.uint32),
                "vl_bits": bits}


class CacheSlot:
    """One sequence of a HybridCache as a B = 1 cache: the descriptor's pointers
    are offset to batch row b (the page pool, when paged, is shared; the page
    table row is b's).  Accepted by every entry point of this module."""

    def __init__(self, parent: HybridCache, b: int):
        if not 0 <= b < parent.B:
            raise HqError(f"slot {b} outside the batch of {parent.B}")
        self.parent, self.b = parent, b
        self.B, self.Hq, self.Hkv, self.D, self.W = 1, parent.Hq, parent.Hkv, parent.D, parent.W
        self.rho_bp, self.cap, self.vl_cap, self.R = parent.rho_bp, parent.cap, parent.vl_cap, parent.R
        sl = lambda t: t[b:b + 1]
        self.kf, self.vf, self.vl_pos = sl(parent.kf), sl(parent.vf), sl(parent.vl_pos)
        self.kr, self.vr, self.qbuf, self.vl_sel = sl(parent.kr), sl(parent.vr), sl(parent.qbuf), sl(parent.vl_sel)
        self.state_t = sl(parent.state_t)
        self.pages = parent.pages if parent.paged else sl(parent.pages)
        self.page_table = sl(parent.page_table) if parent.paged else None
        self.score_acc = sl(parent.score_acc) if parent.score_acc is not None else None
        self.qlse = sl(parent.qlse) if parent.qlse is not None else None
        self.c = HqCacheStruct(1, self.Hq, self.Hkv, self.D, self.W, self.rho_bp, self.cap, self.vl_cap, *[
            t.data_ptr() for t in (self.pages, self.kf, self.vf, self.vl_pos, self.kr, self.vr, self.qbuf, self.vl_sel,
                                   self.state_t)], self.page_table.data_ptr() if parent.paged else None,
            self.score_acc.data_ptr() if self.score_acc is not None else None,
            self.qlse.data_ptr() if self.qlse is not None else None, parent.n_pages, parent.k_bits, parent.v_bits, 0)
        self.k_bits, self.v_bits, self.layout = parent.k_bits, parent.v_bits, parent.layout
        _check(_lib.hq_cache_validate(ctypes.byref(self.c)), "hq_cache_validate (slot)")
        self._ws = {}

    workspace = HybridCache.workspace

    def state(self, b: int = None) -> dict:
        return self.parent.state(self.b)


# ----------------------------------------------------------------------------- entry points

def hq_cache_reset(cache: HybridCache, stream=None):
    _check(_lib.hq_cache_reset(ctypes.byref(cache.c), _stream(stream)), "hq_cache_reset")


def hq_select_vlines(cache: HybridCache, k_dense=None, q_ext=None, scores_out=None, stream=None):
    """Init mode when k_dense [B,Hkv,L,D] and q_ext [B,Hq,nq,D] are given, else decode mode."""
    L = nq = 0
    if k_dense is not None:
        L = k_dense.shape[2]
        nq = q_ext.shape[2]
        _need(k_dense, torch.float16, (cache.B, cache.Hkv, L, cache.D), "k_dense")
        _need(q_ext, torch.float16, (cache.B, cache.Hq, nq, cache.D), "q_ext")
    if scores_out is not None:
        _need(scores_out, torch.float32, (cache.B, cache.Hkv, cache.cap), "scores_out")
    ws = cache.workspace(OP_SELECT, L)
    _check(_lib.hq_select_vlines(ctypes.byref(cache.c), _ptr(k_dense), L, _ptr(q_ext), nq, _ptr(scores_out),
                                 _ptr(ws), ws.numel(), _stream(stream)), "hq_select_vlines")


def hq_pack_merge(cache: HybridCache, k_dense=None, v_dense=None, stream=None):
    """Init mode with dense K/V [B,Hkv,L,D]; merge mode with neither."""
    L = 0
    if k_dense is not None:
        L = k_dense.shape[2]
        _need(k_dense, torch.float16, (cache.B, cache.Hkv, L, cache.D), "k_dense")
        _need(v_dense, torch.float16, (cache.B, cache.Hkv, L, cache.D), "v_dense")
    ws = cache.workspace(OP_MERGE)
    _check(_lib.hq_pack_merge(ctypes.byref(cache.c), _ptr(k_dense), _ptr(v_dense), L, _ptr(ws), ws.numel(),
                              _stream(stream)), "hq_pack_merge")


def hq_decode_attn(cache: HybridCache, q, k_new, v_new, out=None, sm_scale: float = None, stream=None):
    _need(q, torch.float16, (cache.B, cache.Hq, cache.D), "q")
    _need(k_new, torch.float16, (cache.B, cache.Hkv, cache.D), "k_new")
    _need(v_new, torch.float16, (cache.B, cache.Hkv, cache.D), "v_new")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.float16, (cache.B, cache.Hq, cache.D), "out")
    if sm_scale is None:
        sm_scale = cache.D ** -0.5
    ws = cache.workspace(OP_DECODE)
    _check(_lib.hq_decode_attn(ctypes.byref(cache.c), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                               ctypes.c_float(sm_scale), _ptr(ws), ws.numel(), _stream(stream)), "hq_decode_attn")
    return out


def hq_decode_attn_noalloc(cache: HybridCache, q, k_new, v_new, out=None, sm_scale: float = None, stream=None):
    """hq_decode_attn for callers that may not allocate device memory: no
    workspace argument, the library's fixed scratch array is used instead (see
    include/hq.h for its size and sharing rules)."""
    _need(q, torch.float16, (cache.B, cache.Hq, cache.D), "q")
    _need(k_new, torch.float16, (cache.B, cache.Hkv, cache.D), "k_new")
    _need(v_new, torch.float16, (cache.B, cache.Hkv, cache.D), "v_new")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.float16, (cache.B, cache.Hq, cache.D), "out")
    if sm_scale is None:
        sm_scale = cache.D ** -0.5
    _check(_lib.hq_decode_attn_noalloc(ctypes.byref(cache.c), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                       ctypes.c_float(sm_scale), _stream(stream)), "hq_decode_attn_noalloc")
    return out


def hq_prefill_workspace_bytes(B, Hq, Hkv, L, vl_stride, D=HQ_HEAD_DIM) -> int:
    return int(_lib.hq_prefill_workspace_bytes(B, Hq, Hkv, L, D, vl_stride))


def prefill_ws_regions(B, Hq, Hkv, L, D=HQ_HEAD_DIM) -> dict:
    """Byte offsets of the documented prefill workspace regions (include/hq.h):
    the error word, the e4m3 codes of Q and K, the fp16 values of V."""
    Lp = (L + 127) // 128 * 128
    al = lambda x: (x + 1023) // 1024 * 1024
    q8 = al(16)
    k8 = al(q8 + B * Hq * Lp * D)
    v8 = al(k8 + B * Hkv * Lp * D)
    return {"err": 0, "q8": q8, "k8": k8, "v16": v8, "Lp": Lp}


def hq_prefill_attn(q, k, v, vl_pos, n_vl: int, W: int, sm_scale: float = None, out=None, ws=None, stream=None,
                    qk_format: int = PREFILL_E4M3):
    """q [B,Hq,L,D], k/v [B,Hkv,L,D] fp16; vl_pos int32 [B,Hkv,stride] (first n_vl ascending);
    qk_format PREFILL_E4M3 (e4m3 Q, K, V) or PREFILL_INT8_QK (INT8 Q, K and FP16 V) for the quantised keys."""
    B, Hq, L, D = q.shape
    Hkv = k.shape[1]
    _need(q, torch.float16, (B, Hq, L, D), "q")
    _need(k, torch.float16, (B, Hkv, L, D), "k")
    _need(v, torch.float16, (B, Hkv, L, D), "v")
    _need(vl_pos, torch.int32, (B, Hkv, vl_pos.shape[2]), "vl_pos")
    if out is None:
        out = torch.empty_like(q)
    n = hq_prefill_workspace_bytes(B, Hq, Hkv, L, vl_pos.shape[2], D)
    if ws is None:
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    if sm_scale is None:
        sm_scale = D ** -0.5
    _check(_lib.hq_prefill_attn(B, Hq, Hkv, L, D, _ptr(q), _ptr(k), _ptr(v), _ptr(vl_pos), n_vl, vl_pos.shape[2], W,
                                qk_format, ctypes.c_float(sm_scale), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "hq_prefill_attn")
    return out


# ----------------------------------------------------------------------------- rotary positions, 8-bit block cache

class _On:
    """Makes a call's launch stream current with its device, so that what the call allocates belongs to it
    (stream None: the device's current stream)."""

    def __init__(self, index, stream=None):
        if stream is None:
            self.ctx = torch.cuda.device(index)
        else:
            if stream.device.index != index:
                raise HqError(f"stream of {stream.device} for tensors on cuda:{index}")
            self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


# The current device and its current stream's handle, without the Device and
# Stream objects of the torch.cuda functions (2 us and more of a small call).
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_HALVES = (torch.float16, torch.bfloat16)
_ALL = tuple(_DTYPE)


def _rows(t, index, shape, name, dtypes=_HALVES):
    """A tensor of that shape (None: any size) on that CUDA device, its last dimension contiguous."""
    have = t.shape
    ok = len(have) == len(shape) and t.dtype in dtypes and t.is_cuda and t.get_device() == index and \
        (t.stride(-1) == 1 or have[-1] <= 1 or t.numel() == 0)
    if ok:
        for n, m in zip(shape, have):
            if n != m and n is not None:
                ok = False
    if not ok:
        raise HqError(f"{name}: expected {'/'.join(str(d) for d in dtypes)} {tuple(shape)} on cuda:{index} with contiguous "
                      f"rows, got {t.dtype} {tuple(have)} strides {t.stride()} on {t.device}")


def _ints(t, index, shape, name):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous() or not t.is_cuda or t.get_device() != index:
        raise HqError(f"{name}: expected contiguous {torch.int32} {tuple(shape)} on cuda:{index}, got {t.dtype} "
                      f"{tuple(t.shape)} on {t.device}")


def _scratch(t, index, name, dtype=None, shape=None):
    """Memory that a kernel writes as it lies: contiguous, on that CUDA device."""
    if not t.is_cuda or t.get_device() != index or not t.is_contiguous() or (dtype is not None and t.dtype != dtype) or \
            (shape is not None and tuple(t.shape) != shape):
        raise HqError(f"{name}: expected contiguous {dtype or 'memory'} {shape or ''} on cuda:{index}, got {t.dtype} "
                      f"{tuple(t.shape)} on {t.device}")


class _Places:
    """A tensor's bytes by address, for numpy, which does not look at them."""

    def __init__(self, t):
        n = t.element_size()
        self.__array_interface__ = dict(version=3, data=(t.data_ptr(), False), typestr=f"|V{n}", shape=tuple(t.shape),
                                        strides=tuple(s * n for s in t.stride()))


def _overlap(a, b) -> bool:
    """Whether two tensors (strides not negative) share an element's place: exactly, but for strides so unlike that
    numpy gives up on them, which count as apart."""
    pa, pb = a.data_ptr(), b.data_ptr()
    if pa > pb:
        a, b, pa, pb = b, a, pb, pa
    # mostly the one that begins first has ended where the other begins
    if pb - pa >= (a.nbytes if a.is_contiguous() else (sum((n - 1) * s for n, s in zip(a.shape, a.stride())) + 1) * a.element_size()):
        return False
    if a.numel() == 0 or b.numel() == 0:
        return False
    try:
        return bool(np.shares_memory(np.asarray(_Places(a)), np.asarray(_Places(b)), max_work=100000))
    except np.exceptions.TooHardError:
        return False


def _output(call, t, name, other, x):
    """An output of the caller's: each element in a place of its own, apart from those of x."""
    if 0 in t.stride() and any(s == 0 and n > 1 for n, s in zip(t.shape, t.stride())):
        raise HqError(f"{call}: elements of {name} share places, strides {t.stride()}")
    if _overlap(t, x):
        raise HqError(f"{call}: {name} overlaps {other}")


class RopeTable:
    """Frequencies of ``rot`` rotated elements (include/hq.h, hq_rope_freqs), on the device."""

    def __init__(self, rot: int, base: float = 10000.0, kind: int = ROPE_PLAIN, factor: float = 1.0, orig_len: float = 0,
                 low: float = 0, high: float = 0, device="cuda"):
        f = np.zeros(max(rot, 0) // 2, dtype=np.uint64)
        amp = _F()
        _check(_lib.hq_rope_freqs(rot, base, kind, factor, orig_len, low, high, f.ctypes.data, ctypes.byref(amp)), "hq_rope_freqs")
        self.rot, self.amp = rot, amp.value
        self.freqs = torch.from_numpy(f.view(np.int64)).to(device)
        self.index = self.freqs.get_device()
        self._ptr = self.freqs.data_ptr()


def hq_rope(q, k, pos, table: RopeTable, layout: int = ROPE_HALF, grad: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [B, T, Hq, D] and k [B, T, Hkv, D] (or None) at pos int32 [B, T]; without a batch
    dimension [T, H, D] and [T].  Strided views are taken as they are; q_out, k_out may be q, k themselves.
    ``grad``: the transposed rotation (gradients of q and k from those of the outputs).  Returns (q_out, k_out).
    Where q or k requires grad the outputs do, too, to any order; q_out and k_out are refused then."""
    dev = table.index
    if dev < 0:
        raise HqError("hq_rope: the table is not on a CUDA device")
    if stream is not None or _device() != dev:
        with _On(dev, stream):
            return hq_rope(q, k, pos, table, layout, grad, q_out, k_out)
    if (q.requires_grad or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        if q_out is not None or k_out is not None:
            raise HqError("hq_rope: q_out and k_out have no gradient, and q or k requires one (torch.no_grad, or leave them out)")
        return _Rope.apply(q, k, pos, table, layout, grad)
    shape = q.shape
    n = len(shape)
    if n != 4 and n != 3:
        raise HqError(f"q: expected [B, T, H, D] or [T, H, D], got {tuple(shape)}")
    lead, D = shape[:-2], shape[-1]
    _ints(pos, dev, lead, "pos")
    dt = q.dtype
    _rows(q, dev, shape, "q", _ALL)
    if q_out is None:
        q_out = torch.empty_like(q)
    else:
        _rows(q_out, dev, shape, "q_out", (dt,))
        if q_out.data_ptr() != q.data_ptr():
            _output("hq_rope", q_out, "q_out", "q", q)
    a, q_out = _rope_side(q, q_out, n)
    b = None
    if k is not None:
        _rows(k, dev, (*lead, None, D), "k", (dt,))
        if k_out is None:
            k_out = torch.empty_like(k)
        else:
            _rows(k_out, dev, k.shape, "k_out", (dt,))
            if k_out.data_ptr() != k.data_ptr():
                _output("hq_rope", k_out, "k_out", "k", k)
        b, k_out = _rope_side(k, k_out, n)
    st = _lib.hq_rope(_DTYPE[dt], lead[0] if n == 4 else 1, lead[-1], D, table.rot, layout, 1 if grad else 0, a, b,
                      pos.data_ptr(), table._ptr, table.amp, _raw_stream(dev))
    if st:
        _check(st, "hq_rope")
    return q_out, k_out if k is not None else None


class _Rope(torch.autograd.Function):
    """hq_rope in a graph: its gradient is the call with the rotation transposed."""

    @staticmethod
    def forward(ctx, q, k, pos, table, layout, grad):
        ctx.save_for_backward(pos)
        ctx.how = table, layout, not grad
        ctx.set_materialize_grads(False)
        return hq_rope(q, k, pos, table, layout, grad)

    @staticmethod
    def backward(ctx, *g):
        # of outputs that are used, for inputs that ask; expanded gradients (a sum's) have no rows
        g = [x.contiguous() if x is not None and need and x.stride(-1) != 1 else x if need else None
             for x, need in zip(g, ctx.needs_input_grad)]
        pos, = ctx.saved_tensors
        if g[0] is not None:
            g = hq_rope(g[0], g[1], pos, *ctx.how)
        elif g[1] is not None:
            g[1] = hq_rope(g[1], None, pos, *ctx.how)[0]
        return *g, None, None, None, None


def _rope_side(x, y, n):
    """A tensor's part of the call, and its output: empty_like's follows the order of x's strides, which for windows one
    element apart is not that of rows, and is made anew then."""
    xs, ys = x.stride(), y.stride()
    if ys[-1] != 1 and y.shape[-1] > 1 and y.numel():
        y = x.new_empty(x.shape)
        ys = y.stride()
    if n == 3:
        return HqRopeTensor(x.data_ptr(), y.data_ptr(), 0, xs[0], xs[1], 0, ys[0], ys[1], x.shape[1], 0), y
    return HqRopeTensor(x.data_ptr(), y.data_ptr(), xs[0], xs[1], xs[2], ys[0], ys[1], ys[2], x.shape[2], 0), y


_SCRATCH = {}  # hq_kv8_attn's, by device and launch stream


class Kv8Cache:
    """Device buffers of one layer's 8-bit block cache (layout: include/hq.h, struct hq_kv8_cache).

    ``paged=True`` keeps the blocks in a pool of ``n_pages`` pages (default: what the batch can use) with a page
    table [B, Hkv, cap/64] (``page_order`` fills it, else in order).  ``pages``, ``page_table``, ``tail_k``,
    ``tail_v`` and ``tail_scale`` may be given as tensors of the documented layout instead."""

    def __init__(self, B: int, Hkv: int, cap: int, fmt: int = KV8_E4M3, device="cuda", D: int = HQ_HEAD_DIM,
                 paged: bool = False, n_pages: int = None, page_order=None, pages=None, page_table=None, tail_k=None,
                 tail_v=None, tail_scale=None):
        cap = ((cap + 127) // 128) * 128
        self.B, self.Hkv, self.D, self.cap, self.fmt, self.npg = B, Hkv, D, cap, fmt, cap // PAGE_POSITIONS
        dev = pages.device if pages is not None else torch.device(device)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)
        if page_table is None and paged:
            n_pages = n_pages if n_pages is not None else B * Hkv * self.npg
            order = torch.arange(B * Hkv * self.npg, dtype=torch.int32) if page_order is None else \
                torch.as_tensor(page_order, dtype=torch.int32)
            page_table = order.reshape(B, Hkv, self.npg).to(dev).contiguous()
        if pages is None:
            pages = z((n_pages if n_pages is not None else B * Hkv * self.npg, KV8_PAGE_BYTES), torch.uint8) \
                if page_table is not None else z((B, Hkv, self.npg, KV8_PAGE_BYTES), torch.uint8)
        self.pages, self.page_table = pages, page_table
        dev = pages.device
        if page_table is not None:
            _ints(page_table, dev.index, (B, Hkv, self.npg), "page_table")
            _need(pages, torch.uint8, (pages.shape[0], KV8_PAGE_BYTES), "pages")
        else:
            _need(pages, torch.uint8, (B, Hkv, self.npg, KV8_PAGE_BYTES), "pages")
        self.tail_k = tail_k if tail_k is not None else z((B, Hkv, 2, 64 * D), torch.float16)
        self.tail_v = tail_v if tail_v is not None else z((B, Hkv, 2, 64 * D), torch.float16)
        self.tail_scale = tail_scale if tail_scale is not None else z((B, Hkv, 2, KV8_TAIL), torch.float32)
        _need(self.tail_k, torch.float16, (B, Hkv, 2, 64 * D), "tail_k")
        _need(self.tail_v, torch.float16, (B, Hkv, 2, 64 * D), "tail_v")
        _need(self.tail_scale, torch.float32, (B, Hkv, 2, KV8_TAIL), "tail_scale")
        self.err = z((B,), torch.int32)
        self.device, self.index = self.err.device, self.err.get_device()
        for name in ("tail_k", "tail_v", "tail_scale"):
            if getattr(self, name).get_device() != self.index:
                raise HqError(f"{name}: on {getattr(self, name).device}, the pages on {self.device}")
        self.c = HqKv8CacheStruct(B, Hkv, D, cap, fmt, pages.shape[0] if page_table is not None else 0, *[
            None if t is None else t.data_ptr() for t in (pages, page_table, self.tail_k, self.tail_v, self.tail_scale, self.err)])
        self.ref = ctypes.byref(self.c)
        _check(_lib.hq_kv8_validate(self.ref), "hq_kv8_validate")
        self._ws, self._ws_bytes = {}, {}

    def errors(self) -> list:
        """Every sequence's DEVERR_* bits."""
        bits = self.err.cpu().tolist()
        if any(b & DEVERR_TIMEOUT for b in bits):
            for stream_ptr in self._ws:  # nothing of a call that gave up is used again
                _SCRATCH.pop((self.index, stream_ptr), None)
            self._ws.clear()
        return bits

    def workspace(self, Hq: int, max_new: int, stream_ptr: int) -> torch.Tensor:
        """Scratch of an attention call with zeroed counters, one per launch stream for the caches of all layers: calls on
        different streams may run at the same time.  A captured call gets its own from the graph's memory pool, its
        counters cleared in the graph by a fill in front of the kernel: replays of two graphs share nothing.  (Scratch
        of the caller's, zeroed once and kept for the graph, spares the fill.)"""
        n = self._ws_bytes.get((Hq, max_new))
        if n is None:
            n = int(_lib.hq_kv8_attn_workspace_bytes(self.ref, Hq, max_new))
            if n == 0:
                raise HqError(f"hq_kv8_attn: {Hq} query heads over {self.Hkv} kv heads, {max_new} new tokens")
            self._ws_bytes[(Hq, max_new)] = n
        capturing = torch._C._cuda_isCurrentStreamCapturing()
        w = None if capturing else _SCRATCH.get((self.index, stream_ptr))
        if w is None or w.numel() < n:
            w = torch.empty(n, dtype=torch.uint8, device=self.device)
            w[:KV8_WS_ZERO].zero_()
            if not capturing:
                _SCRATCH[(self.index, stream_ptr)] = w
        if not capturing:
            self._ws[stream_ptr] = w
        return w


def hq_kv8_append(cache: Kv8Cache, k, v, cu, kv_len, stream=None):
    """Append rows cu[b] .. cu[b+1]-1 of k, v [N, Hkv, D] (fp16 or bf16) to sequence b as its positions
    kv_len[b] - n_b .. kv_len[b] - 1; cu int32 [B+1], kv_len int32 [B] (new tokens included)."""
    dev = cache.index
    if stream is not None or _device() != dev:
        with _On(dev, stream):
            return hq_kv8_append(cache, k, v, cu, kv_len)
    _rows(k, dev, (None, cache.Hkv, cache.D), "k")
    _rows(v, dev, k.shape, "v", (k.dtype,))
    _ints(cu, dev, (cache.B + 1,), "cu")
    _ints(kv_len, dev, (cache.B,), "kv_len")
    ks, vs = k.stride(), v.stride()
    st = _lib.hq_kv8_append(cache.ref, _DTYPE[k.dtype], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                            k.shape[0], cu.data_ptr(), kv_len.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "hq_kv8_append")


def hq_kv8_read(cache: Kv8Cache, kv_len, start: int = 0, n: int = None, dtype=torch.float16, k_out=None, v_out=None,
                zero_rest: bool = True, stream=None):
    """Positions start .. start+n-1 (default: to the capacity) of every sequence, dequantised: (k, v), each
    [B, Hkv, n, D].  Rows at or past kv_len[b] are zeroed, or with zero_rest=False left as they are."""
    dev = cache.index
    if stream is not None or _device() != dev:
        with _On(dev, stream):
            return hq_kv8_read(cache, kv_len, start, n, dtype, k_out, v_out, zero_rest)
    if n is None:
        n = cache.cap - start
    _ints(kv_len, dev, (cache.B,), "kv_len")
    if k_out is None and v_out is None:
        if not zero_rest:
            raise HqError("hq_kv8_read: zero_rest=False needs k_out, v_out")
        if n < 0 or dtype not in _DTYPE:
            raise HqError(f"hq_kv8_read: {n} positions of {dtype}")
        k_out = torch.empty((cache.B, cache.Hkv, n, cache.D), dtype=dtype, device=cache.device)
        v_out = torch.empty_like(k_out)
    elif k_out is None or v_out is None:
        raise HqError("hq_kv8_read: give both of k_out, v_out or neither")
    else:
        _rows(k_out, dev, (cache.B, cache.Hkv, n, cache.D), "k_out", _ALL)
        _rows(v_out, dev, k_out.shape, "v_out", (k_out.dtype,))
        if k_out.stride() != v_out.stride():
            raise HqError("hq_kv8_read: k_out and v_out need the same strides")
        _output("hq_kv8_read", k_out, "k_out", "v_out", v_out)
    os_ = k_out.stride()
    st = _lib.hq_kv8_read(cache.ref, _DTYPE[k_out.dtype], kv_len.data_ptr(), start, n, k_out.data_ptr(), v_out.data_ptr(),
                          os_[0], os_[1], os_[2], 1 if zero_rest else 0, _raw_stream(dev))
    if st:
        _check(st, "hq_kv8_read")
    return k_out, v_out


def hq_kv8_attn(cache: Kv8Cache, q, cu, kv_len, max_new: int, sm_scale: float = None, window: int = 0, out=None,
                lse=None, return_lse: bool = False, ws=None, stream=None):
    """Attention of the newest tokens (appended before): q [N, Hq, D] holds sequence b's queries as rows
    cu[b] .. cu[b+1]-1, at most max_new of them, at its last positions; causal, with window > 0 over that many
    positions.  Returns out [N, Hq, D] (``out`` must not overlap q), with return_lse (out, lse float [N, Hq], base 2).
    ``ws``: scratch of the caller's (hq_kv8_attn_workspace_bytes, its first KV8_WS_ZERO bytes zeroed once), in place of
    the stream's: not for two calls that can run at once, nor for two graphs that can."""
    dev = cache.index
    if stream is not None or _device() != dev:
        with _On(dev, stream):
            return hq_kv8_attn(cache, q, cu, kv_len, max_new, sm_scale, window, out, lse, return_lse, ws)
    _rows(q, dev, (None, None, cache.D), "q")
    _ints(cu, dev, (cache.B + 1,), "cu")
    _ints(kv_len, dev, (cache.B,), "kv_len")
    N, Hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty_like(q)
    else:
        _rows(out, dev, q.shape, "out", (q.dtype,))
        _output("hq_kv8_attn", out, "out", "q", q)
    if lse is None:
        if return_lse:
            lse = q.new_empty((N, Hq), dtype=torch.float32)
    else:
        _scratch(lse, dev, "lse", torch.float32, (N, Hq))
    s = _raw_stream(dev)
    if ws is None:
        ws = cache.workspace(Hq, max_new, s)
    else:
        _scratch(ws, dev, "ws")
    qs, os_ = q.stride(), out.stride()
    st = _lib.hq_kv8_attn(cache.ref, _DTYPE[q.dtype], q.data_ptr(), qs[0], qs[1], Hq, N, cu.data_ptr(), kv_len.data_ptr(),
                          max_new, window, cache.D ** -0.5 if sm_scale is None else sm_scale, out.data_ptr(), os_[0], os_[1],
                          None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes, s)
    if st:
        _check(st, "hq_kv8_attn")
    return (out, lse) if return_lse else out


def hq_diag_stream_read(buf, sink, ctas_per_sm: int = 2, stream=None):
    """Read-only HBM streaming pass over a device tensor (measurement helper)."""
    _check(_lib.hq_diag_stream_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), ctas_per_sm,
                                    _stream(stream)), "hq_diag_stream_read")
