"""Python binding of libbeam.so (ctypes). Argument marshalling only: every step runs in the
library's CUDA kernels; torch supplies device memory and streams.

The functions carry the C names (beam_boundary_norm, beam_qkv_gate, beam_attn, beam_route,
beam_moe, beam_dense_mlp, ...) and take torch tensors. There is no fallback: if the library
is not built, or a call returns an error status, a BeamError is raised.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbeam.so")

BEAM_KV_BF16, BEAM_KV_FP8_E4M3 = 0, 1
BEAM_ATTN_SWA_ROPE, BEAM_ATTN_NOPE_SSMAX = 0, 1
BEAM_PAGED_BF16, BEAM_PAGED_FP8, BEAM_PAGED_NVFP4 = 0, 1, 2
DEV_BAD_POSITION, DEV_BAD_SEQ, DEV_BAD_EXPERT, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEV_BAD_PAGE = 0x10


class BeamError(RuntimeError):
    pass


class KVCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("num_seqs", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("window", ctypes.c_int32)]


class LayerCfgC(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_q", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("rope_theta", ctypes.c_float), ("ssmax_base", ctypes.c_float),
                ("ssmax_exp", ctypes.c_float), ("eps", ctypes.c_float),
                ("n_experts", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("d_ff_expert", ctypes.c_int32), ("d_ff_dense", ctypes.c_int32),
                ("route_scale", ctypes.c_float)]


class PagedKVC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("block_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("window", ctypes.c_int32)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_SIGS = {
    "beam_boundary_norm": [_P, _P, _P, _P, _P, _I, _I, _I, _F, _P],
    "beam_qkv_gate": [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _Z, _P],
    "beam_attn": [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _Z, _P],
    "beam_route": [_P, _P, _P, _P, _I, _P, _P, _P, _P, _Z, _P],
    "beam_moe": [_P, _P, _P, _P, _P, _P, _I, _P, _P, _Z, _P],
    "beam_moe_nvfp4": [_P, _P, _P, _P, _P, _I, _P, _P, _Z, _P],
    "beam_moe_fp8": [_P, _P, _P, _P, _P, _I, _P, _P, _Z, _P],
    "beam_dense_mlp": [_P, _P, _P, _P, _I, _P, _P, _Z, _P],
    "beam_workspace_bytes": [_P, _I, _I],
    "beam_kv_cache_bytes": [_I, _I, _I, _I, _I],
    "beam_get_device_status": [_P, ctypes.POINTER(ctypes.c_uint32)],
    "beam_status_string": [_I],
    "beam_launch_count": [],
    "beam_last_cuda_error": [],
    "beam_gemm_bf16": [_P, _I, _I, _I, _P, _I, _I, _P, _I, _I, _P],
    "beam_route_noalloc": [_P, _P, _P, _P, _I, _P, _P, _P],
    "beam_lm_head": [_P, _P, _I, _I, _I, _F, _P, _P],
    "beam_selftest_wait_timeout": [_P],
    "beam_paged_kv_write": [_P, _P, _I, _P, _P, _I, _P, _P],
    "beam_paged_kv_read": [_P, _P, _P, _P, _I, _I, _P, _P],
    "beam_paged_attn": [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _Z, _P],
    "beam_paged_workspace_bytes": [_P, _I, _I],
    "beam_paged_kv_bytes": [_I, _I, _I, _I, _I],
}
_RES = {"beam_workspace_bytes": _Z, "beam_kv_cache_bytes": _Z,
        "beam_paged_workspace_bytes": _Z, "beam_paged_kv_bytes": _Z,
        "beam_status_string": ctypes.c_char_p, "beam_launch_count": ctypes.c_uint64,
        "beam_last_cuda_error": ctypes.c_char_p}

_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise BeamError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() or "
                            "hybrid_attention_moe_gb300/build.py")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _RES.get(name, ctypes.c_int)
        _lib = L
    return _lib


def _check(status, what):
    if status != 0:
        msg = lib().beam_status_string(status).decode()
        if status == 3:
            msg += " [" + lib().beam_last_cuda_error().decode() + "]"
        raise BeamError(f"{what} failed: {msg} ({status})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclasses.dataclass
class LayerCfg:
    hidden: int
    n_q: int
    n_kv: int
    head_dim: int
    kind: int
    n_experts: int
    n_groups: int
    topk_groups: int
    topk: int
    d_ff_expert: int
    d_ff_dense: int
    rope_theta: float = 10000.0
    ssmax_base: float = 2048.0
    ssmax_exp: float = 0.1
    eps: float = 1e-6
    route_scale: float = 2.5

    @classmethod
    def from_shape(cls, shape, kind):
        return cls(hidden=shape.hidden, n_q=shape.n_q, n_kv=shape.n_kv,
                   head_dim=shape.head_dim, kind=kind, n_experts=shape.n_experts,
                   n_groups=shape.n_groups, topk_groups=shape.topk_groups, topk=shape.topk,
                   d_ff_expert=shape.d_ff_expert, d_ff_dense=shape.d_ff_dense,
                   rope_theta=shape.rope_theta, ssmax_base=shape.ssmax_base,
                   ssmax_exp=shape.ssmax_exp, eps=shape.eps, route_scale=shape.route_scale)

    def c(self):
        return LayerCfgC(self.hidden, self.n_q, self.n_kv, self.head_dim, self.kind,
                         self.rope_theta, self.ssmax_base, self.ssmax_exp, self.eps,
                         self.n_experts, self.n_groups, self.topk_groups, self.topk,
                         self.d_ff_expert, self.d_ff_dense, self.route_scale)

    def __setattr__(self, name, value):
        self.__dict__.pop("_kept", None)
        self.__dict__[name] = value

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_kept"}   # an address of this process

    def _ref(self):
        """Reference to a C struct of the present values, built again after a change."""
        kept = self.__dict__.get("_kept")
        if kept is None:
            kept = self.__dict__["_kept"] = ctypes.byref(self.c())
        return kept


@dataclasses.dataclass
class KVCache:
    """One layer's cache: k, v tensors [S][Hkv][capacity][D] (bf16, or uint8 e4m3 codes)."""
    k: torch.Tensor
    v: torch.Tensor
    window: int = 0
    k_scale: float = 1.0
    v_scale: float = 1.0

    @property
    def fp8(self):
        return self.k.dtype == torch.uint8

    def c(self):
        return KVCacheC(self.k.data_ptr(), self.v.data_ptr(),
                        BEAM_KV_FP8_E4M3 if self.fp8 else BEAM_KV_BF16, self.k_scale,
                        self.v_scale, self.k.shape[0], self.k.shape[2], self.window)


def _want(device, name, t, dtype, *shapes):
    """Refuses a tensor that the library would read as something else: another type or device,
    gaps between its elements, or none of the shapes (a number: any shape of so many elements)."""
    if (t.dtype != dtype or not t.is_contiguous() or t.get_device() != device or
            not (t.shape in shapes or t.numel() in shapes)):
        raise BeamError(f"{name}: contiguous {dtype} {' or '.join(map(str, shapes))} on cuda:{device} is wanted, "
                        f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _on_device(cache):
    """The cache's device, which has to be the current one: the library launches there."""
    dev = torch._C._cuda_getDevice()
    if cache.device != dev:
        raise BeamError(f"the cache is on cuda:{cache.device}, but the current device is cuda:{dev}")
    return dev


def _raw_stream(stream, device):
    """The handle of `stream`, or of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


class PagedKVCache:
    """One layer's pages (beam_paged_kv in include/beam.h).

    k, v        [num_pages][n_kv][page_size][D] bf16, or uint8 codes: [...][D] e4m3 (FP8), or
                [...][D/2] e2m1 pairs (NVFP4, recognised by its block_scale)
    page_table  [num_seqs][pages per sequence] int32
    row_scale   [num_pages][n_kv][2][page_size] uint8; None for bf16
    block_scale [num_pages][n_kv][2][page_size][D/16] uint8; NVFP4 only
    window      0 for full attention, else the sliding window
    The tensors are checked once, here, and must not be replaced afterwards (their contents may
    change, the page table's among them); the window may be set again."""

    page_size, num_pages = 256, 2 ** 31 - 1   # the largest; a cache holds its own

    @property
    def window(self):
        return self._window

    @window.setter
    def window(self, value):
        self._window = int(value)
        if "_c" in self.__dict__:   # what the kernels read
            self._c.window = self._window

    def __reduce__(self):
        """Copies and pickles by the tensors: the C struct holds addresses of this cache."""
        return (type(self), (self.k, self.v, self.page_table, self.row_scale, self.block_scale, self.window))

    @property
    def positions(self):
        """Positions that a sequence's row of the page table reaches."""
        return self.page_table.shape[1] * self.page_size

    def __init__(self, k, v, page_table, row_scale=None, block_scale=None, window=0):
        if k.dim() != 4 or page_table.dim() != 2:
            raise BeamError("PagedKVCache: k and v are [num_pages][n_kv][page_size][...], "
                            "page_table [num_seqs][pages]")
        pages, n_kv, size, width = k.shape
        code = torch.bfloat16 if row_scale is None else torch.uint8
        dev = k.get_device()
        _want(dev, "k", k, code, k.numel())
        _want(dev, "v", v, code, tuple(k.shape))
        _want(dev, "page_table", page_table, torch.int32, page_table.numel())
        self.dtype = BEAM_PAGED_BF16
        if row_scale is not None:
            _want(dev, "row_scale", row_scale, torch.uint8, (pages, n_kv, 2, size))
            self.dtype = BEAM_PAGED_FP8
        if block_scale is not None:
            if row_scale is None:
                raise BeamError("PagedKVCache: block_scale without row_scale")
            width *= 2
            _want(dev, "block_scale", block_scale, torch.uint8, (pages, n_kv, 2, size, width // 16))
            self.dtype = BEAM_PAGED_NVFP4
        if dev < 0:
            raise BeamError("PagedKVCache: the tensors must be on a CUDA device")
        self.k, self.v, self.page_table = k, v, page_table
        self.row_scale, self.block_scale, self.window = row_scale, block_scale, window
        self.num_pages, self.n_kv, self.page_size, self.head_dim = pages, n_kv, size, width
        self.device = dev
        self._c = PagedKVC(k.data_ptr(), v.data_ptr(),
                           0 if row_scale is None else row_scale.data_ptr(),
                           0 if block_scale is None else block_scale.data_ptr(),
                           page_table.data_ptr(), self.dtype, pages, size, n_kv, width,
                           page_table.shape[0], page_table.shape[1], self.window)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages, page_size, n_kv, head_dim, page_table, dtype=BEAM_PAGED_BF16,
              window=0):
        """Pages of zeros on the page table's device."""
        dev = page_table.device
        width = {BEAM_PAGED_BF16: head_dim, BEAM_PAGED_FP8: head_dim,
                 BEAM_PAGED_NVFP4: head_dim // 2}[dtype]
        kind = torch.bfloat16 if dtype == BEAM_PAGED_BF16 else torch.uint8
        dims = (num_pages, n_kv, page_size, width)
        row = block = None
        if dtype != BEAM_PAGED_BF16:
            row = torch.zeros((num_pages, n_kv, 2, page_size), dtype=torch.uint8, device=dev)
        if dtype == BEAM_PAGED_NVFP4:
            block = torch.zeros((num_pages, n_kv, 2, page_size, head_dim // 16),
                                dtype=torch.uint8, device=dev)
        return cls(torch.zeros(dims, dtype=kind, device=dev),
                   torch.zeros(dims, dtype=kind, device=dev), page_table, row, block, window)


def capturing():
    """Whether the current stream's work goes into a CUDA graph, which keeps its addresses."""
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


class Workspace:
    """Device scratch for the library calls, grown on demand (256-byte aligned). A buffer that a
    captured call got stays allocated for its replays when a larger one takes its place."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = None
        self.held = []

    def get(self, nbytes):
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        if capturing() and all(self.buf is not x for x in self.held):
            self.held.append(self.buf)
        return self.buf


def workspace_bytes(cfg: LayerCfg, T: int, max_pos: int) -> int:
    c = cfg.c()
    return lib().beam_workspace_bytes(ctypes.byref(c), T, max_pos)


def kv_cache_bytes(num_seqs, n_kv, capacity, head_dim, fp8=False) -> int:
    return lib().beam_kv_cache_bytes(num_seqs, n_kv, capacity, head_dim,
                                     BEAM_KV_FP8_E4M3 if fp8 else BEAM_KV_BF16)


def beam_boundary_norm(x, h, u_out, w_post, w_pre, n, eps, stream=None):
    T, H = h.shape
    _check(lib().beam_boundary_norm(_ptr(x), _ptr(h), _ptr(u_out), _ptr(w_post), _ptr(w_pre),
                                    T, H, n, eps, _stream(stream)), "beam_boundary_norm")


def beam_qkv_gate(cfg: LayerCfg, u, w_qkvg, q_norm_w, k_norm_w, seq_id, pos, q_out, g_out,
                  cache: KVCache, ws: torch.Tensor, stream=None):
    c, kc = cfg.c(), cache.c()
    _check(lib().beam_qkv_gate(ctypes.byref(c), _ptr(u), _ptr(w_qkvg), _ptr(q_norm_w),
                               _ptr(k_norm_w), _ptr(seq_id), _ptr(pos), u.shape[0], _ptr(q_out),
                               _ptr(g_out), ctypes.byref(kc), _ptr(ws), ws.numel(),
                               _stream(stream)), "beam_qkv_gate")


def beam_attn(cfg: LayerCfg, q, g, gate_bias, cache: KVCache, seq_id, pos, max_pos, w_o, out,
              ws: torch.Tensor, stream=None, max_q_per_seq=None):
    """max_q_per_seq: most tokens of one sequence in the call (1 for decode); None = T."""
    c, kc = cfg.c(), cache.c()
    mq = q.shape[0] if max_q_per_seq is None else int(max_q_per_seq)
    _check(lib().beam_attn(ctypes.byref(c), _ptr(q), _ptr(g), _ptr(gate_bias), ctypes.byref(kc),
                           _ptr(seq_id), _ptr(pos), q.shape[0], int(max_pos), max(1, mq),
                           _ptr(w_o), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "beam_attn")


def beam_route(cfg: LayerCfg, u, w_router, corr_bias, logits, topk_idx, topk_w,
               ws: torch.Tensor, stream=None):
    c = cfg.c()
    _check(lib().beam_route(ctypes.byref(c), _ptr(u), _ptr(w_router), _ptr(corr_bias),
                            u.shape[0], _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(ws),
                            ws.numel(), _stream(stream)), "beam_route")


def beam_moe(cfg: LayerCfg, u, topk_idx, topk_w, w_gate_up, w_down, out, ws: torch.Tensor,
             stream=None):
    c = cfg.c()
    _check(lib().beam_moe(ctypes.byref(c), _ptr(u), _ptr(topk_idx), _ptr(topk_w),
                          _ptr(w_gate_up), _ptr(w_down), u.shape[0], _ptr(out), _ptr(ws),
                          ws.numel(), _stream(stream)), "beam_moe")


def paged_workspace_bytes(cfg: LayerCfg, T: int, max_pos: int) -> int:
    c = cfg.c()
    return lib().beam_paged_workspace_bytes(ctypes.byref(c), T, max_pos)


def paged_kv_bytes(num_pages, n_kv, page_size, head_dim, dtype=BEAM_PAGED_BF16) -> int:
    return lib().beam_paged_kv_bytes(num_pages, n_kv, page_size, head_dim, dtype)


def beam_paged_kv_write(k, v, seq_id, pos, cache: PagedKVCache, stream=None):
    """k, v [T][n_kv][D] bf16 (rows of a token contiguous, any stride between tokens that is a
    multiple of 8; or [T][n_kv*D], contiguous) into the cache's pages."""
    dev, bf, i32 = _on_device(cache), torch.bfloat16, torch.int32
    n_kv, D = cache.n_kv, cache.head_dim
    T, step = k.size(0), n_kv * D
    # one test of everything for rows that lie side by side; others, and what is wrong, below
    if not (k.dtype is bf and (k.shape == (T, n_kv, D) or k.shape == (T, step)) and
            k.is_contiguous() and k.get_device() == dev and
            v.dtype is bf and v.shape == k.shape and v.is_contiguous() and v.get_device() == dev and
            seq_id.dtype is i32 and seq_id.numel() == T and seq_id.is_contiguous() and
            seq_id.get_device() == dev and pos.dtype is i32 and pos.numel() == T and
            pos.is_contiguous() and pos.get_device() == dev):
        _want(dev, "seq_id", seq_id, i32, T)
        _want(dev, "pos", pos, i32, T)
        for name, x in (("k", k), ("v", v)):
            if x.dtype != bf or x.shape != (T, n_kv, D) or x.get_device() != dev:
                raise BeamError(f"beam_paged_kv_write: {name} must be bfloat16 ({T}, {n_kv}, {D}) "
                                f"on cuda:{dev}, got {x.dtype} {tuple(x.shape)} on {x.device}")
            if T and (x.stride(2) != 1 or (n_kv > 1 and x.stride(1) != D)):
                raise BeamError(f"beam_paged_kv_write: the rows of a token of {name} must be "
                                f"contiguous, got strides {x.stride()}")
        if T > 1:
            step = k.stride(0)
            if v.stride(0) != step:
                raise BeamError("beam_paged_kv_write: k and v have different strides between tokens")
    st = lib().beam_paged_kv_write(k.data_ptr(), v.data_ptr(), step, seq_id.data_ptr(),
                                   pos.data_ptr(), T, cache._ref, _raw_stream(stream, dev))
    if st:
        _check(st, "beam_paged_kv_write")


def beam_paged_kv_read(cache: PagedKVCache, seq_id, first, last, max_len, dst: KVCache,
                       stream=None):
    """Positions first[i]..last[i] of sequence seq_id[i] into row i of the contiguous BF16 cache
    dst, slot (p-1) % capacity."""
    dev, i32, k, v = _on_device(cache), torch.int32, dst.k, dst.v
    N = seq_id.numel()
    rows, _, cap, _ = k.shape
    dims = (rows, cache.n_kv, cap, cache.head_dim)
    if not (seq_id.dtype is i32 and seq_id.is_contiguous() and seq_id.get_device() == dev and
            first.dtype is i32 and first.numel() == N and first.is_contiguous() and
            first.get_device() == dev and last.dtype is i32 and last.numel() == N and
            last.is_contiguous() and last.get_device() == dev and k.dtype is torch.bfloat16 and
            k.shape == dims and k.is_contiguous() and k.get_device() == dev and
            v.dtype is torch.bfloat16 and v.shape == dims and v.is_contiguous() and
            v.get_device() == dev):
        for name, x in (("seq_id", seq_id), ("first", first), ("last", last)):
            _want(dev, name, x, i32, N)
        for name, x in (("dst.k", k), ("dst.v", v)):
            _want(dev, name, x, torch.bfloat16, dims)
    kc = KVCacheC(k.data_ptr(), v.data_ptr(), BEAM_KV_BF16, 1.0, 1.0, rows, cap, dst.window)
    st = lib().beam_paged_kv_read(cache._ref, seq_id.data_ptr(), first.data_ptr(),
                                  last.data_ptr(), N, int(max_len), ctypes.byref(kc),
                                  _raw_stream(stream, dev))
    if st:
        _check(st, "beam_paged_kv_read")


def beam_paged_attn(cfg: LayerCfg, q, g, gate_bias, cache: PagedKVCache, seq_id, pos, max_pos,
                    w_o, out, ws: torch.Tensor, stream=None):
    """Decode attention over the pages. q, g [T][n_q][D] or [T][n_q*D]; g, gate_bias None: no gate;
    out [T][hidden], or of q's shapes where w_o is None."""
    dev, bf, i32 = _on_device(cache), torch.bfloat16, torch.int32
    T, n_q = q.size(0), cfg.n_q
    row = n_q * cfg.head_dim
    width = row if w_o is None else cfg.hidden
    heads, flat = (T, n_q, cfg.head_dim), (T, row)
    if (g is None) != (gate_bias is None):
        raise BeamError("beam_paged_attn: g and gate_bias go together")
    # one test of everything; what is wrong is looked for where it fails
    if not (q.dtype is bf and (q.shape == heads or q.shape == flat) and q.is_contiguous() and
            q.get_device() == dev and out.dtype is bf and
            (out.shape == (T, width) or (w_o is None and out.shape == heads)) and
            out.is_contiguous() and out.get_device() == dev and seq_id.dtype is i32 and seq_id.numel() == T and
            seq_id.is_contiguous() and seq_id.get_device() == dev and pos.dtype is i32 and
            pos.numel() == T and pos.is_contiguous() and pos.get_device() == dev and
            ws.is_contiguous() and ws.get_device() == dev):
        _want(dev, "q", q, bf, heads, flat)
        _want(dev, "out", out, bf, (T, width), *([heads] if w_o is None else []))
        _want(dev, "seq_id", seq_id, i32, T)
        _want(dev, "pos", pos, i32, T)
        _want(dev, "ws", ws, ws.dtype, ws.numel())
    pg = pb = pw = None
    if g is not None:
        if not (g.dtype is bf and (g.shape == flat or g.shape == heads) and g.is_contiguous() and
                g.get_device() == dev and gate_bias.dtype is bf and gate_bias.numel() == n_q and
                gate_bias.is_contiguous() and gate_bias.get_device() == dev):
            _want(dev, "g", g, bf, flat, heads)
            _want(dev, "gate_bias", gate_bias, bf, n_q)
        pg, pb = g.data_ptr(), gate_bias.data_ptr()
    if w_o is not None:
        _want(dev, "w_o", w_o, bf, (width, row))
        pw = w_o.data_ptr()
    st = lib().beam_paged_attn(cfg._ref(), q.data_ptr(), pg, pb, cache._ref, seq_id.data_ptr(),
                               pos.data_ptr(), T, int(max_pos), pw, out.data_ptr(), ws.data_ptr(),
                               ws.nbytes, _raw_stream(stream, dev))
    if st:
        _check(st, "beam_paged_attn")


class NvFp4ExpertsC(ctypes.Structure):
    _fields_ = [("gate_up", ctypes.c_void_p), ("gate_up_scale", ctypes.c_void_p),
                ("gate_up_global", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("down_scale", ctypes.c_void_p), ("down_global", ctypes.c_void_p)]


def beam_moe_nvfp4(cfg: LayerCfg, u, topk_idx, topk_w, experts: dict, out, ws: torch.Tensor,
                   stream=None):
    """experts: the tensors of synth.expert_weights_nvfp4 (gate_up, gate_up_scale,
    gate_up_global, down, down_scale, down_global)."""
    c = cfg.c()
    w = NvFp4ExpertsC(*[_ptr(experts[k]) for k in ("gate_up", "gate_up_scale", "gate_up_global",
                                                    "down", "down_scale", "down_global")])
    _check(lib().beam_moe_nvfp4(ctypes.byref(c), _ptr(u), _ptr(topk_idx), _ptr(topk_w),
                                ctypes.byref(w), u.shape[0], _ptr(out), _ptr(ws), ws.numel(),
                                _stream(stream)), "beam_moe_nvfp4")


class Fp8ExpertsC(ctypes.Structure):
    _fields_ = [("gate_up", ctypes.c_void_p), ("gate_up_scale", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("down_scale", ctypes.c_void_p)]


def beam_moe_fp8(cfg: LayerCfg, u, topk_idx, topk_w, experts: dict, out, ws: torch.Tensor,
                 stream=None):
    """experts: the tensors of synth.expert_weights_fp8 (gate_up, gate_up_scale, down,
    down_scale)."""
    c = cfg.c()
    w = Fp8ExpertsC(*[_ptr(experts[k]) for k in ("gate_up", "gate_up_scale", "down",
                                                  "down_scale")])
    _check(lib().beam_moe_fp8(ctypes.byref(c), _ptr(u), _ptr(topk_idx), _ptr(topk_w),
                              ctypes.byref(w), u.shape[0], _ptr(out), _ptr(ws), ws.numel(),
                              _stream(stream)), "beam_moe_fp8")


def beam_dense_mlp(cfg: LayerCfg, u, w_gate_up, w_down, out, ws: torch.Tensor, stream=None):
    c = cfg.c()
    _check(lib().beam_dense_mlp(ctypes.byref(c), _ptr(u), _ptr(w_gate_up), _ptr(w_down),
                                u.shape[0], _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "beam_dense_mlp")


def beam_get_device_status(stream=None) -> int:
    bits = ctypes.c_uint32(0)
    _check(lib().beam_get_device_status(_stream(stream), ctypes.byref(bits)),
           "beam_get_device_status")
    return bits.value


def beam_launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(lib().beam_launch_count())


def beam_gemm_bf16(a, b, c, stream=None):
    """c = a @ b.T with a [M][K], b [N][K] bf16 and c [M][N] float32 or bfloat16."""
    M, K = a.shape
    N = b.shape[0]
    _check(lib().beam_gemm_bf16(_ptr(a), M, K, a.stride(0), _ptr(b), N, b.stride(0), _ptr(c),
                                c.stride(0), int(c.dtype == torch.bfloat16), _stream(stream)),
           "beam_gemm_bf16")


def beam_lm_head(u, w_lm, logits, softcap=30.0, stream=None):
    """logits [T][V] fp32 = softcap * tanh((u w_lm^T) / softcap); u [T][H] bf16 (final-normed),
    w_lm [V][H] bf16; softcap <= 0: no cap."""
    T, H = u.shape
    V = w_lm.shape[0]
    _check(lib().beam_lm_head(_ptr(u), _ptr(w_lm), T, H, V, float(softcap), _ptr(logits),
                              _stream(stream)), "beam_lm_head")


def beam_route_noalloc(cfg: LayerCfg, u, w_router, corr_bias, topk_idx, topk_w, stream=None):
    """beam_route without caller scratch (the logits live in the library's static array)."""
    c = cfg.c()
    _check(lib().beam_route_noalloc(ctypes.byref(c), _ptr(u), _ptr(w_router), _ptr(corr_bias),
                                    u.shape[0], _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "beam_route_noalloc")


def beam_selftest_wait_timeout(stream=None):
    """Runs the library's bounded on-device wait against a barrier nothing completes (see
    include/beam.h); the status word then holds DEV_TIMEOUT."""
    _check(lib().beam_selftest_wait_timeout(_stream(stream)), "beam_selftest_wait_timeout")
