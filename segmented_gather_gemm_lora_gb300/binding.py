"""Thin Python binding of liblora_sgmv.so (the C ABI in include/lora_sgmv.h,
include/lora_pool.h, include/lora_train.h and include/lora_f8.h).

Argument marshalling only: every step of the LoRA path runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  There is
no fallback: if the library cannot be built or loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

import numpy as np
import torch

from . import build as _build

# ---------------------------------------------------------------- C structs --

LORA_OK = 0
LORA_ERR_INVALID_ARG = -1
LORA_ERR_UNSUPPORTED = -2
LORA_ERR_CUDA = -3
LORA_ERR_WORKSPACE = -4
LORA_DERR_BAD_ADAPTER = 1
LORA_DERR_BAD_PAGE = 2
LORA_DERR_BAD_RANK = 4
LORA_DERR_TIMEOUT = 8
LORA_MAX_RANK = 64
LORA_MAX_ADAPTERS = 32768
LORA_SHORT_MAX_TOKENS = 24
LORA_TILE_M = 128
LORA_BGMV_STATIC_ADAPTERS = 1
LORA_SEG_GROUP = 0
LORA_SEG_CONTIGUOUS = 1
LORA_FIXED_SCRATCH_MAX_TOKENS = 16384
LORA_MAX_PROJ = 4
LORA_DERR_BAD_LABEL = 16
LORA_DERR_BAD_SEQ = 32
LORA_DERR_NONFINITE = 64
LORA_LOGITS_BF16 = 0
LORA_LOGITS_F32 = 1
LORA_PREF_SIGMOID = 0
LORA_PREF_HINGE = 1
LORA_PREF_IPO = 2
LORA_PREF_AVERAGE = 1
LORA_STATE_F32 = 0
LORA_STATE_E4M3 = 1
LORA_ADAMW_BLOCK = 64
LORA_ADAMW_ZERO_GRAD = 1
LORA_TOPK_MAX = 256
LORA_DISTILL_FORWARD = 0
LORA_DISTILL_REVERSE = 1
LORA_DISTILL_JSD = 2
LORA_F8_E4M3 = 0
LORA_F8_E5M2 = 1
LORA_F8_FROM_BF16 = 0
LORA_F8_FROM_F32 = 1
LORA_F8_BLOCK = 128
LORA_F8_POW2 = 1

EXPORTED = (
    "lora_segments_buffer_bytes",
    "lora_segments_carve",
    "lora_segments_build",
    "lora_sgmv_shrink",
    "lora_sgmv_expand",
    "lora_apply",
    "lora_apply_f32y",
    "lora_apply_multi",
    "lora_sgmv_backward",
    "lora_apply_fixed_scratch",
    "lora_bgmv",
    "lora_bgmv_ex",
    "lora_base_apply",
    "lora_pool_pages_needed",
    "lora_status_string",
    "lora_abi_version",
    "lora_launch_count",
    "lora_debug_wait_probe",
    "lora_debug_gather_width",
    "lora_pool_mgr_create",
    "lora_pool_mgr_destroy",
    "lora_pool_mgr_page_list_len",
    "lora_pool_mgr_free_pages",
    "lora_pool_resident_rank",
    "lora_pool_pin",
    "lora_pool_unpin",
    "lora_pool_mgr_reserve",
    "lora_pool_mgr_release",
    "lora_pool_load",
    "lora_pool_evict",
    "lora_pool_mgr_stats",
    "lora_token_logprobs",
    "lora_preference_workspace_bytes",
    "lora_preference_loss",
    "lora_policy_loss",
    "lora_adamw_init",
    "lora_grad_sumsq_workspace_bytes",
    "lora_grad_sumsq",
    "lora_adamw_step",
    "lora_topk_logits",
    "lora_distill_loss",
    "lora_f8_quantize",
    "lora_base_f8",
    "lora_base_f8_backward",
)


class lora_adapter_desc_t(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("scale", ctypes.c_float),
                ("a_page0", ctypes.c_int32), ("b_page0", ctypes.c_int32)]


class lora_pool_view_t(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_list", ctypes.c_void_p), ("n_page_list", ctypes.c_int64),
                ("adapters", ctypes.c_void_p), ("n_adapters", ctypes.c_int32),
                ("page_elems", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32)]


class lora_proj_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("view", lora_pool_view_t)]


class lora_pool_stats_t(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_int64), ("loads", ctypes.c_int64), ("refused", ctypes.c_int64),
                ("evictions", ctypes.c_int64), ("pages_loaded", ctypes.c_int64),
                ("resident", ctypes.c_int32), ("pinned", ctypes.c_int32)]


class lora_segments_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("max_long_units", ctypes.c_int32),
                ("token_perm", ctypes.c_void_p), ("seg_indptr", ctypes.c_void_p),
                ("seg_adapter", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("short_units", ctypes.c_void_p), ("long_units", ctypes.c_void_p),
                ("scratch", ctypes.c_void_p), ("h_scratch", ctypes.c_void_p),
                ("k_partials", ctypes.c_void_p)]


class lora_pref_opts_t(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("flags", ctypes.c_uint32), ("beta", ctypes.c_float),
                ("label_smoothing", ctypes.c_float), ("margin", ctypes.c_float), ("grad_scale", ctypes.c_float)]


class lora_policy_opts_t(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("grad_scale", ctypes.c_float)]


class lora_train_proj_t(ctypes.Structure):
    _fields_ = [("view", lora_pool_view_t), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class lora_adamw_hyper_t(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int32), ("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("max_norm", ctypes.c_float), ("grad_scale", ctypes.c_float)]


class lora_distill_opts_t(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("temperature", ctypes.c_float), ("mix", ctypes.c_float),
                ("kd_weight", ctypes.c_float), ("ce_weight", ctypes.c_float), ("grad_scale", ctypes.c_float)]


class lora_f8_matrix_t(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("scale_row", ctypes.c_int64), ("scale_col", ctypes.c_int64), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("block_rows", ctypes.c_int32), ("type", ctypes.c_int32)]


class LoraError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))
        self.status = status


_lib = None


def lib():
    """The loaded library (built in-tree first if its sources are newer)."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.lora_launch_count.restype = ctypes.c_uint64
        L.lora_launch_count.argtypes = []
        L.lora_debug_wait_probe.restype = None
        L.lora_debug_wait_probe.argtypes = [ctypes.c_int64]
        L.lora_debug_gather_width.restype = ctypes.c_int32
        L.lora_debug_gather_width.argtypes = [ctypes.POINTER(lora_pool_view_t), ctypes.c_int32]
        L.lora_segments_buffer_bytes.restype = sz
        L.lora_segments_buffer_bytes.argtypes = [i32]
        L.lora_segments_carve.restype = i32
        L.lora_segments_carve.argtypes = [vp, sz, i32, ctypes.POINTER(lora_segments_t)]
        L.lora_segments_build.restype = i32
        L.lora_segments_build.argtypes = [vp, i32, i32, i32, ctypes.POINTER(lora_segments_t), vp, vp]
        seg_p = ctypes.POINTER(lora_segments_t)
        view_p = ctypes.POINTER(lora_pool_view_t)
        L.lora_sgmv_shrink.restype = i32
        L.lora_sgmv_shrink.argtypes = [vp, i64, vp, i64, seg_p, view_p, vp, vp]
        L.lora_sgmv_expand.restype = i32
        L.lora_sgmv_expand.argtypes = [vp, i64, vp, i64, seg_p, view_p, vp, vp]
        L.lora_apply.restype = i32
        L.lora_apply.argtypes = [vp, i64, vp, i64, seg_p, view_p, vp, vp]
        L.lora_apply_f32y.restype = i32
        L.lora_apply_f32y.argtypes = [vp, i64, vp, i64, vp, i64, seg_p, view_p, vp, vp]
        L.lora_sgmv_backward.restype = i32
        L.lora_sgmv_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i64, seg_p, view_p, vp, vp]
        L.lora_apply_multi.restype = i32
        L.lora_apply_multi.argtypes = [ctypes.POINTER(lora_proj_t), i32, seg_p, vp, vp]
        L.lora_apply_fixed_scratch.restype = i32
        L.lora_apply_fixed_scratch.argtypes = [vp, i64, vp, i64, seg_p, view_p, vp, vp]
        L.lora_bgmv.restype = i32
        L.lora_bgmv.argtypes = [vp, i64, vp, i64, vp, i32, view_p, vp, vp]
        L.lora_base_apply.restype = i32
        L.lora_base_apply.argtypes = [vp, i64, vp, i64, vp, i64, vp, seg_p, view_p, vp, vp]
        L.lora_bgmv_ex.restype = i32
        L.lora_bgmv_ex.argtypes = [vp, i64, vp, i64, vp, i32, view_p, ctypes.c_uint32, vp, vp]
        L.lora_pool_pages_needed.restype = i64
        L.lora_pool_pages_needed.argtypes = [i32, i32, i32, i32]
        L.lora_status_string.restype = ctypes.c_char_p
        L.lora_status_string.argtypes = [i32]
        L.lora_abi_version.restype = i32
        L.lora_abi_version.argtypes = []
        i32p = ctypes.POINTER(ctypes.c_int32)
        L.lora_pool_mgr_create.restype = i32
        L.lora_pool_mgr_create.argtypes = [i64, i32, i32, i32, i32, i32, ctypes.POINTER(vp)]
        L.lora_pool_mgr_destroy.restype = None
        L.lora_pool_mgr_destroy.argtypes = [vp]
        L.lora_pool_mgr_page_list_len.restype = i64
        L.lora_pool_mgr_page_list_len.argtypes = [vp]
        L.lora_pool_mgr_free_pages.restype = i64
        L.lora_pool_mgr_free_pages.argtypes = [vp]
        L.lora_pool_resident_rank.restype = i32
        L.lora_pool_resident_rank.argtypes = [vp, i32]
        L.lora_pool_pin.restype = i32
        L.lora_pool_pin.argtypes = [vp, i32]
        L.lora_pool_unpin.restype = i32
        L.lora_pool_unpin.argtypes = [vp, i32]
        L.lora_pool_mgr_reserve.restype = i32
        L.lora_pool_mgr_reserve.argtypes = [vp, i32, i32, i32p, i32, i32p, i32p, i32, i32p]
        L.lora_pool_mgr_release.restype = i32
        L.lora_pool_mgr_release.argtypes = [vp, i32]
        L.lora_pool_load.restype = i32
        L.lora_pool_load.argtypes = [vp, i32, i32, ctypes.c_float, vp, vp, view_p, vp]
        L.lora_pool_evict.restype = i32
        L.lora_pool_evict.argtypes = [vp, i32, view_p, vp]
        L.lora_pool_mgr_stats.restype = i32
        L.lora_pool_mgr_stats.argtypes = [vp, ctypes.POINTER(lora_pool_stats_t)]
        u32, proj_p = ctypes.c_uint32, ctypes.POINTER(lora_train_proj_t)
        L.lora_token_logprobs.restype = i32
        L.lora_token_logprobs.argtypes = [vp, i64, i32, vp, i32, i32, vp, vp, vp, vp]
        L.lora_preference_workspace_bytes.restype = sz
        L.lora_preference_workspace_bytes.argtypes = [i32, i32]
        L.lora_preference_loss.restype = i32
        L.lora_preference_loss.argtypes = [vp, i64, i32, vp, vp, vp, i32, i32, i32, ctypes.POINTER(lora_pref_opts_t),
                                           vp, vp, vp, i64, vp, sz, vp, vp]
        L.lora_policy_loss.restype = i32
        L.lora_policy_loss.argtypes = [vp, i64, i32, vp, vp, vp, vp, vp, i32, i32, ctypes.POINTER(lora_policy_opts_t),
                                       vp, vp, vp, vp, i64, vp, vp]
        L.lora_adamw_init.restype = i32
        L.lora_adamw_init.argtypes = [proj_p, i32, i32, vp, i32, vp, vp]
        L.lora_grad_sumsq_workspace_bytes.restype = sz
        L.lora_grad_sumsq_workspace_bytes.argtypes = [proj_p, i32, i32]
        L.lora_grad_sumsq.restype = i32
        L.lora_grad_sumsq.argtypes = [proj_p, i32, vp, i32, i32, vp, vp, sz, vp, vp]
        L.lora_adamw_step.restype = i32
        L.lora_adamw_step.argtypes = [proj_p, i32, i32, vp, i32, vp, vp, u32, vp, vp]
        L.lora_topk_logits.restype = i32
        L.lora_topk_logits.argtypes = [vp, i64, i32, vp, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp]
        L.lora_distill_loss.restype = i32
        L.lora_distill_loss.argtypes = [vp, i64, i32, vp, vp, vp, i32, vp, vp, i32, i32,
                                        ctypes.POINTER(lora_distill_opts_t), vp, vp, vp, vp, i64, vp, vp]
        f8_p = ctypes.POINTER(lora_f8_matrix_t)
        L.lora_f8_quantize.restype = i32
        L.lora_f8_quantize.argtypes = [vp, i64, i32, f8_p, u32, vp, vp]
        for f in (L.lora_base_f8, L.lora_base_f8_backward):
            f.restype = i32
            f.argtypes = [f8_p, f8_p, vp, i64, i32, vp, vp]
        _lib = L
    return _lib


def library_path() -> str:
    return _build.LIB


def status_string(status: int) -> str:
    return lib().lora_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != LORA_OK:
        raise LoraError(status, what)


def _handle(stream) -> int:
    """A stream's handle as a plain integer."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _stream(stream) -> ctypes.c_void_p:
    return ctypes.c_void_p(_handle(stream))


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    return int(t.stride(0))


# ------------------------------------------------------------ device views --

class PoolView:
    """A projection's paged adapter pool on the device plus its C view."""

    def __init__(self, pool: torch.Tensor, page_list: torch.Tensor, adapters: torch.Tensor,
                 page_elems: int, max_rank: int, d_in: int, d_out: int):
        self.pool = pool  # bf16 (or int16 bits) [n_pages, page_elems]
        self.page_list = page_list  # int32
        self.adapters = adapters  # uint8 [n_adapters * 16] or int32 [n_adapters, 4]
        self.c = lora_pool_view_t(
            pool.data_ptr(), pool.numel() // page_elems, page_list.data_ptr(), page_list.numel(),
            adapters.data_ptr(), adapters.numel() * adapters.element_size() // 16, page_elems,
            max_rank, d_in, d_out)

    @classmethod
    def from_host(cls, host_pool, device="cuda"):
        """Upload a workloads.AdapterPool."""
        pool = torch.from_numpy(host_pool.pool.view(np.int16)).to(device).view(torch.bfloat16)
        pl = torch.from_numpy(np.ascontiguousarray(host_pool.page_list, dtype=np.int32)).to(device)
        desc = torch.from_numpy(np.ascontiguousarray(host_pool.desc).view(np.uint8)).to(device)
        return cls(pool, pl, desc, host_pool.page_elems, host_pool.max_rank, host_pool.d_in,
                   host_pool.d_out)

    @property
    def d_in(self):
        return self.c.d_in

    @property
    def d_out(self):
        return self.c.d_out


class Segments:
    """A device buffer carved into the segment arrays for T tokens."""

    def __init__(self, T: int, device="cuda"):
        nbytes = int(lib().lora_segments_buffer_bytes(T))
        self.buf = torch.zeros(max(nbytes, 16) // 4 + 4, dtype=torch.int32, device=device)
        self.c = lora_segments_t()
        _check(lib().lora_segments_carve(_ptr(self.buf), self.buf.numel() * 4, T, ctypes.byref(self.c)),
               "lora_segments_carve")
        self.T = T

    def _view(self, ptr_field: str, n: int) -> torch.Tensor:
        off = (getattr(self.c, ptr_field) - self.buf.data_ptr()) // 4
        return self.buf[off: off + n]

    @property
    def meta(self) -> torch.Tensor:
        return self._view("meta", 8)

    def host(self):
        """(perm, indptr, seg_adapter, n_tokens, short_units, long_units [n, 2]) on the host."""
        meta = self.meta.cpu().numpy()
        n_segs, n_tok, n_short, n_long = (int(v) for v in meta[:4])
        perm = self._view("token_perm", n_tok).cpu().numpy()
        indptr = self._view("seg_indptr", n_segs + 1).cpu().numpy()
        seg_ad = self._view("seg_adapter", n_segs).cpu().numpy()
        short = self._view("short_units", n_short).cpu().numpy()
        long_ = self._view("long_units", 2 * n_long).cpu().numpy().reshape(-1, 2)
        return perm, indptr, seg_ad, n_tok, short, long_


# ------------------------------------------------------------ entry points --

def lora_segments_buffer_bytes(T: int) -> int:
    return int(lib().lora_segments_buffer_bytes(T))


def lora_pool_pages_needed(rank: int, d_in: int, d_out: int, page_elems: int) -> int:
    return int(lib().lora_pool_pages_needed(rank, d_in, d_out, page_elems))


def lora_status_string(status: int) -> str:
    return status_string(status)


def lora_abi_version() -> int:
    return int(lib().lora_abi_version())


def lora_segments_build(token_adapter: torch.Tensor, n_adapters: int, seg: Segments,
                        mode: int = LORA_SEG_GROUP, err: Optional[torch.Tensor] = None, stream=None):
    T = int(token_adapter.numel())
    _check(lib().lora_segments_build(_ptr(token_adapter), T, n_adapters, mode, ctypes.byref(seg.c),
                                     _ptr(err), _stream(stream)), "lora_segments_build")


def lora_sgmv_shrink(x: torch.Tensor, h: torch.Tensor, seg: Segments, view: PoolView,
                     err: Optional[torch.Tensor] = None, stream=None):
    _check(lib().lora_sgmv_shrink(_ptr(x), _ld(x), _ptr(h), _ld(h), ctypes.byref(seg.c),
                                  ctypes.byref(view.c), _ptr(err), _stream(stream)),
           "lora_sgmv_shrink")


def lora_sgmv_expand(h: torch.Tensor, y: torch.Tensor, seg: Segments, view: PoolView,
                     err: Optional[torch.Tensor] = None, stream=None):
    _check(lib().lora_sgmv_expand(_ptr(h), _ld(h), _ptr(y), _ld(y), ctypes.byref(seg.c),
                                  ctypes.byref(view.c), _ptr(err), _stream(stream)),
           "lora_sgmv_expand")


def lora_apply(x: torch.Tensor, y: torch.Tensor, seg: Segments, view: PoolView,
               err: Optional[torch.Tensor] = None, stream=None):
    _check(lib().lora_apply(_ptr(x), _ld(x), _ptr(y), _ld(y), ctypes.byref(seg.c),
                            ctypes.byref(view.c), _ptr(err), _stream(stream)), "lora_apply")


def lora_apply_f32y(x: torch.Tensor, y0: torch.Tensor, yf: torch.Tensor, seg: Segments, view: PoolView,
                    err: Optional[torch.Tensor] = None, stream=None):
    """lora_apply with the result written as fp32 into yf (y0 bf16 is only read)."""
    _check(lib().lora_apply_f32y(_ptr(x), _ld(x), _ptr(y0), _ld(y0), _ptr(yf), _ld(yf),
                                 ctypes.byref(seg.c), ctypes.byref(view.c), _ptr(err), _stream(stream)),
           "lora_apply_f32y")


def lora_apply_multi(calls, seg: Segments, err: Optional[torch.Tensor] = None, stream=None):
    """Several projections on one batch in one grouped call: `calls` is a list of
    (x, y, view) with the same d_in; projections may share x."""
    arr = (lora_proj_t * len(calls))()
    for i, (x, y, view) in enumerate(calls):
        arr[i].x = _ptr(x).value
        arr[i].ldx = _ld(x)
        arr[i].y = _ptr(y).value
        arr[i].ldy = _ld(y)
        arr[i].view = view.c
    _check(lib().lora_apply_multi(arr, len(calls), ctypes.byref(seg.c), _ptr(err), _stream(stream)),
           "lora_apply_multi")


def lora_sgmv_backward(x: torch.Tensor, dy: torch.Tensor, dx: Optional[torch.Tensor], grad_pool: torch.Tensor,
                       hu: torch.Tensor, seg: Segments, view: PoolView, err: Optional[torch.Tensor] = None,
                       stream=None):
    """Adapter gradients: dA_i, dB_i added into grad_pool (fp32, the pool's page layout),
    dx += the adapter path's contribution (bf16 in place, or None).  hu: fp32 workspace
    [2 * T, ldh]."""
    ldh = _ld(hu)
    _check(lib().lora_sgmv_backward(_ptr(x), _ld(x), _ptr(dy), _ld(dy), _ptr(dx), _ld(dx) if dx is not None else 0,
                                    _ptr(grad_pool), _ptr(hu), ldh, ctypes.byref(seg.c), ctypes.byref(view.c),
                                    _ptr(err), _stream(stream)), "lora_sgmv_backward")


def apply_kernel_names():
    """Names of the kernels one lora_apply call may launch, in launch order."""
    return ["gather_kernel", "fused_tc_kernel"]


def lora_apply_fixed_scratch(x: torch.Tensor, y: torch.Tensor, seg: Segments, view: PoolView,
                             err: Optional[torch.Tensor] = None, stream=None):
    """lora_apply with its intermediate in the library's fixed device array: for callers
    that cannot allocate a workspace (see include/lora_sgmv.h).  Calls that may overlap on
    the GPU share that array and must be serialised by the caller."""
    _check(lib().lora_apply_fixed_scratch(_ptr(x), _ld(x), _ptr(y), _ld(y), ctypes.byref(seg.c),
                                          ctypes.byref(view.c), _ptr(err), _stream(stream)),
           "lora_apply_fixed_scratch")


def debug_wait_probe(cycles: int) -> None:
    """Test-only: arm (cycles > 0) or disarm the kernels' timeout probe."""
    lib().lora_debug_wait_probe(int(cycles))


def debug_gather_width(shapes) -> int:
    """Test-only, host only: the gather kernel's cluster width for a call over projections
    of the given (d_in, d_out) shapes, before the launcher's occupancy narrowing."""
    arr = (lora_pool_view_t * max(1, len(shapes)))()
    for i, (d_in, d_out) in enumerate(shapes):
        arr[i].d_in, arr[i].d_out = int(d_in), int(d_out)
    return int(lib().lora_debug_gather_width(arr, len(shapes)))


def launch_count() -> int:
    """Kernels the library has launched in this process (a recorded graph counts once)."""
    return int(lib().lora_launch_count())


def lora_base_apply(x: torch.Tensor, w0: torch.Tensor, y: torch.Tensor, token_adapter: torch.Tensor, seg: Segments,
                    view: PoolView, err: Optional[torch.Tensor] = None, stream=None):
    """y = bf16(x W0^T + s_i (x A_i^T) B_i), y written only; w0 bf16 [d_out, ldw >= d_in]."""
    _check(lib().lora_base_apply(_ptr(x), _ld(x), _ptr(w0), _ld(w0), _ptr(y), _ld(y), _ptr(token_adapter),
                                 ctypes.byref(seg.c), ctypes.byref(view.c), _ptr(err), _stream(stream)),
           "lora_base_apply")


def lora_bgmv(x: torch.Tensor, y: torch.Tensor, token_adapter: torch.Tensor, view: PoolView,
              err: Optional[torch.Tensor] = None, stream=None, static_adapters: bool = False):
    """static_adapters: lora_bgmv_ex with LORA_BGMV_STATIC_ADAPTERS (see include/lora_sgmv.h)."""
    T = int(token_adapter.numel())
    if static_adapters:
        _check(lib().lora_bgmv_ex(_ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(token_adapter), T, ctypes.byref(view.c),
                                  LORA_BGMV_STATIC_ADAPTERS, _ptr(err), _stream(stream)), "lora_bgmv_ex")
    else:
        _check(lib().lora_bgmv(_ptr(x), _ld(x), _ptr(y), _ld(y), _ptr(token_adapter), T,
                               ctypes.byref(view.c), _ptr(err), _stream(stream)), "lora_bgmv")



# ---------------------------------------------------------- pool residency --

def _host_bits(m, rows: int, cols: int) -> tuple:
    """(pointer, owner) of a host bf16 matrix [rows, cols]: a contiguous CPU tensor of
    bfloat16 / int16 / uint16 or a numpy uint16 / int16 array."""
    if isinstance(m, torch.Tensor):
        if m.device.type != "cpu" or m.element_size() != 2 or not m.is_contiguous():
            raise ValueError("expected a contiguous 2-byte CPU tensor")
        if m.numel() != rows * cols:
            raise ValueError("expected %d x %d elements" % (rows, cols))
        return ctypes.c_void_p(m.data_ptr()), m
    a = np.ascontiguousarray(m)
    if a.dtype.itemsize != 2 or a.size != rows * cols:
        raise ValueError("expected a %d x %d array of 2-byte elements" % (rows, cols))
    return ctypes.c_void_p(a.ctypes.data), a


def lora_pool_mgr_create(n_pages: int, page_elems: int, n_adapters: int, max_rank: int,
                         d_in: int, d_out: int) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(lib().lora_pool_mgr_create(n_pages, page_elems, n_adapters, max_rank, d_in, d_out,
                                      ctypes.byref(h)), "lora_pool_mgr_create")
    return h


def lora_pool_mgr_destroy(mgr: ctypes.c_void_p) -> None:
    lib().lora_pool_mgr_destroy(mgr)


def lora_pool_mgr_page_list_len(mgr) -> int:
    return int(lib().lora_pool_mgr_page_list_len(mgr))


def lora_pool_mgr_free_pages(mgr) -> int:
    return int(lib().lora_pool_mgr_free_pages(mgr))


def lora_pool_resident_rank(mgr, adapter: int) -> int:
    return int(lib().lora_pool_resident_rank(mgr, adapter))


def lora_pool_pin(mgr, adapter: int) -> None:
    _check(lib().lora_pool_pin(mgr, adapter), "lora_pool_pin")


def lora_pool_unpin(mgr, adapter: int) -> None:
    _check(lib().lora_pool_unpin(mgr, adapter), "lora_pool_unpin")


def lora_pool_mgr_reserve(mgr, adapter: int, rank: int, pages_cap: int, evicted_cap: int):
    """(pages, evicted) as int32 arrays: the pages the adapter now holds (empty if it was
    already resident with this rank) and the adapters evicted for them, in order."""
    pages = (ctypes.c_int32 * max(1, pages_cap))()
    evicted = (ctypes.c_int32 * max(1, evicted_cap))()
    n_p, n_e = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().lora_pool_mgr_reserve(mgr, adapter, rank, pages, pages_cap, ctypes.byref(n_p), evicted,
                                       evicted_cap, ctypes.byref(n_e)), "lora_pool_mgr_reserve")
    return (np.frombuffer(pages, dtype=np.int32)[: n_p.value].copy(),
            np.frombuffer(evicted, dtype=np.int32)[: n_e.value].copy())


def lora_pool_mgr_release(mgr, adapter: int) -> None:
    _check(lib().lora_pool_mgr_release(mgr, adapter), "lora_pool_mgr_release")


def lora_pool_load(mgr, adapter: int, rank: int, scale: float, A, B, view: PoolView, stream=None):
    """A: host bf16 [rank, d_in], B: host bf16 [rank, d_out] (tensors or uint16 arrays).  A
    pinned tensor is copied asynchronously: keep it unchanged until the stream passes."""
    pa, _ = _host_bits(A, rank, view.d_in)
    pb, _ = _host_bits(B, rank, view.d_out)
    _check(lib().lora_pool_load(mgr, adapter, rank, float(scale), pa, pb, ctypes.byref(view.c),
                                _stream(stream)), "lora_pool_load")


def lora_pool_mgr_stats(mgr) -> dict:
    st = lora_pool_stats_t()
    _check(lib().lora_pool_mgr_stats(mgr, ctypes.byref(st)), "lora_pool_mgr_stats")
    return {name: int(getattr(st, name)) for name, _ in lora_pool_stats_t._fields_}


def lora_pool_evict(mgr, adapter: int, view: PoolView, stream=None) -> None:
    _check(lib().lora_pool_evict(mgr, adapter, ctypes.byref(view.c), _stream(stream)), "lora_pool_evict")


class PoolManager:
    """One projection's pool residency (include/lora_pool.h): a host-side manager plus,
    from device_view(), the device pool, page list and descriptors it fills."""

    def __init__(self, n_pages: int, page_elems: int, n_adapters: int, max_rank: int,
                 d_in: int, d_out: int):
        self.h = lora_pool_mgr_create(n_pages, page_elems, n_adapters, max_rank, d_in, d_out)
        self.n_pages, self.page_elems, self.n_adapters = n_pages, page_elems, n_adapters
        self.max_rank, self.d_in, self.d_out = max_rank, d_in, d_out

    def close(self):
        if self.h is not None and self.h.value:
            lora_pool_mgr_destroy(self.h)
        self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def page_list_len(self) -> int:
        return lora_pool_mgr_page_list_len(self.h)

    @property
    def slots_per_adapter(self) -> int:
        return self.page_list_len // self.n_adapters

    @property
    def free_pages(self) -> int:
        return lora_pool_mgr_free_pages(self.h)

    def stats(self) -> dict:
        """hits, loads, refused, evictions, pages_loaded, resident, pinned."""
        return lora_pool_mgr_stats(self.h)

    def resident_rank(self, adapter: int) -> int:
        return lora_pool_resident_rank(self.h, adapter)

    def pin(self, adapter: int):
        lora_pool_pin(self.h, adapter)

    def unpin(self, adapter: int):
        lora_pool_unpin(self.h, adapter)

    def reserve(self, adapter: int, rank: int):
        return lora_pool_mgr_reserve(self.h, adapter, rank, self.slots_per_adapter, self.n_adapters)

    def release(self, adapter: int):
        lora_pool_mgr_release(self.h, adapter)

    def device_view(self, device="cuda") -> PoolView:
        """A zeroed device pool, page list and descriptor array of this manager's geometry."""
        pool = torch.zeros(self.n_pages, self.page_elems, dtype=torch.bfloat16, device=device)
        pl = torch.zeros(self.page_list_len, dtype=torch.int32, device=device)
        desc = torch.zeros(self.n_adapters * 16, dtype=torch.uint8, device=device)
        return PoolView(pool, pl, desc, self.page_elems, self.max_rank, self.d_in, self.d_out)

    def load(self, adapter: int, rank: int, scale: float, A, B, view: PoolView, stream=None):
        lora_pool_load(self.h, adapter, rank, scale, A, B, view, stream)

    def evict(self, adapter: int, view: PoolView, stream=None):
        lora_pool_evict(self.h, adapter, view, stream)


# ------------------------------------------------- training: losses on logits --

def _logits(t: torch.Tensor):
    """(address, row stride, dtype code, T, V) of a [T, V] matrix of logits."""
    code = _LOGITS_CODE.get(t.dtype)
    if code is None:
        raise ValueError("expected bfloat16 or float32 logits")
    T, V = t.shape
    ld, one = t.stride()
    if one != 1 and V > 1:
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    if T <= 1:
        ld = max(ld, V)  # the stride of a matrix of one row says nothing
    elif ld < V:
        raise ValueError("expected rows that do not overlap (a row stride of at least %d, got %d)" % (V, ld))
    return t.data_ptr(), ld, code, T, V


_LOGITS_CODE = {torch.bfloat16: LORA_LOGITS_BF16, torch.float32: LORA_LOGITS_F32}


def _rows(t: Optional[torch.Tensor], n: int, dtype, what: str) -> int:
    """Address of a contiguous vector of n elements of a type, 0 of none.  (Addresses as plain
    integers: these calls are short, and a ctypes object for each argument costs as much as a check.)"""
    if t is None:
        return 0
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected %d contiguous elements of %s" % (what, n, dtype))
    return t.data_ptr()


@functools.lru_cache(maxsize=64)
def _opts(kind, *values):
    """A structure of options by reference: a training run passes the same few again and again.
    Plain numbers only, which are their own key: a tensor's is its identity, not its value."""
    return ctypes.byref(kind(*values))


def _addr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _grad_of(logits: torch.Tensor, dlogits: Optional[torch.Tensor]):
    if dlogits is None:
        return 0, 0
    if dlogits is not logits and (dlogits.shape != logits.shape or dlogits.dtype is not logits.dtype):
        raise ValueError("dlogits: expected the shape and type of the logits")
    return _logits(dlogits)[:2]


def lora_token_logprobs(logits: torch.Tensor, labels: torch.Tensor, logp: torch.Tensor,
                        lse: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None):
    """logp[t] = logits[t, labels[t]] - lse[t]; logits [T, V] bf16 or fp32, labels int32 [T] (< 0: not counted)."""
    p, ld, code, T, V = _logits(logits)
    f32 = torch.float32
    _check(lib().lora_token_logprobs(p, ld, code, _rows(labels, T, torch.int32, "labels"), T, V,
                                     _rows(logp, T, f32, "logp"), _rows(lse, T, f32, "lse"), _addr(err),
                                     _handle(stream)), "lora_token_logprobs")


def preference_workspace(T: int, n_pairs: int, device="cuda") -> torch.Tensor:
    """A workspace for lora_preference_loss over T rows and n_pairs pairs."""
    return torch.empty(int(lib().lora_preference_workspace_bytes(T, n_pairs)), dtype=torch.uint8, device=device)


def lora_preference_loss(logits: torch.Tensor, labels: torch.Tensor, seq_indptr: torch.Tensor, loss: torch.Tensor,
                         seq_logp: Optional[torch.Tensor], dlogits: Optional[torch.Tensor], workspace: torch.Tensor,
                         ref_logp: Optional[torch.Tensor] = None, kind: int = LORA_PREF_SIGMOID, beta: float = 0.1,
                         label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                         grad_scale: float = 1.0, err: Optional[torch.Tensor] = None, stream=None):
    """Paired preference loss and its gradient (see include/lora_train.h): sequence s is rows
    seq_indptr[s] .. seq_indptr[s + 1], pair p sequences 2p (chosen) and 2p + 1 (rejected).
    dlogits may be the logits (the gradient takes their place) or None."""
    p, ld, code, T, V = _logits(logits)
    n = int(loss.numel())
    f32 = torch.float32
    opts = _opts(lora_pref_opts_t, int(kind), LORA_PREF_AVERAGE if average else 0, float(beta), float(label_smoothing),
                 float(margin), float(grad_scale))
    dp, ldd = _grad_of(logits, dlogits)
    _check(lib().lora_preference_loss(p, ld, code, _rows(labels, T, torch.int32, "labels"),
                                      _rows(ref_logp, T, f32, "ref_logp"),
                                      _rows(seq_indptr, 2 * n + 1, torch.int32, "seq_indptr"), n, T, V,
                                      opts, _rows(loss, n, f32, "loss"),
                                      _rows(seq_logp, 2 * n, f32, "seq_logp"), dp, ldd, _addr(workspace),
                                      workspace.nbytes, _addr(err), _handle(stream)),
           "lora_preference_loss")


def lora_policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                     logp: torch.Tensor, loss: torch.Tensor, kl: Optional[torch.Tensor],
                     dlogits: Optional[torch.Tensor], ref_logp: Optional[torch.Tensor] = None,
                     weight: Optional[torch.Tensor] = None, clip_low: float = 0.2, clip_high: float = 0.2,
                     kl_coef: float = 0.0, grad_scale: float = 1.0, err: Optional[torch.Tensor] = None, stream=None):
    """Clipped policy loss with a KL term, per row, and its gradient (see include/lora_train.h).
    dlogits may be the logits (the gradient takes their place) or None."""
    p, ld, code, T, V = _logits(logits)
    f32 = torch.float32
    opts = _opts(lora_policy_opts_t, float(clip_low), float(clip_high), float(kl_coef), float(grad_scale))
    dp, ldd = _grad_of(logits, dlogits)
    _check(lib().lora_policy_loss(p, ld, code, _rows(labels, T, torch.int32, "labels"),
                                  _rows(old_logp, T, f32, "old_logp"), _rows(ref_logp, T, f32, "ref_logp"),
                                  _rows(advantage, T, f32, "advantage"), _rows(weight, T, f32, "weight"), T, V,
                                  opts, _rows(logp, T, f32, "logp"), _rows(loss, T, f32, "loss"),
                                  _rows(kl, T, f32, "kl"), dp, ldd, _addr(err), _handle(stream)), "lora_policy_loss")


def _one_device(stream, first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The stream's handle.  Refuses tensors that do not all lie on the current CUDA device, and a stream of another one:
    the library launches on the current device, and would read their addresses there."""
    d = first.get_device()
    if d < 0:
        raise ValueError("expected tensors on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("expected tensors on one CUDA device")
    if d != torch._C._cuda_getDevice():
        raise ValueError("expected tensors on the current CUDA device (%d)" % torch.cuda.current_device())
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(d)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != d:
        raise ValueError("expected a stream of the tensors' device")
    return _handle(stream)


def _err_word(err: Optional[torch.Tensor]) -> int:
    if err is None:
        return 0
    if err.dtype is not torch.int32 or err.numel() < 1:
        raise ValueError("err: expected an element of torch.int32")
    return err.data_ptr()


def lora_topk_logits(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, tail: Optional[torch.Tensor] = None,
                     temperature: float = 1.0, labels: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                     stream=None):
    """The k largest logits of each row, largest first (ids int32 and values fp32 [T, k]; equal ones by rising
    index), and tail[t] = log of the sum of exp(logit / temperature) over the others.  labels int32 [T]: rows with a
    negative label list nothing.  See include/lora_train.h."""
    handle = _one_device(stream, logits, ids, values, tail, labels, err)
    p, ld, code, T, V = _logits(logits)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError("ids: expected a row for each row of logits")
    k = ids.shape[1]
    i32, f32 = torch.int32, torch.float32
    _check(lib().lora_topk_logits(p, ld, code, _rows(labels, T, i32, "labels"), T, V, k, float(temperature),
                                  _rows(ids, T * k, i32, "ids"), _rows(values, T * k, f32, "values"),
                                  _rows(tail, T, f32, "tail"), _err_word(err), handle), "lora_topk_logits")


def lora_distill_loss(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, loss: torch.Tensor,
                      kd: Optional[torch.Tensor], dlogits: Optional[torch.Tensor], tail: Optional[torch.Tensor] = None,
                      labels: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      ce: Optional[torch.Tensor] = None, kind: int = LORA_DISTILL_FORWARD, mix: float = 0.5,
                      temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0, grad_scale: float = 1.0,
                      err: Optional[torch.Tensor] = None, stream=None):
    """Divergence of a student's logits from a teacher's list (ids, values [T, k] and tail, as lora_topk_logits
    leaves them), with the labels' cross-entropy, per row, and its gradient (see include/lora_train.h).  dlogits may
    be the logits (the gradient takes their place) or None."""
    handle = _one_device(stream, logits, ids, values, loss, kd, dlogits, tail, labels, weight, ce, err)
    p, ld, code, T, V = _logits(logits)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError("ids: expected a row for each row of logits")
    k = ids.shape[1]
    i32, f32 = torch.int32, torch.float32
    opts = _opts(lora_distill_opts_t, int(kind), float(temperature), float(mix), float(kd_weight), float(ce_weight),
                 float(grad_scale))
    dp, ldd = _grad_of(logits, dlogits)
    _check(lib().lora_distill_loss(p, ld, code, _rows(ids, T * k, i32, "ids"), _rows(values, T * k, f32, "values"),
                                   _rows(tail, T, f32, "tail"), k, _rows(labels, T, i32, "labels"),
                                   _rows(weight, T, f32, "weight"), T, V, opts, _rows(loss, T, f32, "loss"),
                                   _rows(kd, T, f32, "kd"), _rows(ce, T, f32, "ce"), dp, ldd, _err_word(err),
                                   handle), "lora_distill_loss")


# --------------------------------------------------- training: optimizer step --

class TrainProj:
    """One projection's training state beside its pool: gradients, moments and optional fp32
    weights, all laid out like the pool (lora_train_proj_t).  fp32 moments, or e4m3 codes
    (float8_e4m3fn or uint8) with bf16 scales."""

    def __init__(self, view: PoolView, grad: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                 master: Optional[torch.Tensor] = None, m_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        n = view.c.n_pages * view.c.page_elems
        if (m_scale is None) != (v_scale is None):
            raise ValueError("m_scale, v_scale: expected both (8-bit moments) or none")
        self.state = LORA_STATE_F32 if m_scale is None else LORA_STATE_E4M3
        f32, bf16 = (torch.float32,), (torch.bfloat16,)
        moment = f32 if self.state == LORA_STATE_F32 else (torch.float8_e4m3fn, torch.uint8)
        for name, t, count, types in (("grad", grad, n, f32), ("m", m, n, moment), ("v", v, n, moment),
                                      ("master", master, n, f32), ("m_scale", m_scale, n // LORA_ADAMW_BLOCK, bf16),
                                      ("v_scale", v_scale, n // LORA_ADAMW_BLOCK, bf16)):
            if t is None:
                continue
            if t.numel() < count or t.dtype not in types or not t.is_contiguous():
                raise ValueError("%s: expected %d contiguous elements of %s" % (name, count, " or ".join(map(str, types))))
        self.view, self.grad, self.m, self.v = view, grad, m, v
        self.master, self.m_scale, self.v_scale = master, m_scale, v_scale
        self.c = lora_train_proj_t(view.c, *(_addr(t) or None for t in (grad, master, m, v, m_scale, v_scale)))

    @classmethod
    def zeros(cls, view: PoolView, state: int = LORA_STATE_F32, master: bool = False):
        """Zeroed state for a view (run lora_adamw_init for the adapters that train: it fills master)."""
        dev = view.pool.device
        n = view.c.n_pages * view.c.page_elems
        grad = torch.zeros(n, dtype=torch.float32, device=dev)
        w = torch.zeros(n, dtype=torch.float32, device=dev) if master else None
        if state == LORA_STATE_F32:
            return cls(view, grad, torch.zeros_like(grad), torch.zeros_like(grad), master=w)
        m, v = (torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
        ms, vs = (torch.zeros(n // LORA_ADAMW_BLOCK, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return cls(view, grad, m, v, master=w, m_scale=ms, v_scale=vs)


class TrainSet:
    """The projections whose adapters step together (lora_train_proj_t array)."""

    def __init__(self, projs):
        self.projs = list(projs)
        if not self.projs or any(p.state != self.projs[0].state for p in self.projs):
            raise ValueError("expected projections with moments of one kind")
        self.state = self.projs[0].state
        self.n = len(self.projs)
        self.n_adapters = int(self.projs[0].view.c.n_adapters)
        self.c = (lora_train_proj_t * self.n)(*(p.c for p in self.projs))

    def sumsq_workspace(self, n_ids: int) -> torch.Tensor:
        """A workspace for lora_grad_sumsq over n_ids adapters."""
        n = int(lib().lora_grad_sumsq_workspace_bytes(self.c, self.n, n_ids))
        return torch.empty(n, dtype=torch.uint8, device=self.projs[0].grad.device)


def adamw_hyper(n_adapters: int, step=1, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_norm=0.0,
                grad_scale=1.0, device="cuda") -> torch.Tensor:
    """A device array of n_adapters lora_adamw_hyper_t as fp32 [n_adapters, 8] (column 0 holds the
    step's int32 bits: view(torch.int32)[:, 0]); each argument is a value or one value per adapter."""
    h = np.zeros((n_adapters, 8), dtype=np.float32)
    h.view(np.int32)[:, 0] = step
    for k, value in enumerate((lr, beta1, beta2, eps, weight_decay, max_norm, grad_scale)):
        h[:, 1 + k] = value
    return torch.from_numpy(h).to(device)


def _ids(ids: torch.Tensor):
    if ids.dtype is not torch.int32 or not ids.is_contiguous():
        raise ValueError("ids: expected contiguous elements of torch.int32")
    return ids.data_ptr(), ids.numel()


def lora_adamw_init(train: TrainSet, ids: torch.Tensor, err: Optional[torch.Tensor] = None, stream=None):
    """Zero the listed adapters' gradients and moments; master takes the pool's weights."""
    p, n = _ids(ids)
    _check(lib().lora_adamw_init(train.c, train.n, train.state, p, n, _addr(err), _handle(stream)), "lora_adamw_init")


def lora_grad_sumsq(train: TrainSet, ids: torch.Tensor, sumsq: torch.Tensor, workspace: torch.Tensor,
                    accumulate: bool = False, err: Optional[torch.Tensor] = None, stream=None):
    """sumsq[i] = (accumulate: +=) the sum of squares of adapter i's gradients, for the listed ids."""
    p, n = _ids(ids)
    _check(lib().lora_grad_sumsq(train.c, train.n, p, n, 1 if accumulate else 0,
                                 _rows(sumsq, train.n_adapters, torch.float32, "sumsq"), _addr(workspace),
                                 workspace.nbytes, _addr(err), _handle(stream)),
           "lora_grad_sumsq")


def lora_adamw_step(train: TrainSet, ids: torch.Tensor, hyper: torch.Tensor, sumsq: Optional[torch.Tensor] = None,
                    zero_grad: bool = False, err: Optional[torch.Tensor] = None, stream=None):
    """One AdamW step of the listed adapters in place (see include/lora_train.h); hyper: see adamw_hyper."""
    p, n = _ids(ids)
    if hyper.nbytes != 32 * train.n_adapters or not hyper.is_contiguous():
        raise ValueError("hyper: expected %d settings of 32 bytes" % train.n_adapters)
    _check(lib().lora_adamw_step(train.c, train.n, train.state, p, n, _addr(hyper),
                                 _rows(sumsq, train.n_adapters, torch.float32, "sumsq"),
                                 LORA_ADAMW_ZERO_GRAD if zero_grad else 0, _addr(err), _handle(stream)),
           "lora_adamw_step")


# ------------------------------------------------------------- base in 8 bits --

_F8_CODE = {torch.float8_e4m3fn: LORA_F8_E4M3, torch.float8_e5m2: LORA_F8_E5M2}
_F8_TORCH = {code: t for t, code in _F8_CODE.items()}
_F8_FROM = {torch.bfloat16: LORA_F8_FROM_BF16, torch.float32: LORA_F8_FROM_F32}


class F8Matrix:
    """An 8-bit matrix (lora_f8_matrix_t): codes [rows, cols] of float8_e4m3fn or float8_e5m2 whose rows start on
    16-byte boundaries, and fp32 scales [rows / block_rows, cols / 128] (rounded up) of any strides.  block_rows: 1
    (activations, gradients) or 128 (weights)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, block_rows: int = 1):
        code = _F8_CODE.get(codes.dtype)
        if code is None or codes.dim() != 2:
            raise ValueError("codes: expected a matrix of float8_e4m3fn or float8_e5m2")
        if block_rows not in (1, LORA_F8_BLOCK):
            raise ValueError("block_rows: expected 1 or %d" % LORA_F8_BLOCK)
        rows, cols = codes.shape
        ld = codes.stride(0)
        if rows <= 1:
            ld = max(ld, -(-cols // 16) * 16) // 16 * 16  # the stride of a matrix of one row says nothing
        if cols < 1 or (cols > 1 and codes.stride(1) != 1) or ld % 16 or ld < cols or codes.data_ptr() % 16:
            raise ValueError("codes: expected rows of consecutive elements on 16-byte boundaries")
        if scales.dtype is not torch.float32 or tuple(scales.shape) != (-(-rows // block_rows), -(-cols // LORA_F8_BLOCK)):
            raise ValueError("scales: expected torch.float32 of [%d, %d]"
                             % (-(-rows // block_rows), -(-cols // LORA_F8_BLOCK)))
        self.codes, self.scales, self.block_rows, self.type = codes, scales, block_rows, code
        self.c = lora_f8_matrix_t(codes.data_ptr() or None, ld, scales.data_ptr() or None, scales.stride(0), scales.stride(1),
                                  rows, cols, block_rows, code)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, type: int = LORA_F8_E4M3, device="cuda"):
        """Room for a matrix: rows padded to 16 bytes, the scales of a group of 128 columns side by side for all the
        rows (block_rows 1), the layout the product reads fastest."""
        codes = torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=device).view(_F8_TORCH[type])[:, :cols]
        groups, blocks = -(-cols // LORA_F8_BLOCK), -(-rows // block_rows)
        scales = torch.empty(groups, blocks, device=device).t() if block_rows == 1 else torch.empty(blocks, groups, device=device)
        return cls(codes, scales, block_rows)


def _plain(t: torch.Tensor, rows: int, cols: int, what: str):
    """(address, row stride, type code) of a plain [rows, cols] matrix beside 8-bit ones."""
    code = _F8_FROM.get(t.dtype)
    if code is None or t.shape != (rows, cols):
        raise ValueError("%s: expected bfloat16 or float32 of [%d, %d]" % (what, rows, cols))
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("%s: expected a row-major matrix with unit column stride" % what)
    if rows <= 1:
        ld = max(ld, cols)
    elif ld < cols:
        raise ValueError("%s: expected rows that do not overlap" % what)
    return t.data_ptr(), ld, code


def lora_f8_quantize(x: torch.Tensor, q: F8Matrix, pow2: bool = False, err: Optional[torch.Tensor] = None, stream=None):
    """Quantise x (bf16 or fp32, q's shape) into q; pow2: scales are powers of two (see include/lora_f8.h)."""
    handle = _one_device(stream, x, q.codes, q.scales, err)
    p, ld, code = _plain(x, q.c.rows, q.c.cols, "x")
    _check(lib().lora_f8_quantize(p, ld, code, q.ref, LORA_F8_POW2 if pow2 else 0, _err_word(err), handle),
           "lora_f8_quantize")


def lora_base_f8(x: F8Matrix, w: F8Matrix, y: torch.Tensor, err: Optional[torch.Tensor] = None, stream=None):
    """y = x W0^T, written only (bf16 or fp32): x [T, d_in] in groups of a row, w [d_out, d_in] in blocks of 128 rows."""
    handle = _one_device(stream, y, x.codes, x.scales, w.codes, w.scales, err)
    p, ld, code = _plain(y, x.c.rows, w.c.rows, "y")
    _check(lib().lora_base_f8(x.ref, w.ref, p, ld, code, _err_word(err), handle), "lora_base_f8")


def lora_base_f8_backward(dy: F8Matrix, w: F8Matrix, dx: torch.Tensor, err: Optional[torch.Tensor] = None, stream=None):
    """dx = dy W0, written only (bf16 or fp32): the gradient of lora_base_f8's input (the base is frozen)."""
    handle = _one_device(stream, dx, dy.codes, dy.scales, w.codes, w.scales, err)
    p, ld, code = _plain(dx, dy.c.rows, w.c.cols, "dx")
    _check(lib().lora_base_f8_backward(dy.ref, w.ref, p, ld, code, _err_word(err), handle), "lora_base_f8_backward")
