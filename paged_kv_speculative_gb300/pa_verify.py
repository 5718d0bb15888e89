"""Python binding of the C ABI in ``include/pa_verify.h``.

Argument marshalling only: every step of the attention runs in the CUDA
library ``_lib/libpa_verify.so``. There is no fallback; if the library is
missing or fails to load, every entry point raises.

Functions keep the C names without the ``pa_verify_`` prefix: ``plan``,
``run``, ``free``, ``device_errors``, ``last_error``. ``VerifyAttention``
bundles a plan with its device workspace, ``ChunkAttention`` a batch shape of
``pa_chunk_attention`` with its workspace, ``PagePool`` the caches of a pool with
the workspace of the page operations.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Sequence

import torch

from . import _build

KV_BF16 = 0
KV_FP8_E4M3 = 1
OUT_BF16 = 0
OUT_F32 = 1

OK = 0
ERR_INVALID = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_NOMEM = -5

KERNEL_AUTO = 0
KERNEL_WARP_MMA = 1
KERNEL_TCGEN05 = 2

DEVERR_PAGE_RANGE = 1
DEVERR_LENGTHS = 2
DEVERR_TIMEOUT = 4
DEVERR_NO_PAGES = 8
DEVERR_REFS = 16

ROPE_HALVES = 0
ROPE_NEIGHBOURS = 1

# every symbol include/pa_verify.h declares
EXPORTED = ("pa_verify_plan", "pa_verify_plan_get_info", "pa_verify_run", "pa_verify_free",
            "pa_verify_device_errors", "pa_verify_last_error", "pa_verify_profile_enable",
            "pa_verify_profile_read", "pa_kv_write", "pa_greedy_verdict_workspace_bytes",
            "pa_greedy_verdict", "pa_verify_run_static", "pa_verify_plan_dynamic", "pa_verify_plan_get_cta_starts",
            "pa_verify_debug_stall", "pa_verify_plan_get_second", "pa_pages_fork", "pa_pages_workspace_bytes",
            "pa_pages_resize", "pa_pages_compact", "pa_pages_copy", "pa_rope_write", "pa_chunk_workspace_bytes",
            "pa_chunk_attention")


class PaVerifyError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pa_verify status {status}: {message}")
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_seqs", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "kv_dtype", "out_dtype",
        "num_pages", "block_table_stride", "split_override", "sm_count", "kernel")]


class KvWriteDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_kv_heads", "head_dim", "kv_dtype", "num_pages")]


class PagesDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "block_table_stride", "num_pages")]


class PoolDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_pages", "num_kv_heads", "head_dim", "kv_dtype", "num_layers")]


class RopeDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_tokens", "num_q_heads", "num_kv_heads", "head_dim", "rot_dim",
                                               "num_axes", "pairs", "kv_dtype", "num_pages")]
                + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")])


class ChunkDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_seqs", "num_tokens", "num_q_heads", "num_kv_heads", "head_dim",
                                               "page_size", "kv_dtype", "num_pages", "block_table_stride", "sm_count")]
                + [("q_stride", ctypes.c_int64)])


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("num_units", ctypes.c_int32), ("chunk_tokens", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
        ("rows_max", ctypes.c_int32), ("warps", ctypes.c_int32), ("max_splits", ctypes.c_int32),
        ("needs_combine", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("kv_bytes", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_size_t), ("kernel", ctypes.c_int32), ("dynamic", ctypes.c_int32),
        ("flat", ctypes.c_int32), ("total_tiles", ctypes.c_int32), ("device_table", ctypes.c_int32),
        ("launches", ctypes.c_int32), ("split_pairs", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_}


_lib = None


def lib(path: Optional[str] = None):
    """Loads the library (it must have been built: ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library {p} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(p)
    vp, sz, i32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32)
    L.pa_verify_plan.argtypes = [ctypes.POINTER(Desc), i32p, i32p, ctypes.POINTER(vp), ctypes.POINTER(sz)]
    L.pa_verify_plan.restype = ctypes.c_int
    L.pa_verify_plan_dynamic.argtypes = [ctypes.POINTER(Desc), ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(vp),
                                         ctypes.POINTER(sz)]
    L.pa_verify_plan_dynamic.restype = ctypes.c_int
    L.pa_verify_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    L.pa_verify_plan_get_info.restype = ctypes.c_int
    L.pa_verify_plan_get_cta_starts.argtypes = [vp, i32p, ctypes.c_int32]
    L.pa_verify_plan_get_cta_starts.restype = ctypes.c_int
    L.pa_verify_plan_get_second.argtypes = [vp]
    L.pa_verify_plan_get_second.restype = vp
    L.pa_verify_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, sz, vp]
    L.pa_verify_run.restype = ctypes.c_int
    L.pa_verify_run_static.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp]
    L.pa_verify_run_static.restype = ctypes.c_int
    L.pa_verify_debug_stall.argtypes = [vp, ctypes.c_int32, ctypes.c_uint32]
    L.pa_verify_debug_stall.restype = ctypes.c_int
    L.pa_verify_free.argtypes = [vp]
    L.pa_verify_free.restype = None
    L.pa_verify_device_errors.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, vp]
    L.pa_verify_device_errors.restype = ctypes.c_int
    L.pa_verify_profile_enable.argtypes = [vp, ctypes.c_int]
    L.pa_verify_profile_enable.restype = ctypes.c_int
    L.pa_verify_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float)]
    L.pa_verify_profile_read.restype = ctypes.c_int
    L.pa_kv_write.argtypes = [ctypes.POINTER(KvWriteDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.pa_kv_write.restype = ctypes.c_int
    L.pa_greedy_verdict_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
    L.pa_greedy_verdict_workspace_bytes.restype = ctypes.c_size_t
    L.pa_greedy_verdict.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32] + [vp] * 7 + [sz, vp]
    L.pa_greedy_verdict.restype = ctypes.c_int
    L.pa_pages_fork.argtypes = [ctypes.POINTER(PagesDesc)] + [vp] * 5 + [ctypes.c_int32, vp, vp]
    L.pa_pages_workspace_bytes.argtypes = [ctypes.POINTER(PagesDesc)]
    L.pa_pages_workspace_bytes.restype = sz
    L.pa_pages_resize.argtypes = [ctypes.POINTER(PagesDesc)] + [vp] * 8 + [sz, vp]
    L.pa_pages_compact.argtypes = [ctypes.POINTER(PagesDesc)] + [vp] * 10 + [sz, vp]
    L.pa_pages_copy.argtypes = [ctypes.POINTER(PoolDesc), vp, vp, ctypes.c_int32] + [vp] * 7
    L.pa_rope_write.argtypes = [ctypes.POINTER(RopeDesc)] + [vp] * 14
    L.pa_chunk_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
    L.pa_chunk_workspace_bytes.restype = sz
    L.pa_chunk_attention.argtypes = [ctypes.POINTER(ChunkDesc)] + [vp] * 8 + [ctypes.c_float, vp, vp, sz, vp]
    for f in (L.pa_pages_fork, L.pa_pages_resize, L.pa_pages_compact, L.pa_pages_copy, L.pa_rope_write,
              L.pa_chunk_attention):
        f.restype = ctypes.c_int
    L.pa_verify_last_error.argtypes = []
    L.pa_verify_last_error.restype = ctypes.c_char_p
    if path is None:
        _lib = L
    return L


def last_error() -> str:
    return lib().pa_verify_last_error().decode()


def _check(status: int):
    if status != OK:
        raise PaVerifyError(status, last_error())


class Plan:
    """A host-side plan (owns the C handle)."""

    def __init__(self, handle: int, desc: Desc, workspace_bytes: int, owned: bool = True):
        self.handle = handle
        self.desc = desc
        self.workspace_bytes = workspace_bytes
        self.owned = owned
        info = PlanInfo()
        _check(lib().pa_verify_plan_get_info(handle, ctypes.byref(info)))
        self.info = info

    def second(self) -> Optional["Plan"]:
        """The second launch of a two-launch plan (a view owned by this plan), or None."""
        h = lib().pa_verify_plan_get_second(self.handle)
        if not h:
            return None
        v = Plan(h, self.desc, self.workspace_bytes, owned=False)
        v.parent = self  # keeps the owner alive while the view is used
        return v

    def cta_starts(self) -> list:
        """A static flat plan's CTA ranges: CTA c covers flat tiles [s[c], s[c + 1])."""
        buf = (ctypes.c_int32 * (self.info.num_units + 1))()
        n = lib().pa_verify_plan_get_cta_starts(self.handle, buf, len(buf))
        _check(min(n, 0))
        return list(buf[:n])

    def free(self):
        if self.handle and self.owned:
            lib().pa_verify_free(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _runnable(p: Plan):
    if not p.owned:
        raise ValueError("the second launch of a two-launch plan runs only as part of its plan")


def plan(num_q_heads: int, num_kv_heads: int, head_dim: int, kv_dtype: int, out_dtype: int, num_pages: int,
         block_table_stride: int, context_lens: Sequence[int], query_lens: Sequence[int],
         split_override: int = 0, sm_count: int = 0, page_size: int = 16, kernel: int = KERNEL_AUTO) -> Plan:
    """pa_verify_plan with host lengths; raises PaVerifyError on refusal."""
    n = len(context_lens)
    d = Desc(num_seqs=n, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim,
             page_size=page_size, kv_dtype=kv_dtype, out_dtype=out_dtype, num_pages=num_pages,
             block_table_stride=block_table_stride, split_override=split_override, sm_count=sm_count,
             kernel=kernel)
    arr = ctypes.c_int32 * max(1, n)
    cl = arr(*[int(x) for x in context_lens])
    ql = arr(*[int(x) for x in query_lens])
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib().pa_verify_plan(ctypes.byref(d), cl, ql, ctypes.byref(h), ctypes.byref(ws)))
    return Plan(h.value, d, ws.value)


def plan_dynamic(num_q_heads: int, num_kv_heads: int, head_dim: int, kv_dtype: int, out_dtype: int, num_pages: int,
                 block_table_stride: int, capacity: int, max_context_len: int, max_query_len: int,
                 sm_count: int = 0, kernel: int = KERNEL_AUTO) -> Plan:
    """pa_verify_plan_dynamic: a capacity plan whose lengths are read on the device each run."""
    d = Desc(num_seqs=capacity, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim, page_size=16,
             kv_dtype=kv_dtype, out_dtype=out_dtype, num_pages=num_pages, block_table_stride=block_table_stride,
             split_override=0, sm_count=sm_count, kernel=kernel)
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib().pa_verify_plan_dynamic(ctypes.byref(d), int(max_context_len), int(max_query_len), ctypes.byref(h),
                                        ctypes.byref(ws)))
    return Plan(h.value, d, ws.value)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def run(p: Plan, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: Optional[torch.Tensor],
        v_scale: Optional[torch.Tensor], block_table: torch.Tensor, context_lens: torch.Tensor,
        query_lens: torch.Tensor, softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor,
        stream: Optional[torch.cuda.Stream] = None):
    """pa_verify_run on device tensors (enqueued on ``stream`` or torch's current stream)."""
    _runnable(p)
    _need(q, "q", torch.bfloat16)
    for t, nm in ((k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out"), (workspace, "workspace")):
        _need(t, nm)
    for t, nm in ((block_table, "block_table"), (context_lens, "context_lens"), (query_lens, "query_lens")):
        _need(t, nm, torch.int32)
    for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is not None:
            _need(t, nm, torch.float32)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    _check(lib().pa_verify_run(p.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                               _ptr(block_table), _ptr(context_lens), _ptr(query_lens), float(softmax_scale),
                               _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                               s.cuda_stream))


def run_static(p: Plan, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               k_scale: Optional[torch.Tensor], v_scale: Optional[torch.Tensor], block_table: torch.Tensor,
               context_lens: torch.Tensor, query_lens: torch.Tensor, softmax_scale: float, out: torch.Tensor,
               stream: Optional[torch.cuda.Stream] = None):
    """pa_verify_run_static: like ``run`` but with the library's fixed device
    scratch instead of a workspace, for callers that cannot allocate."""
    _runnable(p)
    _need(q, "q", torch.bfloat16)
    for t, nm in ((k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
        _need(t, nm)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    _check(lib().pa_verify_run_static(p.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                      _ptr(v_scale), _ptr(block_table), _ptr(context_lens), _ptr(query_lens),
                                      float(softmax_scale), _ptr(out), s.cuda_stream))


def device_errors(workspace: Optional[torch.Tensor], clear: bool = False,
                  stream: Optional[torch.cuda.Stream] = None) -> int:
    """The device error word of ``workspace``; ``None`` reads the fixed scratch of ``run_static``."""
    s = stream if stream is not None else torch.cuda.current_stream(
        workspace.device if workspace is not None else None)
    flags = ctypes.c_uint32()
    _check(lib().pa_verify_device_errors(_ptr(workspace), ctypes.byref(flags), int(bool(clear)), s.cuda_stream))
    return int(flags.value)


def rescale_count(workspace: torch.Tensor) -> int:
    """Word 1 of a workspace header: in-segment rescales of the output accumulator so far."""
    return int(workspace[4:8].view(torch.int32).item())


def debug_stall(p: Plan, stall_cta: int, wait_limit_us: int = 0):
    """pa_verify_debug_stall: bounded-wait test hook (stall_cta = -1 and 0 restore the defaults)."""
    _check(lib().pa_verify_debug_stall(p.handle, int(stall_cta), int(wait_limit_us)))


def profile_enable(p: Plan, enable: bool = True):
    _check(lib().pa_verify_profile_enable(p.handle, int(bool(enable))))


def profile_read(p: Plan):
    """(split kernel ms, combine kernel ms) of the last profiled run."""
    a, b = ctypes.c_float(), ctypes.c_float()
    _check(lib().pa_verify_profile_read(p.handle, ctypes.byref(a), ctypes.byref(b)))
    return float(a.value), float(b.value)


def free(p: Plan):
    p.free()


def kv_write(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, k_scale: Optional[torch.Tensor], v_scale: Optional[torch.Tensor],
             kv_dtype: int, error_flags: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """pa_kv_write: stores new tokens' K/V rows [n, Hkv, D] into their slots."""
    _need(k_new, "k_new", torch.bfloat16)
    _need(v_new, "v_new", torch.bfloat16)
    _need(slot_mapping, "slot_mapping", torch.int64)
    _need(k_cache, "k_cache")
    _need(v_cache, "v_cache")
    n, hkv, d = k_new.shape
    desc = KvWriteDesc(num_tokens=n, num_kv_heads=hkv, head_dim=d, kv_dtype=kv_dtype, num_pages=k_cache.shape[0])
    s = stream if stream is not None else torch.cuda.current_stream(k_new.device)
    _check(lib().pa_kv_write(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
                             _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(error_flags), s.cuda_stream))


class VerifyAttention:
    """A plan plus a zero-initialised device workspace for one batch shape."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, kv_dtype: int, num_pages: int,
                 block_table_stride: int, context_lens: Sequence[int], query_lens: Sequence[int],
                 out_dtype: int = OUT_F32, split_override: int = 0, device: Optional[torch.device] = None,
                 kernel: int = KERNEL_AUTO):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self.plan = plan(num_q_heads, num_kv_heads, head_dim, kv_dtype, out_dtype, num_pages, block_table_stride,
                             context_lens, query_lens, split_override=split_override, kernel=kernel)
        self.out_dtype = out_dtype
        self.num_q_heads = num_q_heads
        self.head_dim = head_dim
        self.workspace = torch.zeros(max(256, self.plan.workspace_bytes), dtype=torch.uint8, device=self.device)

    @property
    def info(self) -> dict:
        return self.plan.info.as_dict()

    def new_out(self) -> torch.Tensor:
        T = self.plan.info.num_tokens
        dt = torch.float32 if self.out_dtype == OUT_F32 else torch.bfloat16
        return torch.empty((T, self.num_q_heads, self.head_dim), dtype=dt, device=self.device)

    def __call__(self, q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, query_lens,
                 softmax_scale: float, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        if out is None:
            out = self.new_out()
        run(self.plan, q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, query_lens,
            softmax_scale, out, self.workspace, stream)
        return out

    def device_errors(self, clear: bool = False) -> int:
        return device_errors(self.workspace, clear=clear)


def greedy_verdict(logits: torch.Tensor, input_ids: torch.Tensor, query_lens: torch.Tensor,
                   workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """pa_greedy_verdict: (target_ids [T], accepted [B], next_token [B]) int32 device tensors."""
    _need(logits, "logits", torch.bfloat16)
    _need(input_ids, "input_ids", torch.int32)
    _need(query_lens, "query_lens", torch.int32)
    T, V = logits.shape
    B = query_lens.shape[0]
    dev = logits.device
    need = lib().pa_greedy_verdict_workspace_bytes(T, V)
    if workspace is None:
        workspace = torch.zeros(max(256, need), dtype=torch.uint8, device=dev)
    tgt = torch.empty(T, dtype=torch.int32, device=dev)
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(lib().pa_greedy_verdict(B, T, V, _ptr(logits), _ptr(input_ids), _ptr(query_lens), _ptr(tgt), _ptr(acc),
                                   _ptr(nxt), _ptr(workspace), workspace.numel(), s.cuda_stream))
    return tgt, acc, nxt


# ------------------------------------------------------------------ prompts: pages, rotary writes, chunk attention
# These calls take few microseconds on the device, so their checks are written as one expression of plain attribute reads
# each (about 0.1 us a read); what failed is found out afterwards, by _explain.
_BF16, _F32, _F64, _I32, _I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
_FP8_TYPES = (torch.uint8, torch.float8_e4m3fn)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


_fast_module = None


def _fast():
    """csrc/pa_fast.cpp, which makes the plain case of these calls in one step, or False when it is not built."""
    global _fast_module
    if _fast_module is None:
        _fast_module = False
        path = _build.fast_path()
        if os.path.exists(path):
            spec = importlib.util.spec_from_file_location("pa_fast", path)
            m = importlib.util.module_from_spec(spec)
            try:
                spec.loader.exec_module(m)
            except ImportError:  # something it links is not there
                return False
            L = lib()
            m.init(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                L.pa_rope_write, L.pa_chunk_attention, L.pa_pages_fork, L.pa_pages_resize, L.pa_pages_compact, L.pa_pages_copy)])
            _fast_module = m
    return _fast_module


def _fast_result(r):
    if type(r) is int:
        raise PaVerifyError(r, last_error())
    return r


def _launch(dev: int, stream: Optional[torch.cuda.Stream], fn, *args):
    """Calls ``fn(*args, stream)`` with device ``dev`` current (``stream``: None = torch's current stream of that device)."""
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == torch.cuda.current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != OK:
        raise PaVerifyError(rc, last_error())


def _empty(shape, dtype, device: torch.device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new tensor that belongs to the stream of the call that fills it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _zeroed(n: int, dtype, device: torch.device) -> torch.Tensor:
    """Zeros that a call on any stream finds as zeros: the current stream, which fills them, is waited for."""
    with torch.cuda.device(device):
        t = torch.zeros(n, dtype=dtype, device=device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
    return t


def _explain(dev: int, **wanted):
    """Raises for the first of ``name=(tensor, dtype, shape)`` that is not contiguous, of that type and shape (None: any) on
    device ``dev``."""
    for name, (t, dtype, shape) in wanted.items():
        if t is None:
            raise ValueError(f"{name} is needed")
        _need(t, name, dtype)
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError("arguments do not belong together")


def _rows(t: torch.Tensor, name: str) -> int:
    """Elements between the tokens of a [T, heads, D] bf16 tensor whose heads are contiguous and whose tokens do not overlap (in
    the C ABI a stride of 0 means contiguous, so an expanded tensor must not get there)."""
    if t.dtype is _BF16 and t.dim() == 3 and t.is_cuda:
        n, h, d = t.shape
        s0, s1, s2 = t.stride()
        if s2 == 1 and (h == 1 or s1 == d):
            if n <= 1:
                return h * d
            if s0 >= h * d:
                return s0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    raise ValueError(f"{name} must be [tokens, heads, head_dim] with contiguous heads and tokens that do not overlap")


def _caches_ok(dev: int, k_cache, v_cache, k_scale, v_scale, kv_dtype: int, num_kv_heads: int, head_dim: int,
               num_pages: Optional[int] = None):
    """Checks a layer's caches [num_pages, Hkv, 16, D], bf16 or E4M3 codes (float8_e4m3fn or uint8), and, for FP8, their scales
    [num_pages, Hkv, 16]."""
    types = _FP8_TYPES if kv_dtype == KV_FP8_E4M3 else (_BF16,)
    shape = k_cache.shape
    if (shape[1:] == (num_kv_heads, 16, head_dim) and (num_pages is None or shape[0] == num_pages) and v_cache.shape == shape
            and k_cache.dtype in types and v_cache.dtype in types and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_cache.get_device() == dev and v_cache.get_device() == dev):
        if kv_dtype != KV_FP8_E4M3:
            return
        n = shape[0] * num_kv_heads * 16
        if (k_scale is not None and v_scale is not None and k_scale.dtype is _F32 and v_scale.dtype is _F32
                and k_scale.numel() == n and v_scale.numel() == n and k_scale.is_contiguous() and v_scale.is_contiguous()
                and k_scale.get_device() == dev and v_scale.get_device() == dev):
            return
        _explain(dev, k_scale=(k_scale, _F32, (shape[0], num_kv_heads, 16)), v_scale=(v_scale, _F32, (shape[0], num_kv_heads, 16)))
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype not in types:
            raise ValueError(f"{name} must be {' or '.join(map(str, types))}, got {t.dtype}")
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, name)
        pages = num_pages if num_pages is not None else k_cache.shape[0]
        if t.get_device() != dev or tuple(t.shape) != (pages, num_kv_heads, 16, head_dim):
            _explain(dev, **{name: (t, None, (pages, num_kv_heads, 16, head_dim))})
    raise ValueError("k_cache and v_cache do not belong together")


def rope_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
               pair_axis: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               k_scale: Optional[torch.Tensor], v_scale: Optional[torch.Tensor], kv_dtype: int,
               q_out: Optional[torch.Tensor] = None, pairs: int = ROPE_HALVES,
               error_flags: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """pa_rope_write: rotates q and k by positions [axes, T] and stores k, v into their slots; returns q_out.

    q, k and v may be views of one projection's output (any token stride, contiguous heads)."""
    if stream is None and _fast():
        r = _fast_module.rope(q, k, v, positions, inv_freq, pair_axis, slot_mapping, k_cache, v_cache, k_scale, v_scale, kv_dtype,
                              q_out, pairs, error_flags)
        if r is not None:
            return _fast_result(r)
    qs, ks, vs = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    n, hq, d = q.shape
    hkv, dev, half = k.shape[1], q.get_device(), inv_freq.shape[0]
    if k.shape != (n, hkv, d) or v.shape != (n, hkv, d):
        raise ValueError(f"k and v must be [{n}, kv heads, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    if q_out is None:
        q_out, os_ = _empty((n, hq, d), _BF16, q.device, stream), hq * d
    else:
        os_ = _rows(q_out, "q_out")
        if q_out.shape != q.shape:
            raise ValueError(f"q_out must be {tuple(q.shape)}, got {tuple(q_out.shape)}")
    if positions.dim() != 2:
        raise ValueError(f"positions must be [axes, {n}], got {tuple(positions.shape)}")
    axes = positions.shape[0]
    if not (positions.dtype is _I32 and positions.shape[1] == n and positions.is_contiguous() and positions.get_device() == dev
            and inv_freq.dtype is _F64 and inv_freq.shape == (half,) and inv_freq.is_contiguous() and inv_freq.get_device() == dev
            and pair_axis.dtype is _I32 and pair_axis.shape == (half,) and pair_axis.is_contiguous()
            and pair_axis.get_device() == dev and slot_mapping.dtype is _I64 and slot_mapping.shape == (n,)
            and slot_mapping.is_contiguous() and slot_mapping.get_device() == dev and k.get_device() == dev
            and v.get_device() == dev and q_out.get_device() == dev
            and (error_flags is None or (error_flags.get_device() == dev and error_flags.element_size() == 4))):
        _explain(dev, positions=(positions, _I32, (axes, n)), inv_freq=(inv_freq, _F64, (half,)),
                 pair_axis=(pair_axis, _I32, (half,)), slot_mapping=(slot_mapping, _I64, (n,)))
    _caches_ok(dev, k_cache, v_cache, k_scale, v_scale, kv_dtype, hkv, d)
    desc = RopeDesc(n, hq, hkv, d, 2 * half, axes, pairs, kv_dtype, k_cache.shape[0], qs, ks, vs, os_)
    fp8 = kv_dtype == KV_FP8_E4M3
    _launch(dev, stream, lib().pa_rope_write, ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(),
            inv_freq.data_ptr(), pair_axis.data_ptr(), slot_mapping.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr() if fp8 else None, v_scale.data_ptr() if fp8 else None,
            None if error_flags is None else error_flags.data_ptr())
    return q_out


class ChunkAttention:
    """pa_chunk_attention for batches of up to ``max_seqs`` sequences, with a zero-initialised device workspace (the object has
    to live until its calls have run; making one waits for the current stream)."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, kv_dtype: int, num_pages: int,
                 block_table_stride: int, max_seqs: int = 1024, device: Optional[torch.device] = None):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.max_seqs = max_seqs
        self.num_q_heads, self.num_kv_heads, self.head_dim, self.kv_dtype = num_q_heads, num_kv_heads, head_dim, kv_dtype
        self.num_pages, self.block_table_stride = num_pages, block_table_stride
        self.sm_count = torch.cuda.get_device_properties(self.device).multi_processor_count
        need = lib().pa_chunk_workspace_bytes(ctypes.byref(self._desc(max_seqs, 0, 0)))
        if need == 0:
            raise PaVerifyError(ERR_UNSUPPORTED, last_error())
        self.workspace = _zeroed(need, torch.uint8, self.device)
        self._plain = (num_q_heads, num_kv_heads, head_dim, kv_dtype, num_pages, block_table_stride, max_seqs, self.sm_count,
                       self.workspace.data_ptr(), need, self.device.index)

    def _desc(self, num_seqs: int, num_tokens: int, q_stride: int) -> ChunkDesc:
        return ChunkDesc(num_seqs, num_tokens, self.num_q_heads, self.num_kv_heads, self.head_dim, 16, self.kv_dtype,
                         self.num_pages, self.block_table_stride, self.sm_count, q_stride)

    def __call__(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: Optional[torch.Tensor],
                 v_scale: Optional[torch.Tensor], block_table: torch.Tensor, context_lens: torch.Tensor,
                 query_lens: torch.Tensor, softmax_scale: float, out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """q [T, Hq, D] (any token stride); rows of ``out`` behind the last sequence are left as they were."""
        if stream is None and _fast():
            r = _fast_module.chunk(self._plain, q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, query_lens,
                                   softmax_scale, out)
            if r is not None:
                return _fast_result(r)
        stride, dev = _rows(q, "q"), self.device.index
        tokens, n = q.shape[0], context_lens.shape[0]
        shape = (tokens, self.num_q_heads, self.head_dim)
        if q.shape != shape or n > self.max_seqs:
            raise ValueError(f"q must be [tokens, {self.num_q_heads}, {self.head_dim}] for up to {self.max_seqs} sequences, got "
                             f"{tuple(q.shape)} and {n} sequences")
        if out is None:
            out = _empty(shape, _BF16, self.device, stream)
        if not (out.dtype is _BF16 and out.shape == shape and out.is_contiguous() and out.get_device() == dev
                and block_table.dtype is _I32 and block_table.shape == (n, self.block_table_stride) and block_table.is_contiguous()
                and block_table.get_device() == dev and context_lens.dtype is _I32 and context_lens.dim() == 1
                and context_lens.is_contiguous() and context_lens.get_device() == dev and query_lens.dtype is _I32
                and query_lens.shape == (n,) and query_lens.is_contiguous() and query_lens.get_device() == dev
                and q.get_device() == dev):
            _explain(dev, out=(out, _BF16, shape), block_table=(block_table, _I32, (n, self.block_table_stride)),
                     context_lens=(context_lens, _I32, (n,)), query_lens=(query_lens, _I32, (n,)))
        _caches_ok(dev, k_cache, v_cache, k_scale, v_scale, self.kv_dtype, self.num_kv_heads, self.head_dim, self.num_pages)
        fp8 = self.kv_dtype == KV_FP8_E4M3
        _launch(dev, stream, lib().pa_chunk_attention, ctypes.byref(self._desc(n, tokens, stride)), q.data_ptr(),
                k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr() if fp8 else None, v_scale.data_ptr() if fp8 else None,
                block_table.data_ptr(), context_lens.data_ptr(), query_lens.data_ptr(), softmax_scale, out.data_ptr(),
                self.workspace.data_ptr(), self.workspace.numel())
        return out

    def device_errors(self, clear: bool = False) -> int:
        with torch.cuda.device(self.device):
            return device_errors(self.workspace, clear=clear)


class PagePool:
    """The page operations on one pool: its layers' caches, a workspace and an error word.

    The block table [B, stride], the lengths [B] and the reference counts [num_pages] (int32 device tensors) are the
    caller's and travel with each call. ``k_caches`` / ``v_caches``: one [num_pages, Hkv, 16, D] tensor a layer, bf16,
    or E4M3 codes (as float8_e4m3fn or uint8) with ``k_scales`` / ``v_scales`` [num_pages, Hkv, 16]. The pool has to live until
    its calls have run; making one waits for the current stream."""

    def __init__(self, k_caches: Sequence[torch.Tensor], v_caches: Sequence[torch.Tensor],
                 k_scales: Optional[Sequence[torch.Tensor]] = None, v_scales: Optional[Sequence[torch.Tensor]] = None):
        if not k_caches or len(v_caches) != len(k_caches):
            raise ValueError("k_caches and v_caches must hold one tensor a layer")
        first = k_caches[0]
        if first.dim() != 4 or not first.is_cuda:
            raise ValueError("caches must be [num_pages, kv heads, 16, head_dim] CUDA tensors")
        self.kv_dtype = KV_FP8_E4M3 if first.element_size() == 1 else KV_BF16
        fp8 = self.kv_dtype == KV_FP8_E4M3
        self.device, self.dev, self.num_pages, hkv, d = first.device, first.get_device(), first.shape[0], first.shape[1], first.shape[3]
        for group, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            if (group is not None) != fp8 or (fp8 and len(group) != len(k_caches)):
                raise ValueError(f"{name} must hold one tensor a layer for 8-bit caches and be None for bf16")
        for i, (k, v) in enumerate(zip(k_caches, v_caches)):
            _caches_ok(self.dev, k, v, k_scales[i] if fp8 else None, v_scales[i] if fp8 else None, self.kv_dtype, hkv, d, self.num_pages)
        self.caches = (list(k_caches), list(v_caches), list(k_scales or ()), list(v_scales or ()))  # keeps them alive
        self.desc = PoolDesc(self.num_pages, hkv, d, self.kv_dtype, len(k_caches))
        array = ctypes.c_void_p * len(k_caches)
        self.pointers = [array(*[t.data_ptr() for t in g]) if g else None for g in self.caches]
        need = lib().pa_pages_workspace_bytes(ctypes.byref(PagesDesc(0, 1, self.num_pages)))
        if need == 0:
            raise PaVerifyError(ERR_UNSUPPORTED, last_error())
        self.errors = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.workspace = _zeroed(need, torch.uint8, self.device)
        self._scratch = (self.errors.data_ptr(), self.workspace.data_ptr(), need)
        self._pool = _fast().pool_new(self.num_pages, hkv, d, self.kv_dtype, self.dev, *self._scratch,
                                      *[[t.data_ptr() for t in g] for g in self.caches]) if _fast() else None

    def _tables(self, block_table, context_lens, ref_counts) -> PagesDesc:
        dev = self.dev
        if block_table.dim() != 2:
            raise ValueError("block_table must be [sequences, entries]")
        n, stride = block_table.shape
        if not (block_table.dtype is _I32 and block_table.is_contiguous() and block_table.get_device() == dev
                and context_lens.dtype is _I32 and context_lens.shape == (n,) and context_lens.is_contiguous()
                and context_lens.get_device() == dev and ref_counts.dtype is _I32 and ref_counts.shape == (self.num_pages,)
                and ref_counts.is_contiguous() and ref_counts.get_device() == dev):
            _explain(dev, block_table=(block_table, _I32, None), context_lens=(context_lens, _I32, (n,)),
                     ref_counts=(ref_counts, _I32, (self.num_pages,)))
        return PagesDesc(n, stride, self.num_pages)

    def fork(self, block_table, context_lens, ref_counts, parents, children, stream=None):
        """pa_pages_fork: row children[i] shares row parents[i]'s pages."""
        if stream is None and self._pool is not None:
            r = _fast_module.fork(self._pool, block_table, context_lens, ref_counts, parents, children)
            if r is not None:
                _fast_result(r if r is not True else None)
                return
        desc, dev = self._tables(block_table, context_lens, ref_counts), self.dev
        n = parents.shape[0]
        if not (parents.dtype is _I32 and parents.dim() == 1 and parents.is_contiguous() and parents.get_device() == dev
                and children.dtype is _I32 and children.shape == (n,) and children.is_contiguous() and children.get_device() == dev):
            _explain(dev, parents=(parents, _I32, (n,)), children=(children, _I32, (n,)))
        _launch(dev, stream, lib().pa_pages_fork, ctypes.byref(desc), block_table.data_ptr(), context_lens.data_ptr(),
                ref_counts.data_ptr(), parents.data_ptr(), children.data_ptr(), n, self._scratch[0])

    def resize(self, block_table, context_lens, ref_counts, new_lens, stream=None):
        """pa_pages_resize: lengths to new_lens (negative: as they are); returns (copy_src, copy_dst) for ``copy``."""
        if stream is None and self._pool is not None:
            r = _fast_module.resize(self._pool, block_table, context_lens, ref_counts, new_lens)
            if r is not None:
                return _fast_result(r)
        desc, dev = self._tables(block_table, context_lens, ref_counts), self.dev
        n = block_table.shape[0]
        if not (new_lens.dtype is _I32 and new_lens.shape == (n,) and new_lens.is_contiguous() and new_lens.get_device() == dev):
            _explain(dev, new_lens=(new_lens, _I32, (n,)))
        src, dst = _empty(n, _I32, self.device, stream), _empty(n, _I32, self.device, stream)
        _launch(dev, stream, lib().pa_pages_resize, ctypes.byref(desc), block_table.data_ptr(), context_lens.data_ptr(),
                ref_counts.data_ptr(), new_lens.data_ptr(), src.data_ptr(), dst.data_ptr(), *self._scratch)
        return src, dst

    def compact(self, block_table, context_lens, ref_counts, in_place: bool = False, stream=None):
        """pa_pages_compact: (block_table, ref_counts, copy_src, copy_dst, num_moves), new tensors or rewritten in place."""
        if stream is None and self._pool is not None:
            r = _fast_module.compact(self._pool, block_table, context_lens, ref_counts, in_place)
            if r is not None:
                return _fast_result(r)
        desc = self._tables(block_table, context_lens, ref_counts)
        new = lambda shape: _empty(shape, _I32, self.device, stream)
        table, ref = (block_table, ref_counts) if in_place else (new(block_table.shape), new(self.num_pages))
        src, dst, moves = new(self.num_pages // 2), new(self.num_pages // 2), new(1)
        _launch(self.dev, stream, lib().pa_pages_compact, ctypes.byref(desc), block_table.data_ptr(), context_lens.data_ptr(),
                ref_counts.data_ptr(), table.data_ptr(), ref.data_ptr(), src.data_ptr(), dst.data_ptr(), moves.data_ptr(),
                *self._scratch)
        return table, ref, src, dst, moves

    def copy(self, copy_src, copy_dst, num_pairs: Optional[torch.Tensor] = None, stream=None):
        """pa_pages_copy: pages copy_src[i] to copy_dst[i] in every layer (num_pairs: a device count, as ``compact`` gives)."""
        if stream is None and self._pool is not None:
            r = _fast_module.copy(self._pool, copy_src, copy_dst, num_pairs)
            if r is not None:
                _fast_result(r if r is not True else None)
                return
        n, dev = copy_src.shape[0], self.dev
        if not (copy_src.dtype is _I32 and copy_src.dim() == 1 and copy_src.is_contiguous() and copy_src.get_device() == dev
                and copy_dst.dtype is _I32 and copy_dst.shape == (n,) and copy_dst.is_contiguous() and copy_dst.get_device() == dev
                and (num_pairs is None or (num_pairs.dtype is _I32 and num_pairs.shape == (1,) and num_pairs.get_device() == dev))):
            _explain(dev, copy_src=(copy_src, _I32, (n,)), copy_dst=(copy_dst, _I32, (n,)),
                     **({} if num_pairs is None else {"num_pairs": (num_pairs, _I32, (1,))}))
        k, v, ks, vs = self.pointers
        _launch(dev, stream, lib().pa_pages_copy, ctypes.byref(self.desc), copy_src.data_ptr(), copy_dst.data_ptr(), n,
                None if num_pairs is None else num_pairs.data_ptr(), k, v, ks, vs, self._scratch[0])

    def device_errors(self, clear: bool = False) -> int:
        """The DEVERR_* bits of the calls so far (waits for the device's current stream)."""
        flags = int(self.errors.item())
        if clear:
            self.errors.zero_()
        return flags
