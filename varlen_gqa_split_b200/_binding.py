"""Binding of libvgqa (include/varlen_gqa.h): argument marshalling only, by
ctypes and, for the cache operators, by the native module _lib/_marshal.*.so
(built for one torch and one interpreter, which its name carries; loaded with
the first of these calls).

Every step of the attention runs in the library's CUDA kernels; this module
checks dtypes, shapes and devices of torch tensors, passes their device
pointers and the current CUDA stream, and turns ATTN_* codes into exceptions.
There is no fallback: if the library is missing or no sm_100 device is
present, the calls raise.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import sys
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libvgqa.so")
MARSHAL_PATH = os.path.join(_HERE, "_lib", f"_marshal.{sys.implementation.cache_tag}.torch-{torch.__version__}.so")

ATTN_OK = 0
ATTN_VARIANT_AUTO, ATTN_VARIANT_SIMT, ATTN_VARIANT_MMA, ATTN_VARIANT_TC = 0, 1, 2, 3
ATTN_COMBINE_AUTO, ATTN_COMBINE_KERNEL, ATTN_COMBINE_FUSED = 0, 1, 2
ATTN_DEV_ERR_OFFSETS = 0x1
ATTN_DEV_ERR_Q_TOO_LONG = 0x2
ATTN_DEV_ERR_K_TOO_LONG = 0x4
ATTN_DEV_ERR_TIMEOUT = 0x8
ATTN_DEV_ERR_PAGE = 0x10
ATTN_DTYPE_BF16, ATTN_DTYPE_F16, ATTN_DTYPE_F32 = 0, 1, 2
ATTN_ROPE_HALF, ATTN_ROPE_INTERLEAVED = 0, 1

EXPORTED = ("attn_plan", "attn_plan_ex", "attn_plan_info", "attn_run", "attn_run_strided", "attn_run_paged",
            "attn_run_rows", "attn_run_paged_rows", "attn_merge_lse", "attn_check_error", "attn_destroy", "attn_strerror", "attn_rope_create",
            "attn_rope_destroy", "attn_rope_apply", "attn_append_paged", "attn_key_weights", "attn_key_weights_paged",
            "attn_evict_paged")


class Overrides(ctypes.Structure):
    _fields_ = [("nsplit", ctypes.c_int), ("block_n", ctypes.c_int), ("variant", ctypes.c_int),
                ("stages", ctypes.c_int), ("combine", ctypes.c_int), ("ctas", ctypes.c_int),
                ("deterministic", ctypes.c_int), ("wait_limit_us", ctypes.c_int), ("test_stall", ctypes.c_int)]


class PlanDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "B_max", "s_max", "Hq", "Hkv", "D", "max_q", "G", "variant", "nsplit", "chunk", "block_n",
        "stages", "rows_per_block", "row_tiles", "grid_x", "grid_y", "grid_z", "ctas", "deterministic", "combine",
        "combine_blocks",
        "smem_bytes", "num_sms")] + [("scratch_bytes", ctypes.c_size_t)]


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (code {code})")


_lock = threading.Lock()
_lib = None


class _Unloaded:
    """Stands for the marshalling module until one of its functions is asked for."""

    def __getattr__(self, name):
        global _marshal
        lib()
        with _lock:
            if isinstance(_marshal, _Unloaded):
                if not os.path.exists(MARSHAL_PATH):
                    raise RuntimeError(f"the cache operators' binding is not built for this torch and interpreter "
                                       f"({MARSHAL_PATH}); run `python -m varlen_gqa_split_b200.build`")
                loader = importlib.machinery.ExtensionFileLoader("_marshal", MARSHAL_PATH)
                m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
                loader.exec_module(m)
                m.bind(LIB_PATH)
                _marshal = m
        return getattr(_marshal, name)


_marshal = _Unloaded()   # native marshalling of the cache operators


def lib() -> ctypes.CDLL:
    """Load libvgqa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libvgqa.so not built ({LIB_PATH}); run "
                               "`python -m varlen_gqa_split_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, i32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
        L.attn_plan.argtypes = [ctypes.POINTER(vp), i, i, i, i, i, i]
        L.attn_plan.restype = i
        L.attn_plan_ex.argtypes = [ctypes.POINTER(vp), i, i, i, i, i, i, ctypes.POINTER(Overrides)]
        L.attn_plan_ex.restype = i
        L.attn_plan_info.argtypes = [vp, ctypes.POINTER(PlanDesc)]
        L.attn_plan_info.restype = i
        L.attn_run.argtypes = [vp, vp, vp, vp, i32p, i32p, vp, vp, vp]
        L.attn_run.restype = i
        L.attn_run_strided.argtypes = [vp, vp, vp, vp, i32p, i32p, vp, vp, ctypes.c_int64, ctypes.c_int64, vp]
        L.attn_run_strided.restype = i
        i64 = ctypes.c_int64
        L.attn_run_paged.argtypes = [vp, vp, vp, vp, i64, i64, i, i, i32p, i, i32p, i32p, vp, vp, vp]
        L.attn_run_paged.restype = i
        L.attn_run_rows.argtypes = [vp, vp, i64, vp, vp, i64, i64, i64, i32p, i32p, vp, vp, vp]
        L.attn_run_rows.restype = i
        L.attn_run_paged_rows.argtypes = [vp, vp, i64, vp, vp, i64, i64, i, i, i32p, i, i32p, i32p, vp, vp, vp]
        L.attn_run_paged_rows.restype = i
        L.attn_merge_lse.argtypes = [i, vp, vp, i64, i32p, i, i, i, vp, vp, vp]
        L.attn_merge_lse.restype = i
        L.attn_check_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.attn_check_error.restype = i
        L.attn_destroy.argtypes = [vp]
        L.attn_destroy.restype = None
        L.attn_strerror.argtypes = [i]
        L.attn_strerror.restype = ctypes.c_char_p
        f32 = ctypes.c_float
        L.attn_rope_create.argtypes = [ctypes.POINTER(vp), i, i, i, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_int32), i, f32]
        L.attn_rope_create.restype = i
        L.attn_rope_destroy.argtypes = [vp]
        L.attn_rope_destroy.restype = None
        L.attn_rope_apply.argtypes = [vp, i, vp, i64, i64, i, i32p, i64, i, vp, i64, vp]
        L.attn_rope_apply.restype = i
        cache = [i64, i64, i, i, i32p, i]            # page_stride, token_stride, page_size, num_pages, table, bt_stride
        L.attn_append_paged.argtypes = ([vp, vp, vp, i64, vp, i64, vp, i64, i64, i32p, i64, vp, vp, vp] + cache +
                                        [i32p, i32p, vp])
        L.attn_append_paged.restype = i
        ledger = [i32p, i32p, vp, f32, vp, vp, i64, i32p, i32p, vp]
        L.attn_key_weights.argtypes = [vp, vp, i64, vp, i64, i64] + ledger
        L.attn_key_weights.restype = i
        L.attn_key_weights_paged.argtypes = [vp, vp, i64, vp] + cache + ledger
        L.attn_key_weights_paged.restype = i
        L.attn_evict_paged.argtypes = [vp, vp, i32p, i32p, i32p, i, i, vp, i32p, i64, vp, vp] + cache + [i32p, i32p, vp]
        L.attn_evict_paged.restype = i
        _lib = L
        return L


def merge_lse(outs, lses, cu_q, out=None, lse=None, stream=None):
    """out, lse = merge_lse(outs, lses, cu_q[, out, lse, stream]): combine the
    attention results of n disjoint key ranges (attn_merge_lse).

    outs [n, T_q, Hq, D] bf16 and lses [n, T_q, Hq] fp32 contiguous CUDA
    tensors; cu_q int32 [B_max + 1]; only tokens [cu_q[0], cu_q[B_max]) are
    written."""
    if outs.dtype != torch.bfloat16 or not outs.is_cuda or not outs.is_contiguous() or outs.dim() != 4:
        raise ValueError("outs must be a contiguous bf16 CUDA tensor [n, T_q, Hq, D]")
    n, T_q, Hq, D = outs.shape
    if lses.dtype != torch.float32 or not lses.is_contiguous() or tuple(lses.shape) != (n, T_q, Hq):
        raise ValueError("lses must be a contiguous fp32 tensor [n, T_q, Hq]")
    if cu_q.dtype != torch.int32 or not cu_q.is_cuda or not cu_q.is_contiguous() or cu_q.dim() != 1:
        raise ValueError("cu_q must be a contiguous int32 CUDA tensor")
    if out is None:
        out = _made(stream, torch.empty, T_q, Hq, D, dtype=torch.bfloat16, device=outs.device)
    if lse is None:
        lse = _made(stream, torch.empty, T_q, Hq, dtype=torch.float32, device=outs.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (T_q, Hq, D) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor [T_q, Hq, D]")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (T_q, Hq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [T_q, Hq]")
    rc = lib().attn_merge_lse(int(n), outs.data_ptr(), lses.data_ptr(), int(T_q), cu_q.data_ptr(),
                              int(cu_q.numel() - 1), int(Hq), int(D), out.data_ptr(), lse.data_ptr(),
                              _stream_ptr(stream))
    _check(rc, "attn_merge_lse")
    return out, lse


def strerror(code: int) -> str:
    return lib().attn_strerror(int(code)).decode()


def _check(code: int, where: str):
    if code != ATTN_OK:
        raise AttnError(code, where)


# the current stream's handle without building a Stream object (3 us a call),
# where this torch has the shortcut
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_ptr(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_raw_device())
    return torch.cuda.current_stream().cuda_stream


def _made(stream, make, *args, **kw):
    """A result that the caller did not pass.  It is made, and filled, on the
    stream that the call runs on: a fill on another one could come after the
    kernel, and the allocator could hand the memory of a dropped result to that
    other stream while the kernel still writes it."""
    if stream is None:
        return make(*args, **kw)
    with _on(stream):
        return make(*args, **kw)


def _on(stream):
    """The context in which `stream` (torch's, or anything with a cuda_stream) is the current one."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


class _Turn(torch.autograd.Function):
    """A recorded rotation; its backward is the transpose (which is recorded in turn)."""

    @staticmethod
    def forward(ctx, x, pos, rope, grad):
        ctx.save_for_backward(pos)
        ctx.rope, ctx.grad = rope, grad
        return rope._launch(x, pos, None, grad, None)

    @staticmethod
    def backward(ctx, g):
        T, H, D = g.shape
        # a gradient may come expanded or permuted
        if (D > 1 and g.stride(2) != 1) or (H > 1 and g.stride(1) != D) or (T > 1 and g.stride(0) < H * D):
            g = g.contiguous()
        return ctx.rope.apply(g, *ctx.saved_tensors, grad=not ctx.grad), None, None, None


def rope_table(n_pairs, sections=None, *, base=10000.0, restart=False):
    """freqs, axes for Rope: pair i of n turns with base^(-i / n) radians per
    position.  sections: pairs per axis, in order (None: one axis for all);
    restart=True begins the frequencies anew in each section."""
    sections = [n_pairs] if sections is None else list(sections)
    if sum(sections) != n_pairs or min(sections) < 0:
        raise ValueError("sections must add up to n_pairs")
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    if restart:
        freqs = [float(base) ** (-i / n) for n in sections for i in range(n)]
    else:
        freqs = [float(base) ** (-i / n_pairs) for i in range(n_pairs)]
    return freqs, axes


class Rope:
    """Rotary positions with several axes (attn_rope_create).

    Rope(D, freqs, axes=None, *, n_axes=None, layout="half", scale=1.0):
    pair i of a head of D elements turns by pos[axes[i]] * freqs[i] radians;
    layout "half" pairs elements (i, i + n), "interleaved" (2 i, 2 i + 1);
    elements past the 2 n paired ones stay as they are; scale multiplies the
    cosines and sines.  Holds no device memory: one table serves every device
    and stream."""

    def __init__(self, D, freqs, axes=None, *, n_axes=None, layout="half", scale=1.0):
        self._h = None
        n = len(freqs)
        axes = [0] * n if axes is None else [int(a) for a in axes]
        if len(axes) != n:
            raise ValueError("axes must name one axis for each frequency")
        if layout not in ("half", "interleaved"):
            raise ValueError('layout must be "half" or "interleaved"')
        self.D, self.n_pairs, self.layout, self.scale = int(D), n, layout, float(scale)
        self.n_axes = int(n_axes) if n_axes is not None else max(axes, default=0) + 1
        h = ctypes.c_void_p()
        rc = lib().attn_rope_create(ctypes.byref(h), self.D, n, self.n_axes,
                                    (ctypes.c_double * max(n, 1))(*[float(f) for f in freqs]),
                                    (ctypes.c_int32 * max(n, 1))(*axes),
                                    ATTN_ROPE_HALF if layout == "half" else ATTN_ROPE_INTERLEAVED, self.scale)
        _check(rc, "attn_rope_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def apply(self, x, pos, out=None, *, grad=False, stream=None):
        """out = rope.apply(x, pos[, out, grad, stream]): rotate x [T, H, D]
        (bf16, fp16 or fp32; heads contiguous within a token, token stride
        free) by pos [n_axes, T] int32.  grad=True applies the transpose: x is
        the gradient of a rotated tensor, out that of its input.  out may be x
        itself; it is allocated packed when not given.  Where x requires grad,
        the rotation is recorded for autograd (not with out)."""
        grad = bool(grad)
        if torch.is_grad_enabled() and (getattr(x, "requires_grad", False) or getattr(out, "requires_grad", False)):
            if out is not None:
                raise ValueError("out records no gradient: leave it out, or call under no_grad")
            if stream is None:
                return _Turn.apply(x, pos, self, grad)
            with _on(stream):
                return _Turn.apply(x, pos, self, grad)
        return self._launch(x, pos, out, grad, stream)

    def _launch(self, x, pos, out, grad, stream):
        if self._h is None:
            raise AttnError(-3, "attn_rope_apply")
        if out is None:
            out = _made(stream, torch.empty_like, x, memory_format=torch.contiguous_format)
        rc = _marshal.rope_apply(self._h.value, self.D, self.n_axes, _raw_device(), x, pos, out, grad,
                                 _stream_ptr(stream))
        if rc:
            _check(rc, "attn_rope_apply")
        return out

    def close(self):
        if self._h is not None:
            lib().attn_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Plan:
    """A plan: launch shape, split count and scratch fixed from constants.

    Plan(B_max, s_max, Hq, Hkv, D, max_q=1, *, nsplit=0, block_n=0, variant=0,
    stages=0, combine=0, ctas=0, deterministic=0, wait_limit_us=0, test_stall=0) -- the
    keyword choices override the planner (0 = its own; deterministic=1 asks
    for static tile shares, -1 for run-time balancing of shared units;
    wait_limit_us bounds one device wait; test_stall=1 is the test hook of
    attn_overrides that makes the first call's merge waits run out).  Its calls
    are for inference: autograd does not record them."""

    def __init__(self, B_max, s_max, Hq, Hkv, D, max_q=1, *, nsplit=0, block_n=0, variant=0,
                 stages=0, combine=0, ctas=0, deterministic=0, wait_limit_us=0, test_stall=0):
        L = lib()
        h = ctypes.c_void_p()
        if nsplit or block_n or variant or stages or combine or ctas or deterministic or wait_limit_us or test_stall:
            o = Overrides(int(nsplit), int(block_n), int(variant), int(stages), int(combine), int(ctas),
                          int(deterministic), int(wait_limit_us), int(test_stall))
            rc = L.attn_plan_ex(ctypes.byref(h), int(B_max), int(s_max), int(Hq), int(Hkv), int(D),
                                int(max_q), ctypes.byref(o))
        else:
            rc = L.attn_plan(ctypes.byref(h), int(B_max), int(s_max), int(Hq), int(Hkv), int(D),
                             int(max_q))
        _check(rc, "attn_plan")
        self._h = h
        self.device = torch.cuda.current_device()
        self.info = self._info()
        # what the native marshalling checks tensors against
        self._args = (h.value, *(self.info[n] for n in ("B_max", "Hq", "Hkv", "D")), self.device, self.info["s_max"])

    def _info(self) -> dict:
        d = PlanDesc()
        _check(lib().attn_plan_info(self._h, ctypes.byref(d)), "attn_plan_info")
        return {name: getattr(d, name) for name, _ in PlanDesc._fields_}

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def run(self, q, k, v, cu_q, cu_k, out=None, lse=None, stream=None):
        """out, lse = plan.run(q, k, v, cu_q, cu_k[, out, lse, stream]).

        q [T_q, Hq, D] bf16 contiguous CUDA tensor; k / v [T_kv, Hkv, D] bf16
        CUDA tensors whose heads are contiguous within a token -- packed, or
        views into a larger buffer with a token stride (e.g. the halves of a
        fused [T, 2, Hkv, D] cache).  Goes through attn_run_rows;
        cu_q / cu_k int32 CUDA tensors with B_max + 1 entries; out / lse are
        allocated when not given (pass them for graph capture)."""
        out, lse = self._check_common(q, cu_q, cu_k, out, lse, "attn_run", stream)
        i = self.info
        for name, t in (("k", k), ("v", v)):
            if t.dtype != torch.bfloat16 or not t.is_cuda:
                raise TypeError(f"{name} must be a bf16 CUDA tensor")
            if t.dim() != 3 or t.shape[1:] != (i["Hkv"], i["D"]):
                raise ValueError(f"{name} must be [T_kv, {i['Hkv']}, {i['D']}]")
            if t.stride(2) != 1 or t.stride(1) != i["D"] or (t.shape[0] > 1 and t.stride(0) < i["Hkv"] * i["D"]):
                raise ValueError(f"{name} must keep each token's heads contiguous (strides (s, D, 1), s >= Hkv*D)")
        packed = i["Hkv"] * i["D"]
        ks = k.stride(0) if k.shape[0] > 1 else packed
        vs = v.stride(0) if v.shape[0] > 1 else packed
        rc = lib().attn_run_rows(self._h, q.data_ptr(), q.shape[0], k.data_ptr(), v.data_ptr(),
                                 min(k.shape[0], v.shape[0]), ks, vs, cu_q.data_ptr(), cu_k.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), _stream_ptr(stream))
        _check(rc, "attn_run")
        return out, lse

    def run_paged(self, q, k_cache, v_cache, block_table, cu_q, cu_k, out=None, lse=None, stream=None):
        """out, lse = plan.run_paged(q, k_cache, v_cache, block_table, cu_q, cu_k[, out, lse, stream]).

        k_cache / v_cache [num_pages, page_size, Hkv, D] bf16 CUDA tensors
        (each token's heads contiguous; token and page strides free, so the
        halves of a [num_pages, 2, page_size, Hkv, D] cache work);
        block_table [B_max, n] int32 CUDA tensor, row b listing the pages of
        sequence b in key order (n >= ceil(s_max / page_size), row stride
        free); cu_k supplies the key lengths only.  Goes through
        attn_run_paged_rows."""
        out, lse = self._check_common(q, cu_q, cu_k, out, lse, "attn_run_paged", stream)
        i = self.info
        shape = None
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype != torch.bfloat16 or not t.is_cuda:
                raise TypeError(f"{name} must be a bf16 CUDA tensor")
            if t.dim() != 4 or t.shape[2:] != (i["Hkv"], i["D"]):
                raise ValueError(f"{name} must be [num_pages, page_size, {i['Hkv']}, {i['D']}]")
            if t.stride(3) != 1 or t.stride(2) != i["D"]:
                raise ValueError(f"{name} must keep each token's heads contiguous")
            if shape is not None and (t.shape != shape or t.stride() != k_cache.stride()):
                raise ValueError("k_cache and v_cache must have the same shape and strides")
            shape = t.shape
        n_pages, page_size = int(shape[0]), int(shape[1])
        tok = k_cache.stride(1) if page_size > 1 else i["Hkv"] * i["D"]
        pstride = k_cache.stride(0) if n_pages > 1 else page_size * tok
        bt = block_table
        if bt.dtype != torch.int32 or not bt.is_cuda or bt.dim() != 2 or bt.shape[0] != i["B_max"] or bt.stride(1) != 1:
            raise ValueError("block_table must be an int32 CUDA tensor [B_max, n] with unit column stride")
        if bt.shape[1] * page_size < i["s_max"]:
            raise ValueError("block_table rows must cover s_max keys")
        rc = lib().attn_run_paged_rows(self._h, q.data_ptr(), q.shape[0], k_cache.data_ptr(), v_cache.data_ptr(),
                                       int(pstride), int(tok), page_size, n_pages, bt.data_ptr(), int(bt.stride(0)),
                                       cu_q.data_ptr(), cu_k.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       _stream_ptr(stream))
        _check(rc, "attn_run_paged")
        return out, lse

    def append_paged(self, k, v, k_cache, v_cache, block_table, cu_q, cu_k, *, q=None, pos=None, rope=None,
                     q_out=None, stream=None):
        """q_out = plan.append_paged(k, v, k_cache, v_cache, block_table, cu_q, cu_k, *[, q, pos, rope, q_out, stream]).

        Writes the new tokens' k / v [T_q, Hkv, D] (token stride free) to their
        places in the paged cache, rotating k, and q [T_q, Hq, D] into q_out,
        by rope at pos [n_axes, T_q] (rope None: no rotation).  cu_k counts the
        new tokens, as run_paged takes it.  q_out may be a packed q itself; it
        is allocated when q is given without it, and None without q.  Goes
        through attn_append_paged."""
        if self._h is None:
            raise AttnError(-5, "attn_append_paged")
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
        elif q_out is None:
            q_out = _made(stream, torch.empty_like, q, memory_format=torch.contiguous_format)
        rp = n_axes = 0
        if rope is not None:
            if rope._h is None:
                raise AttnError(-3, "attn_append_paged")
            if pos is None:
                raise ValueError("rope needs pos")
            if rope.D != self.info["D"]:
                raise ValueError("rope's head size is not the plan's")
            rp, n_axes = rope._h.value, rope.n_axes
        elif pos is not None:
            raise ValueError("pos without rope")
        rc = _marshal.append_paged(self._args, rp, n_axes, k, v, k_cache, v_cache, block_table, cu_q, cu_k, q, pos, q_out,
                                   _stream_ptr(stream))
        if rc:
            _check(rc, "attn_append_paged")
        return q_out

    def _key_weights(self, where, q, k, block_table, cu_q, cu_k, lse, weight_in, decay, out, seen, born, stream):
        if self._h is None:
            raise AttnError(-5, where)
        if out is None:
            like = weight_in if weight_in is not None else born
            i = self.info
            out = _made(stream, torch.zeros, (i["B_max"], i["Hkv"], i["s_max"] if like is None else like.shape[-1]),
                        dtype=torch.float32, device=q.device)
        rc = _marshal.key_weights(self._args, q, k, block_table, cu_q, cu_k, lse, weight_in, decay, out, seen, born,
                                  _stream_ptr(stream))
        if rc:
            _check(rc, where)
        return out

    def key_weights(self, q, k, cu_q, cu_k, lse, weight_in=None, *, decay=1.0, out=None, seen=None, born=None,
                    stream=None):
        """out = plan.key_weights(q, k, cu_q, cu_k, lse[, weight_in, decay, out, seen, born, stream]).

        The attention weight each key is given, added to decay * weight_in
        (both [B_max, Hkv, ld >= s_max] fp32; out may be weight_in; it is
        allocated, zero past the sequences, when not given).  q, k, cu_q, cu_k
        as in run(), lse its result.  With seen [B_max] and born [B_max, Hkv,
        ld] int32, the births of the present tokens are written.  Goes through
        attn_key_weights."""
        return self._key_weights("attn_key_weights", q, k, None, cu_q, cu_k, lse, weight_in, decay, out, seen, born,
                                 stream)

    def key_weights_paged(self, q, k_cache, block_table, cu_q, cu_k, lse, weight_in=None, *, decay=1.0, out=None,
                          seen=None, born=None, stream=None):
        """key_weights over a paged cache (k_cache and block_table as in
        run_paged).  Goes through attn_key_weights_paged."""
        if block_table is None:
            raise ValueError("block_table must be a tensor")
        return self._key_weights("attn_key_weights_paged", q, k_cache, block_table, cu_q, cu_k, lse, weight_in, decay,
                                 out, seen, born, stream)

    def evict_paged(self, weight, born, seen, keep, k_cache, v_cache, block_table, cu_k, *, sink=0, recent=0,
                    weight_out=None, born_out=None, cu_k_out=None, stream=None):
        """weight_out, born_out, cu_k_out = plan.evict_paged(weight, born, seen, keep, k_cache, v_cache, block_table,
        cu_k, *[, sink, recent, weight_out, born_out, cu_k_out, stream]).

        Cuts every sequence to min(length, keep[b]) keys in each KV head, the
        ones of the highest weight, those born among the first `sink` or last
        `recent` of its seen[b] tokens first; K and V rows move within the
        cache, and the ledger (weight fp32 and born int32, [B_max, Hkv, ld])
        with them, in place unless weight_out / born_out are given.  cu_k_out
        [B_max + 1] gets the offsets of the new lengths.  Goes through
        attn_evict_paged."""
        if self._h is None:
            raise AttnError(-5, "attn_evict_paged")
        if weight_out is None:
            weight_out = weight
        if born_out is None:
            born_out = born
        if cu_k_out is None:
            cu_k_out = _made(stream, torch.empty_like, cu_k)
        rc = _marshal.evict_paged(self._args, weight, born, seen, keep, k_cache, v_cache, block_table, cu_k, sink, recent,
                                  weight_out, born_out, cu_k_out, _stream_ptr(stream))
        if rc:
            _check(rc, "attn_evict_paged")
        return weight_out, born_out, cu_k_out

    def _check_common(self, q, cu_q, cu_k, out, lse, where, stream):
        if self._h is None:
            raise AttnError(-5, where)
        i = self.info
        if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
            raise TypeError("q must be a contiguous bf16 CUDA tensor")
        if q.dim() != 3 or q.shape[1:] != (i["Hq"], i["D"]):
            raise ValueError(f"q must be [T_q, {i['Hq']}, {i['D']}]")
        for name, t in (("cu_q", cu_q), ("cu_k", cu_k)):
            if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != i["B_max"] + 1:
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of B_max+1 entries")
        if out is None:
            out = _made(stream, torch.empty_like, q)
        if lse is None:
            lse = _made(stream, torch.empty, q.shape[0], i["Hq"], dtype=torch.float32, device=q.device)
        if out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be a contiguous bf16 tensor shaped like q")
        if lse.dtype != torch.float32 or lse.shape != (q.shape[0], i["Hq"]) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous fp32 tensor [T_q, Hq]")
        return out, lse

    def check_error(self, stream=None) -> int:
        """Synchronise, then read and clear the sticky device error bits."""
        f = ctypes.c_uint32(0)
        _check(lib().attn_check_error(self._h, _stream_ptr(stream), ctypes.byref(f)), "attn_check_error")
        return int(f.value)

    def close(self):
        if self._h is not None:
            lib().attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
