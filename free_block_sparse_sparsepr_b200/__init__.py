"""Python binding of the SparsePR attention library (libsparsepr.so, sm_100a).

Argument marshalling only: every step of the call runs in the CUDA kernels
behind the C ABI declared in include/sparsepr.h. PyTorch provides device
memory and streams. There is no CPU fallback: if the shared library is
missing, importing the binding's entry points raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import re

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libsparsepr.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "sparsepr.h")

FLAG_HARD_DROP_ONLY = 1 << 0
FLAG_RIDGE_ONLY = 1 << 1
FLAG_RBAR_UNPROJECTED = 1 << 2
FLAG_UNIFORM_WEIGHTS = 1 << 3
FLAG_TOPMASS = 1 << 4
FLAG_PROBES_UNIFORM = 1 << 5     # ablation: probes on a uniform grid of the original token order
FLAG_PROBES_RANDOM = 1 << 6      # ablation: probes drawn at random (seeded SplitMix64)
FLAG_SEMANTIC_PARTITION = 1 << 7  # ablation: k-means on the raw keys and the raw mean query
FLAG_STAGE_TIMING = 1 << 8
FLAG_TEST_STALL = 1 << 9          # test only: the dense kernel's first bounded wait runs out
FLAG_TEST_STALL_BWD = 1 << 11     # test only: the same for the backward passes' kernel
FLAG_BWD_SPLIT_DS = 1 << 10       # backward passes: dS as two bf16 parts in dQ, at the price of an eighth product

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "workspace allocation failed",
          4: "CUDA error", 5: "device wait timed out", 6: "device-side check failed"}

_p = ctypes.c_void_p


class Config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("N", ctypes.c_int),
                ("d", ctypes.c_int), ("block", ctypes.c_int), ("Gk", ctypes.c_int), ("Gq", ctypes.c_int),
                ("rK", ctypes.c_int), ("rQ", ctypes.c_int), ("M", ctypes.c_int), ("r", ctypes.c_int),
                ("kmeans_iters", ctypes.c_int), ("lam", ctypes.c_float), ("rho_exec", ctypes.c_float),
                ("flags", ctypes.c_uint), ("seed", ctypes.c_ulonglong)]


class Partition(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("kgroup", "qgroup", "kperm", "koff", "qperm", "qoff", "kcent", "radial",
                                  "probe", "probe_pos", "weights", "features", "topmass")]


class Route(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("rowptr", "kg", "scores", "pairs")]


class Fit(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("obar", "Rbar", "A", "U", "Bm", "c0", "rank", "R", "Odense", "Osp")]


class Stats(ctypes.Structure):
    _fields_ = [("route_density", ctypes.c_double), ("rho_exec", ctypes.c_double),
                ("useful_pairs", ctypes.c_double), ("stage_ms", ctypes.c_float * 8),
                ("device_status", ctypes.c_int)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int),
                ("layout", ctypes.c_int), ("axes", ctypes.c_int), ("dtype", ctypes.c_int), ("width", ctypes.c_int * 3),
                ("stride_b", ctypes.c_longlong), ("stride_n", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("pos_stride_b", ctypes.c_longlong), ("amplitude", ctypes.c_double), ("freq", ctypes.c_double * 64)]


class SparsePRError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({code})")
        self.code = code


SHARED_ROWS = 8   # rows per query group in the shared-support diagnostic (SPARSEPR_SHARED_ROWS)

_lib = None


def header_functions() -> list[str]:
    """Names of the entry points that include/sparsepr.h declares."""
    txt = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+(sparsepr_\w+)\s*\(", txt, re.M)))


def load_library() -> ctypes.CDLL:
    """Load libsparsepr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m free_block_sparse_sparsepr_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    st = ctypes.c_int
    H = _p
    sig = {
        "sparsepr_status_string": (ctypes.c_char_p, [st]),
        "sparsepr_version": (ctypes.c_int, []),
        "sparsepr_create": (st, [ctypes.POINTER(Config), ctypes.POINTER(_p)]),
        "sparsepr_destroy": (st, [H]),
        "sparsepr_workspace_bytes": (st, [H, ctypes.POINTER(ctypes.c_size_t)]),
        "sparsepr_partition": (st, [H, _p, _p, ctypes.POINTER(Partition), _p]),
        "sparsepr_route": (st, [H, _p, ctypes.POINTER(Partition), ctypes.POINTER(Route), _p]),
        "sparsepr_permute": (st, [H, _p, _p, _p, ctypes.POINTER(Partition), _p, _p, _p, _p]),
        "sparsepr_blocksparse_attn": (st, [H, _p, _p, _p, ctypes.POINTER(Partition), ctypes.POINTER(Route),
                                           _p, _p, _p]),
        "sparsepr_probe_fit": (st, [H, _p, _p, _p, ctypes.POINTER(Partition), _p, ctypes.POINTER(Fit), _p]),
        "sparsepr_writeback": (st, [H, ctypes.POINTER(Partition), _p, ctypes.POINTER(Fit), _p, _p]),
        "sparsepr_attention": (st, [H, _p, _p, _p, _p, _p]),
        "sparsepr_attention_host": (st, [H, _p, _p, _p, _p, _p]),
        "sparsepr_dense_attn": (st, [H, _p, _p, _p, _p, _p]),
        "sparsepr_dense_attn_lse": (st, [H, _p, _p, _p, _p, _p, _p]),
        "sparsepr_attn_bwd_workspace": (st, [H, ctypes.POINTER(ctypes.c_size_t)]),
        "sparsepr_dense_attn_bwd_workspace": (st, [H, ctypes.POINTER(ctypes.c_size_t)]),
        "sparsepr_dense_attn_bwd": (st, [H] + [_p] * 10 + [ctypes.c_size_t, _p]),
        "sparsepr_blocksparse_attn_bwd": (st, [H, _p, _p, _p, ctypes.POINTER(Partition), ctypes.POINTER(Route)]
                                          + [_p] * 7 + [ctypes.c_size_t, _p]),
        "sparsepr_rope": (st, [ctypes.POINTER(RopeConfig), _p, _p, _p, _p]),
        "sparsepr_rope_bwd": (st, [ctypes.POINTER(RopeConfig), _p, _p, _p, _p]),
        "sparsepr_get_stats": (st, [H, ctypes.POINTER(Stats)]),
        "sparsepr_device_status": (st, [H, ctypes.POINTER(ctypes.c_int)]),
        "sparsepr_last_launch_count": (st, [H, ctypes.POINTER(ctypes.c_int)]),
        "sparsepr_set_stage_events": (st, [H, ctypes.c_void_p]),
        "sparsepr_shared_support_workspace": (st, [H, ctypes.POINTER(ctypes.c_size_t),
                                                   ctypes.POINTER(ctypes.c_size_t)]),
        "sparsepr_shared_support": (st, [H, _p, _p, ctypes.POINTER(Partition), _p, _p, _p, ctypes.c_size_t, _p]),
        "sparsepr_affine_diagnostics_workspace": (st, [H, ctypes.POINTER(ctypes.c_size_t)]),
        "sparsepr_affine_diagnostics": (st, [H, _p, _p, _p, _p, ctypes.c_size_t, _p]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _check(fn: str, code: int):
    if code != 0:
        raise SparsePRError(fn, code)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context with `device` current and, if `stream` is given, that stream current too, so that
    memory taken inside belongs to the stream that uses it."""
    import torch

    if stream is None and device.index == torch.cuda.current_device():
        return _HERE
    if stream is not None and not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"stream on {stream.device} for tensors on {device}")
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(device))
    if stream is not None:
        ctx.enter_context(torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int)
                                            else stream))
    return ctx


def _stream_on(device, stream) -> int:
    """_stream on a given device (looking that device up anew costs microseconds a call)."""
    if stream is None:
        return _current_raw_stream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _current_raw_stream(index: int) -> int:
    """The current stream's pointer; torch's Stream object costs a microsecond where its raw getter is not there."""
    global _current_raw_stream
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_raw_stream = raw or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current_raw_stream(index)


def _want(name, t, shape, dtype, device):
    """Refuse a tensor argument that the C ABI would read or write wrongly."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


class _DevArray:
    """Zero-copy __cuda_array_interface__ view of handle-owned device memory."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"data": (ptr, False), "shape": tuple(shape), "typestr": typestr,
                                         "version": 3, "strides": None}


def device_view(ptr: int, shape, dtype):
    """torch tensor viewing `ptr` (valid until the handle overwrites or frees it)."""
    import torch

    typestr = {torch.float32: "<f4", torch.int32: "<i4", torch.int64: "<i8", torch.int16: "<i2"}[dtype]
    return torch.as_tensor(_DevArray(ptr, shape, typestr), device="cuda")


class SparsePR:
    """One configured SparsePR call on the current CUDA device (owns the workspace).

    No call is an autograd function: results carry no graph whatever their inputs require. dense_attn and
    blocksparse_attn have their gradients in dense_attn_bwd and blocksparse_attn_bwd, the other steps none."""

    def __init__(self, B, Hq, Hkv, N, d, Gk, Gq, block=128, rK=48, rQ=64, M=64, r=16, kmeans_iters=10,
                 lam=0.1, rho_exec=0.22, flags=0, seed=0):
        self.lib = load_library()
        self.cfg = Config(B, Hq, Hkv, N, d, block, Gk, Gq, rK, rQ, M, r, kmeans_iters, lam, rho_exec, flags,
                          seed)
        h = _p()
        _check("sparsepr_create", self.lib.sparsepr_create(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.h = h
        self._bwd_bytes = {"sparsepr_dense_attn_bwd": self.attn_bwd_workspace_bytes(dense_only=True),
                           "sparsepr_blocksparse_attn_bwd": self.attn_bwd_workspace_bytes()}
        try:
            import torch

            self.device = torch.device("cuda", torch.cuda.current_device())     # the handle's
        except (ImportError, AssertionError, RuntimeError):      # no torch, or one without CUDA: host buffers only
            self.device = None

    @classmethod
    def from_workload(cls, w, flags=0, **kw):
        args = dict(B=w.B, Hq=w.Hq, Hkv=w.Hkv, N=w.N, d=w.d, Gk=w.Gk, Gq=w.Gq, block=w.block, rK=w.rK,
                    rQ=w.rQ, M=w.M, r=w.r, kmeans_iters=w.kmeans_iters, lam=w.lam, rho_exec=w.rho,
                    flags=flags, seed=w.seed)
        args.update(kw)
        return cls(**args)

    # ------------------------------------------------------------------ lifetime
    def close(self):
        if getattr(self, "h", None):
            self.lib.sparsepr_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def P(self):
        return self.cfg.B * self.cfg.Hkv

    @property
    def Hp(self):
        return self.cfg.B * self.cfg.Hq

    def workspace_bytes(self) -> int:
        n = ctypes.c_size_t()
        _check("sparsepr_workspace_bytes", self.lib.sparsepr_workspace_bytes(self.h, ctypes.byref(n)))
        return n.value

    # ------------------------------------------------------------------ steps
    def partition(self, Q, K, stream=None) -> Partition:
        out = Partition()
        _check("sparsepr_partition", self.lib.sparsepr_partition(self.h, _ptr(Q), _ptr(K), ctypes.byref(out),
                                                                 _stream(stream)))
        return out

    def route(self, Q, part: Partition, stream=None) -> Route:
        out = Route()
        _check("sparsepr_route", self.lib.sparsepr_route(self.h, _ptr(Q), ctypes.byref(part), ctypes.byref(out),
                                                         _stream(stream)))
        return out

    def permute(self, Q, K, V, part: Partition, Qp=None, Kp=None, Vp=None, stream=None):
        _check("sparsepr_permute", self.lib.sparsepr_permute(self.h, _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(part),
                                                             _ptr(Qp), _ptr(Kp), _ptr(Vp), _stream(stream)))

    def blocksparse_attn(self, Qp, Kp, Vp, part: Partition, route: Route, Osp, lse=None, stream=None):
        _check("sparsepr_blocksparse_attn",
               self.lib.sparsepr_blocksparse_attn(self.h, _ptr(Qp), _ptr(Kp), _ptr(Vp), ctypes.byref(part),
                                                  ctypes.byref(route), _ptr(Osp), _ptr(lse), _stream(stream)))

    def probe_fit(self, Q, K, V, part: Partition, Osp, stream=None) -> Fit:
        out = Fit()
        _check("sparsepr_probe_fit", self.lib.sparsepr_probe_fit(self.h, _ptr(Q), _ptr(K), _ptr(V),
                                                                 ctypes.byref(part), _ptr(Osp), ctypes.byref(out),
                                                                 _stream(stream)))
        return out

    def shared_support(self, Q, K, part: Partition, max_workspace_bytes: int = 8 << 30, stream=None):
        """Shared-route support diagnostic: (row_frac [B*Hkv, Gq, SHARED_ROWS], union_frac
        [B*Hkv, Gq]) as fp32 device tensors; the workspace (device memory through torch) holds
        as many KV heads' logits per pass as max_workspace_bytes allows (at least one)."""
        import torch

        lo, hi = ctypes.c_size_t(), ctypes.c_size_t()
        _check("sparsepr_shared_support_workspace",
               self.lib.sparsepr_shared_support_workspace(self.h, ctypes.byref(lo), ctypes.byref(hi)))
        nbytes = max(lo.value, min(hi.value, max_workspace_bytes))
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        P = self.cfg.B * self.cfg.Hkv
        row_frac = torch.empty((P, self.cfg.Gq, SHARED_ROWS), dtype=torch.float32, device="cuda")
        union_frac = torch.empty((P, self.cfg.Gq), dtype=torch.float32, device="cuda")
        _check("sparsepr_shared_support",
               self.lib.sparsepr_shared_support(self.h, _ptr(Q), _ptr(K), ctypes.byref(part), _ptr(row_frac),
                                                _ptr(union_frac), _ptr(ws), nbytes, _stream(stream)))
        return row_frac, union_frac

    def affine_diagnostics(self, Q, K, V, stream=None):
        """Affine-explainable fraction and affine-orthogonal energy of each query head's hard-drop
        residual (dense output minus the uncorrected sparse output), as a [B*Hq, 2] fp64 device
        tensor; runs the partition, routing, sparse attention and the dense baseline."""
        import torch

        part = self.partition(Q, K, stream)
        route = self.route(Q, part, stream)
        Qp, Kp, Vp, Osp = (torch.empty_like(t) for t in (Q, K, V, Q))
        self.permute(Q, K, V, part, Qp, Kp, Vp, stream)
        self.blocksparse_attn(Qp, Kp, Vp, part, route, Osp, None, stream)
        Os, Od = torch.empty_like(Q), torch.empty_like(Q)
        self.writeback(part, Osp, None, Os, stream)
        self.dense_attn(Q, K, V, Od, stream)
        n = ctypes.c_size_t()
        _check("sparsepr_affine_diagnostics_workspace",
               self.lib.sparsepr_affine_diagnostics_workspace(self.h, ctypes.byref(n)))
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        out = torch.empty((self.cfg.B * self.cfg.Hq, 2), dtype=torch.float64, device="cuda")
        _check("sparsepr_affine_diagnostics",
               self.lib.sparsepr_affine_diagnostics(self.h, _ptr(Os), _ptr(Od), _ptr(out), _ptr(ws), n.value,
                                                    _stream(stream)))
        return out, Os, Od

    def writeback(self, part: Partition, Osp, fit: Fit | None, O, stream=None):
        _check("sparsepr_writeback", self.lib.sparsepr_writeback(self.h, ctypes.byref(part), _ptr(Osp),
                                                                 ctypes.byref(fit) if fit is not None else None,
                                                                 _ptr(O), _stream(stream)))

    def attention(self, Q, K, V, O=None, stream=None):
        if O is None:
            import torch

            O = torch.empty_like(Q)
        _check("sparsepr_attention", self.lib.sparsepr_attention(self.h, _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                                                 _stream(stream)))
        return O

    def attention_host(self, Q, K, V, O, stream=None):
        """Whole call on HOST tensors (pinned for full copy speed); synchronises the stream."""
        _check("sparsepr_attention_host", self.lib.sparsepr_attention_host(self.h, _ptr(Q), _ptr(K), _ptr(V),
                                                                           _ptr(O), _stream(stream)))
        return O

    def dense_attn(self, Q, K, V, O=None, stream=None, lse=None):
        """Dense attention; with `lse` (fp32 [B, Hq, N]) the rows' log softmax denominators are written too."""
        if lse is not None:
            import torch

            _want("lse", lse, (self.cfg.B, self.cfg.Hq, self.cfg.N), torch.float32, self.device)
        if O is None:
            import torch

            O = torch.empty_like(Q)
        _check("sparsepr_dense_attn", self.lib.sparsepr_dense_attn_lse(self.h, _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                                                       _ptr(lse), _stream(stream)))
        return O

    # ------------------------------------------------------------------ backward passes
    def attn_bwd_workspace_bytes(self, dense_only=False) -> int:
        """Workspace of either backward pass, or what dense_attn_bwd alone needs."""
        n = ctypes.c_size_t()
        fn = "sparsepr_dense_attn_bwd_workspace" if dense_only else "sparsepr_attn_bwd_workspace"
        _check(fn, getattr(self.lib, fn)(self.h, ctypes.byref(n)))
        return n.value

    def _bwd(self, name, call, Q, K, V, O, lse, dO, dQ, dK, dV, need_dq, need_dkv, workspace, stream):
        import torch

        c = self.cfg
        B, Hq, Hkv, N, d = c.B, c.Hq, c.Hkv, c.N, c.d
        qs, ks = (B, Hq, N, d), (B, Hkv, N, d)
        if not need_dq and not need_dkv:
            raise ValueError("no gradient asked for")
        if (dQ is not None and not need_dq) or ((dK is not None or dV is not None) and not need_dkv):
            raise ValueError("an output is given for a gradient that is not asked for")
        bf16, dev = torch.bfloat16, self.device
        _want("Q", Q, qs, bf16, dev)
        _want("K", K, ks, bf16, dev)
        _want("V", V, ks, bf16, dev)
        _want("O", O, qs, bf16, dev)
        _want("lse", lse, (B, Hq, N), torch.float32, dev)
        _want("dO", dO, qs, bf16, dev)
        for label, t, shape in (("dQ", dQ, qs), ("dK", dK, ks), ("dV", dV, ks)):
            if t is not None:
                _want(label, t, shape, bf16, dev)
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace: expected contiguous memory on {dev}")
        with _on(dev, stream):
            if need_dq and dQ is None:
                dQ = torch.empty_like(Q)
            if need_dkv:
                dK = torch.empty_like(K) if dK is None else dK
                dV = torch.empty_like(V) if dV is None else dV
            if workspace is None:
                workspace = torch.empty(self._bwd_bytes[name], dtype=torch.uint8, device=dev)
            _check(name, call(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), lse.data_ptr(), dO.data_ptr(),
                              _ptr(dQ), _ptr(dK), _ptr(dV), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream_on(dev, stream)))
        return dQ, dK, dV

    def dense_attn_bwd(self, Q, K, V, O, lse, dO, dQ=None, dK=None, dV=None, need_dq=True, need_dkv=True,
                       workspace=None, stream=None):
        """Gradients (dQ, dK, dV) of dense_attn from its output O and lse and the gradient dO of O (None for
        one that need_dq / need_dkv leave out). workspace: attn_bwd_workspace_bytes(dense_only=True) of device
        memory that a program may keep; None takes it from torch for this call."""
        return self._bwd("sparsepr_dense_attn_bwd",
                         lambda *a: self.lib.sparsepr_dense_attn_bwd(self.h, *a),
                         Q, K, V, O, lse, dO, dQ, dK, dV, need_dq, need_dkv, workspace, stream)

    def blocksparse_attn_bwd(self, Qp, Kp, Vp, part: Partition, route: Route, Osp, lse, dOsp, dQ=None, dK=None,
                             dV=None, need_dq=True, need_dkv=True, workspace=None, stream=None):
        """Gradients of permute followed by blocksparse_attn, with the partition and the route held constant (and of
        writeback without a fit; the correction of one with a fit, or of `attention`, has no gradient here):
        group-major Qp, Kp, Vp, Osp, lse and dOsp in (dOsp: permute of the original-order gradient), dQ, dK
        and dV in the original token order out. workspace: attn_bwd_workspace_bytes(). A partition or route
        whose buffers the handle owns is overwritten by the handle's next call: keep copies (partition_views,
        route_views) across calls."""
        return self._bwd("sparsepr_blocksparse_attn_bwd",
                         lambda q, k, v, *a: self.lib.sparsepr_blocksparse_attn_bwd(
                             self.h, q, k, v, ctypes.byref(part), ctypes.byref(route), *a),
                         Qp, Kp, Vp, Osp, lse, dOsp, dQ, dK, dV, need_dq, need_dkv, workspace, stream)

    # ------------------------------------------------------------------ introspection
    def stats(self) -> dict:
        s = Stats()
        _check("sparsepr_get_stats", self.lib.sparsepr_get_stats(self.h, ctypes.byref(s)))
        names = ["partition", "route", "permute", "attention", "probe_fit", "writeback", "unused", "total"]
        return {"route_density": s.route_density, "rho_exec": s.rho_exec, "useful_pairs": s.useful_pairs,
                "stage_ms": {n: s.stage_ms[i] for i, n in enumerate(names) if n != "unused"},
                "device_status": s.device_status}

    def device_status(self) -> int:
        v = ctypes.c_int()
        _check("sparsepr_device_status", self.lib.sparsepr_device_status(self.h, ctypes.byref(v)))
        return v.value

    def set_stage_events(self, events):
        """Record the next calls' 7 stage boundaries into these torch.cuda.Event objects (None: stop)."""
        if events is None:
            _check("sparsepr_set_stage_events", self.lib.sparsepr_set_stage_events(self.h, None))
            return
        assert len(events) == 7
        arr = (ctypes.c_void_p * 7)(*[e.cuda_event for e in events])
        self._events_keepalive = (events, arr)
        _check("sparsepr_set_stage_events", self.lib.sparsepr_set_stage_events(self.h, ctypes.cast(arr, ctypes.c_void_p)))

    def last_launch_count(self) -> int:
        v = ctypes.c_int()
        _check("sparsepr_last_launch_count", self.lib.sparsepr_last_launch_count(self.h, ctypes.byref(v)))
        return v.value

    # ------------------------------------------------------------------ views of handle-owned buffers
    def partition_views(self, part: Partition) -> dict:
        import torch

        c, P, N = self.cfg, self.P, self.cfg.N
        M = 0 if (c.flags & FLAG_HARD_DROP_ONLY) else c.M
        v = {"kperm": device_view(part.kperm, (P, N), torch.int32), "koff": device_view(part.koff, (P, c.Gk + 1), torch.int32),
             "qperm": device_view(part.qperm, (P, N), torch.int32), "qoff": device_view(part.qoff, (P, c.Gq + 1), torch.int32),
             "kgroup": device_view(part.kgroup, (P, N), torch.int32), "qgroup": device_view(part.qgroup, (P, N), torch.int32),
             "kcent": device_view(part.kcent, (P, c.Gk, c.d), torch.float32),
             "radial": device_view(part.radial, (P, N), torch.float32)}
        if part.features:
            DP = c.d if c.flags & FLAG_SEMANTIC_PARTITION else (c.rK + 15) // 16 * 16
            v["features"] = device_view(part.features, (P, N, DP), torch.float32)
        if part.topmass:
            v["topmass"] = device_view(part.topmass, (P, c.rK), torch.float32)
        if M:
            v["probe"] = device_view(part.probe, (P, M), torch.int32)
            v["probe_pos"] = device_view(part.probe_pos, (P, M), torch.int32)
            v["weights"] = device_view(part.weights, (P, M), torch.float32)
        return v

    def route_views(self, route: Route) -> dict:
        import torch

        c, P = self.cfg, self.P
        return {"rowptr": device_view(route.rowptr, (P, c.Gq + 1), torch.int32),
                "kg": device_view(route.kg, (P, c.Gq * c.Gk), torch.int32),
                "scores": device_view(route.scores, (P, c.Gq, c.Gk), torch.float32),
                "pairs": device_view(route.pairs, (P,), torch.int64)}

    def fit_views(self, fit: Fit) -> dict:
        import torch

        c, Hp = self.cfg, self.Hp
        return {"obar": device_view(fit.obar, (Hp, c.d), torch.float32),
                "Rbar": device_view(fit.Rbar, (Hp, c.d), torch.float32),
                "A": device_view(fit.A, (Hp, c.d, c.d), torch.float32),
                "U": device_view(fit.U, (Hp, c.d, c.r), torch.float32),
                "Bm": device_view(fit.Bm, (Hp, c.r, c.d), torch.float32),
                "c0": device_view(fit.c0, (Hp, c.r), torch.float32),
                "rank": device_view(fit.rank, (Hp,), torch.int32),
                "R": device_view(fit.R, (Hp, c.M, c.d), torch.float32),
                "Odense": device_view(fit.Odense, (Hp, c.M, c.d), torch.float32),
                "Osp": device_view(fit.Osp, (Hp, c.M, c.d), torch.float32)}


class Rope:
    """Rotary positions of Q and K: from a model's token-major tensors into the head-major bf16
    layout of the attention calls (`forward`), and the gradient back (`backward`). No autograd function:
    results carry no graph whatever their inputs require, the gradient is a call of its own.

    widths  rotated elements of each axis, even: (w,) for a sequence (w < d rotates part of the head),
            (frame, row, column) for video tokens
    layout  "interleaved": pairs (2i, 2i + 1) of an axis' section; "half": pairs (i, i + w/2)
    scaling "none": freq_i = base^(-2i/w)
            "linear": freq_i / factor (positions interpolated into the trained range)
            "ntk": base * factor^(w / (w - 2)) in place of base
            "yarn": pairs that turn at least beta_fast times within trained_length keep freq_i, those that
            turn at most beta_slow times take freq_i / factor, a linear ramp over the pair index between;
            turned pairs are multiplied by 0.1 ln(factor) + 1 where factor is above 1
    amplitude  factor of the turned pairs; None: the scaling's own"""

    def __init__(self, d, widths, layout="half", base=10000.0, scaling="none", factor=1.0, trained_length=None,
                 beta_fast=32.0, beta_slow=1.0, amplitude=None):
        widths = tuple(int(w) for w in widths)
        if d not in (64, 128):
            raise ValueError(f"head dimension {d}: 64 or 128")
        if not 1 <= len(widths) <= 3 or any(w < 2 or w % 2 for w in widths) or sum(widths) > d:
            raise ValueError(f"widths {widths}: one to three even widths of at least 2, at most {d} together")
        if layout not in ("interleaved", "half"):
            raise ValueError(f"layout {layout!r}: 'interleaved' or 'half'")
        if not base > 1.0 or not factor > 0.0:
            raise ValueError("base must be above 1 and factor above 0")
        if scaling == "yarn" and not (trained_length and trained_length > 0 and beta_fast > beta_slow > 0.0):
            raise ValueError("yarn needs trained_length and beta_fast > beta_slow > 0")
        self.d, self.widths = d, widths
        self.layout = 0 if layout == "interleaved" else 1
        self.freq = [f for w in widths for f in self._frequencies(w, float(base), scaling, float(factor),
                                                                  trained_length, beta_fast, beta_slow)]
        if amplitude is None:
            amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
        self.amplitude = float(amplitude)
        self.lib = load_library()
        self._plans = {}
        import torch

        self._int32, self._bf16 = torch.int32, torch.bfloat16

    @staticmethod
    def _frequencies(w, base, scaling, factor, trained, beta_fast, beta_slow):
        if scaling == "ntk":
            base = base * factor ** (w / max(w - 2, 1))
        freq = [base ** (-2.0 * i / w) for i in range(w // 2)]
        if scaling in ("none", "ntk"):
            return freq
        if scaling == "linear":
            return [f / factor for f in freq]
        if scaling != "yarn":
            raise ValueError(f"scaling {scaling!r}: 'none', 'linear', 'ntk' or 'yarn'")

        def pair(turns):   # index at which a pair turns that often within the trained length
            return w * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), w - 1)
        slow = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(w // 2)]
        return [f / factor * s + f * (1.0 - s) for f, s in zip(freq, slow)]

    def _config(self, model, pos):
        """The call's plan for this shape, strides and type, checked when first met, and the head-major shape."""
        key = (model.shape, model.stride(), model.dtype, pos.shape)
        c = self._plans.get(key)
        if c is None:
            c = self._plan(model, pos)
            if len(self._plans) >= 256:
                self._plans.clear()
            self._plans[key] = c
        if pos.dtype is not self._int32 or pos.device != model.device or not pos.is_contiguous() or not model.is_cuda:
            raise ValueError(f"positions: expected a contiguous int32 tensor on {model.device} (a CUDA device), got "
                             f"{pos.dtype} on {pos.device}")
        return c

    def _plan(self, model, pos):
        import torch

        if model.dim() != 4 or model.shape[3] != self.d or model.stride(3) != 1 or 0 in model.shape:
            raise ValueError(f"expected a token-major tensor [B, N, H, {self.d}] with contiguous heads, got "
                             f"{tuple(model.shape)} with strides {model.stride()}")
        if model.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"token-major tensor of {model.dtype}: bfloat16 or float32")
        B, N, H, d = model.shape
        axes = len(self.widths)
        if tuple(pos.shape) not in ((N, axes), (B, N, axes)):
            raise ValueError(f"positions: expected [{N}, {axes}] or [{B}, {N}, {axes}], got {tuple(pos.shape)}")
        c = RopeConfig(B, H, N, d, self.layout, axes, 1 if model.dtype == torch.float32 else 0,
                       (ctypes.c_int * 3)(*self.widths), *model.stride()[:3], N * axes if pos.dim() == 3 else 0,
                       self.amplitude, (ctypes.c_double * 64)(*self.freq))
        return ctypes.byref(c), (B, H, N, d)

    def forward(self, x, pos, out=None, stream=None):
        """x [B, N, H, d] bf16 or fp32 (any strides of 16-byte multiples, e.g. a slice of a fused projection)
        turned by int32 positions [N, axes] or [B, N, axes]: bf16 [B, H, N, d]."""
        cfg, shape = self._config(x, pos)
        dev, bf16 = x.device, self._bf16
        with _on(dev, stream):
            if out is None:
                out = x.new_empty(shape) if x.dtype is bf16 else x.new_empty(shape, dtype=bf16)
            else:
                _want("out", out, shape, bf16, dev)
            _check("sparsepr_rope", self.lib.sparsepr_rope(cfg, x.data_ptr(), pos.data_ptr(), out.data_ptr(),
                                                           _stream_on(dev, stream)))
        return out

    def backward(self, dy, pos, out=None, dtype=None, stream=None):
        """Gradient dy bf16 [B, H, N, d] of forward's output -> gradient of x, [B, N, H, d] of `dtype` (bf16
        unless given) or written into `out` (any strides of 16-byte multiples whose rows do not overlap)."""
        if dy.dim() != 4 or not dy.is_cuda or out is not None and dtype not in (None, out.dtype):
            raise ValueError("dy must be [B, H, N, d] on a CUDA device, and dtype that of out")
        B, H, N, d = dy.shape
        dev = dy.device
        _want("dy", dy, (B, H, N, d), self._bf16, dev)
        with _on(dev, stream):
            if out is None:
                out = dy.new_empty((B, N, H, d)) if dtype is None else dy.new_empty((B, N, H, d), dtype=dtype)
            elif tuple(out.shape) != (B, N, H, d) or out.device != dev:
                raise ValueError(f"out: expected [{B}, {N}, {H}, {d}] on {dev}, got {tuple(out.shape)} on {out.device}")
            cfg, _ = self._config(out, pos)
            _check("sparsepr_rope_bwd", self.lib.sparsepr_rope_bwd(cfg, dy.data_ptr(), pos.data_ptr(), out.data_ptr(),
                                                                   _stream_on(dev, stream)))
        return out


def partition_from_tensors(t: dict) -> Partition:
    """Partition struct pointing at caller-owned device tensors (for handing a partition in)."""
    p = Partition()
    for name in ("kgroup", "qgroup", "kperm", "koff", "qperm", "qoff", "kcent", "radial", "probe", "probe_pos",
                 "weights", "features"):
        if name in t and t[name] is not None:
            setattr(p, name, t[name].data_ptr())
    return p


def route_from_tensors(t: dict) -> Route:
    r = Route()
    for name in ("rowptr", "kg", "scores", "pairs"):
        if name in t and t[name] is not None:
            setattr(r, name, t[name].data_ptr())
    return r


__all__ = ["SparsePR", "Rope", "RopeConfig", "SparsePRError", "Config", "Partition", "Route", "Fit", "Stats", "load_library",
           "header_functions", "partition_from_tensors", "route_from_tensors", "device_view", "LIB_PATH",
           "FLAG_HARD_DROP_ONLY", "FLAG_RIDGE_ONLY", "FLAG_RBAR_UNPROJECTED", "FLAG_UNIFORM_WEIGHTS", "FLAG_TOPMASS",
           "FLAG_PROBES_UNIFORM", "FLAG_PROBES_RANDOM", "FLAG_BWD_SPLIT_DS", "FLAG_SEMANTIC_PARTITION", "SHARED_ROWS",
           "FLAG_STAGE_TIMING"]
