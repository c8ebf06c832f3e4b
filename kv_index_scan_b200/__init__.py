"""Python binding of libkvscan.so: the B200 per-step top-k sparse-attention
decode path (Fathom bit-plane index scan, top-k, hot-buffer gather, sparse GQA
attention, and the lightning-indexer variant), and beside it a paged K/V cache
(PagedKV and the paged_* functions).

This module only marshals arguments: it allocates output tensors with torch,
passes raw device pointers and the current CUDA stream to the C ABI declared in
include/kvscan.h, and raises on a non-OK status. Every step runs in the CUDA
kernels of the library; there is no CPU fallback. Importing fails loudly when
the library has not been built.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvscan.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m kv_index_scan_b200.build` "
        "(nvcc, sm_100a). There is no fallback implementation.")

_lib = ctypes.CDLL(LIB_PATH)

KVS_OK, KVS_EINVAL, KVS_EUNSUPPORTED, KVS_ECUDA, KVS_EWORKSPACE, KVS_ETIMEOUT, KVS_EBOUNDS = range(7)
KVS_F32, KVS_BF16 = 0, 1
KVS_SCAN_FATHOM, KVS_SCAN_LIGHTNING = 0, 1
STATUS_NAMES = {0: "KVS_OK", 1: "KVS_EINVAL", 2: "KVS_EUNSUPPORTED", 3: "KVS_ECUDA",
                4: "KVS_EWORKSPACE", 5: "KVS_ETIMEOUT", 6: "KVS_EBOUNDS"}

P = ctypes.c_void_p
I32 = ctypes.c_int32
I64 = ctypes.c_int64
SZ = ctypes.c_size_t
F32 = ctypes.c_float


class FathomIndexC(ctypes.Structure):
    _fields_ = [("planes", P), ("kmin", P), ("kstep", P), ("kvar", P), ("R", I32), ("G", I32),
                ("D", I32), ("W", I32), ("host_mapped", I32)]


class PlanC(ctypes.Structure):
    _fields_ = [("t", P), ("plane_idx", P), ("plane_w", P), ("C", P), ("B", I32)]


class ScanArgsC(ctypes.Structure):
    _fields_ = [("kind", I32), ("R", I32), ("n_max", I32), ("n", P), ("ix", ctypes.POINTER(FathomIndexC)),
                ("plan", ctypes.POINTER(PlanC)), ("kidx", P), ("qidx", P), ("widx", P), ("Hi", I32),
                ("Dl", I32), ("block", I32)]


class DecodeArgsC(ctypes.Structure):
    _fields_ = [("q", P), ("q_dtype", I32), ("H", I32), ("ix", ctypes.POINTER(FathomIndexC)),
                ("plan", ctypes.POINTER(PlanC)), ("k", I32), ("n", P), ("n_max", I32),
                ("slot_map", P), ("hotK", P), ("hotV", P), ("S", I32), ("fullK", P), ("fullV", P),
                ("idx_in", P), ("idx_shared", I32), ("scale", F32), ("out", P), ("lse", P),
                ("idx", P), ("slots", P), ("misses", P)]


class PagedKVC(ctypes.Structure):
    _fields_ = [("K", P), ("V", P), ("page_stride", I64), ("head_stride", I64), ("token_stride", I64),
                ("table", P), ("table_ld", I64), ("n", P), ("R", I32), ("G", I32), ("D", I32), ("page", I32),
                ("max_pages", I32), ("num_pages", I32)]


class PagedDecodeArgsC(ctypes.Structure):
    _fields_ = [("kv", ctypes.POINTER(PagedKVC)), ("q", P), ("q_dtype", I32), ("H", I32), ("window", I32),
                ("sinks", I32), ("scale", F32), ("out", P), ("lse", P), ("mass", P), ("mass_out", P)]


class PagedPromptArgsC(ctypes.Structure):
    _fields_ = [("kv", ctypes.POINTER(PagedKVC)), ("q", P), ("q_ld", I64), ("cu", P), ("T", I32), ("H", I32),
                ("window", I32), ("sinks", I32), ("scale", F32), ("out", P), ("out_ld", I64), ("lse", P)]


class PagedEvictArgsC(ctypes.Structure):
    _fields_ = [("kv", ctypes.POINTER(PagedKVC)), ("mass", P), ("pos", P), ("seen", P), ("budget", I32),
                ("sinks", I32), ("recent", I32), ("mass_out", P), ("pos_out", P), ("n_out", P), ("src", P)]


def _declare():
    L = _lib
    L.kvs_abi_version.restype = I32
    L.kvs_last_error.restype = ctypes.c_char_p
    L.kvs_build_fathom_index.argtypes = [P, P, I32, I32, I32, I32, I32, P, P, P, P, P, SZ, P, P]
    L.kvs_build_fathom_index.restype = I32
    L.kvs_build_index_workspace_size.argtypes = [I32, I32, I32]
    L.kvs_build_index_workspace_size.restype = SZ
    L.fathom_plan_bits.argtypes = [P, I32, ctypes.POINTER(FathomIndexC), I32, ctypes.POINTER(PlanC), P, P]
    L.fathom_plan_bits.restype = I32
    L.index_scan.argtypes = [ctypes.POINTER(ScanArgsC), P, P, P]
    L.index_scan.restype = I32
    L.topk_select.argtypes = [P, I64, P, I32, I32, I32, I32, P, P, P, SZ, P, P]
    L.topk_select.restype = I32
    L.kvs_topk_workspace_size.argtypes = [I32, I32, I32, I32, I32]
    L.kvs_topk_workspace_size.restype = SZ
    L.sparse_gather.argtypes = [P, I32, P, P, P, I32, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P]
    L.sparse_gather.restype = I32
    L.sparse_decode_attn.argtypes = [P, I32, P, P, P, I32, I32, I32, I32, I32, F32, P, P, P, SZ, P, P]
    L.sparse_decode_attn.restype = I32
    L.kvs_attn_workspace_size.argtypes = [I32, I32, I32, I32]
    L.kvs_attn_workspace_size.restype = SZ
    L.sparse_decode_attn_noalloc.argtypes = [P, I32, P, P, P, I32, I32, I32, I32, I32, F32, P, P, P, P]
    L.sparse_decode_attn_noalloc.restype = I32
    L.decode_step.argtypes = [ctypes.POINTER(DecodeArgsC), P, SZ, P, P]
    L.decode_step.restype = I32
    L.kvs_decode_step_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32]
    L.kvs_decode_step_workspace_size.restype = SZ
    L.kvs_decode_step_workspace_size_host.argtypes = [I32, I32, I32, I32, I32, I32]
    L.kvs_decode_step_workspace_size_host.restype = SZ
    L.decode_step_timed.argtypes = [ctypes.POINTER(DecodeArgsC), P, SZ, P, P, ctypes.POINTER(P), I32]
    L.decode_step_timed.restype = I32
    L.kvs_append_token.argtypes = [P, P, P, I32, I32, I32, I32, P, I32, P, P, P, P, P, P, P, P, P, I32,
                                   P, P]
    L.kvs_append_token.restype = I32
    L.kvs_selftest_scan_timeout.argtypes = [ctypes.POINTER(FathomIndexC), ctypes.POINTER(PlanC), P, I32,
                                            P, I64, P, P]
    L.kvs_selftest_scan_timeout.restype = I32
    L.kvs_paged_append.argtypes = [ctypes.POINTER(PagedKVC), P, P, I64, P, I32, P, P, P, P, P]
    L.kvs_paged_append.restype = I32
    L.paged_decode_attn.argtypes = [ctypes.POINTER(PagedDecodeArgsC), P, SZ, P, P]
    L.paged_decode_attn.restype = I32
    L.kvs_paged_decode_workspace_size.argtypes = [I32, I32, I32, I32]
    L.kvs_paged_decode_workspace_size.restype = SZ
    L.kvs_selftest_paged_decode_timeout.argtypes = [ctypes.POINTER(PagedDecodeArgsC), P, SZ, I32, I64, P, P]
    L.kvs_selftest_paged_decode_timeout.restype = I32
    L.paged_prompt_attn.argtypes = [ctypes.POINTER(PagedPromptArgsC), P, SZ, P, P]
    L.paged_prompt_attn.restype = I32
    L.kvs_paged_prompt_workspace_size.argtypes = [I32] * 7
    L.kvs_paged_prompt_workspace_size.restype = SZ
    L.kvs_paged_prompt_workspace_bound.argtypes = [I32] * 7
    L.kvs_paged_prompt_workspace_bound.restype = SZ
    L.kvs_selftest_paged_prompt_timeout.argtypes = [ctypes.POINTER(PagedPromptArgsC), I32, I64, P, P]
    L.kvs_selftest_paged_prompt_timeout.restype = I32
    L.kvs_paged_evict.argtypes = [ctypes.POINTER(PagedEvictArgsC), P, SZ, P, P]
    L.kvs_paged_evict.restype = I32
    L.kvs_paged_evict_workspace_size.argtypes = [I32, I32, I32]
    L.kvs_paged_evict_workspace_size.restype = SZ


_declare()


class KvsError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.kvs_last_error().decode(errors="replace")
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int, where: str):
    if status != KVS_OK:
        raise KvsError(status, where)


def abi_version() -> int:
    return _lib.kvs_abi_version()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, MappedHostStore):
        return t.ptr
    return t.data_ptr()


def _stream(stream=None) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _u16(t):
    return t.view(torch.int16) if isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16 else t


def plane_words(n_max: int) -> int:
    """Words per bit plane: ceil(n_max / 32) rounded up to a multiple of 4."""
    return ((n_max + 31) // 32 + 3) // 4 * 4


class FathomIndex:
    """The 4-bit channel-major bit-plane K index (tensors owned by torch).

    planes int32 [R][G][D][4][W] (u32 bit patterns), kmin/kstep/kvar f32 [R][G][D].
    `planes_ptr` overrides the planes address (a mapped pinned host alias).
    """

    def __init__(self, planes, kmin, kstep, kvar, planes_ptr: int | None = None,
                 host_mapped: bool = False):
        self.planes, self.kmin, self.kstep, self.kvar = planes, kmin, kstep, kvar
        self.R, self.G, self.D, _, self.W = planes.shape
        self.planes_ptr = planes_ptr
        self.host_mapped = host_mapped

    def c(self) -> FathomIndexC:
        pp = self.planes_ptr if self.planes_ptr is not None else self.planes.data_ptr()
        return FathomIndexC(pp, _ptr(self.kmin), _ptr(self.kstep), _ptr(self.kvar), self.R, self.G,
                            self.D, self.W, int(self.host_mapped))


class MappedHostIndex(FathomIndex):
    """A FathomIndex whose planes live in mapped pinned host memory
    (cudaHostAlloc with cudaHostAllocMapped); the scan reads them over the host
    link through the device alias from cudaHostGetDevicePointer. The host
    buffer is freed when this object is."""

    def __init__(self, index: FathomIndex):
        from cuda.bindings import runtime as rt
        self._rt = rt
        nbytes = index.planes.numel() * 4
        err, hptr = rt.cudaHostAlloc(nbytes, rt.cudaHostAllocMapped | rt.cudaHostAllocPortable)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaHostAlloc: {err}")
        self._hptr = hptr
        err, dptr = rt.cudaHostGetDevicePointer(hptr, 0)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaHostGetDevicePointer: {err}")
        torch.cuda.synchronize()
        err, = rt.cudaMemcpy(hptr, index.planes.data_ptr(), nbytes,
                             rt.cudaMemcpyKind.cudaMemcpyDeviceToHost)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaMemcpy: {err}")
        super().__init__(index.planes, index.kmin, index.kstep, index.kvar, planes_ptr=int(dptr),
                         host_mapped=True)
        self.nbytes = nbytes

    def __del__(self):
        try:
            self._rt.cudaFreeHost(self._hptr)
        except Exception:
            pass


class MappedHostStore:
    """A full K or V store in mapped pinned host memory (cudaHostAlloc with
    cudaHostAllocMapped): the host tier of the pages' system. `ptr` is its
    device alias, which decode_step reads over the host link (only the missing
    selected rows). Built from a bf16 device tensor [R][G][n_max][D]; the host
    buffer is freed when this object is."""

    def __init__(self, t: torch.Tensor):
        from cuda.bindings import runtime as rt
        self._rt = rt
        self.shape = tuple(t.shape)
        self.nbytes = t.numel() * t.element_size()
        err, hptr = rt.cudaHostAlloc(self.nbytes, rt.cudaHostAllocMapped | rt.cudaHostAllocPortable)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaHostAlloc: {err}")
        self._hptr = hptr
        err, dptr = rt.cudaHostGetDevicePointer(hptr, 0)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaHostGetDevicePointer: {err}")
        torch.cuda.synchronize()
        err, = rt.cudaMemcpy(hptr, t.data_ptr(), self.nbytes, rt.cudaMemcpyKind.cudaMemcpyDeviceToHost)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaMemcpy: {err}")
        self.ptr = int(dptr)

    def __del__(self):
        try:
            self._rt.cudaFreeHost(self._hptr)
        except Exception:
            pass


class Plan:
    """Per-(r, g) bit allocation: t u8 [R][G][D], plane_idx int16 [R][G][B]
    (u16 plane ids c*4+p), plane_w f32 [R][G][B], C f32 [R][G]."""

    def __init__(self, R: int, G: int, D: int, B: int, device):
        self.B = B
        self.t = torch.empty(R, G, D, dtype=torch.uint8, device=device)
        self.plane_idx = torch.empty(R, G, max(B, 1), dtype=torch.int16, device=device)
        self.plane_w = torch.empty(R, G, max(B, 1), dtype=torch.float32, device=device)
        self.C = torch.empty(R, G, dtype=torch.float32, device=device)

    def c(self) -> PlanC:
        return PlanC(_ptr(self.t), _ptr(self.plane_idx), _ptr(self.plane_w), _ptr(self.C), self.B)


def _n_tensor(n, R: int, device) -> torch.Tensor:
    if isinstance(n, torch.Tensor):
        return n.to(device=device, dtype=torch.int32).contiguous()
    if isinstance(n, int):
        n = [n] * R
    return torch.tensor(list(n), dtype=torch.int32, device=device)


def build_fathom_index(K: torch.Tensor, n, W: int | None = None, stream=None,
                       dev_status=None) -> FathomIndex:
    """a0: K bf16 [R][G][n_max][D] -> FathomIndex (kvs_build_fathom_index)."""
    R, G, n_max, D = K.shape
    W = plane_words(n_max) if W is None else W
    dev = K.device
    nt = _n_tensor(n, R, dev)
    planes = torch.empty(R, G, D, 4, W, dtype=torch.int32, device=dev)
    kmin = torch.empty(R, G, D, dtype=torch.float32, device=dev)
    kstep = torch.empty_like(kmin)
    kvar = torch.empty_like(kmin)
    wsb = _lib.kvs_build_index_workspace_size(R, G, D)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    st = _lib.kvs_build_fathom_index(_ptr(_u16(K)), _ptr(nt), R, G, n_max, D, W, _ptr(planes),
                                     _ptr(kmin), _ptr(kstep), _ptr(kvar), _ptr(ws), ws.numel(),
                                     _ptr(dev_status), _stream(stream))
    _check(st, "kvs_build_fathom_index")
    return FathomIndex(planes, kmin, kstep, kvar)


def fathom_plan_bits(q: torch.Tensor, index: FathomIndex, B: int, plan: Plan | None = None,
                     stream=None, dev_status=None) -> Plan:
    """a1: q f32 [R][G][H][D] -> Plan."""
    R, G, H, D = q.shape
    plan = plan or Plan(R, G, D, B, q.device)
    ix, pc = index.c(), plan.c()
    st = _lib.fathom_plan_bits(_ptr(q), H, ctypes.byref(ix), B, ctypes.byref(pc), _ptr(dev_status),
                               _stream(stream))
    _check(st, "fathom_plan_bits")
    return plan


def index_scan_fathom(index: FathomIndex, plan: Plan, n, n_max: int, scores=None, stream=None,
                      dev_status=None) -> torch.Tensor:
    """a2 (Fathom): scores f32 [R][G][n_max] (-inf past n[r])."""
    dev = index.kmin.device
    nt = _n_tensor(n, index.R, dev)
    if scores is None:
        scores = torch.empty(index.R, index.G, n_max, dtype=torch.float32, device=dev)
    ix, pc = index.c(), plan.c()
    a = ScanArgsC(KVS_SCAN_FATHOM, index.R, n_max, _ptr(nt), ctypes.pointer(ix), ctypes.pointer(pc),
                  None, None, None, 0, 0, 0)
    _check(_lib.index_scan(ctypes.byref(a), _ptr(scores), _ptr(dev_status), _stream(stream)),
           "index_scan(fathom)")
    return scores


def index_scan_lightning(kidx: torch.Tensor, qidx: torch.Tensor, w: torch.Tensor, n,
                         block: int = 64, scores=None, stream=None, dev_status=None) -> torch.Tensor:
    """a2 (lightning): kidx e4m3 codes u8 [R][n_max][Dl], qidx bf16 [R][Hi][Dl], w f32 [R][Hi]
    -> block scores f32 [R][ceil(n_max/block)] (token scores when block == 1)."""
    R, n_max, Dl = kidx.shape
    Hi = qidx.shape[1]
    nt = _n_tensor(n, R, kidx.device)
    nb = (n_max + block - 1) // block
    if scores is None:
        scores = torch.empty(R, nb, dtype=torch.float32, device=kidx.device)
    a = ScanArgsC(KVS_SCAN_LIGHTNING, R, n_max, _ptr(nt), None, None, _ptr(kidx), _ptr(_u16(qidx)),
                  _ptr(w), Hi, Dl, block)
    _check(_lib.index_scan(ctypes.byref(a), _ptr(scores), _ptr(dev_status), _stream(stream)),
           "index_scan(lightning)")
    return scores


def topk_select(scores: torch.Tensor, n, k: int, block: int = 1, want_vals: bool = False,
                idx=None, stream=None, dev_status=None):
    """a3: scores f32 [R][G][ld] (or [R][ld]) -> idx int32 [R][G][k] (and vals)."""
    s3 = scores if scores.dim() == 3 else scores.unsqueeze(1)
    R, G, ld = s3.shape
    nt = _n_tensor(n, R, scores.device)
    if idx is None:
        idx = torch.empty(R, G, k, dtype=torch.int32, device=scores.device)
    vals = torch.empty(R, G, k, dtype=torch.float32, device=scores.device) if want_vals else None
    wsb = _lib.kvs_topk_workspace_size(R, G, ld, k, block)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=scores.device)
    st = _lib.topk_select(_ptr(s3), ld, _ptr(nt), R, G, k, block, _ptr(idx), _ptr(vals), _ptr(ws),
                          ws.numel(), _ptr(dev_status), _stream(stream))
    _check(st, "topk_select")
    if scores.dim() == 2:
        idx = idx.squeeze(1)
        vals = vals.squeeze(1) if vals is not None else None
    return (idx, vals) if want_vals else idx


def sparse_gather(idx, slot_map, hotK, hotV, fullK, fullV, n, stream=None, dev_status=None):
    """a4: -> (gK, gV bf16 [R][G][k][D], slots int32 [R][G][k], misses int32 [R][G])."""
    R, G, k = idx.shape
    S = hotK.shape[2]
    n_max, D = fullK.shape[2], fullK.shape[3]
    dev = idx.device
    nt = _n_tensor(n, R, dev)
    gK = torch.empty(R, G, k, D, dtype=torch.bfloat16, device=dev)
    gV = torch.empty_like(gK)
    slots = torch.empty(R, G, k, dtype=torch.int32, device=dev)
    misses = torch.empty(R, G, dtype=torch.int32, device=dev)
    st = _lib.sparse_gather(_ptr(idx), k, _ptr(slot_map), _ptr(_u16(hotK)), _ptr(_u16(hotV)), S,
                            _ptr(_u16(fullK)), _ptr(_u16(fullV)), _ptr(nt), n_max, R, G, D,
                            _ptr(_u16(gK)), _ptr(_u16(gV)), _ptr(slots), _ptr(misses),
                            _ptr(dev_status), _stream(stream))
    _check(st, "sparse_gather")
    return gK, gV, slots, misses


def sparse_decode_attn(q, K, V, k_eff=None, scale: float | None = None, want_lse: bool = True,
                       stream=None, dev_status=None):
    """a5: q f32/bf16 [R][G][H][D], K/V bf16 [R][G][k][D] -> (out f32 [R][G][H][D], lse)."""
    R, G, H, D = q.shape
    k = K.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.empty(R, G, H, D, dtype=torch.float32, device=q.device)
    lse = torch.empty(R, G, H, dtype=torch.float32, device=q.device) if want_lse else None
    wsb = _lib.kvs_attn_workspace_size(R, G, H, k)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=q.device)
    qd = KVS_BF16 if q.dtype == torch.bfloat16 else KVS_F32
    st = _lib.sparse_decode_attn(_ptr(_u16(q)), qd, _ptr(_u16(K)), _ptr(_u16(V)), _ptr(k_eff), R, G,
                                 H, D, k, scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                 _ptr(dev_status), _stream(stream))
    _check(st, "sparse_decode_attn")
    return out, lse


def _require(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def sparse_decode_attn_noalloc(q, K, V, out, lse=None, k_eff=None, scale: float | None = None,
                               stream=None, dev_status=None):
    """a5 without a workspace, into caller-provided out (and lse): the library
    keeps the split-K scratch in a fixed device array (see include/kvscan.h).
    out must be f32 [R][G][H][D] and lse f32 [R][G][H], contiguous, on q's
    device; k_eff (nullable) int32 [R][G]."""
    R, G, H, D = q.shape
    k = K.shape[2]
    for name, t, shape, dt in (("out", out, (R, G, H, D), torch.float32),
                               ("lse", lse, (R, G, H), torch.float32),
                               ("k_eff", k_eff, (R, G), torch.int32)):
        if t is None:
            _require(name != "out", "out is required")
            continue
        _require(t.dtype == dt, f"{name} must be {dt}, got {t.dtype}")
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        _require(t.is_contiguous(), f"{name} must be contiguous")
        _require(t.device == q.device, f"{name} must be on {q.device}")
    _require(tuple(K.shape) == (R, G, k, D) and tuple(V.shape) == (R, G, k, D),
             "K and V must be [R][G][k][D]")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    qd = KVS_BF16 if q.dtype == torch.bfloat16 else KVS_F32
    st = _lib.sparse_decode_attn_noalloc(_ptr(_u16(q)), qd, _ptr(_u16(K)), _ptr(_u16(V)), _ptr(k_eff),
                                         R, G, H, D, k, scale, _ptr(out), _ptr(lse),
                                         _ptr(dev_status), _stream(stream))
    _check(st, "sparse_decode_attn_noalloc")
    return out, lse


def append_token(index: FathomIndex, Knew, Vnew, n: torch.Tensor, fullK, fullV, slot_map=None,
                 hot_slot=None, hot_tok=None, hotK=None, hotV=None, stream=None, dev_status=None):
    """Per-step write-back (kvs_append_token): the new token Knew/Vnew bf16
    [R][G][D] of every request joins its rows at position n[r] -- its 4-bit
    codes (the index's own quantiser) into the planes, its K/V rows into the
    full store, optionally a hot slot (hot_slot int32 [R][G], with hot_tok
    int32 [R][G][S] the token each slot holds) -- and n (device int32 [R]) is
    advanced in place."""
    R, G, D = Knew.shape
    n_max = fullK.shape[2]
    if n.dtype != torch.int32 or not n.is_contiguous() or n.device != Knew.device:
        raise ValueError("n must be a contiguous device int32 tensor on Knew's device")
    S = hotK.shape[2] if hotK is not None else 0
    st = _lib.kvs_append_token(_ptr(_u16(Knew)), _ptr(_u16(Vnew)), _ptr(n), R, G, D, n_max,
                               _ptr(index.planes), index.W, _ptr(index.kmin), _ptr(index.kstep),
                               _ptr(_u16(fullK)), _ptr(_u16(fullV)), _ptr(slot_map), _ptr(hot_slot),
                               _ptr(hot_tok), _ptr(_u16(hotK)), _ptr(_u16(hotV)), S,
                               _ptr(dev_status), _stream(stream))
    _check(st, "kvs_append_token")


def selftest_scan_timeout(index: FathomIndex, plan: Plan, n, n_max: int, wait_cycles: int,
                          dev_status: torch.Tensor, stream=None):
    """kvs_selftest_scan_timeout: the HBM scan with a withheld producer
    arrival, so that its bounded waits run out; dev_status (device int32)
    receives KVS_ETIMEOUT. For tests of the failure path."""
    nt = _n_tensor(n, index.R, index.kmin.device)
    scores = torch.empty(index.R, index.G, n_max, dtype=torch.float32, device=index.kmin.device)
    ix, pc = index.c(), plan.c()
    st = _lib.kvs_selftest_scan_timeout(ctypes.byref(ix), ctypes.byref(pc), _ptr(nt), n_max,
                                        _ptr(scores), wait_cycles, _ptr(dev_status), _stream(stream))
    _check(st, "kvs_selftest_scan_timeout")


def decode_step_workspace_size(R, G, H, n_max, k, B) -> int:
    return int(_lib.kvs_decode_step_workspace_size(R, G, H, n_max, k, B))


class DecodeStep:
    """a6 with persistent, caller-owned buffers (like a graph-captured decode
    layer): outputs and workspace are allocated once, each call only launches."""

    def __init__(self, index: FathomIndex, n, n_max: int, H: int, B: int, k: int, fullK, fullV,
                 slot_map=None, hotK=None, hotV=None, scale: float | None = None,
                 q_dtype=torch.float32, device=None):
        dev = device or index.kmin.device
        self.index, self.H, self.B, self.k, self.n_max = index, H, B, k, n_max
        R, G, D = index.R, index.G, index.D
        self.R, self.G, self.D = R, G, D
        self.n = _n_tensor(n, R, dev)
        self.fullK, self.fullV, self.slot_map, self.hotK, self.hotV = fullK, fullV, slot_map, hotK, hotV
        self.S = hotK.shape[2] if hotK is not None else 0
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.plan = Plan(R, G, D, B, dev)
        self.out = torch.empty(R, G, H, D, dtype=torch.float32, device=dev)
        self.lse = torch.empty(R, G, H, dtype=torch.float32, device=dev)
        self.idx = torch.empty(R, G, k, dtype=torch.int32, device=dev)
        self.slots = torch.empty(R, G, k, dtype=torch.int32, device=dev)
        self.misses = torch.empty(R, G, dtype=torch.int32, device=dev)
        # a full store in host memory (MappedHostStore) needs the staging too
        self.full_on_host = isinstance(fullK, MappedHostStore)
        wsb = (int(_lib.kvs_decode_step_workspace_size_host(R, G, H, n_max, k, B)) if self.full_on_host
               else decode_step_workspace_size(R, G, H, n_max, k, B))
        self.ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
        self.q_dtype = KVS_BF16 if q_dtype == torch.bfloat16 else KVS_F32
        self._ix = index.c()
        self._plan = self.plan.c()

    def args(self, q, idx_in=None, idx_shared: bool = False, out=None) -> DecodeArgsC:
        return DecodeArgsC(
            _ptr(_u16(q)), self.q_dtype, self.H, ctypes.pointer(self._ix), ctypes.pointer(self._plan),
            self.k, _ptr(self.n), self.n_max, _ptr(self.slot_map), _ptr(_u16(self.hotK)),
            _ptr(_u16(self.hotV)), self.S, _ptr(_u16(self.fullK)), _ptr(_u16(self.fullV)),
            _ptr(idx_in), int(idx_shared), self.scale, _ptr(self.out if out is None else out),
            _ptr(self.lse), _ptr(self.idx), _ptr(self.slots), _ptr(self.misses))

    def __call__(self, q, idx_in=None, idx_shared: bool = False, stream=None, dev_status=None,
                 out=None):
        a = self.args(q, idx_in, idx_shared, out)
        st = _lib.decode_step(ctypes.byref(a), _ptr(self.ws), self.ws.numel(), _ptr(dev_status),
                              _stream(stream))
        _check(st, "decode_step")
        return self.out if out is None else out

    DECODE_STAGES = ("allocation", "scan", "selection", "attention")

    def timed(self, q, events, idx_in=None, idx_shared: bool = False, stream=None,
              dev_status=None, out=None):
        """decode_step_timed: as __call__, recording the 5 torch.cuda.Event(enable_timing=True)
        objects in `events` at the stage boundaries (see DECODE_STAGES)."""
        if len(events) != len(self.DECODE_STAGES) + 1:
            raise ValueError(f"{len(self.DECODE_STAGES) + 1} events needed")
        s = stream if stream is not None else torch.cuda.current_stream()
        for e in events:  # make sure each event exists (torch creates it lazily)
            e.record(s)
        evs = (P * len(events))(*[e.cuda_event for e in events])
        a = self.args(q, idx_in, idx_shared, out)
        st = _lib.decode_step_timed(ctypes.byref(a), _ptr(self.ws), self.ws.numel(),
                                    _ptr(dev_status), _stream(s), evs, len(events))
        _check(st, "decode_step_timed")
        return self.out if out is None else out


def decode_step(q, index: FathomIndex, n, B: int, k: int, fullK, fullV, slot_map=None, hotK=None,
                hotV=None, scale=None, idx_in=None, idx_shared=False, stream=None):
    """a6 one-shot: returns (out, lse, idx, slots, misses, plan)."""
    R, G, H, D = q.shape
    step = DecodeStep(index, n, fullK.shape[2], H, B, k, fullK, fullV, slot_map, hotK, hotV, scale,
                      q_dtype=q.dtype)
    step(q, idx_in=idx_in, idx_shared=idx_shared, stream=stream)
    return step.out, step.lse, step.idx, step.slots, step.misses, step.plan


# ----------------------------------------------------------------------------- the paged K/V cache

def _elsewhere(dev: torch.device, stream) -> bool:
    """Whether a call has to go into a context first: its tensors' device is not the current one, or it has a
    stream of its own."""
    return stream is not None or torch.cuda.current_device() != dev.index


def _on(dev: torch.device, stream):
    """That context: dev current and, where one is given, `stream` current too, so that what the call
    allocates belongs to the stream that uses it."""
    if stream is None:
        return torch.cuda.device(dev)
    _require(stream.device == dev, f"the stream is on {stream.device}, the cache on {dev}")
    return torch.cuda.stream(stream)


def _raw_stream(dev: torch.device) -> int:
    """The current stream of dev, as its handle (torch.cuda.current_stream builds an object around it)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _need(name: str, t, shape, dtype, dev):
    """t, if it is a contiguous tensor of this shape and type on dev."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        what = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else repr(type(t))
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on {dev}, got {what}")
    return t


def _check_ws(ws, dev):
    if not (ws.device == dev and ws.dtype is torch.uint8 and ws.is_contiguous()):
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev}")


def _status_ptr(t, dev):
    """The status word's address. Kernels write there, so a tensor of another type or in ordinary host memory is
    refused (a raw address is the caller's word)."""
    if isinstance(t, torch.Tensor) and not (t.dtype is torch.int32 and t.numel() >= 1
                                            and (t.device == dev or (t.device.type == "cpu" and t.is_pinned()))):
        raise ValueError(f"dev_status must be an int32 tensor on {dev} or in pinned host memory, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return _ptr(t)


def _counts(**values):
    """Every value fits the C boundary's int32 and is not negative."""
    for name, v in values.items():
        if not (isinstance(v, int) and 0 <= v < 2147483648):
            raise ValueError(f"{name} must be an int from 0 to 2^31 - 1, got {v!r}")


class PagedKV:
    """A paged K/V cache (tensors owned by torch).

    k_pages, v_pages bf16 [num_pages][G][page][128], of the same strides, the last dimension contiguous
    (a pool laid out [num_pages][page][G][128] is passed as its .transpose(1, 2)); table int32
    [R][max_pages], the pages of each request in order; n int32 [R], the tokens each holds. The tensors
    are read by later calls as they are then: n and table may change in place, in a captured graph too. The
    attributes k_pages, v_pages, table and n stay these tensors; others make another PagedKV.
    """

    _KEPT = frozenset(("k_pages", "v_pages", "table", "n"))

    def __setattr__(self, name, value):
        # the C descriptor points to these tensors' memory (`x.n += 1` assigns the same tensor)
        if name in self._KEPT and self.__dict__.get(name, value) is not value:
            raise ValueError(f"{name} stays the tensor it was made with: change that one in place (.copy_), or make "
                             "another cache")
        object.__setattr__(self, name, value)

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, n: torch.Tensor):
        for name, t, dt, dims in (("k_pages", k_pages, torch.bfloat16, 4), ("v_pages", v_pages, torch.bfloat16, 4),
                                  ("table", table, torch.int32, 2), ("n", n, torch.int32, 1)):
            _require(isinstance(t, torch.Tensor) and t.dtype == dt and t.dim() == dims,
                     f"{name} must be a {dt} tensor of {dims} dimensions")
            _require(t.device == k_pages.device and t.is_cuda, f"{name} must be on k_pages' CUDA device")
            _require(t.stride(-1) == 1 or t.shape[-1] == 1, f"{name} must be contiguous in its last dimension")
        _require(k_pages.shape == v_pages.shape and k_pages.stride() == v_pages.stride(),
                 "k_pages and v_pages must have the same shape and strides")
        _require(k_pages.numel() > 0, f"k_pages must not be empty, got {tuple(k_pages.shape)}")
        self.num_pages, self.G, self.page, self.D = k_pages.shape
        self.R, self.max_pages = table.shape
        _require(n.shape[0] == self.R, f"n must have {self.R} entries, got {n.shape[0]}")
        self.k_pages, self.v_pages, self.table, self.n = k_pages, v_pages, table, n
        self.device = k_pages.device
        self.cap = self.max_pages * self.page
        # the stride of a dimension of one entry says nothing
        st = [x if k > 1 else self.D for x, k in zip(k_pages.stride(), k_pages.shape)]
        self._c = PagedKVC(k_pages.data_ptr(), v_pages.data_ptr(), st[0], st[1], st[2], table.data_ptr(),
                           table.stride(0) if self.R > 1 else self.max_pages, n.data_ptr(), self.R, self.G, self.D,
                           self.page, self.max_pages, self.num_pages)
        self._ref = ctypes.pointer(self._c)
        self._state_shape = torch.Size((self.R, self.G, self.cap))
        self._r_shape, self._cu_shape = torch.Size((self.R,)), torch.Size((self.R + 1,))
        self._ws_bytes = {}  # what the library asks for, by call and sizes

    def _state(self, name, t, dtype):
        return None if t is None else _need(name, t, self._state_shape, dtype, self.device).data_ptr()

    def _workspace(self, query, *sizes):
        """What the library asks for, or None where that is nothing."""
        nb = self._ws_bytes.get((query, sizes))
        if nb is None:
            if len(self._ws_bytes) > 1000:  # a prompt's size depends on its tokens
                self._ws_bytes.clear()
            nb = self._ws_bytes[query, sizes] = int(getattr(_lib, query)(self.R, self.G, *sizes))
        return torch.empty(nb, dtype=torch.uint8, device=self.device) if nb else None


def paged_append(cache: PagedKV, Knew: torch.Tensor, Vnew: torch.Tensor, cu=None, mass=None, pos=None, seen=None,
                 stream=None, dev_status=None):
    """Writes the newest tokens' rows into their pages (kvs_paged_append): Knew, Vnew bf16 [T][G][128],
    packed by request with cu int32 [R+1] (None: one token each). cache.n already counts them. mass f32 and
    pos int32 [R][G][cap] get 0 and the token's place (counted by seen int32 [R])."""
    dev = cache.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return paged_append(cache, Knew, Vnew, cu, mass, pos, seen, None, dev_status)
    shape = Knew.shape
    if not (len(shape) == 3 and Vnew.shape == shape and shape[1] == cache.G and shape[2] == cache.D
            and Knew.dtype is torch.bfloat16 and Vnew.dtype is torch.bfloat16 and Knew.device == dev
            and Vnew.device == dev):
        raise ValueError(f"Knew and Vnew must be bf16 [T][{cache.G}][{cache.D}] on {dev}")
    st = Knew.stride()
    _require(Vnew.stride() == st and st[2] == 1 and (st[1] == cache.D or cache.G == 1),
             "Knew and Vnew must have the same strides, their heads contiguous")
    T = shape[0]
    ld = st[0] if T > 1 else cache.G * cache.D
    cup = None if cu is None else _need("cu", cu, cache._cu_shape, torch.int32, dev).data_ptr()
    sp = None if seen is None else _need("seen", seen, cache._r_shape, torch.int32, dev).data_ptr()
    mp, pp = cache._state("mass", mass, torch.float32), cache._state("pos", pos, torch.int32)
    st_ptr = None if dev_status is None else _status_ptr(dev_status, dev)
    _check(_lib.kvs_paged_append(cache._ref, Knew.data_ptr(), Vnew.data_ptr(), ld, cup, T, mp, pp, sp,
                                 st_ptr, _raw_stream(dev)), "kvs_paged_append")


def paged_decode_workspace(cache: PagedKV, H: int, weights: bool = False) -> torch.Tensor:
    """A workspace for paged_decode_attn, for callers that keep one (calls that may run at the same time
    need one each)."""
    if _elsewhere(cache.device, None):
        with _on(cache.device, None):
            return paged_decode_workspace(cache, H, weights)
    return cache._workspace("kvs_paged_decode_workspace_size", H, cache.cap if weights else 0)


def paged_decode_attn(q: torch.Tensor, cache: PagedKV, window: int = 0, sinks: int = 0, scale: float | None = None,
                      out=None, lse=None, mass=None, mass_out=None, ws=None, stream=None, dev_status=None):
    """Attention of each request's newest token over its cache: q f32/bf16 [R][G][H][128] -> (out f32
    [R][G][H][128], lse f32 [R][G][H]). window > 0: only the last `window` tokens and the first `sinks`.
    mass f32 [R][G][cap]: every visible token's softmax weights, summed over the H heads, are added to it
    (in place, or into mass_out)."""
    dev, R, G, D = cache.device, cache.R, cache.G, cache.D
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return paged_decode_attn(q, cache, window, sinks, scale, out, lse, mass, mass_out, ws, None, dev_status)
    _counts(window=window, sinks=sinks)
    shape, bf16 = q.shape, q.dtype is torch.bfloat16
    if not (len(shape) == 4 and shape[0] == R and shape[1] == G and shape[3] == D
            and (bf16 or q.dtype is torch.float32) and q.device == dev and q.is_contiguous()):
        raise ValueError(f"q must be contiguous f32 or bf16 [{R}][{G}][H][{D}] on {dev}, got {q.dtype} {tuple(shape)} "
                         f"on {q.device}")
    H = shape[2]
    if out is None:
        out = torch.empty(R, G, H, D, dtype=torch.float32, device=dev)
    else:
        _need("out", out, shape, torch.float32, dev)
    if lse is None:
        lse = torch.empty(R, G, H, dtype=torch.float32, device=dev)
    else:
        _need("lse", lse, shape[:3], torch.float32, dev)
    mp = cache._state("mass", mass, torch.float32)
    mo = mp if mass_out is None else cache._state("mass_out", mass_out, torch.float32)
    if ws is None:
        ws = paged_decode_workspace(cache, H, mass is not None)
    else:
        _check_ws(ws, dev)
    a = PagedDecodeArgsC(cache._ref, q.data_ptr(), KVS_BF16 if bf16 else KVS_F32, H, window, sinks,
                         1.0 / math.sqrt(D) if scale is None else scale, out.data_ptr(), lse.data_ptr(), mp, mo)
    st_ptr = None if dev_status is None else _status_ptr(dev_status, dev)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
    _check(_lib.paged_decode_attn(ctypes.byref(a), wp, wn, st_ptr, _raw_stream(dev)), "paged_decode_attn")
    return out, lse


def selftest_paged_decode_timeout(q: torch.Tensor, cache: PagedKV, warp: int, wait_cycles: int,
                                  dev_status: torch.Tensor, stream=None):
    """kvs_selftest_paged_decode_timeout: paged_decode_attn of bf16 queries with one warp of every block giving
    up a wait; dev_status (device int32) receives KVS_ETIMEOUT. For tests of the failure path."""
    dev = cache.device
    with _on(dev, stream):
        H = q.shape[2]
        _require(1 <= H <= 8, f"1 to 8 query heads a KV head, got {H}")
        _need("q", q, (cache.R, cache.G, H, cache.D), torch.bfloat16, dev)
        out = torch.empty(q.shape, dtype=torch.float32, device=dev)
        ws = paged_decode_workspace(cache, H)
        a = PagedDecodeArgsC(cache._ref, q.data_ptr(), KVS_BF16, H, 0, 0, 1.0, out.data_ptr(), None, None, None)
        _check(_lib.kvs_selftest_paged_decode_timeout(ctypes.byref(a), ws.data_ptr(), ws.numel(), warp, wait_cycles,
                                                      _status_ptr(dev_status, dev), _raw_stream(dev)),
               "kvs_selftest_paged_decode_timeout")


def paged_prompt_workspace(cache: PagedKV, H: int, T: int, window: int = 0, sinks: int = 0):
    """A workspace for every paged_prompt_attn of up to T queries with H query heads a KV head, this window and
    these sinks, for callers that keep one (None: no such call needs any)."""
    if _elsewhere(cache.device, None):
        with _on(cache.device, None):
            return paged_prompt_workspace(cache, H, T, window, sinks)
    _counts(H=H, T=T, window=window, sinks=sinks)
    return cache._workspace("kvs_paged_prompt_workspace_bound", H, T, cache.cap, window, sinks)


def paged_evict_workspace(cache: PagedKV, budget: int) -> torch.Tensor:
    """A workspace for paged_evict down to `budget` or less, for callers that keep one."""
    if _elsewhere(cache.device, None):
        with _on(cache.device, None):
            return paged_evict_workspace(cache, budget)
    _counts(budget=budget)
    return cache._workspace("kvs_paged_evict_workspace_size", budget)


def paged_prompt_attn(q: torch.Tensor, cu: torch.Tensor, cache: PagedKV, window: int = 0, sinks: int = 0,
                      scale: float | None = None, out=None, lse=None, ws=None, stream=None, dev_status=None):
    """Causal attention of the newest tokens of each request over its cache: q bf16 [T][G*H][128], packed by
    request with cu int32 [R+1] -> (out bf16 [T][G*H][128], lse f32 [T][G*H]). window > 0: each token sees
    itself and the window - 1 before it, and the first `sinks`. Rows from cu[R] on are left as they are
    (zero in an `out` and `lse` made here)."""
    dev = cache.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return paged_prompt_attn(q, cu, cache, window, sinks, scale, out, lse, ws, None, dev_status)
    _counts(window=window, sinks=sinks)
    shape = q.shape
    if not (len(shape) == 3 and q.dtype is torch.bfloat16 and q.device == dev and shape[2] == cache.D
            and shape[1] % cache.G == 0):
        raise ValueError(f"q must be bf16 [T][{cache.G}*H][{cache.D}] on {dev}")
    T, Hq, D = shape
    _need("cu", cu, cache._cu_shape, torch.int32, dev)
    if out is None:
        out = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    else:
        if not (out.shape == shape and out.dtype is torch.bfloat16 and out.device == dev):
            raise ValueError(f"out must be bf16 {tuple(shape)} on {dev}")
    qs, os_ = q.stride(), out.stride()
    if not (qs[2] == 1 and os_[2] == 1 and (Hq == 1 or (qs[1] == D and os_[1] == D))):
        raise ValueError("q and out must have contiguous heads")
    if lse is None:
        lse = torch.zeros(T, Hq, dtype=torch.float32, device=dev)
    else:
        _need("lse", lse, (T, Hq), torch.float32, dev)
    ld = (qs[0], os_[0]) if T > 1 else (Hq * D, Hq * D)
    a = PagedPromptArgsC(cache._ref, q.data_ptr(), ld[0], cu.data_ptr(), T, Hq // cache.G, window, sinks,
                         1.0 / math.sqrt(D) if scale is None else scale, out.data_ptr(), ld[1], lse.data_ptr())
    if ws is None:
        ws = cache._workspace("kvs_paged_prompt_workspace_size", Hq // cache.G, T, cache.cap, window,
                              sinks)
    else:
        _check_ws(ws, dev)
    st_ptr = None if dev_status is None else _status_ptr(dev_status, dev)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
    _check(_lib.paged_prompt_attn(ctypes.byref(a), wp, wn, st_ptr, _raw_stream(dev)), "paged_prompt_attn")
    return out, lse


def selftest_paged_prompt_timeout(q: torch.Tensor, cu: torch.Tensor, cache: PagedKV, warp: int, wait_cycles: int,
                                  dev_status: torch.Tensor, stream=None):
    """kvs_selftest_paged_prompt_timeout: paged_prompt_attn with one warp of every block giving up; dev_status
    (device int32) receives KVS_ETIMEOUT. For tests of the failure path."""
    dev = cache.device
    with _on(dev, stream):
        T, Hq, D = q.shape
        _need("q", q, (T, Hq, cache.D), torch.bfloat16, dev)
        _need("cu", cu, cache._cu_shape, torch.int32, dev)
        _require(Hq % cache.G == 0, f"q must have a multiple of {cache.G} heads")
        out = torch.empty_like(q)
        a = PagedPromptArgsC(cache._ref, q.data_ptr(), Hq * D, cu.data_ptr(), T, Hq // cache.G, 0, 0, 1.0,
                             out.data_ptr(), Hq * D, None)
        _check(_lib.kvs_selftest_paged_prompt_timeout(ctypes.byref(a), warp, wait_cycles, _status_ptr(dev_status, dev),
                                                      _raw_stream(dev)), "kvs_selftest_paged_prompt_timeout")


def paged_evict(cache: PagedKV, mass: torch.Tensor, budget: int, sinks: int = 0, recent: int = 0, pos=None,
                seen=None, mass_out=None, pos_out=None, n_out=None, src=None, ws=None, stream=None,
                dev_status=None) -> torch.Tensor:
    """Cuts every request that holds more than `budget` tokens down to `budget`, for each KV head by itself
    (kvs_paged_evict): kept are tokens placed (pos int32 [R][G][cap]; None: slot i holds token i) before
    `sinks` or among the last `recent` of the `seen` int32 [R] (None: cache.n), then those of largest mass f32
    [R][G][cap]. Kept rows behind the budget move into freed slots; mass, pos and cache.n are updated in
    place unless mass_out, pos_out and n_out are given. -> src int32 [R][G][budget]: the slot each token was
    in (-1 behind the last)."""
    dev = cache.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return paged_evict(cache, mass, budget, sinks, recent, pos, seen, mass_out, pos_out, n_out, src, ws, None,
                               dev_status)
    _counts(budget=budget, sinks=sinks, recent=recent)
    mp = cache._state("mass", mass, torch.float32)
    _require(mp is not None, "mass is required")
    mo = mp if mass_out is None else cache._state("mass_out", mass_out, torch.float32)
    pp = cache._state("pos", pos, torch.int32)
    _require(pp is not None or pos_out is None, "pos_out without pos")
    po = pp if pos_out is None else cache._state("pos_out", pos_out, torch.int32)
    sp = None if seen is None else _need("seen", seen, cache._r_shape, torch.int32, dev).data_ptr()
    no = (cache.n if n_out is None else _need("n_out", n_out, cache._r_shape, torch.int32, dev)).data_ptr()
    if not 1 <= budget <= 1 << 30:
        raise ValueError(f"budget must be from 1 to 2^30, got {budget}")
    if src is None:
        src = torch.empty(cache.R, cache.G, budget, dtype=torch.int32, device=dev)
    else:
        _need("src", src, (cache.R, cache.G, budget), torch.int32, dev)
    if ws is None:
        ws = cache._workspace("kvs_paged_evict_workspace_size", budget)
    else:
        _check_ws(ws, dev)
    a = PagedEvictArgsC(cache._ref, mp, pp, sp, budget, sinks, recent, mo, po, no, src.data_ptr())
    st_ptr = None if dev_status is None else _status_ptr(dev_status, dev)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
    _check(_lib.kvs_paged_evict(ctypes.byref(a), wp, wn, st_ptr, _raw_stream(dev)), "kvs_paged_evict")
    return src
