"""ctypes binding of libag (include/ag.h): argument marshalling only.

Every function here forwards to the C ABI of the same name; all work on the
device happens in the library's HIP kernels.  There is no fallback: if
libag.so is missing or fails to load, every call raises.

Device memory and streams come from PyTorch (a torch uint8 tensor can serve
as the heap's slab via ``Heap.wrap``); pointers are passed as integers.
"""

from __future__ import annotations

import ctypes
import os
from array import array
from operator import attrgetter
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libag.so")

AG_OK, AG_ERR_INVALID_ARG, AG_ERR_UNSUPPORTED, AG_ERR_OUT_OF_MEMORY, AG_ERR_HIP = range(5)
STATUS_NAMES = {0: "AG_OK", 1: "AG_ERR_INVALID_ARG", 2: "AG_ERR_UNSUPPORTED",
                3: "AG_ERR_OUT_OF_MEMORY", 4: "AG_ERR_HIP"}
AG_F16, AG_BF16, AG_F32 = 0, 1, 2
DTYPE_CODES = {"f16": AG_F16, "bf16": AG_BF16, "f32": AG_F32}
ELEM_BYTES = {"f16": 2, "bf16": 2, "f32": 4}
AG_MAX_WORLD = 8
AG_NOALLOC_MAX_RANKS = 64
AG_REGION_ALIGN = 2 << 20


class AgError(RuntimeError):
    def __init__(self, status: int, message: str, call: str):
        self.status = status
        self.message = message
        super().__init__(f"{call}: {STATUS_NAMES.get(status, status)}: {message}")


class Geometry(ctypes.Structure):
    _fields_ = [("slab_addr", ctypes.c_uint64), ("bytes_per_rank", ctypes.c_uint64),
                ("n_ranks", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("num_cus", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("group_rank", ctypes.c_int32), ("vec_bytes", ctypes.c_int32),
                ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
                ("n_programs", ctypes.c_int32), ("threads", ctypes.c_int32), ("lds_bytes", ctypes.c_int32),
                ("vectors_per_thread", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64), ("total_tiles", ctypes.c_int64),
                ("rank_block_offset", ctypes.c_uint64), ("bytes_read", ctypes.c_uint64),
                ("bytes_written", ctypes.c_uint64), ("flops", ctypes.c_double),
                ("dest_group", ctypes.c_int32), ("schedule", ctypes.c_int32),
                ("tile_order", ctypes.c_int32), ("tiles_per_ticket", ctypes.c_int32),
                ("ticket_wait", ctypes.c_int32), ("reserved_plan", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


AG_SCHEDULE_TILES, AG_SCHEDULE_PARTITIONED = 0, 1
SCHEDULES = {"tiles": AG_SCHEDULE_TILES, "partitioned": AG_SCHEDULE_PARTITIONED}
AG_ORDER_AUTO, AG_ORDER_STRIDE, AG_ORDER_TICKETS = 0, 1, 2
TILE_ORDERS = {"auto": AG_ORDER_AUTO, "stride": AG_ORDER_STRIDE, "tickets": AG_ORDER_TICKETS}
AG_B_K_CONTIGUOUS, AG_B_N_CONTIGUOUS = 0, 1
B_LAYOUTS = {"k": AG_B_K_CONTIGUOUS, "n": AG_B_N_CONTIGUOUS}


class CopyOptions(ctypes.Structure):
    _fields_ = [("dest_group", ctypes.c_int32), ("schedule", ctypes.c_int32), ("tile_order", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 5)]


class GemmOptions(ctypes.Structure):
    _fields_ = [("b_layout", ctypes.c_int32), ("reserved", ctypes.c_int32 * 7)]


AG_ACT_NONE, AG_ACT_RELU, AG_ACT_GELU, AG_ACT_GELU_TANH, AG_ACT_SILU = range(5)
ACTS = {"none": AG_ACT_NONE, "relu": AG_ACT_RELU, "gelu": AG_ACT_GELU, "gelu_tanh": AG_ACT_GELU_TANH,
        "silu": AG_ACT_SILU}
AG_ADAMW_BLOCK = 256


def _fields(ctype, names):
    return [(name, ctype) for name in names.split()]


class LinearArgs(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_void_p, "x w bias residual y z") +
                _fields(ctypes.c_int64, "ldx ldw ldr ldy ldz M N K") +
                _fields(ctypes.c_int32, "dtype act") + [("reserved", ctypes.c_int32 * 6)])


class LinearBackwardArgs(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_void_p, "dy z x w dx dw db") +
                _fields(ctypes.c_int64, "lddy ldz ldx ldw lddx lddw M N K") +
                _fields(ctypes.c_int32, "dtype act dw_dtype accumulate") + [("reserved", ctypes.c_int32 * 4)])


class ProductPlan(ctypes.Structure):
    _fields_ = _fields(ctypes.c_int32, "variant tile_m tile_n tile_k full_tiles splits n_programs packed")


class LinearPlan(ctypes.Structure):
    _fields_ = ([("product", ProductPlan), ("product_dw", ProductPlan)] +
                _fields(ctypes.c_uint64, "workspace_bytes bytes_read bytes_written") +
                [("flops", ctypes.c_double)] + _fields(ctypes.c_int32, "launches reserved"))


class AdamwTensor(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_void_p, "param grad exp_avg exp_avg_sq exp_avg_scale exp_avg_sq_scale master") +
                [("n", ctypes.c_int64)])


class AdamwHyper(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_double, "lr beta1 beta2 eps weight_decay grad_scale") +
                [("step", ctypes.c_int64)] + _fields(ctypes.c_void_p, "dev_step dev_lr dev_grad_scale") +
                [("seed", ctypes.c_uint64), ("stochastic", ctypes.c_int32), ("reserved", ctypes.c_int32 * 5)])


def _options(dest_group=0, schedule=0, tile_order=0) -> CopyOptions:
    o = CopyOptions()
    o.dest_group = dest_group
    o.schedule = SCHEDULES[schedule] if isinstance(schedule, str) else schedule
    o.tile_order = TILE_ORDERS[tile_order] if isinstance(tile_order, str) else tile_order
    return o


_lib: Optional[ctypes.CDLL] = None

_c_int, _c_size, _c_i64, _c_u64, _vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
_HEAP_PP = ctypes.POINTER(ctypes.c_void_p)

_SIGNATURES = {
    "ag_heap_region_bytes": [_c_size, ctypes.POINTER(ctypes.c_size_t)],
    "ag_heap_create": [_c_int, _c_size, _HEAP_PP],
    "ag_heap_wrap": [_vp, _c_int, _c_size, _HEAP_PP],
    "ag_heap_view": [_vp, _c_int, _HEAP_PP],
    "ag_heap_destroy": [_vp],
    "ag_heap_alloc": [_vp, _c_size, _c_size, ctypes.POINTER(ctypes.c_size_t)],
    "ag_heap_reset": [_vp],
    "ag_heap_rank_ptr": [_vp, _c_int, _c_size, ctypes.POINTER(ctypes.c_void_p)],
    "ag_heap_base_table": [_vp, ctypes.POINTER(ctypes.c_void_p)],
    "ag_heap_geometry": [_vp, ctypes.POINTER(Geometry)],
    "ag_heap_info": [_vp, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                     ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_void_p)],
    "ag_heap_clear_tickets": [_vp, _vp],
    "ag_all_gather": [_vp, _c_int, _c_int, _c_int, _vp, _c_size, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                      _c_int, _vp],
    "ag_plan_all_gather": [ctypes.POINTER(Geometry), _c_int, _c_int, _c_int, _c_u64, _c_size, _c_i64, _c_i64,
                           _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(Plan)],
    "ag_all_gather_ex": [_vp, _c_int, _c_int, _c_int, _vp, _c_size, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                         _c_int, ctypes.POINTER(CopyOptions), _vp],
    "ag_plan_all_gather_ex": [ctypes.POINTER(Geometry), _c_int, _c_int, _c_int, _c_u64, _c_size, _c_i64, _c_i64,
                              _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(CopyOptions), ctypes.POINTER(Plan)],
    "ag_all_gather_noalloc": [_vp, _c_int, _c_int, _c_int, _vp, _c_size, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                              _c_int, ctypes.POINTER(CopyOptions), _vp],
    "ag_all_to_all": [_vp, _c_int, _c_int, _c_int, _vp, _c_size, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                      _c_int, _vp],
    "ag_plan_all_to_all": [ctypes.POINTER(Geometry), _c_int, _c_int, _c_int, _c_u64, _c_size, _c_i64, _c_i64,
                           _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(Plan)],
    "ag_all_to_all_ex": [_vp, _c_int, _c_int, _c_int, _vp, _c_size, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                         _c_int, ctypes.POINTER(CopyOptions), _vp],
    "ag_plan_all_to_all_ex": [ctypes.POINTER(Geometry), _c_int, _c_int, _c_int, _c_u64, _c_size, _c_i64, _c_i64,
                              _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(CopyOptions), ctypes.POINTER(Plan)],
    "ag_gemm_all_gather": [_vp, _c_int, _c_int, _c_int, _vp, _c_i64, _vp, _c_i64, _c_size, _c_i64, _c_i64,
                           _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int, _vp],
    "ag_plan_gemm_all_gather": [ctypes.POINTER(Geometry), _c_int, _c_int, _c_int, _c_u64, _c_i64, _c_u64, _c_i64,
                                _c_size, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int,
                                ctypes.POINTER(Plan)],
    "ag_gemm_all_gather_ex": [_vp, _c_int, _c_int, _c_int, _vp, _c_i64, _vp, _c_i64, _c_size, _c_i64, _c_i64,
                              _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(GemmOptions), _vp],
    "ag_plan_gemm_all_gather_ex": [ctypes.POINTER(Geometry), _c_int, _c_int, _c_int, _c_u64, _c_i64, _c_u64,
                                   _c_i64, _c_size, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   ctypes.POINTER(GemmOptions), ctypes.POINTER(Plan)],
    "ag_linear": [ctypes.POINTER(LinearArgs), _vp, _c_size, _vp],
    "ag_plan_linear": [ctypes.POINTER(LinearArgs), _c_int, ctypes.POINTER(LinearPlan)],
    "ag_linear_backward": [ctypes.POINTER(LinearBackwardArgs), _vp, _c_size, _vp],
    "ag_plan_linear_backward": [ctypes.POINTER(LinearBackwardArgs), _c_int, ctypes.POINTER(LinearPlan)],
    "ag_adamw_create": [ctypes.POINTER(AdamwTensor), _c_i64, _c_int, _c_int, _c_int, _HEAP_PP],
    "ag_adamw_destroy": [_vp],
    "ag_adamw_step": [_vp, ctypes.POINTER(AdamwHyper), _vp],
    "ag_adamw_read_states": [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp],
}


def lib() -> ctypes.CDLL:
    """The loaded libag.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m gemm_all_gather_amd.build` "
                               "(there is no fallback implementation)")
        l = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name in ("ag_status_string", "ag_last_error_message", "ag_version"):
            getattr(l, name).restype = ctypes.c_char_p
        l.ag_status_string.argtypes = [ctypes.c_int]
        _lib = l
    return _lib


def _check(status: int, call: str) -> None:
    if status != AG_OK:
        msg = lib().ag_last_error_message().decode()
        raise AgError(status, msg, call)


def version() -> str:
    return lib().ag_version().decode()


def heap_region_bytes(bytes_per_rank: int) -> int:
    """The region stride ag_heap_create uses for bytes_per_rank (the layout to give ag_heap_wrap too)."""
    out = ctypes.c_size_t(0)
    _check(lib().ag_heap_region_bytes(bytes_per_rank, ctypes.byref(out)), "ag_heap_region_bytes")
    return out.value


def _ptr(x) -> int:
    """Integer device address of a tensor (data_ptr) or an int."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream) -> Optional[int]:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _dtype(d) -> int:
    if isinstance(d, int):
        return d
    if isinstance(d, str):
        return DTYPE_CODES[d]
    import torch
    return {torch.float16: AG_F16, torch.bfloat16: AG_BF16, torch.float32: AG_F32}[d]


class Heap:
    """A handle of the symmetric heap: the root (rank -1) or a view of one rank."""

    def __init__(self, handle: int, keepalive=None):
        self._h = ctypes.c_void_p(handle)
        self._keepalive = keepalive

    @classmethod
    def create(cls, n_ranks: int, bytes_per_rank: int) -> "Heap":
        h = ctypes.c_void_p()
        _check(lib().ag_heap_create(n_ranks, bytes_per_rank, ctypes.byref(h)), "ag_heap_create")
        return cls(h.value)

    @classmethod
    def wrap(cls, slab, n_ranks: int, bytes_per_rank: int) -> "Heap":
        """Heap over caller memory (a device tensor of n_ranks*bytes_per_rank bytes, kept alive here)."""
        h = ctypes.c_void_p()
        _check(lib().ag_heap_wrap(_ptr(slab), n_ranks, bytes_per_rank, ctypes.byref(h)), "ag_heap_wrap")
        return cls(h.value, keepalive=slab)

    def view(self, rank: int) -> "Heap":
        h = ctypes.c_void_p()
        _check(lib().ag_heap_view(self._h, rank, ctypes.byref(h)), "ag_heap_view")
        return Heap(h.value, keepalive=self)

    def destroy(self) -> None:
        if self._h is not None and self._h.value:
            lib().ag_heap_destroy(self._h)
        self._h = None

    close = destroy

    def __del__(self):
        try:
            if self._h is not None and self._h.value and _lib is not None:
                _lib.ag_heap_destroy(self._h)
                self._h = None
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("heap handle already destroyed")
        return self._h

    def alloc(self, nbytes: int, align: int = 256) -> int:
        off = ctypes.c_size_t()
        _check(lib().ag_heap_alloc(self.handle, nbytes, align, ctypes.byref(off)), "ag_heap_alloc")
        return off.value

    def reset(self) -> None:
        _check(lib().ag_heap_reset(self.handle), "ag_heap_reset")

    def rank_ptr(self, rank: int, offset: int = 0) -> int:
        p = ctypes.c_void_p()
        _check(lib().ag_heap_rank_ptr(self.handle, rank, offset, ctypes.byref(p)), "ag_heap_rank_ptr")
        return p.value or 0

    def base_table(self) -> int:
        p = ctypes.c_void_p()
        _check(lib().ag_heap_base_table(self.handle, ctypes.byref(p)), "ag_heap_base_table")
        return p.value or 0

    def geometry(self) -> Geometry:
        g = Geometry()
        _check(lib().ag_heap_geometry(self.handle, ctypes.byref(g)), "ag_heap_geometry")
        return g

    def info(self) -> dict:
        """ag_heap_info: n_ranks, rank (-1 for the root handle), bytes_per_rank, base_table (device address)."""
        n, r, s, t = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t(), ctypes.c_void_p()
        _check(lib().ag_heap_info(self.handle, ctypes.byref(n), ctypes.byref(r), ctypes.byref(s), ctypes.byref(t)),
               "ag_heap_info")
        return {"n_ranks": n.value, "rank": r.value, "bytes_per_rank": s.value, "base_table": t.value or 0}

    def clear_tickets(self, stream=None) -> None:
        """ag_heap_clear_tickets: zero every rank's tile counters on stream."""
        _check(lib().ag_heap_clear_tickets(self.handle, _stream(stream)), "ag_heap_clear_tickets")


def plan_all_gather(geom: Geometry, W, rank_start, rank_stride, input_addr, out_offset, M_local, N, dtype,
                    tile_m=0, tile_n=0, n_programs=0) -> Plan:
    p = Plan()
    _check(lib().ag_plan_all_gather(ctypes.byref(geom), W, rank_start, rank_stride, _ptr(input_addr), out_offset,
                                    M_local, N, _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(p)),
           "ag_plan_all_gather")
    return p


def all_gather(heap: Heap, W, rank_start, rank_stride, input, out_offset, M_local, N, dtype,
               tile_m=0, tile_n=0, n_programs=0, stream=None) -> None:
    _check(lib().ag_all_gather(heap.handle, W, rank_start, rank_stride, _ptr(input), out_offset, M_local, N,
                               _dtype(dtype), tile_m, tile_n, n_programs, _stream(stream)), "ag_all_gather")


def plan_all_gather_ex(geom: Geometry, W, rank_start, rank_stride, input_addr, out_offset, M_local, N, dtype,
                       tile_m=0, tile_n=0, n_programs=0, dest_group=0, schedule=0, tile_order=0) -> Plan:
    p = Plan()
    o = _options(dest_group, schedule, tile_order)
    _check(lib().ag_plan_all_gather_ex(ctypes.byref(geom), W, rank_start, rank_stride, _ptr(input_addr), out_offset,
                                       M_local, N, _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(o),
                                       ctypes.byref(p)), "ag_plan_all_gather_ex")
    return p


def all_gather_ex(heap: Heap, W, rank_start, rank_stride, input, out_offset, M_local, N, dtype,
                  tile_m=0, tile_n=0, n_programs=0, dest_group=0, schedule=0, stream=None, tile_order=0) -> None:
    o = _options(dest_group, schedule, tile_order)
    _check(lib().ag_all_gather_ex(heap.handle, W, rank_start, rank_stride, _ptr(input), out_offset, M_local, N,
                                  _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(o), _stream(stream)),
           "ag_all_gather_ex")


def all_gather_noalloc(heap: Heap, W, rank_start, rank_stride, input, out_offset, M_local, N, dtype,
                       tile_m=0, tile_n=0, n_programs=0, dest_group=0, schedule=0, stream=None,
                       tile_order=0) -> None:
    """ag_all_gather_noalloc: ag_all_gather_ex whose tile counter is the library's fixed device array."""
    o = _options(dest_group, schedule, tile_order)
    _check(lib().ag_all_gather_noalloc(heap.handle, W, rank_start, rank_stride, _ptr(input), out_offset, M_local, N,
                                       _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(o), _stream(stream)),
           "ag_all_gather_noalloc")


def plan_all_to_all(geom: Geometry, W, rank_start, rank_stride, input_addr, out_offset, M_chunk, N, dtype,
                    tile_m=0, tile_n=0, n_programs=0) -> Plan:
    p = Plan()
    _check(lib().ag_plan_all_to_all(ctypes.byref(geom), W, rank_start, rank_stride, _ptr(input_addr), out_offset,
                                    M_chunk, N, _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(p)),
           "ag_plan_all_to_all")
    return p


def all_to_all(heap: Heap, W, rank_start, rank_stride, input, out_offset, M_chunk, N, dtype,
               tile_m=0, tile_n=0, n_programs=0, stream=None) -> None:
    _check(lib().ag_all_to_all(heap.handle, W, rank_start, rank_stride, _ptr(input), out_offset, M_chunk, N,
                               _dtype(dtype), tile_m, tile_n, n_programs, _stream(stream)), "ag_all_to_all")


def plan_all_to_all_ex(geom: Geometry, W, rank_start, rank_stride, input_addr, out_offset, M_chunk, N, dtype,
                       tile_m=0, tile_n=0, n_programs=0, dest_group=0, schedule=0, tile_order=0) -> Plan:
    p = Plan()
    o = _options(dest_group, schedule, tile_order)
    _check(lib().ag_plan_all_to_all_ex(ctypes.byref(geom), W, rank_start, rank_stride, _ptr(input_addr), out_offset,
                                       M_chunk, N, _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(o),
                                       ctypes.byref(p)), "ag_plan_all_to_all_ex")
    return p


def all_to_all_ex(heap: Heap, W, rank_start, rank_stride, input, out_offset, M_chunk, N, dtype,
                  tile_m=0, tile_n=0, n_programs=0, dest_group=0, schedule=0, stream=None, tile_order=0) -> None:
    o = _options(dest_group, schedule, tile_order)
    _check(lib().ag_all_to_all_ex(heap.handle, W, rank_start, rank_stride, _ptr(input), out_offset, M_chunk, N,
                                  _dtype(dtype), tile_m, tile_n, n_programs, ctypes.byref(o), _stream(stream)),
           "ag_all_to_all_ex")


def plan_gemm_all_gather(geom: Geometry, W, rank_start, rank_stride, a_addr, lda, b_addr, ldb, out_offset,
                         M_local, N, K, dtype, tile_m=0, tile_n=0, tile_k=0, n_programs=0) -> Plan:
    p = Plan()
    _check(lib().ag_plan_gemm_all_gather(ctypes.byref(geom), W, rank_start, rank_stride, _ptr(a_addr), lda,
                                         _ptr(b_addr), ldb, out_offset, M_local, N, K, _dtype(dtype), tile_m,
                                         tile_n, tile_k, n_programs, ctypes.byref(p)), "ag_plan_gemm_all_gather")
    return p


def gemm_all_gather(heap: Heap, W, rank_start, rank_stride, A, lda, B, ldb, out_offset, M_local, N, K, dtype,
                    tile_m=0, tile_n=0, tile_k=0, n_programs=0, stream=None) -> None:
    _check(lib().ag_gemm_all_gather(heap.handle, W, rank_start, rank_stride, _ptr(A), lda, _ptr(B), ldb,
                                    out_offset, M_local, N, K, _dtype(dtype), tile_m, tile_n, tile_k, n_programs,
                                    _stream(stream)), "ag_gemm_all_gather")


def _gemm_options(b_layout=0) -> GemmOptions:
    o = GemmOptions()
    o.b_layout = B_LAYOUTS[b_layout] if isinstance(b_layout, str) else b_layout
    return o


def plan_gemm_all_gather_ex(geom: Geometry, W, rank_start, rank_stride, a_addr, lda, b_addr, ldb, out_offset,
                            M_local, N, K, dtype, tile_m=0, tile_n=0, tile_k=0, n_programs=0, b_layout=0) -> Plan:
    """b_layout: "k" (element (k,n) at B[n*ldb + k]) or "n" (at B[k*ldb + n])."""
    p = Plan()
    o = _gemm_options(b_layout)
    _check(lib().ag_plan_gemm_all_gather_ex(ctypes.byref(geom), W, rank_start, rank_stride, _ptr(a_addr), lda,
                                            _ptr(b_addr), ldb, out_offset, M_local, N, K, _dtype(dtype), tile_m,
                                            tile_n, tile_k, n_programs, ctypes.byref(o), ctypes.byref(p)),
           "ag_plan_gemm_all_gather_ex")
    return p


def gemm_all_gather_ex(heap: Heap, W, rank_start, rank_stride, A, lda, B, ldb, out_offset, M_local, N, K, dtype,
                       tile_m=0, tile_n=0, tile_k=0, n_programs=0, b_layout=0, stream=None) -> None:
    o = _gemm_options(b_layout)
    _check(lib().ag_gemm_all_gather_ex(heap.handle, W, rank_start, rank_stride, _ptr(A), lda, _ptr(B), ldb,
                                       out_offset, M_local, N, K, _dtype(dtype), tile_m, tile_n, tile_k, n_programs,
                                       ctypes.byref(o), _stream(stream)), "ag_gemm_all_gather_ex")


def _act(act) -> int:
    return ACTS[act] if isinstance(act, str) else act


def _workspace(workspace):
    """Address and bytes of a workspace: a tensor, or None."""
    if workspace is None:
        return 0, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _linear_args(M, N, K, dtype, act, x, w, y, bias, residual, z, ldx, ldw, ldr, ldy, ldz) -> LinearArgs:
    return LinearArgs(_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y), _ptr(z), ldx, ldw, ldr, ldy, ldz, M, N, K,
                      _dtype(dtype), _act(act))


def plan_linear(x, w, y, M, N, K, dtype, act="none", bias=None, residual=None, z=None, ldx=0, ldw=0, ldr=0, ldy=0,
                ldz=0, num_cus=0) -> LinearPlan:
    p = LinearPlan()
    a = _linear_args(M, N, K, dtype, act, x, w, y, bias, residual, z, ldx, ldw, ldr, ldy, ldz)
    _check(lib().ag_plan_linear(ctypes.byref(a), num_cus, ctypes.byref(p)), "ag_plan_linear")
    return p


def linear(x, w, y, M, N, K, dtype, act="none", bias=None, residual=None, z=None, ldx=0, ldw=0, ldr=0, ldy=0, ldz=0,
           workspace=None, stream=None) -> None:
    """y = act(x w^T + bias) + residual; z, if given, receives the pre-activation (ag_linear)."""
    a = _linear_args(M, N, K, dtype, act, x, w, y, bias, residual, z, ldx, ldw, ldr, ldy, ldz)
    ws, nbytes = _workspace(workspace)
    _check(lib().ag_linear(ctypes.byref(a), ws, nbytes, _stream(stream)), "ag_linear")


def _backward_args(M, N, K, dtype, act, dy, x, w, z, dx, dw, db, lddy, ldx, ldw, ldz, lddx, lddw, dw_dtype,
                   accumulate) -> LinearBackwardArgs:
    return LinearBackwardArgs(_ptr(dy), _ptr(z), _ptr(x), _ptr(w), _ptr(dx), _ptr(dw), _ptr(db), lddy, ldz, ldx, ldw,
                              lddx, lddw, M, N, K, _dtype(dtype), _act(act),
                              _dtype(dtype if dw_dtype is None else dw_dtype), int(accumulate))


def plan_linear_backward(dy, x, w, M, N, K, dtype, act="none", z=None, dx=None, dw=None, db=None, lddy=0, ldx=0, ldw=0,
                         ldz=0, lddx=0, lddw=0, dw_dtype=None, accumulate=False, num_cus=0) -> LinearPlan:
    p = LinearPlan()
    a = _backward_args(M, N, K, dtype, act, dy, x, w, z, dx, dw, db, lddy, ldx, ldw, ldz, lddx, lddw, dw_dtype,
                       accumulate)
    _check(lib().ag_plan_linear_backward(ctypes.byref(a), num_cus, ctypes.byref(p)), "ag_plan_linear_backward")
    return p


def linear_backward(dy, x, w, M, N, K, dtype, act="none", z=None, dx=None, dw=None, db=None, lddy=0, ldx=0, ldw=0,
                    ldz=0, lddx=0, lddw=0, dw_dtype=None, accumulate=False, workspace=None, stream=None) -> None:
    """The gradients dx, dw and db that are given, from dy and the stored pre-activation z (ag_linear_backward)."""
    a = _backward_args(M, N, K, dtype, act, dy, x, w, z, dx, dw, db, lddy, ldx, ldw, ldz, lddx, lddw, dw_dtype,
                       accumulate)
    ws, nbytes = _workspace(workspace)
    _check(lib().ag_linear_backward(ctypes.byref(a), ws, nbytes, _stream(stream)), "ag_linear_backward")


def _reachable(tensors) -> bool:
    """Whether kernels can reach the tensors' elements: device memory, or pinned host memory."""
    import torch
    return min(map(torch.Tensor.get_device, tensors), default=0) >= 0 or \
        all(t.is_cuda or t.numel() == 0 or t.is_pinned() for t in tensors)


def _scalar(x, name, dtype) -> int:
    """Address of a device scalar: None, an address, or a tensor whose first element the kernel reads."""
    if x is None or isinstance(x, int):
        return x or 0
    import torch
    if x.dtype != getattr(torch, dtype) or x.numel() < 1:
        raise ValueError(f"{name} is not a tensor of one {dtype}")
    if not _reachable([x]):
        raise ValueError(f"{name} lies in host memory that is not pinned")
    return int(x.data_ptr())


class AdamW:
    """ag_adamw: a device table of tensors, made once; ``step`` updates all of them in one launch.

    Lists (or other iterables) of device tensors, equally many, each contiguous; 8-bit states are int8 and uint8
    tensors with their fp32 block maxima in exp_avg_scales and exp_avg_sq_scales.  The tensors are kept alive here,
    whatever becomes of the lists, and must keep their addresses (clear gradients in place).
    """

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, masters=None, exp_avg_scales=None,
                 exp_avg_sq_scales=None):
        import torch
        # tuples of the tensors: the caller's lists may change while the device table holds these addresses
        parts = [part if part is None else tuple(part) for part in
                 (params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales, exp_avg_sq_scales, masters)]
        params, grads, exp_avgs = parts[:3]
        count = len(params)
        if any(part is not None and len(part) != count for part in parts):
            raise ValueError("the lists of tensors differ in length")
        state8 = count > 0 and exp_avgs[0].dtype == torch.int8
        wanted = [None, None, torch.int8 if state8 else torch.float32, torch.uint8 if state8 else torch.float32,
                  torch.float32, torch.float32, torch.float32]
        for i, (part, dtype) in enumerate(zip(parts, wanted)):
            if part is None:
                continue
            for t, p in zip(part, params):
                need = -(-p.numel() // AG_ADAMW_BLOCK) if i in (4, 5) else p.numel()     # block maxima
                if not t.is_contiguous() or t.numel() != need or t.dtype != (dtype or part[0].dtype):
                    raise ValueError(f"a tensor is not contiguous, not of {need} elements or not {dtype or part[0].dtype}")
            if not _reachable(part):
                raise ValueError("a tensor lies in host memory that is not pinned")
        table = (AdamwTensor * max(1, count))()
        for i, p in enumerate(params):
            table[i] = AdamwTensor(*(_ptr(part[i]) if part is not None else 0 for part in parts), p.numel())
        h = ctypes.c_void_p()
        _check(lib().ag_adamw_create(table, count, _dtype(params[0].dtype) if count else AG_F32,
                                     _dtype(grads[0].dtype) if count else AG_F32, 8 if state8 else 32,
                                     ctypes.byref(h)), "ag_adamw_create")
        self._h = h
        self._keepalive = parts
        self._sizes = [p.numel() for p in params]
        T = torch.Tensor
        self._reads = T.numel, T.is_contiguous, attrgetter("dtype"), T.get_device, T.data_ptr, {torch.float32}
        self._pointers = _vp * count

    def destroy(self) -> None:
        if self._h is not None and self._h.value:
            lib().ag_adamw_destroy(self._h)
        self._h = None

    close = destroy

    def __del__(self):
        try:
            if getattr(self, "_h", None) is not None and _lib is not None:
                _lib.ag_adamw_destroy(self._h)
                self._h = None
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("optimizer handle already destroyed")
        return self._h

    def step(self, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0, seed=None,
             dev_step=None, dev_lr=None, dev_grad_scale=None, stream=None) -> None:
        """One AdamW step; a seed (8-bit states) turns stochastic rounding on (ag_adamw_step).

        dev_step (int64), dev_lr and dev_grad_scale (fp32) are one-element device tensors or device addresses.
        """
        y = AdamwHyper(lr, beta1, beta2, eps, weight_decay, grad_scale, step, _scalar(dev_step, "dev_step", "int64"),
                       _scalar(dev_lr, "dev_lr", "float32"), _scalar(dev_grad_scale, "dev_grad_scale", "float32"),
                       0 if seed is None else seed, 0 if seed is None else 1)
        _check(lib().ag_adamw_step(self.handle, ctypes.byref(y), _stream(stream)), "ag_adamw_step")

    def _addresses(self, outputs):
        """The outputs' addresses, each tensor checked first (by whole lists: there may be hundreds a call)."""
        if int in set(map(type, outputs)):      # addresses among them are taken as they are
            at = [t if isinstance(t, int) else self._addresses_of([t], [n])[0] for t, n in zip(outputs, self._sizes * 2)]
            return array("Q", at)
        return self._addresses_of(outputs, self._sizes * 2)

    def _addresses_of(self, tensors, sizes):
        numel, contiguous, dtype, device, data_ptr, fp32 = self._reads
        if list(map(numel, tensors)) != sizes or not all(map(contiguous, tensors)) or not fp32.issuperset(map(dtype, tensors)):
            raise ValueError("an output is not contiguous, not of its parameter's elements or not fp32")
        if min(map(device, tensors), default=0) < 0 and not _reachable(tensors):
            raise ValueError("an output lies in host memory that is not pinned")
        return array("Q", map(data_ptr, tensors))

    def read_states(self, exp_avgs, exp_avg_sqs, stream=None) -> None:
        """The fp32 values of 8-bit states, into two lists of fp32 tensors, contiguous and of each parameter's
        elements (or device addresses of as many floats) (ag_adamw_read_states)."""
        m, v, n = tuple(exp_avgs), tuple(exp_avg_sqs), len(self._sizes)
        if len(m) != n or len(v) != n:
            raise ValueError("the lists of tensors differ in length")
        at = self._addresses(m + v)
        m, v = self._pointers.from_buffer(at), self._pointers.from_buffer(at, n * at.itemsize)
        _check(lib().ag_adamw_read_states(self.handle, m, v, _stream(stream)), "ag_adamw_read_states")
