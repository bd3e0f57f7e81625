"""ctypes binding of libmoe (include/moe.h): argument marshalling only.

Every function here passes raw device pointers, sizes and the current CUDA
stream to the C ABI of the same name; all the layer's work runs in the
library's kernels. Tensors are torch tensors on the GPU (PyTorch provides the
device memory and the stream), except where a name ends in ``_host``.

Importing this module raises if libmoe.so has not been built: there is no
fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_OVERFLOW", 6: "MOE_ERR_HOST"}
BF16, FP16, FP32 = 0, 1, 2
ACT_NONE, ACT_SWIGLU = 0, 1
DEV_BAD_INDEX, DEV_BAD_SLOT, DEV_NONFINITE, DEV_MISS_OVERFLOW, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10

_P = C.c_void_p
_I = C.c_int
_I32 = C.c_int32
_SZ = C.c_size_t


class QPool(C.Structure):
    _fields_ = [("base", _P), ("slot_bytes", C.c_int64), ("num_slots", _I32), ("fmt", _I32), ("d", _I32),
                ("f", _I32)]


class QMatrix(C.Structure):
    _fields_ = [("codes", _P), ("hi", _P), ("scale", _P), ("min", _P)]


class Q4Weights(C.Structure):
    _fields_ = [("codes", _P), ("scale", _P), ("min", _P), ("num_slots", _I32), ("N", _I32), ("K", _I32),
                ("group", _I32)]
    tensors = ()    # kept alive; empty where the addresses were filled in by hand


class Swap(C.Structure):
    _fields_ = [("slot", _I32), ("layer_in", _I32), ("expert_in", _I32), ("layer_out", _I32), ("expert_out", _I32)]


class Miss(C.Structure):
    _fields_ = [("layer", _I32), ("expert", _I32), ("token", _I32), ("j", _I32), ("gate", C.c_float)]


MISS_BYTES = C.sizeof(Miss)

# name -> (restype, argtypes), mirroring include/moe.h
SIGNATURES = {
    "moe_status_str": (C.c_char_p, [_I]),
    "moe_version": (_I, []),
    "moe_expert_bytes": (_SZ, [_I, _I, _I]),
    "moe_pack_expert": (_I, [_I, _I, _I, C.POINTER(QMatrix), C.POINTER(QMatrix), C.POINTER(QMatrix), _P, _P]),
    "moe_pack_expert_host": (_I, [_I, _I, _I, C.POINTER(QMatrix), C.POINTER(QMatrix), C.POINTER(QMatrix), _P]),
    "moe_unpack_expert_host": (_I, [_I, _I, _I, _P, C.POINTER(QMatrix), C.POINTER(QMatrix), C.POINTER(QMatrix)]),
    "moe_route": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_permute_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_permute": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "moe_cache_lookup": (_I, [_P, _I32, _I32, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _I32, _P, _P, _P]),
    "moe_expert_ffn_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_expert_ffn_q2": (_I, [C.POINTER(QPool), _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P,
                               _P]),
    "moe_expert_ffn_q3": (_I, [C.POINTER(QPool), _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P,
                               _P]),
    "moe_expert_ffn_q2_noalloc": (_I, [C.POINTER(QPool), _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                       _P]),
    "moe_combine": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_layer_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_layer_decode": (_I, [C.POINTER(QPool), _P, _I32, _I32, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                              _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P, _P]),
    "moe_stack_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_stack_decode": (_I, [C.POINTER(QPool), _I, _P, _P, _I32, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                              _P, _I32, _P, _P, _P, _SZ, _P, _P]),
    "moe_complete_misses_host": (_I, [_I, _I, _I, _P, _I, _P, _I32, _I32, _P, _I, _P, _I]),
    "moe_debug_wait_probe": (_I, [_P, C.c_uint32, _P, _P, _P]),
    "moe_linear_q4": (_I, [_P, _I32, _P, _I, _I, _I, _P, _I, _P]),
    "moe_expert_linear_q4": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P]),
    "moe_expert_gemm": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I, _P, _P]),
    "moe_expert_gemm_dgrad": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P]),
    "moe_expert_gemm_wgrad": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _P]),
    "moe_swiglu": (_I, [_P, _I, C.c_int64, _I, _P, _P]),
    "moe_swiglu_backward": (_I, [_P, _P, _I, C.c_int64, _I, _P, _P]),
    "moe_miss_engine_create": (_I, [_I, C.POINTER(_P)]),
    "moe_miss_engine_submit": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _I32, _I32, _P, _I, _P]),
    "moe_miss_engine_wait": (_I, [_P]),
    "moe_miss_engine_destroy": (None, [_P]),
    "moe_cache_policy_bytes": (_SZ, [_I, _I]),
    "moe_cache_policy_init": (_I, [_P, _SZ, _I, _I, _I, _I, _I]),
    "moe_cache_policy_observe": (_I, [_P, _I, _P, _I, _I]),
    "moe_cache_policy_observe_counts": (_I, [_P, _P, _I]),
    "moe_cache_policy_plan": (_I32, [_P, _P, _P, _I32]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoe.so is not built ({LIB_PATH}); run `python -m bit_expert_ffn_fp32_b200.build`")
    lib = C.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {lib.moe_status_str(code).decode()}")
        self.code = code


def check(fn: str, code: int) -> None:
    if code != MOE_OK:
        raise MoeError(fn, code)


def ptr(t) -> int | None:
    """Device (or host) address of a tensor/array, None for None."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data  # numpy


def stream_handle(stream=None) -> int | None:
    """cudaStream_t of a torch stream, by default the current GPU's current one."""
    if stream is not None:
        return stream.cuda_stream or None
    if _Types.device is None:
        _Types.load()
    return _Types.raw_stream(_Types.device()) or None


def qmatrix(codes, scale, mn=None, hi=None) -> QMatrix:
    return QMatrix(ptr(codes), ptr(hi), ptr(scale), ptr(mn))


def qpool(base, slot_bytes: int, num_slots: int, fmt: int, d: int, f: int) -> QPool:
    return QPool(ptr(base), slot_bytes, num_slots, fmt, d, f)


# ------------------------------------------------------------------ thin wrappers
def expert_bytes(fmt: int, d: int, f: int) -> int:
    return int(lib.moe_expert_bytes(fmt, d, f))


def pack_expert(fmt, d, f, gate: QMatrix, up: QMatrix, down: QMatrix, dst_ptr: int, stream=None) -> None:
    check("moe_pack_expert", lib.moe_pack_expert(fmt, d, f, C.byref(gate), C.byref(up), C.byref(down), dst_ptr,
                                                 stream_handle(stream)))


def pack_expert_host(fmt, d, f, gate: QMatrix, up: QMatrix, down: QMatrix, dst_ptr: int) -> None:
    check("moe_pack_expert_host", lib.moe_pack_expert_host(fmt, d, f, C.byref(gate), C.byref(up), C.byref(down),
                                                           dst_ptr))


def unpack_expert_host(fmt, d, f, src_ptr: int, gate: QMatrix, up: QMatrix, down: QMatrix) -> None:
    check("moe_unpack_expert_host", lib.moe_unpack_expert_host(fmt, d, f, src_ptr, C.byref(gate), C.byref(up),
                                                               C.byref(down)))


def route(x, Wr, bias, T, d, E, k, logits, topk_idx, topk_w, dev_status=None, stream=None) -> None:
    check("moe_route", lib.moe_route(ptr(x), ptr(Wr), ptr(bias), T, d, E, k, ptr(logits), ptr(topk_idx),
                                     ptr(topk_w), ptr(dev_status), stream_handle(stream)))


def permute_workspace_bytes(T, k, E) -> int:
    return int(lib.moe_permute_workspace_bytes(T, k, E))


def permute(topk_idx, T, k, E, counts, offsets, sorted_tok, sorted_j, inv, active, ws=None, ws_bytes=0,
            dev_status=None, stream=None) -> None:
    check("moe_permute", lib.moe_permute(ptr(topk_idx), T, k, E, ptr(counts), ptr(offsets), ptr(sorted_tok),
                                         ptr(sorted_j), ptr(inv), ptr(active), ptr(ws), ws_bytes, ptr(dev_status),
                                         stream_handle(stream)))


def cache_lookup(slot_of, num_slots, layer, topk_idx, topk_w, offsets, sorted_tok, sorted_j, T, k, E,
                 slot_of_pair, miss, miss_count, miss_cap, dev_status=None, stream=None, expert_counts=None) -> None:
    check("moe_cache_lookup", lib.moe_cache_lookup(ptr(slot_of), num_slots, layer, ptr(topk_idx), ptr(topk_w),
                                                   ptr(offsets), ptr(sorted_tok), ptr(sorted_j), T, k, E,
                                                   ptr(slot_of_pair), ptr(miss), ptr(miss_count), miss_cap,
                                                   ptr(expert_counts), ptr(dev_status), stream_handle(stream)))


def expert_ffn_workspace_bytes(T, k, d, f) -> int:
    return int(lib.moe_expert_ffn_workspace_bytes(T, k, d, f))


def expert_ffn(pool: QPool, slot_of, x, T, d, f, E, k, offsets, sorted_tok, sorted_j, active, topk_w, out, ws,
               ws_bytes, dev_status=None, stream=None) -> None:
    fn = lib.moe_expert_ffn_q2 if pool.fmt == 2 else lib.moe_expert_ffn_q3
    name = "moe_expert_ffn_q2" if pool.fmt == 2 else "moe_expert_ffn_q3"
    check(name, fn(C.byref(pool), ptr(slot_of), ptr(x), T, d, f, E, k, ptr(offsets), ptr(sorted_tok),
                   ptr(sorted_j), ptr(active), ptr(topk_w), ptr(out), ptr(ws), ws_bytes, ptr(dev_status),
                   stream_handle(stream)))


def expert_ffn_q2_noalloc(pool: QPool, slot_of, x, T, d, f, E, k, offsets, sorted_tok, sorted_j, active, topk_w,
                          out, dev_status=None, stream=None) -> None:
    """moe_expert_ffn_q2 with the library's built-in scratch instead of a workspace."""
    check("moe_expert_ffn_q2_noalloc",
          lib.moe_expert_ffn_q2_noalloc(C.byref(pool), ptr(slot_of), ptr(x), T, d, f, E, k, ptr(offsets),
                                        ptr(sorted_tok), ptr(sorted_j), ptr(active), ptr(topk_w), ptr(out),
                                        ptr(dev_status), stream_handle(stream)))


def combine(y_perm, inv, topk_w, slot_of_pair, y_shared, T, k, d, y, stream=None) -> None:
    check("moe_combine", lib.moe_combine(ptr(y_perm), ptr(inv), ptr(topk_w), ptr(slot_of_pair), ptr(y_shared), T,
                                         k, d, ptr(y), stream_handle(stream)))


def layer_decode_workspace_bytes(T, k, f, E) -> int:
    return int(lib.moe_layer_decode_workspace_bytes(T, k, f, E))


def layer_decode(pool: QPool, slot_of, shared_slot: int, layer: int, x, Wr, bias, T, d, f, E, k, logits=None,
                 topk_idx=None, topk_w=None, counts=None, offsets=None, sorted_tok=None, sorted_j=None, inv=None,
                 active=None, slot_of_pair=None, miss=None, miss_count=None, miss_cap=0, y=None, ws=None,
                 ws_bytes=0, dev_status=None, stream=None, expert_counts=None) -> None:
    check("moe_layer_decode",
          lib.moe_layer_decode(C.byref(pool), ptr(slot_of), shared_slot, layer, ptr(x), ptr(Wr), ptr(bias), T, d, f,
                               E, k, ptr(logits), ptr(topk_idx), ptr(topk_w), ptr(counts), ptr(offsets),
                               ptr(sorted_tok), ptr(sorted_j), ptr(inv), ptr(active), ptr(slot_of_pair), ptr(miss),
                               ptr(miss_count), miss_cap, ptr(expert_counts), ptr(y), ptr(ws), ws_bytes,
                               ptr(dev_status), stream_handle(stream)))


def stack_decode(pool: QPool, L: int, slot_of, shared_slot, layer0: int, x, Wr, bias, T, d, f, E, k, topk_idx=None,
                 topk_w=None, slot_of_pair=None, miss=None, miss_count=None, miss_cap=0, y=None, ws=None,
                 ws_bytes=0, dev_status=None, stream=None, expert_counts=None) -> None:
    check("moe_stack_decode",
          lib.moe_stack_decode(C.byref(pool), L, ptr(slot_of), ptr(shared_slot), layer0, ptr(x), ptr(Wr), ptr(bias),
                               T, d, f, E, k, ptr(topk_idx), ptr(topk_w), ptr(slot_of_pair), ptr(miss),
                               ptr(miss_count), miss_cap, ptr(expert_counts), ptr(y), ptr(ws), ws_bytes,
                               ptr(dev_status), stream_handle(stream)))


def expert_table(E: int, experts: dict) -> C.Array:
    """moe_qmatrix [E][3] (gate, up, down) for the experts given as
    {e: canonical expert dict}; absent experts get NULL matrices. The arrays
    must stay alive while the table is used."""
    tab = (QMatrix * (3 * E))()
    for e, ex in experts.items():
        for i, m in enumerate(("gate", "up", "down")):
            tab[3 * e + i] = qmatrix(ex[m]["codes"], ex[m]["scale"], ex[m]["min"], ex[m]["hi"])
    return tab


def complete_misses_host(fmt: int, d: int, f: int, experts: C.Array, E: int, miss, n: int, layer: int, x, T: int, y,
                         nthreads: int = 0) -> None:
    """Host completion of a layer's miss list (host arrays: experts from
    expert_table, miss records, x uint16 [T][d], y float32 [T][d] accumulated
    in place)."""
    check("moe_complete_misses_host",
          lib.moe_complete_misses_host(fmt, d, f, C.cast(experts, _P), E, ptr(miss), n, layer, ptr(x), T, ptr(y),
                                       nthreads))


class MissEngine:
    """moe_miss_engine: host worker threads completing miss lists as they are
    published (see include/moe.h). Submitted arrays must stay alive until
    wait() returns; the engine keeps references to them until then."""

    def __init__(self, nthreads: int = 0):
        h = _P()
        check("moe_miss_engine_create", lib.moe_miss_engine_create(nthreads, C.byref(h)))
        self.h = h
        self._keep = []

    def submit(self, fmt: int, d: int, f: int, experts: C.Array, E: int, miss, count, miss_cap: int, layer: int, x,
               T: int, y) -> None:
        """miss: host records (e.g. a pinned tensor the GPU writes), count: host
        int32 whose value becomes >= 0 when the records are complete."""
        self._keep.append((experts, miss, count, x, y))
        check("moe_miss_engine_submit",
              lib.moe_miss_engine_submit(self.h, fmt, d, f, C.cast(experts, _P), E, ptr(miss), ptr(count), miss_cap,
                                         layer, ptr(x), T, ptr(y)))

    def wait(self) -> None:
        code = lib.moe_miss_engine_wait(self.h)
        self._keep.clear()
        check("moe_miss_engine_wait", code)

    def close(self) -> None:
        if self.h:
            lib.moe_miss_engine_destroy(self.h)
            self.h = None
            self._keep.clear()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class CachePolicy:
    """Host expert-cache policy (moe_cache_policy_*): counts of routed pairs,
    halved every `epoch` tokens, and slot plans against an [L][E] slot table."""

    def __init__(self, L: int, E: int, S: int, epoch: int, margin: int = 0):
        import numpy as np

        n = int(lib.moe_cache_policy_bytes(L, E))
        if n == 0:
            raise MoeError("moe_cache_policy_bytes", 2)
        self.L, self.E, self.S = L, E, S
        self.state = np.zeros(n, np.uint8)
        check("moe_cache_policy_init", lib.moe_cache_policy_init(self.state.ctypes.data, n, L, E, S, epoch, margin))

    def observe(self, layer: int, topk_idx) -> None:
        import numpy as np

        idx = np.ascontiguousarray(topk_idx, dtype=np.int32)
        T, k = idx.shape
        check("moe_cache_policy_observe", lib.moe_cache_policy_observe(self.state.ctypes.data, layer, idx.ctypes.data,
                                                                       T, k))

    def observe_counts(self, counts, tokens: int) -> None:
        """A window of `tokens` token steps from per-expert counts (int32 [L][E])."""
        import numpy as np

        c = np.ascontiguousarray(counts, dtype=np.int32)
        check("moe_cache_policy_observe_counts",
              lib.moe_cache_policy_observe_counts(self.state.ctypes.data, c.ctypes.data, tokens))

    def plan(self, slot_of, max_swaps: int) -> list:
        """Update slot_of (int32 [L][E] numpy, in place); the changes as tuples
        (slot, layer_in, expert_in, layer_out, expert_out)."""
        buf = (Swap * max(1, max_swaps))()
        n = int(lib.moe_cache_policy_plan(self.state.ctypes.data, slot_of.ctypes.data, buf, max_swaps))
        if n < 0:
            raise MoeError("moe_cache_policy_plan", -n)
        return [(buf[i].slot, buf[i].layer_in, buf[i].expert_in, buf[i].layer_out, buf[i].expert_out)
                for i in range(n)]


def debug_wait_probe(counter, target: int, elapsed_ns, dev_status, stream=None) -> None:
    """moe_debug_wait_probe: the library's bounded waits against a counter below
    target and an mbarrier phase nothing completes (device tensors)."""
    check("moe_debug_wait_probe", lib.moe_debug_wait_probe(ptr(counter), target, ptr(elapsed_ns), ptr(dev_status),
                                                           stream_handle(stream)))


# ------------------------------------------------------------------ 4-bit and unquantised products, gradients
class _Types:
    """torch's types and their moe_dtype codes, once torch is loaded."""
    code: dict = {}
    int32 = device = raw_stream = None

    @classmethod
    def load(cls) -> None:
        import torch
        # the handle alone, where torch has it: torch.cuda.current_stream() builds a Stream around it (3.4 us a call
        # against 0.3)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.raw_stream = staticmethod(raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
        cls.int32 = torch.int32
        # last, what callers look at to see whether the rest is there: another thread may look meanwhile; int16
        # tensors hold bf16 bits, as for the layer's x
        cls.device = torch.cuda.current_device
        cls.code = {torch.bfloat16: BF16, torch.int16: BF16, torch.float16: FP16, torch.float32: FP32}


def dtype_code(t) -> int:
    """moe_dtype of a tensor (int16 = bf16 bits)."""
    if not _Types.code:
        _Types.load()
    code = _Types.code.get(t.dtype)
    if code is None:
        raise ValueError(f"no moe_dtype for {t.dtype}: bfloat16 (or int16 bits), float16 and float32 are known")
    return code


def _address(t, n: int, dev: int) -> int:
    """Address of a tensor, looked at before it goes to the library: contiguous,
    on GPU `dev`, of n elements at least."""
    if t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"a contiguous tensor of {n} or more elements on GPU {dev} is wanted, got {tuple(t.shape)}, "
                         f"strides {t.stride()}, on {t.device}")
    return t.data_ptr()


def _table(t, n: int, dev: int) -> int | None:
    """_address of an int32 table, None for None."""
    if t is None:
        return None
    if t.dtype != _Types.int32:
        raise ValueError(f"an int32 tensor is wanted, got {t.dtype}")
    return _address(t, n, dev)


def _stream_on(stream, dev: int) -> int | None:
    """stream_handle where the current GPU is known."""
    return (_Types.raw_stream(dev) if stream is None else stream.cuda_stream) or None


def _place_of(t) -> int:
    """The GPU of a tensor, which has to be the current one: the library launches there."""
    if _Types.device is None:
        _Types.load()
    dev = t.get_device()
    if dev < 0:
        raise ValueError("GPU tensors are wanted")
    if dev != _Types.device():
        raise ValueError(f"the tensors are on GPU {dev}, the current GPU is {_Types.device()}")
    return dev


def q4_weights(codes, scale, min, group: int) -> Q4Weights:
    """moe_q4weights over codes uint8 [slots][N][K/2], scale and min fp16
    [slots][N][K/group] (min None: w = s*(q-8)); one matrix may leave the slots
    out. The description keeps the tensors alive."""
    import torch
    if codes.dtype != torch.uint8 or codes.dim() not in (2, 3):
        raise ValueError("codes: uint8 [slots][N][K/2]")
    slots, N, half = codes.shape if codes.dim() == 3 else (1, *codes.shape)
    if group not in (32, 64, 128) or 2 * half % group:
        raise ValueError("group: 32, 64 or 128, a divisor of K")
    for t in (scale, min):
        if t is not None and (t.dtype not in (torch.float16, torch.int16) or
                              t.shape != (*codes.shape[:-1], 2 * half // group)):
            raise ValueError("scale, min: fp16 [slots][N][K/group]")
    for t in (codes, scale, min):
        if t is not None and not (t.is_contiguous() and t.device == codes.device):
            raise ValueError("codes, scale, min: contiguous, on one GPU")
    w = Q4Weights(ptr(codes), ptr(scale), ptr(min), slots, N, 2 * half, group)
    w.tensors = (codes, scale, min)
    return w


def linear_q4(W: Q4Weights, slot: int, x, T: int, out, act: int = ACT_NONE, stream=None) -> None:
    """out[t] = W[slot] x[t]; out [T][N] (SwiGLU: [T][N/2]) in x's type or fp32."""
    dev = _place_of(W.tensors[0] if W.tensors else x)
    code = lib.moe_linear_q4(C.addressof(W), slot, _address(x, T * W.K, dev), dtype_code(x), T, act,
                             _address(out, T * W.N // (1 + (act == ACT_SWIGLU)), dev), dtype_code(out),
                             _stream_on(stream, dev))
    if code:
        raise MoeError("moe_linear_q4", code)


def expert_linear_q4(W: Q4Weights, slot_of, x, T: int, E: int, k: int, offsets, sorted_tok, active, out,
                     act: int = ACT_NONE, dev_status=None, stream=None) -> None:
    """out[s] = W[slot_of[e]] x_s for the sorted pairs s of every active expert e
    (x_s = x[sorted_tok[s]], or x[s] with sorted_tok None)."""
    dev, P = _place_of(W.tensors[0] if W.tensors else x), T * k
    code = lib.moe_expert_linear_q4(C.addressof(W), _table(slot_of, E, dev),
                                    _address(x, (P if sorted_tok is None else T) * W.K, dev), dtype_code(x), T, E, k,
                                    _table(offsets, E + 1, dev), _table(sorted_tok, P, dev),
                                    _table(active, E + 1, dev), act,
                                    _address(out, P * W.N // (1 + (act == ACT_SWIGLU)), dev), dtype_code(out),
                                    _table(dev_status, 1, dev), _stream_on(stream, dev))
    if code:
        raise MoeError("moe_expert_linear_q4", code)


def expert_gemm(a, W, T: int, E: int, k: int, N: int, K: int, offsets, sorted_tok, out, dev_status=None,
                stream=None) -> None:
    """out[s] = W[e] a_s for the sorted pairs s of every expert e
    (a_s = a[sorted_tok[s]], or a[s] with sorted_tok None). Only dev_status
    (int32 [1]) tells of a wait that gave up, here and in the two gradients."""
    dev, P, dt = _place_of(W), T * k, dtype_code(a)
    if dtype_code(W) != dt:
        raise ValueError("a and W have one type")
    code = lib.moe_expert_gemm(_address(a, (P if sorted_tok is None else T) * K, dev), _address(W, E * N * K, dev), dt,
                               T, E, k, N, K, _table(offsets, E + 1, dev), _table(sorted_tok, P, dev),
                               _address(out, P * N, dev), dtype_code(out), _table(dev_status, 1, dev),
                               _stream_on(stream, dev))
    if code:
        raise MoeError("moe_expert_gemm", code)


def expert_gemm_dgrad(dy, W, T: int, E: int, k: int, N: int, K: int, offsets, da, dev_status=None,
                      stream=None) -> None:
    """da[s] = W[e]^T dy[s] for the sorted pairs s of every expert e."""
    dev, P, dt = _place_of(W), T * k, dtype_code(dy)
    if dtype_code(W) != dt:
        raise ValueError("dy and W have one type")
    code = lib.moe_expert_gemm_dgrad(_address(dy, P * N, dev), _address(W, E * N * K, dev), dt, T, E, k, N, K,
                                     _table(offsets, E + 1, dev), _address(da, P * K, dev), dtype_code(da),
                                     _table(dev_status, 1, dev), _stream_on(stream, dev))
    if code:
        raise MoeError("moe_expert_gemm_dgrad", code)


def expert_gemm_wgrad(dy, a, T: int, E: int, k: int, N: int, K: int, offsets, sorted_tok, dW, base=None,
                      dev_status=None, stream=None) -> None:
    """dW[e] = base[e] + sum over expert e's sorted pairs s of dy[s] a_s^T (base
    None: zeros; base may be dW)."""
    dev, P, dt, odt = _place_of(dW), T * k, dtype_code(dy), dtype_code(dW)
    if dtype_code(a) != dt or (base is not None and dtype_code(base) != odt):
        raise ValueError("dy and a have one type, base and dW have one type")
    code = lib.moe_expert_gemm_wgrad(_address(dy, P * N, dev), _address(a, (P if sorted_tok is None else T) * K, dev),
                                     dt, T, E, k, N, K, _table(offsets, E + 1, dev), _table(sorted_tok, P, dev),
                                     None if base is None else _address(base, E * N * K, dev),
                                     _address(dW, E * N * K, dev), odt, _table(dev_status, 1, dev),
                                     _stream_on(stream, dev))
    if code:
        raise MoeError("moe_expert_gemm_wgrad", code)


def swiglu(gu, rows: int, f: int, h, stream=None) -> None:
    """h = silu(g) * u for rows [g | u] of gu."""
    dev, dt = _place_of(gu), dtype_code(gu)
    if dtype_code(h) != dt:
        raise ValueError("gu and h have one type")
    code = lib.moe_swiglu(_address(gu, rows * 2 * f, dev), dt, rows, f, _address(h, rows * f, dev),
                          _stream_on(stream, dev))
    if code:
        raise MoeError("moe_swiglu", code)


def swiglu_backward(gu, dh, rows: int, f: int, dgu, stream=None) -> None:
    """dgu = the gradient of swiglu to [g | u], given dh."""
    dev, dt = _place_of(gu), dtype_code(gu)
    if dtype_code(dh) != dt or dtype_code(dgu) != dt:
        raise ValueError("gu, dh and dgu have one type")
    code = lib.moe_swiglu_backward(_address(gu, rows * 2 * f, dev), _address(dh, rows * f, dev), dt, rows, f,
                                   _address(dgu, rows * 2 * f, dev), _stream_on(stream, dev))
    if code:
        raise MoeError("moe_swiglu_backward", code)
