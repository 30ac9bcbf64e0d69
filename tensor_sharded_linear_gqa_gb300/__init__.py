"""Python binding of libtpgqa, the tensor-parallel sharded linear block on GB300.

Argument marshalling only: every function forwards to the C entry point of the
same name (declared in include/tpgqa.h); every step of the computation runs in
the library's CUDA kernels. There is no CPU fallback: the first call loads
``libtpgqa.so`` and raises ImportError when it is missing (build it with
``python -m tensor_sharded_linear_gqa_gb300.build``).

Tensors are passed either as ``TpTensor`` or as 2-D CUDA ``torch.Tensor`` views
with unit column stride (float32 or bfloat16; float8_e4m3fn or uint8 where a call
takes it). Per-rank arguments are Python
sequences. ``stream`` is a ``torch.cuda.Stream``, a raw ``cudaStream_t`` int, or
None for the current torch stream.
"""
from __future__ import annotations

import ctypes
import functools
import importlib
import operator
import os
import struct
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtpgqa.so")


# ---- constants (mirror include/tpgqa.h) ------------------------------------
TP_OK = 0
STATUS_NAMES = ["TP_OK", "TP_ERR_INVALID_ARG", "TP_ERR_TP_SIZE_NOT_POW2", "TP_ERR_NOT_DIVISIBLE",
                "TP_ERR_GQA_SHAPE", "TP_ERR_DTYPE", "TP_ERR_ALIGNMENT", "TP_ERR_RANK_FAILED",
                "TP_ERR_TIMEOUT", "TP_ERR_CUDA", "TP_ERR_WORKSPACE", "TP_ERR_UNSUPPORTED",
                "TP_ERR_BAD_TOKEN", "TP_ERR_BAD_LENGTH"]
for _i, _n in enumerate(STATUS_NAMES):
    globals()[_n] = _i
TP_F32, TP_BF16, TP_E4M3, TP_U8 = 0, 1, 2, 3
TP_SHARD_COLUMN, TP_SHARD_ROW, TP_SHARD_VOCAB, TP_SHARD_REPLICATED = 0, 1, 2, 3
TP_COMM_NONE, TP_COMM_ALL_REDUCE, TP_COMM_ALL_GATHER, TP_COMM_REDUCE_SCATTER = 0, 1, 2, 3
TP_W_Q, TP_W_K, TP_W_V, TP_W_O, TP_W_GATE, TP_W_UP, TP_W_DOWN, TP_W_COUNT = range(8)
WEIGHT_NAMES = ["q_proj", "k_proj", "v_proj", "o_proj", "gate_proj", "up_proj", "down_proj"]
TP_COMBINE_NONE, TP_COMBINE_FUSED, TP_COMBINE_RING, TP_COMBINE_RING_FUSED, TP_COMBINE_RING_SHARED = 0, 1, 2, 3, 4
TP_RING_STEPS, TP_RING_FUSED, TP_RING_FUSED_SHARED = 0, 1, 2
TP_ACT_NONE, TP_ACT_RELU, TP_ACT_GELU, TP_ACT_SILU = 0, 1, 2, 3
ACTIVATIONS = {"none": TP_ACT_NONE, "relu": TP_ACT_RELU, "gelu": TP_ACT_GELU, "silu": TP_ACT_SILU}
TP_MOE_EXPERT_PARALLEL, TP_MOE_WITHIN_EXPERT = 0, 1
TP_ROTARY_HALVES, TP_ROTARY_NEIGHBOURS = 0, 1


class TpTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64)]


class TpDims(ctypes.Structure):
    _fields_ = [("tp_size", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("ffn", ctypes.c_int32)]


class TpRankShard(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("q_head_begin", ctypes.c_int32),
                ("q_head_end", ctypes.c_int32), ("kv_head_begin", ctypes.c_int32),
                ("kv_head_end", ctypes.c_int32), ("kv_replicated", ctypes.c_int32),
                ("strategy", ctypes.c_int32 * TP_W_COUNT), ("comm", ctypes.c_int32 * TP_W_COUNT),
                ("range_begin", ctypes.c_int64 * TP_W_COUNT),
                ("range_end", ctypes.c_int64 * TP_W_COUNT)]


class TpMoeDims(ctypes.Structure):
    _fields_ = [("tp_size", ctypes.c_int32), ("mode", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64)]


class TPError(RuntimeError):
    def __init__(self, status: int, where: str):
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else f"status {status}"
        extra = ""
        if status == 9:  # TP_ERR_CUDA
            extra = f" (cudaError {int(_lib.tp_last_cuda_error())})"
        super().__init__(f"{where}: {name}{extra}")
        self.status = status
        self.name = name


_P = ctypes.POINTER
_T = _P(TpTensor)
_S = ctypes.c_void_p  # cudaStream_t
_A = ctypes.c_void_p


class _I32:
    """A 32-bit integer argument: ctypes itself would cut a larger one to its low bits."""

    @classmethod
    def from_param(cls, x):
        if isinstance(x, ctypes.c_int32):
            return x
        x = operator.index(x)
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"out of range: {x}")
        return ctypes.c_int32(x)


_SIGS = {
    "tp_plan_create": ([_P(TpDims), _P(ctypes.c_void_p)], ctypes.c_int),
    "tp_plan_destroy": ([ctypes.c_void_p], ctypes.c_int),
    "tp_plan_dims": ([ctypes.c_void_p, _P(TpDims)], ctypes.c_int),
    "tp_plan_query_rank": ([ctypes.c_void_p, ctypes.c_int32, _P(TpRankShard)], ctypes.c_int),
    "tp_plan_q_to_kv": ([ctypes.c_void_p, ctypes.c_int32, _P(ctypes.c_int32), ctypes.c_int32],
                        ctypes.c_int),
    "tp_column_linear": ([ctypes.c_int32, _T, _T, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_row_linear": ([ctypes.c_int32, _T, _T, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_reduce_scatter": ([ctypes.c_int32, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_reduce_scatter_bf16": ([ctypes.c_int32, _T, _T, _S], ctypes.c_int),
    "tp_column_linear_chunks": ([ctypes.c_int32, _T, _T, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_ring_all_gather": ([ctypes.c_int32, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_allreduce_ring": ([ctypes.c_int32, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_all_gather": ([ctypes.c_int32, _T, _T, ctypes.c_int32, ctypes.c_int32, _S], ctypes.c_int),
    "tp_vocab_embedding": ([ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, _T, _T, ctypes.c_int32, _S],
                           ctypes.c_int),
    "tp_vocab_lm_head": ([ctypes.c_int32, _T, _T, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_attn_core_workspace_size": ([ctypes.c_void_p, ctypes.c_int64], ctypes.c_size_t),
    "tp_attn_core": ([ctypes.c_void_p, _T, _T, _T, _T, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, _S],
                     ctypes.c_int),
    "tp_moe_workspace_size": ([_P(TpMoeDims), ctypes.c_int64], ctypes.c_size_t),
    "tp_moe_block": ([_P(TpMoeDims), _T, ctypes.c_void_p, ctypes.c_void_p, _T, _T, _T, _T, ctypes.c_int32,
                      ctypes.c_void_p, ctypes.c_size_t, _S], ctypes.c_int),
    "tp_gate_up_swiglu": ([ctypes.c_void_p, _T, _T, _T, _T, _S], ctypes.c_int),
    "tp_mlp_block_workspace_size": ([ctypes.c_void_p, ctypes.c_int64], ctypes.c_size_t),
    "tp_mlp_block": ([ctypes.c_void_p, _T, _T, _T, _T, _T, ctypes.c_int32, ctypes.c_void_p,
                      ctypes.c_size_t, _S], ctypes.c_int),
    "tp_mlp_block_static": ([ctypes.c_void_p, _T, _T, _T, _T, _T, ctypes.c_int32, _S], ctypes.c_int),
    "tp_mlp_block_static_max_bytes": ([], ctypes.c_size_t),
    "tp_qkv_proj": ([ctypes.c_void_p, _T, _T, _T, _T, _T, _T, _T, _S], ctypes.c_int),
    "tp_attn_proj": ([ctypes.c_void_p, _T, _T, _T, _T, _T, _T, _T, _T, _T, _T, ctypes.c_int32,
                      _S], ctypes.c_int),
    # descriptors by address: an arr(), byref() or the address of packed ones
    "tp_add_rmsnorm": ([ctypes.c_int32, _A, _A, _A, ctypes.c_float, _A, _A, _A, _S], ctypes.c_int),
    "tp_linear_epilogue": ([ctypes.c_int32, ctypes.c_int32, _A, _A, _A, _A, _A, ctypes.c_int32, _A, _A, _S], ctypes.c_int),
    "tp_prefix_attn_workspace_size": ([_A, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32],
                                      ctypes.c_size_t),
    "tp_prefix_attn": ([_A, ctypes.c_int64, _A, _A, _A, _A, _A, _A, _A, _A, _A, _A, ctypes.c_size_t, _S], ctypes.c_int),
    "tp_cache_evict": ([_A, ctypes.c_int64, _A, _A, _A, _A, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _A, _A, _A, _A,
                        _A, _S], ctypes.c_int),
    "tp_rotary": ([_A, ctypes.c_int64, _A, _I32, _A, _I32, _A, _I32, _I32, _A, _A, _A,
                   _A, _S], ctypes.c_int),
    "tp_window_attn_workspace_size": ([_A, ctypes.c_int64, ctypes.c_int64, _I32, _I32], ctypes.c_size_t),
    "tp_window_attn": ([_A, _A, _A, _A, _I32, _I32, _A, _A, ctypes.c_size_t, _S], ctypes.c_int),
    "tp_cache4_store": ([_A, ctypes.c_int64, _A, _A, _A, _A, _A, _A, _A, _A, _S], ctypes.c_int),
    "tp_cache4_load": ([_A, ctypes.c_int64, _A, _A, _A, _A, _A, _A, _A, _S], ctypes.c_int),
    "tp_cache4_attn_workspace_size": ([_A, ctypes.c_int64, ctypes.c_int64, _I32, _I32], ctypes.c_size_t),
    "tp_cache4_attn": ([_A, ctypes.c_int64, _A, _A, _A, _A, _A, _A, _I32, _I32, _A, _A, ctypes.c_size_t,
                        _S], ctypes.c_int),
    "tp_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "tp_last_cuda_error": ([], ctypes.c_int32),
    "tp_set_rank_health": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_int),
    "tp_device_status": ([_S, _P(ctypes.c_int32)], ctypes.c_int),
    "tp_set_wait_budget": ([ctypes.c_int64], ctypes.c_int),
    "tp_debug_wait_timeout": ([_S], ctypes.c_int),
    "tp_launch_count": ([], ctypes.c_uint64),
    "tp_version": ([], ctypes.c_char_p),
}
EXPORTED = tuple(_SIGS)


class _Lib:
    """The loaded libtpgqa.so; loading fails loudly when the library is missing."""

    def __init__(self):
        self._cdll = None

    def __getattr__(self, name):
        if self._cdll is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -m tensor_sharded_linear_gqa_gb300.build); there is no CPU fallback")
            cdll = ctypes.CDLL(LIB_PATH)
            for n, (args, res) in _SIGS.items():
                f = getattr(cdll, n)
                f.argtypes = args
                f.restype = res
                setattr(self, n, f)  # found directly from now on
            self._cdll = cdll
        return getattr(self._cdll, name)


_lib = _Lib()


def load() -> ctypes.CDLL:
    """Loads the library now (raises ImportError if it is missing) and returns it."""
    _lib.tp_version  # noqa: B018
    return _lib._cdll


def _check(status: int, where: str) -> None:
    if status != TP_OK:
        raise TPError(status, where)


# ---- marshalling ------------------------------------------------------------
# A descriptor is packed straight into the argument's buffer: building it field by
# field through ctypes costs about as long as the rest of a small call.
_DESC = struct.Struct("=Qiiqqq")
_DTYPES: dict = {}


_loading = threading.RLock()
_loaded = False


def _load_describe():
    """The same in C, for plain tensors (a small call's issue time is mostly this), loaded by the first
    tensor that is described: importing the package maps no object. None where it is not built (an
    interpreter without its headers): interpreted code does it all."""
    if not _loaded:
        with _loading:
            if not _loaded:
                _first_use()
    return _describe


def _types(torch) -> dict:
    return {torch.float32: TP_F32, torch.bfloat16: TP_BF16, torch.float8_e4m3fn: TP_E4M3, torch.uint8: TP_U8}


def _first_use() -> None:
    """Other threads may call meanwhile: they find the functions below, which wait for the lock, until
    everything that they need is in place. (The import itself already puts _describe into this module.)"""
    global _describe, _matrix, _matrices, _row, _vector, _bytes, _DTYPES, _loaded
    types = {}
    try:
        import torch  # the module reads tensors through torch's own libraries
        types = _types(torch)
    except Exception:  # none, or one that does not load: descriptors, addresses and streams may be given as they are
        pass
    try:
        module = importlib.import_module("._describe", __name__)
    except (ImportError, OSError):  # not built, or linked to another torch's libraries
        _describe = None
        _matrix = _row = lambda t, to, device=-1: False  # noqa: E731
        _vector, _bytes = lambda t, kind, n, device=-1: None, lambda t, device=-1: None  # noqa: E731
        _matrices = lambda seq, n, to, device=-1: 0  # noqa: E731
    else:
        if types:
            module.dtypes(*types)
            module.reads_torch(f"{torch.version.__version__} {torch.version.git_version}")
        _describe = module
        _matrix, _matrices, _row = module.matrix, module.matrices, module.row
        _vector, _bytes = module.vector, module.bytes
    _DTYPES = types
    _loaded = True


def __getattr__(name):
    if name == "_describe":
        return _load_describe()
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def _dtypes() -> dict:
    global _DTYPES
    _load_describe()
    if not _DTYPES:  # no torch on the first use: says why, or it is there by now
        import torch
        _DTYPES = _types(torch)
    return _DTYPES


def _matrix(*args):
    """_describe.matrix; _load_describe puts it in this one's place, as for the next four."""
    _load_describe()
    return _matrix(*args)


def _matrices(*args):
    _load_describe()
    return _matrices(*args)


def _row(*args):
    _load_describe()
    return _row(*args)


def _vector(*args):
    _load_describe()
    return _vector(*args)


def _bytes(*args):
    _load_describe()
    return _bytes(*args)


def _fields(t) -> tuple:
    """(ptr, dtype, reserved, rows, cols, ld) of a TpTensor or a 2-D CUDA torch tensor."""
    if isinstance(t, TpTensor):
        return t.ptr or 0, t.dtype, t.reserved, t.rows, t.cols, t.ld
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("expected a 2-D tensor")
    rows, cols = shape
    ld, step = t.stride()
    dt = (_DTYPES or _dtypes()).get(t.dtype)
    if rows and cols:
        if step != 1:
            raise ValueError("expected unit stride along columns")
        if dt is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        return t.data_ptr(), dt, 0, rows, cols, ld if rows > 1 else max(ld, cols)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return 0, dt, 0, rows, cols, ld if rows > 1 else max(ld, cols, 1)


def _tensor(t) -> TpTensor:
    if isinstance(t, TpTensor):
        return t
    return TpTensor(*_fields(t))


def tensor(t) -> TpTensor:
    """TpTensor view of a 2-D CUDA torch tensor with unit column stride (or a TpTensor)."""
    out = _tensor(t)
    if out is not t:
        out.device = _gpu_of(t)
    return out


_devices = None  # GPUs that torch sees


def _device() -> int:
    """The GPU on which the tensors of a call must lie: the current one, on which its kernels run (the
    library sees addresses only, and another GPU's would fault there). -1 where there is only one."""
    global _devices
    if _devices is None:
        try:
            import torch
            _devices = torch.cuda.device_count()
        except Exception:  # no torch: no tensors of it
            _devices = 0
    if _devices < 2:
        return -1
    import torch
    return torch.cuda.current_device()


def _gpu_of(t):
    """The GPU of a tensor or of a descriptor made by tensor(); None: not known."""
    at = getattr(t, "device", None)
    return at if at is None or isinstance(at, int) else at.index if at.type == "cuda" else None


def _lies_on(device: int, at) -> None:
    if at is not None and at != device:
        raise ValueError(f"a tensor on cuda:{at}, the current device is cuda:{device}")


_ARRAYS: dict = {}  # array type by length


def _arr(seq):
    if isinstance(seq, ctypes.Array):  # an arr() the caller keeps
        return seq
    if not isinstance(seq, (list, tuple)):
        seq = list(seq)
    n = len(seq)
    kind = _ARRAYS.get(n)
    if kind is None:
        kind = _ARRAYS[n] = TpTensor * max(n, 1)
    buf = bytearray(_DESC.size * max(n, 1))
    at = 0
    for t in seq:
        _DESC.pack_into(buf, at, *_fields(t))
        at += _DESC.size
    return kind.from_buffer(buf)


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_stream() -> int:
    """The current torch stream's handle, by the binding's own accessor where torch has it
    (torch.cuda.current_stream() builds a Stream object for it first)."""
    global _current_stream
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    torch.cuda.current_stream()  # initialises CUDA
    if raw is not None and device is not None:
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream()


# ---- plan -----------------------------------------------------------------------
class Plan:
    """Owner of a tp_plan*; freed with tp_plan_destroy."""

    def __init__(self, handle: int, dims: TpDims):
        self.handle = handle
        self.dims = dims
        # read on every call: ranks, and copies of K/V (one per rank, or one where they are replicated)
        self.ranks = int(dims.tp_size)
        self.sources = 1 if dims.num_kv_heads < dims.tp_size else self.ranks

    @property
    def tp_size(self) -> int:
        return self.dims.tp_size

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            _lib.tp_plan_destroy(h)
            self.handle = None


def tp_plan_create(tp_size: int, hidden: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   ffn: int) -> Plan:
    d = TpDims(tp_size, hidden, num_q_heads, num_kv_heads, head_dim, ffn)
    h = ctypes.c_void_p()
    _check(_lib.tp_plan_create(ctypes.byref(d), ctypes.byref(h)), "tp_plan_create")
    return Plan(h.value, d)


def tp_plan_destroy(plan: Plan) -> None:
    if plan.handle:
        _check(_lib.tp_plan_destroy(plan.handle), "tp_plan_destroy")
        plan.handle = None


def tp_plan_query_rank(plan: Plan, rank: int) -> dict:
    s = TpRankShard()
    _check(_lib.tp_plan_query_rank(plan.handle, rank, ctypes.byref(s)), "tp_plan_query_rank")
    return {
        "rank": s.rank,
        "q_heads": (s.q_head_begin, s.q_head_end),
        "kv_heads": (s.kv_head_begin, s.kv_head_end),
        "kv_replicated": bool(s.kv_replicated),
        "strategy": {WEIGHT_NAMES[i]: s.strategy[i] for i in range(TP_W_COUNT)},
        "comm": {WEIGHT_NAMES[i]: s.comm[i] for i in range(TP_W_COUNT)},
        "ranges": {WEIGHT_NAMES[i]: (s.range_begin[i], s.range_end[i]) for i in range(TP_W_COUNT)},
    }


def tp_plan_q_to_kv(plan: Plan, rank: int) -> list:
    cap = max(plan.dims.num_q_heads, 1)
    out = (ctypes.c_int32 * cap)()
    _check(_lib.tp_plan_q_to_kv(plan.handle, rank, out, cap), "tp_plan_q_to_kv")
    s = tp_plan_query_rank(plan, rank)
    return [out[j] for j in range(s["q_heads"][1] - s["q_heads"][0])]


# ---- linear layers and collectives ---------------------------------------------
def tp_column_linear(tp_size: int, x, w, y, gather: bool, stream=None) -> None:
    xs = _tensor(x)
    _check(_lib.tp_column_linear(tp_size, ctypes.byref(xs), _arr(w), _arr(y), int(gather),
                                 _stream(stream)), "tp_column_linear")


def tp_row_linear(tp_size: int, x, w, y, combine: int, stream=None) -> None:
    _check(_lib.tp_row_linear(tp_size, _arr(x), _arr(w), _arr(y), combine, _stream(stream)),
           "tp_row_linear")


def tp_reduce_scatter(tp_size: int, bufs, mode: int = TP_RING_STEPS, stream=None) -> None:
    _check(_lib.tp_reduce_scatter(tp_size, _arr(bufs), mode, _stream(stream)), "tp_reduce_scatter")


def tp_reduce_scatter_bf16(tp_size: int, partials, out, stream=None) -> None:
    """Ring reduce-scatter of f32 partials; chunk r of out[r] receives the bf16 sum."""
    _check(_lib.tp_reduce_scatter_bf16(tp_size, _arr(partials), _arr(out), _stream(stream)),
           "tp_reduce_scatter_bf16")


def tp_column_linear_chunks(tp_size: int, x_chunks, w, y, gather: bool, stream=None) -> None:
    """Column-parallel linear whose input rows [c*T/N, (c+1)*T/N) are read from x_chunks[c]."""
    _check(_lib.tp_column_linear_chunks(tp_size, _arr(x_chunks), _arr(w), _arr(y), int(gather),
                                        _stream(stream)), "tp_column_linear_chunks")


def tp_ring_all_gather(tp_size: int, bufs, mode: int = TP_RING_STEPS, stream=None) -> None:
    _check(_lib.tp_ring_all_gather(tp_size, _arr(bufs), mode, _stream(stream)),
           "tp_ring_all_gather")


def tp_allreduce_ring(tp_size: int, bufs, mode: int = TP_RING_STEPS, stream=None) -> None:
    _check(_lib.tp_allreduce_ring(tp_size, _arr(bufs), mode, _stream(stream)), "tp_allreduce_ring")


def tp_all_gather(tp_size: int, shards, outs, axis: int, stream=None) -> None:
    outs = list(outs)
    _check(_lib.tp_all_gather(tp_size, _arr(shards), _arr(outs), len(outs), axis, _stream(stream)),
           "tp_all_gather")


def ids_ptr(ids) -> int:
    """Device address of a contiguous int32 CUDA tensor of token ids (0 when empty)."""
    if str(ids.dtype) != "torch.int32" or not ids.is_contiguous():
        raise TypeError("token ids must be a contiguous int32 tensor")
    return ids.data_ptr() if ids.numel() else 0


def tp_vocab_embedding(tp_size: int, ids, table, outs, stream=None) -> None:
    """Rows ids[i] of the vocab-sharded table (table[r] = rank r's slice) into
    every output (1 shared copy or tp_size copies)."""
    outs = list(outs)
    _check(_lib.tp_vocab_embedding(tp_size, ids_ptr(ids), ids.numel(), _arr(table), _arr(outs), len(outs),
                                   _stream(stream)), "tp_vocab_embedding")


def tp_vocab_lm_head(tp_size: int, x, w, logits, gather: bool, stream=None) -> None:
    xs = _tensor(x)
    _check(_lib.tp_vocab_lm_head(tp_size, ctypes.byref(xs), _arr(w), _arr(logits), int(gather),
                                 _stream(stream)), "tp_vocab_lm_head")


def tp_attn_core_workspace_size(plan: Plan, tokens: int) -> int:
    return int(_lib.tp_attn_core_workspace_size(plan.handle, tokens))


def tp_attn_core(plan: Plan, q, k, v, a, causal: bool, workspace, stream=None) -> None:
    """q[r], a[r]: rank r's [T x Hq_r*d] bf16; k, v: one entry per rank, or one
    shared entry when the plan replicates K/V; workspace: a CUDA byte tensor."""
    _check(_lib.tp_attn_core(plan.handle, _arr(q), _arr(k), _arr(v), _arr(a), int(causal),
                             workspace.data_ptr(), workspace.numel(), _stream(stream)), "tp_attn_core")


def moe_dims(tp_size: int, mode: int, num_experts: int, top_k: int, hidden: int, ffn: int) -> TpMoeDims:
    return TpMoeDims(tp_size, mode, num_experts, top_k, hidden, ffn)


def tp_moe_workspace_size(dims: TpMoeDims, tokens: int) -> int:
    return int(_lib.tp_moe_workspace_size(ctypes.byref(dims), tokens))


_DTYPE_NAMES: dict = {}  # str(dtype) by dtype: formatting it costs more than the rest of the check
_VECTOR_KINDS = {"torch.float32": TP_F32, "torch.int32": 4}  # the extension module's names of them


def _dev_ptr(t, dtype: str, n: int | None = None, what: str = "", device: int = -1) -> int:
    """Address of a contiguous CUDA tensor (0 when empty). The library sees no length, so where it
    takes one from elsewhere (n), the tensor's is held against it here. device: as _device gives it."""
    at = _vector(t, _VECTOR_KINDS[dtype], -1 if n is None else n, device)
    if at is not None:
        return at
    if device >= 0:
        _lies_on(device, _gpu_of(t))
    name = _DTYPE_NAMES.get(t.dtype)
    if name is None:
        name = _DTYPE_NAMES[t.dtype] = str(t.dtype)
    if name != dtype or not t.is_contiguous():
        raise TypeError(f"expected a contiguous {dtype} tensor")
    have = t.numel()
    if n is not None and have != n:
        raise ValueError(f"{what} must have {n} entries, not {have}")
    if have == 0:
        return 0
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def tp_moe_block(dims: TpMoeDims, x, topk_ids, topk_w, w_gate, w_up, w_down, y, combine: int, workspace,
                 stream=None) -> None:
    """topk_ids: int32 [T x k] CUDA tensor; topk_w: float32 [T x k]; workspace: a
    CUDA byte tensor of at least tp_moe_workspace_size bytes."""
    xs = _tensor(x)
    _check(_lib.tp_moe_block(ctypes.byref(dims), ctypes.byref(xs), _dev_ptr(topk_ids, "torch.int32"),
                             _dev_ptr(topk_w, "torch.float32"), _arr(w_gate), _arr(w_up), _arr(w_down),
                             _arr(y), combine, workspace.data_ptr(), workspace.numel(), _stream(stream)),
           "tp_moe_block")


def tp_gate_up_swiglu(plan: Plan, x, w_gate, w_up, h, stream=None) -> None:
    xs = _tensor(x)
    _check(_lib.tp_gate_up_swiglu(plan.handle, ctypes.byref(xs), _arr(w_gate), _arr(w_up), _arr(h),
                                  _stream(stream)), "tp_gate_up_swiglu")


def tp_mlp_block_workspace_size(plan: Plan, tokens: int) -> int:
    return int(_lib.tp_mlp_block_workspace_size(plan.handle, tokens))


def tp_mlp_block(plan: Plan, x, w_gate, w_up, w_down, y, combine: int, workspace,
                 workspace_bytes: int | None = None, stream=None) -> None:
    """``workspace`` is a CUDA torch tensor (any dtype) or a raw device pointer int."""
    if isinstance(workspace, int) or workspace is None:
        wptr, wbytes = workspace, workspace_bytes or 0
    else:
        wptr = workspace.data_ptr()
        wbytes = workspace.numel() * workspace.element_size()
    xs = _tensor(x)
    _check(_lib.tp_mlp_block(plan.handle, ctypes.byref(xs), _arr(w_gate), _arr(w_up),
                             _arr(w_down), _arr(y), combine, wptr, wbytes, _stream(stream)),
           "tp_mlp_block")


def tp_mlp_block_static(plan: Plan, x, w_gate, w_up, w_down, y, combine: int, stream=None) -> None:
    """tp_mlp_block without a workspace argument, for callers that cannot allocate
    device memory: H lives in the library's fixed 16 MiB scratch array. Calls on
    one device share that array, so calls that overlap on the GPU race."""
    xs = _tensor(x)
    _check(_lib.tp_mlp_block_static(plan.handle, ctypes.byref(xs), _arr(w_gate), _arr(w_up),
                                    _arr(w_down), _arr(y), combine, _stream(stream)),
           "tp_mlp_block_static")


def tp_mlp_block_static_max_bytes() -> int:
    return int(_lib.tp_mlp_block_static_max_bytes())


def tp_qkv_proj(plan: Plan, x, w_q, w_k, w_v, q, k, v, stream=None) -> None:
    xs = _tensor(x)
    _check(_lib.tp_qkv_proj(plan.handle, ctypes.byref(xs), _arr(w_q), _arr(w_k), _arr(w_v), _arr(q),
                            _arr(k), _arr(v), _stream(stream)), "tp_qkv_proj")


def tp_attn_proj(plan: Plan, x, w_q, w_k, w_v, q, k, v, a, w_o, y, combine: int,
                 stream=None) -> None:
    xs = _tensor(x)
    _check(_lib.tp_attn_proj(plan.handle, ctypes.byref(xs), _arr(w_q), _arr(w_k), _arr(w_v),
                             _arr(q), _arr(k), _arr(v), _arr(a), _arr(w_o), _arr(y), combine,
                             _stream(stream)), "tp_attn_proj")


# ---- between the projections ----------------------------------------------------
class _Scratch:
    """Descriptors of the call being made, one buffer per thread (the library reads them during the
    call only). Each method packs tensors and returns the address: a small call spends less time
    on its kernels than building ctypes objects for its arguments would take."""

    __slots__ = ("buf", "base", "room", "used", "device")

    def __init__(self, room: int):
        self.buf = bytearray(_DESC.size * room)
        self.base = ctypes.addressof((ctypes.c_char * len(self.buf)).from_buffer(self.buf))
        self.room, self.used = room, 0  # tensors; bytes
        self.device = -1  # the GPU on which they must lie, -1: not asked

    def one(self, t):
        """A single descriptor; None for None."""
        if t is None:
            return None
        at = self.used
        self.used = at + _DESC_SIZE
        if not (_matrix(t, self.base + at) if self.device < 0 else _matrix(t, self.base + at, self.device)):
            if self.device >= 0:
                _lies_on(self.device, _gpu_of(t))
            _PACK(self.buf, at, *_fields(t))  # no plain tensor, the first of all, or an error's words
        return self.base + at

    def many(self, seq, n: int):
        """A per-rank argument with at least n entries; an arr() the caller keeps goes as it is."""
        if len(seq) < n:
            raise ValueError(f"expected {n} tensors, one per rank or kv source")
        if isinstance(seq, ctypes.Array):
            if self.device >= 0:
                for at in getattr(seq, "devices", ()):
                    _lies_on(self.device, at)
            return seq
        first = self.base + self.used
        done = _matrices(seq, n, first) if self.device < 0 else _matrices(seq, n, first, self.device)
        self.used += done * _DESC_SIZE
        for i in range(done, n):
            self.one(seq[i])
        return first

    def row(self, t):
        """A vector: its 1-D tensor is the [1 x n] view that the library takes."""
        if t is None:
            return None
        at = self.used
        if not _row(t, self.base + at):
            return self.one(t if type(t) is TpTensor or t.dim() != 1 else t.unsqueeze(0))
        self.used = at + _DESC_SIZE
        return self.base + at


_DESC_SIZE, _PACK = _DESC.size, _DESC.pack_into
_local = threading.local()


def _args(most: int, device: int = -1) -> _Scratch:
    """The thread's scratch, emptied, with room for `most` tensors."""
    s = getattr(_local, "scratch", None)
    if s is None or s.room < most:
        s = _local.scratch = _Scratch(max(most, 256))
    s.used, s.device = 0, device
    return s


def _scale_ptr(t, of, dim: int, what: str):
    """Address of the scales of `of`'s rows (dim 0) or columns (1); None for None."""
    if t is None:
        return None
    n = (of.rows, of.cols)[dim] if isinstance(of, TpTensor) else of.shape[dim]
    return _dev_ptr(t, "torch.float32", n, what)


def tp_add_rmsnorm(x, residual, weight, eps: float, residual_out, y, y_scale=None, stream=None) -> None:
    """z = sum of x (one tensor or a list of per-rank partials) + residual, to residual_out;
    y = z * rsqrt(mean(z^2) + eps) * weight, in bf16, or as e4m3 codes with y_scale [T]."""
    many = isinstance(x, (list, tuple, ctypes.Array))
    n = len(x) if many else 1
    a = _args(n + 4)
    st = _lib.tp_add_rmsnorm(n, a.many(x, n) if many else a.one(x), a.one(residual), a.row(weight), eps,
                             a.one(residual_out), a.one(y), _scale_ptr(y_scale, y, 0, "y_scale"), _stream(stream))
    if st:
        raise TPError(st, "tp_add_rmsnorm")


def tp_linear_epilogue(tp_size: int, shard: int, x, w, y, bias=None, activation: int = TP_ACT_NONE, residual=None,
                       x_scale=None, w_scale=None, stream=None) -> None:
    """y = activation(x w^T * x_scale * w_scale + bias) + residual. shard: TP_SHARD_COLUMN (x: [X],
    w: the ranks' weight rows) or TP_SHARD_ROW (x, w: the ranks' slices of the input features)."""
    a = _args(2 * tp_size + 3 if tp_size > 0 else 3)
    to = a.one(y)
    st = _lib.tp_linear_epilogue(tp_size, shard, a.many(x, tp_size if shard == TP_SHARD_ROW else 1),
                                 _scale_ptr(x_scale, y, 0, "x_scale"), a.many(w, tp_size), _scale_ptr(w_scale, y, 1, "w_scale"),
                                 a.row(bias), activation, a.one(residual), to, _stream(stream))
    if st:
        raise TPError(st, "tp_linear_epilogue")


def tp_prefix_attn_workspace_size(plan: Plan, batch: int, prefix: int, capacity: int, weights: bool) -> int:
    return int(_lib.tp_prefix_attn_workspace_size(plan.handle, batch, prefix, capacity, int(weights)))


def _kv_sources(plan: Plan) -> int:
    return plan.sources


def tp_prefix_attn(plan: Plan, q, k_prefix, v_prefix, k_own, v_own, lengths, a, workspace, weight_in=None, weight_out=None,
                   stream=None) -> None:
    """One new token per sequence over the shared prefix and the sequence's own cache. q, a: one
    entry per rank; caches and weights: one per kv source; workspace: a CUDA byte tensor."""
    if not workspace.is_contiguous() or not (workspace.is_cuda or workspace.numel() == 0):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    n, src = plan.dims.tp_size, _kv_sources(plan)
    g = _args(2 * n + 6 * src)
    st = _lib.tp_prefix_attn(plan.handle, lengths.numel(), g.many(q, n), g.many(k_prefix, src), g.many(v_prefix, src),
                             g.many(k_own, src), g.many(v_own, src), _dev_ptr(lengths, "torch.int32"),
                             None if weight_in is None else g.many(weight_in, src),
                             None if weight_out is None else g.many(weight_out, src), g.many(a, n), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream(stream))
    if st:
        raise TPError(st, "tp_prefix_attn")


def tp_cache_evict(plan: Plan, lengths, k, v, weight, budget: int, n_first: int, n_recent: int, k_out, v_out, weight_out,
                   lengths_out, kept, stream=None) -> None:
    """Keeps `budget` positions of every sequence and kv head: the first n_first, the last
    n_recent and the heaviest between. k, v, weight and their outputs: one entry per kv source."""
    batch, src = lengths.numel(), _kv_sources(plan)
    a = _args(6 * src)
    st = _lib.tp_cache_evict(plan.handle, batch, _dev_ptr(lengths, "torch.int32"), a.many(k, src), a.many(v, src),
                             a.many(weight, src), budget, n_first, n_recent, a.many(k_out, src), a.many(v_out, src),
                             a.many(weight_out, src), _dev_ptr(lengths_out, "torch.int32", batch, "lengths_out"),
                             _dev_ptr(kept, "torch.int32", batch * plan.dims.num_kv_heads * budget, "kept"), _stream(stream))
    if st:
        raise TPError(st, "tp_cache_evict")


# ---- long contexts ----------------------------------------------------------------
def rotary_axes(sections) -> ctypes.Array:
    """The `axis` argument of tp_rotary for axes that take their pairs one after the other:
    sections[x] pairs of axis x."""
    axis = [x for x, n in enumerate(sections) for _ in range(n)]
    return (ctypes.c_int32 * len(axis))(*axis)


def _workspace(t, device: int = -1) -> tuple:
    """(address, bytes) of a workspace tensor; None is an empty one."""
    if t is None:
        return None, 0
    at = _bytes(t, device)
    if at is not None:
        return at
    if device >= 0:
        _lies_on(device, _gpu_of(t))
    size = t.numel() * t.element_size()
    if not t.is_contiguous() or not (t.is_cuda or size == 0):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return t.data_ptr(), size


_entries: dict = {}


def _entry(name: str):
    """The library's call tp_<name>, by way of the extension module where that is built."""
    fn = _entries.get(name)
    if fn is None:
        fn = getattr(_lib, "tp_" + name)
        if _load_describe() is not None:
            fn = functools.partial(getattr(_describe, name), ctypes.cast(fn, ctypes.c_void_p).value)
        _entries[name] = fn
    return fn


def tp_rotary(plan: Plan, positions, freq, q, k, q_out, k_out, axis=None, layout: int = TP_ROTARY_HALVES,
              inverse: bool = False, stream=None) -> None:
    """Rotates pairs of values of q's and k's heads by positions[axis] * freq. positions: int32 [T] or
    [axes x T]; freq: f32 [pairs]; axis: per pair (rotary_axes), None: all 0. q, q_out: one entry
    per rank, k, k_out: one per kv source; q or k may be None with its output."""
    n, src, pairs = plan.ranks, plan.sources, freq.numel()
    device = _device()
    if positions.dim() not in (1, 2):
        raise ValueError("positions must be [T] or [axes x T]")
    axes, tokens = (1, positions.shape[0]) if positions.dim() == 1 else positions.shape
    if axis is not None:
        if not isinstance(axis, ctypes.Array):
            if any(not 0 <= x < axes for x in axis):
                raise ValueError(f"axis must have entries in [0, {axes})")
            axis = (ctypes.c_int32 * len(axis))(*axis)
        if axis._type_ is not ctypes.c_int32 or len(axis) != pairs:
            raise ValueError(f"axis must have {pairs} entries, one per pair")
    g = _args(2 * n + 2 * src, device)
    st = _entry("rotary")(plan.handle, tokens, _dev_ptr(positions, "torch.int32", device=device), axes,
                          _dev_ptr(freq, "torch.float32", device=device), pairs, axis, layout, int(inverse),
                          None if q is None else g.many(q, n), None if k is None else g.many(k, src),
                          None if q_out is None else g.many(q_out, n), None if k_out is None else g.many(k_out, src),
                          _stream(stream))
    if st:
        raise TPError(st, "tp_rotary")


def tp_window_attn_workspace_size(plan: Plan, tokens: int, keys: int, window: int, sinks: int) -> int:
    return int(_lib.tp_window_attn_workspace_size(plan.handle, tokens, keys, window, sinks))


def tp_window_attn(plan: Plan, q, k, v, window: int, sinks: int, a, workspace=None, stream=None) -> None:
    """The last T of S tokens over a sliding window and the first `sinks` tokens. q, a: one entry per
    rank; k, v: one per kv source; workspace: a CUDA byte tensor."""
    n, src = plan.ranks, plan.sources
    device = _device()
    ws, size = _workspace(workspace, device)
    g = _args(2 * n + 2 * src, device)
    st = _entry("window_attn")(plan.handle, g.many(q, n), g.many(k, src), g.many(v, src), window, sinks, g.many(a, n), ws, size,
                               _stream(stream))
    if st:
        raise TPError(st, "tp_window_attn")


def tp_cache4_store(plan: Plan, lengths, k, v, k_codes, k_scale, v_codes, v_scale, counts=None, stream=None) -> None:
    """Stores the rows of k and v (batch * n tokens) behind the lengths[b] positions that the 4-bit
    caches hold. All but lengths and counts: one entry per kv source."""
    batch, src = lengths.numel(), plan.sources
    device = _device()
    g = _args(6 * src, device)
    st = _entry("cache4_store")(plan.handle, batch, _dev_ptr(lengths, "torch.int32", device=device),
                                None if counts is None else _dev_ptr(counts, "torch.int32", batch, "counts", device),
                                g.many(k, src), g.many(v, src), g.many(k_codes, src), g.many(k_scale, src), g.many(v_codes, src),
                                g.many(v_scale, src), _stream(stream))
    if st:
        raise TPError(st, "tp_cache4_store")


def tp_cache4_load(plan: Plan, first, k_codes, k_scale, v_codes, v_scale, k_out, v_out, stream=None) -> None:
    """Positions first[b] .. of every sequence from the 4-bit caches into k_out and v_out (batch * n
    rows). All but first: one entry per kv source."""
    src, device = plan.sources, _device()
    g = _args(6 * src, device)
    st = _entry("cache4_load")(plan.handle, first.numel(), _dev_ptr(first, "torch.int32", device=device),
                               g.many(k_codes, src), g.many(k_scale, src), g.many(v_codes, src), g.many(v_scale, src), g.many(k_out, src),
                               g.many(v_out, src), _stream(stream))
    if st:
        raise TPError(st, "tp_cache4_load")


def tp_cache4_attn_workspace_size(plan: Plan, batch: int, capacity: int, window: int, sinks: int) -> int:
    return int(_lib.tp_cache4_attn_workspace_size(plan.handle, batch, capacity, window, sinks))


def tp_cache4_attn(plan: Plan, q, k_codes, k_scale, v_codes, v_scale, lengths, window: int, sinks: int, a, workspace=None,
                   stream=None) -> None:
    """One new token per sequence over the 4-bit caches, a sliding window and the first `sinks` tokens.
    q, a: one entry per rank; caches: one per kv source; workspace: a CUDA byte tensor."""
    n, src = plan.ranks, plan.sources
    device = _device()
    ws, size = _workspace(workspace, device)
    g = _args(2 * n + 4 * src, device)
    st = _entry("cache4_attn")(plan.handle, lengths.numel(), g.many(q, n), g.many(k_codes, src), g.many(k_scale, src),
                               g.many(v_codes, src), g.many(v_scale, src), _dev_ptr(lengths, "torch.int32", device=device),
                               window, sinks, g.many(a, n), ws, size, _stream(stream))
    if st:
        raise TPError(st, "tp_cache4_attn")


# ---- status and diagnostics ---------------------------------------------------
def tp_status_str(status: int) -> str:
    return _lib.tp_status_str(status).decode()


def tp_last_cuda_error() -> int:
    return int(_lib.tp_last_cuda_error())


def tp_set_rank_health(rank: int, healthy: bool) -> None:
    _check(_lib.tp_set_rank_health(rank, int(healthy)), "tp_set_rank_health")


def tp_device_status(stream=None) -> tuple:
    """(status, raw word): synchronises the stream and reads/clears the device status word."""
    word = ctypes.c_int32(0)
    st = _lib.tp_device_status(_stream(stream), ctypes.byref(word))
    return st, word.value


def tp_set_wait_budget(nanoseconds: int) -> None:
    _check(_lib.tp_set_wait_budget(nanoseconds), "tp_set_wait_budget")


def tp_debug_wait_timeout(stream=None) -> None:
    _check(_lib.tp_debug_wait_timeout(_stream(stream)), "tp_debug_wait_timeout")


def tp_launch_count() -> int:
    """Kernel launches the library has enqueued in this process so far."""
    return int(_lib.tp_launch_count())


def tp_version() -> str:
    return _lib.tp_version().decode()


def arr(seq):
    """ctypes array of TpTensor for a per-rank argument (kept alive by the caller)."""
    if isinstance(seq, ctypes.Array):
        return seq
    seq = list(seq)
    out = _arr(seq)
    out.devices = frozenset(_gpu_of(t) for t in seq) - {None}
    return out


class Prepared:
    """A C entry point with its arguments marshalled once, for tight loops: calling
    it makes only the ctypes call. Raises TPError on a non-OK status."""

    def __init__(self, fn_name: str, *args):
        self.fn = getattr(_lib, fn_name)
        self.name = fn_name
        self.args = args  # keeps the ctypes objects alive

    def __call__(self) -> None:
        st = self.fn(*self.args)
        if st != TP_OK:
            raise TPError(st, self.name)


def raw_status(fn_name: str, *args) -> int:
    """Calls a C entry point with ready-made ctypes arguments and returns its status
    (for tests of the error paths)."""
    return getattr(_lib, fn_name)(*args)
