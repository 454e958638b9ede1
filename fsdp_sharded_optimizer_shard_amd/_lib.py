"""ctypes binding of libzeroshard (include/zero_shard.h).  Argument
marshalling only: every step of the path runs in the HIP library.

Buffers may be given as torch tensors (their data_ptr() is passed) or as raw
integer device addresses.  A tensor is checked before the call: its dtype,
that it is contiguous, and that it holds every element the call touches (from
the layout's unit range), so that an undersized buffer raises ValueError here
instead of being read or written past its end by a kernel.  Raw addresses are
passed as they are.  `stream` defaults to torch's current stream on the
current device.  Errors of the library raise ZeroShardError with its message.
There is no fallback: if the library is missing this module fails to import.
"""
import ctypes
import os
from typing import Optional, Sequence

# torch first: its ROCm build ships its own HIP runtime (same soname,
# libamdhip64.so.7).  Loading torch before the library makes the library bind
# to that runtime, so device pointers and streams from torch are valid in it;
# loading the library first would put a second HIP runtime in the process.
import torch  # noqa: E402,F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzeroshard.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run __graft_entry__.build() or "
        "python -m fsdp_sharded_optimizer_shard_amd.build")

_lib = ctypes.CDLL(LIB_PATH)

# enums (zero_shard.h)
OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_OOM, ERR_HIP, ERR_UNSUPPORTED = range(6)
DDP, STAGE1, STAGE2, STAGE3, FSDP, MEGATRON_DO = range(6)
BF16, FP32 = 0, 1
INDEX_FULL, INDEX_SHARD = 0, 1
K_INNER, K_OUTER = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
SAVED_BF16, SAVED_E4M3 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
STATE_FP32, STATE_E4M3 = 0, 1
MIX_STEP_STREAMS, MIX_READS, MIX_WRITES = 0, 1, 2
MAX_RANKS_PER_CALL = 64
NOALLOC_MAX_PARTIALS = 524288
STATE_CHUNK_MIN, STATE_CHUNK_MAX = 4, 1 << 24     # zero_layout_chunk_state bounds
STATE_CHUNK_DEFAULT = 8192                         # the measured best on MI355X
GRAD_CHUNK_DEFAULT = 16384                         # chunked gradients, likewise
XENT_PIECE_ELEMS = 67108864                        # dz elements of a head's piece, by default

STRATEGY = {"ddp": DDP, "zero1": STAGE1, "zero1_allreduce": STAGE1, "zero2": STAGE2,
            "zero3": STAGE3, "fsdp": FSDP, "fsdp2": FSDP, "megatron_do": MEGATRON_DO}

ACTIVATION = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
              "silu": ACT_SILU}

SCORE = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


class _Grads(ctypes.Structure):
    _fields_ = [("ptrs", ctypes.POINTER(ctypes.c_void_p)), ("index", ctypes.POINTER(ctypes.c_uint8)),
                ("n", _I32), ("dtype", _I32), ("index_all", _I32), ("chunk", _I32)]


class AdamCfg(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("decoupled", _I32), ("step", _I64)]


def adam_cfg(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, decoupled=False,
             step=1) -> AdamCfg:
    return AdamCfg(lr, beta1, beta2, eps, weight_decay, int(bool(decoupled)), int(step))


class AdamTableEntry(ctypes.Structure):
    _fields_ = [(k, ctypes.c_float) for k in ("lr", "beta1", "beta2", "eps", "weight_decay",
                                               "one_minus_beta1", "one_minus_beta2", "bias1",
                                               "bias2", "decay")] + \
               [("has_decay", _I32), ("decoupled", _I32)]


_lib.zero_shard_init.argtypes = [ctypes.POINTER(_P), _I32, _I32, _I32, _I32, ctypes.POINTER(_I64)]
_lib.zero_shard_init.restype = _I32
_lib.zero_shard_init_rows.argtypes = [ctypes.POINTER(_P), _I32, _I32, _I32, _I32,
                                      ctypes.POINTER(_I64), ctypes.POINTER(_I64)]
_lib.zero_shard_init_rows.restype = _I32
_lib.zero_layout_rows.argtypes = [_P, _I32] + [ctypes.POINTER(_I64)] * 3
_lib.zero_layout_rows.restype = _I32
_lib.zero_shard_destroy.argtypes = [_P]
_lib.zero_shard_destroy.restype = None
_lib.zero_layout_info.argtypes = [_P] + [ctypes.POINTER(_I64)] * 2 + [ctypes.POINTER(_I32)] * 4
_lib.zero_layout_info.restype = _I32
_lib.zero_layout_query.argtypes = [_P, _I32] + [ctypes.POINTER(_I64)] * 6
_lib.zero_layout_query.restype = _I32
_lib.zero_layout_chunk_state.argtypes = [_P, _I64, ctypes.POINTER(_P)]
_lib.zero_layout_chunk_state.restype = _I32
_lib.zero_layout_state.argtypes = [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]
_lib.zero_layout_state.restype = _I32
_lib.zero_reduce_shard.argtypes = [_P, _I32, _I32, ctypes.POINTER(_Grads), _P, _I32, _P, _I64,
                                   _P]
_lib.zero_reduce_shard.restype = _I32
_lib.zero_reduce_partials_count.argtypes = [_P, _I32, _I32]
_lib.zero_reduce_partials_count.restype = _I64
_lib.zero_clip_coef.argtypes = [_P, _I64, ctypes.c_float, _P, _P, _P]
_lib.zero_clip_coef.restype = _I32
_lib.zero_adam_step.argtypes = [_P, _I32, _I32, ctypes.POINTER(AdamCfg), _P, _I32, _P,
                                ctypes.POINTER(_Grads), _P, _P, _P, _P, _I32, _P]
_lib.zero_adam_step.restype = _I32
_lib.zero_adam_step_clip_noalloc.argtypes = [_P, _I32, _I32, ctypes.POINTER(AdamCfg),
                                             ctypes.c_float, ctypes.POINTER(_Grads), _P, _P, _P,
                                             _P, _P, _I32, _P, _P]
_lib.zero_adam_step_clip_noalloc.restype = _I32
_lib.zero_adam_table_fill.argtypes = [ctypes.POINTER(AdamCfg), _I64, _P]
_lib.zero_adam_table_fill.restype = _I32
_lib.zero_adam_step_table.argtypes = [_P, _I32, _I32, _P, _I64, _P, _P, _I32, _P,
                                      ctypes.POINTER(_Grads), _P, _P, _P, _P, _I32, _P]
_lib.zero_adam_step_table.restype = _I32
_lib.zero_step_advance.argtypes = [_P, _P]
_lib.zero_step_advance.restype = _I32
_lib.zero_gather_params.argtypes = [_P, _I32, _I32, ctypes.POINTER(ctypes.c_void_p), _I32, _P, _P]
_lib.zero_gather_params.restype = _I32


class _UnitIO(ctypes.Structure):
    _fields_ = [("rank_grads", ctypes.POINTER(ctypes.c_void_p)),
                ("peer_shards", ctypes.POINTER(ctypes.c_void_p)), ("unit_full", _P)]


_lib.zero_fsdp_sweep.argtypes = [_P, _I32, _I32, ctypes.POINTER(AdamCfg), _I32, _I32,
                                 ctypes.POINTER(_UnitIO), _P, _P, _P, _I32, _P, _P]
_lib.zero_fsdp_sweep.restype = _I32
_lib.zero_fsdp_sweep_table.argtypes = [_P, _I32, _I32, _P, _I64, _P, _I32, _I32,
                                       ctypes.POINTER(_UnitIO), _P, _P, _P, _I32, _P, _P]
_lib.zero_fsdp_sweep_table.restype = _I32
_lib.zero_gemm_bf16.argtypes = [_I64, _I64, _I64, _P, _I64, _I32, _P, _I64, _I32, _P, _I64, _I32,
                                _P]
_lib.zero_gemm_bf16.restype = _I32
_lib.zero_gemm_bf16_nt.argtypes = [_I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _P]
_lib.zero_gemm_bf16_nt.restype = _I32
_lib.zero_transpose_bf16.argtypes = [_I64, _I64, _P, _I64, _P, _I64, _P]
_lib.zero_transpose_bf16.restype = _I32
_lib.zero_fsdp_linear_forward.argtypes = [_P, _I32, ctypes.POINTER(ctypes.c_void_p), _I64, _P, _P,
                                          _P, _I32, _P]
_lib.zero_fsdp_linear_forward.restype = _I32
_lib.zero_fsdp_linear_backward.argtypes = [_P, _I32, ctypes.POINTER(ctypes.c_void_p), _I64, _P,
                                           _P, _P, _P, _I32, _P, _P]
_lib.zero_fsdp_linear_backward.restype = _I32


class _Saved(ctypes.Structure):
    _fields_ = [("data", _P), ("ld", _I64), ("scales", _P), ("ld_scales", _I64), ("format", _I32)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("bias", _P), ("residual", _P), ("ldr", _I64), ("preact", _P), ("output", _P), ("bias_dtype", _I32), ("residual_dtype", _I32),
                ("act", _I32)]


_SP = ctypes.POINTER(_Saved)
_EP = ctypes.POINTER(_Epilogue)
_PP = ctypes.POINTER(ctypes.c_void_p)
_lib.zero_saved_write.argtypes = [_I64, _I64, _P, _I64, _I32, _SP, _P]
_lib.zero_saved_write.restype = _I32
_lib.zero_saved_read.argtypes = [_I64, _I64, _SP, _P, _I64, _I32, _P]
_lib.zero_saved_read.restype = _I32
_lib.zero_gemm_bf16_epilogue.argtypes = [_I64, _I64, _I64, _P, _I64, _I32, _P, _I64, _I32, _P, _I64,
                                         _I32, _EP, _P]
_lib.zero_gemm_bf16_epilogue.restype = _I32
_lib.zero_act_backward.argtypes = [_I64, _I64, _P, _I64, _I32, _I32, _SP, _P, _I64, _P, _P, _I64, _P]
_lib.zero_act_backward.restype = _I32
_lib.zero_act_backward_workspace.argtypes = [_I64, _I64]
_lib.zero_act_backward_workspace.restype = _I64
_lib.zero_gemm_saved_bf16.argtypes = [_I64, _I64, _I64, _SP, _P, _I64, _P, _I64, _I32, _P]
_lib.zero_gemm_saved_bf16.restype = _I32
_lib.zero_gemm_grouped_rows_bf16.argtypes = [_I32, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _I32,
                                             _I64, _P, _I64, _I32, _EP, _P]
_lib.zero_gemm_grouped_rows_bf16.restype = _I32
_lib.zero_gemm_grouped_depth_bf16.argtypes = [_I32, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P,
                                              _I64, _I64, _I32, _P]
_lib.zero_gemm_grouped_depth_bf16.restype = _I32
_lib.zero_fsdp_linear_act_forward.argtypes = [_P, _I32, _PP, _I64, _P, _P, _EP, _P, _I32, _P]
_lib.zero_fsdp_linear_act_forward.restype = _I32
_lib.zero_fsdp_linear_act_backward.argtypes = [_P, _I32, _PP, _I64, _SP, _I32, _SP, _P, _P, _P, _P,
                                               _I32, _P, _P, _P, _I64, _P]
_lib.zero_fsdp_linear_act_backward.restype = _I32
_lib.zero_fsdp_experts_forward.argtypes = [_P, _I32, _I32, _PP, _P, _I64, _P, _P, _EP, _P, _I32, _P]
_lib.zero_fsdp_experts_forward.restype = _I32
_lib.zero_fsdp_experts_backward.argtypes = [_P, _I32, _I32, _PP, _P, _I64, _P, _P, _P, _P, _I32, _P,
                                            _P]
_lib.zero_fsdp_experts_backward.restype = _I32


class _Router(ctypes.Structure):
    _fields_ = [(k, _I32) for k in ("n_experts", "top_k", "n_groups", "top_groups", "group_best",
                                    "score", "renormalize")] + [("scale", ctypes.c_float)]


class _Tensor(ctypes.Structure):
    _fields_ = [("n", _I64)] + [(k, _P) for k in ("master", "grad", "param", "m", "v", "m_scales",
                                                  "v_scales")] + [("decay", _I32)]


_RP = ctypes.POINTER(_Router)
_TP = ctypes.POINTER(_Tensor)
_F32, _U64 = ctypes.c_float, ctypes.c_uint64
_lib.zero_layer_norm_forward.argtypes = [_I64, _I64, _P, _I64, _I32, _P, _P, _I32, _F32, _P, _I64,
                                         _I32, _P, _P, _P]
_lib.zero_layer_norm_forward.restype = _I32
_lib.zero_layer_norm_backward.argtypes = [_I64, _I64, _P, _I64, _I32, _P, _I64, _I32, _P, _I32, _P,
                                          _P, _P, _I64, _P, _I64, _I32, _P, _P, _P, _I64, _P]
_lib.zero_layer_norm_backward.restype = _I32
_lib.zero_layer_norm_workspace.argtypes = [_I64, _I64]
_lib.zero_layer_norm_workspace.restype = _I64
_lib.zero_route_forward.argtypes = [_RP, _I64, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _I64, _P]
_lib.zero_route_forward.restype = _I32
_lib.zero_route_workspace.argtypes = [_RP, _I64]
_lib.zero_route_workspace.restype = _I64
_lib.zero_route_backward.argtypes = [_RP, _I64, _P, _I64, _I32, _P, _P, _P, _I64, _I32, _P]
_lib.zero_route_backward.restype = _I32
_lib.zero_experts_dispatch.argtypes = [_I64, _I32, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P]
_lib.zero_experts_dispatch.restype = _I32
_lib.zero_experts_combine.argtypes = [_I64, _I32, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _P, _I64,
                                      _I32, _P]
_lib.zero_experts_combine.restype = _I32
_lib.zero_experts_combine_backward.argtypes = [_I64, _I32, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _P,
                                               _I64, _P, _P]
_lib.zero_experts_combine_backward.restype = _I32
_lib.zero_linear_xent_forward.argtypes = [_I64, _I64, _I64, _P, _I64, _P, _I64, _I32, _P, _P, _P, _P,
                                          _I64, _P]
_lib.zero_linear_xent_forward.restype = _I32
_lib.zero_linear_xent_backward.argtypes = [_I64, _I64, _I64, _P, _I64, _P, _I64, _I32, _P, _P, _P, _P,
                                           _I64, _I32, _P, _I64, _I32, _I64, _P, _I64, _P]
_lib.zero_linear_xent_backward.restype = _I32
_lib.zero_linear_xent_workspace.argtypes = [_I64, _I64, _I64, _I32, _I64]
_lib.zero_linear_xent_workspace.restype = _I64
_lib.zero_fsdp_head_forward.argtypes = [_P, _I32, _PP, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P]
_lib.zero_fsdp_head_forward.restype = _I32
_lib.zero_fsdp_head_backward.argtypes = [_P, _I32, _PP, _I32, _I64, _P, _P, _P, _P, _P, _P, _I32, _P,
                                         _I64, _P, _I64, _P]
_lib.zero_fsdp_head_backward.restype = _I32
_lib.zero_adam_tensors.argtypes = [_I32, _TP, _I32, _I32, ctypes.POINTER(AdamCfg), _U64, _P, _P]
_lib.zero_adam_tensors.restype = _I32
_lib.zero_adam_tensors_table.argtypes = [_I32, _TP, _I32, _I32, _P, _I64, _P, _U64, _P, _P]
_lib.zero_adam_tensors_table.restype = _I32
_lib.zero_tensors_sumsq.argtypes = [_I32, _TP, _I32, _P, _I64, _P]
_lib.zero_tensors_sumsq.restype = _I32
_lib.zero_tensors_partials_count.argtypes = [_I32, _TP]
_lib.zero_tensors_partials_count.restype = _I64
_lib.zero_adam_state_read.argtypes = [_I64, _P, _P, _I32, _P, _I32, _P]
_lib.zero_adam_state_read.restype = _I32
_lib.zero_stream_mix.argtypes = [_I32, ctypes.POINTER(ctypes.c_void_p), _I32, _P, _P, _P, _P,
                                 _I64, _I64, _I64, _P]
_lib.zero_stream_mix.restype = _I32
_lib.zero_grad_accumulate.argtypes = [_P, _P, _I64, _P]
_lib.zero_grad_accumulate.restype = _I32
_lib.zero_status_str.argtypes = [_I32]
_lib.zero_status_str.restype = ctypes.c_char_p
_lib.zero_last_error.argtypes = []
_lib.zero_last_error.restype = ctypes.c_char_p

EXPORTS = ("zero_shard_init", "zero_shard_init_rows", "zero_layout_rows", "zero_shard_destroy",
           "zero_layout_info", "zero_layout_query", "zero_layout_chunk_state", "zero_layout_state",
           "zero_reduce_shard",
           "zero_reduce_partials_count", "zero_clip_coef", "zero_adam_step",
           "zero_adam_step_clip_noalloc",
           "zero_adam_table_fill", "zero_adam_step_table", "zero_step_advance", "zero_gather_params",
           "zero_grad_accumulate", "zero_stream_mix", "zero_fsdp_sweep", "zero_fsdp_sweep_table", "zero_gemm_bf16",
           "zero_gemm_bf16_nt",
           "zero_transpose_bf16", "zero_fsdp_linear_forward", "zero_fsdp_linear_backward",
           "zero_saved_write", "zero_saved_read", "zero_gemm_bf16_epilogue", "zero_act_backward",
           "zero_act_backward_workspace", "zero_gemm_saved_bf16", "zero_gemm_grouped_rows_bf16",
           "zero_gemm_grouped_depth_bf16", "zero_fsdp_linear_act_forward",
           "zero_fsdp_linear_act_backward", "zero_fsdp_experts_forward",
           "zero_fsdp_experts_backward",
           "zero_layer_norm_forward", "zero_layer_norm_backward", "zero_layer_norm_workspace",
           "zero_route_forward", "zero_route_workspace", "zero_route_backward",
           "zero_experts_dispatch", "zero_experts_combine", "zero_experts_combine_backward",
           "zero_linear_xent_forward", "zero_linear_xent_backward", "zero_linear_xent_workspace",
           "zero_fsdp_head_forward", "zero_fsdp_head_backward",
           "zero_adam_tensors", "zero_adam_tensors_table", "zero_tensors_sumsq",
           "zero_tensors_partials_count", "zero_adam_state_read",
           "zero_status_str", "zero_last_error")


class ZeroShardError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        msg = _lib.zero_last_error().decode(errors="replace")
        super().__init__(f"{fn}: {_lib.zero_status_str(status).decode()} ({status}): {msg}")


def _check(status: int, fn: str) -> None:
    if status != OK:
        raise ZeroShardError(status, fn)


def _addr(x) -> Optional[int]:
    """Device address of a buffer: None, a raw int address, or a tensor that
    lives on the GPU (a host tensor's pointer would fault inside a kernel,
    so it is refused here)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if getattr(x, "is_cuda", True) is False:
        raise ValueError("buffers passed to libzeroshard must be GPU tensors (got one on "
                         f"{getattr(x, 'device', 'the host')})")
    return x.data_ptr()


_DTYPES = {
    "fp32": (torch.float32,),
    "fp64": (torch.float64,),
    "bf16": (torch.int16, torch.uint16, torch.bfloat16),   # bf16 bit patterns
    "int64": (torch.int64,),
    "int32": (torch.int32,),
    "bytes8": (torch.uint8, torch.bool),
    "codes": (torch.uint8, torch.float8_e4m3fn),           # one byte each
}


def _need(x, what: str, count: Optional[int], kind: str) -> None:
    """A tensor argument must be of `kind`, contiguous, and hold at least
    `count` elements (bytes for kind "bytes").  None, raw addresses and an
    unknown count (an invalid range, reported by the library) pass."""
    if x is None or x.__class__ is int or not hasattr(x, "numel"):
        return
    if x.is_cuda is False:
        raise ValueError(f"{what}: buffers passed to libzeroshard must be GPU tensors (got one "
                         f"on {x.device})")
    if count is None:
        return
    if kind == "bytes":
        have = x.numel() * x.element_size()
    else:
        if x.dtype not in _DTYPES[kind]:
            raise ValueError(f"{what}: dtype {x.dtype}, expected one of "
                             f"{', '.join(str(d) for d in _DTYPES[kind])}")
        have = x.numel()
    if have < count:
        raise ValueError(f"{what} holds {have} {'bytes' if kind == 'bytes' else 'elements'}, "
                         f"the call touches {count}")
    if not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _kind(dtype: int) -> str:
    return "fp32" if dtype == FP32 else "bf16"


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Layout:
    """An owned zero_layout (host memory).  Use shard_init() to make one."""

    def __init__(self, handle: int, units: Sequence[int]):
        self._h = handle
        self.units = list(units)
        self._uq = None
        self._lens = {}
        self._state = None

    def _unit_table(self):
        """Every unit's query(), read once (a layout never changes)."""
        if self._uq is None:
            self._uq = [self.query(u) for u in range(self.info()["n_units"])]
        return self._uq

    def range_lens(self, unit_begin: int, unit_end: int):
        """(shard-indexed, full-indexed) element counts of a unit range, or
        (None, None) for a range the library will refuse."""
        key = (unit_begin, unit_end)
        r = self._lens.get(key)
        if r is None:
            r = self._lens[key] = self._range_lens(unit_begin, unit_end)
        return r

    def _range_lens(self, unit_begin, unit_end):
        q = self._unit_table()
        if not (0 <= unit_begin <= unit_end <= len(q)):
            return None, None
        if unit_begin == unit_end:
            return 0, 0
        a, b = q[unit_begin], q[unit_end - 1]
        return (b["shard_off"] + b["shard_len"] - a["shard_off"],
                b["flat_off"] + b["padded_len"] - a["flat_off"])

    @property
    def handle(self) -> int:
        if not self._h:
            raise ValueError("layout is destroyed")
        return self._h

    def destroy(self) -> None:
        if self._h and _lib is not None:   # _lib may already be gone at exit
            _lib.zero_shard_destroy(self._h)
        self._h = None

    __del__ = destroy

    def info(self) -> dict:
        f, s = _I64(), _I64()
        nu, wn, r, st = _I32(), _I32(), _I32(), _I32()
        _check(_lib.zero_layout_info(self.handle, ctypes.byref(f), ctypes.byref(s), ctypes.byref(nu),
                                     ctypes.byref(wn), ctypes.byref(r), ctypes.byref(st)),
               "zero_layout_info")
        return {"flat_len": f.value, "shard_len": s.value, "n_units": nu.value,
                "world_n": wn.value, "rank": r.value, "strategy": st.value}

    def query(self, unit: int) -> dict:
        v = [_I64() for _ in range(6)]
        _check(_lib.zero_layout_query(self.handle, unit, *[ctypes.byref(x) for x in v]),
               "zero_layout_query")
        keys = ("numel", "padded_len", "flat_off", "shard_len", "shard_off", "rank_flat_off")
        return dict(zip(keys, (x.value for x in v)))

    def rows(self, unit: int) -> dict:
        v = [_I64() for _ in range(3)]
        _check(_lib.zero_layout_rows(self.handle, unit, *[ctypes.byref(x) for x in v]),
               "zero_layout_rows")
        return dict(zip(("cols", "first_row", "row_count"), (x.value for x in v)))

    def chunk_state(self, chunk: int) -> "Layout":
        """A copy of this layout whose master, m and v form one buffer in
        chunks of `chunk` elements (0: three arrays); see state_views()."""
        h = _P()
        _check(_lib.zero_layout_chunk_state(self.handle, chunk, ctypes.byref(h)),
               "zero_layout_chunk_state")
        return Layout(h.value, self.units)

    def _state_format(self):
        if self._state is None:
            e, n = _I64(), _I64()
            _check(_lib.zero_layout_state(self.handle, ctypes.byref(e), ctypes.byref(n)),
                   "zero_layout_state")
            self._state = (e.value, n.value)
        return self._state

    @property
    def state_chunk(self) -> int:
        """0 for three state arrays, else the chunk E of the one state buffer."""
        return self._state_format()[0]

    @property
    def state_len(self) -> int:
        """Floats of the state: shard_len per array, or the chunked buffer's length."""
        return self._state_format()[1]

    def state_views(self, state):
        """(master, m, v) for a chunked layout: views of one state tensor of
        state_len floats starting at 0, E and 2E, as the library expects."""
        E = self.state_chunk
        if E == 0:
            raise ValueError("this layout keeps master, m and v as three arrays")
        if state.numel() != self.state_len:
            raise ValueError(f"state: expected {self.state_len} floats, got {state.numel()}")
        return state[0:], state[E:], state[2 * E:]

    def state_count(self, unit_begin: int, unit_end: int):
        """Floats each of master, m and v must hold from its pointer for a
        call over [unit_begin, unit_end), or None for a range the library
        will refuse.  A chunked state is addressed by absolute shard index."""
        shard, _ = self.range_lens(unit_begin, unit_end)
        E = self.state_chunk
        if shard is None or E == 0 or shard == 0:
            return shard
        last = self._unit_table()[unit_end - 1]
        i = last["shard_off"] + last["shard_len"] - 1     # highest shard index touched
        return (i // E) * 3 * E + i % E + 1

    def grad_count(self, unit_begin: int, unit_end: int, chunk: int):
        """Elements each rank's pointer into chunked gradients (chunk E) must
        reach for a call over [unit_begin, unit_end): the range's last
        element i sits at (i // E) N E + i % E (None as above)."""
        shard, _ = self.range_lens(unit_begin, unit_end)
        if shard is None or chunk == 0 or shard == 0:
            return shard
        i, E = shard - 1, chunk
        return (i // E) * self.info()["world_n"] * E + i % E + 1

    def grad_len(self, chunk: int, unit_begin: int = 0, unit_end: Optional[int] = None) -> int:
        """Elements of one buffer holding all N ranks' gradients for the
        range's part of this shard (the whole shard by default) in chunks of
        `chunk`: ceil(S / E) rows of N chunks."""
        if chunk <= 0:
            raise ValueError(f"chunk must be positive (got {chunk})")
        ue = self.info()["n_units"] if unit_end is None else unit_end
        shard, _ = self.range_lens(unit_begin, ue)
        if shard is None:
            raise ValueError(f"unit range [{unit_begin}, {ue}) is outside the layout")
        return -(-shard // chunk) * self.info()["world_n"] * chunk

    @property
    def flat_len(self) -> int:
        return self.info()["flat_len"]

    @property
    def shard_len(self) -> int:
        return self.info()["shard_len"]


def shard_init(strategy, world_n: int, rank: int, unit_numel: Sequence[int]) -> Layout:
    s = STRATEGY[strategy] if isinstance(strategy, str) else int(strategy)
    arr = (_I64 * len(unit_numel))(*[int(u) for u in unit_numel]) if len(unit_numel) else None
    h = _P()
    _check(_lib.zero_shard_init(ctypes.byref(h), s, world_n, rank, len(unit_numel), arr),
           "zero_shard_init")
    return Layout(h.value, unit_numel)


def shard_init_rows(strategy, world_n: int, rank: int, shapes) -> Layout:
    """FSDP2-style layout: one unit per (rows, cols) parameter."""
    s = STRATEGY[strategy] if isinstance(strategy, str) else int(strategy)
    n = len(shapes)
    rows = (_I64 * max(1, n))(*[int(r) for r, _ in shapes])
    cols = (_I64 * max(1, n))(*[int(c) for _, c in shapes])
    h = _P()
    _check(_lib.zero_shard_init_rows(ctypes.byref(h), s, world_n, rank, n, rows, cols),
           "zero_shard_init_rows")
    return Layout(h.value, [int(r) * int(c) for r, c in shapes])


class Grads:
    """Marshalled zero_grads; keeps its ctypes arrays alive."""

    def __init__(self, bufs, dtype: int = BF16, index=INDEX_FULL, chunk: int = 0):
        self._keep = list(bufs)              # keeps tensors alive; sliceable by callers
        ptrs = [_addr(b) for b in bufs]
        self._ptrs = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
        self._index = None
        idx_all = INDEX_FULL
        if isinstance(index, int):
            idx_all = index
        else:
            self._index = (ctypes.c_uint8 * len(index))(*[int(i) for i in index])
        self.s = _Grads(self._ptrs, self._index, len(ptrs), dtype, idx_all, chunk)
        self._checked = None

    @classmethod
    def chunked(cls, buf, n: int, chunk: int, dtype: int = BF16, full=None):
        """N ranks' shard-indexed gradients interleaved in one buffer in
        chunks of `chunk` elements (Layout.grad_len long): rank q's pointer
        is the buffer's start + q * chunk.  `full` maps ranks whose
        gradient is a full-indexed buffer of its own (a rank's own main
        gradient) to that buffer; their slots in `buf` are not read."""
        full = full or {}
        bufs = [full[q] if q in full else buf[q * chunk:] for q in range(n)]
        index = ([INDEX_FULL if q in full else INDEX_SHARD for q in range(n)] if full
                 else INDEX_SHARD)
        return cls(bufs, dtype, index, chunk)

    @property
    def chunk(self) -> int:
        return self.s.chunk

    def ref(self):
        return ctypes.byref(self.s)

    def check(self, layout, unit_begin: int, unit_end: int) -> None:
        """Each rank buffer holds what a call over [unit_begin, unit_end)
        reads from it.  The buffers of a Grads never change, so a range
        checked once is not checked again."""
        shard, full = layout.range_lens(unit_begin, unit_end)
        if self.chunk and shard is not None:
            shard = layout.grad_count(unit_begin, unit_end, self.chunk)
        lens = (shard, full)
        if lens == self._checked:
            return
        for q, b in enumerate(self._keep):
            mode = self.s.index_all if self._index is None else self._index[q]
            _need(b, f"gradient buffer of rank {q}", full if mode == INDEX_FULL else shard,
                  _kind(self.s.dtype))
        if None not in lens:
            self._checked = lens


def reduce_partials_count(layout: Layout, unit_begin: int, unit_end: int) -> int:
    return _lib.zero_reduce_partials_count(layout.handle, unit_begin, unit_end)


def reduce_shard(layout: Layout, unit_begin: int, unit_end: int, grads: Grads, out,
                 sumsq_partials=None, n_partials: int = 0, stream=None,
                 out_index: int = INDEX_SHARD) -> None:
    shard, full = layout.range_lens(unit_begin, unit_end)
    if grads is not None:
        grads.check(layout, unit_begin, unit_end)
    _need(out, "out", full if out_index == INDEX_FULL else shard, "fp32")
    _need(sumsq_partials, "sumsq_partials", n_partials, "fp64")
    _check(_lib.zero_reduce_shard(layout.handle, unit_begin, unit_end, grads.ref() if grads else None,
                                  _addr(out), out_index, _addr(sumsq_partials), n_partials,
                                  _stream(stream)),
           "zero_reduce_shard")


def clip_coef(partials, n: int, max_norm: float, coef_out, norm_out=None, stream=None) -> None:
    _need(partials, "partials", n, "fp64")
    _need(coef_out, "coef_out", 1, "fp32")
    _need(norm_out, "norm_out", 1, "fp64")
    _check(_lib.zero_clip_coef(_addr(partials), n, max_norm, _addr(coef_out), _addr(norm_out),
                               _stream(stream)), "zero_clip_coef")


def _check_step(layout, unit_begin, unit_end, master, m, v, param_out, param_index,
                grad_fp32=None, grad_index=INDEX_SHARD, clip_coef=None, grads=None):
    lens = layout.range_lens(unit_begin, unit_end)
    shard, full = lens
    sc = layout.state_count(unit_begin, unit_end)
    _need(master, "master", sc, "fp32")
    _need(m, "m", sc, "fp32")
    _need(v, "v", sc, "fp32")
    _need(param_out, "param_out", full if param_index == INDEX_FULL else shard, "bf16")
    if grad_fp32 is not None:
        _need(grad_fp32, "grad_fp32", full if grad_index == INDEX_FULL else shard, "fp32")
    if clip_coef is not None:
        _need(clip_coef, "clip_coef", 1, "fp32")
    if grads is not None:
        grads.check(layout, unit_begin, unit_end)


def adam_step(layout: Layout, unit_begin: int, unit_end: int, cfg: AdamCfg, master, m, v,
              param_out, param_index: int = INDEX_FULL, grad_fp32=None, clip_coef=None,
              grads: Optional[Grads] = None, stream=None, grad_index: int = INDEX_SHARD) -> None:
    _check_step(layout, unit_begin, unit_end, master, m, v, param_out, param_index, grad_fp32,
                grad_index, clip_coef, grads)
    _check(_lib.zero_adam_step(layout.handle, unit_begin, unit_end, ctypes.byref(cfg),
                               _addr(grad_fp32), grad_index, _addr(clip_coef),
                               grads.ref() if grads else None,
                               _addr(master), _addr(m), _addr(v), _addr(param_out), param_index,
                               _stream(stream)), "zero_adam_step")


def adam_step_clip_noalloc(layout: Layout, unit_begin: int, unit_end: int, cfg: AdamCfg,
                           max_norm: float, grads: Grads, grad_out, master, m, v, param_out,
                           param_index: int = INDEX_FULL, norm_out=None, stream=None) -> None:
    """The clipped two-pass step with the library's static scratch (no
    device allocation): reduce with partials, clip coefficient, Adam."""
    _check_step(layout, unit_begin, unit_end, master, m, v, param_out, param_index,
                grad_fp32=grad_out, grads=grads)
    _need(norm_out, "norm_out", 1, "fp64")
    _check(_lib.zero_adam_step_clip_noalloc(layout.handle, unit_begin, unit_end,
                                            ctypes.byref(cfg), max_norm,
                                            grads.ref() if grads else None, _addr(grad_out),
                                            _addr(master), _addr(m), _addr(v), _addr(param_out),
                                            param_index, _addr(norm_out), _stream(stream)),
           "zero_adam_step_clip_noalloc")


def adam_table(cfgs):
    """Host table of step scalars, one entry per configuration (entry k is
    used when the device step counter holds k + 1): an array of
    AdamTableEntry; bytes(table) is what goes to the device."""
    n = len(cfgs)
    arr = (AdamCfg * max(1, n))(*cfgs)
    out = (AdamTableEntry * max(1, n))()
    _check(_lib.zero_adam_table_fill(arr, n, out), "zero_adam_table_fill")
    return out


def adam_table_device(cfgs, device="cuda"):
    """adam_table(cfgs) copied into a device uint8 tensor."""
    import torch
    t = adam_table(cfgs)
    return torch.frombuffer(bytearray(bytes(t)), dtype=torch.uint8).to(device)


def adam_step_table(layout: Layout, unit_begin: int, unit_end: int, table, n_entries: int,
                    step_counter, master, m, v, param_out, param_index: int = INDEX_FULL,
                    grad_fp32=None, clip_coef=None, grads: Optional[Grads] = None, stream=None,
                    grad_index: int = INDEX_SHARD) -> None:
    _check_step(layout, unit_begin, unit_end, master, m, v, param_out, param_index, grad_fp32,
                grad_index, clip_coef, grads)
    _need(table, "table", n_entries * ctypes.sizeof(AdamTableEntry), "bytes")
    _need(step_counter, "step_counter", 1, "int64")
    _check(_lib.zero_adam_step_table(layout.handle, unit_begin, unit_end, _addr(table), n_entries,
                                     _addr(step_counter), _addr(grad_fp32), grad_index,
                                     _addr(clip_coef), grads.ref() if grads else None,
                                     _addr(master), _addr(m), _addr(v), _addr(param_out),
                                     param_index, _stream(stream)), "zero_adam_step_table")


def step_advance(step_counter, stream=None) -> None:
    _need(step_counter, "step_counter", 1, "int64")
    _check(_lib.zero_step_advance(_addr(step_counter), _stream(stream)), "zero_step_advance")


def gather_params(layout: Layout, unit_begin: int, unit_end: int, shards, param_full,
                  stream=None) -> None:
    shard, full = layout.range_lens(unit_begin, unit_end)
    for q, x in enumerate(shards):
        _need(x, f"shard of rank {q}", shard, "bf16")
    _need(param_full, "param_full", full, "bf16")
    ptrs = [_addr(s) for s in shards]
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    _check(_lib.zero_gather_params(layout.handle, unit_begin, unit_end, arr, len(ptrs),
                                   _addr(param_full), _stream(stream)), "zero_gather_params")


def _parts(layout: Layout) -> int:
    """Slices per unit: world_n, or 1 for a DDP layout."""
    i = layout.info()
    return 1 if i["strategy"] == DDP else i["world_n"]


def _need_len(what: str, seq, n: int) -> None:
    # The library reads exactly n entries of these host arrays; a shorter
    # list would have it read past the ctypes array.
    if len(seq) != n:
        raise ValueError(f"{what}: expected {n} entries, got {len(seq)}")


def _unit_ios(layout: Layout, unit_begin: int, unit_end: int, units, grad_dtype=BF16,
              grad_chunk=0):
    if 0 <= unit_begin <= unit_end:
        _need_len("units", units, unit_end - unit_begin)
        n, parts = layout.info()["world_n"], _parts(layout)
        table = layout._unit_table()
        for i, (grads, peers, full) in enumerate(units):
            _need_len("rank_grads", grads, n)
            _need_len("peer_shards", peers, parts)
            if unit_begin + i < len(table):
                u = unit_begin + i
                q = table[u]
                count = (layout.grad_count(u, u + 1, grad_chunk) if grad_chunk else
                         q["shard_len"])
                for k, x in enumerate(grads):
                    _need(x, f"unit {u} gradient of rank {k}", count, _kind(grad_dtype))
                for k, x in enumerate(peers):
                    _need(x, f"unit {unit_begin + i} shard of rank {k}", q["shard_len"], "bf16")
                _need(full, f"unit {unit_begin + i} buffer", q["padded_len"], "bf16")
    keep = []
    arr = (_UnitIO * max(1, len(units)))()
    for i, (grads, peers, full) in enumerate(units):
        g = (ctypes.c_void_p * max(1, len(grads)))(*[_addr(x) for x in grads])
        p = (ctypes.c_void_p * max(1, len(peers)))(*[_addr(x) for x in peers])
        keep += [g, p]
        arr[i] = _UnitIO(g, p, _addr(full))
    return arr, keep


def fsdp_sweep(layout: Layout, unit_begin: int, unit_end: int, cfg: AdamCfg, grad_dtype: int,
               units, master, m, v, max_inflight: int = 2, step_stream=None,
               gather_stream=None, grad_chunk: int = 0) -> None:
    """units: one (rank_grads, peer_shards, unit_full) per unit of the range;
    rank_grads are world_n buffers and peer_shards one per slice (world_n,
    or 1 under DDP; None allowed).  gather_stream defaults to step_stream
    (sequential).  grad_chunk E > 0: every unit's rank_grads are the
    pointers of one chunked receive buffer over the shard (Grads.chunked)."""
    arr, keep = _unit_ios(layout, unit_begin, unit_end, units, grad_dtype, grad_chunk)
    sc = layout.state_count(unit_begin, unit_end)
    for name, x in (("master", master), ("m", m), ("v", v)):
        _need(x, name, sc, "fp32")
    ss = _stream(step_stream)
    gs = ss if gather_stream is None else _stream(gather_stream)
    _check(_lib.zero_fsdp_sweep(layout.handle, unit_begin, unit_end, ctypes.byref(cfg), grad_dtype,
                                grad_chunk, arr, _addr(master), _addr(m), _addr(v), max_inflight,
                                ss, gs),
           "zero_fsdp_sweep")


def fsdp_sweep_table(layout: Layout, unit_begin: int, unit_end: int, table, n_entries: int,
                     step_counter, grad_dtype: int, units, master, m, v, max_inflight: int = 2,
                     step_stream=None, gather_stream=None, grad_chunk: int = 0) -> None:
    """fsdp_sweep with the step scalars of table[*step_counter - 1] (device
    table and counter); advances the counter once, after the last unit."""
    arr, keep = _unit_ios(layout, unit_begin, unit_end, units, grad_dtype, grad_chunk)
    sc = layout.state_count(unit_begin, unit_end)
    for name, x in (("master", master), ("m", m), ("v", v)):
        _need(x, name, sc, "fp32")
    _need(table, "table", n_entries * ctypes.sizeof(AdamTableEntry), "bytes")
    _need(step_counter, "step_counter", 1, "int64")
    ss = _stream(step_stream)
    gs = ss if gather_stream is None else _stream(gather_stream)
    _check(_lib.zero_fsdp_sweep_table(layout.handle, unit_begin, unit_end, _addr(table),
                                      n_entries, _addr(step_counter), grad_dtype, grad_chunk,
                                      arr,
                                      _addr(master), _addr(m), _addr(v), max_inflight, ss, gs),
           "zero_fsdp_sweep_table")


def _operand_extent(rows: int, K: int, ld: int, order: int) -> int:
    """Elements from an operand's start to its last one read."""
    if rows <= 0 or K <= 0:
        return 0
    return (rows - 1) * ld + K if order == K_INNER else (K - 1) * ld + rows


def gemm_bf16(M: int, N: int, K: int, A, lda: int, a_order: int, B, ldb: int, b_order: int, C,
              ldc: int, c_dtype: int = FP32, stream=None) -> None:
    if M > 0 and N > 0 and K >= 0:
        _need(A, "A", _operand_extent(M, K, lda, a_order), "bf16")
        _need(B, "B", _operand_extent(N, K, ldb, b_order), "bf16")
        _need(C, "C", (M - 1) * ldc + N, _kind(c_dtype))
    _check(_lib.zero_gemm_bf16(M, N, K, _addr(A), lda, a_order, _addr(B), ldb, b_order, _addr(C),
                               ldc, c_dtype, _stream(stream)), "zero_gemm_bf16")


def gemm_bf16_nt(M: int, N: int, K: int, A, lda: int, B, ldb: int, C, ldc: int,
                 c_dtype: int = FP32, stream=None) -> None:
    if M > 0 and N > 0 and K >= 0:
        _need(A, "A", _operand_extent(M, K, lda, K_INNER), "bf16")
        _need(B, "B", _operand_extent(N, K, ldb, K_INNER), "bf16")
        _need(C, "C", (M - 1) * ldc + N, _kind(c_dtype))
    _check(_lib.zero_gemm_bf16_nt(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, c_dtype,
                                  _stream(stream)), "zero_gemm_bf16_nt")


def transpose_bf16(rows: int, cols: int, src, lds: int, dst, ldd: int, stream=None) -> None:
    if rows > 0 and cols > 0:
        _need(src, "src", (rows - 1) * lds + cols, "bf16")
        _need(dst, "dst", (cols - 1) * ldd + rows, "bf16")
    _check(_lib.zero_transpose_bf16(rows, cols, _addr(src), lds, _addr(dst), ldd, _stream(stream)),
           "zero_transpose_bf16")


def _ptrs(bufs):
    return (ctypes.c_void_p * max(1, len(bufs)))(*[_addr(b) for b in bufs])


def _layer_dims(layout: Layout, unit: int):
    """(in, out, shard, padded) of a linear layer's unit, or None if the unit
    does not exist (the library reports that)."""
    table = layout._unit_table()
    if not 0 <= unit < len(table):
        return None
    q = table[unit]
    cols = layout.rows(unit)["cols"]
    return q["numel"] // cols, cols, q["shard_len"], q["padded_len"]


def _check_layer(layout, unit, w_shards, w_full, batch):
    d = _layer_dims(layout, unit)
    if d is None or batch < 0:
        return None
    for q, x in enumerate(w_shards):
        _need(x, f"W shard of rank {q}", d[2], "bf16")
    _need(w_full, "w_full", d[3], "bf16")
    return d


def fsdp_linear_forward(layout: Layout, unit: int, w_shards, batch: int, x, w_full, y,
                        y_dtype: int = BF16, stream=None) -> None:
    _need_len("w_shards", w_shards, _parts(layout))
    d = _check_layer(layout, unit, w_shards, w_full, batch)
    if d is not None:
        _need(x, "x", batch * d[0], "bf16")
        _need(y, "y", batch * d[1], _kind(y_dtype))
    _check(_lib.zero_fsdp_linear_forward(layout.handle, unit, _ptrs(w_shards), batch, _addr(x),
                                         _addr(w_full), _addr(y), y_dtype, _stream(stream)),
           "zero_fsdp_linear_forward")


def fsdp_linear_backward(layout: Layout, unit: int, w_shards, batch: int, x, dy, w_full, dx,
                         dw_full, dx_dtype: int = BF16, stream=None) -> None:
    _need_len("w_shards", w_shards, _parts(layout))
    d = _check_layer(layout, unit, w_shards, w_full, batch)
    if d is not None:
        _need(x, "x", batch * d[0], "bf16")
        _need(dy, "dy", batch * d[1], "bf16")
        _need(dx, "dx", batch * d[0], _kind(dx_dtype))
        _need(dw_full, "dw_full", d[3], "fp32")
    _check(_lib.zero_fsdp_linear_backward(layout.handle, unit, _ptrs(w_shards), batch, _addr(x),
                                          _addr(dy), _addr(w_full), _addr(dx), dx_dtype,
                                          _addr(dw_full), _stream(stream)),
           "zero_fsdp_linear_backward")


# ------------------------------------------------------- layer operators --

class _Call:
    """The buffers of one call: each checked like _need and turned into its
    address, all on one device, which is the one that the default stream
    belongs to.  Small calls last as long as their arguments' checks, so a
    good tensor passes in a handful of lookups."""
    __slots__ = ("device",)

    def __init__(self):
        self.device = None

    def __call__(self, x, what: str, count: Optional[int], kind: str) -> Optional[int]:
        if x is None or x.__class__ is int:
            return x
        if not (count is not None and x.is_cuda and x.dtype in _DTYPES[kind] and x.numel() >= count
                and x.is_contiguous()):
            _need(x, what, count, kind)
        if self.device is None:
            self.device = x.get_device()
        elif x.get_device() != self.device:
            raise ValueError(f"tensors of one call on two devices ({self.device} and "
                             f"{x.get_device()})")
        return x.data_ptr()

    def stream(self, stream) -> Optional[int]:
        if stream is not None:
            return _stream(stream)
        current = torch.cuda.current_device()
        if self.device is not None and self.device != current:
            raise ValueError(f"tensors on device {self.device}, but the current device is "
                             f"{current}: switch to it, or give a stream of it")
        return _raw_stream(current)


# The current stream's handle without a Stream object around it, where this
# torch has that; a Stream costs as much as the rest of a call's checks.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _extent(rows: int, ld: int, cols: int) -> Optional[int]:
    """Elements from a matrix's start to its last one (None: a size that the
    library refuses)."""
    if rows < 0 or cols < 0 or ld < cols:
        return None
    return 0 if rows == 0 or cols == 0 else (rows - 1) * ld + cols


class Saved:
    """A rows x cols activation matrix kept for the backward pass: bf16
    (`scales` None), or 8-bit codes with one exponent byte per 32 rows of a
    column.  Keeps its buffers alive."""
    __slots__ = ("data", "scales", "format", "s", "ref")

    def __init__(self, data, ld: int, scales=None, ld_scales: int = 0):
        self.data, self.scales = data, scales
        self.format = SAVED_BF16 if scales is None else SAVED_E4M3
        self.s = _Saved(_addr(data), ld, _addr(scales), ld_scales, self.format)
        self.ref = ctypes.byref(self.s)

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Saved":
        """An 8-bit checkpoint of rows x cols with buffers of its own."""
        ld, lds = -(-max(cols, 1) // 16) * 16, -(-max(cols, 1) // 4) * 4
        return cls(torch.empty((max(rows, 1), ld), dtype=torch.uint8, device=device), ld,
                   torch.empty((max(-(-rows // 32), 1), lds), dtype=torch.uint8, device=device), lds)

    def check(self, call: _Call, what: str, rows: int, cols: int):
        """Checks the buffers for rows x cols; the C argument."""
        s = self.s
        if self.format == SAVED_BF16:
            call(self.data, what, _extent(rows, s.ld, cols), "bf16")
        else:
            call(self.data, what, _extent(rows, s.ld, cols), "codes")
            call(self.scales, what, _extent((rows + 31) // 32, s.ld_scales, cols), "codes")
        return self.ref


def _act(act) -> int:
    if isinstance(act, str):
        if act not in ACTIVATION:
            raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTIVATION)})")
        return ACTIVATION[act]
    return int(act)


def _dtype_of(x, given: int) -> int:
    """ZERO_FP32 for a float32 tensor, ZERO_BF16 for another tensor, `given`
    for a raw address."""
    if x is None or x.__class__ is int:
        return given
    return FP32 if x.dtype == torch.float32 else BF16


class Epilogue:
    """C = act(z) + residual with z = A B + bias; `preact` keeps z, `output`
    keeps C in 8 bits.  `act` is a name of ACTIVATION or its number; the
    types of bias and residual are taken from tensors, else bias_dtype and
    residual_dtype (raw addresses).  Keeps its buffers alive."""
    __slots__ = ("bias", "residual", "preact", "output", "s", "ref")

    def __init__(self, bias=None, act=ACT_NONE, residual=None, ldr: int = 0, preact: Optional[Saved] = None,
                 output: Optional[Saved] = None, bias_dtype: int = BF16, residual_dtype: int = BF16):
        self.bias, self.residual, self.preact, self.output = bias, residual, preact, output
        self.s = _Epilogue(_addr(bias), _addr(residual), ldr,
                           None if preact is None else ctypes.addressof(preact.s),
                           None if output is None else ctypes.addressof(output.s),
                           _dtype_of(bias, bias_dtype), _dtype_of(residual, residual_dtype),
                           _act(act))
        self.ref = ctypes.byref(self.s)

    def check(self, call: _Call, M: int, N: int):
        """Checks the buffers for an M x N product; the C argument."""
        if self.bias is not None:
            call(self.bias, "bias", N if N >= 0 else None, _kind(self.s.bias_dtype))
        if self.residual is not None:
            call(self.residual, "residual", _extent(M, self.s.ldr, N), _kind(self.s.residual_dtype))
        if self.preact is not None:
            self.preact.check(call, "preact", M, N)
        if self.output is not None:
            self.output.check(call, "output", M, N)
        return self.ref


def saved_write(rows: int, cols: int, x, ldx: int, out: Saved, x_dtype: Optional[int] = None,
                stream=None) -> None:
    """x (rows x cols, bf16 or fp32: taken from the tensor, BF16 for a raw
    address unless given) into the 8-bit checkpoint `out`."""
    if x_dtype is None:
        x_dtype = _dtype_of(x, BF16)
    call = _Call()
    xp = call(x, "x", _extent(rows, ldx, cols), _kind(x_dtype))
    _check(_lib.zero_saved_write(rows, cols, xp, ldx, x_dtype, out.check(call, "out", rows, cols),
                                 call.stream(stream)), "zero_saved_write")


def saved_read(rows: int, cols: int, saved: Saved, out, ldo: int, out_dtype: Optional[int] = None,
               stream=None) -> None:
    """The values of an 8-bit checkpoint, exact in bf16 and in fp32."""
    if out_dtype is None:
        out_dtype = _dtype_of(out, BF16)
    call = _Call()
    op = call(out, "out", _extent(rows, ldo, cols), _kind(out_dtype))
    _check(_lib.zero_saved_read(rows, cols, saved.check(call, "saved", rows, cols), op, ldo, out_dtype,
                                call.stream(stream)), "zero_saved_read")


def _operand_count(rows: int, K: int, ld: int, order: int) -> Optional[int]:
    return _operand_extent(rows, K, ld, order) if K >= 0 else None


def gemm_bf16_epilogue(M: int, N: int, K: int, A, lda: int, a_order: int, B, ldb: int, b_order: int,
                       C, ldc: int, c_dtype: int = FP32, epilogue: Optional[Epilogue] = None,
                       stream=None) -> None:
    """gemm_bf16 with bias, activation, residual and kept outputs."""
    call = _Call()
    Ap = call(A, "A", _operand_count(M, K, lda, a_order), "bf16")
    Bp = call(B, "B", _operand_count(N, K, ldb, b_order), "bf16")
    Cp = call(C, "C", _extent(M, ldc, N), _kind(c_dtype))
    ep = None if epilogue is None else epilogue.check(call, M, N)
    _check(_lib.zero_gemm_bf16_epilogue(M, N, K, Ap, lda, a_order, Bp, ldb, b_order, Cp, ldc,
                                        c_dtype, ep, call.stream(stream)), "zero_gemm_bf16_epilogue")


def act_backward_workspace(rows: int, cols: int) -> int:
    """Floats of workspace that dbias of rows x cols needs."""
    return _lib.zero_act_backward_workspace(rows, cols)


def _numel(x) -> int:
    """Elements of a workspace; a raw address is taken at its caller's word."""
    return 0 if x is None else (1 << 62) if x.__class__ is int else x.numel()


def _sums(call: _Call, rows: int, cols: int, dbias, workspace):
    """dbias and its workspace, checked."""
    if dbias is None:
        return None, None
    return (call(dbias, "dbias", max(cols, 0), "fp32"),
            call(workspace, "workspace", act_backward_workspace(rows, cols), "fp32"))


def act_backward(rows: int, cols: int, dy, ldy: int, act, preact: Optional[Saved], dz, ldz: int,
                 dbias=None, workspace=None, dy_dtype: Optional[int] = None, stream=None) -> None:
    """dz = dy act'(preact) in bf16 and dbias = its column sums in fp32."""
    if dy_dtype is None:
        dy_dtype = _dtype_of(dy, BF16)
    call = _Call()
    dyp = call(dy, "dy", _extent(rows, ldy, cols), _kind(dy_dtype))
    zp = None if preact is None else preact.check(call, "preact", rows, cols)
    dzp = call(dz, "dz", _extent(rows, ldz, cols), "bf16")
    dbp, wp = _sums(call, rows, cols, dbias, workspace)
    _check(_lib.zero_act_backward(rows, cols, dyp, ldy, dy_dtype, _act(act), zp, dzp, ldz, dbp, wp,
                                  _numel(workspace), call.stream(stream)), "zero_act_backward")


def gemm_saved_bf16(M: int, N: int, K: int, A: Saved, B, ldb: int, C, ldc: int, c_dtype: int = FP32,
                    stream=None) -> None:
    """C = A^T B from a kept K x M operand and a K x N bf16 one."""
    call = _Call()
    Ap = A.check(call, "A", K, M)
    Bp = call(B, "B", _extent(K, ldb, N), "bf16")
    Cp = call(C, "C", _extent(M, ldc, N), _kind(c_dtype))
    _check(_lib.zero_gemm_saved_bf16(M, N, K, Ap, Bp, ldb, Cp, ldc, c_dtype, call.stream(stream)),
           "zero_gemm_saved_bf16")


def _offsets(call: _Call, offsets, n_groups: int) -> Optional[int]:
    return call(offsets, "offsets", n_groups + 1 if n_groups >= 1 else None, "int64")


def _stacked(n: int, stride: int, each: Optional[int]) -> Optional[int]:
    """Elements of n matrices `stride` apart, the last `each` long."""
    return None if n < 1 or each is None else (n - 1) * stride + each


def gemm_grouped_rows_bf16(n_groups: int, offsets, rows: int, N: int, K: int, A, lda: int, B,
                           ldb: int, b_order: int, stride_b: int, C, ldc: int, c_dtype: int = BF16,
                           epilogue: Optional[Epilogue] = None, stream=None) -> None:
    """C[r] = epilogue(A[r] B_e) for the rows r of group e; `offsets` is a
    device int64 tensor of n_groups + 1."""
    call = _Call()
    op = _offsets(call, offsets, n_groups)
    Ap = call(A, "A", _operand_count(rows, K, lda, K_INNER), "bf16")
    Bp = call(B, "B", _stacked(n_groups, stride_b, _operand_count(N, K, ldb, b_order))
              if rows > 0 and N > 0 else 0, "bf16")
    Cp = call(C, "C", _extent(rows, ldc, N), _kind(c_dtype))
    ep = None if epilogue is None else epilogue.check(call, rows, N)
    _check(_lib.zero_gemm_grouped_rows_bf16(n_groups, op, rows, N, K, Ap, lda, Bp, ldb, b_order,
                                            stride_b, Cp, ldc, c_dtype, ep, call.stream(stream)),
           "zero_gemm_grouped_rows_bf16")


def gemm_grouped_depth_bf16(n_groups: int, offsets, rows: int, M: int, N: int, A, lda: int, B,
                            ldb: int, C, ldc: int, stride_c: int, c_dtype: int = FP32,
                            stream=None) -> None:
    """C_e = sum over the rows r of group e of A[r]^T B[r]."""
    call = _Call()
    op = _offsets(call, offsets, n_groups)
    Ap = call(A, "A", _extent(rows, lda, M), "bf16")
    Bp = call(B, "B", _extent(rows, ldb, N), "bf16")
    Cp = call(C, "C", _stacked(n_groups, stride_c, _extent(M, ldc, N)), _kind(c_dtype))
    _check(_lib.zero_gemm_grouped_depth_bf16(n_groups, op, rows, M, N, Ap, lda, Bp, ldb, Cp, ldc,
                                             stride_c, c_dtype, call.stream(stream)),
           "zero_gemm_grouped_depth_bf16")


def _layer_buffers(call: _Call, layout: Layout, unit: int, w_shards, w_full):
    """(the unit's (in, out, shard, padded) or None, the shards' pointers,
    w_full's), checked."""
    _need_len("w_shards", w_shards, _parts(layout))
    d = _layer_dims(layout, unit)
    shard, padded = (None, None) if d is None else d[2:]
    ptrs = [call(x, f"W shard of rank {q}", shard, "bf16") for q, x in enumerate(w_shards)]
    return d, (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs), call(w_full, "w_full", padded, "bf16")


def _times(rows: int, cols: Optional[int]) -> Optional[int]:
    return None if cols is None or rows < 0 else rows * cols


def fsdp_linear_act_forward(layout: Layout, unit: int, w_shards, batch: int, x, w_full, y,
                            epilogue: Optional[Epilogue] = None, y_dtype: int = BF16,
                            stream=None) -> None:
    """fsdp_linear_forward with an epilogue."""
    call = _Call()
    d, wp, wf = _layer_buffers(call, layout, unit, w_shards, w_full)
    inf, out = (None, None) if d is None else d[:2]
    xp = call(x, "x", _times(batch, inf), "bf16")
    yp = call(y, "y", _times(batch, out), _kind(y_dtype))
    ep = None if epilogue is None else epilogue.ref if d is None else epilogue.check(call, batch, out)
    _check(_lib.zero_fsdp_linear_act_forward(layout.handle, unit, wp, batch, xp, wf, ep, yp, y_dtype,
                                             call.stream(stream)), "zero_fsdp_linear_act_forward")


def fsdp_linear_act_backward(layout: Layout, unit: int, w_shards, batch: int, x: Saved, act,
                             preact: Optional[Saved], dy, w_full, dz, dx, dw_full, dbias=None,
                             workspace=None, dx_dtype: int = BF16, stream=None) -> None:
    """fsdp_linear_backward through the epilogue, from the kept x and z."""
    call = _Call()
    d, wp, wf = _layer_buffers(call, layout, unit, w_shards, w_full)
    inf, out, padded = (None, None, None) if d is None else (d[0], d[1], d[3])
    xr = x.ref if d is None else x.check(call, "x", batch, inf)
    zr = None if preact is None else \
        preact.ref if d is None else preact.check(call, "preact", batch, out)
    dyp = call(dy, "dy", _times(batch, out), "bf16")
    dzp = call(dz, "dz", _times(batch, out), "bf16")
    dxp = call(dx, "dx", _times(batch, inf), _kind(dx_dtype))
    dwp = call(dw_full, "dw_full", padded, "fp32")
    dbp, wsp = _sums(call, batch, 0 if d is None else out, dbias, workspace)
    _check(_lib.zero_fsdp_linear_act_backward(layout.handle, unit, wp, batch, xr, _act(act), zr, dyp,
                                              wf, dzp, dxp, dx_dtype, dwp, dbp, wsp,
                                              _numel(workspace), call.stream(stream)),
           "zero_fsdp_linear_act_backward")


def _expert_buffers(call: _Call, layout: Layout, unit: int, n_experts: int, w_shards, offsets, w_full):
    """_layer_buffers with one expert's in, and the offsets' pointer."""
    d, wp, wf = _layer_buffers(call, layout, unit, w_shards, w_full)
    op = _offsets(call, offsets, n_experts)
    if d is None or n_experts < 1 or d[0] % n_experts:
        return None, wp, wf, op
    return (d[0] // n_experts, *d[1:]), wp, wf, op


def fsdp_experts_forward(layout: Layout, unit: int, n_experts: int, w_shards, offsets, rows: int, x,
                         w_full, y, epilogue: Optional[Epilogue] = None, y_dtype: int = BF16,
                         stream=None) -> None:
    """The grouped forward of an expert layer whose weights (n_experts * in
    rows x out) are one row-sharded unit."""
    call = _Call()
    d, wp, wf, op = _expert_buffers(call, layout, unit, n_experts, w_shards, offsets, w_full)
    inf, out = (None, None) if d is None else d[:2]
    xp = call(x, "x", _times(rows, inf), "bf16")
    yp = call(y, "y", _times(rows, out), _kind(y_dtype))
    ep = None if epilogue is None else epilogue.ref if d is None else epilogue.check(call, rows, out)
    _check(_lib.zero_fsdp_experts_forward(layout.handle, unit, n_experts, wp, op, rows, xp, wf, ep, yp,
                                          y_dtype, call.stream(stream)), "zero_fsdp_experts_forward")


def fsdp_experts_backward(layout: Layout, unit: int, n_experts: int, w_shards, offsets, rows: int,
                          x, dy, w_full, dx, dw_full, dx_dtype: int = BF16, stream=None) -> None:
    """The grouped dx and the experts' dW (dw_full: the padded unit, fp32)."""
    call = _Call()
    d, wp, wf, op = _expert_buffers(call, layout, unit, n_experts, w_shards, offsets, w_full)
    inf, out, padded = (None, None, None) if d is None else (d[0], d[1], d[3])
    xp = call(x, "x", _times(rows, inf), "bf16")
    dyp = call(dy, "dy", _times(rows, out), "bf16")
    dxp = call(dx, "dx", _times(rows, inf), _kind(dx_dtype))
    dwp = call(dw_full, "dw_full", padded, "fp32")
    _check(_lib.zero_fsdp_experts_backward(layout.handle, unit, n_experts, wp, op, rows, xp, dyp, wf,
                                           dxp, dx_dtype, dwp, call.stream(stream)),
           "zero_fsdp_experts_backward")


# ---------------------------------------------------- training operators --

def layer_norm_forward(rows: int, cols: int, x, ldx: int, gain, bias, eps: float, y, ldy: int,
                       mean=None, rstd=None, x_dtype: int = BF16, param_dtype: int = BF16,
                       y_dtype: int = BF16, stream=None) -> None:
    """y = (x - mean) rstd gain + bias, row by row; mean and rstd (fp32) are kept for the
    backward pass if given.  Types are taken from tensors; the *_dtype arguments
    are those of raw addresses."""
    call = _Call()
    xt, yt = _dtype_of(x, x_dtype), _dtype_of(y, y_dtype)
    pt = _dtype_of(bias if gain is None or gain.__class__ is int else gain, param_dtype)
    n = max(cols, 0)
    xp = call(x, "x", _extent(rows, ldx, cols), _kind(xt))
    gp = call(gain, "gain", n, _kind(pt))
    bp = call(bias, "bias", n, _kind(pt))
    yp = call(y, "y", _extent(rows, ldy, cols), _kind(yt))
    mp = call(mean, "mean", max(rows, 0), "fp32")
    rp = call(rstd, "rstd", max(rows, 0), "fp32")
    _check(_lib.zero_layer_norm_forward(rows, cols, xp, ldx, xt, gp, bp, pt, eps, yp, ldy, yt, mp, rp,
                                        call.stream(stream)), "zero_layer_norm_forward")


def layer_norm_workspace(rows: int, cols: int) -> int:
    """Floats of workspace that dgain and dbias need."""
    return _lib.zero_layer_norm_workspace(rows, cols)


def layer_norm_backward(rows: int, cols: int, dy, lddy: int, x, ldx: int, gain, mean, rstd, dx,
                        lddx: int, dgain=None, dbias=None, workspace=None, residual=None,
                        ldr: int = 0, dy_dtype: int = BF16, x_dtype: int = BF16,
                        param_dtype: int = BF16, dx_dtype: int = BF16, stream=None) -> None:
    """dx, with the gradient `residual` that reaches x past the norm added, and the sums
    dgain and dbias."""
    call = _Call()
    yt, xt, pt, dt = (_dtype_of(t, d) for t, d in ((dy, dy_dtype), (x, x_dtype), (gain, param_dtype),
                                                   (dx, dx_dtype)))
    n, r = max(cols, 0), max(rows, 0)
    yp = call(dy, "dy", _extent(rows, lddy, cols), _kind(yt))
    xp = call(x, "x", _extent(rows, ldx, cols), _kind(xt))
    gp = call(gain, "gain", n, _kind(pt))
    mp = call(mean, "mean", r, "fp32")
    rp = call(rstd, "rstd", r, "fp32")
    sp = call(residual, "residual", _extent(rows, ldr, cols), _kind(dt))
    dp = call(dx, "dx", _extent(rows, lddx, cols), _kind(dt))
    dgp = call(dgain, "dgain", n, "fp32")
    dbp = call(dbias, "dbias", n, "fp32")
    need = layer_norm_workspace(rows, cols) if dgain is not None or dbias is not None else 0
    wp = call(workspace, "workspace", need, "fp32")
    _check(_lib.zero_layer_norm_backward(rows, cols, yp, lddy, yt, xp, ldx, xt, gp, pt, mp, rp, sp, ldr,
                                         dp, lddx, dt, dgp, dbp, wp, _numel(workspace),
                                         call.stream(stream)), "zero_layer_norm_backward")


class Router:
    """How tokens choose experts: `top_k` of `n_experts` by softmax or sigmoid scores,
    from the `top_groups` best of `groups` equal runs of experts, a group ranked by
    its `group_best` (1 or 2) best experts; weights renormalised and scaled."""
    __slots__ = ("s", "ref")

    def __init__(self, n_experts: int, top_k: int, score="softmax", groups: int = 1,
                 top_groups: int = 1, group_best: int = 1, renormalize: bool = True,
                 scale: float = 1.0):
        if isinstance(score, str):
            if score not in SCORE:
                raise ValueError(f"unknown score {score!r} (one of {', '.join(SCORE)})")
            score = SCORE[score]
        self.s = _Router(n_experts, top_k, groups, top_groups, group_best, score,
                         int(bool(renormalize)), scale)
        self.ref = ctypes.byref(self.s)


def route_workspace(router: Router, tokens: int) -> int:
    """int32 of workspace that routing `tokens` tokens needs."""
    return _lib.zero_route_workspace(router.ref, tokens)


def route_forward(router: Router, tokens: int, logits, ldl: int, experts, weights, offsets, rows_of,
                  workspace=None, bias=None, active=None, logits_dtype: int = BF16,
                  stream=None) -> None:
    """Each token's experts and weights (tokens x top_k), the experts' offsets for the
    grouped products and each choice's row when sorted by expert."""
    call = _Call()
    lt, E = _dtype_of(logits, logits_dtype), router.s.n_experts
    n, e = max(tokens, 0) * max(router.s.top_k, 0), max(E, 0)
    lp = call(logits, "logits", _extent(tokens, ldl, E), _kind(lt))
    ep = call(experts, "experts", n, "int32")
    wp = call(weights, "weights", n, "fp32")
    op = call(offsets, "offsets", e + 1, "int64")
    rp = call(rows_of, "rows_of", n, "int32")
    sp = call(workspace, "workspace", route_workspace(router, tokens), "int32")
    bp = call(bias, "bias", e, "fp32")
    ap = call(active, "active", max(tokens, 0), "bytes8")
    _check(_lib.zero_route_forward(router.ref, tokens, lp, ldl, lt, bp, ap, ep, wp, op, rp, sp,
                                   _numel(workspace), call.stream(stream)), "zero_route_forward")


def route_backward(router: Router, tokens: int, logits, ldl: int, experts, dweights, dlogits,
                   ldd: int, logits_dtype: int = BF16, dlogits_dtype: int = BF16,
                   stream=None) -> None:
    """dlogits from dweights, the choice held fixed."""
    call = _Call()
    lt, dt, E = _dtype_of(logits, logits_dtype), _dtype_of(dlogits, dlogits_dtype), router.s.n_experts
    n = max(tokens, 0) * max(router.s.top_k, 0)
    lp = call(logits, "logits", _extent(tokens, ldl, E), _kind(lt))
    ep = call(experts, "experts", n, "int32")
    wp = call(dweights, "dweights", n, "fp32")
    dp = call(dlogits, "dlogits", _extent(tokens, ldd, E), _kind(dt))
    _check(_lib.zero_route_backward(router.ref, tokens, lp, ldl, lt, ep, wp, dp, ldd, dt,
                                    call.stream(stream)), "zero_route_backward")


def experts_dispatch(tokens: int, top_k: int, cols: int, x, ldx: int, rows_of, rows: int, out, ldo: int,
                     weights=None, stream=None) -> None:
    """out[rows_of[t, j]] = (weights[t, j]) x[t], bf16."""
    call = _Call()
    n = max(tokens, 0) * max(top_k, 0)
    xp = call(x, "x", _extent(tokens, ldx, cols), "bf16")
    rp = call(rows_of, "rows_of", n, "int32")
    wp = call(weights, "weights", n, "fp32")
    op = call(out, "out", _extent(rows, ldo, cols), "bf16")
    _check(_lib.zero_experts_dispatch(tokens, top_k, cols, xp, ldx, rp, wp, rows, op, ldo,
                                      call.stream(stream)), "zero_experts_dispatch")


def experts_combine(tokens: int, top_k: int, cols: int, src, lds: int, rows: int, rows_of, y, ldy: int,
                    weights=None, residual=None, ldr: int = 0, y_dtype: int = BF16,
                    stream=None) -> None:
    """y[t] = sum over j of (weights[t, j]) src[rows_of[t, j]] (+ residual[t])."""
    call = _Call()
    yt, n = _dtype_of(y, y_dtype), max(tokens, 0) * max(top_k, 0)
    sp = call(src, "src", _extent(rows, lds, cols), "bf16")
    rp = call(rows_of, "rows_of", n, "int32")
    wp = call(weights, "weights", n, "fp32")
    ep = call(residual, "residual", _extent(tokens, ldr, cols), "bf16")
    yp = call(y, "y", _extent(tokens, ldy, cols), _kind(yt))
    _check(_lib.zero_experts_combine(tokens, top_k, cols, sp, lds, rows, rp, wp, ep, ldr, yp, ldy, yt,
                                     call.stream(stream)), "zero_experts_combine")


def experts_combine_backward(tokens: int, top_k: int, cols: int, dy, lddy: int, rows: int, rows_of,
                             weights, src, lds: int, dsrc, ldds: int, dweights, stream=None) -> None:
    """dsrc[rows_of[t, j]] = weights[t, j] dy[t] and dweights[t, j] = dy[t] . src[rows_of[t, j]]."""
    call = _Call()
    n = max(tokens, 0) * max(top_k, 0)
    yp = call(dy, "dy", _extent(tokens, lddy, cols), "bf16")
    rp = call(rows_of, "rows_of", n, "int32")
    wp = call(weights, "weights", n, "fp32")
    sp = call(src, "src", _extent(rows, lds, cols), "bf16")
    dp = call(dsrc, "dsrc", _extent(rows, ldds, cols), "bf16")
    dwp = call(dweights, "dweights", n, "fp32")
    _check(_lib.zero_experts_combine_backward(tokens, top_k, cols, yp, lddy, rows, rp, wp, sp, lds, dp,
                                              ldds, dwp, call.stream(stream)),
           "zero_experts_combine_backward")


def linear_xent_workspace(rows: int, vocab: int, hidden: int, backward: bool = False,
                          piece: int = 0) -> int:
    """Floats of workspace of the loss, or of its gradient."""
    return _lib.zero_linear_xent_workspace(rows, vocab, hidden, int(bool(backward)), piece)


def _head_extent(vocab: int, hidden: int, ld: int, order: int) -> Optional[int]:
    return _extent(hidden, ld, vocab) if order == K_OUTER else _extent(vocab, ld, hidden)


def linear_xent_forward(rows: int, vocab: int, hidden: int, x, ldx: int, w, ldw: int, w_order: int,
                        targets, loss, lse, workspace, stream=None) -> None:
    """loss and lse of softmax(x W) against targets (int64; one outside [0, vocab) is none)."""
    call = _Call()
    r = max(rows, 0)
    xp = call(x, "x", _extent(rows, ldx, hidden), "bf16")
    wp = call(w, "w", _head_extent(vocab, hidden, ldw, w_order), "bf16")
    tp = call(targets, "targets", r, "int64")
    lp = call(loss, "loss", r, "fp32")
    ep = call(lse, "lse", r, "fp32")
    sp = call(workspace, "workspace", linear_xent_workspace(rows, vocab, hidden), "fp32")
    _check(_lib.zero_linear_xent_forward(rows, vocab, hidden, xp, ldx, wp, ldw, w_order, tp, lp, ep, sp,
                                         _numel(workspace), call.stream(stream)),
           "zero_linear_xent_forward")


def linear_xent_backward(rows: int, vocab: int, hidden: int, x, ldx: int, w, ldw: int, w_order: int,
                         targets, lse, dloss, dx, lddx: int, dw, lddw: int, piece: int, workspace,
                         dx_dtype: int = BF16, dw_dtype: int = FP32, stream=None) -> None:
    """dx and dw from the rows' dloss; piece 0: the default pieces of the vocabulary."""
    call = _Call()
    dxt, dwt, r = _dtype_of(dx, dx_dtype), _dtype_of(dw, dw_dtype), max(rows, 0)
    xp = call(x, "x", _extent(rows, ldx, hidden), "bf16")
    wp = call(w, "w", _head_extent(vocab, hidden, ldw, w_order), "bf16")
    tp = call(targets, "targets", r, "int64")
    ep = call(lse, "lse", r, "fp32")
    lp = call(dloss, "dloss", r, "fp32")
    dxp = call(dx, "dx", _extent(rows, lddx, hidden), _kind(dxt))
    dwp = call(dw, "dw", _head_extent(vocab, hidden, lddw, w_order), _kind(dwt))
    sp = call(workspace, "workspace", linear_xent_workspace(rows, vocab, hidden, True, piece), "fp32")
    _check(_lib.zero_linear_xent_backward(rows, vocab, hidden, xp, ldx, wp, ldw, w_order, tp, ep, lp, dxp,
                                          lddx, dxt, dwp, lddw, dwt, piece, sp, _numel(workspace),
                                          call.stream(stream)), "zero_linear_xent_backward")


def _head(call: _Call, layout: Layout, unit: int, w_shards, w_full, w_order: int, batch: int, x, targets):
    """(vocab, hidden, the padded unit's elements; None where the unit does not exist), and the
    arguments every head call begins with, checked."""
    d, wp, wf = _layer_buffers(call, layout, unit, w_shards, w_full)
    hidden, vocab, padded = (None, None, None) if d is None else (d[0], d[1], d[3])
    if d is not None and w_order == K_INNER:
        hidden, vocab = vocab, hidden
    xp = call(x, "x", _times(batch, hidden), "bf16")
    tp = call(targets, "targets", max(batch, 0), "int64")
    return vocab, hidden, padded, wp, wf, xp, tp


def fsdp_head_forward(layout: Layout, unit: int, w_shards, w_order: int, batch: int, x, w_full, targets,
                      loss, lse, workspace, stream=None) -> None:
    """The loss of a head whose W is a row-sharded unit."""
    call = _Call()
    vocab, hidden, _, wp, wf, xp, tp = _head(call, layout, unit, w_shards, w_full, w_order, batch, x,
                                             targets)
    r = max(batch, 0)
    lp = call(loss, "loss", r, "fp32")
    ep = call(lse, "lse", r, "fp32")
    sp = call(workspace, "workspace",
              None if vocab is None else linear_xent_workspace(batch, vocab, hidden), "fp32")
    _check(_lib.zero_fsdp_head_forward(layout.handle, unit, wp, w_order, batch, xp, wf, tp, lp, ep, sp,
                                       _numel(workspace), call.stream(stream)),
           "zero_fsdp_head_forward")


def fsdp_head_backward(layout: Layout, unit: int, w_shards, w_order: int, batch: int, x, w_full, targets,
                       lse, dloss, dx, dw_full, piece: int, workspace, dx_dtype: int = BF16,
                       stream=None) -> None:
    """dx, and dW as the padded unit in fp32."""
    call = _Call()
    vocab, hidden, padded, wp, wf, xp, tp = _head(call, layout, unit, w_shards, w_full, w_order, batch,
                                                  x, targets)
    dxt, r = _dtype_of(dx, dx_dtype), max(batch, 0)
    ep = call(lse, "lse", r, "fp32")
    lp = call(dloss, "dloss", r, "fp32")
    dxp = call(dx, "dx", _times(batch, hidden), _kind(dxt))
    dwp = call(dw_full, "dw_full", padded, "fp32")
    sp = call(workspace, "workspace",
              None if vocab is None else linear_xent_workspace(batch, vocab, hidden, True, piece), "fp32")
    _check(_lib.zero_fsdp_head_backward(layout.handle, unit, wp, w_order, batch, xp, wf, tp, ep, lp, dxp,
                                        dxt, dwp, piece, sp, _numel(workspace), call.stream(stream)),
           "zero_fsdp_head_backward")


class TensorList:
    """The tensors of one optimizer step, described once: a list each of masters (fp32),
    gradients (all bf16 or all fp32; None until set_grads, and for a tensor without
    elements), parameters (bf16, or None), m and v (fp32, or 8-bit codes with m_scales and
    v_scales), and whether weight decay applies (default: to all).  Tensors are contiguous,
    of any shape; no two may share memory.  Keeps its buffers alive."""
    __slots__ = ("s", "n", "state", "grad_dtype", "device", "sizes", "_keep")

    def __init__(self, masters, grads, params, m, v, m_scales=None, v_scales=None, decay=None):
        self.n = len(masters)
        self.state = STATE_FP32 if m_scales is None else STATE_E4M3
        none = [None] * self.n
        lists = {"master": masters, "param": none if params is None else params, "m": m, "v": v,
                 "m_scales": none if m_scales is None else m_scales,
                 "v_scales": none if v_scales is None else v_scales}
        for name, x in lists.items():
            _need_len(name, x, self.n)
        # the tensors, not the caller's lists, which may change
        lists = {name: tuple(x) for name, x in lists.items()}
        decay = [True] * self.n if decay is None else decay
        _need_len("decay", decay, self.n)
        self.s = (_Tensor * max(1, self.n))()
        call, seen = _Call(), set()
        kinds = {"master": "fp32", "param": "bf16", "m": "fp32", "v": "fp32"}
        if self.state == STATE_E4M3:
            kinds.update({"m": "codes", "v": "codes", "m_scales": "codes", "v_scales": "codes"})
        self.sizes = [x.numel() for x in lists["master"]]
        for i, size in enumerate(self.sizes):
            d = self.s[i]
            d.n, d.decay = size, int(bool(decay[i]))
            for name, kind in kinds.items():
                x = lists[name][i]
                if x is None and name != "param":
                    raise ValueError(f"tensor {i}: {name} is required")
                count = -(-size // 32) if name.endswith("scales") else size
                p = call(x, f"{name} of tensor {i}", count, kind)
                if p and size:
                    if p in seen:
                        raise ValueError(f"{name} of tensor {i} is given twice")
                    seen.add(p)
                setattr(d, name, p)
        self.device, self.grad_dtype, self._keep = call.device, BF16, [lists]
        if grads is not None:
            self.set_grads(grads)

    def set_grads(self, grads) -> None:
        """Other gradient tensors for the next steps.  A list that is refused changes
        nothing."""
        _need_len("grads", grads, self.n)
        grads = tuple(grads)
        call = _Call()
        call.device = self.device
        kind, pointers = None, []
        for i, x in enumerate(grads):
            if kind is None and x is not None:
                kind = _dtype_of(x, BF16)
            pointers.append(call(x, f"gradient of tensor {i}", self.sizes[i], _kind(kind or BF16)))
        for d, p in zip(self.s, pointers):
            d.grad = p
        self.grad_dtype = BF16 if kind is None else kind
        self._keep[1:] = [grads]

    def partials_count(self) -> int:
        """fp64 partial sums that tensors_sumsq writes."""
        return _lib.zero_tensors_partials_count(self.n, self.s)

    def _call(self) -> _Call:
        call = _Call()
        call.device = self.device
        return call


def adam_tensors(tensors: TensorList, cfg: AdamCfg, seed: int = 0, clip_coef=None, stream=None) -> None:
    """One Adam / AdamW step of every tensor of the list."""
    call = tensors._call()
    cp = call(clip_coef, "clip_coef", 1, "fp32")
    _check(_lib.zero_adam_tensors(tensors.n, tensors.s, tensors.state, tensors.grad_dtype,
                                  ctypes.byref(cfg), seed & (2 ** 64 - 1), cp, call.stream(stream)),
           "zero_adam_tensors")


def adam_tensors_table(tensors: TensorList, table, n_entries: int, step_counter, seed: int = 0,
                       clip_coef=None, stream=None) -> None:
    """adam_tensors with the scalars of table[*step_counter - 1] (device table and counter)."""
    call = tensors._call()
    _need(table, "table", n_entries * ctypes.sizeof(AdamTableEntry), "bytes")
    sp = call(step_counter, "step_counter", 1, "int64")
    cp = call(clip_coef, "clip_coef", 1, "fp32")
    _check(_lib.zero_adam_tensors_table(tensors.n, tensors.s, tensors.state, tensors.grad_dtype,
                                        _addr(table), n_entries, sp, seed & (2 ** 64 - 1), cp,
                                        call.stream(stream)), "zero_adam_tensors_table")


def tensors_sumsq(tensors: TensorList, partials, stream=None) -> None:
    """The gradients' sums of squares, for clip_coef: partials_count() fp64."""
    call = tensors._call()
    n = tensors.partials_count()
    pp = call(partials, "partials", n, "fp64")
    _check(_lib.zero_tensors_sumsq(tensors.n, tensors.s, tensors.grad_dtype, pp, _numel(partials),
                                   call.stream(stream)), "zero_tensors_sumsq")


def adam_state_read(n: int, codes, scales, out, second: bool = False, out_dtype: int = BF16,
                    stream=None) -> None:
    """What n 8-bit state codes stand for: m, or with `second` v."""
    call = _Call()
    ot, k = _dtype_of(out, out_dtype), max(n, 0)
    cp = call(codes, "codes", k, "codes")
    sp = call(scales, "scales", -(-k // 32), "codes")
    op = call(out, "out", k, _kind(ot))
    _check(_lib.zero_adam_state_read(n, cp, sp, int(bool(second)), op, ot, call.stream(stream)),
           "zero_adam_state_read")


def stream_mix(kind: int, grads, master, m, v, param, n: int, stream=None,
               state_chunk: int = 0, grad_chunk: int = 0) -> None:
    """zero_stream_mix: the fused step's memory traffic without its
    arithmetic (kind MIX_STEP_STREAMS), its reads alone (MIX_READS) or its
    writes alone (MIX_WRITES), over n elements; state_chunk E > 0 takes
    master, m, v in the chunked format (m = master + E, v = master + 2E),
    grad_chunk G > 0 the rank gradients chunked (grads[q] = grads[0] + qG)."""

    def count(E, k):
        return n if E <= 0 or n <= 0 else ((n - 1) // E) * k * E + (n - 1) % E + 1

    for q, x in enumerate(grads):
        _need(x, f"gradient buffer of rank {q}", count(grad_chunk, len(grads)), "bf16")
    sc = count(state_chunk, 3)
    for name, x in (("master", master), ("m", m), ("v", v)):
        _need(x, name, sc, "fp32")
    _need(param, "param", n, "bf16")
    _check(_lib.zero_stream_mix(kind, _ptrs(grads), len(grads), _addr(master), _addr(m), _addr(v),
                                _addr(param), n, state_chunk, grad_chunk, _stream(stream)),
           "zero_stream_mix")


def grad_accumulate(main_grad, micro_bf16, n: int, stream=None) -> None:
    _need(main_grad, "main_grad", n, "fp32")
    _need(micro_bf16, "micro_bf16", n, "bf16")
    _check(_lib.zero_grad_accumulate(_addr(main_grad), _addr(micro_bf16), n, _stream(stream)),
           "zero_grad_accumulate")


def raw():
    """The ctypes library object (for tests of the exported symbols)."""
    return _lib
