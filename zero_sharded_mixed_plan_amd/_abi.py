"""ctypes binding of libzero_shard.so: the C ABI declared in include/zero_shard.h.

Argument marshalling only; every step of the computation runs in the library.
Functions keep the C names.  Device pointers are plain integers (e.g. a torch
tensor's data_ptr()); `stream` is a hipStream_t as an integer (0 = null stream).
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Tuple

# ZERO_SHARD_LIB selects another build of the same library (e.g. a tuning variant)
LIB_PATH = os.environ.get("ZERO_SHARD_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libzero_shard.so")

ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ENOMEM, ZERO_EHIP, ZERO_EIO = 0, -1, -2, -3, -4, -5
ZERO_F32, ZERO_BF16, ZERO_F16 = 0, 1, 2
ZERO_STATE_SEPARATE, ZERO_STATE_TILED = 0, 1
ZERO_STATE_TILE = 2048
ZERO_GRAD_SHARD, ZERO_GRAD_FULL = 0, 1
DTYPE_CODES = {"f32": ZERO_F32, "bf16": ZERO_BF16, "f16": ZERO_F16}
DTYPE_BYTES = {ZERO_F32: 4, ZERO_BF16: 2, ZERO_F16: 2}

# every symbol the header declares
EXPORTS = [
    "zero_plan", "zero_plan_dim0", "zero_plan_free", "zero_plan_shard_numel", "zero_plan_total_numel",
    "zero_plan_padded_numel", "zero_plan_world", "zero_plan_num_buckets", "zero_plan_num_tensors",
    "zero_plan_bucket", "zero_plan_tensor", "zero_plan_rank_segment", "zero_plan_bytes",
    "zero_state_numel", "zero_workspace_bytes", "zero_plan_piece_table_bytes", "zero_plan_attach_piece_table",
    "zero_reduce_shard", "zero_shard_norm", "zero_noalloc_max_shard", "zero_reduce_norm_noalloc",
    "zero_adam_step", "zero_scaler_init", "zero_scaler_update", "zero_scaler_inv_scale", "zero_plan_hash",
    "zero_checkpoint_save", "zero_checkpoint_load", "zero_stream_copy", "zero_last_error", "zero_version",
    "zero_dropout", "zero_embed_lookup", "zero_embed_grad", "zero_embed_grad_ws_bytes",
    "zero_pack8", "zero_unpack8", "zero_rms_norm", "zero_rms_norm_grad", "zero_rms_grad_ws_bytes",
    "zero_gated", "zero_gated_grad", "zero_gated_input_grad", "zero_gated_weight_grad", "zero_gated_ws_bytes",
]


class ZeroError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class zero_adam_args_t(ctypes.Structure):
    _fields_ = [
        ("rank", ctypes.c_int32),
        ("grad", ctypes.c_void_p),
        ("grad_ld", ctypes.c_int64),
        ("grad_dtype", ctypes.c_int),
        ("grad_count", ctypes.c_int32),
        ("grad_layout", ctypes.c_int32),
        ("inv_scale", ctypes.c_float),
        ("g_stash", ctypes.c_void_p),
        ("clip_coef", ctypes.c_void_p),
        ("state_layout", ctypes.c_int32),
        ("master_in", ctypes.c_void_p),
        ("m_in", ctypes.c_void_p),
        ("v_in", ctypes.c_void_p),
        ("master_out", ctypes.c_void_p),
        ("m_out", ctypes.c_void_p),
        ("v_out", ctypes.c_void_p),
        ("gather", ctypes.c_void_p),
        ("param_dtype", ctypes.c_int),
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
        ("step", ctypes.c_int64),
        ("skip_in", ctypes.c_void_p),
        ("overflow_out", ctypes.c_void_p),
        ("ev_begin", ctypes.c_void_p),
        ("ev_end", ctypes.c_void_p),
        ("ctl", ctypes.c_void_p),
    ]


class zero_scaler_t(ctypes.Structure):
    _fields_ = [
        ("scale", ctypes.c_float),
        ("growth_tracker", ctypes.c_int32),
        ("growth_factor", ctypes.c_float),
        ("backoff_factor", ctypes.c_float),
        ("growth_interval", ctypes.c_int32),
    ]


class zero_step_ctl_t(ctypes.Structure):
    """Step control kept in device memory (this is its host image)."""
    _fields_ = [
        ("step", ctypes.c_int64),
        ("skipped", ctypes.c_int64),
        ("lr", ctypes.c_double),
        ("scaler", zero_scaler_t),
        ("dynamic", ctypes.c_int32),
        ("k", ctypes.c_float * 8),
    ]


class zero_ckpt_meta_t(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int64), ("scaler", zero_scaler_t)]


class zero_drop_t(ctypes.Structure):
    _fields_ = [
        ("p", ctypes.c_double),
        ("seed", ctypes.c_uint64),
        ("site", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
        ("step", ctypes.c_int64),
        ("step_dev", ctypes.c_void_p),
        ("row0", ctypes.c_int64),
    ]


class zero_embed_args_t(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("ld_table", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("id0", ctypes.c_int64),
        ("table_dtype", ctypes.c_int),
        ("id_bytes", ctypes.c_int32),
        ("ids", ctypes.c_void_p),
        ("n_ids", ctypes.c_int64),
        ("dim", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("pos_table", ctypes.c_void_p),
        ("ld_pos", ctypes.c_int64),
        ("pos_rows", ctypes.c_int64),
        ("pos", ctypes.c_void_p),
        ("pos_period", ctypes.c_int64),
        ("out", ctypes.c_void_p),
        ("ld_out", ctypes.c_int64),
        ("out_dtype", ctypes.c_int),
        ("drop", ctypes.c_void_p),
    ]


class zero_embed_grad_args_t(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p),
        ("ld_dy", ctypes.c_int64),
        ("dy_dtype", ctypes.c_int),
        ("id_bytes", ctypes.c_int32),
        ("ids", ctypes.c_void_p),
        ("period", ctypes.c_int64),
        ("n_ids", ctypes.c_int64),
        ("dim", ctypes.c_int64),
        ("id0", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("grad_dtype", ctypes.c_int),
        ("grad", ctypes.c_void_p),
        ("ld_grad", ctypes.c_int64),
        ("accumulate", ctypes.c_int32),
        ("drop", ctypes.c_void_p),
        ("ws", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_int64),
    ]


class zero_held_t(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("ld_codes", ctypes.c_int64),
        ("scales", ctypes.c_void_p),
        ("ld_scales", ctypes.c_int64),
    ]


class zero_rms_args_t(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("ld_x", ctypes.c_int64),
        ("x_dtype", ctypes.c_int),
        ("res_dtype", ctypes.c_int),
        ("residual", ctypes.c_void_p),
        ("ld_res", ctypes.c_int64),
        ("total", ctypes.c_void_p),
        ("ld_total", ctypes.c_int64),
        ("weight", ctypes.c_void_p),
        ("weight_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("out", ctypes.c_void_p),
        ("ld_out", ctypes.c_int64),
        ("held", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("eps", ctypes.c_double),
    ]


class zero_rms_grad_args_t(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p),
        ("ld_dy", ctypes.c_int64),
        ("dy_dtype", ctypes.c_int),
        ("h_dtype", ctypes.c_int),
        ("h", ctypes.c_void_p),
        ("ld_h", ctypes.c_int64),
        ("held", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("weight_dtype", ctypes.c_int),
        ("dweight_dtype", ctypes.c_int),
        ("dres", ctypes.c_void_p),
        ("ld_dres", ctypes.c_int64),
        ("dh", ctypes.c_void_p),
        ("ld_dh", ctypes.c_int64),
        ("dweight", ctypes.c_void_p),
        ("accumulate", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ws", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_int64),
    ]


class zero_gated_args_t(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("dim", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("act", ctypes.c_int),
        ("x", ctypes.c_void_p),
        ("ld_x", ctypes.c_int64),
        ("w_gate", ctypes.c_void_p),
        ("ld_w_gate", ctypes.c_int64),
        ("w_up", ctypes.c_void_p),
        ("ld_w_up", ctypes.c_int64),
        ("a", ctypes.c_void_p),
        ("ld_a", ctypes.c_int64),
        ("g", ctypes.c_void_p),
        ("ld_g", ctypes.c_int64),
        ("u", ctypes.c_void_p),
        ("ld_u", ctypes.c_int64),
        ("g8", ctypes.c_void_p),
        ("u8", ctypes.c_void_p),
        ("da", ctypes.c_void_p),
        ("ld_da", ctypes.c_int64),
        ("dg", ctypes.c_void_p),
        ("ld_dg", ctypes.c_int64),
        ("du", ctypes.c_void_p),
        ("ld_du", ctypes.c_int64),
        ("dx", ctypes.c_void_p),
        ("ld_dx", ctypes.c_int64),
        ("dw_gate", ctypes.c_void_p),
        ("ld_dw_gate", ctypes.c_int64),
        ("dw_up", ctypes.c_void_p),
        ("ld_dw_up", ctypes.c_int64),
        ("dw_dtype", ctypes.c_int),
        ("accumulate", ctypes.c_int32),
        ("ws", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_int64),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library once.  Fails loudly when it has not been built."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def load(path: str, required: bool = True) -> ctypes.CDLL:
    """Load one build of the library from `path` and declare its C signatures
    (required=False skips entry points an older build does not export)."""
    # torch first: the library must bind to the HIP runtime torch already uses
    # for the device memory and streams it hands over (one runtime per process)
    import torch  # noqa: F401
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m zero_sharded_mixed_plan_amd.build` (hipcc, gfx950)")
    L = ctypes.CDLL(path)
    i32, i64, vp, f32, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double
    P64, P32 = ctypes.POINTER(i64), ctypes.POINTER(i32)
    sig = {
        "zero_plan": (ctypes.c_int, [P64, i32, i32, i64, ctypes.POINTER(vp)]),
        "zero_plan_dim0": (ctypes.c_int, [P64, P64, i32, i32, ctypes.POINTER(vp)]),
        "zero_plan_free": (None, [vp]),
        "zero_plan_shard_numel": (i64, [vp]),
        "zero_plan_total_numel": (i64, [vp]),
        "zero_plan_padded_numel": (i64, [vp]),
        "zero_plan_world": (i32, [vp]),
        "zero_plan_num_buckets": (i32, [vp]),
        "zero_plan_num_tensors": (i32, [vp]),
        "zero_plan_bucket": (ctypes.c_int, [vp, i32, P64, P64, P64, P64, P32, P32]),
        "zero_plan_tensor": (ctypes.c_int, [vp, i32, P32, P64]),
        "zero_plan_rank_segment": (ctypes.c_int, [vp, i32, i32, P64, P64, P64]),
        "zero_plan_bytes": (ctypes.c_int, [vp, i32, ctypes.POINTER(f64), P64]),
        "zero_state_numel": (i64, [vp, i32]),
        "zero_workspace_bytes": (ctypes.c_size_t, [vp]),
        "zero_plan_piece_table_bytes": (i64, [vp]),
        "zero_plan_attach_piece_table": (ctypes.c_int, [vp, i32, vp, i64]),
        "zero_reduce_shard": (ctypes.c_int, [vp, i32, vp, i64, i32, i32, ctypes.c_int, f32, vp, vp, i32, vp, vp]),
        "zero_shard_norm": (ctypes.c_int, [vp, vp, f64, f64, vp, vp, vp, vp]),
        "zero_noalloc_max_shard": (i64, []),
        "zero_reduce_norm_noalloc": (ctypes.c_int, [vp, i32, vp, i64, i32, i32, ctypes.c_int, f32, vp, f64, f64,
                                                    vp, vp, vp, vp, vp]),
        "zero_adam_step": (ctypes.c_int, [vp, ctypes.POINTER(zero_adam_args_t), vp]),
        "zero_scaler_init": (ctypes.c_int, [ctypes.POINTER(zero_scaler_t), f32, f32, f32, i32]),
        "zero_scaler_update": (ctypes.c_int, [ctypes.POINTER(zero_scaler_t), i32]),
        "zero_scaler_inv_scale": (f32, [ctypes.POINTER(zero_scaler_t)]),
        "zero_plan_hash": (ctypes.c_uint64, [vp]),
        "zero_checkpoint_save": (ctypes.c_int, [vp, i32, ctypes.c_char_p, i32, vp, vp, vp,
                                                ctypes.POINTER(zero_ckpt_meta_t), vp]),
        "zero_checkpoint_load": (ctypes.c_int, [vp, i32, ctypes.c_char_p, i32, vp, vp, vp,
                                                ctypes.POINTER(zero_ckpt_meta_t), vp]),
        "zero_stream_copy": (ctypes.c_int, [vp, vp, i64, vp]),
        "zero_dropout": (ctypes.c_int, [vp, i64, ctypes.c_int, vp, i64, vp, i64, ctypes.c_int, i64, i64, vp, vp]),
        "zero_embed_lookup": (ctypes.c_int, [vp, vp]),
        "zero_embed_grad": (ctypes.c_int, [vp, vp]),
        "zero_embed_grad_ws_bytes": (i64, [i64, i64, i64]),
        "zero_pack8": (ctypes.c_int, [vp, i64, ctypes.c_int, i64, i64, vp, vp]),
        "zero_unpack8": (ctypes.c_int, [vp, i64, i64, vp, i64, ctypes.c_int, vp]),
        "zero_rms_norm": (ctypes.c_int, [vp, vp]),
        "zero_rms_norm_grad": (ctypes.c_int, [vp, vp]),
        "zero_rms_grad_ws_bytes": (i64, [i64, i64]),
        "zero_gated": (ctypes.c_int, [vp, vp]),
        "zero_gated_grad": (ctypes.c_int, [vp, vp]),
        "zero_gated_input_grad": (ctypes.c_int, [vp, vp]),
        "zero_gated_weight_grad": (ctypes.c_int, [vp, vp]),
        "zero_gated_ws_bytes": (i64, [i64, i64, i64]),
        "zero_last_error": (ctypes.c_char_p, []),
        "zero_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        if not required and not hasattr(L, name):
            continue
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def _check(rc: int) -> None:
    if rc != ZERO_OK:
        raise ZeroError(rc, lib().zero_last_error().decode())


def zero_last_error() -> str:
    return lib().zero_last_error().decode()


def zero_version() -> str:
    return lib().zero_version().decode()


# ---------------------------------------------------------------------------
# planner
# ---------------------------------------------------------------------------

class Plan:
    """Owner of a zero_plan_t handle."""

    def __init__(self, numels, world: int, bucket_cap: int = 0, *, _handle=None):
        L = lib()
        if _handle is None:
            arr = (ctypes.c_int64 * len(numels))(*[int(n) for n in numels])
            h = ctypes.c_void_p()
            _check(L.zero_plan(arr, len(numels), int(world), int(bucket_cap), ctypes.byref(h)))
            _handle = h
        self._h = _handle
        self.world = int(world)

    @classmethod
    def dim0(cls, shapes, world: int) -> "Plan":
        """Per-parameter dim-0 layout (zero_plan_dim0) of parameters of the given shapes."""
        rows, row_numel = [], []
        for sh in shapes:
            sh = tuple(int(x) for x in sh)
            rows.append(sh[0] if sh else 1)
            k = 1
            for x in sh[1:]:
                k *= x
            row_numel.append(k)
        n = len(rows)
        h = ctypes.c_void_p()
        _check(lib().zero_plan_dim0((ctypes.c_int64 * n)(*rows), (ctypes.c_int64 * n)(*row_numel), n,
                                    int(world), ctypes.byref(h)))
        return cls(None, world, _handle=h)

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise ValueError("plan already freed")
        return self._h

    def free(self) -> None:
        if getattr(self, "_h", None) is not None:
            lib().zero_plan_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    @property
    def shard_numel(self) -> int:
        return lib().zero_plan_shard_numel(self.handle)

    @property
    def total_numel(self) -> int:
        return lib().zero_plan_total_numel(self.handle)

    @property
    def padded_numel(self) -> int:
        return lib().zero_plan_padded_numel(self.handle)

    @property
    def num_buckets(self) -> int:
        return lib().zero_plan_num_buckets(self.handle)

    @property
    def num_tensors(self) -> int:
        return lib().zero_plan_num_tensors(self.handle)

    def bucket(self, b: int) -> Tuple[int, int, int, int, int, int]:
        """(base, numel, padded, shard, first_tensor, n_tensors)"""
        o = [ctypes.c_int64() for _ in range(4)] + [ctypes.c_int32() for _ in range(2)]
        _check(lib().zero_plan_bucket(self.handle, b, *[ctypes.byref(x) for x in o]))
        return tuple(x.value for x in o)

    def tensor(self, i: int) -> Tuple[int, int]:
        """(bucket, flat offset)"""
        b, off = ctypes.c_int32(), ctypes.c_int64()
        _check(lib().zero_plan_tensor(self.handle, i, ctypes.byref(b), ctypes.byref(off)))
        return b.value, off.value

    def rank_segment(self, rank: int, b: int) -> Tuple[int, int, int]:
        """(gather_off, local_off, valid)"""
        o = [ctypes.c_int64() for _ in range(3)]
        _check(lib().zero_plan_rank_segment(self.handle, rank, b, *[ctypes.byref(x) for x in o]))
        return tuple(x.value for x in o)

    def segments(self, rank: int) -> List[Tuple[int, int, int, int]]:
        """(gather_off, local_off, seg_len, valid) per bucket."""
        out = []
        for b in range(self.num_buckets):
            go, lo, valid = self.rank_segment(rank, b)
            out.append((go, lo, self.bucket(b)[3], valid))
        return out

    def tensor_offsets(self) -> List[int]:
        return [self.tensor(i)[1] for i in range(self.num_tensors)]

    def bytes(self, stage: int) -> Tuple[float, int]:
        f, p = ctypes.c_double(), ctypes.c_int64()
        _check(lib().zero_plan_bytes(self.handle, stage, ctypes.byref(f), ctypes.byref(p)))
        return f.value, p.value

    def piece_table_bytes(self) -> int:
        """Device bytes of one rank's piece table (16 per piece)."""
        return lib().zero_plan_piece_table_bytes(self.handle)

    def attach_piece_table(self, rank: int, table: int, nbytes: int) -> None:
        """Write rank's piece table into device memory `table` and attach it
        (one launch per step for any number of pieces); table=0 detaches."""
        _check(lib().zero_plan_attach_piece_table(self.handle, int(rank), table or None, int(nbytes)))

    def workspace_bytes(self) -> int:
        return lib().zero_workspace_bytes(self.handle)

    def state_numel(self, layout: int) -> int:
        n = lib().zero_state_numel(self.handle, layout)
        if n < 0:
            raise ZeroError(ZERO_EINVAL, "unknown state layout")
        return n


# ---------------------------------------------------------------------------
# device operations
# ---------------------------------------------------------------------------

def zero_reduce_shard(plan: Plan, grad: int, grad_ld: int, grad_dtype: int, inv_scale: float,
                      g_out: int, ws: int, want_sumsq: bool, stream: int = 0,
                      grad_count: int = 0, grad_layout: int = ZERO_GRAD_SHARD, rank: int = 0,
                      ctl: int = 0) -> None:
    """grad_count: gradient buffers summed (0 = N, one per rank; 1 = a stored
    reduce-scatter output, or with grad_layout ZERO_GRAD_FULL one all-reduced
    full gradient read at `rank`'s pieces).  ctl: device address of a
    zero_step_ctl_t whose loss scale replaces inv_scale (0 = none)."""
    _check(lib().zero_reduce_shard(plan.handle, int(rank), grad, grad_ld, grad_count, grad_layout, grad_dtype,
                                   inv_scale, g_out or None, ws, 1 if want_sumsq else 0, ctl or None,
                                   stream or None))


def zero_shard_norm(plan: Plan, ws: int, other_ranks_sumsq: float, max_norm: float,
                    overflow_out: int, sumsq_out: int, clip_coef_out: int, stream: int = 0) -> None:
    _check(lib().zero_shard_norm(plan.handle, ws, other_ranks_sumsq, max_norm, overflow_out or None,
                                 sumsq_out or None, clip_coef_out or None, stream or None))


ZERO_NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def zero_noalloc_max_shard() -> int:
    return int(lib().zero_noalloc_max_shard())


def zero_reduce_norm_noalloc(plan: Plan, grad: int, grad_ld: int, grad_dtype: int, inv_scale: float,
                             g_out: int, other_ranks_sumsq: float, max_norm: float, overflow_out: int,
                             sumsq_out: int, clip_coef_out: int, stream: int = 0, grad_count: int = 0,
                             grad_layout: int = ZERO_GRAD_SHARD, rank: int = 0, ctl: int = 0) -> None:
    """zero_reduce_shard + zero_shard_norm with the library's fixed workspace
    (for callers that cannot allocate device memory)."""
    _check(lib().zero_reduce_norm_noalloc(plan.handle, int(rank), grad, grad_ld, grad_count, grad_layout,
                                          grad_dtype, inv_scale, g_out or None, other_ranks_sumsq, max_norm,
                                          overflow_out or None, sumsq_out or None, clip_coef_out or None,
                                          ctl or None, stream or None))


def zero_adam_step(plan: Plan, args: zero_adam_args_t, stream: int = 0) -> None:
    _check(lib().zero_adam_step(plan.handle, ctypes.byref(args), stream or None))


# ---------------------------------------------------------------------------
# loss scale and sharded checkpoints (host)
# ---------------------------------------------------------------------------

class Scaler:
    """Dynamic loss scale (zero_scaler_t): update() after every step with its
    overflow flag; inv_scale is what the step multiplies the gradient by."""

    def __init__(self, init_scale: float = 65536.0, growth_factor: float = 2.0,
                 backoff_factor: float = 0.5, growth_interval: int = 2000):
        self.s = zero_scaler_t()
        _check(lib().zero_scaler_init(ctypes.byref(self.s), init_scale, growth_factor, backoff_factor,
                                      int(growth_interval)))

    def update(self, overflow: bool) -> None:
        _check(lib().zero_scaler_update(ctypes.byref(self.s), 1 if overflow else 0))

    @property
    def scale(self) -> float:
        return self.s.scale

    @property
    def growth_tracker(self) -> int:
        return self.s.growth_tracker

    @property
    def inv_scale(self) -> float:
        return lib().zero_scaler_inv_scale(ctypes.byref(self.s))


def zero_plan_hash(plan: Plan) -> int:
    return lib().zero_plan_hash(plan.handle)


def zero_checkpoint_save(plan: Plan, rank: int, path: str, state_layout: int, master: int, m: int, v: int,
                         step: int, scaler: zero_scaler_t, stream: int = 0) -> None:
    meta = zero_ckpt_meta_t(step=int(step), scaler=scaler)
    _check(lib().zero_checkpoint_save(plan.handle, int(rank), os.fsencode(path), int(state_layout),
                                      master or None, m or None, v or None, ctypes.byref(meta),
                                      stream or None))


def zero_checkpoint_load(plan: Plan, rank: int, path: str, state_layout: int, master: int, m: int, v: int,
                         stream: int = 0) -> zero_ckpt_meta_t:
    """Returns the saved metadata (step and scaler)."""
    meta = zero_ckpt_meta_t()
    _check(lib().zero_checkpoint_load(plan.handle, int(rank), os.fsencode(path), int(state_layout),
                                      master or None, m or None, v or None, ctypes.byref(meta),
                                      stream or None))
    return meta


def zero_stream_copy(dst: int, src: int, nbytes: int, stream: int = 0) -> None:
    _check(lib().zero_stream_copy(dst, src, int(nbytes), stream or None))


# ---------------------------------------------------------------------------
# the model's input layer
# ---------------------------------------------------------------------------

def zero_dropout(x: int, ld_x: int, x_dtype: int, residual: int, ld_res: int, out: int, ld_out: int,
                 out_dtype: int, rows: int, cols: int, drop: "zero_drop_t | None", stream: int = 0) -> None:
    """residual 0: none; drop None: nothing is dropped."""
    _check(lib().zero_dropout(x or None, ld_x, x_dtype, residual or None, ld_res, out or None, ld_out, out_dtype,
                              rows, cols, ctypes.addressof(drop) if drop is not None else None, stream or None))


def zero_embed_lookup(args: zero_embed_args_t, stream: int = 0) -> None:
    _check(lib().zero_embed_lookup(ctypes.addressof(args), stream or None))


def zero_embed_grad_ws_bytes(n_ids: int, rows: int, dim: int) -> int:
    """Workspace bytes of zero_embed_grad; 0 for sizes out of range."""
    return int(lib().zero_embed_grad_ws_bytes(n_ids, rows, dim))


def zero_embed_grad(args: zero_embed_grad_args_t, stream: int = 0) -> None:
    _check(lib().zero_embed_grad(ctypes.addressof(args), stream or None))


# ---------------------------------------------------------------------------
# the pre-norm gated feed-forward sub-layer
# ---------------------------------------------------------------------------

def zero_pack8(x: int, ld_x: int, x_dtype: int, rows: int, cols: int, held: zero_held_t, stream: int = 0) -> None:
    _check(lib().zero_pack8(x or None, ld_x, x_dtype, rows, cols, ctypes.addressof(held), stream or None))


def zero_unpack8(held: zero_held_t, rows: int, cols: int, out: int, ld_out: int, out_dtype: int,
                 stream: int = 0) -> None:
    _check(lib().zero_unpack8(ctypes.addressof(held), rows, cols, out or None, ld_out, out_dtype, stream or None))


def zero_rms_norm(args: zero_rms_args_t, stream: int = 0) -> None:
    _check(lib().zero_rms_norm(ctypes.addressof(args), stream or None))


def zero_rms_grad_ws_bytes(rows: int, cols: int) -> int:
    """Workspace bytes of zero_rms_norm_grad; 0 for sizes out of range."""
    return int(lib().zero_rms_grad_ws_bytes(rows, cols))


def zero_rms_norm_grad(args: zero_rms_grad_args_t, stream: int = 0) -> None:
    _check(lib().zero_rms_norm_grad(ctypes.addressof(args), stream or None))


def zero_gated_ws_bytes(tokens: int, dim: int, hidden: int) -> int:
    """Workspace bytes of the gated block's product calls; 0 for sizes out of range."""
    return int(lib().zero_gated_ws_bytes(tokens, dim, hidden))


def zero_gated(args: zero_gated_args_t, stream: int = 0) -> None:
    _check(lib().zero_gated(ctypes.addressof(args), stream or None))


def zero_gated_grad(args: zero_gated_args_t, stream: int = 0) -> None:
    _check(lib().zero_gated_grad(ctypes.addressof(args), stream or None))


def zero_gated_input_grad(args: zero_gated_args_t, stream: int = 0) -> None:
    _check(lib().zero_gated_input_grad(ctypes.addressof(args), stream or None))


def zero_gated_weight_grad(args: zero_gated_args_t, stream: int = 0) -> None:
    _check(lib().zero_gated_weight_grad(ctypes.addressof(args), stream or None))


def adam_args(**kw) -> zero_adam_args_t:
    """Build a zero_adam_args_t; unspecified pointers are NULL, inv_scale 1."""
    a = zero_adam_args_t()
    a.inv_scale = 1.0
    for k, v in kw.items():
        if not hasattr(a, k):
            raise TypeError(f"unknown field {k}")
        setattr(a, k, v)
    return a
