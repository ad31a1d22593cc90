"""GB300-native ZeRO-DP partitioned mixed-precision optimizer step.

A thin ctypes binding of ``libzero_gb300.so`` (C ABI in ``include/zero.h``):
the functions here have the C names and only marshal arguments -- every step
of the path runs in the library's CUDA kernels.  Pointers may be given as
torch tensors (their ``data_ptr()``) or as integers.  A nonzero status raises
``ZeroError`` with the library's message.

Importing this package loads the compiled library; if it has not been built
(``python zero_dp_partitioned_gb300/build.py``) the import fails -- there is
no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libzero_gb300.so")

ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_EWORKSPACE, ZERO_ECUDA, ZERO_ELIMIT = 0, -1, -2, -3, -4, -5
ZERO_F16, ZERO_BF16, ZERO_F32, ZERO_E4M3, ZERO_I32, ZERO_I64 = 1, 2, 3, 4, 5, 6
ZERO_MX4_ROWS, ZERO_MX4_TILES = 0, 1
ZERO_SILU, ZERO_GELU_TANH = 0, 1
ZERO_PLAN_PADDED, ZERO_PLAN_UNPADDED = 0, 1
ZERO_MAX_SLICES = ZERO_MAX_SHARDS = 64


class ZeroError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{msg} (status {code})")
        self.code = code


class zero_hyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("max_grad_norm", ctypes.c_float),
                ("step", ctypes.c_int64)]


class zero_shard(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("grad_offset", ctypes.c_int64), ("param_offset", ctypes.c_int64),
                ("master_in", ctypes.c_void_p), ("m_in", ctypes.c_void_p), ("v_in", ctypes.c_void_p),
                ("master_out", ctypes.c_void_p), ("m_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p),
                ("grad_shard", ctypes.c_void_p)]


class zero_stats(ctypes.Structure):
    _fields_ = [("sumsq", ctypes.c_double), ("overflow", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class zero_chain(ctypes.Structure):
    _fields_ = [("cur", ctypes.c_int32), ("reserved", ctypes.c_int32), ("step", ctypes.c_int64),
                ("loss_scale", ctypes.c_double), ("applied", ctypes.c_int64), ("skipped", ctypes.c_int64),
                ("failed", ctypes.c_int64), ("min_loss_scale", ctypes.c_double)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_ if not k.startswith("reserved")}


class zero_result(ctypes.Structure):
    _fields_ = [("overflow", ctypes.c_int32), ("applied", ctypes.c_int32), ("path", ctypes.c_int32),
                ("status", ctypes.c_int32), ("sumsq", ctypes.c_double), ("grad_norm", ctypes.c_double),
                ("clip_coef", ctypes.c_double), ("grad_mult", ctypes.c_float), ("reserved", ctypes.c_float)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_ if not k.startswith("reserved")}


class zero_mat(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]
    device = None                          # of the tensor that mat() was given, -1: not a GPU


class zero_mx4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64), ("layout", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]
    device = None                          # of the tensors that mx4() was given or made, -1: not a GPU

    @property
    def tensors(self):
        """The (data, scales) buffers that mx4() was given or made."""
        data, scales, n = self.buffers
        return (data, scales) if n is None else (data[:n], data[n:])


class zero_drop(ctypes.Structure):
    _fields_ = [("seed", ctypes.c_uint64), ("site", ctypes.c_uint32), ("p", ctypes.c_float), ("step", ctypes.c_int64),
                ("chain", ctypes.c_void_p)]
    device = None                          # of the chain's tensor, None: an address or none


assert ctypes.sizeof(zero_drop) == 32
assert ctypes.sizeof(zero_mat) == 24 and ctypes.sizeof(zero_mx4) == 48
assert ctypes.sizeof(zero_hyper) == 32 and ctypes.sizeof(zero_shard) == 80
assert ctypes.sizeof(zero_stats) == 16 and ctypes.sizeof(zero_result) == 48 and ctypes.sizeof(zero_chain) == 56

_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGS = {
    "zero_plan": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "zero_plan_intersections": (_I, [_P, _P, _I, _I64, _I64, _P]),
    "zero_mem_model": (_I, [ctypes.c_double, ctypes.c_double, _I, _I, _P]),
    "zero_mem_model_plan": (_I, [_I64, _I64, ctypes.c_double, _I, _I, _I64, _I64, _P]),
    "zero_comm_volume": (_I, [ctypes.c_double, _I, _I, _I, _P]),
    "zero_plan_round_robin": (_I, [_I, _I, _P]),
    "zero_workspace_bytes": (ctypes.c_size_t, []),
    "zero_shard_step": (_I, [_P, _I, _I, _P, _I, _P, _I, _P, ctypes.c_float, ctypes.c_double, _I, _P,
                             ctypes.c_size_t, _P, _P]),
    "zero_shard_init": (_I, [_P, _I, _P, _I, _P]),
    "zero_shard_reduce": (_I, [_P, _I, _I, _P, _I, _I, _P, _P, ctypes.c_size_t, _P]),
    "zero_shard_apply": (_I, [_P, _I, _I, _P, _I, _P, ctypes.c_float, _P, ctypes.c_double, _I, _P, ctypes.c_size_t,
                              _P, _P]),
    "zero3_gather_layer": (_I, [_P, _I, _I64, _I, _P, _P]),
    "zero3_gather_segments": (_I, [_P, _P, _I, _I, _P, _P]),
    "zero3_gather_bulk": (_I, [_P, _P, _I, _I, _P, _I, _P, _P]),
    "zero3_reduce_bucket": (_I, [_P, _I, _I, _I64, _I, _P, _I, _P, _P, ctypes.c_size_t, _P]),
    "zero_shard_step_noalloc": (_I, [_P, _I, _I, _P, _I, _P, _I, _P, ctypes.c_float, ctypes.c_double, _I, _P, _P]),
    "zero_adam_scalar_table": (_I, [_P, _I64, _I64, _P]),
    "zero_shard_step_chained": (_I, [_P, _I, _I, _P, _I, _P, _I, _P, _P, _I64, _I64, _P, ctypes.c_double, _I, _P,
                                     ctypes.c_size_t, _P, _P]),
    "zero_shard_apply_chained": (_I, [_P, _I, _I, _P, _I, _P, _P, _I64, _I64, _P, _P, ctypes.c_double, _I, _P,
                                      ctypes.c_size_t, _P, _P]),
    "zero_shard_step_partial": (_I, [_P, _I, _I, _P, _I, _P, _I, _P, ctypes.c_float, _P, _I64, _I64, _P, _I, _P, _P,
                                     ctypes.c_size_t, _P]),
    "zero_shard_step_commit": (_I, [_P, _I, _P, _I, ctypes.c_float, _I64, _I64, _P, _P, ctypes.c_double, _I, _P, _P]),
    "zero_shard_step_host": (_I, [_P, _I, _I, _P, _I, _P, _I, _P, _P, ctypes.c_float, ctypes.c_double, _I, _P,
                                  ctypes.c_size_t, _P, ctypes.c_size_t, _P, _P]),
    "zero_norm_forward": (_I, [_P, _P, _P, _I64, _I64, ctypes.c_float, _P, _P, _P, _I64, _P, _P]),
    "zero_norm_backward": (_I, [_P, _P, _P, _I64, _I64, _P, _P, _P, _P, _I, _P, ctypes.c_size_t, _P]),
    "zero_norm_workspace_bytes": (ctypes.c_size_t, [_I64]),
    "zero_distill_loss": (_I, [_P, _I64, _I64, _P, _P, _I, _P, ctypes.c_float, _P, ctypes.c_float, _P, _P, _P, _P,
                               _P]),
    "zero_distill_backward": (_I, [_P, _I64, _I64, _P, _P, _I, _P, ctypes.c_float, _P, ctypes.c_float, _P, _P, _P,
                                   _P]),
    "zero_mx4_bytes": (_I, [_I64, _I64, _I, _P, _P, _P]),
    "zero_mx4_quantize": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "zero_mx4_dequantize": (_I, [_P, _P, _P]),
    "zero_mx4_tile_scales": (_I, [_P, _P, _P]),
    "zero_mx4_matmul": (_I, [_P, _P, ctypes.c_float, _P, _P, _P]),
    "zero_dropout": (_I, [_P, _P, _I64, _I64, _P, _P, _P]),
    "zero_layernorm_forward": (_I, [_P, _P, _P, _P, _P, _I64, _I64, ctypes.c_float, _P, _P, _P, _P, _P]),
    "zero_layernorm_backward": (_I, [_P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, ctypes.c_size_t,
                                     _P]),
    "zero_layernorm_workspace_bytes": (ctypes.c_size_t, [_I64]),
    "zero_gated_forward": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]),
    "zero_gated_forward_workspace_bytes": (ctypes.c_size_t, [_P, _P, _P, _I64, _I64, _I64]),
    "zero_gated_backward": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _I, _P,
                                 ctypes.c_size_t, _P, _P]),
    "zero_gated_backward_workspace_bytes": (ctypes.c_size_t, [_P, _P, _P, _P, _P, _I64, _I64, _I64]),
    "zero_last_error": (ctypes.c_char_p, []),
}
# every symbol include/zero.h declares
EXPORTS = tuple(_SIGS)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python zero_dp_partitioned_gb300/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _ptr(x):
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _stream(stream):
    if stream is not None:
        return _ptr(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)
    return _current_stream()


_raw_stream = None
_gpus = 0                                  # of this process; 0: not known yet


def _current_stream():
    """torch's current stream on the current device (None without a GPU), by the
    calls under torch.cuda.current_stream(): its Stream object alone costs as
    much as a small kernel (2.8 us on the host that drives a GB300).  They are
    not public; a torch without them is asked by the public calls."""
    return _raw_stream[0](_raw_stream[1]()) if _raw_stream or _find_raw_stream() else None


def _current_device():
    """torch's current device (-1 without a GPU)."""
    return _raw_stream[1]() if _raw_stream or _find_raw_stream() else -1


def _find_raw_stream():
    global _raw_stream, _gpus
    if _raw_stream is None:
        import torch
        if not torch.cuda.is_available():
            return None
        torch.cuda.init()
        calls = tuple(getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if None in calls:
            calls = (lambda d: torch.cuda.current_stream(d).cuda_stream, torch.cuda.current_device)
        _raw_stream, _gpus = calls, torch.cuda.device_count()
    return _raw_stream


def _check(rc):
    if rc < 0:
        raise ZeroError(rc, lib.zero_last_error().decode())
    return rc


def _ptrs(xs):
    return (ctypes.c_void_p * max(1, len(xs)))(*[_ptr(x) for x in xs])


# ------------------------------------------------------------------ host-only calls
def zero_plan(numels, world_size, mode=ZERO_PLAN_PADDED):
    n = len(numels)
    arr = (ctypes.c_int64 * max(1, n))(*numels)
    t_off = (ctypes.c_int64 * max(1, n))()
    r_off = (ctypes.c_int64 * world_size)()
    r_num = (ctypes.c_int64 * world_size)()
    padded, pad = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.zero_plan(arr, n, world_size, mode, t_off, r_off, r_num, ctypes.byref(padded), ctypes.byref(pad)))
    return {"tensor_offsets": list(t_off)[:n], "rank_offsets": list(r_off), "rank_numels": list(r_num),
            "padded_total": padded.value, "padding": pad.value}


def zero_plan_intersections(tensor_offsets, numels, rank_offset, rank_numel):
    n = len(numels)
    t = (ctypes.c_int64 * max(1, n))(*tensor_offsets)
    m = (ctypes.c_int64 * max(1, n))(*numels)
    out = (ctypes.c_int64 * (4 * max(1, n)))()
    k = _check(lib.zero_plan_intersections(t, m, n, rank_offset, rank_numel, out))
    return [tuple(out[4 * i:4 * i + 4]) for i in range(k)]


def zero_mem_model(psi, K, n_d, stage):
    b = ctypes.c_double()
    _check(lib.zero_mem_model(psi, K, n_d, stage, ctypes.byref(b)))
    return b.value


def zero_mem_model_plan(flat_numel, shard_numel, K, stage, state_sets=1, fp32_temp_numel=0, b16_temp_numel=0):
    """Plan-exact bytes of one rank: dict of params, grads, states, temp, total."""
    out = (ctypes.c_double * 5)()
    _check(lib.zero_mem_model_plan(flat_numel, shard_numel, K, stage, state_sets, fp32_temp_numel, b16_temp_numel,
                                   out))
    return dict(zip(("params", "grads", "states", "temp", "total"), list(out)))


def zero_comm_volume(psi, n_d, stage, ring=False):
    v = ctypes.c_double()
    _check(lib.zero_comm_volume(psi, n_d, stage, int(ring), ctypes.byref(v)))
    return v.value


def zero_plan_round_robin(n_tensors, world_size):
    out = (ctypes.c_int64 * max(1, n_tensors))()
    _check(lib.zero_plan_round_robin(n_tensors, world_size, out))
    return list(out)[:n_tensors]


def zero_workspace_bytes():
    return lib.zero_workspace_bytes()


# ------------------------------------------------------------------ device calls
def shard(numel, grad_offset, param_offset, master_in, m_in, v_in, master_out=None, m_out=None, v_out=None,
          grad_shard=None) -> zero_shard:
    """A zero_shard; *_out default to *_in (in-place)."""
    return zero_shard(numel, grad_offset, param_offset, _ptr(master_in), _ptr(m_in), _ptr(v_in),
                      _ptr(master_out if master_out is not None else master_in),
                      _ptr(m_out if m_out is not None else m_in),
                      _ptr(v_out if v_out is not None else v_in), _ptr(grad_shard))


def hyper(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, max_grad_norm=0.0, step=1) -> zero_hyper:
    return zero_hyper(lr, beta1, beta2, eps, weight_decay, max_grad_norm, step)


def zero_shard_step(grad_slices, grad_dtype, shards, flat_param, param_dtype, hyper, loss_scale,
                    extra_sumsq, extra_overflow, workspace, workspace_bytes, result, stream=None):
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_step(_ptrs(grad_slices), len(grad_slices), grad_dtype, sh, len(shards), _ptr(flat_param),
                               param_dtype, ctypes.byref(hyper), loss_scale, extra_sumsq, int(extra_overflow),
                               _ptr(workspace), workspace_bytes, _ptr(result), _stream(stream)))


def zero_shard_step_host(host_grad_slices, grad_dtype, shards, flat_param, param_dtype, host_param, hyper,
                         loss_scale, extra_sumsq, extra_overflow, staging, staging_bytes, workspace, workspace_bytes,
                         result, stream=None):
    """zero_shard_step with the gradients in page-locked host memory and the
    updated parameters copied back to page-locked host memory (host_param,
    laid out as flat_param; None = no copy down): the library copies the
    slices up chunk by chunk into the device ring `staging` while the chunks
    already up are reduced and updated."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_step_host(_ptrs(host_grad_slices), len(host_grad_slices), grad_dtype, sh, len(shards),
                                    _ptr(flat_param), param_dtype, _ptr(host_param), ctypes.byref(hyper), loss_scale,
                                    extra_sumsq, int(extra_overflow), _ptr(staging), staging_bytes, _ptr(workspace),
                                    workspace_bytes, _ptr(result), _stream(stream)))


def zero_shard_step_noalloc(grad_slices, grad_dtype, shards, flat_param, param_dtype, hyper, loss_scale,
                            extra_sumsq, extra_overflow, result, stream=None):
    """zero_shard_step without caller scratch (for callers that cannot allocate
    device memory): the library's built-in scratch array stands in for the
    workspace and the two-pass path's reduced-gradient buffers."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_step_noalloc(_ptrs(grad_slices), len(grad_slices), grad_dtype, sh, len(shards),
                                       _ptr(flat_param), param_dtype, ctypes.byref(hyper), loss_scale, extra_sumsq,
                                       int(extra_overflow), _ptr(result), _stream(stream)))


def zero_shard_init(shards, flat_param, param_dtype, stream=None):
    """Before the first step: every shard's master_in = fp32(its 16-bit
    parameters in flat_param), m_in = v_in = 0."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_init(sh, len(shards), _ptr(flat_param), param_dtype, _stream(stream)))


def zero_shard_reduce(grad_slices, grad_dtype, shards, accumulate, stats, workspace, workspace_bytes, stream=None):
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_reduce(_ptrs(grad_slices), len(grad_slices), grad_dtype, sh, len(shards), int(accumulate),
                                 _ptr(stats), _ptr(workspace), workspace_bytes, _stream(stream)))


def zero_shard_apply(shards, grad_dtype, flat_param, param_dtype, hyper, loss_scale, stats, extra_sumsq,
                     extra_overflow, workspace, workspace_bytes, result, stream=None):
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_apply(sh, len(shards), grad_dtype, _ptr(flat_param), param_dtype, ctypes.byref(hyper),
                                loss_scale, _ptr(stats), extra_sumsq, int(extra_overflow), _ptr(workspace),
                                workspace_bytes, _ptr(result), _stream(stream)))


def zero3_gather_layer(part_ptrs, unit_numel, dtype, layer_out, stream=None):
    _check(lib.zero3_gather_layer(_ptrs(part_ptrs), len(part_ptrs), unit_numel, dtype, _ptr(layer_out),
                                  _stream(stream)))


def zero3_gather_segments(segment_ptrs, segment_numels, dtype, layer_out, stream=None):
    n = len(segment_ptrs)
    lens = (ctypes.c_int64 * max(1, n))(*segment_numels)
    _check(lib.zero3_gather_segments(_ptrs(segment_ptrs), lens, n, dtype, _ptr(layer_out), _stream(stream)))


def zero3_gather_bulk(segment_ptrs, segment_numels, dtype, layer_out, n_ctas, status, stream=None):
    """The gather on at most n_ctas CTAs (0 = one per SM), moved by the TMA unit
    when every segment agrees with its slot modulo 16 bytes; status: device
    int32 (zero-filled by the caller), bit 0 set if a wait ran out."""
    n = len(segment_ptrs)
    lens = (ctypes.c_int64 * max(1, n))(*segment_numels)
    _check(lib.zero3_gather_bulk(_ptrs(segment_ptrs), lens, n, dtype, _ptr(layer_out), int(n_ctas), _ptr(status),
                                 _stream(stream)))


def zero3_reduce_bucket(bucket_ptrs, owner, unit_numel, grad_dtype, grad_part, accumulate, stats, workspace,
                        workspace_bytes, stream=None):
    _check(lib.zero3_reduce_bucket(_ptrs(bucket_ptrs), len(bucket_ptrs), owner, unit_numel, grad_dtype,
                                   _ptr(grad_part), int(accumulate), _ptr(stats), _ptr(workspace), workspace_bytes,
                                   _stream(stream)))


def zero_adam_scalar_table(hyper, t0, n):
    """The step-dependent AdamW scalars (lr / (1 - b1^t), 1 / sqrt(1 - b2^t)) for
    t = t0 .. t0 + n - 1, as a host float32 array of 2 n values."""
    import numpy as np
    out = np.zeros(2 * int(n), np.float32)
    _check(lib.zero_adam_scalar_table(ctypes.byref(hyper), int(t0), int(n), out.ctypes.data))
    return out


def chain(step=1, loss_scale=1.0, cur=0, min_loss_scale=0.0):
    """A zero_chain to copy to the device (56 bytes) as the start of a chain;
    min_loss_scale <= 0 leaves the library's floor of 2^-126."""
    return zero_chain(cur, 0, step, loss_scale, 0, 0, 0, min_loss_scale)


def read_chain(t) -> zero_chain:
    """A zero_chain from a 56-byte tensor (device or host)."""
    b = bytes(t.detach().cpu().view(-1).numpy().tobytes()) if hasattr(t, "detach") else bytes(t)
    return zero_chain.from_buffer_copy(b[:ctypes.sizeof(zero_chain)])


def zero_shard_step_chained(grad_slices, grad_dtype, shards, flat_param, param_dtype, hyper, scalar_table, table_t0,
                            n_table, chain_dev, extra_sumsq, extra_overflow, workspace, workspace_bytes, result,
                            stream=None):
    """One step with its bookkeeping (t, S, the state set in use) in the device
    zero_chain chain_dev; scalar_table: device float32, 2 n_table values."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_step_chained(_ptrs(grad_slices), len(grad_slices), grad_dtype, sh, len(shards),
                                       _ptr(flat_param), param_dtype, ctypes.byref(hyper), _ptr(scalar_table),
                                       int(table_t0), int(n_table), _ptr(chain_dev), extra_sumsq,
                                       int(extra_overflow), _ptr(workspace), workspace_bytes, _ptr(result),
                                       _stream(stream)))


def zero_shard_apply_chained(shards, grad_dtype, flat_param, param_dtype, hyper, scalar_table, table_t0, n_table,
                             chain_dev, stats, extra_sumsq, extra_overflow, workspace, workspace_bytes, result,
                             stream=None):
    """The apply pass with t, S and the state set in use read from the device
    zero_chain chain_dev, which it then updates; shards may update in place."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_apply_chained(sh, len(shards), grad_dtype, _ptr(flat_param), param_dtype,
                                        ctypes.byref(hyper), _ptr(scalar_table), int(table_t0), int(n_table),
                                        _ptr(chain_dev), _ptr(stats), extra_sumsq, int(extra_overflow),
                                        _ptr(workspace), workspace_bytes, _ptr(result), _stream(stream)))


def zero_shard_step_partial(grad_slices, grad_dtype, shards, flat_param, param_dtype, hyper, loss_scale, accumulate,
                            stats, workspace, workspace_bytes, scalar_table=None, table_t0=1, n_table=0,
                            chain_dev=None, stream=None):
    """A fused pass over some shards of a step, adding their statistics to
    stats; the step is decided later by zero_shard_step_commit.  With
    chain_dev, t, S and the state set in use come from the device chain."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_step_partial(_ptrs(grad_slices), len(grad_slices), grad_dtype, sh, len(shards),
                                       _ptr(flat_param), param_dtype, ctypes.byref(hyper), loss_scale,
                                       _ptr(scalar_table), int(table_t0), int(n_table), _ptr(chain_dev),
                                       int(accumulate), _ptr(stats), _ptr(workspace), workspace_bytes,
                                       _stream(stream)))


def zero_shard_step_commit(shards, flat_param, param_dtype, loss_scale, stats, extra_sumsq, extra_overflow, result,
                           table_t0=1, n_table=0, chain_dev=None, stream=None):
    """The decision of a step made of partial fused passes: the result from
    their statistics, the parameters restored on a skip, the chain updated."""
    sh = (zero_shard * max(1, len(shards)))(*shards)
    _check(lib.zero_shard_step_commit(sh, len(shards), _ptr(flat_param), param_dtype, loss_scale, int(table_t0),
                                      int(n_table), _ptr(chain_dev), _ptr(stats), extra_sumsq, int(extra_overflow),
                                      _ptr(result), _stream(stream)))


def read_result(t) -> zero_result:
    """A zero_result from a 48-byte tensor (device or host)."""
    b = bytes(t.detach().cpu().view(-1).numpy().tobytes()) if hasattr(t, "detach") else bytes(t)
    return zero_result.from_buffer_copy(b[:ctypes.sizeof(zero_result)])


def read_stats(t) -> zero_stats:
    b = bytes(t.detach().cpu().view(-1).numpy().tobytes())
    return zero_stats.from_buffer_copy(b[:ctypes.sizeof(zero_stats)])


# ------------------------------------------------------------------ layer operators
# Most calls of a layer take a few microseconds on the GPU, so the arguments
# are marshalled with few Python operations: a tensor's zero_mat is packed as
# bytes, whose address ctypes passes.
_MAT_DTYPES = {"torch.float16": ZERO_F16, "torch.bfloat16": ZERO_BF16, "torch.float32": ZERO_F32,
               "torch.float8_e4m3fn": ZERO_E4M3, "torch.int32": ZERO_I32, "torch.int64": ZERO_I64}
_codes = {}                                # torch dtype -> zero_dtype, filled as they are met
_pack_mat = struct.Struct("=Qqii").pack


def _code(dtype):
    code = _MAT_DTYPES.get(str(dtype))
    if code is None:
        raise ZeroError(ZERO_EINVAL, f"no zero_mat of {dtype}")
    _codes[dtype] = code
    return code


def mat(data, ld=None, dtype=None) -> zero_mat:
    """A zero_mat of a torch tensor (two dimensions with adjacent columns, or
    one: a single row), or of an address with its row distance and dtype."""
    if not hasattr(data, "data_ptr"):
        return zero_mat(_ptr(data), ld or 0, dtype or 0, 0)
    code = _code(data.dtype)
    if data.dim() not in (1, 2) or (data.shape[-1] > 1 and data.stride(-1) != 1):
        raise ZeroError(ZERO_EINVAL, "a zero_mat has one or two dimensions and adjacent columns")
    m = zero_mat(data.data_ptr(), data.stride(0) if data.dim() == 2 else data.shape[0], code, 0)
    m.tensor = data                        # kept alive with the argument
    m.device = data.get_device()
    return m


def _elsewhere(device, what):
    raise ZeroError(ZERO_EINVAL, f"{what} is not on a GPU" if device < 0 else
                    f"{what} is on GPU {device}, not on the current one")


def _mat(x, rows, cols, what):
    """A matrix argument: None, a zero_mat, or a tensor of exactly rows x cols
    (of one dimension: a single row) with adjacent columns."""
    if x is None:
        return None
    if isinstance(x, zero_mat):
        if x.device is not None and (x.device < 0 or x.device != _current_device()):
            _elsewhere(x.device, what)
        return ctypes.byref(x)
    code = _codes.get(x.dtype) or _code(x.dtype)
    shape, step = x.shape, x.stride()
    if len(shape) == 1:
        shape, step = (1, shape[0]), (shape[0], step[0])
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ZeroError(ZERO_EINVAL, f"{what} is {tuple(x.shape)}, not {rows} x {cols}")
    if step[1] != 1 and cols > 1:
        raise ZeroError(ZERO_EINVAL, f"{what}: its columns are not adjacent")
    if not x.is_cuda or (_gpus != 1 and x.get_device() != _current_device()):
        _elsewhere(x.get_device(), what)
    return _pack_mat(x.data_ptr(), step[0], code, 0)


def _vec(x, n, what):
    """An array argument: None, an address, or a tensor of at least n contiguous
    fp32 values."""
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if x.numel() < n or (_codes.get(x.dtype) or _code(x.dtype)) != ZERO_F32 or not x.is_contiguous():
            raise ZeroError(ZERO_EINVAL, f"{what} must be {n} contiguous float32 values")
        if not x.is_cuda or (_gpus != 1 and x.get_device() != _current_device()):
            _elsewhere(x.get_device(), what)
        return x.data_ptr()
    return int(x)


def _buf(x, n, what, code=ZERO_EINVAL):
    """A buffer argument: None, an address, or a tensor of at least n contiguous
    bytes."""
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if x.numel() * x.element_size() < n or not x.is_contiguous():
            raise ZeroError(code, f"{what} must be at least {n} contiguous bytes")
        if not x.is_cuda or (_gpus != 1 and x.get_device() != _current_device()):
            _elsewhere(x.get_device(), what)
        return x.data_ptr()
    return int(x)


def zero_norm_forward(x, residual, weight, rows, cols, eps, h_out, y, y_scale, scale_block, rstd, stream=None):
    """h = x + residual, y = RMSnorm(h) * weight per row; y in x's type, or
    float8_e4m3fn with a scale per row (scale_block 0) or per 128 columns."""
    n = rows * (-(-cols // scale_block) if scale_block > 0 else 1)
    _check(lib.zero_norm_forward(_mat(x, rows, cols, "x"), _mat(residual, rows, cols, "residual"),
                                 _mat(weight, 1, cols, "weight"), rows, cols, eps, _mat(h_out, rows, cols, "h_out"),
                                 _mat(y, rows, cols, "y"), _vec(y_scale, n, "y_scale"), scale_block,
                                 _vec(rstd, rows, "rstd"), _stream(stream)))


def zero_norm_workspace_bytes(cols):
    return lib.zero_norm_workspace_bytes(cols)


def zero_norm_backward(dy, h, weight, rows, cols, rstd, dh, dx, dw, accumulate, workspace, workspace_bytes,
                       stream=None):
    """dx (of x and residual alike) and dw of zero_norm_forward."""
    _check(lib.zero_norm_backward(_mat(dy, rows, cols, "dy"), _mat(h, rows, cols, "h"),
                                  _mat(weight, 1, cols, "weight"), rows, cols, _vec(rstd, rows, "rstd"),
                                  _mat(dh, rows, cols, "dh"), _mat(dx, rows, cols, "dx"), _mat(dw, 1, cols, "dw"),
                                  int(accumulate), _buf(workspace, workspace_bytes, "workspace", ZERO_EWORKSPACE),
                                  workspace_bytes, _stream(stream)))


def zero_distill_loss(logits, rows, cols, ids, teacher, k, teacher_lse, temperature, row_weight, grad_scale, chain_dev,
                      loss, lse, dlogits, stream=None):
    """The rows' losses against the teacher's k logits and, with dlogits, the
    gradient, scaled by grad_scale and by the loss scale of the device chain."""
    _check(lib.zero_distill_loss(_mat(logits, rows, cols, "logits"), rows, cols, _mat(ids, rows, k, "ids"),
                                 _mat(teacher, rows, k, "teacher"), k, _vec(teacher_lse, rows, "teacher_lse"),
                                 temperature, _vec(row_weight, rows, "row_weight"), grad_scale,
                                 _buf(chain_dev, ctypes.sizeof(zero_chain), "chain_dev"),
                                 _vec(loss, rows, "loss"), _vec(lse, rows, "lse"),
                                 _mat(dlogits, rows, cols, "dlogits"), _stream(stream)))


def zero_distill_backward(logits, rows, cols, ids, teacher, k, teacher_lse, temperature, row_weight, grad_scale,
                          chain_dev, lse, dlogits, stream=None):
    """The gradient alone, from the lse that zero_distill_loss stored."""
    _check(lib.zero_distill_backward(_mat(logits, rows, cols, "logits"), rows, cols, _mat(ids, rows, k, "ids"),
                                     _mat(teacher, rows, k, "teacher"), k, _vec(teacher_lse, rows, "teacher_lse"),
                                     temperature, _vec(row_weight, rows, "row_weight"), grad_scale,
                                     _buf(chain_dev, ctypes.sizeof(zero_chain), "chain_dev"),
                                     _vec(lse, rows, "lse"), _mat(dlogits, rows, cols, "dlogits"), _stream(stream)))


@functools.lru_cache(maxsize=1024)
def zero_mx4_bytes(rows, cols, layout=ZERO_MX4_TILES):
    """(ld, data bytes, scale bytes) of a 4-bit matrix."""
    ld, data, scales = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib.zero_mx4_bytes(rows, cols, layout, ctypes.byref(ld), ctypes.byref(data), ctypes.byref(scales)))
    return ld.value, data.value, scales.value


def mx4(rows, cols, data=None, scales=None, layout=ZERO_MX4_TILES, device=None) -> zero_mx4:
    """A zero_mx4 over given buffers (torch uint8 tensors or addresses), or over
    new ones on `device` (None: the current GPU); rows follow one another
    without gaps."""
    ld, n_data, n_scales = zero_mx4_bytes(rows, cols, layout)
    if data is None and scales is None:
        import torch
        buf = torch.empty(n_data + n_scales, dtype=torch.uint8, device="cuda" if device is None else device)
        at = buf.data_ptr()
        m = zero_mx4(at, at + n_data, rows, cols, ld, layout, 0)
        m.buffers = (buf, None, n_data)    # kept alive with the argument
        m.device = buf.get_device()
        return m
    if data is None or scales is None:
        raise ZeroError(ZERO_EINVAL, "data and scales: both or neither")
    for t, n, what in ((data, n_data, "data"), (scales, n_scales, "scales")):
        if hasattr(t, "data_ptr") and (t.numel() * t.element_size() < n or not t.is_contiguous()):
            raise ZeroError(ZERO_EINVAL, f"{what} must be at least {n} contiguous bytes")
    m = zero_mx4(_ptr(data), _ptr(scales), rows, cols, ld, layout, 0)
    m.buffers = (data, scales, None)
    on = {t.get_device() for t in (data, scales) if hasattr(t, "data_ptr")}
    if len(on) == 2 and min(on) >= 0:
        raise ZeroError(ZERO_EINVAL, "data and scales are on two GPUs")
    m.device = min(on) if on else None
    return m


def _mx4(x, what):
    if x is None:
        return None
    if x.device is not None and (x.device < 0 or (_gpus != 1 and x.device != _current_device())):
        _elsewhere(x.device, what)
    return ctypes.byref(x)


def zero_mx4_quantize(src, rows, cols, out, out_t, stream=None):
    """src to 4 bits along its rows (out) and along its columns (out_t: cols x
    rows); either may be None."""
    _check(lib.zero_mx4_quantize(_mat(src, rows, cols, "src"), rows, cols, _mx4(out, "out"), _mx4(out_t, "out_t"),
                                 _stream(stream)))


def zero_mx4_dequantize(src, dst, stream=None):
    """The values of a 4-bit matrix in dst's type."""
    d = None if src is None else _mat(dst, src.rows, src.cols, "dst")
    _check(lib.zero_mx4_dequantize(_mx4(src, "src"), d, _stream(stream)))


def zero_mx4_tile_scales(src, dst, stream=None):
    """Scales gathered row by row (ZERO_MX4_ROWS) to the product's tiles."""
    _check(lib.zero_mx4_tile_scales(_mx4(src, "src"), _mx4(dst, "dst"), _stream(stream)))


def zero_mx4_matmul(a, b, alpha, d, status, stream=None):
    """d = alpha a b^T of two 4-bit matrices; status: device int32 (zero-filled by
    the caller), bit 0 set if a wait ran out."""
    m = None if a is None or b is None else _mat(d, a.rows, b.rows, "d")
    _check(lib.zero_mx4_matmul(_mx4(a, "a"), _mx4(b, "b"), alpha, m, _buf(status, 4, "status"), _stream(stream)))


def drop(p, seed, site=0, step=0, chain_dev=None) -> zero_drop:
    """A dropout: the probability of dropping, the run's 64-bit seed, the place in
    the model, and the step, or the device zero_chain whose step is taken when
    the kernel runs.  A chain's step moves once an applied step: micro-batches
    that add to one step's gradients need sites (or seeds) of their own, or they
    drop the same elements."""
    d = zero_drop(int(seed) & 0xFFFFFFFFFFFFFFFF, int(site) & 0xFFFFFFFF, p, int(step),
                  _buf(chain_dev, ctypes.sizeof(zero_chain), "chain_dev"))
    if hasattr(chain_dev, "data_ptr"):
        d.tensor = chain_dev               # kept alive with the argument
        d.device = chain_dev.get_device()
    return d


def _drop(d):
    if d is None:
        return None
    if d.device is not None and _gpus != 1 and d.device != _current_device():
        _elsewhere(d.device, "drop's chain")
    return ctypes.byref(d)


def zero_dropout(x, residual, rows, cols, drop, y, stream=None):
    """y = dropout(x) + residual; the gradient of x is the same call on dy."""
    _check(lib.zero_dropout(_mat(x, rows, cols, "x"), _mat(residual, rows, cols, "residual"), rows, cols, _drop(drop),
                            _mat(y, rows, cols, "y"), _stream(stream)))


def zero_layernorm_forward(x, residual, drop, weight, bias, rows, cols, eps, h_out, y, mean, rstd, stream=None):
    """h = dropout(x) + residual, y = layernorm(h) * weight + bias per row."""
    _check(lib.zero_layernorm_forward(_mat(x, rows, cols, "x"), _mat(residual, rows, cols, "residual"), _drop(drop),
                                      _mat(weight, 1, cols, "weight"), _mat(bias, 1, cols, "bias"), rows, cols, eps,
                                      _mat(h_out, rows, cols, "h_out"), _mat(y, rows, cols, "y"),
                                      _vec(mean, rows, "mean"), _vec(rstd, rows, "rstd"), _stream(stream)))


def zero_layernorm_workspace_bytes(cols):
    return lib.zero_layernorm_workspace_bytes(cols)


def zero_layernorm_backward(dy, h, weight, rows, cols, mean, rstd, dh, drop, dr, dx, dw, db, accumulate, workspace,
                            workspace_bytes, stream=None):
    """dr (of the residual), dx (of x, behind the dropout), dw and db of
    zero_layernorm_forward."""
    _check(lib.zero_layernorm_backward(_mat(dy, rows, cols, "dy"), _mat(h, rows, cols, "h"),
                                       _mat(weight, 1, cols, "weight"), rows, cols, _vec(mean, rows, "mean"),
                                       _vec(rstd, rows, "rstd"), _mat(dh, rows, cols, "dh"), _drop(drop),
                                       _mat(dr, rows, cols, "dr"), _mat(dx, rows, cols, "dx"), _mat(dw, 1, cols, "dw"),
                                       _mat(db, 1, cols, "db"), int(accumulate),
                                       _buf(workspace, workspace_bytes, "workspace", ZERO_EWORKSPACE),
                                       workspace_bytes, _stream(stream)))


def zero_gated_forward_workspace_bytes(x, gate_w, up_w, rows, cols, ff):
    """0 for few rows, and where the rows of x and of the weights start on 16-byte
    boundaries."""
    return lib.zero_gated_forward_workspace_bytes(_mat(x, rows, cols, "x"), _mat(gate_w, ff, cols, "gate_w"),
                                                  _mat(up_w, ff, cols, "up_w"), rows, cols, ff)


def zero_gated_forward(x, gate_w, up_w, rows, cols, ff, act, h, gate, up, workspace, workspace_bytes, status,
                       stream=None):
    """h = act(x gate_w^T) * (x up_w^T), and, with gate and up, both projections;
    status: device int32 (zero-filled by the caller), bit 0 set if a wait ran
    out."""
    _check(lib.zero_gated_forward(_mat(x, rows, cols, "x"), _mat(gate_w, ff, cols, "gate_w"),
                                  _mat(up_w, ff, cols, "up_w"), rows, cols, ff, act, _mat(h, rows, ff, "h"),
                                  _mat(gate, rows, ff, "gate"), _mat(up, rows, ff, "up"),
                                  _buf(workspace, workspace_bytes, "workspace", ZERO_EWORKSPACE), workspace_bytes,
                                  _buf(status, 4, "status"), _stream(stream)))


def zero_gated_backward_workspace_bytes(x, gate_w, up_w, dgate, dup, rows, cols, ff):
    """Room for copies of those whose rows do not start on 16-byte boundaries, and
    for the parts of dx's sum where few rows and columns leave most of the GPU
    idle."""
    return lib.zero_gated_backward_workspace_bytes(_mat(x, rows, cols, "x"), _mat(gate_w, ff, cols, "gate_w"),
                                                   _mat(up_w, ff, cols, "up_w"), _mat(dgate, rows, ff, "dgate"),
                                                   _mat(dup, rows, ff, "dup"), rows, cols, ff)


def zero_gated_backward(dh, gate, up, x, gate_w, up_w, rows, cols, ff, act, dgate, dup, dx, dgate_w, dup_w, accumulate,
                        workspace, workspace_bytes, status, stream=None):
    """dgate and dup (the projections' gradients, stored), and of them dx and the
    weights' gradients."""
    _check(lib.zero_gated_backward(_mat(dh, rows, ff, "dh"), _mat(gate, rows, ff, "gate"), _mat(up, rows, ff, "up"),
                                   _mat(x, rows, cols, "x"), _mat(gate_w, ff, cols, "gate_w"),
                                   _mat(up_w, ff, cols, "up_w"), rows, cols, ff, act, _mat(dgate, rows, ff, "dgate"),
                                   _mat(dup, rows, ff, "dup"), _mat(dx, rows, cols, "dx"),
                                   _mat(dgate_w, ff, cols, "dgate_w"), _mat(dup_w, ff, cols, "dup_w"), int(accumulate),
                                   _buf(workspace, workspace_bytes, "workspace", ZERO_EWORKSPACE), workspace_bytes,
                                   _buf(status, 4, "status"), _stream(stream)))
