"""Python binding of libtp (the C ABI declared in include/tp.h).

Argument marshalling only: every function has the C entry point's name and argument order, accepts
torch tensors (or raw integer addresses) where the C side takes device pointers, lists of them where
it takes a host array of shard pointers, and an optional ``stream`` (default: torch's current
stream). A non-OK status raises ``TPError``. All work runs in the library's CUDA kernels; there is no
fallback path: importing this package fails if libtp.so has not been built.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtp.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python tensor_sharded_matmul_b200/build.py` "
                      "(or __graft_entry__.build()); there is no fallback implementation")

_lib = C.CDLL(LIB_PATH)

# ---- enums (values of include/tp.h) ----------------------------------------------------------
TP_OK, TP_EINVAL, TP_ESHAPE, TP_EDIVIS, TP_EALIGN, TP_ECUDA, TP_ETIMEOUT, TP_EUNSUPPORTED, TP_ENOSPACE = range(9)
TP_F32, TP_BF16, TP_BF16_RING = 0, 1, 2
TP_ACT_NONE, TP_ACT_GELU, TP_ACT_GELU_TANH, TP_ACT_SWIGLU = 0, 1, 2, 3
TP_OUT_PARTIALS, TP_OUT_RS, TP_OUT_AR, TP_OUT_RS_AG = 0, 1, 2, 3
TP_CASE1_LOCAL = 0
TP_CASE2_ALLGATHER, TP_CASE2_ALLREDUCE = 0, 1
TP_CASE3_ALLREDUCE, TP_CASE3_RS_B, TP_CASE3_RS_F = 0, 1, 2
TP_CASE4_GATHER_X, TP_CASE4_GATHER_W = 0, 1
TP_MAX_SHARDS = 16
TP_GATE_SOFTMAX, TP_GATE_TOPK = 0, 1
TP_MAX_EXPERTS, TP_MAX_TOPK = 1024, 16

EXPORTED = (
    "tp_status_str", "tp_last_error", "tp_device_status", "tp_set_wait_budget", "tp_selftest_wait_timeout",
    "tp_num_sms", "tp_shard_cols", "tp_shard_rows", "tp_shard_gate_up", "tp_shard_qkv", "tp_reduce_scatter",
    "tp_all_gather", "tp_all_reduce", "tp_grouped_gemm", "tp_column_linear", "tp_row_linear", "tp_row_linear_reduce", "tp_mlp_fwd",
    "tp_sharded_matmul_ws_bytes", "tp_sharded_matmul_choose", "tp_sharded_matmul", "tp_layer_fwd", "tp_mlp_fwd_noalloc",
    "tp_column_linear_sp", "tp_mlp_fwd_sp", "tp_all_to_all", "tp_grouped_gemm_t", "tp_mlp_bwd",
    "tp_moe_route_ws_bytes", "tp_moe_route", "tp_moe_route_bwd", "tp_ragged_linear", "tp_ragged_linear_dx",
    "tp_ragged_linear_dw", "tp_moe_combine", "tp_moe_combine_bwd", "tp_moe_mlp_ws_bytes", "tp_moe_mlp_fwd",
    "tp_moe_mlp_bwd", "tp_lora_plan_ws_bytes", "tp_lora_plan", "tp_lora_ws_bytes", "tp_lora_linear",
)

_vp, _i64, _i32, _u64, _sz = C.c_void_p, C.c_int64, C.c_int, C.c_uint64, C.c_size_t
_pp = C.POINTER(C.c_void_p)

_SIGS = {
    "tp_status_str": (C.c_char_p, [_i32]),
    "tp_last_error": (C.c_char_p, []),
    "tp_device_status": (_i32, [_i32, C.POINTER(C.c_uint32)]),
    "tp_set_wait_budget": (None, [_u64]),
    "tp_selftest_wait_timeout": (_i32, [_u64, _vp]),
    "tp_num_sms": (_i32, []),
    "tp_shard_cols": (_i32, [_vp, _i64, _i64, _i64, _i32, _vp, _vp]),
    "tp_shard_rows": (_i32, [_vp, _i64, _i64, _i64, _i32, _vp, _vp]),
    "tp_shard_gate_up": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _vp]),
    "tp_shard_qkv": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _vp]),
    "tp_reduce_scatter": (_i32, [_pp, _pp, _i64, _i64, _i32, _i32, _i32, _vp]),
    "tp_all_gather": (_i32, [_pp, _pp, _i64, _i64, _i32, _i32, _i32, _vp]),
    "tp_all_reduce": (_i32, [_pp, _pp, _i64, _i64, _i32, _i32, _vp]),
    "tp_all_to_all": (_i32, [_pp, _pp, _i64, _i64, _i32, _i32, _i32, _i32, _vp]),
    "tp_grouped_gemm": (_i32, [_i32, _pp, _pp, _pp, _i64, _i64, _i64, _i32, _i32, _vp]),
    "tp_grouped_gemm_t": (_i32, [_i32, _pp, _i32, _pp, _i32, _pp, _i64, _i64, _i64, _i32, _vp]),
    "tp_mlp_bwd": (_i32, [_vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _pp, _vp]),
    "tp_column_linear": (_i32, [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp]),
    "tp_row_linear": (_i32, [_vp, _i64, _i64, _i64, _i32, _vp, _pp, _vp]),
    "tp_row_linear_reduce": (_i32, [_vp, _i64, _i64, _i64, _i32, _vp, _i32, _i32, _pp, _pp, _vp]),
    "tp_mlp_fwd": (_i32, [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _pp, _i32, _pp, _vp]),
    "tp_mlp_fwd_noalloc": (_i32, [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _i32, _pp, _vp]),
    "tp_column_linear_sp": (_i32, [_pp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp]),
    "tp_mlp_fwd_sp": (_i32, [_pp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _pp, _vp]),
    "tp_sharded_matmul_ws_bytes": (_sz, [_i32, _i32, _i64, _i64, _i64, _i32]),
    "tp_sharded_matmul_choose": (_i32, [_i32, _i64, _i64, _i64, _i32, C.POINTER(C.c_int)]),
    "tp_sharded_matmul": (_i32, [_i32, _i32, _pp, _pp, _i64, _i64, _i64, _i32, _pp, _i32, _vp, _sz, _vp]),
    "tp_layer_fwd": (_i32, [_vp, _pp, _i64, _i64, _i32, _i32, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _pp,
                            _vp, _vp, _pp, _pp, _vp]),
    "tp_moe_route_ws_bytes": (_sz, [_i64, _i32, _i32]),
    "tp_moe_route": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "tp_moe_route_bwd": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "tp_ragged_linear": (_i32, [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _i64, _i32, _vp, _vp, _i32, _vp, _vp]),
    "tp_ragged_linear_dx": (_i32, [_vp, _vp, _i64, _i32, _i64, _i64, _vp, _i32, _vp, _vp, _vp]),
    "tp_ragged_linear_dw": (_i32, [_vp, _i64, _vp, _vp, _vp, _i64, _i32, _i64, _i64, _vp, _i32, _vp]),
    "tp_moe_combine": (_i32, [_vp, _i32, _i64, _vp, _vp, _i64, _i64, _i32, _vp, _i32, _vp]),
    "tp_moe_combine_bwd": (_i32, [_vp, _i32, _vp, _i32, _i64, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "tp_moe_mlp_ws_bytes": (_sz, [_i64, _i32, _i32]),
    "tp_moe_mlp_fwd": (_i32, [_vp, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _i32] + [_vp] * 11 + [_i32, _vp, _sz, _vp]),
    "tp_moe_mlp_bwd": (_i32, [_vp, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _i32] + [_vp] * 16 + [_i32, _vp, _vp]),
    "tp_lora_plan_ws_bytes": (_sz, [_i64, _i32]),
    "tp_lora_plan": (_i32, [_vp, _i64, _i32, _vp, _vp, _vp, _sz, _vp]),
    "tp_lora_ws_bytes": (_sz, [_i64, _i32]),
    "tp_lora_linear": (_i32, [_vp, _i64, _i64, _i64, _i32, _vp, _i32, _i32] + [_vp] * 7 + [_sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class TPError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.tp_status_str(status).decode()
        detail = _lib.tp_last_error().decode()
        super().__init__(f"{where}: {msg} ({detail})" if detail else f"{where}: {msg}")


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _ptrs(xs):
    if xs is None:
        return None
    arr = (C.c_void_p * len(xs))(*[_ptr(x) for x in xs])
    return C.cast(arr, _pp)


_raw_stream = None


def _current_stream():
    """torch's current stream of the current device as an address (None without a GPU). torch's raw getter spares
    the stream object that current_stream() builds: 0.4 against 3.9 us a call."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        if not torch.cuda.is_available():
            return None
        torch.cuda.init()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and device is not None:
            _raw_stream = lambda: raw(device())                            # noqa: E731
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, *args):
    st = getattr(_lib, name)(*args)
    if st != TP_OK:
        raise TPError(st, name)


# ---- status -----------------------------------------------------------------------------------
def tp_status_str(status: int) -> str:
    return _lib.tp_status_str(status).decode()


def tp_last_error() -> str:
    return _lib.tp_last_error().decode()


def tp_device_status(clear: int = 1):
    """Returns (status, site) after synchronising; does not raise."""
    where = C.c_uint32(0)
    st = _lib.tp_device_status(clear, C.byref(where))
    return st, where.value


def tp_set_wait_budget(cycles: int) -> None:
    _lib.tp_set_wait_budget(cycles)


def tp_selftest_wait_timeout(budget_cycles: int, stream=None) -> None:
    _call("tp_selftest_wait_timeout", budget_cycles, _stream(stream))


def tp_num_sms() -> int:
    return _lib.tp_num_sms()


# ---- layouts ----------------------------------------------------------------------------------
def tp_shard_cols(w, ld, K, N, t, out, stream=None):
    _call("tp_shard_cols", _ptr(w), ld, K, N, t, _ptr(out), _stream(stream))


def tp_shard_rows(w, ld, K, N, t, out, stream=None):
    _call("tp_shard_rows", _ptr(w), ld, K, N, t, _ptr(out), _stream(stream))


def tp_shard_gate_up(w_gate, ld_g, w_up, ld_u, h, F, t, out, stream=None):
    _call("tp_shard_gate_up", _ptr(w_gate), ld_g, _ptr(w_up), ld_u, h, F, t, _ptr(out), _stream(stream))


def tp_shard_qkv(w_q, ld_q, w_k, ld_k, w_v, ld_v, h, n_h, n_kv, d_h, t, out, stream=None):
    _call("tp_shard_qkv", _ptr(w_q), ld_q, _ptr(w_k), ld_k, _ptr(w_v), ld_v, h, n_h, n_kv, d_h, t, _ptr(out),
          _stream(stream))


# ---- collectives ------------------------------------------------------------------------------
def tp_reduce_scatter(ins, outs, rows, cols, axis, dtype, t, stream=None):
    _call("tp_reduce_scatter", _ptrs(ins), _ptrs(outs), rows, cols, axis, dtype, t, _stream(stream))


def tp_all_gather(ins, outs, rows, cols, axis, dtype, t, stream=None):
    _call("tp_all_gather", _ptrs(ins), _ptrs(outs), rows, cols, axis, dtype, t, _stream(stream))


def tp_all_reduce(ins, outs, rows, cols, dtype, t, stream=None):
    _call("tp_all_reduce", _ptrs(ins), _ptrs(outs), rows, cols, dtype, t, _stream(stream))


def tp_all_to_all(ins, outs, rows, cols, split_axis, concat_axis, dtype, t, stream=None):
    _call("tp_all_to_all", _ptrs(ins), _ptrs(outs), rows, cols, split_axis, concat_axis, dtype, t, _stream(stream))


# ---- GEMMs, MLP, cases, layer -----------------------------------------------------------------
def tp_grouped_gemm(groups, a, b, c, M, N, K, act, c_dtype, stream=None):
    _call("tp_grouped_gemm", groups, _ptrs(a), _ptrs(b), _ptrs(c), M, N, K, act, c_dtype, _stream(stream))


def tp_grouped_gemm_t(groups, a, trans_a, b, trans_b, c, M, N, K, c_dtype, stream=None):
    _call("tp_grouped_gemm_t", groups, _ptrs(a), trans_a, _ptrs(b), trans_b, _ptrs(c), M, N, K, c_dtype,
          _stream(stream))


def tp_mlp_bwd(x, dy, N, h, F, t, act, w_in, w_down, h_pre, z, dz_ws, dh_ws, dw_in, dw_down, dx, stream=None):
    _call("tp_mlp_bwd", _ptr(x), _ptr(dy), N, h, F, t, act, _ptr(w_in), _ptr(w_down), _ptr(h_pre), _ptr(z),
          _ptr(dz_ws), _ptr(dh_ws), _ptr(dw_in), _ptr(dw_down), _ptrs(dx), _stream(stream))


def tp_column_linear(x, N, k, n, t, act, w, y, stream=None):
    _call("tp_column_linear", _ptr(x), N, k, n, t, act, _ptr(w), _ptr(y), _stream(stream))


def tp_row_linear(x, N, k, n, t, w, partials, stream=None):
    _call("tp_row_linear", _ptr(x), N, k, n, t, _ptr(w), _ptrs(partials), _stream(stream))


def tp_row_linear_reduce(x, N, k, n, t, w, mode, axis, out, partials=None, stream=None):
    _call("tp_row_linear_reduce", _ptr(x), N, k, n, t, _ptr(w), mode, axis, _ptrs(out), _ptrs(partials),
          _stream(stream))


def tp_mlp_fwd(x, N, h, F, t, act, w_in, w_down, z_ws, partials, mode, out, stream=None):
    _call("tp_mlp_fwd", _ptr(x), N, h, F, t, act, _ptr(w_in), _ptr(w_down), _ptr(z_ws), _ptrs(partials), mode,
          _ptrs(out), _stream(stream))


def tp_mlp_fwd_noalloc(x, N, h, F, t, act, w_in, w_down, mode, out, stream=None):
    """tp_mlp_fwd for callers that cannot allocate device memory: the scratch is a fixed array inside
    the library (TP_MLP_NOALLOC_SCRATCH_BYTES); see include/tp.h for its limits and sharing rules."""
    _call("tp_mlp_fwd_noalloc", _ptr(x), N, h, F, t, act, _ptr(w_in), _ptr(w_down), mode, _ptrs(out),
          _stream(stream))


TP_MLP_NOALLOC_SCRATCH_BYTES = 32 << 20


def tp_column_linear_sp(x, N, k, n, t, act, w, y, stream=None):
    _call("tp_column_linear_sp", _ptrs(x), N, k, n, t, act, _ptr(w), _ptr(y), _stream(stream))


def tp_mlp_fwd_sp(x, N, h, F, t, act, w_in, w_down, z_ws, out, stream=None):
    _call("tp_mlp_fwd_sp", _ptrs(x), N, h, F, t, act, _ptr(w_in), _ptr(w_down), _ptr(z_ws), _ptrs(out),
          _stream(stream))


def tp_sharded_matmul_ws_bytes(case_id, strategy, B, D, F, t) -> int:
    return int(_lib.tp_sharded_matmul_ws_bytes(case_id, strategy, B, D, F, t))


def tp_sharded_matmul_choose(case_id, B, D, F, t) -> int:
    """The strategy the pages' cost rule picks for case 1, 2 or 4 (see include/tp.h)."""
    out = C.c_int(-1)
    _call("tp_sharded_matmul_choose", case_id, B, D, F, t, C.byref(out))
    return out.value


def tp_sharded_matmul(case_id, strategy, x, w, B, D, F, t, c, c_dtype, ws, ws_bytes, stream=None):
    _call("tp_sharded_matmul", case_id, strategy, _ptrs(x), _ptrs(w), B, D, F, t, _ptrs(c), c_dtype, _ptr(ws),
          ws_bytes, _stream(stream))


def tp_layer_fwd(x, o, N, h, n_h, n_kv, d_h, F, t, w_qkv, w_o, w_gu, w_down, qkv_out, h1, h1_bf16, z_ws, partials,
                 y, stream=None):
    _call("tp_layer_fwd", _ptr(x), _ptrs(o), N, h, n_h, n_kv, d_h, F, t, _ptr(w_qkv), _ptr(w_o), _ptr(w_gu),
          _ptr(w_down), _ptr(qkv_out), _ptrs(h1), _ptr(h1_bf16), _ptr(z_ws), _ptrs(partials), _ptrs(y),
          _stream(stream))


# ---- mixture-of-experts MLP and adapters --------------------------------------------------------
def tp_moe_route_ws_bytes(N, E, k) -> int:
    return int(_lib.tp_moe_route_ws_bytes(N, E, k))


def tp_moe_route(logits, dtype, N, E, k, gate, expert, weight, slot, offsets, row_token, ws, ws_bytes, stream=None):
    _call("tp_moe_route", _ptr(logits), dtype, N, E, k, gate, _ptr(expert), _ptr(weight), _ptr(slot), _ptr(offsets),
          _ptr(row_token), _ptr(ws), ws_bytes, _stream(stream))


def tp_moe_route_bwd(logits, dtype, N, E, k, gate, expert, dweight, dlogits, stream=None):
    _call("tp_moe_route_bwd", _ptr(logits), dtype, N, E, k, gate, _ptr(expert), _ptr(dweight), _ptr(dlogits),
          _stream(stream))


def tp_ragged_linear(x, x_rows, row_index, offsets, R, E, k, n, act, w, y, y_dtype, pre=None, stream=None):
    _call("tp_ragged_linear", _ptr(x), x_rows, _ptr(row_index), _ptr(offsets), R, E, k, n, act, _ptr(w), _ptr(y), y_dtype,
          _ptr(pre), _stream(stream))


def tp_ragged_linear_dx(dy, offsets, R, E, k, n, w, act, h_pre, dx, stream=None):
    _call("tp_ragged_linear_dx", _ptr(dy), _ptr(offsets), R, E, k, n, _ptr(w), act, _ptr(h_pre), _ptr(dx), _stream(stream))


def tp_ragged_linear_dw(x, x_rows, row_index, dy, offsets, R, E, k, n, dw, dw_dtype, stream=None):
    _call("tp_ragged_linear_dw", _ptr(x), x_rows, _ptr(row_index), _ptr(dy), _ptr(offsets), R, E, k, n, _ptr(dw), dw_dtype,
          _stream(stream))


def tp_moe_combine(u, u_dtype, R, weight, slot, N, h, k, y, y_dtype, stream=None):
    _call("tp_moe_combine", _ptr(u), u_dtype, R, _ptr(weight), _ptr(slot), N, h, k, _ptr(y), y_dtype, _stream(stream))


def tp_moe_combine_bwd(dy, dy_dtype, u, u_dtype, R, weight, slot, N, h, k, du, dweight, stream=None):
    _call("tp_moe_combine_bwd", _ptr(dy), dy_dtype, _ptr(u), u_dtype, R, _ptr(weight), _ptr(slot), N, h, k, _ptr(du),
          _ptr(dweight), _stream(stream))


def tp_moe_mlp_ws_bytes(N, E, k) -> int:
    return int(_lib.tp_moe_mlp_ws_bytes(N, E, k))


def tp_moe_mlp_fwd(x, N, h, F, E, k, gate, act, logits, logits_dtype, w_in, w_down, expert, weight, slot, offsets,
                   row_token, h_pre, z, u, y, y_dtype, ws, ws_bytes, stream=None):
    _call("tp_moe_mlp_fwd", _ptr(x), N, h, F, E, k, gate, act, _ptr(logits), logits_dtype, _ptr(w_in), _ptr(w_down),
          _ptr(expert), _ptr(weight), _ptr(slot), _ptr(offsets), _ptr(row_token), _ptr(h_pre), _ptr(z), _ptr(u), _ptr(y),
          y_dtype, _ptr(ws), ws_bytes, _stream(stream))


def tp_moe_mlp_bwd(x, dy, N, h, F, E, k, gate, act, logits, logits_dtype, w_in, w_down, expert, weight, slot, offsets,
                   row_token, h_pre, z, u, du_ws, dh_ws, dweight_ws, dw_in, dw_down, dx, dx_dtype, dlogits, stream=None):
    _call("tp_moe_mlp_bwd", _ptr(x), _ptr(dy), N, h, F, E, k, gate, act, _ptr(logits), logits_dtype, _ptr(w_in),
          _ptr(w_down), _ptr(expert), _ptr(weight), _ptr(slot), _ptr(offsets), _ptr(row_token), _ptr(h_pre), _ptr(z),
          _ptr(u), _ptr(du_ws), _ptr(dh_ws), _ptr(dweight_ws), _ptr(dw_in), _ptr(dw_down), _ptr(dx), dx_dtype,
          _ptr(dlogits), _stream(stream))


def tp_lora_plan_ws_bytes(N, L) -> int:
    return int(_lib.tp_lora_plan_ws_bytes(N, L))


def tp_lora_plan(id, N, L, offsets, row_token, ws, ws_bytes, stream=None):
    _call("tp_lora_plan", _ptr(id), N, L, _ptr(offsets), _ptr(row_token), _ptr(ws), ws_bytes, _stream(stream))


def tp_lora_ws_bytes(N, rank) -> int:
    return int(_lib.tp_lora_ws_bytes(N, rank))


def tp_lora_linear(x, N, k, n, t, w, L, rank, a, b, scale, offsets, row_token, y, ws, ws_bytes, stream=None):
    _call("tp_lora_linear", _ptr(x), N, k, n, t, _ptr(w), L, rank, _ptr(a), _ptr(b), _ptr(scale), _ptr(offsets),
          _ptr(row_token), _ptr(y), _ptr(ws), ws_bytes, _stream(stream))
