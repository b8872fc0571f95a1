"""ctypes binding of libhstu.so (include/hstu.h), argument marshalling only.

Every function has the name of the C entry point it calls and takes torch
tensors (for device memory) or plain integers.  PyTorch supplies device
memory and the current CUDA stream; every step of the computation runs in
the library's CUDA kernels.  If libhstu.so is missing the first call raises
``HstuError``: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Dict, List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhstu.so")

HSTU_BF16, HSTU_FP32, HSTU_FP16 = 0, 1, 2
STATUS_NAMES = {0: "HSTU_OK", 1: "HSTU_ERR_INVALID_ARG", 2: "HSTU_ERR_UNSUPPORTED",
                3: "HSTU_ERR_WORKSPACE", 4: "HSTU_ERR_CUDA", 5: "HSTU_ERR_BAD_OFFSETS",
                6: "HSTU_ERR_TIMEOUT", 7: "HSTU_ERR_BAD_TIMESTAMPS", 8: "HSTU_ERR_BAD_IDS"}

# Every symbol include/hstu.h declares.
EXPORTED = ["hstu_workspace_size", "hstu_layer_fwd", "hstu_stack_fwd", "hstu_mfalcon_rank",
            "hstu_bwd_workspace_size", "hstu_layer_bwd", "hstu_stack_bwd",
            "hstu_layer_fwd_noalloc", "hstu_sl_embed_workspace_size", "hstu_sl_embed",
            "hstu_sl_embed_ids", "hstu_embed_workspace_size", "hstu_embed_fwd",
            "hstu_embed_bwd_workspace_size", "hstu_embed_bwd", "hstu_embed_bwd_rows",
            "hstu_grad_norm_workspace_size", "hstu_grad_norm", "hstu_grad_norm_after",
            "hstu_adamw_workspace_size", "hstu_adamw_step",
            "hstu_sl_keep_count", "hstu_bf16_to_f16", "hstu_retrieval_workspace_size",
            "hstu_retrieval_topk", "hstu_retrieval_fallback_taken",
            "hstu_transformer_workspace_size",
            "hstu_transformer_layer_fwd",
            "hstu_read_status", "hstu_debug_offsets", "hstu_debug_keep_z",
            "hstu_debug_wait_test",
            "hstu_trace_enable", "hstu_trace_only", "hstu_trace_read",
            "hstu_kernel_name", "hstu_launch_count", "hstu_last_error", "hstu_set_option",
            "hstu_status_string",
            "hstu_version"]


class HstuError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.code, self.code)}")


class LayerDesc(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("n_pos_buckets", ctypes.c_int32), ("n_time_buckets", ctypes.c_int32),
                ("pos_sub_bits", ctypes.c_int32), ("time_sub_bits", ctypes.c_int32),
                ("ln_eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("W1", ctypes.c_void_p), ("b1", ctypes.c_void_p), ("W2", ctypes.c_void_p),
                ("b2", ctypes.c_void_p), ("ln_gamma", ctypes.c_void_p),
                ("ln_beta", ctypes.c_void_p), ("rab_pos", ctypes.c_void_p),
                ("rab_time", ctypes.c_void_p), ("W1_f16", ctypes.c_void_p),
                ("W2_f16", ctypes.c_void_p)]


GRAD_KEYS = ("dW1", "db1", "dW2", "db2", "dln_gamma", "dln_beta", "drab_pos", "drab_time")


class LayerGrads(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in GRAD_KEYS]


class TransformerWeights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("ln1_gamma", "ln1_beta", "W_qkv", "W_o", "ln2_gamma",
                                               "ln2_beta", "W_1", "b_1", "W_2", "b_2")]


class AdamWTensor(ctypes.Structure):
    """hstu_adamw_tensor."""
    _fields_ = [("n", ctypes.c_int64), ("row_len", ctypes.c_int64), ("max_rows", ctypes.c_int64),
                ("row_ids", ctypes.c_void_p), ("n_rows", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("param", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("copy_f16", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("weight_decay", ctypes.c_double),
                ("grad_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("state_bits", ctypes.c_int32)]


class AdamWArgs(ctypes.Structure):
    """hstu_adamw_args."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p),
                ("seed", ctypes.c_uint64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libhstu.so (built in-tree by ``build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise HstuError(4, f"libhstu.so not found at {LIB_PATH}; build it with "
                           "`python -m hstu_sequential_transducer_layer_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, sz, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    pdesc = ctypes.POINTER(LayerDesc)
    pw = ctypes.POINTER(LayerWeights)
    L.hstu_workspace_size.argtypes = [pdesc, i32, i64, i64, i64, i64, i64, i32]
    L.hstu_workspace_size.restype = sz
    L.hstu_layer_fwd.argtypes = [pdesc, i64, i64, i64, vp, vp, pw, vp, vp, vp, sz, vp]
    L.hstu_layer_fwd.restype = i32
    L.hstu_stack_fwd.argtypes = [pdesc, i32, pw, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp]
    L.hstu_stack_fwd.restype = i32
    L.hstu_mfalcon_rank.argtypes = [pdesc, i32, pw, i64, i64, i64, vp, vp, vp, i64, i64, vp, vp,
                                    vp, i32, vp, vp, vp, sz, vp]
    L.hstu_mfalcon_rank.restype = i32
    pg = ctypes.POINTER(LayerGrads)
    L.hstu_bwd_workspace_size.argtypes = [pdesc, i32, i64, i64, i64]
    L.hstu_bwd_workspace_size.restype = sz
    L.hstu_layer_bwd.argtypes = [pdesc, pw, i64, i64, i64, vp, vp, vp, vp, vp, pg, vp, sz, vp]
    L.hstu_layer_bwd.restype = i32
    L.hstu_stack_bwd.argtypes = [pdesc, i32, pw, i64, i64, i64, vp, vp, vp, vp, vp, pg, vp, sz, vp]
    L.hstu_stack_bwd.restype = i32
    L.hstu_layer_fwd_noalloc.argtypes = [pdesc, i64, i64, i64, vp, vp, pw, vp, vp, vp]
    L.hstu_layer_fwd_noalloc.restype = i32
    L.hstu_sl_embed_workspace_size.argtypes = []
    L.hstu_sl_embed_workspace_size.restype = sz
    L.hstu_sl_keep_count.argtypes = [i64]
    L.hstu_sl_keep_count.restype = i64
    L.hstu_bf16_to_f16.argtypes = [vp, vp, i64, vp]
    L.hstu_bf16_to_f16.restype = i32
    L.hstu_retrieval_workspace_size.argtypes = [i64, i64, i32, i32, i32]
    L.hstu_retrieval_workspace_size.restype = sz
    L.hstu_retrieval_topk.argtypes = [i64, i64, i32, vp, vp, i64, vp, i32, vp, vp, vp, sz, vp]
    L.hstu_retrieval_topk.restype = i32
    L.hstu_retrieval_fallback_taken.argtypes = [vp, sz, ctypes.POINTER(ctypes.c_int32), vp]
    L.hstu_retrieval_fallback_taken.restype = i32
    L.hstu_transformer_workspace_size.argtypes = [i32, i32, i32, i64, i64]
    L.hstu_transformer_workspace_size.restype = sz
    L.hstu_transformer_layer_fwd.argtypes = [i32, i32, i32, ctypes.c_float,
                                             ctypes.POINTER(TransformerWeights), i64, i64, i64, vp,
                                             vp, vp, vp, sz, vp]
    L.hstu_transformer_layer_fwd.restype = i32
    L.hstu_sl_embed.argtypes = [i64, i64, i64, vp, vp, vp, ctypes.c_uint64, vp, i64, vp, i64, i32,
                                vp, vp, vp, vp, sz, vp]
    L.hstu_sl_embed.restype = i32
    L.hstu_sl_embed_ids.argtypes = [i64, i64, i64, vp, vp, vp, ctypes.c_uint64, vp, i64, vp, i64,
                                    i32, vp, vp, vp, vp, vp, sz, vp]
    L.hstu_sl_embed_ids.restype = i32
    f32, pt = ctypes.c_float, ctypes.POINTER(AdamWTensor)
    for name in ("hstu_embed_workspace_size", "hstu_grad_norm_workspace_size",
                 "hstu_adamw_workspace_size"):
        getattr(L, name).argtypes = []
        getattr(L, name).restype = sz
    L.hstu_embed_fwd.argtypes = [i64, vp, vp, i32, i64, i32, i64, i64, f32, vp, i32, i64, vp, sz,
                                 vp]
    L.hstu_embed_fwd.restype = i32
    L.hstu_embed_bwd_workspace_size.argtypes = [i64, i64, i32]
    L.hstu_embed_bwd_workspace_size.restype = sz
    L.hstu_embed_bwd.argtypes = [i64, vp, vp, i32, i64, i64, i32, i64, f32, i32, vp, i32, i64, vp,
                                 sz, vp]
    L.hstu_embed_bwd.restype = i32
    L.hstu_embed_bwd_rows.argtypes = [i64, vp, vp, i32, i64, i64, i32, i64, f32, vp, vp, i32, i64,
                                      vp, vp, sz, vp]
    L.hstu_embed_bwd_rows.restype = i32
    L.hstu_grad_norm.argtypes = [pt, i32, ctypes.c_double, vp, vp, sz, vp]
    L.hstu_grad_norm.restype = i32
    L.hstu_grad_norm_after.argtypes = [pt, i32, ctypes.c_double, vp, vp, vp, sz, vp]
    L.hstu_grad_norm_after.restype = i32
    L.hstu_adamw_step.argtypes = [vp, pt, i32, vp, sz, vp]  # hstu_adamw_args, packed or by address
    L.hstu_adamw_step.restype = i32
    L.hstu_read_status.argtypes = [vp, sz, vp]
    L.hstu_read_status.restype = i32
    L.hstu_debug_offsets.argtypes = [pdesc, i64, i64, i64, ctypes.POINTER(sz),
                                     ctypes.POINTER(sz), ctypes.POINTER(sz)]
    L.hstu_debug_offsets.restype = i32
    L.hstu_debug_keep_z.argtypes = [i32]
    L.hstu_debug_keep_z.restype = i32
    L.hstu_debug_wait_test.argtypes = [ctypes.c_uint32, i32]
    L.hstu_debug_wait_test.restype = i32
    L.hstu_trace_enable.argtypes = [i32]
    L.hstu_trace_enable.restype = i32
    L.hstu_trace_only.argtypes = [i32]
    L.hstu_trace_only.restype = i32
    L.hstu_trace_read.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_float), i32]
    L.hstu_trace_read.restype = i32
    L.hstu_kernel_name.argtypes = [i32]
    L.hstu_kernel_name.restype = ctypes.c_char_p
    L.hstu_launch_count.argtypes = []
    L.hstu_launch_count.restype = i64
    L.hstu_set_option.argtypes = [ctypes.c_char_p, i64]
    L.hstu_set_option.restype = i32
    L.hstu_last_error.argtypes = []
    L.hstu_last_error.restype = ctypes.c_char_p
    L.hstu_status_string.argtypes = [i32]
    L.hstu_status_string.restype = ctypes.c_char_p
    L.hstu_version.argtypes = []
    L.hstu_version.restype = i32
    _lib = L
    return L


# ---------------------------------------------------------------- marshalling
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _nbytes(t) -> int:
    return int(t.numel() * t.element_size())


def _check(code: int, where: str) -> None:
    if code != 0:
        if code == 4:  # HSTU_ERR_CUDA: name the failing runtime call
            where = f"{where} ({lib().hstu_last_error().decode()})"
        raise HstuError(code, where)


def make_desc(d_model, n_heads, d_qk, d_v, n_pos_buckets, n_time_buckets, pos_sub_bits,
              time_sub_bits, ln_eps=1e-6, dtype="bf16") -> LayerDesc:
    dt = HSTU_BF16 if dtype in ("bf16", HSTU_BF16) else HSTU_FP32
    return LayerDesc(d_model, n_heads, d_qk, d_v, n_pos_buckets, n_time_buckets, pos_sub_bits,
                     time_sub_bits, float(ln_eps), dt)


def weights_struct(w: Dict[str, object]) -> LayerWeights:
    """LayerWeights from a dict of device tensors (W1, b1, W2, b2, ln_gamma,
    ln_beta, rab_pos, rab_time)."""
    return LayerWeights(*[_ptr(w[k]) for k in ("W1", "b1", "W2", "b2", "ln_gamma", "ln_beta",
                                                "rab_pos", "rab_time")],
                        *[_ptr(w[k]) if w.get(k) is not None else None
                          for k in ("W1_f16", "W2_f16")])


def weights_array(ws: Sequence[Dict[str, object]]):
    arr = (LayerWeights * len(ws))()
    for i, w in enumerate(ws):
        arr[i] = weights_struct(w)
    return arr


def weights_to_device(weights: Sequence[Dict[str, np.ndarray]], dtype: str, device) -> List[Dict]:
    """Copy a list of per-layer numpy weight dicts to the device (dense
    weights in the layer dtype, rab tables fp32)."""
    import torch
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = []
    for w in weights:
        d = {}
        for k in ("W1", "b1", "W2", "b2", "ln_gamma", "ln_beta"):
            d[k] = torch.from_numpy(np.ascontiguousarray(w[k], np.float32)).to(device=device, dtype=tdt)
        for k in ("rab_pos", "rab_time"):
            d[k] = torch.from_numpy(np.ascontiguousarray(w[k], np.float32)).to(device)
        out.append(d)
    return out


# ---------------------------------------------------------------- entry points
def hstu_workspace_size(desc: LayerDesc, n_layers: int, B: int, total_tokens: int, max_len: int,
                        total_cands: int = 0, max_cands: int = 0, microbatch: int = 0) -> int:
    n = lib().hstu_workspace_size(ctypes.byref(desc), n_layers, B, total_tokens, max_len,
                                  total_cands, max_cands, microbatch)
    if n == 0:
        raise HstuError(1, "hstu_workspace_size")
    return int(n)


def hstu_layer_fwd(desc, B, total_tokens, max_len, offsets, X, weights, timestamps, out,
                   workspace, stream=None) -> None:
    ws = weights if isinstance(weights, LayerWeights) else weights_struct(weights)
    _check(lib().hstu_layer_fwd(ctypes.byref(desc), B, total_tokens, max_len, _ptr(offsets),
                                _ptr(X), ctypes.byref(ws), _ptr(timestamps), _ptr(out),
                                _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "hstu_layer_fwd")


NOALLOC_SCRATCH_BYTES = 64 << 20  # HSTU_NOALLOC_SCRATCH_BYTES


def hstu_layer_fwd_noalloc(desc, B, total_tokens, max_len, offsets, X, weights, timestamps, out,
                           stream=None) -> None:
    """One layer in the library's fixed device scratch (no workspace argument)."""
    ws = weights if isinstance(weights, LayerWeights) else weights_struct(weights)
    _check(lib().hstu_layer_fwd_noalloc(ctypes.byref(desc), B, total_tokens, max_len,
                                        _ptr(offsets), _ptr(X), ctypes.byref(ws),
                                        _ptr(timestamps), _ptr(out), _stream(stream)),
           "hstu_layer_fwd_noalloc")


def hstu_sl_embed_workspace_size() -> int:
    return int(lib().hstu_sl_embed_workspace_size())


def hstu_bf16_to_f16(src, dst, stream=None) -> None:
    """fp16 copy of a bf16 device tensor (same shape) through the library."""
    _check(lib().hstu_bf16_to_f16(_ptr(src), _ptr(dst), int(src.numel()), _stream(stream)),
           "hstu_bf16_to_f16")


def hstu_retrieval_workspace_size(n_users, n_items, d, K, from_rows=False) -> int:
    n = lib().hstu_retrieval_workspace_size(n_users, n_items, d, K, 1 if from_rows else 0)
    if n == 0:
        raise HstuError(1, "hstu_retrieval_workspace_size")
    return int(n)


def hstu_retrieval_topk(H, E, K, out_scores, out_ids, workspace, user_offsets=None,
                        n_users=None, stream=None) -> None:
    """Top-K catalog items per user (see include/hstu.h).  H: bf16 [n_users, d]
    user vectors, or with user_offsets the encoder output [rows, d]; E: bf16
    [n_items, d]."""
    U = int(n_users if n_users is not None else
            (user_offsets.numel() - 1 if user_offsets is not None else H.shape[0]))
    rows = int(H.shape[0]) if user_offsets is not None else 0
    _check(lib().hstu_retrieval_topk(U, int(E.shape[0]), int(E.shape[1]), _ptr(H),
                                     _ptr(user_offsets), rows, _ptr(E), int(K), _ptr(out_scores),
                                     _ptr(out_ids), _ptr(workspace), _nbytes(workspace),
                                     _stream(stream)),
           "hstu_retrieval_topk")


def hstu_retrieval_fallback_taken(workspace, stream=None) -> bool:
    v = ctypes.c_int32(0)
    _check(lib().hstu_retrieval_fallback_taken(_ptr(workspace), _nbytes(workspace),
                                               ctypes.byref(v), _stream(stream)),
           "hstu_retrieval_fallback_taken")
    return bool(v.value)


def hstu_transformer_workspace_size(d_model, n_heads, d_ff, B, total_tokens) -> int:
    n = lib().hstu_transformer_workspace_size(d_model, n_heads, d_ff, B, total_tokens)
    if n == 0:
        raise HstuError(1, "hstu_transformer_workspace_size")
    return int(n)


def hstu_transformer_layer_fwd(d_model, n_heads, d_ff, ln_eps, weights, B, total_tokens, max_len,
                               offsets, X, out, workspace, stream=None) -> None:
    """The softmax-Transformer comparator layer (see include/hstu.h); `weights`
    is a TransformerWeights struct or a dict of device tensors."""
    if not isinstance(weights, TransformerWeights):
        weights = TransformerWeights(*[_ptr(weights[k]) for k, _ in TransformerWeights._fields_])
    _check(lib().hstu_transformer_layer_fwd(d_model, n_heads, d_ff, float(ln_eps),
                                            ctypes.byref(weights), B, total_tokens, max_len,
                                            _ptr(offsets), _ptr(X), _ptr(out), _ptr(workspace),
                                            _nbytes(workspace), _stream(stream)),
           "hstu_transformer_layer_fwd")


def hstu_sl_keep_count(n: int) -> int:
    return int(lib().hstu_sl_keep_count(int(n)))


def hstu_sl_embed(B, raw_total, max_raw_len, raw_offsets, raw_ids, raw_timestamps, seed,
                  content_table, action_table, out_offsets, out_X, out_timestamps, workspace,
                  stream=None) -> None:
    """Stochastic Length + token embedding on the device (see include/hstu.h);
    the tables are bf16 [rows, d] device tensors."""
    _check(lib().hstu_sl_embed(B, raw_total, max_raw_len, _ptr(raw_offsets), _ptr(raw_ids),
                               _ptr(raw_timestamps), int(seed) & ((1 << 64) - 1),
                               _ptr(content_table), int(content_table.shape[0]),
                               _ptr(action_table), int(action_table.shape[0]),
                               int(content_table.shape[1]), _ptr(out_offsets), _ptr(out_X),
                               _ptr(out_timestamps), _ptr(workspace), _nbytes(workspace),
                               _stream(stream)),
           "hstu_sl_embed")


def hstu_sl_embed_ids(B, raw_total, max_raw_len, raw_offsets, raw_ids, raw_timestamps, seed,
                      content_table, action_table, out_offsets, out_X, out_timestamps, out_ids,
                      workspace, stream=None) -> None:
    """hstu_sl_embed that also writes each kept token's row in the two tables
    taken as one (see include/hstu.h)."""
    _check(lib().hstu_sl_embed_ids(B, raw_total, max_raw_len, _ptr(raw_offsets), _ptr(raw_ids),
                                   _ptr(raw_timestamps), int(seed) & ((1 << 64) - 1),
                                   _ptr(content_table), int(content_table.shape[0]),
                                   _ptr(action_table), int(action_table.shape[0]),
                                   int(content_table.shape[1]), _ptr(out_offsets), _ptr(out_X),
                                   _ptr(out_timestamps), _ptr(out_ids), _ptr(workspace),
                                   _nbytes(workspace), _stream(stream)),
           "hstu_sl_embed_ids")


# ------------------------------------------------------ embedding and optimizer
# Small calls are bound by this file's own time: what every one of them needs
# of torch is looked up once (_torch_names).
_DTYPES = _FP32 = _INT64 = _current_device = _current_raw_stream = None


def _torch_names() -> None:
    global _DTYPES, _FP32, _INT64, _current_device, _current_raw_stream
    import torch
    _FP32, _INT64, _current_device = torch.float32, torch.int64, torch.cuda.current_device
    # the stream's address without the stream object that torch.cuda.current_stream() builds
    # (4 us of a call that takes 8)
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _DTYPES = {torch.bfloat16: HSTU_BF16, torch.float32: HSTU_FP32, torch.float16: HSTU_FP16}


def _dtype(t, where: str) -> int:
    if _DTYPES is None:
        _torch_names()
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise HstuError(2, f"{where}: {t.dtype} tensor")
    return code


def _need(ok: bool, where: str, what: str) -> None:
    if not ok:
        raise HstuError(1, f"{where}: {what}")


def _here(where: str, *tensors) -> int:
    """The current CUDA device, which every tensor must be on (kernels are
    launched there)."""
    if _DTYPES is None:
        _torch_names()
    dev = _current_device() if tensors[0].is_cuda else -2
    for t in tensors:
        if t.get_device() != dev:
            raise HstuError(1, f"{where}: a tensor on {t.device}, not on the current CUDA device")
    return dev


def stream_handle(stream) -> int:
    """The integer handle of `stream` (None: the current one)."""
    if stream is not None:
        return _stream(stream)
    if _DTYPES is None:
        _torch_names()
    return _current_raw_stream(_current_device())


def _raw_stream(stream, dev: int) -> int:
    return _current_raw_stream(dev) if stream is None else _stream(stream)


def _rows(t, where: str, name: str) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    if t.is_contiguous() and t.dim() == 2:
        return t.shape[1]
    _need(t.dim() == 2 and (t.shape[1] == 1 or t.stride(1) == 1), where,
          f"{name}: rows of a matrix, contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(int(t.shape[1]), t.stride(0))


def _i64(t, where: str, name: str) -> None:
    if _DTYPES is None:
        _torch_names()
    if t.dtype != _INT64 or not t.is_contiguous():
        raise HstuError(1, f"{where}: {name}: a contiguous int64 tensor")


def hstu_embed_workspace_size() -> int:
    return int(lib().hstu_embed_workspace_size())


def hstu_embed_fwd(ids, table, out, workspace, scale: float = 1.0, pad_id: int = -1,
                   stream=None) -> None:
    """out[t] = scale * table[ids[t]] (see include/hstu.h).  ids: int64 [T];
    table [R, d] and out [T, d]: bf16, fp16 or fp32, rows contiguous."""
    w = "hstu_embed_fwd"
    dev = _here(w, ids, table, out, workspace)
    _i64(ids, w, "ids")
    ldt, ldo = _rows(table, w, "table"), _rows(out, w, "out")
    (R, d), T = table.shape, ids.numel()
    if tuple(out.shape) != (T, d):
        raise HstuError(1, f"{w}: out: [ids, table's columns]")
    code = lib().hstu_embed_fwd(T, ids.data_ptr(), table.data_ptr(), _dtype(table, w), R, d, ldt,
                                pad_id, scale, out.data_ptr(), _dtype(out, w), ldo,
                                workspace.data_ptr(), _nbytes(workspace), _raw_stream(stream, dev))
    if code != 0:
        _check(code, w)


def hstu_embed_bwd_workspace_size(n_tokens: int, n_rows: int, d: int) -> int:
    n = int(lib().hstu_embed_bwd_workspace_size(n_tokens, n_rows, d))
    if n == 0:
        raise HstuError(1, "hstu_embed_bwd_workspace_size")
    return n


def hstu_embed_bwd(ids, dY, dE, workspace, scale: float = 1.0, pad_id: int = -1,
                   accumulate: bool = False, stream=None) -> None:
    """dE[r] = scale * sum of dY[t] over the tokens of row r, every row of the
    table's gradient written, or added into it (see include/hstu.h)."""
    w = "hstu_embed_bwd"
    dev = _here(w, ids, dY, dE, workspace)
    _i64(ids, w, "ids")
    ldy, lde = _rows(dY, w, "dY"), _rows(dE, w, "dE")
    (R, d), T = dE.shape, ids.numel()
    if tuple(dY.shape) != (T, d):
        raise HstuError(1, f"{w}: dY: [ids, dE's columns]")
    code = lib().hstu_embed_bwd(T, ids.data_ptr(), dY.data_ptr(), _dtype(dY, w), ldy, R, d, pad_id,
                                scale, 1 if accumulate else 0, dE.data_ptr(), _dtype(dE, w), lde,
                                workspace.data_ptr(), _nbytes(workspace), _raw_stream(stream, dev))
    if code != 0:
        _check(code, w)


def hstu_embed_bwd_rows(ids, dY, n_rows: int, row_ids, rows, n_unique, workspace,
                        scale: float = 1.0, pad_id: int = -1, stream=None) -> None:
    """The touched rows of that gradient only: row_ids (int64, ascending), rows
    and their number n_unique (int64 [1]); row_ids and rows hold min(ids,
    n_rows) entries (see include/hstu.h)."""
    w = "hstu_embed_bwd_rows"
    dev = _here(w, ids, dY, row_ids, rows, n_unique, workspace)
    for t, name in ((ids, "ids"), (row_ids, "row_ids"), (n_unique, "n_unique")):
        _i64(t, w, name)
    ldy, ldr = _rows(dY, w, "dY"), _rows(rows, w, "rows")
    (have, d), T = rows.shape, ids.numel()
    cap = min(T, int(n_rows))
    if tuple(dY.shape) != (T, d):
        raise HstuError(1, f"{w}: dY: [ids, rows' columns]")
    if row_ids.numel() < cap or have < cap or n_unique.numel() < 1:
        raise HstuError(1, f"{w}: row_ids, rows: min(ids, n_rows) entries")
    code = lib().hstu_embed_bwd_rows(T, ids.data_ptr(), dY.data_ptr(), _dtype(dY, w), ldy,
                                     int(n_rows), d, pad_id, scale, row_ids.data_ptr(),
                                     rows.data_ptr(), _dtype(rows, w), ldr, n_unique.data_ptr(),
                                     workspace.data_ptr(), _nbytes(workspace),
                                     _raw_stream(stream, dev))
    if code != 0:
        _check(code, w)


class GradTensors:
    """A list of gradients laid out once for hstu_grad_norm: dicts with "grad"
    (contiguous, bf16, fp16 or fp32) and, where only the first rows of it count,
    "n_rows" (int64 [1] on the device).

    The list keeps the tensors and takes their addresses here, not at the
    calls: it is for buffers that stay, whose contents change.  A gradient that
    is allocated anew needs a new list; the old one goes on using the old
    tensor."""

    def __init__(self, tensors: Sequence[Dict[str, object]]):
        self.tensors = [dict(t) for t in tensors]  # keeps the memory alive
        self.n = len(self.tensors)
        self.array = (AdamWTensor * max(1, self.n))()
        self.device = None
        for c, t in zip(self.array, self.tensors):
            self._fill(c, t)

    def _take(self, t, name: str):
        w = type(self).__name__
        _need(t.is_contiguous() and t.is_cuda, w, f"{name}: a contiguous device tensor")
        if self.device is None:
            self.device = t.get_device()
        _need(t.get_device() == self.device, w, f"{name}: on another device than the rest")
        return _ptr(t)

    def _fill(self, c, t) -> None:
        w = type(self).__name__
        g = t["grad"]
        c.grad, c.grad_dtype, c.n = self._take(g, "grad"), _dtype(g, w), g.numel()
        if t.get("n_rows") is not None:
            _need(g.dim() == 2, w, "grad with n_rows: a matrix")
            _i64(t["n_rows"], w, "n_rows")
            _need(t["n_rows"].numel() == 1, w, "n_rows: int64 [1]")
            c.n_rows = self._take(t["n_rows"], "n_rows")
            c.max_rows, c.row_len = g.shape


class AdamWTensors(GradTensors):
    """A list of tensors laid out once for hstu_adamw_step (and hstu_grad_norm):
    dicts with "param", "grad", "m", "v"; optional "master" (fp32), "copy_f16"
    (fp16), "weight_decay"; with 8-bit states "m" and "v" are uint8 or
    float8_e4m3fn and "m_scale", "v_scale" uint8 (state_scales() of the
    parameter); for a table with a row gradient "row_ids" and "n_rows".  As for
    GradTensors, addresses are taken once."""

    def _fill(self, c, t) -> None:
        import torch
        super()._fill(c, t)
        w = type(self).__name__
        p, g, m, v = (t[k] for k in ("param", "grad", "m", "v"))
        sparse = t.get("row_ids") is not None
        _need(sparse == (t.get("n_rows") is not None), w, "row_ids and n_rows come together")
        if sparse:
            _i64(t["row_ids"], w, "row_ids")
            _need(p.dim() == 2 and g.shape[1] == p.shape[1], w, "grad: rows of param")
            c.row_ids = self._take(t["row_ids"], "row_ids")
            c.max_rows = min(g.shape[0], t["row_ids"].numel())
            if not c.row_ids:
                # no entries, so no address, which would mean a dense gradient: one that is not read
                t["no_row_ids"] = torch.zeros(2, dtype=torch.int64, device=p.device)
                c.row_ids = t["no_row_ids"].data_ptr()
        else:
            _need(g.numel() == p.numel(), w, "grad: the size of param")
        c.n = p.numel()
        c.param, c.param_dtype = self._take(p, "param"), _dtype(p, w)
        for k, dt in (("master", torch.float32), ("copy_f16", torch.float16)):
            if t.get(k) is not None:
                _need(t[k].dtype == dt and t[k].numel() == p.numel(), w, f"{k}: {dt}, as param")
                setattr(c, k, self._take(t[k], k))
        _need(m.dtype == v.dtype and m.numel() == v.numel() == p.numel(), w, "m, v: as param")
        c.m, c.v = self._take(m, "m"), self._take(v, "v")
        _need(m.dtype in (torch.float32, torch.uint8, torch.float8_e4m3fn), w,
              "m, v: fp32, or uint8 or float8_e4m3fn codes")
        c.state_bits = 32 if m.dtype == torch.float32 else 8
        if c.state_bits == 8:
            n = state_scales(p.shape if sparse else (p.numel(),))
            for k in ("m_scale", "v_scale"):
                _need(t.get(k) is not None and t[k].element_size() == 1 and t[k].numel() == n, w,
                      f"{k}: {n} bytes")
                setattr(c, k, self._take(t[k], k))
        c.weight_decay = float(t.get("weight_decay", 0.0))


def state_scales(shape) -> int:
    """Number of scale bytes of 8-bit states: one per 256 elements of a dense
    tensor (shape (n,)), or of each row of a table (shape (rows, d))."""
    n = 1
    for s in shape[:-1]:
        n *= int(s)
    return n * (-(-int(shape[-1]) // 256))


def hstu_grad_norm_workspace_size() -> int:
    return int(lib().hstu_grad_norm_workspace_size())


def hstu_grad_norm(tensors: GradTensors, max_norm: float, out, workspace, stream=None) -> None:
    """out (fp32 [2]): the norm over all gradients, and the factor that clips it
    to max_norm (NaN if the norm is not finite); see include/hstu.h."""
    w = "hstu_grad_norm"
    dev = _norm_args(w, tensors, out, workspace)
    code = lib().hstu_grad_norm(tensors.array, tensors.n, max_norm, out.data_ptr(),
                                workspace.data_ptr(), _nbytes(workspace), _raw_stream(stream, dev))
    if code != 0:
        _check(code, w)


def hstu_grad_norm_after(tensors: GradTensors, max_norm: float, after, out, workspace,
                         stream=None) -> None:
    """hstu_grad_norm of gradients that the call with the workspace `after`
    made: NaN, NaN if that call failed on the device (see include/hstu.h)."""
    w = "hstu_grad_norm_after"
    dev = _norm_args(w, tensors, out, workspace, after)
    _need(_nbytes(after) >= 4, w, "after: a workspace")
    code = lib().hstu_grad_norm_after(tensors.array, tensors.n, max_norm, after.data_ptr(),
                                      out.data_ptr(), workspace.data_ptr(), _nbytes(workspace),
                                      _raw_stream(stream, dev))
    if code != 0:
        _check(code, w)


def _norm_args(w: str, tensors: GradTensors, out, *workspaces) -> int:
    dev = _here(w, out, *workspaces)
    if tensors.device is not None and tensors.device != dev:
        raise HstuError(1, f"{w}: the tensors are on another device")
    if out.dtype != _FP32 or not out.is_contiguous() or out.numel() < 2:
        raise HstuError(1, f"{w}: out: fp32 [2]")
    return dev


def hstu_adamw_workspace_size() -> int:
    return int(lib().hstu_adamw_workspace_size())


def hstu_adamw_step(tensors: AdamWTensors, workspace, lr, step, beta1: float = 0.9,
                    beta2: float = 0.999, eps: float = 1e-8, grad_scale=None, seed: int = 0,
                    stream=None) -> None:
    """One AdamW step of every tensor of the list (see include/hstu.h).  `lr`
    and `step` are numbers, or device tensors (fp32 [1], int64 [1]) read by the
    kernel; grad_scale: fp32 [1] on the device."""
    w = "hstu_adamw_step"
    if not isinstance(tensors, AdamWTensors):
        raise HstuError(1, f"{w}: tensors: an AdamWTensors list")
    dev = _here(w, workspace)
    if tensors.device is not None and tensors.device != dev:
        raise HstuError(1, f"{w}: the tensors are on another device")
    lr_dev = step_dev = scale = 0
    if hasattr(lr, "data_ptr"):
        lr, lr_dev = 0.0, _scalar(lr, _FP32, w, "lr", dev)
    if hasattr(step, "data_ptr"):
        step, step_dev = 1, _scalar(step, _INT64, w, "step", dev)
    if grad_scale is not None:
        scale = _scalar(grad_scale, _FP32, w, "grad_scale", dev)
    # hstu_adamw_args
    args = _pack_args(lr, beta1, beta2, eps, step, step_dev, lr_dev, scale, seed & ((1 << 64) - 1))
    code = lib().hstu_adamw_step(args, tensors.array, tensors.n, workspace.data_ptr(),
                                 _nbytes(workspace), _current_raw_stream(dev) if stream is None
                                 else _stream(stream))
    if code != 0:
        _check(code, w)


_pack_args = struct.Struct("4dq4Q").pack


def _scalar(t, dtype, where: str, name: str, dev: int) -> int:
    """Address of a one-element device tensor."""
    if t.get_device() != dev or t.dtype != dtype or t.numel() != 1:
        raise HstuError(1, f"{where}: {name}: {dtype} [1] on the current device")
    return t.data_ptr()


def hstu_stack_fwd(desc, n_layers, weights, B, total_tokens, max_len, offsets, X, timestamps,
                   out, workspace, stream=None) -> None:
    arr = weights if not isinstance(weights, (list, tuple)) else weights_array(weights)
    _check(lib().hstu_stack_fwd(ctypes.byref(desc), n_layers, arr, B, total_tokens, max_len,
                                _ptr(offsets), _ptr(X), _ptr(timestamps), _ptr(out),
                                _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "hstu_stack_fwd")


def grads_array(gs: Sequence[Dict[str, object]]):
    """LayerGrads array from per-layer dicts of fp32 device tensors."""
    arr = (LayerGrads * len(gs))()
    for i, g in enumerate(gs):
        arr[i] = LayerGrads(*[_ptr(g[k]) for k in GRAD_KEYS])
    return arr


def hstu_bwd_workspace_size(desc: LayerDesc, n_layers: int, B: int, total_tokens: int,
                            max_len: int) -> int:
    n = int(lib().hstu_bwd_workspace_size(ctypes.byref(desc), n_layers, B, total_tokens, max_len))
    if n == 0:
        raise HstuError(1, "hstu_bwd_workspace_size")
    return n


def hstu_layer_bwd(desc, weights, B, total_tokens, max_len, offsets, X, timestamps, dY, dX,
                   grads, workspace, stream=None) -> None:
    w = weights if isinstance(weights, LayerWeights) else weights_struct(weights)
    g = grads if not isinstance(grads, (list, tuple)) else grads_array(grads)
    _check(lib().hstu_layer_bwd(ctypes.byref(desc), ctypes.byref(w), B, total_tokens, max_len,
                                _ptr(offsets), _ptr(X), _ptr(timestamps), _ptr(dY), _ptr(dX), g,
                                _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "hstu_layer_bwd")


def hstu_stack_bwd(desc, n_layers, weights, B, total_tokens, max_len, offsets, X, timestamps, dY,
                   dX, grads, workspace, stream=None) -> None:
    arr = weights if not isinstance(weights, (list, tuple)) else weights_array(weights)
    g = grads if not isinstance(grads, (list, tuple)) else grads_array(grads)
    _check(lib().hstu_stack_bwd(ctypes.byref(desc), n_layers, arr, B, total_tokens, max_len,
                                _ptr(offsets), _ptr(X), _ptr(timestamps), _ptr(dY), _ptr(dX), g,
                                _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "hstu_stack_bwd")


def hstu_mfalcon_rank(desc, n_layers, weights, B, total_hist, max_len, hist_offsets, history,
                      hist_timestamps, total_cands, max_cands, cand_offsets, candidates,
                      request_ts, microbatch, head_vec, scores, workspace, stream=None) -> None:
    arr = weights if not isinstance(weights, (list, tuple)) else weights_array(weights)
    _check(lib().hstu_mfalcon_rank(ctypes.byref(desc), n_layers, arr, B, total_hist, max_len,
                                   _ptr(hist_offsets), _ptr(history), _ptr(hist_timestamps),
                                   total_cands, max_cands, _ptr(cand_offsets), _ptr(candidates),
                                   _ptr(request_ts), microbatch, _ptr(head_vec), _ptr(scores),
                                   _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "hstu_mfalcon_rank")


def hstu_read_status(workspace, stream=None) -> int:
    return int(lib().hstu_read_status(_ptr(workspace), _nbytes(workspace), _stream(stream)))


def hstu_debug_offsets(desc, B, total_tokens, max_len):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().hstu_debug_offsets(ctypes.byref(desc), B, total_tokens, max_len,
                                    ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
           "hstu_debug_offsets")
    return int(a.value), int(b.value), int(c.value)


def hstu_set_option(name: str, value: int) -> None:
    _check(lib().hstu_set_option(name.encode(), int(value)), "hstu_set_option")


def hstu_debug_keep_z(on: bool) -> None:
    _check(lib().hstu_debug_keep_z(1 if on else 0), "hstu_debug_keep_z")


def hstu_debug_wait_test(wait_limit_us: int, inject_stall: int) -> None:
    _check(lib().hstu_debug_wait_test(int(wait_limit_us), int(inject_stall)),
           "hstu_debug_wait_test")


def hstu_trace_enable(max_records: int) -> None:
    _check(lib().hstu_trace_enable(max_records), "hstu_trace_enable")


def hstu_trace_only(kernel_id: int) -> None:
    _check(lib().hstu_trace_only(kernel_id), "hstu_trace_only")


def hstu_trace_read(capacity: int = 1 << 16):
    ids = (ctypes.c_int32 * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = lib().hstu_trace_read(ids, ms, capacity)
    return [(int(ids[i]), float(ms[i])) for i in range(n)]


def hstu_kernel_name(kernel_id: int) -> str:
    return lib().hstu_kernel_name(kernel_id).decode()


def hstu_launch_count() -> int:
    return int(lib().hstu_launch_count())


def hstu_status_string(code: int) -> str:
    return lib().hstu_status_string(code).decode()


def hstu_version() -> int:
    return int(lib().hstu_version())
