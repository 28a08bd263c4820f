"""Thin Python binding of ``libgptq.so`` (argument marshalling only).

The functions named like the C entry points (``gptq_hessian_accumulate``, ``gptq_prepare``,
``gptq_quantize_layer``, ...) take raw device pointers, sizes and a stream handle exactly as
the C ABI does.  The tensor helpers below them (``hessian``, ``prepare``, ``quantize``) only
allocate outputs/workspaces with torch, pass pointers, and raise on a non-OK status: every
step of the computation runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or fails to load, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import re

from . import build_lib

GPTQ_OK = 0
STATUS_NAMES = {
    0: "GPTQ_OK", 1: "GPTQ_ERR_INVALID_ARG", 2: "GPTQ_ERR_NOT_PD", 3: "GPTQ_ERR_NONFINITE",
    4: "GPTQ_ERR_TIMEOUT", 5: "GPTQ_ERR_CUDA", 6: "GPTQ_ERR_UNSUPPORTED", 7: "GPTQ_ERR_WORKSPACE",
}
DTYPES = {"f16": 0, "bf16": 1, "f32": 2}

SCORES = {"softmax": 0, "sigmoid": 1}

_c = ctypes


class Fp8Weights(_c.Structure):
    """``gptq_fp8_weights`` of include/gptq.h."""
    _fields_ = [("codes", _c.c_void_p), ("ld", _c.c_int64), ("next_codes", _c.c_int64),
                ("exps", _c.c_void_p), ("ld_exps", _c.c_int64), ("next_exps", _c.c_int64),
                ("scale", _c.c_void_p), ("bias", _c.c_void_p)]


_Weights = _c.POINTER(Fp8Weights)
_SIGS = {
    "gptq_status_str": (_c.c_char_p, [_c.c_int]),
    "gptq_abi_version": (_c.c_int, []),
    "gptq_kernel_launches": (_c.c_ulonglong, []),
    "gptq_hessian_accumulate": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
                                           _c.c_int64, _c.c_void_p, _c.c_int, _c.c_void_p]),
    "gptq_hessian_host_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_int64, _c.c_int64]),
    "gptq_hessian_accumulate_host": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
                                                _c.c_int64, _c.c_void_p, _c.c_int, _c.c_int64,
                                                _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_prepare_workspace_bytes": (_c.c_size_t, [_c.c_int64]),
    "gptq_prepare": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_float, _c.c_void_p, _c.c_void_p,
                                _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_quantize_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int, _c.c_int]),
    "gptq_quantize_layer": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
                                       _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_int,
                                       _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                       _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_workspace_status": (_c.c_int, [_c.c_void_p, _c.c_void_p]),
    "gptq_recon_error_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_int64, _c.c_int64,
                                                       _c.c_int64]),
    "gptq_recon_error": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
                                    _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_void_p,
                                    _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                    _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_quantize_obq_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64]),
    "gptq_quantize_obq": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
                                     _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p,
                                     _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                     _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_quantize_shared_workspace_bytes": (_c.c_size_t, [_c.c_int, _c.c_void_p, _c.c_int64,
                                                           _c.c_int, _c.c_int]),
    "gptq_quantize_layers_shared": (_c.c_int, [_c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                               _c.c_void_p, _c.c_int64, _c.c_void_p,
                                               _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                                               _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                               _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_quantize_layer_noalloc": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
                                               _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_int,
                                               _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                               _c.c_void_p, _c.c_void_p]),
    "gptq_noalloc_status": (_c.c_int, [_c.c_void_p]),
    "gptq_debug_hessian_lost_stage": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
                                                 _c.c_int64, _c.c_void_p, _c.c_int64,
                                                 _c.c_uint64, _c.c_void_p, _c.c_void_p]),
    "gptq_rmsnorm_fp8": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
                                    _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_float,
                                    _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                    _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_void_p]),
    "gptq_fp8_quantize": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
                                     _c.c_int, _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                     _c.c_void_p]),
    "gptq_fp8_from_codes": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_void_p, _c.c_int64,
                                       _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                       _c.c_int64, _c.c_void_p]),
    "gptq_fp8_matmul_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int64]),
    "gptq_fp8_matmul": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                   _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                   _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int,
                                   _c.c_int64, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_kv8_append": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int,
                                   _c.c_int64, _c.c_int64, _c.c_int, _c.c_int, _c.c_void_p,
                                   _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64,
                                   _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p,
                                   _c.c_void_p]),
    "gptq_kv8_attention_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int,
                                                         _c.c_int, _c.c_int, _c.c_int64]),
    "gptq_kv8_attention": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
                                      _c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p,
                                      _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                      _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_float,
                                      _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                      _c.c_void_p]),
    "gptq_serving_status": (_c.c_int, [_c.c_void_p]),
    "gptq_fp8_linear_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int64, _c.c_int64]),
    "gptq_fp8_linear": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                   _Weights, _c.c_int, _c.c_void_p, _c.c_int64, _c.c_int64,
                                   _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_int64,
                                   _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_fp8_gated": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                  _Weights, _Weights, _c.c_int, _c.c_int64, _c.c_int64,
                                  _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                  _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_fp8_experts_gated": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                          _c.c_void_p, _Weights, _Weights, _c.c_int, _c.c_int,
                                          _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64,
                                          _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int64,
                                          _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_size_t,
                                          _c.c_void_p]),
    "gptq_fp8_experts": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _Weights,
                                    _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int64,
                                    _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_int64,
                                    _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_moe_route_workspace_bytes": (_c.c_size_t, [_c.c_int64, _c.c_int, _c.c_int]),
    "gptq_moe_route": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int,
                                  _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                                  _c.c_float, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                  _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_moe_combine": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int,
                                    _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                    _c.c_int64, _c.c_void_p]),
    "gptq_debug_fp8_gated_lost_copy": (_c.c_int, [
        _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _Weights, _Weights, _c.c_int, _c.c_int,
        _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p,
        _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_uint64, _c.c_void_p, _c.c_size_t,
        _c.c_void_p]),
    "gptq_debug_fp8_matmul_lost_copy": (_c.c_int, [_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                                   _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
                                                   _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p,
                                                   _c.c_int, _c.c_int64, _c.c_int64, _c.c_uint64,
                                                   _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "gptq_debug_kv8_attention_lost_copy": (_c.c_int, [
        _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int, _c.c_int, _c.c_int,
        _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64,
        _c.c_int64, _c.c_void_p, _c.c_int, _c.c_float, _c.c_void_p, _c.c_void_p, _c.c_int64,
        _c.c_uint64, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
}
NOALLOC_SCRATCH_BYTES = 32 << 20  # GPTQ_NOALLOC_SCRATCH_BYTES in include/gptq.h
OBQ_MAX_D_IN = 128                # GPTQ_OBQ_MAX_D_IN in include/gptq.h
MAX_SHARED_LAYERS = 64            # GPTQ_MAX_SHARED_LAYERS in include/gptq.h
FP8_BLOCK = 128                   # elements of K (and weight rows) that share an exponent
KV8_BLOCK = 64                    # GPTQ_KV8_BLOCK in include/gptq.h

_lib = None


class GptqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.status, self.status)}")


def library_path() -> str:
    return build_lib.LIB


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library (once).  Raises if it is missing: build it with
    ``python -m post_weight_quantization_03_gb300.build_lib``."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or library_path()
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: the CUDA library must be built (build_lib.build())")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def declared_symbols(header: str | None = None):
    """Names of the functions ``include/gptq.h`` declares."""
    header = header or os.path.join(build_lib.INCLUDE, "gptq.h")
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gptq_[a-z_0-9]+)\s*\(", text)))


# ---------------------------------------------------------------------------------------
# C entry points, same names and arguments
# ---------------------------------------------------------------------------------------

def gptq_status_str(status):
    return load().gptq_status_str(status).decode()


def gptq_abi_version():
    return load().gptq_abi_version()


def gptq_kernel_launches():
    return load().gptq_kernel_launches()


def gptq_hessian_accumulate(X, xdtype, n_tok, d_in, ldx, H, accumulate, stream):
    return load().gptq_hessian_accumulate(X, xdtype, n_tok, d_in, ldx, H, accumulate, stream)


def gptq_hessian_host_workspace_bytes(xdtype, d_in, chunk_tok):
    return load().gptq_hessian_host_workspace_bytes(xdtype, d_in, chunk_tok)


def gptq_hessian_accumulate_host(X_host, xdtype, n_tok, d_in, ldx, H, accumulate, chunk_tok, ws,
                                 ws_bytes, stream):
    return load().gptq_hessian_accumulate_host(X_host, xdtype, n_tok, d_in, ldx, H, accumulate,
                                               chunk_tok, ws, ws_bytes, stream)


def gptq_prepare_workspace_bytes(d_in):
    return load().gptq_prepare_workspace_bytes(d_in)


def gptq_prepare(H, d_in, damp, U, dead_mask, n_dead, ws, ws_bytes, stream):
    return load().gptq_prepare(H, d_in, damp, U, dead_mask, n_dead, ws, ws_bytes, stream)


def gptq_quantize_workspace_bytes(d_out, d_in, bits, block):
    return load().gptq_quantize_workspace_bytes(d_out, d_in, bits, block)


def gptq_quantize_layer(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, block, qpacked,
                        scale, zero, W_hat, ws, ws_bytes, stream):
    return load().gptq_quantize_layer(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, block,
                                      qpacked, scale, zero, W_hat, ws, ws_bytes, stream)


def gptq_workspace_status(ws, stream):
    return load().gptq_workspace_status(ws, stream)


def gptq_recon_error_workspace_bytes(xdtype, d_out, d_in, n_tok):
    return load().gptq_recon_error_workspace_bytes(xdtype, d_out, d_in, n_tok)


def gptq_recon_error(X, xdtype, n_tok, d_in, ldx, W, wdtype, d_out, ldw, qpacked, bits, scale,
                     zero, err, ws, ws_bytes, stream):
    return load().gptq_recon_error(X, xdtype, n_tok, d_in, ldx, W, wdtype, d_out, ldw, qpacked,
                                   bits, scale, zero, err, ws, ws_bytes, stream)


def gptq_quantize_obq_workspace_bytes(d_out, d_in):
    return load().gptq_quantize_obq_workspace_bytes(d_out, d_in)


def gptq_quantize_obq(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, qpacked, scale, zero,
                      W_hat, order, ws, ws_bytes, stream):
    return load().gptq_quantize_obq(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, qpacked,
                                    scale, zero, W_hat, order, ws, ws_bytes, stream)


def gptq_quantize_shared_workspace_bytes(n_layers, d_out, d_in, bits, block):
    return load().gptq_quantize_shared_workspace_bytes(n_layers, d_out, d_in, bits, block)


def gptq_quantize_layers_shared(n_layers, W, wdtype, d_out, ldw, d_in, U, dead_mask, bits, block,
                                qpacked, scale, zero, W_hat, ws, ws_bytes, stream):
    return load().gptq_quantize_layers_shared(n_layers, W, wdtype, d_out, ldw, d_in, U,
                                              dead_mask, bits, block, qpacked, scale, zero,
                                              W_hat, ws, ws_bytes, stream)


def gptq_quantize_layer_noalloc(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, block,
                                qpacked, scale, zero, W_hat, stream):
    return load().gptq_quantize_layer_noalloc(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits,
                                              block, qpacked, scale, zero, W_hat, stream)


def gptq_noalloc_status(stream):
    return load().gptq_noalloc_status(stream)


def gptq_debug_hessian_lost_stage(X, xdtype, n_tok, d_in, ldx, H, lost_stage, wait_ns, status_ws,
                                  stream):
    return load().gptq_debug_hessian_lost_stage(X, xdtype, n_tok, d_in, ldx, H, lost_stage,
                                                wait_ns, status_ws, stream)


def gptq_rmsnorm_fp8(X, xdtype, rows, d, ldx, R, ldr, weight, wdtype, eps, H, ldh, codes, ldc,
                     exps, lde, rstd, stream):
    return load().gptq_rmsnorm_fp8(X, xdtype, rows, d, ldx, R, ldr, weight, wdtype, eps, H, ldh,
                                   codes, ldc, exps, lde, rstd, stream)


def gptq_fp8_quantize(X, xdtype, rows, d, ldx, row_block, codes, ldc, exps, lde, stream):
    return load().gptq_fp8_quantize(X, xdtype, rows, d, ldx, row_block, codes, ldc, exps, lde,
                                    stream)


def gptq_fp8_from_codes(qpacked, bits, zero, d_out, d_in, codes, ldc, exps, lde, stream):
    return load().gptq_fp8_from_codes(qpacked, bits, zero, d_out, d_in, codes, ldc, exps, lde,
                                      stream)


def gptq_fp8_matmul_workspace_bytes(m, n, k):
    return load().gptq_fp8_matmul_workspace_bytes(m, n, k)


def gptq_fp8_matmul(a, lda, a_exps, ldae, a_scale, w, ldw, w_exps, ldwe, w_scale, m, n, k, out,
                    odtype, ldo, ws, ws_bytes, stream):
    return load().gptq_fp8_matmul(a, lda, a_exps, ldae, a_scale, w, ldw, w_exps, ldwe, w_scale,
                                  m, n, k, out, odtype, ldo, ws, ws_bytes, stream)


def gptq_kv8_append(new_k, k_strides, new_v, v_strides, dtype, n_seq, n_new, n_kv, dim, k, v,
                    k_exps, v_exps, n_blocks, table, ld_table, max_blocks, start, stream):
    return load().gptq_kv8_append(new_k, k_strides, new_v, v_strides, dtype, n_seq, n_new, n_kv,
                                  dim, k, v, k_exps, v_exps, n_blocks, table, ld_table,
                                  max_blocks, start, stream)


def gptq_kv8_attention_workspace_bytes(n_seq, n_new, n_heads, n_kv, dim, max_blocks):
    return load().gptq_kv8_attention_workspace_bytes(n_seq, n_new, n_heads, n_kv, dim,
                                                     max_blocks)


def gptq_kv8_attention(q, q_strides, dtype, n_seq, n_new, n_heads, n_kv, dim, k, v, k_exps,
                       v_exps, n_blocks, table, ld_table, max_blocks, lengths, causal, scale,
                       out, o_strides, ws, ws_bytes, stream):
    return load().gptq_kv8_attention(q, q_strides, dtype, n_seq, n_new, n_heads, n_kv, dim, k, v,
                                     k_exps, v_exps, n_blocks, table, ld_table, max_blocks,
                                     lengths, causal, scale, out, o_strides, ws, ws_bytes,
                                     stream)


def gptq_serving_status(stream):
    return load().gptq_serving_status(stream)


def gptq_fp8_linear_workspace_bytes(rows, n, k):
    return load().gptq_fp8_linear_workspace_bytes(rows, n, k)


def gptq_fp8_linear(a, lda, a_exps, ldae, a_scale, w, act, residual, ldr, m, n, k, out, odtype, ldo,
                    ws, ws_bytes, stream):
    return load().gptq_fp8_linear(a, lda, a_exps, ldae, a_scale, w, act, residual, ldr, m, n, k,
                                  out, odtype, ldo, ws, ws_bytes, stream)


def gptq_fp8_gated(a, lda, a_exps, ldae, a_scale, gate, up, act, m, n, k, codes, ldc, exps, lde, ws,
                   ws_bytes, stream):
    return load().gptq_fp8_gated(a, lda, a_exps, ldae, a_scale, gate, up, act, m, n, k, codes, ldc,
                                 exps, lde, ws, ws_bytes, stream)


def gptq_fp8_experts_gated(a, lda, a_exps, ldae, a_scale, gate, up, act, n_experts, offsets, order,
                           top_k, n_tokens, n, k, codes, ldc, exps, lde, ws, ws_bytes, stream):
    return load().gptq_fp8_experts_gated(a, lda, a_exps, ldae, a_scale, gate, up, act, n_experts,
                                         offsets, order, top_k, n_tokens, n, k, codes, ldc, exps,
                                         lde, ws, ws_bytes, stream)


def gptq_fp8_experts(a, lda, a_exps, ldae, w, act, n_experts, offsets, order, rows, n, k, out,
                     odtype, ldo, ws, ws_bytes, stream):
    return load().gptq_fp8_experts(a, lda, a_exps, ldae, w, act, n_experts, offsets, order, rows, n,
                                   k, out, odtype, ldo, ws, ws_bytes, stream)


def gptq_moe_route_workspace_bytes(n_tokens, n_experts, top_k):
    return load().gptq_moe_route_workspace_bytes(n_tokens, n_experts, top_k)


def gptq_moe_route(logits, dtype, ld, n_tokens, n_experts, top_k, bias, scores, groups, top_groups,
                   group_top, renormalize, scale, ids, weights, offsets, order, ws, ws_bytes,
                   stream):
    return load().gptq_moe_route(logits, dtype, ld, n_tokens, n_experts, top_k, bias, scores,
                                 groups, top_groups, group_top, renormalize, scale, ids, weights,
                                 offsets, order, ws, ws_bytes, stream)


def gptq_moe_combine(y, dtype, ldy, n_tokens, top_k, d, weights, residual, ldr, out, ldo, stream):
    return load().gptq_moe_combine(y, dtype, ldy, n_tokens, top_k, d, weights, residual, ldr, out,
                                   ldo, stream)


def gptq_debug_fp8_gated_lost_copy(a, lda, a_exps, ldae, gate, up, act, n_experts, offsets, order, top_k,
                                   n_tokens, n, k, codes, ldc, exps, lde, lost_copy, wait_ns, ws,
                                   ws_bytes, stream):
    return load().gptq_debug_fp8_gated_lost_copy(a, lda, a_exps, ldae, gate, up, act, n_experts, offsets,
                                                 order, top_k, n_tokens, n, k, codes, ldc, exps, lde,
                                                 lost_copy, wait_ns, ws, ws_bytes, stream)


def gptq_debug_fp8_matmul_lost_copy(a, lda, a_exps, ldae, w, ldw, w_exps, ldwe, m, n, k, out, odtype,
                                    ldo, lost_copy, wait_ns, ws, ws_bytes, stream):
    return load().gptq_debug_fp8_matmul_lost_copy(a, lda, a_exps, ldae, w, ldw, w_exps, ldwe, m, n, k,
                                                  out, odtype, ldo, lost_copy, wait_ns, ws, ws_bytes,
                                                  stream)


def gptq_debug_kv8_attention_lost_copy(q, q_strides, dtype, n_seq, n_new, n_heads, n_kv, dim, k, v,
                                       k_exps, v_exps, n_blocks, table, ld_table, max_blocks, lengths,
                                       causal, scale, out, o_strides, lost_copy, wait_ns, ws,
                                       ws_bytes, stream):
    return load().gptq_debug_kv8_attention_lost_copy(q, q_strides, dtype, n_seq, n_new, n_heads, n_kv,
                                                     dim, k, v, k_exps, v_exps, n_blocks, table,
                                                     ld_table, max_blocks, lengths, causal, scale,
                                                     out, o_strides, lost_copy, wait_ns, ws,
                                                     ws_bytes, stream)


# ---------------------------------------------------------------------------------------
# torch-tensor helpers (marshalling only)
# ---------------------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    m = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, where):
    if status != GPTQ_OK:
        raise GptqError(status, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def workspace(nbytes, device):
    """A 256-byte aligned byte workspace (torch allocations are 256-byte aligned)."""
    torch = _torch()
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def hessian(X, H=None, accumulate=False, stream=None):
    """``H (+)= 2 X^T X`` for token-major X ``[n_tok, d_in]`` (row stride X.stride(0))."""
    torch = _torch()
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a row-major [n_tok, d_in] matrix")
    n, d = X.shape
    if H is None:
        H = torch.empty(d, d, dtype=torch.float32, device=X.device)
        accumulate = False
    _check(gptq_hessian_accumulate(_ptr(X), _dtype_code(X), n, d, X.stride(0), _ptr(H),
                                   1 if accumulate else 0, _stream(stream)),
           "gptq_hessian_accumulate")
    return H


def hessian_host(Xh, H=None, accumulate=False, chunk_tok=0, ws=None, device=None, stream=None):
    """``H (+)= 2 X^T X`` for a token-major HOST matrix ``Xh`` (CPU tensor, pinned for the
    copies to overlap), streamed to the device in chunks of ``chunk_tok`` tokens."""
    torch = _torch()
    if Xh.device.type != "cpu" or Xh.dim() != 2 or Xh.stride(1) != 1:
        raise ValueError("Xh must be a row-major [n_tok, d_in] CPU matrix")
    n, d = Xh.shape
    dev = torch.device(device) if device is not None else (
        H.device if H is not None else torch.device("cuda", torch.cuda.current_device()))
    if H is None:
        H = torch.empty(d, d, dtype=torch.float32, device=dev)
        accumulate = False
    need = gptq_hessian_host_workspace_bytes(_dtype_code(Xh), d, chunk_tok)
    if ws is None:
        ws = workspace(need, H.device)
    _check(gptq_hessian_accumulate_host(ctypes.c_void_p(Xh.data_ptr()), _dtype_code(Xh), n, d,
                                        Xh.stride(0), _ptr(H), 1 if accumulate else 0, chunk_tok,
                                        _ptr(ws), ws.numel(), _stream(stream)),
           "gptq_hessian_accumulate_host")
    return H


def prepare(H, damp=0.01, U=None, dead_mask=None, ws=None, stream=None):
    """Dead columns + damping + ``U`` with ``U^T U = H_damped^-1``.  CONSUMES ``H``.

    Returns ``(U, dead_mask, n_dead)``.
    """
    torch = _torch()
    d = H.shape[0]
    if H.dtype != torch.float32 or not H.is_contiguous() or H.shape != (d, d):
        raise ValueError("H must be a contiguous float32 [d, d] matrix")
    if U is None:
        U = torch.empty(d, d, dtype=torch.float32, device=H.device)
    if dead_mask is None:
        dead_mask = torch.empty(d, dtype=torch.uint8, device=H.device)
    nbytes = gptq_prepare_workspace_bytes(d)
    if ws is None:
        ws = workspace(nbytes, H.device)
    n_dead = ctypes.c_int32(0)
    _check(gptq_prepare(_ptr(H), d, float(damp), _ptr(U), _ptr(dead_mask),
                        ctypes.byref(n_dead), _ptr(ws), ws.numel(), _stream(stream)),
           "gptq_prepare")
    return U, dead_mask, n_dead.value


def packed_words(d_in, bits):
    return ((d_in + 31) // 32) * bits


def quantize(W, U, bits=4, block=128, dead_mask=None, want_w_hat=True, ws=None, stream=None,
             out=None):
    """The GPTQ sweep of one layer.  Returns ``(qpacked, scale, zero, W_hat or None)``."""
    torch = _torch()
    if W.dim() != 2 or W.stride(1) != 1:
        raise ValueError("W must be a row-major [d_out, d_in] matrix")
    m, d = W.shape
    dev = W.device
    if out is None:
        qpacked = torch.empty(m, packed_words(d, bits), dtype=torch.int32, device=dev)
        scale = torch.empty(m, dtype=torch.float32, device=dev)
        zero = torch.empty(m, dtype=torch.int32, device=dev)
        W_hat = torch.empty(m, d, dtype=torch.float32, device=dev) if want_w_hat else None
    else:
        qpacked, scale, zero, W_hat = out
    if ws is None:
        ws = workspace(gptq_quantize_workspace_bytes(m, d, bits, block), dev)
    _check(gptq_quantize_layer(_ptr(W), _dtype_code(W), m, d, W.stride(0), _ptr(U),
                               _ptr(dead_mask), bits, block, _ptr(qpacked), _ptr(scale),
                               _ptr(zero), _ptr(W_hat), _ptr(ws), ws.numel(), _stream(stream)),
           "gptq_quantize_layer")
    return qpacked, scale, zero, W_hat


def _ptr_array(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() if t is not None else None for t in ts])


def quantize_shared(Ws, U, bits=4, block=128, dead_mask=None, want_w_hat=False, ws=None,
                    stream=None):
    """The sweep of several layers sharing U (one stack of rows).  Returns one
    ``(qpacked, scale, zero, W_hat or None)`` tuple per layer."""
    torch = _torch()
    n = len(Ws)
    d = Ws[0].shape[1]
    for W in Ws:
        if W.dim() != 2 or W.stride(1) != 1 or W.shape[1] != d:
            raise ValueError("every W must be a row-major [d_out, d_in] matrix with one d_in")
    dev = Ws[0].device
    outs = []
    for W in Ws:
        m = W.shape[0]
        outs.append((torch.empty(m, packed_words(d, bits), dtype=torch.int32, device=dev),
                     torch.empty(m, dtype=torch.float32, device=dev),
                     torch.empty(m, dtype=torch.int32, device=dev),
                     torch.empty(m, d, dtype=torch.float32, device=dev) if want_w_hat else None))
    d_out = (ctypes.c_int64 * n)(*[W.shape[0] for W in Ws])
    if ws is None:
        ws = workspace(gptq_quantize_shared_workspace_bytes(n, d_out, d, bits, block), dev)
    _check(gptq_quantize_layers_shared(
        n, _ptr_array(Ws), (ctypes.c_int * n)(*[_dtype_code(W) for W in Ws]), d_out,
        (ctypes.c_int64 * n)(*[W.stride(0) for W in Ws]), d, _ptr(U), _ptr(dead_mask), bits,
        block, _ptr_array([o[0] for o in outs]), _ptr_array([o[1] for o in outs]),
        _ptr_array([o[2] for o in outs]),
        _ptr_array([o[3] for o in outs]) if want_w_hat else None, _ptr(ws), ws.numel(),
        _stream(stream)), "gptq_quantize_layers_shared")
    return outs


def quantize_block(groups, bits=(4,), block=128, damp=0.01, chunk_tok=None, overlap=True,
                   stage_events=None, consumers=2):
    """GPTQ over a block of layers grouped by their shared inputs.

    ``groups`` is a list of ``(X, [W, ...])``: X the token-major inputs of the group (on the
    device) and the weights of every layer that reads them.  Per group: H from X, one
    prepare, then one shared sweep of all its layers per bit width.  With ``overlap`` the
    Hessians are accumulated (in chunks of ``chunk_tok`` tokens, or in one call when None) on
    a producer stream, ahead of the prepares and sweeps, which run on ``consumers``
    higher-priority streams taken in turn by group (so one group's sweep can run beside the
    next group's prepare); every step is a call of this library.  Returns
    ``[{bits: [(qpacked, scale, zero, None) per layer]}, ...]`` and the dead-column counts,
    in group order."""
    torch = _torch()
    dev = groups[0][1][0].device
    caller = torch.cuda.current_stream(dev)
    lo, hi = torch.cuda.Stream.priority_range()
    cons_all = ([torch.cuda.Stream(dev, priority=hi) for _ in range(max(1, consumers))]
                if overlap else [caller])
    prod = torch.cuda.Stream(dev, priority=lo) if overlap else caller
    if overlap:
        prod.wait_stream(caller)
        for c in cons_all:
            c.wait_stream(caller)
    Hs, ready = [], []
    for X, _ in groups:
        d = X.shape[1]
        H = torch.empty(d, d, dtype=torch.float32, device=dev)
        if stage_events is not None:
            e0 = torch.cuda.Event(enable_timing=True)
            e0.record(prod)
        step = chunk_tok or max(X.shape[0], 1)
        for t0 in range(0, X.shape[0], step):
            hessian(X[t0:t0 + step], H, accumulate=t0 > 0, stream=prod)
        e = torch.cuda.Event(enable_timing=stage_events is not None)
        e.record(prod)
        if stage_events is not None:
            stage_events.append(("hessian", e0, e))
        Hs.append(H)
        ready.append(e)
    results, n_dead, keep = [], [], []
    for gi, ((X, Ws), H, e) in enumerate(zip(groups, Hs, ready)):
        cons = cons_all[gi % len(cons_all)]
        cons.wait_event(e)
        d = X.shape[1]
        e0 = torch.cuda.Event(enable_timing=True)
        e0.record(cons)
        # every buffer a stream uses stays referenced until the caller has joined the streams
        pws = workspace(gptq_prepare_workspace_bytes(d), dev)
        U, dm, nd = prepare(H, damp, ws=pws, stream=cons)
        e1 = torch.cuda.Event(enable_timing=True)
        e1.record(cons)
        m_rows = (ctypes.c_int64 * len(Ws))(*[W.shape[0] for W in Ws])
        ws = workspace(max(gptq_quantize_shared_workspace_bytes(len(Ws), m_rows, d, b, block)
                           for b in bits), dev)
        res = {}
        for b in bits:
            res[b] = quantize_shared(Ws, U, b, block, dm, ws=ws, stream=cons)
        e2 = torch.cuda.Event(enable_timing=True)
        e2.record(cons)
        if stage_events is not None:
            stage_events.append(("prepare", e0, e1))
            stage_events.append(("quantize", e1, e2))
        results.append(res)
        n_dead.append(nd)
        keep += [U, dm, ws, pws]   # in use on the consumer streams until the waits below
    if overlap:
        for c in cons_all:
            caller.wait_stream(c)
        caller.wait_stream(prod)
    return results, n_dead


def recon_error(X, W, qpacked, bits, scale, zero, ws=None, stream=None):
    """Per-row ``||(W - W_hat) X^T||^2`` from the packed codes (``[d_out]`` fp32)."""
    torch = _torch()
    n, d = X.shape
    m = W.shape[0]
    if X.stride(1) != 1 or W.stride(1) != 1 or W.shape[1] != d:
        raise ValueError("X [n_tok, d_in] and W [d_out, d_in] must be row-major")
    err = torch.empty(m, dtype=torch.float32, device=W.device)
    if ws is None:
        ws = workspace(gptq_recon_error_workspace_bytes(_dtype_code(X), m, d, n), W.device)
    _check(gptq_recon_error(_ptr(X), _dtype_code(X), n, d, X.stride(0), _ptr(W), _dtype_code(W),
                            m, d if W.stride(0) == d else W.stride(0), _ptr(qpacked), bits,
                            _ptr(scale), _ptr(zero), _ptr(err), _ptr(ws), ws.numel(),
                            _stream(stream)), "gptq_recon_error")
    return err


def quantize_obq(W, U, bits=4, dead_mask=None, ws=None, stream=None):
    """OBQ greedy order per row (d_in <= 128).  Returns
    ``(qpacked, scale, zero, W_hat, order)``."""
    torch = _torch()
    m, d = W.shape
    dev = W.device
    qpacked = torch.empty(m, packed_words(d, bits), dtype=torch.int32, device=dev)
    scale = torch.empty(m, dtype=torch.float32, device=dev)
    zero = torch.empty(m, dtype=torch.int32, device=dev)
    W_hat = torch.empty(m, d, dtype=torch.float32, device=dev)
    order = torch.empty(m, d, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(gptq_quantize_obq_workspace_bytes(m, d), dev)
    _check(gptq_quantize_obq(_ptr(W), _dtype_code(W), m, d, W.stride(0), _ptr(U),
                             _ptr(dead_mask), bits, _ptr(qpacked), _ptr(scale), _ptr(zero),
                             _ptr(W_hat), _ptr(order), _ptr(ws), ws.numel(), _stream(stream)),
           "gptq_quantize_obq")
    return qpacked, scale, zero, W_hat, order


# ---------------------------------------------------------------------------------------
# 8-bit serving (helpers of a step that runs for each token: their own cost is host time, so
# they read each tensor attribute once and pass plain integers)
# ---------------------------------------------------------------------------------------

def _lend(stream, *tensors):
    """Tells torch's allocator that buffers made here for a call on ``stream`` are in use there."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _stream_of(device, stream):
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    index = device.index
    return torch._C._cuda_getCurrentRawStream(
        index if index is not None else torch.cuda.current_device())


# The kernels take addresses: every tensor of a call has to be on one GPU (asked for in place, a
# function over the tensors takes twice as long).
_ONE_GPU = "a call's tensors must be on one GPU"


_SERVING_DTYPES = {}


def _serving_dtype(dtype):
    if not _SERVING_DTYPES:
        torch = _torch()
        _SERVING_DTYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    code = _SERVING_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _fp8_empty(rows, d, row_block, device, stream):
    """Codes and exponents of a ``[rows, d]`` e4m3 matrix, in the pitches the library asks for."""
    torch = _torch()
    pitch, kb = (d + 15) & ~15, (d + FP8_BLOCK - 1) // FP8_BLOCK
    erows, epitch = (rows + row_block - 1) // row_block, (kb + 3) & ~3
    # (the last row has its whole pitch too: the kernels read exponents by words)
    codes = torch.empty((rows, pitch), dtype=torch.float8_e4m3fn, device=device)
    exps = torch.empty((erows, epitch), dtype=torch.uint8, device=device)
    if stream is not None:
        _lend(stream, codes, exps)
    if pitch != d:
        codes = codes.as_strided((rows, d), (pitch, 1))
    if epitch != kb:
        exps = exps.as_strided((erows, kb), (epitch, 1))
    return codes, pitch, exps, epitch


def _rows_of(name, t, rows=None, d=None):
    """Row pitch of a row-major matrix of the given size."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (
            d is not None and shape[1] != d) or (stride[1] != 1 and shape[1] != 1):
        want = f"[{'rows' if rows is None else rows}, {'d' if d is None else d}]"
        raise ValueError(f"{name} must be a row-major {want} matrix")
    return stride[0] if shape[0] != 1 else max(stride[0], shape[1])


def rmsnorm_fp8(X, weight, residual=None, eps=1e-6, want_h=True, stream=None):
    """RMS norm with the residual's addition and e4m3 output.

    ``h = X + residual``; returns ``(codes, exps, rstd, h)``: the codes and exponents of
    ``h * weight`` by 1 x 128 blocks and ``rstd`` per row, so that the normalised row is
    ``rstd * 2**(exps - 127) * codes`` (hand ``rstd`` to ``fp8_matmul`` as ``a_scale``).
    ``h`` is X itself when there is no residual, None when ``want_h`` is false."""
    torch = _torch()
    ldx = _rows_of("X", X)
    n, d = X.shape
    dtype, device = X.dtype, X.device
    ldr = 0
    if residual is not None:
        ldr = _rows_of("residual", residual, n, d)
        if residual.dtype != dtype:
            raise TypeError("residual must have X's dtype")
    if weight.shape != (d,) or (d > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be a contiguous [d] vector")
    gpu = X.get_device()
    if gpu < 0 or weight.get_device() != gpu or (residual is not None and residual.get_device() != gpu):
        raise ValueError(_ONE_GPU)
    codes, ldc, exps, lde = _fp8_empty(n, d, 1, device, stream)
    rstd = torch.empty((n,), dtype=torch.float32, device=device)
    h, h_ptr = X, None
    if not want_h:
        h = None
    elif residual is not None:
        h = torch.empty((n, d), dtype=dtype, device=device)
        h_ptr = h.data_ptr()
    if stream is not None:
        _lend(stream, rstd, h)
    _check(load().gptq_rmsnorm_fp8(
        X.data_ptr(), _serving_dtype(dtype), n, d, ldx,
        residual.data_ptr() if residual is not None else None, ldr, weight.data_ptr(),
        _serving_dtype(weight.dtype), eps, h_ptr, d, codes.data_ptr(), ldc, exps.data_ptr(), lde,
        rstd.data_ptr(), _stream_of(device, stream)), "gptq_rmsnorm_fp8")
    return codes, exps, rstd, h


def fp8_quantize(X, row_block=1, stream=None):
    """``(codes, exps)`` of a ``[rows, d]`` matrix by ``row_block x 128`` blocks: 1 for
    activations, 128 for weights."""
    ldx = _rows_of("X", X)
    n, d = X.shape
    if row_block not in (1, FP8_BLOCK):
        raise ValueError(f"row_block must be 1 or {FP8_BLOCK}")
    if X.get_device() < 0:
        raise ValueError(_ONE_GPU)
    codes, ldc, exps, lde = _fp8_empty(n, d, row_block, X.device, stream)
    _check(load().gptq_fp8_quantize(X.data_ptr(), _serving_dtype(X.dtype), n, d, ldx, row_block,
                                    codes.data_ptr(), ldc, exps.data_ptr(), lde,
                                    _stream_of(X.device, stream)), "gptq_fp8_quantize")
    return codes, exps


def fp8_from_codes(qpacked, zero, d_in, bits=4, stream=None):
    """``(codes, exps)`` of a layer from ``quantize``'s packed 2-, 3- or 4-bit codes: exactly
    ``code - zero``, so with ``quantize``'s scale as ``w_scale`` the product's weights are
    exactly W_hat."""
    m = qpacked.shape[0]
    if qpacked.shape != (m, packed_words(d_in, bits)) or not qpacked.is_contiguous() \
            or zero.shape != (m,) or not zero.is_contiguous():
        raise ValueError("qpacked [d_out, ceil(d_in / 32) * bits] and zero [d_out] as quantize "
                         "returns them")
    if qpacked.dtype != zero.dtype or zero.dtype != _torch().int32:
        raise TypeError("qpacked and zero must be int32, as quantize returns them")
    if qpacked.get_device() < 0 or zero.get_device() != qpacked.get_device():
        raise ValueError(_ONE_GPU)
    codes, ldc, exps, lde = _fp8_empty(m, d_in, FP8_BLOCK, qpacked.device, stream)
    _check(load().gptq_fp8_from_codes(qpacked.data_ptr(), bits, zero.data_ptr(), m, d_in,
                                      codes.data_ptr(), ldc, exps.data_ptr(), lde,
                                      _stream_of(qpacked.device, stream)), "gptq_fp8_from_codes")
    return codes, exps


def serving_status(stream=None):
    """Waits for ``stream`` and raises if a device wait of a product (``fp8_matmul``, ``fp8_linear``,
    ``fp8_gated``, ``fp8_experts``, ``fp8_experts_gated``) or of ``kv8_attention`` gave up since the
    last such query, whatever the stream and workspace of the call: its output is then undefined."""
    _check(gptq_serving_status(_stream(stream)), "gptq_serving_status")


# The workspace of a product, and of an attention that cuts no item, is its status block alone.
# Calls without one share a block by device, which is not read back (``serving_status`` tells of a
# wait that gave up): making a tensor takes 3 to 5 us of a call's host time.
_STATUS_BLOCKS = {}


def _status_block(device):
    block = _STATUS_BLOCKS.get(device)
    if block is None:
        torch = _torch()
        block = _STATUS_BLOCKS[device] = torch.empty((256,), dtype=torch.uint8, device=device)
    return block


def fp8_matmul(a, a_exps, w, w_exps, a_scale=None, w_scale=None, out_dtype=None, out=None,
               ws=None, stream=None):
    """``diag(a_scale) A W^T diag(w_scale)`` of e4m3 matrices ``A [m, k]`` (1 x 128 blocks) and
    ``W [n, k]`` (128 x 128 blocks), ``[m, n]`` in float16 or bfloat16 (the default).  ``ws``
    (``gptq_fp8_matmul_workspace_bytes``) keeps the call's status for ``gptq_workspace_status``;
    without one ``serving_status`` tells of it."""
    torch = _torch()
    m, k = a.shape
    n = w.shape[0]
    kb = (k + FP8_BLOCK - 1) // FP8_BLOCK
    lda, ldw = _rows_of("a", a), _rows_of("w", w, n, k)
    ldae = _rows_of("a_exps", a_exps, m, kb)
    ldwe = _rows_of("w_exps", w_exps, (n + FP8_BLOCK - 1) // FP8_BLOCK, kb)
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    if a.dtype != f8 or w.dtype != f8 or a_exps.dtype != u8 or w_exps.dtype != u8:
        raise TypeError("codes are float8_e4m3fn and exponents uint8")
    for name, t, rows in (("a_scale", a_scale, m), ("w_scale", w_scale, n)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (rows,)
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 [{rows}] vector")
    gpu = a.get_device()
    if gpu < 0 or w.get_device() != gpu or a_exps.get_device() != gpu or w_exps.get_device() != gpu \
            or (a_scale is not None and a_scale.get_device() != gpu) \
            or (w_scale is not None and w_scale.get_device() != gpu):
        raise ValueError(_ONE_GPU)
    device = a.device
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=device)
        ldo = n
        if stream is not None:
            _lend(stream, out)
    else:
        ldo = _rows_of("out", out, m, n)
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out must have out_dtype")
        if out.get_device() != gpu:
            raise ValueError(_ONE_GPU)
    lib = load()
    if ws is None:
        ws = _status_block(device)
    elif ws.get_device() != gpu:
        raise ValueError(_ONE_GPU)
    _check(lib.gptq_fp8_matmul(
        a.data_ptr(), lda, a_exps.data_ptr(), ldae,
        a_scale.data_ptr() if a_scale is not None else None, w.data_ptr(), ldw, w_exps.data_ptr(),
        ldwe, w_scale.data_ptr() if w_scale is not None else None, m, n, k, out.data_ptr(),
        _serving_dtype(out.dtype), ldo, ws.data_ptr(), ws.numel(), _stream_of(device, stream)),
        "gptq_fp8_matmul")
    return out


def kv8_cache(n_blocks, n_kv_heads, dim, device=None):
    """An empty 8-bit cache ``(k, v, k_exps, v_exps)`` of ``n_blocks`` blocks of 64 tokens: K
    codes ``[n_blocks, n_kv_heads, 64, dim]``, V codes ``[n_blocks, n_kv_heads, dim, 64]`` and
    an exponent byte per block and head for each."""
    torch = _torch()
    dev = torch.device(device) if device is not None else torch.device(
        "cuda", torch.cuda.current_device())
    k = torch.zeros(n_blocks, n_kv_heads, KV8_BLOCK, dim, dtype=torch.uint8, device=dev)
    v = torch.zeros(n_blocks, n_kv_heads, dim, KV8_BLOCK, dtype=torch.uint8, device=dev)
    exps = [torch.full((n_blocks, n_kv_heads), 127, dtype=torch.uint8, device=dev)
            for _ in range(2)]
    return (k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), *exps)


def _kv8_args(cache, table, seqs, lengths, what):
    """``(n_blocks, n_kv_heads, dim, table pitch, blocks of the table, GPU)`` of matching arguments."""
    torch = _torch()
    k, v, ke, ve = cache
    shape = k.shape
    if len(shape) != 4 or shape[2] != KV8_BLOCK:
        raise ValueError(f"cache k must be [n_blocks, n_kv_heads, {KV8_BLOCK}, dim]")
    nb, kv, _, d = shape
    if v.shape != (nb, kv, d, KV8_BLOCK) or ke.shape != (nb, kv) or ve.shape != (nb, kv):
        raise ValueError("cache v, k_exps, v_exps do not match k")
    f8, u8, i32 = torch.float8_e4m3fn, torch.uint8, torch.int32
    if k.dtype != f8 or v.dtype != f8 or ke.dtype != u8 or ve.dtype != u8:
        raise TypeError("codes are float8_e4m3fn and exponents uint8")
    if not (k.is_contiguous() and v.is_contiguous() and ke.is_contiguous()
            and ve.is_contiguous()):
        raise ValueError("the cache must be contiguous")
    if table.dtype != i32 or lengths.dtype != i32:
        raise TypeError(f"table and {what} must be int32")
    pitch = _rows_of("table", table, seqs)
    if lengths.shape != (seqs,) or not lengths.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [{seqs}] vector")
    gpu = k.get_device()
    if v.get_device() != gpu or ke.get_device() != gpu or ve.get_device() != gpu \
            or table.get_device() != gpu or lengths.get_device() != gpu:
        gpu = -1
    return nb, kv, d, pitch, table.shape[1], gpu


_Strides3 = ctypes.c_int64 * 3


def kv8_append(cache, k, v, table, start, stream=None):
    """Writes new keys and values ``[seqs, new, n_kv_heads, dim]`` into the cache at each
    sequence's tokens ``[start, start + new)``; ``table [seqs, blocks]`` (int32) names the cache
    blocks of each sequence, -1 for none."""
    shape, ks, vs = k.shape, k.stride(), v.stride()
    nb, kv, d, pitch, mb, gpu = _kv8_args(cache, table, shape[0], start, "start")
    if len(shape) != 4 or shape[2] != kv or shape[3] != d or v.shape != shape \
            or k.dtype != v.dtype:
        raise ValueError(f"k and v must be [seqs, new, {kv}, {d}] of one dtype")
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("a head's elements must be contiguous")
    if gpu < 0 or k.get_device() != gpu or v.get_device() != gpu:
        raise ValueError(_ONE_GPU)
    kc, vc, ke, ve = cache
    _check(load().gptq_kv8_append(
        k.data_ptr(), _Strides3(ks[0], ks[1], ks[2]), v.data_ptr(),
        _Strides3(vs[0], vs[1], vs[2]), _serving_dtype(k.dtype), shape[0], shape[1], kv, d,
        kc.data_ptr(), vc.data_ptr(), ke.data_ptr(), ve.data_ptr(), nb, table.data_ptr(), pitch,
        mb, start.data_ptr(), _stream_of(k.device, stream)), "gptq_kv8_append")


def kv8_attention(q, cache, table, lengths, scale=None, causal=True, out=None, ws=None,
                  stream=None):
    """Attention of the last ``new`` tokens' queries ``[seqs, new, heads, dim]`` over the cached
    tokens of each sequence (``lengths`` of them, the new ones included); ``scale`` defaults to
    ``dim ** -0.5``.  Rows that see no token give zeros.  ``ws`` as for ``fp8_matmul``."""
    torch = _torch()
    shape, qs = q.shape, q.stride()
    if len(shape) != 4 or qs[3] != 1:
        raise ValueError("q must be [seqs, new, heads, dim] with a head's elements contiguous")
    n_seq, new, heads, dim = shape
    nb, kv, d, pitch, mb, gpu = _kv8_args(cache, table, n_seq, lengths, "lengths")
    if dim != d:
        raise ValueError(f"q's heads must be {d} wide, as the cache's")
    device, dtype = q.device, q.dtype
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        os_ = out.stride()
        if stream is not None:
            _lend(stream, out)
    else:
        os_ = out.stride()
        if out.shape != shape or out.dtype != dtype or os_[3] != 1:
            raise ValueError("out must match q")
    if gpu < 0 or q.get_device() != gpu or out.get_device() != gpu \
            or (ws is not None and ws.get_device() != gpu):
        raise ValueError(_ONE_GPU)
    kc, vc, ke, ve = cache
    lib = load()
    if ws is None:
        need = lib.gptq_kv8_attention_workspace_bytes(n_seq, new, heads, kv, d, mb)
        if need <= 256:
            ws = _status_block(device)
        else:
            ws = torch.empty((need,), dtype=torch.uint8, device=device)
            if stream is not None:
                _lend(stream, ws)
    _check(lib.gptq_kv8_attention(
        q.data_ptr(), _Strides3(qs[0], qs[1], qs[2]), _serving_dtype(dtype), n_seq, new, heads,
        kv, d, kc.data_ptr(), vc.data_ptr(), ke.data_ptr(), ve.data_ptr(), nb, table.data_ptr(),
        pitch, mb, lengths.data_ptr(), 1 if causal else 0, d ** -0.5 if scale is None else scale,
        out.data_ptr(), _Strides3(os_[0], os_[1], os_[2]), ws.data_ptr(), ws.numel(),
        _stream_of(device, stream)), "gptq_kv8_attention")
    return out


# ---------------------------------------------------------------------------------------
# Feed-forward blocks of quantized layers (their marshalling is compiled, csrc/marshal.cpp)
# ---------------------------------------------------------------------------------------

_MARSHAL = None


def _marshal():
    """The compiled marshalling, loaded once and given the library's entry points."""
    global _MARSHAL
    if _MARSHAL is None:
        lib = load()
        _torch()
        if not os.path.exists(build_lib.MARSHAL):
            raise RuntimeError(f"{build_lib.MARSHAL} is missing: it must be built (build_lib.build(); needs g++ and "
                               "torch's headers)")
        built, here = build_lib.marshal_built_against(), build_lib.marshal_tag()
        if built not in (None, here):
            raise RuntimeError(f"{build_lib.MARSHAL} was built against {built}, this is {here}: it must be built again "
                               "(build_lib.build())")
        from . import _marshal as module
        module.bind(tuple(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "gptq_fp8_linear", "gptq_fp8_gated", "gptq_fp8_experts", "gptq_fp8_experts_gated",
            "gptq_moe_route", "gptq_moe_route_workspace_bytes", "gptq_moe_combine")), _check)
        _MARSHAL = module
    return _MARSHAL


def fp8_linear(a, a_exps, w, w_exps, a_scale=None, w_scale=None, bias=None, act=None, residual=None,
               out_dtype=None, out=None, ws=None, stream=None):
    """``act(diag(a_scale) A W^T diag(w_scale) + bias) + residual`` of ``fp8_matmul``'s operands,
    ``[m, n]`` in float16 or bfloat16 (the default), rounded once.  ``act``: None, "relu", "silu" or
    "gelu"; ``bias``: float32 ``[n]``; ``residual``: ``[m, n]`` of the output's dtype, which may be
    ``out`` itself.  ``ws`` as for ``fp8_matmul``."""
    return (_MARSHAL or _marshal()).fp8_linear(a, a_exps, w, w_exps, a_scale, w_scale, bias, act, residual,
                                               out_dtype, out, ws, stream)


def fp8_gated(a, a_exps, gate, up, a_scale=None, act="silu", ws=None, stream=None):
    """``(codes, exps)``, by 1 x 128 blocks, of ``act(G) * U``: G and U are the products of ``A [m, k]``
    with the weights ``gate`` and ``up``, each ``(codes [n, k], exps[, scale[, bias]])``, as
    ``fp8_linear`` takes them.  What ``fp8_matmul`` or ``fp8_linear`` take as activations (tensors of
    one storage)."""
    return (_MARSHAL or _marshal()).fp8_gated(a, a_exps, gate, up, a_scale, act, ws, stream)


def moe_route(logits, top_k, bias=None, scores="softmax", groups=1, top_groups=None, group_top=2,
              renormalize=True, scale=1.0, ws=None, stream=None):
    """Which experts each token of ``logits [tokens, experts]`` goes to: ``(ids, weights, offsets,
    order)``.

    ``ids [tokens, top_k]`` (int32): the experts of largest score (softmax or sigmoid of the logits)
    plus ``bias`` (float32 ``[experts]``), largest first, the lowest index of equals, among the
    ``top_groups`` best of ``groups`` runs of experts (by the sum of their ``group_top`` largest).
    ``weights`` (float32): their scores without the bias, over their sum with ``renormalize``, times
    ``scale``.  ``order [tokens * top_k]`` lists the assignments ``token * top_k + place`` by expert,
    expert e's from ``offsets[e]`` on: what ``fp8_experts_gated`` and ``fp8_experts`` take.
    Experts whose logit or bias is not finite are never chosen (ids of -1, weights of 0 where too few
    are left); one that only its bias leaves out keeps its part of the softmax's sum.  The four are
    tensors of one storage."""
    if scores not in SCORES:
        raise ValueError(f"scores must be one of {list(SCORES)}")
    if groups == 1:
        top_groups, group_top = 1, 1
    elif top_groups is None:
        top_groups = groups
    return (_MARSHAL or _marshal()).moe_route(logits, top_k, bias, SCORES[scores], groups, top_groups, group_top,
                                              renormalize, scale, ws, stream)


def fp8_experts_gated(a, a_exps, gate, up, offsets, order, top_k, a_scale=None, act="silu", ws=None,
                      stream=None):
    """``fp8_gated`` of each expert's tokens: ``gate`` and ``up`` are ``(codes [experts, n, k], exps[,
    scale[, bias]])``, ``a [tokens, k]``, ``offsets`` and ``order`` as ``moe_route`` returns them.  Row
    p of the codes belongs to position p of the order; rows after the last one are undefined."""
    return (_MARSHAL or _marshal()).fp8_experts_gated(a, a_exps, gate, up, offsets, order, top_k, a_scale, act, ws,
                                                      stream)


def fp8_experts(a, a_exps, w, w_exps, offsets, order, w_scale=None, bias=None, act=None,
                out_dtype=None, out=None, ws=None, stream=None):
    """Each row of ``a [rows, k]`` (in the experts' order, as ``fp8_experts_gated`` returns them) times
    its expert's weights ``w [experts, n, k]``: ``[rows, n]`` with row p at ``order[p]``, so that a
    token's rows lie together for ``moe_combine``.  Rows that the order does not name stay as they
    are.  Otherwise as ``fp8_linear``."""
    return (_MARSHAL or _marshal()).fp8_experts(a, a_exps, w, w_exps, offsets, order, w_scale, bias, act, out_dtype,
                                                out, ws, stream)


def moe_combine(y, weights, residual=None, out=None, stream=None):
    """``residual[t] + sum_j weights[t, j] y[t * top_k + j]``, ``[tokens, d]``: the experts' outputs
    ``y [tokens * top_k, d]`` with ``moe_route``'s weights.  A row whose weight is 0 is left out,
    whatever it holds.  ``out`` may be the residual."""
    return (_MARSHAL or _marshal()).moe_combine(y, weights, residual, out, stream)
