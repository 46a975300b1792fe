"""glq-b200: B200-native (sm_100a) GLQ compressed-weight linear layer.

    y = S_out . H_m . W^ . H_n . (S_in . x)

W^ is stored as 16-bit indices into a 65,536-entry E8 lattice codebook (one
per 8 weights), optionally refined by a uint8 (256-entry) or uint16 (E8)
residual index times a residual scale, times a per-layer weight scale; H is
a normalised (block-diagonal) Walsh-Hadamard transform and S_in / S_out are
random +-1 signs (GLQ project pages: glq 0.5.1 PyPI page, "How it works",
"Bit widths", "Inference kernels"; GLQ v0.3.2 release notes).

This module is argument marshalling over the C ABI of ``libglq_b200.so``
(declared in include/glq.h): every step of the layer runs in the library's
CUDA kernels.  PyTorch is used only for device memory and streams.  There is
no CPU fallback: if the library is missing, the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libglq_b200.so")

GLQ_F16, GLQ_BF16, GLQ_F32 = 0, 1, 2

STATUS = {
    0: "GLQ_OK", 1: "GLQ_ERR_INVALID_ARG", 2: "GLQ_ERR_SHAPE", 3: "GLQ_ERR_DTYPE",
    4: "GLQ_ERR_BPW", 5: "GLQ_ERR_NO_CODEBOOK", 6: "GLQ_ERR_OOM", 7: "GLQ_ERR_CUDA",
    8: "GLQ_ERR_DEVICE_CHECK", 9: "GLQ_ERR_TIMEOUT", 10: "GLQ_ERR_UNSUPPORTED", 11: "GLQ_ERR_CAPTURE",
}

# every symbol include/glq.h declares
EXPORTS = (
    "glq_status_str", "glq_version", "glq_e8_codebook", "glq_codebook_upload",
    "glq_codebook_destroy", "glq_layer_create", "glq_layer_destroy", "glq_layer_reserve",
    "glq_linear", "glq_dequant_reference", "glq_rht_input", "glq_rht_output",
    "glq_layer_check", "glq_layer_info", "glq_gemv_replay", "glq_linear_noalloc", "glq_decode_plan",
    "glq_prefill_replay", "glq_layer_set_fusion", "glq_layer_set_prefill_reconstruct",
    "glq_workspace_info", "glq_workspace_release", "glq_layer_create_stages",
    "glq_layer_set_batch_invariant", "glq_layer_create_shard", "glq_cast",
    "glq_rht_input_operand", "glq_layer_selftest_wait",
    "glq_fp8_quantize", "glq_fp8_create", "glq_fp8_destroy", "glq_fp8_reserve", "glq_fp8_linear",
    "glq_fp8_linear_quantized", "glq_fp8_dequant", "glq_fp8_check", "glq_fp8_info", "glq_fp8_selftest_wait",
    "glq_fp8_plan",
    "glq_moe_create", "glq_moe_destroy", "glq_moe_reserve", "glq_moe_forward", "glq_moe_check", "glq_moe_info",
    "glq_moe_selftest_wait",
)


class GlqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {STATUS.get(status, status)}")
        self.status = status


_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

class MoeConfig(ctypes.Structure):
    """glq_moe_config of include/glq.h."""
    _fields_ = [("experts", _i64), ("d", _i64), ("inter", _i64), ("topk", _i32), ("scoring", _i32),
                ("renormalize", _i32), ("routed_scale", ctypes.c_float)]


# argument / result types of every exported function
_SIGNATURES = {
    "glq_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "glq_version": ([], ctypes.c_char_p),
    "glq_e8_codebook": ([_vp], ctypes.c_int),
    "glq_codebook_upload": ([_vp, _i32, _i32, ctypes.POINTER(_vp)], ctypes.c_int),
    "glq_codebook_destroy": ([_vp], ctypes.c_int),
    "glq_layer_create": ([_i64, _i64, _i32, _vp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float,
                          _vp, _vp, ctypes.POINTER(_vp)], ctypes.c_int),
    "glq_layer_create_stages": ([_i64, _i64, _i32, _vp, _vp, _vp, _vp, ctypes.c_float, _vp,
                                 _vp, _vp, ctypes.POINTER(_vp)], ctypes.c_int),
    "glq_layer_create_shard": ([_i64, _i64, _i32, _vp, _vp, _vp, _vp, ctypes.c_float, _vp,
                                _vp, _vp, _i64, _i64, ctypes.POINTER(_vp)], ctypes.c_int),
    "glq_cast": ([_vp, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_layer_destroy": ([_vp], ctypes.c_int),
    "glq_layer_reserve": ([_vp, _i64], ctypes.c_int),
    "glq_linear": ([_vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_linear_noalloc": ([_vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_dequant_reference": ([_vp, _vp, _vp], ctypes.c_int),
    "glq_rht_input": ([_vp, _vp, ctypes.c_int, _vp, _i64, _vp], ctypes.c_int),
    "glq_rht_output": ([_vp, _vp, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_rht_input_operand": ([_vp, _vp, ctypes.c_int, _vp, _vp, _i64, ctypes.c_int, _vp], ctypes.c_int),
    "glq_layer_selftest_wait": ([_vp, ctypes.c_int, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_layer_check": ([_vp, _vp], ctypes.c_int),
    "glq_gemv_replay": ([_vp, _i64, _vp], ctypes.c_int),
    "glq_prefill_replay": ([_vp, _i64, _vp], ctypes.c_int),
    "glq_layer_set_fusion": ([_vp, ctypes.c_int32], ctypes.c_int),
    "glq_layer_set_prefill_reconstruct": ([_vp, _i64], ctypes.c_int),
    "glq_layer_set_batch_invariant": ([_vp, ctypes.c_int32], ctypes.c_int),
    "glq_decode_plan": ([_vp, _i64, ctypes.POINTER(_i32), ctypes.POINTER(_i32), ctypes.POINTER(_i32),
                         ctypes.POINTER(_i32), ctypes.POINTER(_i32)], ctypes.c_int),
    "glq_layer_info": ([_vp, ctypes.POINTER(_i64), ctypes.POINTER(_i64), ctypes.POINTER(_i32),
                        ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "glq_workspace_info": ([_i32, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "glq_workspace_release": ([_i32], ctypes.c_int),
    "glq_fp8_quantize": ([_vp, ctypes.c_int, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "glq_fp8_create": ([_i64, _i64, _vp, _i64, _vp, _vp, ctypes.POINTER(_vp)], ctypes.c_int),
    "glq_fp8_destroy": ([_vp], ctypes.c_int),
    "glq_fp8_reserve": ([_vp, _i64], ctypes.c_int),
    "glq_fp8_linear": ([_vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_fp8_linear_quantized": ([_vp, _vp, _vp, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_fp8_dequant": ([_vp, _vp, _vp], ctypes.c_int),
    "glq_fp8_check": ([_vp, _vp], ctypes.c_int),
    "glq_fp8_selftest_wait": ([_vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_fp8_plan": ([_vp, _i64] + [ctypes.POINTER(_i32)] * 4 + [ctypes.POINTER(_i64)], ctypes.c_int),
    "glq_fp8_info": ([_vp, ctypes.POINTER(_i64), ctypes.POINTER(_i64), ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "glq_moe_create": ([ctypes.POINTER(MoeConfig), _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_vp)], ctypes.c_int),
    "glq_moe_destroy": ([_vp], ctypes.c_int),
    "glq_moe_reserve": ([_vp, _i64], ctypes.c_int),
    "glq_moe_forward": ([_vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_moe_check": ([_vp, _vp], ctypes.c_int),
    "glq_moe_selftest_wait": ([_vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "glq_moe_info": ([_vp, ctypes.POINTER(MoeConfig), ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
}

_lib = None


def _L():
    """The loaded library (loaded on first use; raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m e8_lattice_codebook_b200.build` "
                "(the GLQ layer has no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
    return _lib


def _ok(st: int, what: str):
    if st != 0:
        raise GlqError(st, what)


# ---------------------------------------------------------------------------
# C-ABI mirrors (same names, same arguments; raw pointers and sizes)
# ---------------------------------------------------------------------------

def glq_status_str(status: int) -> str:
    return _L().glq_status_str(status).decode()


def glq_version() -> str:
    return _L().glq_version().decode()


def glq_e8_codebook() -> np.ndarray:
    """The library's 65,536 x 8 E8 codebook as fp16 bit patterns (uint16)."""
    out = np.zeros((65536, 8), dtype=np.uint16)
    _ok(_L().glq_e8_codebook(out.ctypes.data), "glq_e8_codebook")
    return out


def glq_codebook_upload(fp16_bits: np.ndarray) -> int:
    a = np.ascontiguousarray(fp16_bits, dtype=np.uint16)
    if a.ndim != 2:
        raise ValueError("codebook must be [entries][8]")
    h = _vp()
    _ok(_L().glq_codebook_upload(a.ctypes.data, a.shape[0], a.shape[1], ctypes.byref(h)), "glq_codebook_upload")
    return h.value


def glq_codebook_destroy(handle: int) -> None:
    _ok(_L().glq_codebook_destroy(handle), "glq_codebook_destroy")


def glq_layer_create(m, n, bpw, idx1, idx2, primary, residual, weight_scale, resid_scale,
                     s_in, s_out) -> int:
    idx1 = np.ascontiguousarray(idx1, dtype=np.uint16)
    if idx2 is not None:
        idx2 = np.ascontiguousarray(idx2, dtype=np.uint8 if bpw == 3 else np.uint16)
    s_in = np.ascontiguousarray(s_in, dtype=np.int8)
    s_out = np.ascontiguousarray(s_out, dtype=np.int8)
    if idx1.size != m * (n // 8) or s_in.size != n or s_out.size != m:
        raise ValueError("array sizes do not match m, n")
    if idx2 is not None and idx2.size != idx1.size:
        raise ValueError("idx2 size does not match idx1")
    h = _vp()
    _ok(_L().glq_layer_create(m, n, bpw, idx1.ctypes.data, None if idx2 is None else idx2.ctypes.data,
                          primary, residual, float(weight_scale), float(resid_scale),
                          s_in.ctypes.data, s_out.ctypes.data, ctypes.byref(h)),
        "glq_layer_create")
    return h.value


def stage_bits(bpw: int) -> list:
    """Index widths of the residual stages of a bit width (glq 0.5.1 PyPI
    page, "Bit widths"): 16-bit E8 stages, then an 8-bit stage for odd bpw."""
    if not 2 <= bpw <= 8:
        raise ValueError("bpw must be in 2..8")
    return [16] * ((bpw - 2) // 2) + ([8] if bpw % 2 else [])


def glq_layer_create_stages(m, n, bpw, idx1, idx_res, primary, residual, weight_scale, resid_scales,
                            s_in, s_out) -> int:
    """idx_res: one [m][n/8] index array per residual stage (stage order),
    resid_scales: one scale per stage."""
    bits = stage_bits(bpw)
    idx_res = list(idx_res or [])
    scales = np.ascontiguousarray(list(resid_scales or []), dtype=np.float32)
    if len(idx_res) != len(bits) or scales.size != len(bits):
        raise ValueError(f"bpw {bpw} has {len(bits)} residual stages")
    idx1 = np.ascontiguousarray(idx1, dtype=np.uint16)
    arrays = [np.ascontiguousarray(a, dtype=np.uint16 if b == 16 else np.uint8) for a, b in zip(idx_res, bits)]
    s_in = np.ascontiguousarray(s_in, dtype=np.int8)
    s_out = np.ascontiguousarray(s_out, dtype=np.int8)
    if idx1.size != m * (n // 8) or s_in.size != n or s_out.size != m or any(a.size != idx1.size for a in arrays):
        raise ValueError("array sizes do not match m, n")
    ptrs = (ctypes.c_void_p * max(1, len(arrays)))(*[a.ctypes.data for a in arrays])
    h = _vp()
    _ok(_L().glq_layer_create_stages(m, n, bpw, idx1.ctypes.data, ctypes.cast(ptrs, ctypes.c_void_p) if arrays else None,
                                     primary, residual, float(weight_scale),
                                     scales.ctypes.data if arrays else None, s_in.ctypes.data,
                                     s_out.ctypes.data, ctypes.byref(h)),
        "glq_layer_create_stages")
    return h.value


def _stage_args(m, n, bpw, idx1, idx_res, resid_scales, s_in, s_out):
    bits = stage_bits(bpw)
    idx_res = list(idx_res or [])
    scales = np.ascontiguousarray(list(resid_scales or []), dtype=np.float32)
    if len(idx_res) != len(bits) or scales.size != len(bits):
        raise ValueError(f"bpw {bpw} has {len(bits)} residual stages")
    idx1 = np.ascontiguousarray(idx1, dtype=np.uint16)
    arrays = [np.ascontiguousarray(a, dtype=np.uint16 if b == 16 else np.uint8) for a, b in zip(idx_res, bits)]
    s_in = np.ascontiguousarray(s_in, dtype=np.int8)
    s_out = np.ascontiguousarray(s_out, dtype=np.int8)
    if idx1.size != m * (n // 8) or s_in.size != n or s_out.size != m or any(a.size != idx1.size for a in arrays):
        raise ValueError("array sizes do not match m, n")
    ptrs = (ctypes.c_void_p * max(1, len(arrays)))(*[a.ctypes.data for a in arrays])
    keep = (idx1, arrays, scales, s_in, s_out, ptrs)
    return keep, (ctypes.cast(ptrs, ctypes.c_void_p) if arrays else None), (scales.ctypes.data if arrays else None)


def glq_layer_create_shard(m, n, bpw, idx1, idx_res, primary, residual, weight_scale, resid_scales,
                           s_in, s_out, k_begin, k_end) -> int:
    """The row-parallel part of a layer holding input columns [k_begin, k_end)
    (whole-layer host arrays; idx_res / resid_scales one per residual stage)."""
    keep, pres, pscales = _stage_args(m, n, bpw, idx1, idx_res, resid_scales, s_in, s_out)
    h = _vp()
    _ok(_L().glq_layer_create_shard(m, n, bpw, keep[0].ctypes.data, pres, primary, residual, float(weight_scale),
                                    pscales, keep[3].ctypes.data, keep[4].ctypes.data, int(k_begin), int(k_end),
                                    ctypes.byref(h)),
        "glq_layer_create_shard")
    return h.value


def glq_cast(src_ptr, dst_ptr, dtype, count, stream) -> None:
    _ok(_L().glq_cast(src_ptr, dst_ptr, dtype, int(count), stream), "glq_cast")


def glq_layer_destroy(handle: int) -> None:
    _ok(_L().glq_layer_destroy(handle), "glq_layer_destroy")


def glq_layer_reserve(handle: int, max_B: int) -> None:
    _ok(_L().glq_layer_reserve(handle, max_B), "glq_layer_reserve")


def glq_linear(handle, x_ptr, x_dtype, y_ptr, y_dtype, B, stream) -> None:
    _ok(_L().glq_linear(handle, x_ptr, x_dtype, y_ptr, y_dtype, B, stream), "glq_linear")


def glq_linear_noalloc(handle, x_ptr, x_dtype, y_ptr, y_dtype, B, stream) -> None:
    """glq_linear without device allocation (B <= 16; fixed 8 MiB device scratch)."""
    _ok(_L().glq_linear_noalloc(handle, x_ptr, x_dtype, y_ptr, y_dtype, B, stream),
        "glq_linear_noalloc")


def glq_dequant_reference(handle, w_ptr, stream) -> None:
    _ok(_L().glq_dequant_reference(handle, w_ptr, stream), "glq_dequant_reference")


def glq_rht_input(handle, x_ptr, x_dtype, xr_ptr, B, stream) -> None:
    _ok(_L().glq_rht_input(handle, x_ptr, x_dtype, xr_ptr, B, stream), "glq_rht_input")


def glq_rht_output(handle, z_ptr, y_ptr, y_dtype, B, stream) -> None:
    _ok(_L().glq_rht_output(handle, z_ptr, y_ptr, y_dtype, B, stream), "glq_rht_output")


def glq_rht_input_operand(handle, x_ptr, x_dtype, xh_ptr, info_ptr, B, kernel, stream) -> None:
    _ok(_L().glq_rht_input_operand(handle, x_ptr, x_dtype, xh_ptr, info_ptr, B, kernel, stream),
        "glq_rht_input_operand")


def glq_layer_selftest_wait(handle, kind, arrivals, limit, stream) -> None:
    _ok(_L().glq_layer_selftest_wait(handle, kind, arrivals, limit, stream), "glq_layer_selftest_wait")


def glq_gemv_replay(handle, B, stream) -> None:
    _ok(_L().glq_gemv_replay(handle, B, stream), "glq_gemv_replay")


def glq_prefill_replay(handle, B, stream) -> None:
    _ok(_L().glq_prefill_replay(handle, B, stream), "glq_prefill_replay")


GLQ_FUSE_INPUT, GLQ_FUSE_OUTPUT, GLQ_SPLITK_CLUSTER, GLQ_FUSE_DEFAULT = 1, 2, 4, -1


def glq_layer_set_fusion(handle, flags: int) -> None:
    _ok(_L().glq_layer_set_fusion(handle, int(flags)), "glq_layer_set_fusion")


def glq_layer_set_prefill_reconstruct(handle, min_batch: int) -> None:
    _ok(_L().glq_layer_set_prefill_reconstruct(handle, int(min_batch)), "glq_layer_set_prefill_reconstruct")


def glq_layer_set_batch_invariant(handle, enable: bool) -> None:
    _ok(_L().glq_layer_set_batch_invariant(handle, 1 if enable else 0), "glq_layer_set_batch_invariant")


def glq_layer_check(handle, stream) -> None:
    _ok(_L().glq_layer_check(handle, stream), "glq_layer_check")


def glq_decode_plan(handle, B: int) -> dict:
    vals = [_i32() for _ in range(5)]
    _ok(_L().glq_decode_plan(handle, int(B), *[ctypes.byref(v) for v in vals]), "glq_decode_plan")
    return dict(zip(("warps", "bands", "splits", "cluster", "fused_input"), (v.value for v in vals)))


def glq_workspace_info(device: int) -> int:
    """Bytes of the device's shared workspace (every layer's calls on it use it)."""
    nb = ctypes.c_size_t()
    _ok(_L().glq_workspace_info(int(device), ctypes.byref(nb)), "glq_workspace_info")
    return nb.value


def glq_workspace_release(device: int) -> None:
    _ok(_L().glq_workspace_release(int(device)), "glq_workspace_release")


def glq_layer_info(handle):
    m, n, bpw, nb = _i64(), _i64(), _i32(), ctypes.c_size_t()
    _ok(_L().glq_layer_info(handle, ctypes.byref(m), ctypes.byref(n), ctypes.byref(bpw), ctypes.byref(nb)),
        "glq_layer_info")
    return m.value, n.value, bpw.value, nb.value


def glq_fp8_quantize(x_ptr, x_dtype, B, n, q_ptr, s_ptr, stream) -> None:
    _ok(_L().glq_fp8_quantize(x_ptr, x_dtype, B, n, q_ptr, s_ptr, stream), "glq_fp8_quantize")


def glq_fp8_create(m, n, w_ptr, ldw, scales_ptr, stream) -> int:
    h = _vp()
    _ok(_L().glq_fp8_create(m, n, w_ptr, ldw, scales_ptr, stream, ctypes.byref(h)), "glq_fp8_create")
    return h.value


def glq_fp8_destroy(handle: int) -> None:
    _ok(_L().glq_fp8_destroy(handle), "glq_fp8_destroy")


def glq_fp8_reserve(handle: int, max_B: int) -> None:
    _ok(_L().glq_fp8_reserve(handle, max_B), "glq_fp8_reserve")


def glq_fp8_linear(handle, x_ptr, x_dtype, y_ptr, y_dtype, B, stream) -> None:
    _ok(_L().glq_fp8_linear(handle, x_ptr, x_dtype, y_ptr, y_dtype, B, stream), "glq_fp8_linear")


def glq_fp8_linear_quantized(handle, q_ptr, s_ptr, y_ptr, y_dtype, B, stream) -> None:
    _ok(_L().glq_fp8_linear_quantized(handle, q_ptr, s_ptr, y_ptr, y_dtype, B, stream), "glq_fp8_linear_quantized")


def glq_fp8_dequant(handle, w_ptr, stream) -> None:
    _ok(_L().glq_fp8_dequant(handle, w_ptr, stream), "glq_fp8_dequant")


def glq_fp8_check(handle, stream) -> None:
    _ok(_L().glq_fp8_check(handle, stream), "glq_fp8_check")


def glq_fp8_selftest_wait(handle, arrivals, limit, stream) -> None:
    _ok(_L().glq_fp8_selftest_wait(handle, arrivals, limit, stream), "glq_fp8_selftest_wait")


def glq_fp8_plan(handle, B) -> dict:
    kernel, cluster, clusters, ksplit, items = _i32(), _i32(), _i32(), _i32(), _i64()
    _ok(_L().glq_fp8_plan(handle, B, *(ctypes.byref(v) for v in (kernel, cluster, clusters, ksplit, items))), "glq_fp8_plan")
    return {"kernel": kernel.value, "cluster": cluster.value, "clusters": clusters.value, "ksplit": ksplit.value,
            "items": items.value}


def glq_fp8_info(handle):
    m, n, nb = _i64(), _i64(), ctypes.c_size_t()
    _ok(_L().glq_fp8_info(handle, ctypes.byref(m), ctypes.byref(n), ctypes.byref(nb)), "glq_fp8_info")
    return m.value, n.value, nb.value


GLQ_MOE_SOFTMAX, GLQ_MOE_SIGMOID = 0, 1


def glq_moe_create(config: MoeConfig, gate, gate_scales, up, up_scales, down, down_scales, stream) -> int:
    h = _vp()
    _ok(_L().glq_moe_create(ctypes.byref(config), gate, gate_scales, up, up_scales, down, down_scales, stream,
                            ctypes.byref(h)), "glq_moe_create")
    return h.value


def glq_moe_destroy(handle: int) -> None:
    _ok(_L().glq_moe_destroy(handle), "glq_moe_destroy")


def glq_moe_reserve(handle: int, max_T: int) -> None:
    _ok(_L().glq_moe_reserve(handle, max_T), "glq_moe_reserve")


def glq_moe_forward(handle, x_ptr, x_dtype, logits_ptr, logits_dtype, y_ptr, y_dtype, T, stream) -> None:
    _ok(_L().glq_moe_forward(handle, x_ptr, x_dtype, logits_ptr, logits_dtype, y_ptr, y_dtype, T, stream),
        "glq_moe_forward")


def glq_moe_check(handle, stream) -> None:
    _ok(_L().glq_moe_check(handle, stream), "glq_moe_check")


def glq_moe_selftest_wait(handle, arrivals, limit, stream) -> None:
    _ok(_L().glq_moe_selftest_wait(handle, arrivals, limit, stream), "glq_moe_selftest_wait")


def glq_moe_info(handle):
    c, nb = MoeConfig(), ctypes.c_size_t()
    _ok(_L().glq_moe_info(handle, ctypes.byref(c), ctypes.byref(nb)), "glq_moe_info")
    return {name: getattr(c, name) for name, _ in MoeConfig._fields_}, nb.value


# ---------------------------------------------------------------------------
# torch convenience (device memory and streams only)
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.float16:
        return GLQ_F16
    if dt == torch.bfloat16:
        return GLQ_BF16
    if dt == torch.float32:
        return GLQ_F32
    raise ValueError(f"unsupported dtype {dt}")


def _stream_ptr(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _torch_stream(stream, device):
    """A stream as torch's own object: any that has a `cuda_stream` is taken."""
    cuda = _torch().cuda
    return stream if isinstance(stream, cuda.Stream) else cuda.ExternalStream(stream.cuda_stream, device=device)


def _empty(shape, dtype, device, stream):
    """A call's result, allocated on the stream that will write it: a block of
    the current stream's could still be read by work queued there, which a
    call on another stream does not wait for.  The current stream is recorded
    as a reader, so that the block stays while that has work with it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(current)
    return out


def _used_on(stream, *tensors):
    """Tensors that a call on `stream` reads or writes stay while it does."""
    if stream is not None and stream.cuda_stream != _torch().cuda.current_stream(tensors[0].device).cuda_stream:
        stream = _torch_stream(stream, tensors[0].device)
        for t in tensors:
            t.record_stream(stream)


class Codebook:
    """A device codebook (65,536 x 8 E8 or 256 x 8 residual), fp16 bits on the host."""

    def __init__(self, fp16_bits: np.ndarray):
        self.entries = int(np.asarray(fp16_bits).shape[0])
        self.handle = glq_codebook_upload(fp16_bits)

    @classmethod
    def e8(cls) -> "Codebook":
        return cls(glq_e8_codebook())

    def close(self):
        if self.handle:
            glq_codebook_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GlqLinear:
    """One compressed linear layer on the current CUDA device."""

    def __init__(self, m, n, bpw, idx1, idx2, primary: Codebook, residual: Codebook | None,
                 weight_scale, resid_scale, s_in, s_out):
        """bpw 2-4: idx2 the residual index array (or None) and resid_scale
        a float; bpw 5-8: idx2 a list of the residual stages' index arrays
        and resid_scale a list of their scales (stage order); residual: the
        256-entry codebook of an odd bpw, else None (or the E8 codebook)."""
        self.m, self.n, self.bpw = int(m), int(n), int(bpw)
        self._cbs = (primary, residual)  # keep codebooks alive
        rh = 0 if residual is None else residual.handle
        if self.bpw <= 4:
            self.handle = glq_layer_create(self.m, self.n, self.bpw, idx1, idx2, primary.handle, rh,
                                           weight_scale, resid_scale, s_in, s_out)
        else:
            self.handle = glq_layer_create_stages(self.m, self.n, self.bpw, idx1, idx2, primary.handle, rh,
                                                  weight_scale, resid_scale, s_in, s_out)

    def reserve(self, max_B: int):
        glq_layer_reserve(self.handle, max_B)

    def forward(self, x, out=None, out_dtype=None, stream=None):
        torch = _torch()
        if x.dim() != 2 or x.shape[1] != self.n or not x.is_cuda or not x.is_contiguous():
            raise ValueError("x must be a contiguous CUDA tensor [B][n]")
        B = x.shape[0]
        odt = out_dtype or x.dtype
        if out is None:
            out = (torch.empty((B, self.m), dtype=odt, device=x.device) if stream is None
                   else _empty((B, self.m), odt, x.device, stream))
        if stream is not None:
            _used_on(stream, x, out)
        glq_linear(self.handle, x.data_ptr(), dtype_code(x.dtype), out.data_ptr(),
                   dtype_code(out.dtype), B, _stream_ptr(stream))
        return out

    __call__ = forward

    def dequant(self, stream=None):
        torch = _torch()
        w = _empty((self.m, self.n), torch.float32, torch.device("cuda", torch.cuda.current_device()), stream)
        glq_dequant_reference(self.handle, w.data_ptr(), _stream_ptr(stream))
        return w

    def rht_input(self, x, stream=None):
        torch = _torch()
        xr = _empty((x.shape[0], self.n), torch.float32, x.device, stream)
        _used_on(stream, x)
        glq_rht_input(self.handle, x.data_ptr(), dtype_code(x.dtype), xr.data_ptr(), x.shape[0],
                      _stream_ptr(stream))
        return xr

    RHT_AUTO, RHT_BUTTERFLY, RHT_TENSOR = 0, 1, 2  # kernels of glq_rht_input_operand

    def rht_input_operand(self, x, kernel=0, stream=None):
        """(xh [B][n_pad] fp16 = xr 2^e per row, inv [B] fp32 = 2^-e): the
        tensor-core path's input stage with the chosen kernel."""
        torch = _torch()
        n_pad = (self.n + 127) // 128 * 128
        xh = _empty((x.shape[0], n_pad), torch.float16, x.device, stream)
        info = _empty((x.shape[0], 4), torch.float32, x.device, stream)
        _used_on(stream, x)
        glq_rht_input_operand(self.handle, x.data_ptr(), dtype_code(x.dtype), xh.data_ptr(), info.data_ptr(),
                              x.shape[0], kernel, _stream_ptr(stream))
        return xh, info[:, 2]

    def selftest_wait(self, kind: int, arrivals: int, limit: int, stream=None):
        """One bounded device wait on a barrier `arrivals` of its two arrivals
        reach (kind 0: cycle-bounded, 1: cluster scope, 2: poll-bounded);
        the outcome reads back through check()."""
        glq_layer_selftest_wait(self.handle, kind, arrivals, limit, _stream_ptr(stream))

    def rht_output(self, z, out_dtype=None, stream=None):
        torch = _torch()
        y = _empty((z.shape[0], self.m), out_dtype or torch.float32, z.device, stream)
        _used_on(stream, z)
        glq_rht_output(self.handle, z.data_ptr(), y.data_ptr(), dtype_code(y.dtype), z.shape[0],
                       _stream_ptr(stream))
        return y

    def decode_plan(self, B: int) -> dict:
        return glq_decode_plan(self.handle, B)

    def gemv_replay(self, B, stream=None):
        glq_gemv_replay(self.handle, B, _stream_ptr(stream))

    def set_fusion(self, flags):
        """GLQ_FUSE_* bits; True / False mean both / neither."""
        if flags is True:
            flags = GLQ_FUSE_INPUT | GLQ_FUSE_OUTPUT
        elif flags is False:
            flags = 0
        glq_layer_set_fusion(self.handle, flags)

    def set_prefill_reconstruct(self, min_batch: int):
        """Batches >= min_batch reconstruct W in fp16 first (-1: default)."""
        glq_layer_set_prefill_reconstruct(self.handle, min_batch)

    def set_batch_invariant(self, enable: bool):
        """Every token's output independent of the batch size and path."""
        glq_layer_set_batch_invariant(self.handle, enable)

    def prefill_replay(self, B, stream=None):
        glq_prefill_replay(self.handle, B, _stream_ptr(stream))

    def check(self, stream=None):
        glq_layer_check(self.handle, _stream_ptr(stream))

    def close(self):
        if self.handle:
            glq_layer_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# 8-bit float layers
# ---------------------------------------------------------------------------

FP8_BLOCK = 128
_DTYPE_CODES = {}  # torch dtype -> code, as they are met
_E4M3_F32 = None
_HERE_ALREADY = contextlib.nullcontext()



def _fp8_blocks(v: int) -> int:
    return -(-v // FP8_BLOCK)


_raw_stream = None  # torch's raw handle of a device's current stream, bound by the first call


def _call_stream(index, stream, *tensors):
    """The raw stream of a call on device `index`; tensors used on a stream
    that is not their allocator's current one are recorded there."""
    global _raw_stream
    if _raw_stream is None:
        _raw_stream = _torch()._C._cuda_getCurrentRawStream
    current = _raw_stream(index)
    if stream is None or stream.cuda_stream == current:
        return current
    if tensors:
        _used_on(stream, *tensors)
    return stream.cuda_stream


def _fp8_dtypes():
    global _E4M3_F32
    if _E4M3_F32 is None:
        torch = _torch()
        _E4M3_F32 = (torch.float8_e4m3fn, torch.float32)
    return _E4M3_F32


def _on_device(index):
    """Makes `index` the current device, if it is not."""
    torch = _torch()
    return _HERE_ALREADY if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _dtype_code(t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        code = _DTYPE_CODES[t.dtype] = dtype_code(t.dtype)  # refuses what it does not know
    return code


def _check_input(name, t, cols, index=None):
    if t.dim() != 2 or (cols is not None and t.size(1) != cols) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor [B][{'n' if cols is None else cols}]")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the layer on cuda:{index}")


def _check_output(name, t, shape, index):
    if tuple(t.shape) != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor {list(shape)} on cuda:{index}")


def _e4m3_matrix(name, w, device, dims=2):
    """A CUDA e4m3 tensor with unit column stride and rows of 8-byte steps."""
    torch = _torch()
    if w.dim() != dims or w.dtype != torch.float8_e4m3fn:
        raise ValueError(f"{name} must be a float8_e4m3fn tensor of {dims} dimensions")
    w = w.to(device)
    packed = w.stride(-1) == 1 and w.stride(-2) >= w.shape[-1] and w.stride(-2) % 8 == 0 and w.data_ptr() % 8 == 0
    return w if packed and (dims == 2 or w.is_contiguous()) else w.clone(memory_format=torch.contiguous_format)


def _block_scales(name, s, device, shape):
    torch = _torch()
    s = s.to(device=device, dtype=torch.float32).contiguous()
    if tuple(s.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)} (one scale per {FP8_BLOCK} x {FP8_BLOCK} block), not {list(s.shape)}")
    return s


def fp8_quantize(x, q=None, s=None, stream=None):
    """Activations x [B][n] (fp16, bf16 or fp32) rounded to e4m3 with one fp32
    scale per token and group of 128 columns: (q [B][G * 128], s [G][B]), G =
    ceil(n / 128), columns of q from n zero.  Several Fp8Linear layers can
    then take them (forward_quantized).  Definition: glq_fp8_quantize."""
    _check_input("x", x, None)
    B, n, index = x.size(0), x.size(1), x.get_device()
    e4m3, f32 = _fp8_dtypes()
    G = _fp8_blocks(n)
    if q is None:
        shape = (B, G * FP8_BLOCK)
        q = x.new_empty(shape, dtype=e4m3) if stream is None else _empty(shape, e4m3, x.device, stream)
    else:
        _check_output("q", q, (B, G * FP8_BLOCK), index)
    if s is None:
        s = x.new_empty((G, B), dtype=f32) if stream is None else _empty((G, B), f32, x.device, stream)
    else:
        _check_output("s", s, (G, B), index)
    if q.dtype != e4m3 or s.dtype != f32:
        raise ValueError("q must be float8_e4m3fn and s float32")
    args = (x.data_ptr(), _dtype_code(x), B, n, q.data_ptr(), s.data_ptr(), _call_stream(index, stream, x, q, s))
    with _on_device(index):
        glq_fp8_quantize(*args)
    return q, s


class Fp8Linear:
    """A linear layer y = x W^T with e4m3 weights W [m][n] and one fp32 scale
    per 128 x 128 block; activations are rounded as fp8_quantize does.  The
    weights are copied into the layer."""

    def __init__(self, w, scales):
        """w: float8_e4m3fn [m][n] (m, n multiples of 8), scales: [ceil(m/128)]
        [ceil(n/128)].  Tensors of the CPU go to the current CUDA device.
        Reads them on the current stream and waits for it."""
        torch = _torch()
        self.handle = 0
        self.device = w.device if w.is_cuda else torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        w = _e4m3_matrix("w", w, self.device)
        self.m, self.n = int(w.shape[0]), int(w.shape[1])
        scales = _block_scales("scales", scales, self.device, (_fp8_blocks(self.m), _fp8_blocks(self.n)))
        with torch.cuda.device(self.device):
            self.handle = glq_fp8_create(self.m, self.n, w.data_ptr(), w.stride(0), scales.data_ptr(),
                                         _call_stream(self._index, None))

    def reserve(self, max_B: int):
        glq_fp8_reserve(self.handle, max_B)

    def forward(self, x, out=None, out_dtype=None, stream=None):
        """y [B][m] of x [B][n] (fp16 or bf16) in x's dtype or out_dtype
        (x's or float32)."""
        _check_input("x", x, self.n, self._index)
        B = x.size(0)
        if out is None:
            shape = (B, self.m)
            out = (x.new_empty(shape, dtype=out_dtype) if stream is None
                   else _empty(shape, out_dtype or x.dtype, x.device, stream))
        else:
            _check_output("out", out, (B, self.m), self._index)
        glq_fp8_linear(self.handle, x.data_ptr(), _dtype_code(x), out.data_ptr(), _dtype_code(out), B,
                       _call_stream(self._index, stream, x, out))
        return out

    __call__ = forward

    def forward_quantized(self, q, s, out=None, out_dtype=None, stream=None):
        """y [B][m] (bfloat16 unless out or out_dtype says otherwise) of
        activations as fp8_quantize returns them."""
        torch = _torch()
        G = _fp8_blocks(self.n)
        _check_input("q", q, G * FP8_BLOCK, self._index)
        if q.dtype != torch.float8_e4m3fn:
            raise ValueError("q must be float8_e4m3fn")
        B = q.size(0)
        _check_output("s", s, (G, B), self._index)
        if s.dtype != torch.float32:
            raise ValueError("s must be float32")
        if out is None:
            shape, dtype = (B, self.m), out_dtype or torch.bfloat16
            out = s.new_empty(shape, dtype=dtype) if stream is None else _empty(shape, dtype, s.device, stream)
        else:
            _check_output("out", out, (B, self.m), self._index)
        glq_fp8_linear_quantized(self.handle, q.data_ptr(), s.data_ptr(), out.data_ptr(), _dtype_code(out), B,
                                 _call_stream(self._index, stream, q, s, out))
        return out

    def dequant(self, stream=None):
        """The weights as fp32 [m][n]."""
        torch = _torch()
        w = _empty((self.m, self.n), torch.float32, self.device, stream)
        glq_fp8_dequant(self.handle, w.data_ptr(), _call_stream(self._index, stream, w))
        return w

    def plan(self, B: int) -> dict:
        return glq_fp8_plan(self.handle, B)

    def selftest_wait(self, arrivals: int, limit: int, stream=None):
        """One bounded wait of the kernels on a barrier `arrivals` of its two
        arrivals reach; the outcome reads back through check()."""
        glq_fp8_selftest_wait(self.handle, arrivals, limit, _call_stream(self._index, stream))

    def check(self, stream=None):
        glq_fp8_check(self.handle, _call_stream(self._index, stream))

    def close(self):
        if self.handle:
            glq_fp8_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Fp8Moe:
    """A mixture-of-experts layer for a few tokens, its experts e4m3 with one
    fp32 scale per 128 x 128 block (definition: include/glq.h, "Mixture of
    experts").  The weights are copied into the layer."""

    def __init__(self, gate, gate_scales, up, up_scales, down, down_scales, topk, renormalize=True,
                 scoring=GLQ_MOE_SOFTMAX, routed_scale=1.0):
        """gate, up: float8_e4m3fn [E][inter][d], down: [E][d][inter] (d, inter
        multiples of 8); scales [E][ceil(rows/128)][ceil(cols/128)].  Tensors
        of the CPU go to the current CUDA device.  Reads them on the current
        stream and waits for it."""
        torch = _torch()
        self.handle = 0
        self.device = gate.device if gate.is_cuda else torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        gate, up, down = (_e4m3_matrix(n, w, self.device, 3) for n, w in (("gate", gate), ("up", up), ("down", down)))
        self.experts, self.inter, self.d = (int(v) for v in gate.shape)
        if tuple(up.shape) != tuple(gate.shape) or tuple(down.shape) != (self.experts, self.d, self.inter):
            raise ValueError(f"up must be {list(gate.shape)} and down {[self.experts, self.d, self.inter]}")
        wide, high = _fp8_blocks(self.d), _fp8_blocks(self.inter)
        gate_scales = _block_scales("gate_scales", gate_scales, self.device, (self.experts, high, wide))
        up_scales = _block_scales("up_scales", up_scales, self.device, (self.experts, high, wide))
        down_scales = _block_scales("down_scales", down_scales, self.device, (self.experts, wide, high))
        self.topk = int(topk)
        config = MoeConfig(self.experts, self.d, self.inter, self.topk, int(scoring), int(bool(renormalize)),
                           float(routed_scale))
        with torch.cuda.device(self.device):
            self.handle = glq_moe_create(config, gate.data_ptr(), gate_scales.data_ptr(), up.data_ptr(),
                                         up_scales.data_ptr(), down.data_ptr(), down_scales.data_ptr(),
                                         _call_stream(self._index, None))

    def reserve(self, max_T: int):
        glq_moe_reserve(self.handle, max_T)

    def forward(self, x, logits, out=None, out_dtype=None, stream=None):
        """y [T][d] of x [T][d] (fp16 or bf16) and router logits [T][E]
        (float32 or x's dtype), in x's dtype or out_dtype (x's or float32)."""
        _check_input("x", x, self.d, self._index)
        _check_input("logits", logits, self.experts, self._index)
        T = x.size(0)
        if logits.size(0) != T:
            raise ValueError(f"logits must have {T} rows, as x has")
        if out is None:
            shape = (T, self.d)
            out = (x.new_empty(shape, dtype=out_dtype) if stream is None
                   else _empty(shape, out_dtype or x.dtype, x.device, stream))
        else:
            _check_output("out", out, (T, self.d), self._index)
        glq_moe_forward(self.handle, x.data_ptr(), _dtype_code(x), logits.data_ptr(), _dtype_code(logits),
                        out.data_ptr(), _dtype_code(out), T, _call_stream(self._index, stream, x, logits, out))
        return out

    __call__ = forward

    def selftest_wait(self, arrivals: int, limit: int, stream=None):
        """One bounded wait on the barrier between the kernel's CTAs, of which
        one (arrivals 1) or none (2) is missing; the outcome reads back through
        check(), which has to come before the next call."""
        glq_moe_selftest_wait(self.handle, arrivals, limit, _call_stream(self._index, stream))

    def check(self, stream=None):
        glq_moe_check(self.handle, _call_stream(self._index, stream))

    def close(self):
        if self.handle:
            glq_moe_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
