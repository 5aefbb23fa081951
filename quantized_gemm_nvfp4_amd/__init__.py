"""Python binding of libnvfp4.so (C ABI in include/nvfp4.h).

Argument marshalling only: every step of quantization and matmul runs in the
library's HIP kernels.  Torch provides device memory and the current stream;
nothing here computes on the data.  If the library is missing or the HIP
runtime cannot load it, every call raises -- there is no CPU fallback.

Function names follow the C ABI:

* ``nvfp4_quantize(x, rule=...)``     -> (codes, scales, global_scale); rule absmax /
  four_over_six / mse
* ``nvfp4_gemm(a, w, algo=AUTO)``     -> bf16 [M, N]; a, w are the 3-tuples above
* ``nvfp4_gemm_amax(a, w)``           -> (bf16 [M, N], amax slots of the output)
* ``nvfp4_quantize_amax(x, slots)``   -> nvfp4_quantize(x) with max|x| from the slots
* ``nvfp4_gemm_w4a16(x, w)``          -> bf16 [M, N]; x bf16 (weight-only NVFP4)
* ``int4g_quantize(w, group=128)``    -> (q, scales_fp16)
* ``int4g_gemv(x, q, scales, ...)``   -> bf16 [M, N]
* ``int4g_asym_quantize(w)``          -> (q, scales_fp16, zeros_u8), zero-point INT4
* ``int4g_asym_gemv(x, q, s, z)``     -> bf16 [M, N]
* ``nvfp4_linear(x, w)``              -> quantize x and multiply (one kernel at M <= 2)

The NVFP4 key/value cache and the attention that reads it:

* ``KVCache`` / ``nvfp4_kv_cache(pages, ...)`` -> the cache's buffers
* ``nvfp4_qk_norm_rope(q, k, ...)``   -> (q, k) with their head norms and positions
* ``nvfp4_kv_write(k, v, cache, slots)`` / ``nvfp4_kv_read(cache, slots)`` -> (k, v)
* ``nvfp4_qk_norm_rope_write(q, k, v, ..., cache, slots)`` -> q; both in one launch
* ``nvfp4_kv_attention(q, cache, page_table, kv_lens, ...)`` -> bf16 [T, heads, D]
"""
import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnvfp4.so")

ALGO_AUTO, ALGO_TILED, ALGO_DECODE, ALGO_SIMPLE = 0, 1, 2, 3
STATUS = {0: "NVFP4_OK", 1: "NVFP4_ERR_INVALID_ARG", 2: "NVFP4_ERR_SHAPE", 3: "NVFP4_ERR_ALIGNMENT",
          4: "NVFP4_ERR_UNSUPPORTED", 5: "NVFP4_ERR_HIP"}

# Every symbol include/nvfp4.h declares, with its ctypes signature.
_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, None
SIGNATURES = {
    "nvfp4_abi_version": ([], ctypes.c_int),
    "nvfp4_quantize_workspace_bytes": ([], ctypes.c_size_t),
    "nvfp4_quantize": ([_P, _I64, _I64, _P, _P, _P, _I, _P, _P], ctypes.c_int),
    "nvfp4_quantize_ex": ([_P, _I64, _I64, _P, _P, _P, _I, _I, _P, _P], ctypes.c_int),
    "nvfp4_quantize_noalloc": ([_P, _I64, _I64, _P, _P, _P, _I, _P], ctypes.c_int),
    "nvfp4_gemm": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "nvfp4_gemm_ex": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P], ctypes.c_int),
    "nvfp4_gemm_workspace_bytes": ([_I64, _I64, _I64], ctypes.c_size_t),
    "nvfp4_linear_workspace_bytes": ([_I64, _I64, _I64], ctypes.c_size_t),
    "nvfp4_linear": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "nvfp4_gemm_ws": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "nvfp4_gemm_amax_slots": ([_I64, _I64, _I64], ctypes.c_size_t),
    "nvfp4_gemm_amax": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_size_t, _P, _P], ctypes.c_int),
    "nvfp4_quantize_amax": ([_P, _I64, _I64, _P, _P, _P, _P, _I64, _P], ctypes.c_int),
    "nvfp4_gemm_w4a16": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "nvfp4_gemm_w4a16_ex": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P], ctypes.c_int),
    "int4g_quantize": ([_P, _I64, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "int4g_gemv": ([_P, _P, _P, _P, _I64, _I64, _I64, _I64, _P], ctypes.c_int),
    "int4g_gemv_ex": ([_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _P], ctypes.c_int),
    "int4g_asym_quantize": ([_P, _I64, _I64, _I64, _P, _P, _P, _P], ctypes.c_int),
    "int4g_asym_gemv": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P], ctypes.c_int),
    "int4g_asym_gemv_ex": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _P], ctypes.c_int),
    "nvfp4_quantize_lora_workspace_bytes": ([_I64, _I64, _I64], ctypes.c_size_t),
    "nvfp4_quantize_lora": ([_P, _I64, _I64, _P, _P, _P, _I, _P, _I64, _P, _P, _P], ctypes.c_int),
    "nvfp4_gemm_lora": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "nvfp4_gemm_lora_ex": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _I, _P], ctypes.c_int),
    "nvfp4_kv_write": ([_P, _P, _I64, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "nvfp4_kv_read": ([_P, _P, _I64, _P, _P, _P], ctypes.c_int),
    "nvfp4_qk_norm_rope": ([_P, _I64, _P, _P, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _I64, _I, _P,
                            ctypes.c_float, _I64, _P], ctypes.c_int),
    "nvfp4_qk_norm_rope_write": ([_P, _P, _I64, _P, _P, _I64, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _I, _P,
                                  ctypes.c_float, _P, _I64, _P], ctypes.c_int),
    "nvfp4_kv_attention_workspace_bytes": ([_P, _I64, _I64, _I64, _I64, _I64, _I64], ctypes.c_size_t),
    "nvfp4_kv_attention": ([_P, _P, _I64, _I64, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, ctypes.c_float, _P,
                            _P, ctypes.c_size_t, _P], ctypes.c_int),
    "nvfp4_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "nvfp4_last_error": ([], ctypes.c_char_p),
}

_lib = None


class Nvfp4Error(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def lib():
    """The loaded library (ctypes.CDLL) with argument types set."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m quantized_gemm_nvfp4_amd.build` (or __graft_entry__.build())")
        # torch first: it loads the HIP runtime it ships with, and the
        # library then binds to that same runtime (loaded the other way
        # round, torch can find no device)
        _torch()
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _check(status):
    if status != 0:
        raise Nvfp4Error(status, lib().nvfp4_last_error().decode())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _launch(index, fn, *args):
    """fn(*args, stream) on the current stream of device `index`, the one the
    operands are on, with that device current: a stream's handle (0 for the
    default one) means what it does on the current device, and kernels are
    launched there."""
    native = _torch_module._C                        # loaded with the library fn is from
    if native._cuda_getDevice() == index:
        status = fn(*args, native._cuda_getCurrentRawStream(index))
    else:
        with _torch_module.cuda.device(index):
            status = fn(*args, native._cuda_getCurrentRawStream(index))
    if status:
        _check(status)


def _need(t, dtype, shape, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda/hip) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


SCALE_RULES = {"absmax": 0, "four_over_six": 1, "mse": 2}


def nvfp4_quantize(x, global_scale=None, out=None, rule="absmax"):
    """NVFP4-quantize a bf16 [rows, cols] tensor (cols % 16 == 0).

    global_scale: optional fp32 device tensor [1] to use instead of the
    dynamic amax / 2688.  out: optional (codes, scales, global_scale) buffers.
    rule: block-scale selection, "absmax" (default), "four_over_six" or "mse".
    Returns (codes uint8 [rows, cols/2], scales uint8 [rows, cols/16],
    global_scale fp32 [1]).
    """
    torch = _torch()
    _need(x, torch.bfloat16, None, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, cols = x.shape
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
        g = global_scale if global_scale is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    else:
        codes, scales, g = out
        if global_scale is not None and g is not global_scale:
            raise ValueError("pass the given global scale as out[2]")
    _need(codes, torch.uint8, (rows, cols // 2), "codes")
    _need(scales, torch.uint8, (rows, cols // 16), "scales")
    _need(g, torch.float32, (1,), "global_scale")
    use_given = 1 if global_scale is not None else 0
    ws = None
    if not use_given:
        ws = torch.empty(lib().nvfp4_quantize_workspace_bytes(), dtype=torch.uint8, device=x.device)
    if rule not in SCALE_RULES:
        raise ValueError(f"unknown scale rule {rule!r}; one of {sorted(SCALE_RULES)}")
    _launch(x.get_device(), lib().nvfp4_quantize_ex, _ptr(x), rows, cols, _ptr(codes), _ptr(scales), _ptr(g),
            use_given, SCALE_RULES[rule], _ptr(ws) if ws is not None else None)
    return codes, scales, g


def nvfp4_gemm(a, w, algo=ALGO_AUTO, out=None, workspace=None):
    """bf16 [M, N] = g_a g_w dequant(A) . dequant(W)^T.

    a = (a_codes [M, K/2], a_scales [M, K/16], a_g [1]); w likewise with N rows.
    workspace: optional uint8 device tensor for the K split of the leftover
    tiles (nvfp4_gemm_workspace_bytes); when None one is taken from torch's
    allocator if the shape needs it.
    """
    torch = _torch()
    ac, as_, ag = a
    wc, ws, wg = w
    M, N = ac.shape[0], wc.shape[0]
    K = ac.shape[1] * 2
    _need(ac, torch.uint8, (M, K // 2), "a_codes")
    _need(as_, torch.uint8, (M, K // 16), "a_scales")
    _need(ag, torch.float32, (1,), "a_gscale")
    _need(wc, torch.uint8, (N, K // 2), "w_codes")
    _need(ws, torch.uint8, (N, K // 16), "w_scales")
    _need(wg, torch.float32, (1,), "w_gscale")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=ac.device)
    _need(out, torch.bfloat16, (M, N), "out")
    if workspace is None:
        nbytes = lib().nvfp4_gemm_workspace_bytes(M, N, K)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=ac.device)
    if workspace is not None:
        _need(workspace, torch.uint8, None, "workspace")
    _launch(ac.get_device(), lib().nvfp4_gemm_ws, _ptr(ac), _ptr(as_), _ptr(ag), _ptr(wc), _ptr(ws), _ptr(wg),
            _ptr(out), M, N, K, int(algo), _ptr(workspace) if workspace is not None else None,
            workspace.numel() if workspace is not None else 0)
    return out


def nvfp4_gemm_amax(a, w, out=None, workspace=None, slots=None):
    """nvfp4_gemm that also returns the amax slots of its output (uint32
    device tensor) for nvfp4_quantize_amax.  N % 16 == 0."""
    torch = _torch()
    ac, as_, ag = a
    wc, ws, wg = w
    M, N = ac.shape[0], wc.shape[0]
    K = ac.shape[1] * 2
    _need(ac, torch.uint8, (M, K // 2), "a_codes")
    _need(as_, torch.uint8, (M, K // 16), "a_scales")
    _need(ag, torch.float32, (1,), "a_gscale")
    _need(wc, torch.uint8, (N, K // 2), "w_codes")
    _need(ws, torch.uint8, (N, K // 16), "w_scales")
    _need(wg, torch.float32, (1,), "w_gscale")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=ac.device)
    _need(out, torch.bfloat16, (M, N), "out")
    nslots = lib().nvfp4_gemm_amax_slots(M, N, K)
    if slots is None:
        slots = torch.empty(max(1, nslots), dtype=torch.int32, device=ac.device)
    _need(slots, torch.int32, None, "slots")
    if slots.numel() < nslots:
        raise ValueError(f"slots holds {slots.numel()} values, the call writes {nslots}")
    if workspace is None:
        nbytes = lib().nvfp4_gemm_workspace_bytes(M, N, K)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=ac.device)
    if workspace is not None:
        _need(workspace, torch.uint8, None, "workspace")
    _launch(ac.get_device(), lib().nvfp4_gemm_amax, _ptr(ac), _ptr(as_), _ptr(ag), _ptr(wc), _ptr(ws), _ptr(wg),
            _ptr(out), M, N, K, _ptr(workspace) if workspace is not None else None,
            workspace.numel() if workspace is not None else 0, _ptr(slots))
    return out, slots[:nslots]


def nvfp4_quantize_amax(x, slots, out=None):
    """nvfp4_quantize(x) (absmax rule) with max|x| read from `slots` (as
    nvfp4_gemm_amax returns them for x) instead of a pass over x."""
    torch = _torch()
    _need(x, torch.bfloat16, None, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    _need(slots, torch.int32, None, "slots")
    rows, cols = x.shape
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
        g = torch.empty(1, dtype=torch.float32, device=x.device)
    else:
        codes, scales, g = out
    _need(codes, torch.uint8, (rows, cols // 2), "codes")
    _need(scales, torch.uint8, (rows, cols // 16), "scales")
    _need(g, torch.float32, (1,), "global_scale")
    _launch(x.get_device(), lib().nvfp4_quantize_amax, _ptr(x), rows, cols, _ptr(codes), _ptr(scales), _ptr(g),
            _ptr(slots), slots.numel())
    return codes, scales, g


def nvfp4_gemm_w4a16(x, w, algo=ALGO_AUTO, out=None):
    """bf16 [M, N] = g_w x . dequant(W)^T with x bf16 [M, K] (weight-only)."""
    torch = _torch()
    wc, ws, wg = w
    _need(x, torch.bfloat16, None, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    N = wc.shape[0]
    _need(wc, torch.uint8, (N, K // 2), "w_codes")
    _need(ws, torch.uint8, (N, K // 16), "w_scales")
    _need(wg, torch.float32, (1,), "w_gscale")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (M, N), "out")
    _launch(x.get_device(), lib().nvfp4_gemm_w4a16_ex, _ptr(x), _ptr(wc), _ptr(ws), _ptr(wg), _ptr(out), M, N, K,
            algo)
    return out


def nvfp4_linear(x, w, out=None, x_out=None, workspace=None):
    """Quantize bf16 x [M, K] (absmax rule, g from max|x|) and multiply by
    the NVFP4 weight w: bit-identical to nvfp4_gemm(nvfp4_quantize(x), w).

    One kernel does both when K % 128 == 0 and either M <= 2, K <= 8192 or
    3 <= M <= 16, M * K / 16 <= 3072.  x_out:
    optional (codes, scales, global_scale) buffers for x's NVFP4 form.
    Returns (out bf16 [M, N], (codes, scales, global_scale)).
    """
    torch = _torch()
    wc, ws, wg = w
    _need(x, torch.bfloat16, None, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    N = wc.shape[0]
    _need(wc, torch.uint8, (N, K // 2), "w_codes")
    _need(ws, torch.uint8, (N, K // 16), "w_scales")
    _need(wg, torch.float32, (1,), "w_gscale")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (M, N), "out")
    if x_out is None:
        x_out = (torch.empty((M, K // 2), dtype=torch.uint8, device=x.device),
                 torch.empty((M, K // 16), dtype=torch.uint8, device=x.device),
                 torch.empty(1, dtype=torch.float32, device=x.device))
    xc, xs, xg = x_out
    _need(xc, torch.uint8, (M, K // 2), "x_codes")
    _need(xs, torch.uint8, (M, K // 16), "x_scales")
    _need(xg, torch.float32, (1,), "x_gscale")
    if workspace is None:
        nbytes = lib().nvfp4_linear_workspace_bytes(M, N, K)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    if workspace is not None:
        _need(workspace, torch.uint8, None, "workspace")
    _launch(x.get_device(), lib().nvfp4_linear, _ptr(x), _ptr(wc), _ptr(ws), _ptr(wg), _ptr(out), M, N, K, _ptr(xc),
            _ptr(xs), _ptr(xg), _ptr(workspace) if workspace is not None else None,
            workspace.numel() if workspace is not None else 0)
    return out, x_out


def nvfp4_quantize_lora(x, lora_down, global_scale=None, out=None):
    """nvfp4_quantize (absmax) of x [rows, cols] plus T = x . lora_down^T.

    lora_down: bf16 [r, cols].  out: optional (codes, scales, global_scale,
    t) buffers.  Returns (codes, scales, global_scale, t fp32 [rows, r]).
    """
    torch = _torch()
    _need(x, torch.bfloat16, None, "x")
    if x.dim() != 2 or lora_down.dim() != 2:
        raise ValueError("x and lora_down must be 2-D")
    rows, cols = x.shape
    r = lora_down.shape[0]
    _need(lora_down, torch.bfloat16, (r, cols), "lora_down")
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
        g = global_scale if global_scale is not None else torch.empty(1, dtype=torch.float32, device=x.device)
        t = torch.empty((rows, r), dtype=torch.float32, device=x.device)
    else:
        codes, scales, g, t = out
        if global_scale is not None and g is not global_scale:
            raise ValueError("pass the given global scale as out[2]")
    _need(codes, torch.uint8, (rows, cols // 2), "codes")
    _need(scales, torch.uint8, (rows, cols // 16), "scales")
    _need(g, torch.float32, (1,), "global_scale")
    _need(t, torch.float32, (rows, r), "t")
    ws = torch.empty(lib().nvfp4_quantize_lora_workspace_bytes(rows, cols, r), dtype=torch.uint8, device=x.device)
    _launch(x.get_device(), lib().nvfp4_quantize_lora, _ptr(x), rows, cols, _ptr(codes), _ptr(scales), _ptr(g),
            1 if global_scale is not None else 0, _ptr(lora_down), r, _ptr(t), _ptr(ws))
    return codes, scales, g, t


def nvfp4_gemm_lora(a, w, t, lora_up, algo=ALGO_AUTO, out=None):
    """nvfp4_gemm(a, w) + t . lora_up^T, rounded once to bf16.

    t: fp32 [M, r] (from nvfp4_quantize_lora); lora_up: bf16 [N, r].
    """
    torch = _torch()
    ac, as_, ag = a
    wc, ws, wg = w
    M, N = ac.shape[0], wc.shape[0]
    K = ac.shape[1] * 2
    r = t.shape[1] if t.dim() == 2 else -1
    _need(ac, torch.uint8, (M, K // 2), "a_codes")
    _need(as_, torch.uint8, (M, K // 16), "a_scales")
    _need(ag, torch.float32, (1,), "a_gscale")
    _need(wc, torch.uint8, (N, K // 2), "w_codes")
    _need(ws, torch.uint8, (N, K // 16), "w_scales")
    _need(wg, torch.float32, (1,), "w_gscale")
    _need(t, torch.float32, (M, r), "t")
    _need(lora_up, torch.bfloat16, (N, r), "lora_up")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=ac.device)
    _need(out, torch.bfloat16, (M, N), "out")
    _launch(ac.get_device(), lib().nvfp4_gemm_lora_ex, _ptr(ac), _ptr(as_), _ptr(ag), _ptr(wc), _ptr(ws), _ptr(wg),
            _ptr(t), _ptr(lora_up), r, _ptr(out), M, N, K, int(algo))
    return out


def nvfp4_linear_lora(x, w, lora_down, lora_up, algo=ALGO_AUTO):
    """NVFP4 layer with a run-time low-rank branch: quantize x (computing
    T = x . lora_down^T in the same pass), then the GEMM with T . lora_up^T
    added before the bf16 rounding."""
    codes, scales, g, t = nvfp4_quantize_lora(x, lora_down)
    return nvfp4_gemm_lora((codes, scales, g), w, t, lora_up, algo=algo)


def int4g_quantize(w, group=128, out=None):
    """Symmetric INT4 per-group quantization of a bf16 [N, K] weight.
    Returns (q uint8 [N, K/2], scales fp16 [N, K/group])."""
    torch = _torch()
    _need(w, torch.bfloat16, None, "w")
    N, K = w.shape
    if out is None:
        q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
        s = torch.empty((N, K // group if group else 0), dtype=torch.float16, device=w.device)
    else:
        q, s = out
    _launch(w.get_device(), lib().int4g_quantize, _ptr(w), N, K, group, _ptr(q), _ptr(s))
    return q, s


def int4g_gemv(x, q, scales, group=128, algo=ALGO_AUTO, out=None):
    """W4A16: bf16 [M, N] = x . dequant(q, scales)^T."""
    torch = _torch()
    M, K = x.shape
    N = q.shape[0]
    _need(x, torch.bfloat16, (M, K), "x")
    _need(q, torch.uint8, (N, K // 2), "q")
    _need(scales, torch.float16, (N, K // group), "scales")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (M, N), "out")
    _launch(x.get_device(), lib().int4g_gemv_ex, _ptr(x), _ptr(q), _ptr(scales), _ptr(out), M, N, K, group, int(algo))
    return out


def int4g_asym_quantize(w, group=128, out=None):
    """Asymmetric (zero-point) INT4 per-group quantization of a bf16 [N, K]
    weight.  Returns (q uint8 [N, K/2], scales fp16 [N, K/128], zeros uint8
    [N, K/128])."""
    torch = _torch()
    _need(w, torch.bfloat16, None, "w")
    N, K = w.shape
    if out is None:
        q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
        s = torch.empty((N, K // group), dtype=torch.float16, device=w.device)
        z = torch.empty((N, K // group), dtype=torch.uint8, device=w.device)
    else:
        q, s, z = out
    _need(q, torch.uint8, (N, K // 2), "q")
    _need(s, torch.float16, (N, K // group), "scales")
    _need(z, torch.uint8, (N, K // group), "zeros")
    _launch(w.get_device(), lib().int4g_asym_quantize, _ptr(w), N, K, group, _ptr(q), _ptr(s), _ptr(z))
    return q, s, z


def int4g_asym_gemv(x, q, scales, zeros, group=128, algo=ALGO_AUTO, out=None):
    """bf16 [M, N] = x . (s16 (q - z))^T for the asymmetric INT4 weight."""
    torch = _torch()
    _need(x, torch.bfloat16, None, "x")
    M, K = x.shape
    N = q.shape[0]
    _need(q, torch.uint8, (N, K // 2), "q")
    _need(scales, torch.float16, (N, K // group), "scales")
    _need(zeros, torch.uint8, (N, K // group), "zeros")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (M, N), "out")
    _launch(x.get_device(), lib().int4g_asym_gemv_ex, _ptr(x), _ptr(q), _ptr(scales), _ptr(zeros), _ptr(out), M, N, K,
            group, algo)
    return out


class _CacheStruct(ctypes.Structure):
    """nvfp4_kv_cache of include/nvfp4.h."""
    _fields_ = [(n, _P) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_gscale", "v_gscale")] + \
               [(n, _I64) for n in ("num_pages", "page_size", "kv_heads", "head_dim")]


class KVCache:
    """A paged NVFP4 key/value cache: six device tensors and their sizes.

    k_codes uint8 [pages, heads, page_size, D/2], k_scales uint8 [pages, heads,
    page_size, D/16], v_codes uint8 [pages, heads, page_size/16, D/2, 16],
    v_scales uint8 [pages, heads, page_size/16, D/16, 16]; k_gscale, v_gscale
    fp32 [1].  Slot s is token s % page_size of page s // page_size.

    The attributes are fixed: calls pass a description that holds the tensors'
    addresses.  Write into the tensors in place (``cache.k_gscale.copy_(g)``),
    and make a new KVCache for other tensors or another pool.
    """

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "k_gscale", "v_gscale", "num_pages", "page_size",
                 "kv_heads", "head_dim", "device", "_index", "_struct", "_ref")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_gscale, v_gscale):
        torch = _torch()
        _need(k_codes, torch.uint8, None, "k_codes")
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, heads, page_size, head_dim/2]")
        pages, heads, ps, d2 = k_codes.shape
        _need(k_scales, torch.uint8, (pages, heads, ps, d2 // 8), "k_scales")
        _need(v_codes, torch.uint8, (pages, heads, ps // 16, d2, 16), "v_codes")
        _need(v_scales, torch.uint8, (pages, heads, ps // 16, d2 // 8, 16), "v_scales")
        _need(k_gscale, torch.float32, (1,), "k_gscale")
        _need(v_gscale, torch.float32, (1,), "v_gscale")
        for t in (k_scales, v_codes, v_scales, k_gscale, v_gscale):
            if t.device != k_codes.device:
                raise ValueError("the cache's tensors are on different devices")
        tensors = (k_codes, k_scales, v_codes, v_scales, k_gscale, v_gscale)
        struct = _CacheStruct(*(t.data_ptr() for t in tensors), pages, ps, heads, 2 * d2)
        for name, value in zip(self.__slots__, tensors + (pages, ps, heads, 2 * d2, k_codes.device, k_codes.get_device(),
                                                          struct, ctypes.addressof(struct))):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError(f"{name} of a KVCache is fixed: write into its tensors in place, or make a new KVCache")

    def __delattr__(self, name):
        raise AttributeError(f"{name} of a KVCache is fixed")

    def __reduce__(self):                        # copies describe their own tensors
        return KVCache, (self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.k_gscale, self.v_gscale)


def nvfp4_kv_cache(num_pages, page_size, kv_heads, head_dim, k_gscale=1.0, v_gscale=1.0, device="cuda"):
    """A KVCache of `num_pages` uninitialized pages.

    k_gscale, v_gscale: the global scales the rows are quantized under; a
    value of about amax / 2688 of the rows to come uses the whole scale range
    (1.0 suits rows whose block maxima lie between 0.02 and 2688).
    """
    torch = _torch()

    def buf(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=device)

    return KVCache(buf(num_pages, kv_heads, page_size, head_dim // 2), buf(num_pages, kv_heads, page_size, head_dim // 16),
                   buf(num_pages, kv_heads, page_size // 16, head_dim // 2, 16),
                   buf(num_pages, kv_heads, page_size // 16, head_dim // 16, 16),
                   *(torch.full((1,), float(g), dtype=torch.float32, device=device) for g in (k_gscale, v_gscale)))


# The checks below run on every step of a decode loop, where a call's host
# time is most of its time: one condition for the usual case, and the reason
# looked for only when it fails.

def _rows(t, heads, d, name, index):
    """(tokens, heads, token stride) of a bf16 [tokens, heads, d] tensor whose
    rows are whole (contiguous, or a view of a packed projection)."""
    torch = _torch()
    if type(t) is torch.Tensor or isinstance(t, torch.Tensor):
        if t.dtype is torch.bfloat16 and t.dim() == 3 and t.get_device() == index:
            n, h, w = t.shape
            s0, s1, s2 = t.stride()
            if w == d and s2 == 1 and (s1 == d or h == 1) and (heads is None or h == heads):
                return n, h, s0 if n > 1 else h * d
            if w != d or (heads is not None and h != heads):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [tokens, {heads or 'heads'}, {d}]")
            raise ValueError(f"{name} must have contiguous rows (strides {t.stride()})")
    else:
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda/hip) tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {torch.bfloat16}")
    if t.dim() != 3:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [tokens, {heads or 'heads'}, {d}]")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _data(t, dtype, shape, name, index):
    """Address of a contiguous device tensor of the given type and shape."""
    tensor = _torch().Tensor
    if (type(t) is tensor or isinstance(t, tensor)) and t.dtype is dtype and t.get_device() == index and \
            t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    _need(t, dtype, shape, name)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _like(t, tokens, heads, d, stride):
    """An uninitialized contiguous [tokens, heads, d] tensor of t's type and
    device (empty_like of a contiguous t costs half of what new_empty does)."""
    return _torch().empty_like(t) if stride == heads * d and t.is_contiguous() else t.new_empty((tokens, heads, d))


def nvfp4_kv_write(k, v, cache, slots):
    """Quantize k, v (bf16 [tokens, heads, D]; token strides of a packed
    projection are fine) into the cache at `slots` (int64 [tokens]; negative:
    skip).  Codes and scales are nvfp4_quantize's under the cache's global
    scales."""
    index, d = cache._index, cache.head_dim
    tokens, _, ks = _rows(k, cache.kv_heads, d, "k", index)
    v_tokens, _, vs = _rows(v, cache.kv_heads, d, "v", index)
    if v_tokens != tokens:
        raise ValueError(f"v has {v_tokens} tokens, k has {tokens}")
    sp = _data(slots, _torch().int64, (tokens,), "slots", index)
    _launch(index, lib().nvfp4_kv_write, cache._ref, k.data_ptr(), ks, v.data_ptr(), vs, sp, tokens)


def nvfp4_kv_read(cache, slots, out=None):
    """The cached rows at `slots` (int64 [tokens]) as bf16: (k, v), each
    [tokens, heads, D]; zeros where the slot is padding.  out: optional (k, v)
    buffers."""
    torch = _torch()
    index = cache._index
    sp = _data(slots, torch.int64, None, "slots", index)
    if slots.dim() != 1:
        raise ValueError("slots must be 1-D")
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    if out is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        _data(k, torch.bfloat16, shape, "k", index)
        _data(v, torch.bfloat16, shape, "v", index)
    _launch(index, lib().nvfp4_kv_read, cache._ref, sp, shape[0], k.data_ptr(), v.data_ptr())
    return k, v


def _norm_rope_args(q, k, q_weight, k_weight, cos_sin, positions):
    """The checked operands: (index, d, tokens, q heads, q stride, k heads, k
    stride, weights' addresses, table's address and sizes, positions' address)."""
    torch = _torch()
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [tokens, heads, D] tensor")
    index, d = q.get_device(), q.shape[2]
    if index < 0:
        raise ValueError("q must be a device (cuda/hip) tensor")
    tokens, hq, qs = _rows(q, None, d, "q", index)
    k_tokens, hk, ks = _rows(k, None, d, "k", index)
    if k_tokens != tokens:
        raise ValueError(f"k has {k_tokens} tokens, q has {tokens}")
    bf16 = torch.bfloat16
    qw = _data(q_weight, bf16, (d,), "q_weight", index) if q_weight is not None else None
    kw = _data(k_weight, bf16, (d,), "k_weight", index) if k_weight is not None else None
    if cos_sin is None:
        return index, d, tokens, hq, qs, hk, ks, qw, kw, None, 0, 0, None
    cp = _data(cos_sin, torch.float32, None, "cos_sin", index)
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_pos, rot_dim]")
    max_pos, rot = cos_sin.shape
    # an empty tensor's address is null, which the library takes for a missing
    # argument; it reads no position of no tokens
    pp = _data(positions, torch.int32, (tokens,), "positions", index) or cp
    return index, d, tokens, hq, qs, hk, ks, qw, kw, cp, max_pos, rot, pp


def nvfp4_qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps=1e-6, interleaved=False, out=None):
    """RMS norm of each head of q and k and the rotation of their positions,
    in one pass.

    q: bf16 [tokens, q_heads, D], k: bf16 [tokens, k_heads, D] (views of a
    packed projection are fine).  q_weight, k_weight: bf16 [D] or None.
    cos_sin: fp32 [max_pos, rot_dim], rot_dim/2 cosines then rot_dim/2 sines
    a position, or None (norm only).  positions: int32 [tokens].
    interleaved: rotate the pairs (2i, 2i + 1) instead of (i, i + rot_dim/2).
    out: optional (q, k) buffers; the inputs themselves work in place.
    Returns (q, k).
    """
    index, d, tokens, hq, qs, hk, ks, qw, kw, cp, max_pos, rot, pp = _norm_rope_args(q, k, q_weight, k_weight, cos_sin,
                                                                                     positions)
    if out is None:
        qo, ko, qos, kos = _like(q, tokens, hq, d, qs), _like(k, tokens, hk, d, ks), hq * d, hk * d
    else:
        qo, ko = out
        qn, _, qos = _rows(qo, hq, d, "out q", index)
        kn, _, kos = _rows(ko, hk, d, "out k", index)
        if qn != tokens or kn != tokens:
            raise ValueError(f"out must hold {tokens} tokens")
    _launch(index, lib().nvfp4_qk_norm_rope, q.data_ptr(), qs, qw, qo.data_ptr(), qos, hq, k.data_ptr(), ks, kw,
            ko.data_ptr(), kos, hk, d, cp, max_pos, rot, 1 if interleaved else 0, pp, eps, tokens)
    return qo, ko


def nvfp4_qk_norm_rope_write(q, k, v, q_weight, k_weight, cos_sin, positions, cache, slots, eps=1e-6,
                             interleaved=False, out=None):
    """nvfp4_qk_norm_rope with K and V going straight to the cache: one
    launch, the same q and cache bytes as nvfp4_qk_norm_rope followed by
    nvfp4_kv_write.  Returns q (out: optional buffer; q itself works)."""
    index, d, tokens, hq, qs, hk, ks, qw, kw, cp, max_pos, rot, pp = _norm_rope_args(q, k, q_weight, k_weight, cos_sin,
                                                                                     positions)
    if index != cache._index or d != cache.head_dim or hk != cache.kv_heads:
        raise ValueError(f"k is {tuple(k.shape)} on {k.device}; the cache holds {cache.kv_heads} heads of "
                         f"{cache.head_dim} on {cache.device}")
    v_tokens, _, vs = _rows(v, hk, d, "v", index)
    if v_tokens != tokens:
        raise ValueError(f"v has {v_tokens} tokens, q has {tokens}")
    sp = _data(slots, _torch().int64, (tokens,), "slots", index)
    if out is None:
        out, stride = _like(q, tokens, hq, d, qs), hq * d
    else:
        n, _, stride = _rows(out, hq, d, "out", index)
        if n != tokens:
            raise ValueError(f"out must hold {tokens} tokens")
    _launch(index, lib().nvfp4_qk_norm_rope_write, cache._ref, q.data_ptr(), qs, qw, out.data_ptr(), stride, hq,
            k.data_ptr(), ks, kw, v.data_ptr(), vs, cp, max_pos, rot, 1 if interleaved else 0, pp, eps, sp, tokens)
    return out


@functools.lru_cache(maxsize=1024)
def _attention_workspace(index, pages, page_size, heads, d, q_heads, batch, total, max_q_len, max_kv_len, prefix_len):
    """nvfp4_kv_attention_workspace_bytes; the sizes alone decide it (the
    addresses in the description are not looked at beyond being there)."""
    c = _CacheStruct(*([256] * 6), pages, page_size, heads, d)
    with _torch().cuda.device(index):
        return lib().nvfp4_kv_attention_workspace_bytes(ctypes.addressof(c), q_heads, batch, total, max_q_len, max_kv_len,
                                                        prefix_len)


def nvfp4_kv_attention(q, cache, page_table, kv_lens, q_starts=None, max_q_len=None, max_kv_len=None, prefix_pages=None,
                       prefix_len=0, scale=None, out=None, workspace=None):
    """Causal attention of new tokens over the cache: softmax(scale q K^T) V.

    q: bf16 [T, q_heads, D] (token stride of a packed projection is fine).
    page_table: int32 [batch, width]; kv_lens: int32 [batch], cached tokens of
    each sequence, its new ones included.  q_starts: int32 [batch + 1], the
    rows of q of each sequence (None: one query a sequence); max_q_len: the
    host's upper bound of a sequence's queries (default: all T, which always
    holds; a close one is faster).  max_kv_len: the host's upper bound of kv_lens
    (default: the page table's width).  prefix_pages (int32), prefix_len:
    tokens that every sequence of the batch has in front of its own; they are
    computed once for all.  scale: default D ** -0.5.  Returns bf16
    [T, q_heads, D]; zeros for a query that sees no key.
    """
    torch = _torch()
    index, d = cache._index, cache.head_dim
    total, hq, qs = _rows(q, None, d, "q", index)
    tp = _data(page_table, torch.int32, None, "page_table", index)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, width]")
    batch, width = page_table.shape
    lens = _data(kv_lens, torch.int32, (batch,), "kv_lens", index)
    starts = _data(q_starts, torch.int32, (batch + 1,), "q_starts", index) if q_starts is not None else None
    if max_q_len is None:
        max_q_len = total if starts is not None else 1
    if max_kv_len is None:
        max_kv_len = width * cache.page_size
    prefix = None
    if prefix_len > 0:
        prefix = _data(prefix_pages, torch.int32, None, "prefix_pages", index)
        need = -(-prefix_len // cache.page_size)
        if prefix_pages.numel() < need:
            raise ValueError(f"prefix_pages holds {prefix_pages.numel()} pages, {prefix_len} tokens need {need}")
    if out is None:
        out = _like(q, total, hq, d, qs)
    else:
        _data(out, torch.bfloat16, (total, hq, d), "out", index)
    if workspace is None:
        wp = None
        wn = _attention_workspace(index, cache.num_pages, cache.page_size, cache.kv_heads, d, hq, batch, total, max_q_len,
                                  max_kv_len, prefix_len)
        if wn:
            workspace = torch.empty(wn, dtype=torch.uint8, device=cache.device)
            wp = workspace.data_ptr()
    else:
        wp, wn = _data(workspace, torch.uint8, None, "workspace", index), workspace.numel()
    _launch(index, lib().nvfp4_kv_attention, cache._ref, q.data_ptr(), qs, hq, starts, batch, total, max_q_len, tp,
            width, lens, max_kv_len, prefix, prefix_len, d ** -0.5 if scale is None else scale, out.data_ptr(), wp,
            wn)
    return out
