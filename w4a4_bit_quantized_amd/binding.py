"""ctypes binding of libw4a4 (include/w4a4.h).

Argument marshalling only: dtype/device/contiguity checks on torch tensors,
output allocation with torch, the current torch stream as the HIP stream.
Every step of the computation runs in the library's HIP kernels; there is no
fallback.  The library is loaded on first use and a missing build raises.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

STATUS_NAMES = {0: "W4A4_OK", 1: "W4A4_ERR_NULL", 2: "W4A4_ERR_SHAPE", 3: "W4A4_ERR_ALIGN",
                4: "W4A4_ERR_UNSUPPORTED", 5: "W4A4_ERR_HIP", 6: "W4A4_ERR_SCRATCH"}

_c_i64 = ctypes.c_int64
_c_i32 = ctypes.c_int32
_c_p = ctypes.c_void_p


class Heads(ctypes.Structure):
    """w4a4_heads: one tensor of w4a4_qk_norm_rope."""
    _fields_ = [("x", _c_p), ("x_token_stride", _c_i64), ("x_head_stride", _c_i64), ("heads", _c_i64),
                ("weight", _c_p), ("y", _c_p), ("y_token_stride", _c_i64), ("y_head_stride", _c_i64)]


class KvCache(ctypes.Structure):
    """w4a4_kv_cache: a paged key / value cache."""
    _fields_ = [("k", _c_p), ("v", _c_p), ("pages", _c_i64), ("page_size", _c_i64), ("heads", _c_i64),
                ("k_page_stride", _c_i64), ("k_token_stride", _c_i64), ("k_head_stride", _c_i64),
                ("v_page_stride", _c_i64), ("v_token_stride", _c_i64), ("v_head_stride", _c_i64)]


class Attention(ctypes.Structure):
    """w4a4_attention: the arguments that w4a4_paged_attention and w4a4_tree_attention share."""
    _fields_ = [("q", _c_p), ("q_token_stride", _c_i64), ("q_head_stride", _c_i64),
                ("out", _c_p), ("out_token_stride", _c_i64), ("out_head_stride", _c_i64),
                ("tokens", _c_i64), ("heads", _c_i64), ("page_table", _c_p), ("table_stride", _c_i64),
                ("table_width", _c_i64), ("kv_lens", _c_p), ("q_starts", _c_p), ("batch", _c_i64), ("max_q", _c_i64),
                ("window", _c_i64), ("sinks", _c_i64), ("scale", ctypes.c_float), ("head_dim", _c_i32),
                ("dtype", _c_i32)]


# name -> (restype, argtypes), mirroring include/w4a4.h
SIGNATURES = {
    "w4a4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "w4a4_version": (ctypes.c_int, []),
    "svdq_quantize_act": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p, _c_p]),
    "svdq_quantize_weight": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "svdq_gemm_lowrank": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                         _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p]),
    "svdq_linear_workspace_bytes": (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64]),
    "svdq_linear": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                   _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "svdq_quantize_act_mx": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p,
                                            _c_p]),
    "svdq_quantize_weight_mx": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "svdq_gemm_lowrank_mx": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                            _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p]),
    "svdq_linear_mx_workspace_bytes": (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64]),
    "svdq_linear_mx": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                      _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "w4a4_hadamard_transform": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_p]),
    "svdq_gemm_lowrank_bias": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                              _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p]),
    "svdq_linear_bias": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                        _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "svdq_gemm_lowrank_mx_bias": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                                 _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p]),
    "svdq_lowrank_split": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, ctypes.c_uint64,
                                          _c_i32, _c_p, _c_p, _c_p, _c_p]),
    "svdq_linear_noalloc": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                           _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p]),
    "svdq_linear_mx_bias": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                           _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p, ctypes.c_size_t,
                                           _c_p]),
    "w8a8_quantize_act": (ctypes.c_int, [_c_p, _c_i64, _c_i32, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "w8a8_quantize_weight": (ctypes.c_int, [_c_p, _c_i64, _c_i32, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "w8a8_gemm": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_i32, _c_p]),
    "w8a8_linear_workspace_bytes": (ctypes.c_size_t, [_c_i64, _c_i64]),
    "w8a8_linear": (ctypes.c_int, [_c_p, _c_i64, _c_i32, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32,
                                   _c_p, _c_i64, _c_i32, _c_p, ctypes.c_size_t, _c_p]),
    "w4a4_qk_norm_rope": (ctypes.c_int, [ctypes.POINTER(Heads), ctypes.POINTER(Heads), _c_p, _c_i64, _c_i32, _c_i32,
                                         ctypes.POINTER(ctypes.c_int32), _c_i32, _c_i32, ctypes.c_double,
                                         ctypes.c_float, _c_i32, _c_p]),
    "w4a4_kv_append": (ctypes.c_int, [ctypes.POINTER(Heads), ctypes.POINTER(Heads), ctypes.POINTER(Heads), _c_p, _c_i64,
                                      _c_i32, _c_i32, ctypes.POINTER(ctypes.c_int32), _c_i32, _c_i32, ctypes.c_double,
                                      ctypes.c_float, _c_i32, _c_p, ctypes.POINTER(KvCache), _c_p]),
    "w4a4_attention_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Attention), ctypes.POINTER(KvCache)]),
    "w4a4_paged_attention": (ctypes.c_int, [ctypes.POINTER(Attention), ctypes.POINTER(KvCache), _c_p, ctypes.c_size_t,
                                            _c_p]),
    "w4a4_tree_attention": (ctypes.c_int, [ctypes.POINTER(Attention), ctypes.POINTER(KvCache), _c_p, _c_i64, _c_i64,
                                           _c_p, _c_p, ctypes.c_size_t, _c_p]),
}

# storage type codes of w4a4_hadamard_transform, the w8a8 entry points and w4a4_qk_norm_rope
DTYPE_BF16, DTYPE_F16, DTYPE_F32 = 0, 1, 2
HADAMARD_MAX_BLOCK = 4096


class W4A4Error(RuntimeError):
    """A libw4a4 call returned a non-OK status (or the library is missing)."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


def library_path():
    return os.environ.get("W4A4_LIBRARY", os.path.join(_HERE, "libw4a4.so"))


def test_library_path():
    """The test build (path-forcing hooks read from the environment); only tests load it."""
    return os.path.join(_HERE, "libw4a4_test.so")


def open_library(path):
    """Open one build of the library and declare its C signatures (no caching)."""
    if not os.path.exists(path):
        raise W4A4Error(f"{os.path.basename(path)} is not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load_library():
    """Load libw4a4.so (once) and declare its C signatures."""
    global _LIB
    if _LIB is None:
        _LIB = open_library(library_path())
    return _LIB


def _i32(value, name):
    """``value`` as an int that the C interface's int32 holds (ctypes drops the bits above without a word)."""
    value = int(value)
    if not -0x80000000 <= value <= 0x7FFFFFFF:
        raise ValueError(f"{name} = {value} is out of range")
    return value


def _i64(**values):
    """Refuses ints that the C interface's int64 does not hold (as ``_i32``, for arguments passed on as they are)."""
    for name, value in values.items():
        if not -2 ** 63 <= value < 2 ** 63:
            raise ValueError(f"{name} = {value} is out of range")


def _check(status, what):
    if status != 0:
        name = STATUS_NAMES.get(status, str(status))
        msg = load_library().w4a4_status_string(status).decode()
        raise W4A4Error(f"{what} failed: {name} ({msg})", status)


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dev(t, name, dtypes, device=None, dense=True):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shape(t, name, shape):
    """Raise ValueError unless tensor ``t`` has exactly ``shape`` (the C ABI sees raw pointers, so
    a mis-sized tensor would be read or written past its end)."""
    got = tuple(int(d) for d in t.shape)
    want = tuple(int(d) for d in shape)
    if got != want:
        raise ValueError(f"{name} has shape {got}, expected {want}")


def check_quantize_act_shapes(x, smooth_factor, proj_down):
    """Sizes (M, K, R) of an activation quantizer call, after checking that every tensor agrees."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D (M, K), got shape {tuple(x.shape)}")
    M, K = (int(d) for d in x.shape)
    if proj_down.dim() != 2:
        raise ValueError(f"proj_down must be 2-D (K, R), got shape {tuple(proj_down.shape)}")
    R = int(proj_down.shape[1])
    _shape(smooth_factor, "smooth_factor", (K,))
    _shape(proj_down, "proj_down", (K, R))
    return M, K, R


def check_gemm_shapes(qact, ascales, lora_act, qweight, wscales, proj_up, wcscales, wtscale, y=None, bias=None,
                      group=16, scale_rows=None):
    """Sizes (M, N, K, R) of a GEMM call, after checking every tensor against them.  ``group`` is
    16 (e4m3 scales) or 32 (E8M0); ``scale_rows`` the activation scale row count (default M)."""
    for t, n in ((qact, "qact"), (qweight, "qweight"), (proj_up, "proj_up")):
        if t.dim() != 2:
            raise ValueError(f"{n} must be 2-D, got shape {tuple(t.shape)}")
    M, K = int(qact.shape[0]), 2 * int(qact.shape[1])
    N, R = int(qweight.shape[0]), int(proj_up.shape[1])
    _shape(ascales, "ascales", (K // group, M if scale_rows is None else scale_rows))
    _shape(lora_act, "lora_act", (M, R))
    _shape(qweight, "qweight", (N, K // 2))
    _shape(wscales, "wscales", (K // group, N))
    _shape(proj_up, "proj_up", (N, R))
    _shape(wcscales, "wcscales", (N,))
    if wtscale.numel() != 1:
        raise ValueError(f"wtscale must hold one value, got shape {tuple(wtscale.shape)}")
    if y is not None:
        _shape(y, "out", (M, N))
    if bias is not None:
        _shape(bias, "bias", (N,))
    return M, N, K, R


def check_layer_shapes(M, K, layer, group=16, y=None):
    """Sizes (N, R) of a whole-layer call on an (M, K) input, after checking every checkpoint
    tensor of ``layer`` (and ``out``, ``bias``) against them."""
    qw, pu = layer["qweight"], layer["proj_up"]
    if qw.dim() != 2 or pu.dim() != 2:
        raise ValueError("qweight and proj_up must be 2-D")
    N, R = int(qw.shape[0]), int(pu.shape[1])
    _shape(qw, "qweight", (N, K // 2))
    _shape(layer["wscales"], "wscales", (K // group, N))
    _shape(layer["proj_down"], "proj_down", (K, R))
    _shape(pu, "proj_up", (N, R))
    _shape(layer["smooth_factor"], "smooth_factor", (K,))
    _shape(layer["wcscales"], "wcscales", (N,))
    if layer["wtscale"].numel() != 1:
        raise ValueError(f"wtscale must hold one value, got shape {tuple(layer['wtscale'].shape)}")
    if layer.get("bias") is not None:
        _shape(layer["bias"], "bias", (N,))
    if y is not None:
        _shape(y, "out", (M, N))
    return N, R


def _bytes_dtypes():
    torch = _torch()
    return (torch.uint8, torch.int8)


def _scale_dtypes():
    torch = _torch()
    return (torch.uint8, torch.float8_e4m3fn)


def svdq_linear_workspace_bytes(M, K, R):
    return int(load_library().svdq_linear_workspace_bytes(int(M), int(K), int(R)))


def svdq_quantize_act(x, smooth_factor, proj_down, hadamard_block=0):
    """x (M, K) bf16 -> (qact (M, K/2) u8, ascales (K/16, M) u8, lora_act (M, R) f32)."""
    torch = _torch()
    lib = load_library()
    x = _dev(x, "x", (torch.bfloat16,))
    dev = x.device
    M, K = x.shape
    _dev(smooth_factor, "smooth_factor", (torch.bfloat16,), dev)
    _dev(proj_down, "proj_down", (torch.bfloat16,), dev)
    M, K, R = check_quantize_act_shapes(x, smooth_factor, proj_down)
    qact = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    ascales = torch.empty((K // 16, M), dtype=torch.uint8, device=dev)
    lora = torch.empty((M, R), dtype=torch.float32, device=dev)
    st = lib.svdq_quantize_act(_ptr(x), _ptr(smooth_factor), _ptr(proj_down), M, K, R,
                               _i32(hadamard_block, "hadamard_block"),
                               _ptr(qact), _ptr(ascales), _ptr(lora), _stream(dev))
    _check(st, "svdq_quantize_act")
    return qact, ascales, lora


def svdq_quantize_weight(w, smooth_factor, hadamard_block=0):
    """w (N, K) bf16 -> (qweight (N, K/2) u8, wscales (K/16, N) u8)."""
    torch = _torch()
    lib = load_library()
    w = _dev(w, "w", (torch.bfloat16,))
    dev = w.device
    N, K = w.shape
    _dev(smooth_factor, "smooth_factor", (torch.bfloat16,), dev)
    _shape(smooth_factor, "smooth_factor", (K,))
    qweight = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    wscales = torch.empty((K // 16, N), dtype=torch.uint8, device=dev)
    st = lib.svdq_quantize_weight(_ptr(w), _ptr(smooth_factor), N, K, _i32(hadamard_block, "hadamard_block"),
                                  _ptr(qweight), _ptr(wscales), _stream(dev))
    _check(st, "svdq_quantize_weight")
    return qweight, wscales


def svdq_gemm_lowrank(qact, ascales, lora_act, qweight, wscales, proj_up, wcscales, wtscale, out=None, bias=None):
    """Block-scaled FP4 GEMM + epilogue -> y (M, N) bf16; ``bias`` (N,) bf16 is optional."""
    torch = _torch()
    lib = load_library()
    qact = _dev(qact, "qact", _bytes_dtypes())
    dev = qact.device
    _dev(ascales, "ascales", _scale_dtypes(), dev)
    _dev(lora_act, "lora_act", (torch.float32,), dev)
    _dev(qweight, "qweight", _bytes_dtypes(), dev)
    _dev(wscales, "wscales", _scale_dtypes(), dev)
    _dev(proj_up, "proj_up", (torch.bfloat16,), dev)
    _dev(wcscales, "wcscales", (torch.bfloat16,), dev)
    _dev(wtscale, "wtscale", (torch.bfloat16,), dev)
    if bias is not None:
        _dev(bias, "bias", (torch.bfloat16,), dev)
    M, N, K, R = check_gemm_shapes(qact, ascales, lora_act, qweight, wscales, proj_up, wcscales, wtscale, out, bias)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _dev(y, "y", (torch.bfloat16,), dev)
    if bias is None:
        st = lib.svdq_gemm_lowrank(_ptr(qact), _ptr(ascales), _ptr(lora_act), _ptr(qweight), _ptr(wscales),
                                   _ptr(proj_up), _ptr(wcscales), _ptr(wtscale), M, N, K, R, _ptr(y), _stream(dev))
    else:
        _dev(bias, "bias", (torch.bfloat16,), dev)
        st = lib.svdq_gemm_lowrank_bias(_ptr(qact), _ptr(ascales), _ptr(lora_act), _ptr(qweight), _ptr(wscales),
                                        _ptr(proj_up), _ptr(wcscales), _ptr(wtscale), _ptr(bias), M, N, K, R,
                                        _ptr(y), _stream(dev))
    _check(st, "svdq_gemm_lowrank")
    return y


LAYER_KEYS = ("qweight", "wscales", "proj_down", "proj_up", "smooth_factor", "wcscales", "wtscale")


def svdq_linear(x, layer, hadamard_block=0, workspace=None, out=None):
    """The whole W4A4 layer.  ``x`` (..., K) bf16; leading dims are flattened into M.

    ``layer`` maps the checkpoint names (qweight, wscales, proj_down, proj_up,
    smooth_factor, wcscales, wtscale) to device tensors, and optionally ``bias``
    (N,) bf16.  ``workspace`` (u8, at least svdq_linear_workspace_bytes bytes)
    and ``out`` may be passed to avoid allocation.
    """
    torch = _torch()
    lib = load_library()
    lead = x.shape[:-1]
    x2 = x.reshape(-1, x.shape[-1])
    _dev(x2, "x", (torch.bfloat16,))
    dev = x2.device
    M, K = x2.shape
    t = {k: layer[k] for k in LAYER_KEYS}
    _dev(t["qweight"], "qweight", _bytes_dtypes(), dev)
    _dev(t["wscales"], "wscales", _scale_dtypes(), dev)
    for k in ("proj_down", "proj_up", "smooth_factor", "wcscales", "wtscale"):
        _dev(t[k], k, (torch.bfloat16,), dev)
    if layer.get("bias") is not None:
        _dev(layer["bias"], "bias", (torch.bfloat16,), dev)
    N, R = check_layer_shapes(M, K, layer, group=16, y=out)
    need = int(lib.svdq_linear_workspace_bytes(M, K, R))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", (torch.uint8,), dev)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, the call needs {need}")
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _dev(y, "y", (torch.bfloat16,), dev)
    common = (_ptr(x2), _ptr(t["qweight"]), _ptr(t["wscales"]), _ptr(t["proj_down"]), _ptr(t["proj_up"]),
              _ptr(t["smooth_factor"]), _ptr(t["wcscales"]), _ptr(t["wtscale"]))
    tail = (M, N, K, R, _i32(hadamard_block, "hadamard_block"), _ptr(y), _ptr(workspace), workspace.numel(), _stream(dev))
    bias = layer.get("bias")
    if bias is None:
        st = lib.svdq_linear(*common, *tail)
    else:
        _dev(bias, "bias", (torch.bfloat16,), dev)
        st = lib.svdq_linear_bias(*common, _ptr(bias), *tail)
    _check(st, "svdq_linear")
    return y.reshape(*lead, N)


NOALLOC_SCRATCH_BYTES = 64 << 20  # W4A4_NOALLOC_SCRATCH_BYTES


def svdq_linear_noalloc(x, layer, hadamard_block=0, out=None):
    """``svdq_linear`` through the entry point without allocation: the library's static device
    workspace instead of a caller-provided one (the binding still allocates ``out`` unless given)."""
    torch = _torch()
    lib = load_library()
    lead = x.shape[:-1]
    x2 = x.reshape(-1, x.shape[-1])
    _dev(x2, "x", (torch.bfloat16,))
    dev = x2.device
    M, K = x2.shape
    t = {k: layer[k] for k in LAYER_KEYS}
    _dev(t["qweight"], "qweight", _bytes_dtypes(), dev)
    _dev(t["wscales"], "wscales", _scale_dtypes(), dev)
    for k in ("proj_down", "proj_up", "smooth_factor", "wcscales", "wtscale"):
        _dev(t[k], k, (torch.bfloat16,), dev)
    bias = layer.get("bias")
    if bias is not None:
        _dev(bias, "bias", (torch.bfloat16,), dev)
    N, R = check_layer_shapes(M, K, layer, group=16, y=out)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _dev(y, "y", (torch.bfloat16,), dev)
    st = lib.svdq_linear_noalloc(_ptr(x2), _ptr(t["qweight"]), _ptr(t["wscales"]), _ptr(t["proj_down"]),
                                 _ptr(t["proj_up"]), _ptr(t["smooth_factor"]), _ptr(t["wcscales"]), _ptr(t["wtscale"]),
                                 _ptr(bias), M, N, K, R, _i32(hadamard_block, "hadamard_block"), _ptr(y), _stream(dev))
    _check(st, "svdq_linear_noalloc")
    return y.reshape(*lead, N)


# ---- MXFP4 variant (E2M1 in blocks of 32 with one E8M0 scale per block) ---------------------

def mx_scale_rows(M):
    """Row stride of the MX activation scale tensor: M rounded up to a multiple of 4."""
    return (int(M) + 3) // 4 * 4


def svdq_linear_mx_workspace_bytes(M, K, R):
    return int(load_library().svdq_linear_mx_workspace_bytes(int(M), int(K), int(R)))


def svdq_quantize_act_mx(x, smooth_factor, proj_down, hadamard_block=32):
    """x (M, K) bf16 -> (qact (M, K/2) u8, ascales (K/32, Mp) u8 E8M0, lora_act (M, R) f32)."""
    torch = _torch()
    lib = load_library()
    x = _dev(x, "x", (torch.bfloat16,))
    dev = x.device
    M, K = x.shape
    _dev(smooth_factor, "smooth_factor", (torch.bfloat16,), dev)
    _dev(proj_down, "proj_down", (torch.bfloat16,), dev)
    M, K, R = check_quantize_act_shapes(x, smooth_factor, proj_down)
    qact = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    ascales = torch.empty((K // 32, mx_scale_rows(M)), dtype=torch.uint8, device=dev)
    lora = torch.empty((M, R), dtype=torch.float32, device=dev)
    st = lib.svdq_quantize_act_mx(_ptr(x), _ptr(smooth_factor), _ptr(proj_down), M, K, R,
                                  _i32(hadamard_block, "hadamard_block"),
                                  _ptr(qact), _ptr(ascales), _ptr(lora), _stream(dev))
    _check(st, "svdq_quantize_act_mx")
    return qact, ascales, lora


def svdq_quantize_weight_mx(w, smooth_factor, hadamard_block=32):
    """w (N, K) bf16 -> (qweight (N, K/2) u8, wscales (K/32, N) u8 E8M0)."""
    torch = _torch()
    lib = load_library()
    w = _dev(w, "w", (torch.bfloat16,))
    dev = w.device
    N, K = w.shape
    _dev(smooth_factor, "smooth_factor", (torch.bfloat16,), dev)
    _shape(smooth_factor, "smooth_factor", (K,))
    qweight = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    wscales = torch.empty((K // 32, N), dtype=torch.uint8, device=dev)
    st = lib.svdq_quantize_weight_mx(_ptr(w), _ptr(smooth_factor), N, K, _i32(hadamard_block, "hadamard_block"),
                                     _ptr(qweight), _ptr(wscales), _stream(dev))
    _check(st, "svdq_quantize_weight_mx")
    return qweight, wscales


def svdq_gemm_lowrank_mx(qact, ascales, lora_act, qweight, wscales, proj_up, wcscales, wtscale, out=None,
                         bias=None):
    """MXFP4 GEMM + epilogue -> y (M, N) bf16; ``bias`` (N,) bf16 is optional."""
    torch = _torch()
    lib = load_library()
    qact = _dev(qact, "qact", _bytes_dtypes())
    dev = qact.device
    _dev(ascales, "ascales", (torch.uint8,), dev)
    _dev(lora_act, "lora_act", (torch.float32,), dev)
    _dev(qweight, "qweight", _bytes_dtypes(), dev)
    _dev(wscales, "wscales", (torch.uint8,), dev)
    _dev(proj_up, "proj_up", (torch.bfloat16,), dev)
    _dev(wcscales, "wcscales", (torch.bfloat16,), dev)
    _dev(wtscale, "wtscale", (torch.bfloat16,), dev)
    if bias is not None:
        _dev(bias, "bias", (torch.bfloat16,), dev)
    M, N, K, R = check_gemm_shapes(qact, ascales, lora_act, qweight, wscales, proj_up, wcscales, wtscale, out, bias,
                                   group=32, scale_rows=mx_scale_rows(qact.shape[0]))
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _dev(y, "y", (torch.bfloat16,), dev)
    if bias is None:
        st = lib.svdq_gemm_lowrank_mx(_ptr(qact), _ptr(ascales), _ptr(lora_act), _ptr(qweight), _ptr(wscales),
                                      _ptr(proj_up), _ptr(wcscales), _ptr(wtscale), M, N, K, R, _ptr(y), _stream(dev))
    else:
        _dev(bias, "bias", (torch.bfloat16,), dev)
        st = lib.svdq_gemm_lowrank_mx_bias(_ptr(qact), _ptr(ascales), _ptr(lora_act), _ptr(qweight), _ptr(wscales),
                                           _ptr(proj_up), _ptr(wcscales), _ptr(wtscale), _ptr(bias), M, N, K, R,
                                           _ptr(y), _stream(dev))
    _check(st, "svdq_gemm_lowrank_mx")
    return y


def svdq_linear_mx(x, layer, hadamard_block=32, workspace=None, out=None):
    """The whole MXFP4 layer (``layer`` as for ``svdq_linear``, with MX qweight / wscales; optional ``bias``)."""
    torch = _torch()
    lib = load_library()
    lead = x.shape[:-1]
    x2 = x.reshape(-1, x.shape[-1])
    _dev(x2, "x", (torch.bfloat16,))
    dev = x2.device
    M, K = x2.shape
    t = {k: layer[k] for k in LAYER_KEYS}
    _dev(t["qweight"], "qweight", _bytes_dtypes(), dev)
    _dev(t["wscales"], "wscales", (torch.uint8,), dev)
    for k in ("proj_down", "proj_up", "smooth_factor", "wcscales", "wtscale"):
        _dev(t[k], k, (torch.bfloat16,), dev)
    if layer.get("bias") is not None:
        _dev(layer["bias"], "bias", (torch.bfloat16,), dev)
    N, R = check_layer_shapes(M, K, layer, group=32, y=out)
    need = int(lib.svdq_linear_mx_workspace_bytes(M, K, R))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", (torch.uint8,), dev)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, the call needs {need}")
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _dev(y, "y", (torch.bfloat16,), dev)
    common = (_ptr(x2), _ptr(t["qweight"]), _ptr(t["wscales"]), _ptr(t["proj_down"]), _ptr(t["proj_up"]),
              _ptr(t["smooth_factor"]), _ptr(t["wcscales"]), _ptr(t["wtscale"]))
    tail = (M, N, K, R, _i32(hadamard_block, "hadamard_block"), _ptr(y), _ptr(workspace), workspace.numel(), _stream(dev))
    bias = layer.get("bias")
    if bias is None:
        st = lib.svdq_linear_mx(*common, *tail)
    else:
        _dev(bias, "bias", (torch.bfloat16,), dev)
        st = lib.svdq_linear_mx_bias(*common, _ptr(bias), *tail)
    _check(st, "svdq_linear_mx")
    return y.reshape(*lead, N)


def _rows_view(t, name):
    """(rows, cols, row stride) of a tensor whose last dimension is dense: 2-D with any row stride
    (a column partition of a larger matrix), or any shape that flattens to rows without copying."""
    if t.dim() == 0 or t.stride(-1) != 1:
        raise ValueError(f"{name} must have a dense last dimension")
    cols = t.shape[-1]
    if t.dim() == 1:
        return 1, cols, cols
    if t.dim() == 2:
        if t.shape[0] > 1 and t.stride(0) < cols:
            raise ValueError(f"{name} rows overlap (row stride {t.stride(0)} < {cols})")
        return t.shape[0], cols, t.stride(0) if t.shape[0] > 1 else cols
    if not t.is_contiguous():
        raise ValueError(f"{name} with more than two dimensions must be contiguous")
    return t.numel() // max(cols, 1), cols, cols


def hadamard_transform(x, block=None, inplace=False, out=None):
    """Normalised block Sylvester Hadamard transform of the last dimension, per `block` columns
    (default: the whole last dimension, a power of two up to HADAMARD_MAX_BLOCK); its own inverse.

    x: bf16, f16 or f32 device tensor with a dense last dimension (a 2-D column slice such as
    y[:, start:start + length] is fine).  inplace=True writes into x and returns it; otherwise
    the result goes to `out` (same shape and dtype) or a new tensor."""
    torch = _torch()
    lib = load_library()
    codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise ValueError("x must be a device tensor")
    if x.dtype not in codes:
        raise TypeError(f"x must be bf16, f16 or f32, got {x.dtype}")
    rows, cols, ldx = _rows_view(x, "x")
    block = _i32(cols if block is None else block, "block")
    if inplace:
        y = x
    else:
        y = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else out
        if y.shape != x.shape or y.dtype != x.dtype or y.device != x.device:
            raise ValueError("out must match x in shape, dtype and device")
    _, _, ldy = _rows_view(y, "out")
    st = lib.w4a4_hadamard_transform(_ptr(x), ldx, _ptr(y), ldy, rows, cols, block, codes[x.dtype],
                                     _stream(x.device))
    _check(st, "w4a4_hadamard_transform")
    return y


def svdq_lowrank_split(w, smooth_factor, rank, oversample=16, power_iters=4, seed=0, threads=0):
    """Offline low-rank split of W * smooth_factor on the host (numpy bf16 bit patterns in, out).

    ``w`` (N, K) and ``smooth_factor`` (K,) are uint16 arrays of bf16 bits.  Returns
    (proj_down (K, R), proj_up (N, R), residual (N, K)) as uint16 bf16 bits and the R singular
    values (float32).  The residual already carries the smoothing: quantize it with a
    smooth_factor of ones."""
    import numpy as np
    lib = load_library()
    w = np.ascontiguousarray(w, dtype=np.uint16)
    lam = np.ascontiguousarray(smooth_factor, dtype=np.uint16)
    N, K = w.shape
    R = int(rank)
    pd = np.zeros((K, R), dtype=np.uint16)
    pu = np.zeros((N, R), dtype=np.uint16)
    resid = np.zeros((N, K), dtype=np.uint16)
    sv = np.zeros(max(R, 1), dtype=np.float32)
    st = lib.svdq_lowrank_split(w.ctypes.data, lam.ctypes.data, N, K, R, int(oversample), int(power_iters),
                                int(seed), int(threads), pd.ctypes.data if R else None,
                                pu.ctypes.data if R else None, resid.ctypes.data, sv.ctypes.data)
    _check(st, "svdq_lowrank_split")
    return pd, pu, resid, sv[:R]


# ---- W8A8 layer (int8, one scale per token and per output channel) --------------------------

W8A8_MAX_K = 131056

_DTYPE_CODES = {}


def _dtype_code(dtype, name):
    if not _DTYPE_CODES:
        torch = _torch()
        _DTYPE_CODES.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32})
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bf16, f16 or f32, got {dtype}")
    return code


def _device_tensor(t, name):
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    return t.device


def _dense(t, name, dtype, shape, dev):
    """``t`` is a contiguous tensor of this dtype, shape and device.  (One test in the ordinary case: small
    calls are bound by the host; the general checks word the error.)"""
    if not (isinstance(t, _torch().Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape
            and t.is_contiguous()):
        _dev(t, name, (dtype,), dev)
        _shape(t, name, shape)


def _on(dev, call, *args):
    """``call(*args, stream)`` with ``dev`` current and its current stream (a stream launches on its own
    device only while that device is current)."""
    torch = _TORCH
    index = dev.index
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the stream's handle without a Stream object
    stream = raw(index) if raw is not None else torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == index:
        return call(*args, stream)
    with torch.cuda.device(dev):
        return call(*args, stream)


def _addr(t):
    return t.data_ptr() if t is not None else None


def _w8a8_rows(t, name):
    """(rows, K, row stride, dtype code, device) of a quantizer input."""
    if isinstance(t, _torch().Tensor) and t.is_cuda and t.dim() == 2 and t.is_contiguous():
        rows, K = t.shape
        return rows, K, K, _dtype_code(t.dtype, name), t.device
    dev = _device_tensor(t, name)
    code = _dtype_code(t.dtype, name)
    rows, K, ld = _rows_view(t, name)
    return rows, K, ld, code, dev


def _check_smooth(smooth_factor, K, dev):
    if smooth_factor is not None:
        _dense(smooth_factor, "smooth_factor", _torch().bfloat16, (K,), dev)


def _check_w8a8_weights(qweight, wscales, bias, K, dev):
    torch = _torch()
    if not isinstance(qweight, torch.Tensor) or qweight.dim() != 2:
        _device_tensor(qweight, "qweight")
        raise ValueError(f"qweight must be 2-D (N, K), got shape {tuple(qweight.shape)}")
    N = qweight.shape[0]
    _dense(qweight, "qweight", torch.int8, (N, K), dev)
    _dense(wscales, "wscales", torch.float32, (N,), dev)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,), dev)
    return N


def _w8a8_out(out, x, M, N, out_dtype, default, dev):
    """(y, its row stride, its dtype code): `out` checked, or a new tensor with x's leading dimensions."""
    if out is None:
        dtype = default if out_dtype is None else out_dtype
        code = _dtype_code(dtype, "out_dtype")
        shape = (M, N) if x.dim() == 2 else (*x.shape[:-1], N)
        return x.new_empty(shape) if dtype is x.dtype else x.new_empty(shape, dtype=dtype), N, code
    if (isinstance(out, _torch().Tensor) and out.device == dev and out.shape == (M, N) and out.is_contiguous()
            and (out_dtype is None or out.dtype is out_dtype)):
        return out, N, _dtype_code(out.dtype, "out")
    lead = x.shape[:-1]
    if _device_tensor(out, "out") != dev:
        raise ValueError(f"out is on {out.device}, expected {dev}")
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must have dtype {out_dtype}, got {out.dtype}")
    if tuple(out.shape) not in ((*lead, N), (M, N)):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(*lead, N)}")
    code = _dtype_code(out.dtype, "out")
    return out, _rows_view(out, "out")[2], code


def w8a8_linear_workspace_bytes(M, K):
    return int(load_library().w8a8_linear_workspace_bytes(int(M), int(K)))


def _w8a8_quantize(call, x, name, smooth_factor, hadamard_block):
    torch = _torch()
    rows, K, ld, code, dev = _w8a8_rows(x, name)
    _check_smooth(smooth_factor, K, dev)
    q = torch.empty((rows, K), dtype=torch.int8, device=dev)
    scales = torch.empty((rows,), dtype=torch.float32, device=dev)
    st = _on(dev, call, x.data_ptr(), ld, code, _addr(smooth_factor), rows, K, _i32(hadamard_block, "hadamard_block"),
             q.data_ptr(), scales.data_ptr())
    return st, q, scales


def w8a8_quantize_act(x, smooth_factor=None, hadamard_block=0):
    """x (..., K) bf16, f16 or f32 -> (qact (M, K) int8, ascales (M,) f32), one scale per token.

    x needs a dense last dimension; a 2-D x may be a column partition of a wider matrix (16-byte
    aligned, row stride a multiple of 8).  smooth_factor (K,) bf16 is optional."""
    st, q, scales = _w8a8_quantize(load_library().w8a8_quantize_act, x, "x", smooth_factor, hadamard_block)
    _check(st, "w8a8_quantize_act")
    return q, scales


def w8a8_quantize_weight(w, smooth_factor=None, hadamard_block=0):
    """w (N, K) bf16, f16 or f32 -> (qweight (N, K) int8, wscales (N,) f32), one scale per output channel."""
    st, q, scales = _w8a8_quantize(load_library().w8a8_quantize_weight, w, "w", smooth_factor, hadamard_block)
    _check(st, "w8a8_quantize_weight")
    return q, scales


def w8a8_gemm(qact, ascales, qweight, wscales, bias=None, out=None, out_dtype=None):
    """int8 GEMM -> y (M, N): (qact @ qweight^T) * ascales[:, None] * wscales + bias.

    ``out_dtype`` is bf16 (default), f16 or f32; ``out`` may be a column partition of a wider
    matrix.  ``bias`` (N,) bf16 is optional."""
    torch = _torch()
    lib = load_library()
    dev = _device_tensor(qact, "qact")
    if qact.dim() != 2:
        raise ValueError(f"qact must be 2-D (M, K), got shape {tuple(qact.shape)}")
    M, K = qact.shape
    _dense(qact, "qact", torch.int8, (M, K), dev)
    _dense(ascales, "ascales", torch.float32, (M,), dev)
    N = _check_w8a8_weights(qweight, wscales, bias, K, dev)
    y, ldy, code = _w8a8_out(out, qact, M, N, out_dtype, torch.bfloat16, dev)
    st = _on(dev, lib.w8a8_gemm, qact.data_ptr(), ascales.data_ptr(), qweight.data_ptr(), wscales.data_ptr(),
             _addr(bias), M, N, K, y.data_ptr(), ldy, code)
    _check(st, "w8a8_gemm")
    return y


def w8a8_linear(x, layer, hadamard_block=0, workspace=None, out=None, out_dtype=None):
    """The whole 8-bit layer.  ``x`` (..., K) bf16, f16 or f32; leading dims are flattened into M.

    ``layer`` maps qweight (N, K) int8 and wscales (N,) f32, and optionally smooth_factor (K,) bf16
    and bias (N,) bf16, to device tensors.  ``out_dtype`` defaults to x's.  ``workspace`` (u8, at
    least w8a8_linear_workspace_bytes bytes) and ``out`` may be passed to avoid allocation; without
    them they come from torch's allocator on the current stream.  ``out`` shares no element with x."""
    torch = _torch()
    lib = load_library()
    M, K, ldx, code, dev = _w8a8_rows(x, "x")
    smooth, bias = layer.get("smooth_factor"), layer.get("bias")
    _check_smooth(smooth, K, dev)
    qweight, wscales = layer["qweight"], layer["wscales"]
    N = _check_w8a8_weights(qweight, wscales, bias, K, dev)
    y, ldy, ycode = _w8a8_out(out, x, M, N, out_dtype, x.dtype, dev)
    need = lib.w8a8_linear_workspace_bytes(M, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        if not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and workspace.device == dev
                and workspace.is_contiguous()):
            _dev(workspace, "workspace", (torch.uint8,), dev)
        size = workspace.numel()
        if size < need:
            raise ValueError(f"workspace holds {size} bytes, the call needs {need}")
        need = size
    st = _on(dev, lib.w8a8_linear, x.data_ptr(), ldx, code, qweight.data_ptr(), wscales.data_ptr(), _addr(smooth),
             _addr(bias), M, N, K, _i32(hadamard_block, "hadamard_block"), y.data_ptr(), ldy, ycode,
             workspace.data_ptr(), need)
    _check(st, "w8a8_linear")
    return y


# ---- q / k head norm and rotary positions ----------------------------------------------------

ROPE_LAYOUTS = {"interleaved": 0, "half": 1, "axis_half": 2}
ROPE_NORM, ROPE_SHARED_FREQUENCIES, ROPE_POSITIONS_I64 = 1, 2, 4
ROPE_MAX_HEAD_DIM, ROPE_MAX_AXES = 512, 8
_I32_ARRAYS = {}  # ctypes array types by length


def _heads_view(t, name):
    """(tokens, heads, head_dim, token stride, head stride) of a (T, H, D) or (B, S, H, D) tensor with a
    dense last dimension; the leading two of four dimensions have to flatten without copying."""
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        T, ts = shape[0], st[0]
    elif len(shape) == 4:
        T, ts = shape[1], st[1]
        if shape[0] > 1 and T > 1 and st[0] != T * st[1]:
            raise ValueError(f"{name}'s batch and token dimensions do not flatten (strides {tuple(st)})")
        if T == 1:
            ts = st[0]
        T *= shape[0]
    else:
        raise ValueError(f"{name} must be (tokens, heads, head_dim) or (batch, tokens, heads, head_dim), "
                         f"got shape {tuple(shape)}")
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have a dense last dimension")
    return T, shape[-2], shape[-1], ts, st[-2]


def _rope_side(x, view, out, weight, name, dtype, dev):
    """The descriptor of one tensor, and its output (``out``, or a new contiguous tensor)."""
    t, h, d, ts, hs = view
    if weight is not None:
        _dense(weight, f"{name}_weight", dtype, (d,), dev)
    if out is None:
        torch = _torch()
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        yts, yhs = h * d, d
    elif out is x:
        yts, yhs = ts, hs
    else:
        if not isinstance(out, _torch().Tensor) or out.shape != x.shape or out.dtype != dtype or out.device != dev:
            raise ValueError(f"the output for {name} must match it in shape, dtype and device")
        _, _, _, yts, yhs = _heads_view(out, f"{name}'s output")
    return Heads(x.data_ptr(), ts, hs, h, _addr(weight), out.data_ptr(), yts, yhs), out


def _matching_view(t, name, like, dtype, dev):
    """The view of a tensor with the tokens and head_dim of the view ``like``."""
    if _device_tensor(t, name) != dev or t.dtype != dtype:
        raise ValueError(f"q, k and v must match in dtype and device, {name} is {t.dtype} on {t.device}")
    view = _heads_view(t, name)
    if view[0] != like[0] or view[2] != like[2]:
        raise ValueError(f"{name} has {view[0]} tokens and head_dim {view[2]}, expected {like[0]} and {like[2]}")
    return view


def _rope_positions(positions, axis_dims, T, lead, dev):
    """(address or None, axis_dims as a C array, axes, flag of their type) of T tokens' checked positions."""
    n = len(axis_dims)
    pos, flag = None, 0
    if n:
        torch = _torch()
        if not isinstance(positions, torch.Tensor) or positions.device != dev or not positions.is_contiguous() or (
                positions.dtype is not torch.int32 and positions.dtype is not torch.int64):
            _dev(positions, "positions", (torch.int32, torch.int64), dev)
        shape = positions.shape
        if shape != (T, n) and shape != (*lead, n) and not (n == 1 and (shape == (T,) or shape == lead)):
            raise ValueError(f"positions has shape {tuple(shape)}, expected {(T, n)}")
        if positions.dtype is torch.int64:
            flag = ROPE_POSITIONS_I64
        pos = positions.data_ptr()
    array = _I32_ARRAYS.get(n)
    if array is None:
        array = _I32_ARRAYS[n] = ctypes.c_int32 * n
    dims = array(*axis_dims)
    if dims[:] != [*axis_dims]:  # (see _i32)
        raise ValueError(f"axis_dims {list(axis_dims)} are out of range")
    return pos, dims, n, flag


def qk_norm_rope(q, k, positions, axis_dims, q_weight=None, k_weight=None, eps=1e-6, theta=10000.0,
                 layout="interleaved", shared_frequencies=False, norm=True, inplace=False, q_out=None, k_out=None):
    """RMS norm of each head of q and k and the rotary rotation by one or more position axes, in one pass.

    q (T, Hq, D) and k (T, Hk, D), or (B, S, H, D): bf16, f16 or f32 with a dense last dimension and
    any token and head strides (partitions of a fused projection's output are fine); k may be None.
    positions (T, len(axis_dims)) int32 or int64, contiguous ((T,) for one axis, (B, S, ...) too); axis
    a rotates axis_dims[a] elements, further elements are only normed.  ``layout``: "interleaved"
    pairs (2p, 2p + 1), "half" (p, p + rot / 2), "axis_half" (halves of each axis's slice).
    ``shared_frequencies``: one ladder theta^(-2p / rot) over all pairs instead of one per axis.
    Frequencies are powers of theta only (no table of frequencies, no scaled ladders), axes take pairs in runs.
    norm=False only rotates.  q and k may be one tensor, but not ``inplace``: outputs share no element
    with each other, or with an input that is not theirs.  Returns (q_out, k_out), or q_out when k is None; new
    contiguous tensors unless ``inplace`` or given."""
    torch = _torch()
    lib = load_library()
    dev = _device_tensor(q, "q")
    dtype = q.dtype
    code = _dtype_code(dtype, "q")
    layout_code = ROPE_LAYOUTS.get(layout)
    if layout_code is None:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    view = _heads_view(q, "q")
    T, D = view[0], view[2]
    if inplace:
        if q_out is not None or k_out is not None:
            raise ValueError("inplace takes no outputs")
        q_out, k_out = q, k
    if k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k_out and k_weight need k")
    flags = (ROPE_NORM if norm else 0) | (ROPE_SHARED_FREQUENCIES if shared_frequencies else 0)
    pos, dims, n, pos_flag = _rope_positions(positions, axis_dims, T, q.shape[:-2], dev)
    qs, q_out = _rope_side(q, view, q_out, q_weight, "q", dtype, dev)
    ks = None
    if k is not None:
        ks, k_out = _rope_side(k, _matching_view(k, "k", view, dtype, dev), k_out, k_weight, "k", dtype, dev)
        ks = ctypes.byref(ks)
    st = _on(dev, lib.w4a4_qk_norm_rope, ctypes.byref(qs), ks, pos, T, D, n, dims, layout_code, flags | pos_flag, theta, eps,
             code)
    _check(st, "w4a4_qk_norm_rope")
    return q_out if k is None else (q_out, k_out)


# ---- paged key / value cache -----------------------------------------------------------------

KV_SLOTS_I64 = 8
ATTENTION_MAX_HEAD_DIM = 256


def _kv_cache(k_cache, v_cache, dtype, dev):
    """The descriptor of a cache of two (pages, page_size, heads, head_dim) tensors of this dtype and device."""
    Tensor = _torch().Tensor
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not (isinstance(t, Tensor) and t.dtype is dtype and t.device == dev):
            _dev(t, name, (dtype,), dev, dense=False)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must both be (pages, page_size, heads, head_dim), got shapes "
                         f"{tuple(shape)} and {tuple(v_cache.shape)}")
    ks, vs = k_cache.stride(), v_cache.stride()
    if (ks[3] != 1 or vs[3] != 1) and shape[3] > 1:
        raise ValueError("k_cache and v_cache must have a dense last dimension")
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), shape[0], shape[1], shape[2], *ks[:3], *vs[:3]), shape


def kv_append(q, k, v, positions, axis_dims, slots, k_cache, v_cache, q_weight=None, k_weight=None, eps=1e-6,
              theta=10000.0, layout="interleaved", shared_frequencies=False, norm=True, inplace=False, q_out=None):
    """``qk_norm_rope`` with k's result, and v as it is, stored in a paged cache, in one pass; returns q's result.

    q (T, Hq, D) or None, k and v (T, Hk, D), or (B, S, H, D): bf16 or f16, partitions of a fused projection's output
    are fine.  k_cache and v_cache (pages, page_size, Hk, D) may have any strides with a dense last dimension, whose
    elements do not overlap.  slots (T,) or (B, S) int32 or int64, contiguous: token t goes to page slots[t] // page_size,
    place slots[t] % page_size; a negative slot, or one past the pool, is not stored.  No two tokens have one
    slot.  The other arguments are ``qk_norm_rope``'s."""
    torch = _torch()
    lib = load_library()
    dev = _device_tensor(k, "k")
    dtype = k.dtype
    code = _dtype_code(dtype, "k")
    layout_code = ROPE_LAYOUTS.get(layout)
    if layout_code is None:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    view = _heads_view(k, "k")
    T, h, D, ts, hs = view
    cache, shape = _kv_cache(k_cache, v_cache, dtype, dev)
    if shape[2] != h or shape[3] != D:
        raise ValueError(f"the cache holds {shape[2]} heads of {shape[3]}, k has {h} of {D}")
    if k_weight is not None:
        _dense(k_weight, "k_weight", dtype, (D,), dev)
    ks = Heads(k.data_ptr(), ts, hs, h, _addr(k_weight), None, 0, 0)
    vv = _matching_view(v, "v", view, dtype, dev)
    if vv[1] != h:
        raise ValueError(f"v has {vv[1]} heads, expected {h}")
    vs = Heads(v.data_ptr(), vv[3], vv[4], h, None, None, 0, 0)
    lead = k.shape[:-2]
    if not (isinstance(slots, torch.Tensor) and slots.device == dev and slots.is_contiguous()
            and (slots.dtype is torch.int64 or slots.dtype is torch.int32)):
        _dev(slots, "slots", (torch.int32, torch.int64), dev)
    if slots.shape != (T,) and slots.shape != lead:
        raise ValueError(f"slots has shape {tuple(slots.shape)}, expected {(T,)}")
    flags = (ROPE_NORM if norm else 0) | (ROPE_SHARED_FREQUENCIES if shared_frequencies else 0)
    if slots.dtype is torch.int64:
        flags |= KV_SLOTS_I64
    pos, dims, n, pos_flag = _rope_positions(positions, axis_dims, T, lead, dev)
    qs = None
    if q is not None:
        if inplace:
            if q_out is not None:
                raise ValueError("inplace takes no outputs")
            q_out = q
        qs, q_out = _rope_side(q, _matching_view(q, "q", view, dtype, dev), q_out, q_weight, "q", dtype, dev)
        qs = ctypes.byref(qs)
    elif q_out is not None or q_weight is not None or inplace:
        raise ValueError("q_out, q_weight and inplace need q")
    st = _on(dev, lib.w4a4_kv_append, qs, ctypes.byref(ks), ctypes.byref(vs), pos, T, D, n, dims, layout_code,
             flags | pos_flag, theta, eps, code, slots.data_ptr(), ctypes.byref(cache))
    _check(st, "w4a4_kv_append")
    return q_out


def _attention(name, q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q, scale, window, sinks, workspace, out,
               tree):
    torch = _torch()
    Tensor = torch.Tensor
    lib = load_library()
    dev = _device_tensor(q, "q")
    dtype = q.dtype
    code = _dtype_code(dtype, "q")
    T, H, D, ts, hs = _heads_view(q, "q")
    cache, shape = _kv_cache(k_cache, v_cache, dtype, dev)
    if shape[3] != D or shape[2] == 0 or H % shape[2] != 0:
        raise ValueError(f"q has {H} heads of {D}, the cache {shape[2]} of {shape[3]}")
    if not (isinstance(page_table, Tensor) and page_table.dtype is torch.int32 and page_table.device == dev):
        _dev(page_table, "page_table", (torch.int32,), dev, dense=False)
    if page_table.dim() != 2 or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError("page_table must be (batch, pages of a sequence) with a dense last dimension")
    B, width = page_table.shape
    _dense(kv_lens, "kv_lens", torch.int32, (B,), dev)
    if q_starts is not None:
        _dense(q_starts, "q_starts", torch.int32, (B + 1,), dev)
        most = T if max_q is None else int(max_q)
    else:
        if (B and T % B) or (T and not B):
            raise ValueError(f"{T} queries are not the same number for each of {B} sequences (pass q_starts)")
        if q.dim() == 4 and q.shape[0] != B:
            raise ValueError(f"q holds {q.shape[0]} sequences, page_table {B}")
        most = T // B if B else 0
        if max_q is not None and int(max_q) < most:
            raise ValueError(f"max_q = {max_q}, but every sequence has {most} queries")
    if most < 0:
        raise ValueError(f"max_q = {max_q} is negative")
    _i64(window=window, sinks=sinks)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        ots, ohs = H * D, D
    else:
        if not isinstance(out, Tensor) or out.shape != q.shape or out.dtype is not dtype or out.device != dev:
            raise ValueError("out must match q in shape, dtype and device")
        _, _, _, ots, ohs = _heads_view(out, "out")
    a = Attention(q.data_ptr(), ts, hs, out.data_ptr(), ots, ohs, T, H, page_table.data_ptr(), page_table.stride(0), width,
                  kv_lens.data_ptr(), _addr(q_starts), B, min(most, T), window, sinks, D ** -0.5 if scale is None else scale, D, code)
    ra, rc = ctypes.byref(a), ctypes.byref(cache)
    need = lib.w4a4_attention_workspace_bytes(ra, rc)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        if not (isinstance(workspace, Tensor) and workspace.dtype is torch.uint8 and workspace.device == dev
                and workspace.is_contiguous()):
            _dev(workspace, "workspace", (torch.uint8,), dev)
        size = workspace.numel()
        if size < need:
            raise ValueError(f"workspace holds {size} bytes, the call needs {need}")
        need = size
    if tree is None:
        st = _on(dev, lib.w4a4_paged_attention, ra, rc, workspace.data_ptr(), need)
    else:
        mask, positions = tree
        if not (isinstance(mask, Tensor) and mask.device == dev and (mask.dtype is torch.bool or mask.dtype is torch.uint8)):
            _dev(mask, "tree_mask", (torch.bool, torch.uint8), dev, dense=False)
        if mask.dim() != 2 or mask.shape[0] != T or (mask.stride(1) != 1 and mask.shape[1] > 1):
            raise ValueError(f"tree_mask must be ({T}, drafted tokens) with a dense last dimension, got shape "
                             f"{tuple(mask.shape)}")
        if positions is not None:
            if not (isinstance(positions, Tensor) and positions.numel() == T):
                raise ValueError(f"positions must have {T} elements")
            _dense(positions, "positions", torch.int32, positions.shape, dev)
        elif window:
            raise ValueError("a window needs the drafted tokens' positions")
        st = _on(dev, lib.w4a4_tree_attention, ra, rc, mask.data_ptr(), mask.stride(0), mask.shape[1], _addr(positions),
                 workspace.data_ptr(), need)
    _check(st, name)
    return out


def attention_workspace_bytes(q, k_cache, v_cache, batch, max_q=None, uniform=False):
    """Bytes of workspace of ``paged_attention`` and ``tree_attention`` for q and a cache of these shapes: of a call with q_starts
    and this max_q (default T, as there), or, where ``uniform`` is set, of one without q_starts, which needs no more."""
    T, H, D, ts, hs = _heads_view(q, "q")
    cache, shape = _kv_cache(k_cache, v_cache, q.dtype, q.device)
    if shape[3] != D or shape[2] == 0 or H % shape[2] != 0:
        raise ValueError(f"q has {H} heads of {D}, the cache {shape[2]} of {shape[3]}")
    most = T if max_q is None else max_q
    _i64(batch=batch)
    if uniform:
        if batch < 0 or (batch and T % batch) or (T and not batch):
            raise ValueError(f"{T} queries are not the same number for each of {batch} sequences")
        most = T // batch if batch else 0
        if max_q is not None and max_q < most:
            raise ValueError(f"max_q = {max_q}, but every sequence has {most} queries")
    if most < 0:
        raise ValueError(f"max_q = {max_q} is negative")
    a = Attention(None, ts, hs, None, H * D, D, T, H, None, 0, 0, None, 1, batch, min(most, T), 0, 0, 1.0, D,
                  _dtype_code(q.dtype, "q"))
    need = int(load_library().w4a4_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(cache)))
    if need == 0:  # (a call that is accepted has some)
        raise ValueError(f"attention takes no {tuple(q.shape)} of {q.dtype} with strides {q.stride()}, cache {tuple(shape)} with "
                         f"{k_cache.stride()} and {v_cache.stride()}, batch {batch}")
    return need


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts=None, max_q=None, scale=None, window=0, sinks=0,
                    workspace=None, out=None):
    """Causal attention over a paged cache; a query at position p sees the keys j <= p, with a window only those with
    j > p - window or j < sinks.

    q (T, Hq, D) or (B, S, Hq, D): bf16 or f16, D a multiple of 8 up to 256, Hq a multiple of the cache's heads.
    k_cache, v_cache (pages, page_size, Hk, D) of q's dtype, any strides with a dense last dimension, 16-byte aligned rows.
    page_table (B, width) int32: key j of sequence b is in page page_table[b, j // page_size].  kv_lens (B,)
    int32: a sequence's keys, its queries' own (already appended) among them.  q_starts (B + 1,) int32: sequence b's
    queries, the last of its keys, are rows q_starts[b] .. q_starts[b + 1] - 1 of q; without it, every sequence has
    T / B.  max_q: at least the largest number of queries of a sequence (default T); it chooses the kernel, and any other value
    costs time and workspace (256 decoded tokens, 32 heads of 128 over 8: 34 MB with 1, 149 MB with the default).  scale
    defaults to D ** -0.5.  window 0 is none.  Rows that see no key, and sequences without keys, give zeros; rows of
    no sequence are not written.  ``workspace`` (u8, attention_workspace_bytes) and ``out`` may be passed to avoid
    allocation; calls that may overlap take a workspace each, and out shares no element with the inputs."""
    return _attention("w4a4_paged_attention", q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q, scale, window,
                      sinks, workspace, out, None)


def tree_attention(q, k_cache, v_cache, page_table, kv_lens, tree_mask, q_starts=None, max_q=None, positions=None,
                   scale=None, window=0, sinks=0, workspace=None, out=None):
    """Attention of drafted tokens over a paged cache that holds them as its last keys.

    Query i of sequence b sees drafted token j of the same sequence where tree_mask[q_starts[b] + i, j] is set ((T, widest
    tree) bool or uint8; the token's own bit counts too), and all keys before them: with a window those with
    j > p - window or j < sinks, where p is the query's entry of positions (T elements, int32; not less than the number of
    keys before the tree).  The other arguments are ``paged_attention``'s."""
    return _attention("w4a4_tree_attention", q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q, scale, window,
                      sinks, workspace, out, (tree_mask, positions))
