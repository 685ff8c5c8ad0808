"""ctypes binding of liblatent_moe.so (include/latent_moe.h), argument marshalling only.

Every function here turns torch tensors into device pointers, calls the C entry
point of the same name, and raises ``LmoeError`` on a non-zero status.  No part
of the block is computed in Python; if the shared library is missing, importing
it fails loudly (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblatent_moe.so")

LMOE_F32, LMOE_BF16, LMOE_NVFP4 = 0, 1, 2
_DT = {"f32": LMOE_F32, "bf16": LMOE_BF16, "nvfp4": LMOE_NVFP4}

STATUS = {0: "LMOE_OK", -1: "LMOE_ERR_ARG", -2: "LMOE_ERR_UNSUPPORTED", -3: "LMOE_ERR_ALIGN",
          -4: "LMOE_ERR_WORKSPACE", -5: "LMOE_ERR_CUDA", -6: "LMOE_ERR_TIMEOUT"}


class LmoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_lib().lmoe_status_string(status).decode()})")


class lmoe_config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d_model", ctypes.c_int), ("d_latent", ctypes.c_int),
                ("n_experts", ctypes.c_int), ("d_ff", ctypes.c_int), ("top_k", ctypes.c_int),
                ("eps", ctypes.c_float), ("act_dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int)]


SCALES_ROW_MAJOR, SCALES_BLOCKED = 0, 1   # lmoe_nvfp4_scale_layout


class lmoe_nvfp4_weight(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("scale_layout", ctypes.c_int)]


class lmoe_ex(ctypes.Structure):
    _fields_ = [("router_bias", ctypes.c_void_p), ("forced_idx", ctypes.c_void_p),
                ("topk_idx_out", ctypes.c_void_p), ("topk_w_out", ctypes.c_void_p),
                ("near_tie_count_out", ctypes.c_void_p), ("wait_budget_cycles", ctypes.c_longlong),
                ("stage_events", ctypes.c_void_p), ("next_norm_gamma", ctypes.c_void_p),
                ("next_norm_out", ctypes.c_void_p), ("single_token_path", ctypes.c_int),
                ("separate_expert_gemms", ctypes.c_int), ("cooperative_launch", ctypes.c_int)]

SINGLE_TOKEN_DEFAULT, SINGLE_TOKEN_KERNEL, SINGLE_TOKEN_CHAIN = 0, 1, 2   # lmoe_ex.single_token_path

STAGES = ["prenorm", "router", "topk", "permute", "pooler", "poolnorm", "gate_up", "down", "combine",
          "unpooler", "postnorm"]
NUM_STAGE_EVENTS = len(STAGES) + 1


_LAYOUT_FIELDS = ["xa", "logits", "topk_idx", "topk_w", "counts", "offsets", "row_of", "tok_of",
                  "tiles", "n_tiles", "p", "ss_p", "xe", "xe_scale", "h", "y", "ss_y", "c", "u",
                  "ss_u", "err", "total"]


_LAYOUT_FIELDS_NVFP4 = ["xq", "xq_scale", "xq_rowscale", "xe_rowscale", "h_scale", "c_scale", "c_rowscale"]


class lmoe_fp8_matmul(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("N", ctypes.c_int), ("K", ctypes.c_int), ("n_experts", ctypes.c_int),
                ("a_format", ctypes.c_int), ("b_format", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("accumulate", ctypes.c_int), ("wait_budget_cycles", ctypes.c_longlong),
                ("unpadded_rows", ctypes.c_longlong)]


class lmoe_workspace_layout(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_longlong) for f in _LAYOUT_FIELDS + _LAYOUT_FIELDS_NVFP4]
                + [("xa_cols", ctypes.c_int), ("grouped_splits", ctypes.c_longlong)])


_P = ctypes.c_void_p
_FWD_ARGS = [ctypes.POINTER(lmoe_config), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
             ctypes.c_int, _P, _P, ctypes.c_size_t, _P]
_lib_handle = None


def _lib():
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run latent_mixture_experts_router_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.lmoe_status_string.restype = ctypes.c_char_p
        L.lmoe_status_string.argtypes = [ctypes.c_int]
        for name in ("lmoe_workspace_size", "lmoe_workspace_size_host_io"):
            getattr(L, name).argtypes = [ctypes.POINTER(lmoe_config), ctypes.POINTER(ctypes.c_size_t)]
            getattr(L, name).restype = ctypes.c_int
        L.lmoe_get_workspace_layout.argtypes = [ctypes.POINTER(lmoe_config), ctypes.POINTER(lmoe_workspace_layout)]
        L.lmoe_get_workspace_layout.restype = ctypes.c_int
        L.latent_moe_forward.argtypes = _FWD_ARGS
        L.latent_moe_forward.restype = ctypes.c_int
        L.latent_moe_forward_ex.argtypes = _FWD_ARGS + [ctypes.POINTER(lmoe_ex)]
        L.latent_moe_forward_ex.restype = ctypes.c_int
        L.latent_moe_forward_host_io.argtypes = _FWD_ARGS
        L.latent_moe_forward_host_io.restype = ctypes.c_int
        L.latent_moe_forward_host_io_ex.argtypes = _FWD_ARGS + [ctypes.POINTER(lmoe_ex)]
        L.latent_moe_forward_host_io_ex.restype = ctypes.c_int
        L.lmoe_check_status.argtypes = [ctypes.POINTER(lmoe_config), _P, _P, ctypes.POINTER(ctypes.c_uint32)]
        L.lmoe_check_status.restype = ctypes.c_int
        L.lmoe_wait_selftest.argtypes = [ctypes.POINTER(lmoe_config), _P, ctypes.c_longlong, _P]
        L.lmoe_wait_selftest.restype = ctypes.c_int
        L.lmoe_expert_pair.argtypes = [ctypes.POINTER(lmoe_config), ctypes.POINTER(ctypes.c_int)]
        L.lmoe_expert_pair.restype = ctypes.c_int
        I, LL = ctypes.c_int, ctypes.c_longlong
        L.lmoe_router_losses_workspace_size.argtypes = [I, I, ctypes.POINTER(ctypes.c_size_t)]
        L.lmoe_router_losses.argtypes = [_P, I, LL, _P, _P, _P, I, I, I, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.lmoe_router_grad.argtypes = [_P, I, LL, _P, _P, _P, _P, _P, _P, I, I, I, _P, LL, _P]
        L.lmoe_quantize_fp8_rows.argtypes = [_P, I, LL, _P, LL, LL, I, I, I, _P, _P, _P]
        L.lmoe_quantize_fp8_weight.argtypes = [_P, I, I, I, I, I, I, _P, _P, _P, _P, _P]
        L.lmoe_quantize_fp8_cols.argtypes = [_P, I, LL, _P, LL, LL, I, _P, I, LL, I, I, _P, _P, _P]
        L.lmoe_fp8_padded_rows.argtypes = [LL, I]
        L.lmoe_fp8_padded_rows.restype = LL
        for name in ("lmoe_matmul_fp8", "lmoe_matmul_fp8_wgrad"):
            getattr(L, name).argtypes = [ctypes.POINTER(lmoe_fp8_matmul), _P, _P, _P, _P, _P, _P, _P, _P]
            getattr(L, name).restype = ctypes.c_int
        L.lmoe_fp8_check_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32)]
        L.lmoe_fp8_wait_selftest.argtypes = [LL, _P]
        for name in ("lmoe_fp8_check_status", "lmoe_fp8_wait_selftest",
                     "lmoe_router_losses_workspace_size", "lmoe_router_losses", "lmoe_router_grad",
                     "lmoe_quantize_fp8_rows", "lmoe_quantize_fp8_weight", "lmoe_quantize_fp8_cols"):
            getattr(L, name).restype = ctypes.c_int
        L.lmoe_kernel_launches.restype = ctypes.c_ulonglong
        L.lmoe_kernel_launches.argtypes = []
        _lib_handle = L
    return _lib_handle


def load():
    """Load the shared library (raises ImportError if it is not built)."""
    return _lib()


# ------------------------------------------------------------------ config
@dataclass
class Config:
    T: int
    d_model: int
    d_latent: int
    n_experts: int
    d_ff: int
    top_k: int
    eps: float = 1e-6
    act_dtype: str = "bf16"
    weight_dtype: str = "bf16"
    out_dtype: str = "f32"

    def c(self) -> lmoe_config:
        return lmoe_config(self.T, self.d_model, self.d_latent, self.n_experts, self.d_ff, self.top_k,
                           self.eps, _DT[self.act_dtype], _DT[self.weight_dtype], _DT[self.out_dtype])


def _check(status: int, where: str):
    if status != 0:
        raise LmoeError(status, where)


def _ptr(t) -> int:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _weight_arg(w, keep: list):
    """A dense tensor -> its pointer; an NVFP4 (codes, scales, tensor_scale[, scale_layout])
    tuple -> a pointer to a host lmoe_nvfp4_weight (kept alive in ``keep``).  Without a fourth
    element the scales are declared row-major (which the forward refuses: convert them with
    lmoe_nvfp4_block_scales and pass SCALES_BLOCKED)."""
    if isinstance(w, tuple):
        layout = w[3] if len(w) > 3 else SCALES_ROW_MAJOR
        s = lmoe_nvfp4_weight(_ptr(w[0]), _ptr(w[1]), _ptr(w[2]), int(layout))
        keep.append(s)
        return ctypes.addressof(s)
    return _ptr(w)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def lmoe_workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t()
    c = cfg.c()
    _check(_lib().lmoe_workspace_size(ctypes.byref(c), ctypes.byref(n)), "lmoe_workspace_size")
    return n.value


def lmoe_workspace_size_host_io(cfg: Config) -> int:
    n = ctypes.c_size_t()
    c = cfg.c()
    _check(_lib().lmoe_workspace_size_host_io(ctypes.byref(c), ctypes.byref(n)), "lmoe_workspace_size_host_io")
    return n.value


def lmoe_expert_pair(cfg: Config) -> bool:
    """Whether a call with ``cfg`` runs the grouped gate/up and down GEMMs as one launch."""
    used = ctypes.c_int()
    c = cfg.c()
    _check(_lib().lmoe_expert_pair(ctypes.byref(c), ctypes.byref(used)), "lmoe_expert_pair")
    return bool(used.value)


def lmoe_get_workspace_layout(cfg: Config) -> dict:
    lay = lmoe_workspace_layout()
    c = cfg.c()
    _check(_lib().lmoe_get_workspace_layout(ctypes.byref(c), ctypes.byref(lay)), "lmoe_get_workspace_layout")
    d = {f: getattr(lay, f) for f in _LAYOUT_FIELDS + _LAYOUT_FIELDS_NVFP4}
    d["xa_cols"] = lay.xa_cols
    d["grouped_splits"] = lay.grouped_splits
    return d


def _fwd_args(cfg, x, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool, g_pre,
              g_post, top_k, out, workspace, stream, keep):
    c = cfg.c()
    keep.append(c)
    return [ctypes.byref(c), _ptr(x), _ptr(W_router), _weight_arg(W_pool, keep), _ptr(g_pool),
            _weight_arg(W_gate, keep), _weight_arg(W_up, keep), _weight_arg(W_down, keep), _ptr(g_expert),
            _weight_arg(W_unpool, keep), _ptr(g_pre), _ptr(g_post), int(top_k), _ptr(out),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)]


def latent_moe_forward(cfg, x, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool,
                       g_pre, g_post, top_k, out, workspace, stream=None):
    keep = []
    args = _fwd_args(cfg, x, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool, g_pre,
                     g_post, top_k, out, workspace, stream, keep)
    _check(_lib().latent_moe_forward(*args), "latent_moe_forward")


def latent_moe_forward_ex(cfg, x, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool,
                          g_pre, g_post, top_k, out, workspace, stream=None, router_bias=None,
                          forced_idx=None, topk_idx_out=None, topk_w_out=None, near_tie_count_out=None,
                          wait_budget_cycles=0, stage_events=None, next_norm_gamma=None, next_norm_out=None,
                          single_token_path=0, separate_expert_gemms=False, cooperative_launch=False):
    """``stage_events``: a list of NUM_STAGE_EVENTS torch.cuda.Event(enable_timing=True) or None,
    recorded by the library at the stage boundaries (for per-stage timing; None entries are
    skipped).  ``single_token_path``: with NVFP4 weights and one token, which kernels run
    (SINGLE_TOKEN_DEFAULT, SINGLE_TOKEN_KERNEL or SINGLE_TOKEN_CHAIN; lmoe_ex.single_token_path).
    ``separate_expert_gemms``: gate/up and down as two launches where lmoe_expert_pair() says one.
    ``cooperative_launch``: the single-token persistent kernels launched cooperatively."""
    keep = []
    args = _fwd_args(cfg, x, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool, g_pre,
                     g_post, top_k, out, workspace, stream, keep)
    evs = None
    if stage_events is not None:
        assert len(stage_events) == NUM_STAGE_EVENTS
        for e in stage_events:   # torch creates the CUDA event lazily
            if e is not None and e.cuda_event == 0:
                e.record()
        evs = (ctypes.c_void_p * NUM_STAGE_EVENTS)(*[e.cuda_event if e is not None else None
                                                     for e in stage_events])
        keep.append(evs)
    ex = lmoe_ex(_ptr(router_bias), _ptr(forced_idx), _ptr(topk_idx_out), _ptr(topk_w_out),
                 _ptr(near_tie_count_out), int(wait_budget_cycles),
                 ctypes.cast(evs, ctypes.c_void_p) if evs is not None else None,
                 _ptr(next_norm_gamma), _ptr(next_norm_out), int(single_token_path),
                 1 if separate_expert_gemms else 0, 1 if cooperative_launch else 0)
    _check(_lib().latent_moe_forward_ex(*args, ctypes.byref(ex)), "latent_moe_forward_ex")


def latent_moe_forward_host_io(cfg, x_host, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert,
                               W_unpool, g_pre, g_post, top_k, out_host, workspace, stream=None):
    keep = []
    args = _fwd_args(cfg, x_host, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool,
                     g_pre, g_post, top_k, out_host, workspace, stream, keep)
    _check(_lib().latent_moe_forward_host_io(*args), "latent_moe_forward_host_io")


def latent_moe_forward_host_io_ex(cfg, x_host, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert,
                                  W_unpool, g_pre, g_post, top_k, out_host, workspace, stream=None,
                                  router_bias=None, forced_idx=None, single_token_path=0):
    """latent_moe_forward_host_io with the device-resident routing extensions of lmoe_ex."""
    keep = []
    args = _fwd_args(cfg, x_host, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool,
                     g_pre, g_post, top_k, out_host, workspace, stream, keep)
    ex = lmoe_ex(_ptr(router_bias), _ptr(forced_idx), None, None, None, 0, None, None, None,
                 int(single_token_path), 0, 0)
    _check(_lib().latent_moe_forward_host_io_ex(*args, ctypes.byref(ex)), "latent_moe_forward_host_io_ex")


def lmoe_check_status(cfg, workspace, stream=None) -> tuple[int, int]:
    """(status, raw error word) of the last calls on ``workspace``; synchronises the stream."""
    c = cfg.c()
    word = ctypes.c_uint32()
    st = _lib().lmoe_check_status(ctypes.byref(c), _ptr(workspace), _stream(stream), ctypes.byref(word))
    return st, word.value


def lmoe_wait_selftest(cfg, workspace, budget_cycles: int, stream=None):
    """Run the wait-timeout diagnostic; lmoe_check_status() then reports the timeout."""
    c = cfg.c()
    _check(_lib().lmoe_wait_selftest(ctypes.byref(c), _ptr(workspace), int(budget_cycles), _stream(stream)),
           "lmoe_wait_selftest")


GUARD_BYTES = 256   # LMOE_GUARD_BYTES


def lmoe_workspace_guards(cfg, host_io: bool = False, lib=None) -> list:
    """Byte offsets of the workspace's guard bands (each GUARD_BYTES long)."""
    L = lib or _lib()
    fn = L.lmoe_workspace_guards
    fn.argtypes = [ctypes.POINTER(lmoe_config), ctypes.c_int, _P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    fn.restype = ctypes.c_int
    c = cfg.c()
    n = ctypes.c_int()
    _check(fn(ctypes.byref(c), 1 if host_io else 0, None, 0, ctypes.byref(n)), "lmoe_workspace_guards")
    arr = (ctypes.c_longlong * max(n.value, 1))()
    _check(fn(ctypes.byref(c), 1 if host_io else 0, ctypes.cast(arr, _P), n.value, ctypes.byref(n)),
           "lmoe_workspace_guards")
    return list(arr[:n.value])


def lmoe_validate_routing(cfg, workspace, stream=None, lib=None):
    """Check the routing structures the last call left in ``workspace``; a violation shows in
    lmoe_check_status (LMOE_ERR_ARG, bit 0x20 of the error word)."""
    L = lib or _lib()
    fn = L.lmoe_validate_routing
    fn.argtypes = [ctypes.POINTER(lmoe_config), _P, _P]
    fn.restype = ctypes.c_int
    c = cfg.c()
    _check(fn(ctypes.byref(c), _ptr(workspace), _stream(stream)), "lmoe_validate_routing")


def lmoe_kernel_launches() -> int:
    """Kernels the library has launched in this process."""
    return int(_lib().lmoe_kernel_launches())


def lmoe_permute_noalloc(topk_idx, E: int, offsets, row_of, tok_of, stream=None):
    """Expert-contiguous permutation of ``topk_idx`` [T, k] (int32, device) into ``offsets``
    [E+1], ``row_of`` [T, k] and ``tok_of`` [T*k] without any device allocation: the library's
    fixed scratch array is used instead of a workspace (E <= 1024, T*k <= 65536)."""
    L = _lib()
    fn = L.lmoe_permute_noalloc
    fn.argtypes = [_P, ctypes.c_int, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P]
    fn.restype = ctypes.c_int
    T, k = topk_idx.shape
    # the library looks its scratch up for the current device: make the ids' device current
    # and take the stream from it
    with torch.cuda.device(topk_idx.device):
        st = _stream(stream if stream is not None else torch.cuda.current_stream(topk_idx.device))
        _check(fn(_ptr(topk_idx), T, k, int(E), _ptr(offsets), _ptr(row_of), _ptr(tok_of), st),
               "lmoe_permute_noalloc")


def lmoe_quantize_nvfp4(src, codes, scales, s_row=None, row_scale=True, stream=None):
    """NVFP4-quantise the fp32 rows of ``src`` [rows, K] (device) with the block's activation rule."""
    L = _lib()
    fn = L.lmoe_quantize_nvfp4
    fn.argtypes = [_P, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P]
    fn.restype = ctypes.c_int
    rows, K = src.shape
    _check(fn(_ptr(src), rows, K, 1 if row_scale else 0, _ptr(codes), _ptr(scales), _ptr(s_row),
              _stream(stream)), "lmoe_quantize_nvfp4")


def lmoe_nvfp4_block_scales(src, K: int, block_rows: int = 128, dst=None, stream=None):
    """Row-major E4M3 scales ``src`` [..., rows, K/16] (uint8, device) -> the block layout the
    NVFP4 GEMMs read, in blocks of ``block_rows`` (128, or 64 for W_gate/W_up) rows; returns a
    flat uint8 tensor unless ``dst`` is given."""
    L = _lib()
    fn = L.lmoe_nvfp4_block_scales
    fn.argtypes = [_P, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, _P, _P]
    fn.restype = ctypes.c_int
    rows = src.numel() // (K // 16)
    if dst is None:
        dst = torch.zeros(rows // block_rows * (K // 64) * 512, dtype=torch.uint8, device=src.device)
    _check(fn(_ptr(src), rows, int(K), int(block_rows), _ptr(dst), _stream(stream)),
           "lmoe_nvfp4_block_scales")
    return dst


# ------------------------------------------------------------------ router training, 8-bit products
# These take tensors whose shapes and dtypes say the sizes; what does not fit is refused with a
# ValueError before the library is called.
_FP8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}          # lmoe_fp8_format
_DENSE = {torch.float32: LMOE_F32, torch.bfloat16: LMOE_BF16}
# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _want(t, name, dtypes, shape, device, strided=False):
    """``t``: a CUDA tensor on device number ``device`` of one of ``dtypes`` (or the one) and of
    ``shape``, contiguous (strided: a matrix whose rows are)."""
    if t.dtype is not dtypes and (isinstance(dtypes, torch.dtype) or t.dtype not in dtypes):
        raise ValueError(f"{name}: dtype {t.dtype} is not one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{device}" if device >= 0 else ""))
    if not t.is_contiguous():
        _need(strided, f"{name} must be contiguous")
        _need(t.shape[1] <= 1 or t.stride(1) == 1, f"{name}: rows must be contiguous")
        _need(t.shape[0] <= 1 or t.stride(0) >= t.shape[1], f"{name}: rows overlap")


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _call(fn, where, device, stream, *args):
    """Calls ``fn`` with device number ``device`` current, on ``stream`` or that device's current one."""
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(fn, where, device, stream, *args)
    status = fn(*args, _raw_stream(device) if stream is None else _stream(stream))
    if status != 0:
        raise LmoeError(status, where)


def lmoe_router_losses_workspace_size(T: int, E: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib().lmoe_router_losses_workspace_size(int(T), int(E), ctypes.byref(n)),
           "lmoe_router_losses_workspace_size")
    return n.value


def _router_args(logits, topk_idx, router_bias, row_mask):
    _need(logits.dim() == 2 and topk_idx.dim() == 2, "logits [T, E] and topk_idx [T, k]")
    dev, (T, E), k = logits.get_device(), logits.shape, topk_idx.shape[1]
    _want(logits, "logits", _DENSE, (T, E), dev, strided=True)
    _want(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    if router_bias is not None:
        _want(router_bias, "router_bias", torch.float32, (E,), dev)
    if row_mask is not None:
        _want(row_mask, "row_mask", (torch.uint8, torch.bool), (T,), dev)
    return dev, T, E, k


def lmoe_router_losses(logits, topk_idx, counts, mean_probs, losses, workspace, router_bias=None, row_mask=None,
                       stream=None):
    """Balance loss and z loss of router ``logits`` [T, E] (fp32 or bf16, rows may be strided) with
    the selected experts ``topk_idx`` [T, k] (int32): writes ``losses`` [2] fp32, ``mean_probs``
    [E] fp32 and ``counts`` [E + 1] int32 (slots per expert, then live rows).  ``row_mask`` [T]
    (uint8 or bool): rows that are 0 are left out.  ``workspace``: at least
    lmoe_router_losses_workspace_size(T, E) bytes."""
    dev, T, E, k = _router_args(logits, topk_idx, router_bias, row_mask)
    _want(counts, "counts", torch.int32, (E + 1,), dev)
    _want(mean_probs, "mean_probs", torch.float32, (E,), dev)
    _want(losses, "losses", torch.float32, (2,), dev)
    _need(workspace.get_device() == dev and workspace.is_contiguous(), f"workspace must be contiguous on cuda:{dev}")
    _call(_lib().lmoe_router_losses, "lmoe_router_losses", dev, stream, logits.data_ptr(), _DENSE[logits.dtype],
          _ld(logits), _ptr(router_bias), _ptr(row_mask), topk_idx.data_ptr(), T, E, k, counts.data_ptr(),
          mean_probs.data_ptr(), losses.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())


def lmoe_router_grad(logits, topk_idx, counts, dlogits, topk_w_grad=None, loss_grads=None, router_bias=None,
                     row_mask=None, stream=None):
    """Gradient ``dlogits`` (dtype and shape of ``logits``, which it may be) from the routing
    weights' gradient ``topk_w_grad`` [T, k] fp32 and the losses' gradients ``loss_grads`` [2]
    fp32 (on the device).  ``counts``: as lmoe_router_losses wrote them (None without
    ``loss_grads``)."""
    dev, T, E, k = _router_args(logits, topk_idx, router_bias, row_mask)
    _want(dlogits, "dlogits", logits.dtype, (T, E), dev, strided=True)
    if topk_w_grad is not None:
        _want(topk_w_grad, "topk_w_grad", torch.float32, (T, k), dev)
    if loss_grads is not None:
        _want(loss_grads, "loss_grads", torch.float32, (2,), dev)
    if counts is not None:
        _want(counts, "counts", torch.int32, (E + 1,), dev)
    _call(_lib().lmoe_router_grad, "lmoe_router_grad", dev, stream, logits.data_ptr(), _DENSE[logits.dtype],
          _ld(logits), _ptr(router_bias), _ptr(row_mask), topk_idx.data_ptr(), _ptr(topk_w_grad), _ptr(counts),
          _ptr(loss_grads), T, E, k, dlogits.data_ptr(), _ld(dlogits))


def lmoe_fp8_padded_rows(rows: int, n_experts: int) -> int:
    """Columns that any split of ``rows`` among ``n_experts`` fits in, each padded to blocks of 128."""
    return int(_lib().lmoe_fp8_padded_rows(int(rows), int(n_experts)))


def _routed_src(src, row_index):
    _need(src.dim() == 2, "src [rows, K]")
    dev, (n, K) = src.get_device(), src.shape
    _want(src, "src", _DENSE, (n, K), dev, strided=True)
    if row_index is None:
        return dev, n, K, n
    _need(row_index.dim() == 1, "row_index [rows]")
    _want(row_index, "row_index", torch.int32, row_index.shape, dev)
    return dev, n, K, row_index.shape[0]


def lmoe_quantize_fp8_rows(src, codes, scales, row_index=None, pow2_scales=False, stream=None):
    """Rows of ``src`` [*, K] (fp32 or bf16), gathered by ``row_index`` [rows] (int32; outside src: a
    row of zeros) if given, into 8-bit ``codes`` [rows, K] (its dtype is the format) with a scale
    per 128 elements, ``scales`` [ceil(K/128), rows] fp32."""
    dev, n, K, rows = _routed_src(src, row_index)
    _want(codes, "codes", _FP8, (rows, K), dev)
    _want(scales, "scales", torch.float32, (-(-K // 128), rows), dev)
    _call(_lib().lmoe_quantize_fp8_rows, "lmoe_quantize_fp8_rows", dev, stream, src.data_ptr(), _DENSE[src.dtype],
          _ld(src), _ptr(row_index), n, rows, K, _FP8[codes.dtype], 1 if pow2_scales else 0, codes.data_ptr(),
          scales.data_ptr())


def lmoe_quantize_fp8_weight(src, codes, scales, codes_t=None, scales_t=None, pow2_scales=False, stream=None):
    """Weights ``src`` [N, K] or [E, N, K] (fp32 or bf16) into 8-bit ``codes`` of the same shape with a
    scale per 128 x 128 block, ``scales`` [(E,) ceil(N/128), ceil(K/128)]; ``codes_t``, ``scales_t``:
    also the transposed pair."""
    _need(src.dim() in (2, 3), "src [N, K] or [E, N, K]")
    dev, (N, K), lead = src.get_device(), src.shape[-2:], src.shape[:-2]
    nb, kb = -(-N // 128), -(-K // 128)
    _want(src, "src", _DENSE, src.shape, dev)
    _want(codes, "codes", _FP8, src.shape, dev)
    _want(scales, "scales", torch.float32, (*lead, nb, kb), dev)
    if codes_t is not None:
        _want(codes_t, "codes_t", codes.dtype, (*lead, K, N), dev)
    if scales_t is not None:
        _want(scales_t, "scales_t", torch.float32, (*lead, kb, nb), dev)
    _call(_lib().lmoe_quantize_fp8_weight, "lmoe_quantize_fp8_weight", dev, stream, src.data_ptr(),
          _DENSE[src.dtype], lead[0] if lead else 1, N, K, _FP8[codes.dtype], 1 if pow2_scales else 0,
          codes.data_ptr(), scales.data_ptr(), _ptr(codes_t), _ptr(scales_t))


def lmoe_quantize_fp8_cols(src, codes_t, scales_t, offsets=None, row_index=None, pow2_scales=False, stream=None):
    """The routed rows of ``src`` (as lmoe_quantize_fp8_rows), expert by expert (``offsets`` [E + 1]
    int32; None: one group), each padded to blocks of 128 rows, into transposed 8-bit ``codes_t``
    [K, P] with a scale per 128 rows of a column, ``scales_t`` [P / 128, K] fp32;
    P = lmoe_fp8_padded_rows(rows, E)."""
    dev, n, K, rows = _routed_src(src, row_index)
    E = 1
    if offsets is not None:
        _need(offsets.dim() == 1 and offsets.shape[0] > 1, "offsets [E + 1]")
        E = offsets.shape[0] - 1
        _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    P = lmoe_fp8_padded_rows(rows, E)
    _want(codes_t, "codes_t", _FP8, (K, P), dev)
    _want(scales_t, "scales_t", torch.float32, (P // 128, K), dev)
    _call(_lib().lmoe_quantize_fp8_cols, "lmoe_quantize_fp8_cols", dev, stream, src.data_ptr(), _DENSE[src.dtype],
          _ld(src), _ptr(row_index), n, rows, K, _ptr(offsets), E, P, _FP8[codes_t.dtype],
          1 if pow2_scales else 0, codes_t.data_ptr(), scales_t.data_ptr())


def _fp8_product(fn, where, dev, stream, rows, N, K, E, a, a_scales, b, b_scales, offsets, out, accumulate, status,
                 unpadded=0):
    if offsets is not None:
        _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    if status is not None:
        _want(status, "status", (torch.int32, torch.uint32), (1,), dev)
    shape = lmoe_fp8_matmul(rows, N, K, E, _FP8[a.dtype], _FP8[b.dtype], _DENSE[out.dtype], 1 if accumulate else 0, 0,
                            unpadded)
    _call(fn, where, dev, stream, ctypes.byref(shape), a.data_ptr(), a_scales.data_ptr(), b.data_ptr(),
          b_scales.data_ptr(), _ptr(offsets), out.data_ptr(), _ptr(status))


def _on_device(device, stream, fn):
    with torch.cuda.device(device):   # (None: the current one)
        return fn(_stream(stream))


def lmoe_fp8_check_status(device=None, stream=None) -> tuple[int, int]:
    """(status, error word) of the 8-bit products on ``device`` that were given no ``status`` word since the
    last check: LMOE_ERR_TIMEOUT if a device wait gave up and left a product unfinished.  Synchronises the
    stream."""
    word = ctypes.c_uint32()
    st = _on_device(device, stream, lambda s: _lib().lmoe_fp8_check_status(s, ctypes.byref(word)))
    return st, word.value


def lmoe_fp8_wait_selftest(budget_cycles: int, device=None, stream=None):
    """Run the wait-timeout diagnostic; lmoe_fp8_check_status() then reports the timeout."""
    _check(_on_device(device, stream, lambda s: _lib().lmoe_fp8_wait_selftest(int(budget_cycles), s)),
           "lmoe_fp8_wait_selftest")


def lmoe_matmul_fp8(a, a_scales, w, w_scales, out, offsets=None, status=None, stream=None):
    """``out`` [rows, N] (fp32 or bf16) = ``a`` [rows, K] times ``w`` [N, K] transposed, or, with ``w`` [E, N,
    K] and ``offsets`` [E + 1] (int32), each expert's rows times its own; scales as
    lmoe_quantize_fp8_rows and lmoe_quantize_fp8_weight write them.  ``status`` [1] (int32): error word, for a
    device wait that gives up; None: the device's own word (lmoe_fp8_check_status)."""
    _need(a.dim() == 2 and w.dim() in (2, 3), "a [rows, K] and w [N, K] or [E, N, K]")
    dev, (rows, K), N, lead = a.get_device(), a.shape, w.shape[-2], w.shape[:-2]
    kb = -(-K // 128)
    _want(a, "a", _FP8, (rows, K), dev)
    _want(a_scales, "a_scales", torch.float32, (kb, rows), dev)
    _want(w, "w", _FP8, (*lead, N, K), dev)
    _want(w_scales, "w_scales", torch.float32, (*lead, -(-N // 128), kb), dev)
    _want(out, "out", _DENSE, (rows, N), dev)
    _fp8_product(_lib().lmoe_matmul_fp8, "lmoe_matmul_fp8", dev, stream, rows, N, K, lead[0] if lead else 1, a,
                 a_scales, w, w_scales, offsets, out, False, status)


def lmoe_matmul_fp8_wgrad(dy_t, dy_scales, x_t, x_scales, dw, offsets=None, accumulate=False, status=None,
                          stream=None, rows=None):
    """``dw`` [(E,) N, K] (fp32 or bf16) (+)= each expert's rows of dy transposed times its rows of x, from
    ``dy_t`` [N, P] and ``x_t`` [K, P] as lmoe_quantize_fp8_cols writes them for ``offsets`` [E + 1].  ``rows``: how
    many rows were padded there, to which offsets are clamped; None: offsets must lie within them, or blocks that were
    never written are added.  ``status`` as in lmoe_matmul_fp8."""
    _need(dy_t.dim() == 2 and x_t.dim() == 2 and dw.dim() in (2, 3), "dy_t [N, P], x_t [K, P], dw [(E,) N, K]")
    dev, (N, P), K, lead = dy_t.get_device(), dy_t.shape, x_t.shape[0], dw.shape[:-2]
    _need(P % 128 == 0, "P must be a multiple of 128")
    _need(rows is None or rows != 0 or P == 0, f"rows 0, but {P} padded ones")   # (0 is "not given" to the library)
    _want(dy_t, "dy_t", _FP8, (N, P), dev)
    _want(dy_scales, "dy_scales", torch.float32, (P // 128, N), dev)
    _want(x_t, "x_t", _FP8, (K, P), dev)
    _want(x_scales, "x_scales", torch.float32, (P // 128, K), dev)
    _want(dw, "dw", _DENSE, (*lead, N, K), dev)
    _fp8_product(_lib().lmoe_matmul_fp8_wgrad, "lmoe_matmul_fp8_wgrad", dev, stream, P, N, K, lead[0] if lead else 1,
                 dy_t, dy_scales, x_t, x_scales, offsets, dw, accumulate, status, 0 if rows is None else int(rows))
