"""Local-Hessian NVFP4 weight-scale calibration on AMD Instinct MI355X.

Thin ctypes binding over the C ABI of ``liblh.so`` (declared in
``include/lh.h``).  The functions carry the C names and only marshal
arguments: tensor pointers, strides, dtypes and the current HIP stream.
Every step of the computation runs in the library's HIP kernels; there is no
CPU fallback.  If the library is missing the import raises.

Tensors must live on a ROCm device.  Shapes:
  weights      [c_out, c_in] or [n_groups, c_out, c_in], bf16 or fp32,
               last dim contiguous (any row / group stride)
  activations  channel-major [c_in, N] / [n_groups, c_in, N], or
               token-major   [N, c_in] / [n_groups, N, c_in]
  hessians     fp32 [n_groups, c_in/16, 16, 16]
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblh.so")

LH_DTYPE_F32, LH_DTYPE_BF16, LH_DTYPE_E4M3 = 0, 1, 2
LH_LAYOUT_CHANNEL_MAJOR, LH_LAYOUT_TOKEN_MAJOR = 0, 1
LH_INDEX_I32, LH_INDEX_I64 = 0, 1
LH_RULE_SWEEP, LH_RULE_MAX, LH_RULE_FOUR_OVER_SIX, LH_RULE_AMAX_SEARCH = 0, 1, 2, 3
N_CANDIDATES = 126
BLOCK = 16
CHECKPOINT_BLOCK = 32  # values that share a power of two in an 8-bit checkpoint


class LHError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s (status %d)" % (message, status))
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("liblh.so not built: run __graft_entry__.build() or "
                          "python nvfp4_scale_calibration_amd/_build.py (%s)" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.lh_abi_version.restype = I
    lib.lh_status_string.argtypes = [I]
    lib.lh_status_string.restype = ctypes.c_char_p
    lib.lh_last_error_message.restype = ctypes.c_char_p
    lib.lh_absmax.argtypes = [P, I, I64, I64, I64, I64, I64, P, P]
    lib.lh_absmax.restype = I
    lib.lh_hessian_alpha.argtypes = [F, I64]
    lib.lh_hessian_alpha.restype = F
    lib.lh_hessian_workspace_bytes.argtypes = [I64, I64, I64]
    lib.lh_hessian_workspace_bytes.restype = SZ
    lib.lh_accumulate_hessian.argtypes = [P, I, I, I64, I64, I64, I64, I64, F, F, P, I64, P, SZ, P]
    lib.lh_accumulate_hessian.restype = I
    lib.lh_hessian_ragged_workspace_bytes.argtypes = [I64, I64, I64, I64]
    lib.lh_hessian_ragged_workspace_bytes.restype = SZ
    lib.lh_accumulate_hessian_ragged.argtypes = [P, I, I64, I64, I64, P, I64, I64, P, I64, P, P, SZ, P]
    lib.lh_accumulate_hessian_ragged.restype = I
    lib.lh_sweep_workspace_bytes.argtypes = [I64, I64]
    lib.lh_sweep_workspace_bytes.restype = SZ
    lib.lh_scale_sweep.argtypes = [P, I, I64, I64, I64, I64, I64, P, I64, P, P, P, P, P, SZ, P]
    lib.lh_scale_sweep.restype = I
    lib.lh_select_scales.argtypes = [I, P, I, I64, I64, I64, I64, I64, P, I64, P, P, P, P, P, SZ, P]
    lib.lh_select_scales.restype = I
    lib.lh_scale_sweep_fake_quant.argtypes = [P, I, I64, I64, I64, I64, I64, P, I64, P, P, P, P, P, P, P, P, P,
                                              SZ, P]
    lib.lh_scale_sweep_fake_quant.restype = I
    lib.lh_calibrate_workspace_bytes.argtypes = [I64, I64, I64, I64]
    lib.lh_calibrate_workspace_bytes.restype = SZ
    lib.lh_calibrate_nvfp4.argtypes = [P, I, I64, I64, I64, I64, I64, P, I, I, I64, I64, I64, P, P, I64, P, P, P, P, P,
                                       P, P, P, SZ, P]
    lib.lh_calibrate_nvfp4.restype = I
    lib.lh_calibrate_nvfp4_noalloc.argtypes = [P, I, I64, I64, I64, I64, I64, P, I, I, I64, I64, I64, P, P, I64, P, P,
                                               P, P, P, P, P, P]
    lib.lh_calibrate_nvfp4_noalloc.restype = I
    lib.lh_calibrate_prologue.argtypes = [P, I, I64, I64, I64, I64, I64, P, I, I, I64, I64, I64, P, P, I64, P, SZ, P]
    lib.lh_calibrate_prologue.restype = I
    lib.lh_calibrate_sweep.argtypes = [P, I, I64, I64, I64, I64, I64, P, I64, P, P, P, P, P, P, P, P, P, SZ, P]
    lib.lh_calibrate_sweep.restype = I
    lib.lh_full_hessian.argtypes = [P, I, I64, I64, I64, I64, I64, F, P, I64, I64, P]
    lib.lh_full_hessian.restype = I
    lib.lh_output_error_workspace_bytes.argtypes = [I64, I64, I64]
    lib.lh_output_error_workspace_bytes.restype = SZ
    lib.lh_output_error.argtypes = [P, I, P, I64, I64, I64, I64, I64, I64, I64, P, I64, I64, P, P, SZ, P]
    lib.lh_output_error.restype = I
    lib.lh_scaled_histogram.argtypes = [P, I, I64, I64, I64, I64, I64, P, P, I, F, P, P]
    lib.lh_scaled_histogram.restype = I
    lib.lh_gptq_workspace_bytes.argtypes = [I64, I64]
    lib.lh_gptq_workspace_bytes.restype = SZ
    lib.lh_gptq_prepare.argtypes = [P, I64, I64, F, P, I64, P, SZ, P]
    lib.lh_gptq_prepare.restype = I
    lib.lh_gptq_quantize.argtypes = [P, I, I64, I64, I64, P, P, P, I64, P, I64, P, SZ, P]
    lib.lh_gptq_quantize.restype = I
    lib.lh_fake_quant_nvfp4.argtypes = [P, I, I64, I64, I64, I64, I64, P, P, P, P, P, P, P]
    lib.lh_fake_quant_nvfp4.restype = I
    lib.lh_quantize_nvfp4.argtypes = [P, I, I64, I64, I64, I64, I64, P, P, I, P, P, P, P]
    lib.lh_quantize_nvfp4.restype = I
    lib.lh_linear_nvfp4_workspace_bytes.argtypes = [I, I, I, I64, I64, I64, I64, I64]
    lib.lh_linear_nvfp4_workspace_bytes.restype = SZ
    lib.lh_linear_nvfp4.argtypes = [P, I, I64, I64, I64, I64, P, P, P, I64, I64, P, P, I, I64, I64, P, SZ, P]
    lib.lh_linear_nvfp4.restype = I
    lib.lh_linear_nvfp4_grad.argtypes = [P, I, I64, I64, I64, I64, P, P, P, I64, I64, P, I, I64, I64, P, SZ, P]
    lib.lh_linear_nvfp4_grad.restype = I
    lib.lh_linear_nvfp4_ragged.argtypes = [P, I, I64, I64, I64, P, I64, I64, P, P, P, I64, P, P, I, I64, P, SZ, P]
    lib.lh_linear_nvfp4_ragged.restype = I
    lib.lh_linear_nvfp4_ragged_grad.argtypes = [P, I, I64, I64, I64, P, I64, I64, P, P, P, I64, P, I, I64, P, SZ, P]
    lib.lh_linear_nvfp4_ragged_grad.restype = I
    lib.lh_moe_sort_workspace_bytes.argtypes = [I64, I64, I64]
    lib.lh_moe_sort_workspace_bytes.restype = SZ
    lib.lh_moe_sort.argtypes = [P, I, I64, I64, I64, P, P, P, P, SZ, P]
    lib.lh_moe_sort.restype = I
    lib.lh_moe_dispatch.argtypes = [P, I, I64, I64, I64, P, I64, P, I64, I64, P]
    lib.lh_moe_dispatch.restype = I
    lib.lh_moe_combine.argtypes = [P, I, I64, I64, I64, P, P, I64, I64, P, I64, P]
    lib.lh_moe_combine.restype = I
    lib.lh_moe_combine_grad.argtypes = [P, I, I64, I64, I64, P, I64, I64, P, I64, P, P, I64, P, P]
    lib.lh_moe_combine_grad.restype = I
    lib.lh_lora_workspace_bytes.argtypes = [I, I64, I64, I64, I64, I64]
    lib.lh_lora_workspace_bytes.restype = SZ
    for f in (lib.lh_lora, lib.lh_lora_grad):
        f.argtypes = [P, I, I64, I64, I64, P, P, I, I64, P, P, I, I64, I64, P, P, I64, I64, P, I, I64, P, P, SZ, P]
        f.restype = I
    lib.lh_lora_weight_grad_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I64]
    lib.lh_lora_weight_grad_workspace_bytes.restype = SZ
    lib.lh_lora_weight_grad.argtypes = [P, I, P, I64, I64, P, I, I64, I64, P, P, I64, P, P, I, I64, I64, I64, P, F, P,
                                        P, I, P, SZ, P]
    lib.lh_lora_weight_grad.restype = I
    lib.lh_checkpoint_pack.argtypes = [P, I, I64, I64, I64, P, P, P]
    lib.lh_checkpoint_pack.restype = I
    lib.lh_checkpoint_unpack.argtypes = [P, P, I64, I64, P, I, I64, P]
    lib.lh_checkpoint_unpack.restype = I
    return lib


lib = _load()
EXPORTS = ("lh_abi_version", "lh_status_string", "lh_last_error_message", "lh_absmax", "lh_hessian_alpha",
           "lh_hessian_workspace_bytes", "lh_accumulate_hessian", "lh_hessian_ragged_workspace_bytes",
           "lh_accumulate_hessian_ragged", "lh_sweep_workspace_bytes", "lh_scale_sweep",
           "lh_scale_sweep_fake_quant", "lh_calibrate_workspace_bytes", "lh_calibrate_nvfp4",
           "lh_calibrate_prologue", "lh_calibrate_sweep", "lh_calibrate_nvfp4_noalloc", "lh_select_scales", "lh_fake_quant_nvfp4", "lh_full_hessian", "lh_output_error_workspace_bytes",
           "lh_output_error", "lh_scaled_histogram", "lh_gptq_workspace_bytes", "lh_gptq_prepare",
           "lh_gptq_quantize", "lh_quantize_nvfp4", "lh_linear_nvfp4_workspace_bytes", "lh_linear_nvfp4",
           "lh_linear_nvfp4_grad", "lh_linear_nvfp4_ragged", "lh_linear_nvfp4_ragged_grad",
           "lh_moe_sort_workspace_bytes", "lh_moe_sort", "lh_moe_dispatch", "lh_moe_combine", "lh_moe_combine_grad",
           "lh_lora_workspace_bytes", "lh_lora", "lh_lora_grad", "lh_lora_weight_grad_workspace_bytes",
           "lh_lora_weight_grad", "lh_checkpoint_pack", "lh_checkpoint_unpack")


def _check(status: int) -> None:
    if status != 0:
        msg = lib.lh_last_error_message().decode() or lib.lh_status_string(status).decode()
        raise LHError(status, msg)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor):
    """The current stream of t's device as an integer (the raw call takes a
    tenth of a microsecond, building a Stream object two)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LH_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return LH_DTYPE_BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def _as3(t: torch.Tensor) -> torch.Tensor:
    if t.dim() == 2:
        return t.unsqueeze(0)
    if t.dim() != 3:
        raise ValueError("expected a 2-D or 3-D tensor, got shape %s" % (tuple(t.shape),))
    return t


def _require_device(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("liblh works on device tensors only (got a %s tensor)" % t.device)


def _group_stride(t3: torch.Tensor) -> int:
    return t3.stride(0) if t3.shape[0] > 1 else 0


def _ld(t3: torch.Tensor) -> int:
    """Row stride; a dimension of size 1 has no meaningful stride (torch may
    report 1), so the contiguous extent is passed instead."""
    return t3.stride(1) if t3.shape[1] > 1 else t3.shape[2]


def lh_abi_version() -> int:
    return lib.lh_abi_version()


def lh_absmax(w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Global amax per group: out[g] = max |w[g]| (fp32)."""
    _require_device(w)
    w3 = _as3(w)
    if w3.stride(-1) != 1:
        raise ValueError("last dim of w must be contiguous")
    g, rows, cols = w3.shape
    if out is None:
        out = torch.empty(g, dtype=torch.float32, device=w.device)
    _check(lib.lh_absmax(_ptr(w3), _dtype(w3), rows, cols, _ld(w3), g, _group_stride(w3),
                         _ptr(out), _stream(w)))
    return out


def lh_hessian_alpha(alpha: float, n_tokens: int) -> float:
    """The factor the Hessian calls apply for `alpha` (NaN: fl32(1/N))."""
    return float(lib.lh_hessian_alpha(float(alpha), int(n_tokens)))


def lh_hessian_workspace_bytes(c_in: int, n_tokens: int, n_groups: int = 1) -> int:
    return int(lib.lh_hessian_workspace_bytes(c_in, n_tokens, n_groups))


def lh_accumulate_hessian(x: torch.Tensor, layout: str = "channel", alpha: float | None = None,
                          beta: float = 0.0, h: torch.Tensor | None = None,
                          workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """h = beta * h + alpha * X_b X_b^T for every 16-channel block.

    x: channel-major [.., c_in, N] (layout="channel") or token-major
    [.., N, c_in] (layout="token").  alpha defaults to 1/N (the normalised
    Hessian).  workspace=True allocates the split-token scratch buffer the
    library asks for, False/None runs without one, a uint8 device tensor is
    used as given."""
    _require_device(x, h)
    x3 = _as3(x)
    if x3.stride(-1) != 1:
        raise ValueError("last dim of x must be contiguous")
    lay = {"channel": LH_LAYOUT_CHANNEL_MAJOR, "token": LH_LAYOUT_TOKEN_MAJOR}[layout]
    g = x3.shape[0]
    c_in, n_tok = (x3.shape[1], x3.shape[2]) if lay == LH_LAYOUT_CHANNEL_MAJOR else (x3.shape[2], x3.shape[1])
    nb = c_in // BLOCK
    if alpha is None:
        alpha = float("nan")   # the library applies the normalised Hessian's 1/N
    if h is None:
        h = torch.empty((g, nb, BLOCK, BLOCK), dtype=torch.float32, device=x.device)
        if beta != 0.0:
            raise ValueError("beta != 0 needs an existing h")
    ws, ws_bytes = None, 0
    if workspace is True:
        ws_bytes = lh_hessian_workspace_bytes(c_in, n_tok, g)
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    elif isinstance(workspace, torch.Tensor):
        ws, ws_bytes = workspace, workspace.numel() * workspace.element_size()
    h_gstride = h.stride(0) if h.dim() == 4 and h.shape[0] > 1 else 0
    _check(lib.lh_accumulate_hessian(_ptr(x3), _dtype(x3), lay, c_in, n_tok, _ld(x3), g,
                                     _group_stride(x3), float(alpha), float(beta), _ptr(h), h_gstride,
                                     _ptr(ws), ws_bytes, _stream(x)))
    return h


def lh_hessian_ragged_workspace_bytes(c_in: int, n_rows: int, n_groups: int, max_group_rows: int = 0) -> int:
    return int(lib.lh_hessian_ragged_workspace_bytes(c_in, n_rows, n_groups, max_group_rows))


def lh_accumulate_hessian_ragged(x: torch.Tensor, offsets: torch.Tensor, h: torch.Tensor | None = None,
                                 counts: torch.Tensor | None = None,
                                 workspace: torch.Tensor | bool | None = True,
                                 max_group_rows: int = 0) -> torch.Tensor:
    """Per-group Hessians of token-major x [n_rows, c_in] whose rows
    offsets[g] .. offsets[g+1]-1 (device int64 [n_groups + 1]) belong to
    group g.  Without counts each group with tokens gets S_g / n_g; with a
    device int64 counts tensor the running mean (n_old H + S_g) / (n_old +
    n_g) is kept and counts is advanced.  Groups without tokens keep h (a
    new h starts at zero)."""
    _require_device(x, offsets, h, counts)
    if x.dim() != 2 or x.stride(-1) != 1:
        raise ValueError("x must be a 2-D token-major tensor with contiguous rows")
    if offsets.dtype != torch.int64 or counts is not None and counts.dtype != torch.int64:
        raise TypeError("offsets and counts must be int64")
    n_rows, c_in = x.shape
    g = offsets.numel() - 1
    nb = c_in // BLOCK
    if h is None:
        h = torch.zeros((g, nb, BLOCK, BLOCK), dtype=torch.float32, device=x.device)
    ws, ws_bytes = None, 0
    if workspace is True:
        ws_bytes = lh_hessian_ragged_workspace_bytes(c_in, n_rows, g, max_group_rows)
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    elif isinstance(workspace, torch.Tensor):
        ws, ws_bytes = workspace, workspace.numel() * workspace.element_size()
    h_gstride = h.stride(0) if h.dim() == 4 and h.shape[0] > 1 else 0
    ld = x.stride(0) if n_rows > 1 else c_in
    _check(lib.lh_accumulate_hessian_ragged(_ptr(x), _dtype(x), c_in, ld, n_rows, _ptr(offsets), g,
                                            int(max_group_rows), _ptr(h),
                                            h_gstride, _ptr(counts), _ptr(ws), ws_bytes, _stream(x)))
    return h


def lh_sweep_workspace_bytes(c_in: int, n_groups: int = 1) -> int:
    return int(lib.lh_sweep_workspace_bytes(c_in, n_groups))


def _select(rule, w, h, amax, best_idx, best_err, best_amax, workspace, quant=None):
    _require_device(w, h, amax)
    w3 = _as3(w)
    if w3.stride(-1) != 1:
        raise ValueError("last dim of w must be contiguous")
    g, c_out, c_in = w3.shape
    nb = c_in // BLOCK
    shape = (g, c_out, nb)
    dev = w.device
    if best_idx is None:
        best_idx = torch.empty(shape, dtype=torch.uint8, device=dev)
    if best_err is True:
        best_err = torch.empty(shape, dtype=torch.float32, device=dev)
    if best_amax is True:
        best_amax = torch.empty(shape, dtype=torch.float32, device=dev)
    best_err = best_err if isinstance(best_err, torch.Tensor) else None
    best_amax = best_amax if isinstance(best_amax, torch.Tensor) else None
    h_gstride = h.stride(0) if h is not None and h.dim() == 4 and h.shape[0] > 1 else 0
    ws, ws_bytes = None, 0
    if workspace is True:
        ws_bytes = lh_sweep_workspace_bytes(c_in, g) if h is not None and rule == LH_RULE_SWEEP else 0
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    elif isinstance(workspace, torch.Tensor):
        ws, ws_bytes = workspace, workspace.numel() * workspace.element_size()
    args = (_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3), _ptr(h), h_gstride, _ptr(amax),
            _ptr(best_idx), _ptr(best_err), _ptr(best_amax), _ptr(ws), ws_bytes, _stream(w))
    if quant is not None:
        _check(lib.lh_scale_sweep_fake_quant(*args[:13], *(_ptr(quant[k]) for k in _FQ_KEYS), *args[13:]))
    elif rule is None:
        _check(lib.lh_scale_sweep(*args))
    else:
        _check(lib.lh_select_scales(int(rule), *args))
    return best_idx, best_err, best_amax


def lh_scale_sweep(w: torch.Tensor, h: torch.Tensor, amax: torch.Tensor,
                   best_idx: torch.Tensor | None = None, best_err: torch.Tensor | bool | None = True,
                   best_amax: torch.Tensor | bool | None = True,
                   workspace: torch.Tensor | bool | None = True):
    """Per-block best candidate index (E4M3 code = idx + 1), its error
    dw^T H_b dw and the per-block amax 6 * s_idx.  Returns (idx, err, amax);
    err / amax are None when not requested (False/None).  workspace=True
    allocates the certificate scratch the library asks for (faster skipping),
    False/None runs without it, a device tensor is used as given."""
    if h is None:
        raise ValueError("lh_scale_sweep needs a Hessian (lh_select_scales takes h=None)")
    return _select(None, w, h, amax, best_idx, best_err, best_amax, workspace)


_FQ_KEYS = ("w_q", "packed", "scale_e4m3", "global_scale")


def _fq_outputs(w3, w_q, packed, scale_e4m3, global_scale) -> dict:
    g, c_out, c_in = w3.shape
    dev = w3.device

    def out(req, shape, dtype):
        if isinstance(req, torch.Tensor):
            return req
        return torch.empty(shape, dtype=dtype, device=dev) if req else None

    return dict(w_q=out(w_q, (g, c_out, c_in), torch.float32),
                packed=out(packed, (g, c_out, c_in // 2), torch.uint8),
                scale_e4m3=out(scale_e4m3, (g, c_out, c_in // BLOCK), torch.uint8),
                global_scale=out(global_scale, (g,), torch.float32))


def lh_scale_sweep_fake_quant(w: torch.Tensor, h: torch.Tensor, amax: torch.Tensor,
                              best_idx: torch.Tensor | None = None, best_err: torch.Tensor | bool | None = True,
                              best_amax: torch.Tensor | bool | None = True,
                              w_q: bool | torch.Tensor = True, packed: bool | torch.Tensor = False,
                              scale_e4m3: bool | torch.Tensor = False, global_scale: bool | torch.Tensor = False,
                              workspace: torch.Tensor | bool | None = True) -> dict:
    """lh_scale_sweep and lh_fake_quant_nvfp4 with its indices in one pass.
    Returns a dict with idx, err, amax (as lh_scale_sweep; None when not
    requested) and the requested fake-quant outputs (as lh_fake_quant_nvfp4)."""
    if h is None:
        raise ValueError("lh_scale_sweep_fake_quant needs a Hessian")
    _require_device(w)
    quant = _fq_outputs(_as3(w), w_q, packed, scale_e4m3, global_scale)
    idx, err, bam = _select(None, w, h, amax, best_idx, best_err, best_amax, workspace, quant=quant)
    res = dict(idx=idx, err=err, amax=bam)
    res.update({k: v for k, v in quant.items() if v is not None})
    return res


def lh_calibrate_workspace_bytes(c_out: int, c_in: int, n_tokens: int, n_groups: int = 1) -> int:
    return int(lib.lh_calibrate_workspace_bytes(c_out, c_in, n_tokens, n_groups))


def _calibrate_outputs(w3, x3, layout, out, best_err, best_amax, w_q, packed, scale_e4m3, global_scale):
    g, c_out, c_in = w3.shape
    if layout == "channel":
        lay, n_tok = LH_LAYOUT_CHANNEL_MAJOR, x3.shape[2]
    elif layout == "token":
        lay, n_tok = LH_LAYOUT_TOKEN_MAJOR, x3.shape[1]
    else:
        raise ValueError("layout must be 'channel' or 'token'")
    if n_tok > 0 and x3.stride(-1) != 1:
        raise ValueError("last dim of x must be contiguous")
    nb = c_in // BLOCK
    dev = w3.device
    out = dict(out or {})

    def get(name, req, shape, dtype):
        if name in out:
            return out[name]
        return torch.empty(shape, dtype=dtype, device=dev) if req else None

    res = dict(amax=get("amax", True, (g,), torch.float32),
               h=get("h", True, (g, nb, 16, 16), torch.float32),
               idx=get("idx", True, (g, c_out, nb), torch.uint8),
               err=get("err", best_err, (g, c_out, nb), torch.float32),
               amax_blk=get("amax_blk", best_amax, (g, c_out, nb), torch.float32),
               w_q=get("w_q", w_q, (g, c_out, c_in), torch.float32),
               packed=get("packed", packed, (g, c_out, c_in // 2), torch.uint8),
               scale_e4m3=get("scale_e4m3", scale_e4m3, (g, c_out, nb), torch.uint8),
               global_scale=get("global_scale", global_scale, (g,), torch.float32))
    if n_tok > 0:
        ld_x = _ld(x3)
    else:  # nothing is read; any row stride the boundary accepts
        ld_x = 1 if lay == LH_LAYOUT_CHANNEL_MAJOR else max(c_in, 1)
    return res, lay, n_tok, ld_x


def lh_calibrate_nvfp4(w: torch.Tensor, x: torch.Tensor, layout: str = "channel", out: dict | None = None,
                       best_err: bool = True, best_amax: bool = True, w_q: bool = True, packed: bool = False,
                       scale_e4m3: bool = False, global_scale: bool = False,
                       workspace: torch.Tensor | None = None, split: bool = False) -> dict:
    """The whole path: global amax, normalised local Hessians (x
    [.., c_in, N] channel-major or [.., N, c_in] token-major), the
    126-candidate sweep and the fake-quant of its result.  Returns a dict
    with amax, h, idx and the requested outputs (err, amax_blk, w_q, packed,
    scale_e4m3, global_scale); tensors given in `out` under those names are
    written in place.  split=True makes the same computation as the two calls
    lh_calibrate_prologue and lh_calibrate_sweep."""
    _require_device(w, x)
    w3, x3 = _as3(w), _as3(x)
    if w3.stride(-1) != 1:
        raise ValueError("last dim of w must be contiguous")
    g, c_out, c_in = w3.shape
    res, lay, n_tok, ld_x = _calibrate_outputs(w3, x3, layout, out, best_err, best_amax, w_q, packed, scale_e4m3,
                                               global_scale)
    if workspace is None:
        workspace = torch.empty(max(lh_calibrate_workspace_bytes(c_out, c_in, n_tok, g), 1), dtype=torch.uint8,
                                device=w.device)
    wsb = workspace.numel() * workspace.element_size()
    h = res["h"]
    h_gstride = h.stride(0) if h.dim() == 4 and h.shape[0] > 1 else 0
    wargs = (_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3))
    fq = (_ptr(res["w_q"]), _ptr(res["packed"]), _ptr(res["scale_e4m3"]), _ptr(res["global_scale"]))
    if split:
        _check(lib.lh_calibrate_prologue(*wargs, _ptr(x3), _dtype(x3), lay, n_tok, ld_x, _group_stride(x3),
                                         _ptr(res["amax"]), _ptr(h), h_gstride, _ptr(workspace), wsb, _stream(w)))
        _check(lib.lh_calibrate_sweep(*wargs, _ptr(h), h_gstride, _ptr(res["amax"]), _ptr(res["idx"]),
                                      _ptr(res["err"]), _ptr(res["amax_blk"]), *fq, _ptr(workspace), wsb,
                                      _stream(w)))
    else:
        _check(lib.lh_calibrate_nvfp4(*wargs, _ptr(x3), _dtype(x3), lay, n_tok, ld_x, _group_stride(x3),
                                      _ptr(res["amax"]), _ptr(h), h_gstride, _ptr(res["idx"]), _ptr(res["err"]),
                                      _ptr(res["amax_blk"]), *fq, _ptr(workspace), wsb, _stream(w)))
    return {k: v for k, v in res.items() if v is not None}


def lh_calibrate_nvfp4_noalloc(w: torch.Tensor, x: torch.Tensor, layout: str = "channel", out: dict | None = None,
                               best_err: bool = True, best_amax: bool = True, w_q: bool = True, packed: bool = False,
                               scale_e4m3: bool = False, global_scale: bool = False) -> dict:
    """lh_calibrate_nvfp4 through the entry point that takes no workspace
    (its scratch is a fixed device array in the library, 32 MiB per GPU).
    Outputs given in `out` are written in place; missing ones are created
    here (the C call itself allocates nothing)."""
    _require_device(w, x)
    w3, x3 = _as3(w), _as3(x)
    if w3.stride(-1) != 1:
        raise ValueError("last dim of w must be contiguous")
    g, c_out, c_in = w3.shape
    res, lay, n_tok, ld_x = _calibrate_outputs(w3, x3, layout, out, best_err, best_amax, w_q, packed, scale_e4m3,
                                               global_scale)
    h = res["h"]
    h_gstride = h.stride(0) if h.dim() == 4 and h.shape[0] > 1 else 0
    _check(lib.lh_calibrate_nvfp4_noalloc(_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3), _ptr(x3),
                                          _dtype(x3), lay, n_tok, ld_x, _group_stride(x3), _ptr(res["amax"]), _ptr(h),
                                          h_gstride, _ptr(res["idx"]), _ptr(res["err"]), _ptr(res["amax_blk"]),
                                          _ptr(res["w_q"]), _ptr(res["packed"]), _ptr(res["scale_e4m3"]),
                                          _ptr(res["global_scale"]), _stream(w)))
    return {k: v for k, v in res.items() if v is not None}


def lh_calibrate_prologue(w: torch.Tensor, x: torch.Tensor, amax: torch.Tensor, h: torch.Tensor,
                          workspace: torch.Tensor, layout: str = "channel") -> None:
    """amax, h and the sweep's certificates (left in workspace) for
    lh_calibrate_sweep; output tensors given."""
    _require_device(w, x, amax, h, workspace)
    w3, x3 = _as3(w), _as3(x)
    g, c_out, c_in = w3.shape
    _, lay, n_tok, ld_x = _calibrate_outputs(w3, x3, layout, dict(amax=amax, h=h, idx=None), False, False, False,
                                             False, False, False)
    h_gstride = h.stride(0) if h.dim() == 4 and h.shape[0] > 1 else 0
    _check(lib.lh_calibrate_prologue(_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3), _ptr(x3),
                                     _dtype(x3), lay, n_tok, ld_x, _group_stride(x3), _ptr(amax), _ptr(h), h_gstride,
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(w)))


def lh_calibrate_sweep(w: torch.Tensor, h: torch.Tensor, amax: torch.Tensor, workspace: torch.Tensor,
                       best_idx: torch.Tensor, best_err=None, best_amax=None, w_q=None, packed=None, scale_e4m3=None,
                       global_scale=None) -> None:
    """The sweep and fake-quant with the certificates lh_calibrate_prologue
    left in workspace; output tensors given (None to skip)."""
    _require_device(w, h, amax, workspace, best_idx)
    w3 = _as3(w)
    g, c_out, c_in = w3.shape
    h_gstride = h.stride(0) if h.dim() == 4 and h.shape[0] > 1 else 0
    _check(lib.lh_calibrate_sweep(_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3), _ptr(h),
                                  h_gstride, _ptr(amax), _ptr(best_idx), _ptr(best_err), _ptr(best_amax), _ptr(w_q),
                                  _ptr(packed), _ptr(scale_e4m3), _ptr(global_scale), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(w)))


def lh_select_scales(rule: int, w: torch.Tensor, h: torch.Tensor | None, amax: torch.Tensor,
                     best_idx: torch.Tensor | None = None, best_err: torch.Tensor | bool | None = True,
                     best_amax: torch.Tensor | bool | None = True,
                     workspace: torch.Tensor | bool | None = True):
    """Block scales by rule (LH_RULE_SWEEP / MAX / FOUR_OVER_SIX /
    AMAX_SEARCH) under dw^T H_b dw, or the plain weight error when h is
    None.  Same outputs as lh_scale_sweep."""
    return _select(rule, w, h, amax, best_idx, best_err, best_amax, workspace)


def lh_fake_quant_nvfp4(w: torch.Tensor, best_idx: torch.Tensor, amax: torch.Tensor,
                        w_q: bool | torch.Tensor = True, packed: bool | torch.Tensor = False,
                        scale_e4m3: bool | torch.Tensor = False,
                        global_scale: bool | torch.Tensor = False) -> dict:
    """NVFP4 fake-quant / packing with the chosen block scales.  Returns a
    dict with the requested outputs: w_q [g, c_out, c_in] fp32, packed
    [g, c_out, c_in/2] uint8, scale_e4m3 [g, c_out, c_in/16] uint8,
    global_scale [g] fp32."""
    _require_device(w, best_idx, amax)
    w3 = _as3(w)
    if w3.stride(-1) != 1:
        raise ValueError("last dim of w must be contiguous")
    g, c_out, c_in = w3.shape
    res = _fq_outputs(w3, w_q, packed, scale_e4m3, global_scale)
    _check(lib.lh_fake_quant_nvfp4(_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3),
                                   _ptr(best_idx), _ptr(amax), _ptr(res["w_q"]), _ptr(res["packed"]),
                                   _ptr(res["scale_e4m3"]), _ptr(res["global_scale"]), _stream(w)))
    return {k: v for k, v in res.items() if v is not None}


def lh_full_hessian(x: torch.Tensor, alpha: float | None = None, h: torch.Tensor | None = None) -> torch.Tensor:
    """Full C_in x C_in Hessian alpha X X^T of channel-major x [.., c_in, N]
    (alpha defaults to 1/N)."""
    _require_device(x, h)
    x3 = _as3(x)
    g, c_in, n = x3.shape
    if n > 0 and x3.stride(-1) != 1:
        raise ValueError("last dim of x must be contiguous")
    if alpha is None:
        alpha = float("nan")   # the library applies 1/N
    if h is None:
        h = torch.empty((g, c_in, c_in), dtype=torch.float32, device=x.device)
    h3 = _as3(h)
    ld = _ld(x3) if n > 0 else 1  # no token: nothing is read
    _check(lib.lh_full_hessian(_ptr(x3), _dtype(x3), c_in, n, ld, g, _group_stride(x3), float(alpha),
                               _ptr(h3), _ld(h3), _group_stride(h3), _stream(x)))
    return h


def lh_output_error_workspace_bytes(c_out: int, c_in: int, n_groups: int = 1) -> int:
    return int(lib.lh_output_error_workspace_bytes(c_out, c_in, n_groups))


def lh_output_error(w: torch.Tensor, w_q: torch.Tensor, h_full: torch.Tensor, err: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Per-row d H d^T with d = w_q - w ([n_groups, c_out])."""
    _require_device(w, w_q, h_full, err, workspace)
    w3, q3, h3 = _as3(w), _as3(w_q), _as3(h_full)
    if q3.dtype != torch.float32 or h3.dtype != torch.float32:
        raise TypeError("w_q and h_full must be float32")
    g, c_out, c_in = w3.shape
    if err is None:
        err = torch.empty((g, c_out), dtype=torch.float32, device=w.device)
    if workspace is None:
        workspace = torch.empty(max(lh_output_error_workspace_bytes(c_out, c_in, g), 4), dtype=torch.uint8,
                                device=w.device)
    _check(lib.lh_output_error(_ptr(w3), _dtype(w3), _ptr(q3), c_out, c_in, _ld(w3), _ld(q3), g,
                               _group_stride(w3), _group_stride(q3), _ptr(h3), _ld(h3), _group_stride(h3),
                               _ptr(err), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(w)))
    return err


def lh_scaled_histogram(w: torch.Tensor, best_idx: torch.Tensor, amax: torch.Tensor, n_bins: int = 160,
                        bins_per_unit: float = 20.0, counts: torch.Tensor | None = None) -> torch.Tensor:
    """Counts [n_groups, n_bins + 1] (int64 storage of uint64 counts) of
    W/s = fl32(|w| / s_k), bins of width 1/bins_per_unit, last = overflow."""
    _require_device(w, best_idx, amax, counts)
    w3 = _as3(w)
    g, c_out, c_in = w3.shape
    if counts is None:
        counts = torch.empty((g, n_bins + 1), dtype=torch.int64, device=w.device)
    _check(lib.lh_scaled_histogram(_ptr(w3), _dtype(w3), c_out, c_in, _ld(w3), g, _group_stride(w3),
                                   _ptr(best_idx), _ptr(amax), int(n_bins), float(bins_per_unit), _ptr(counts),
                                   _stream(w)))
    return counts


def lh_gptq_workspace_bytes(c_out: int, c_in: int) -> int:
    return int(lib.lh_gptq_workspace_bytes(c_out, c_in))


def _gptq_ws(c_out, c_in, device, workspace):
    if workspace is not None:
        return workspace
    return torch.empty(max(lh_gptq_workspace_bytes(c_out, c_in), 16), dtype=torch.uint8, device=device)


def lh_gptq_prepare(h_full: torch.Tensor, damp: float = 0.01, u: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Upper u with (H + damp mean(diag H) I)^-1 = u^T u, from one layer's
    full Hessian [c_in, c_in] (fp32)."""
    _require_device(h_full, u, workspace)
    h2 = h_full.reshape(h_full.shape[-2], h_full.shape[-1])
    c_in = h2.shape[0]
    if u is None:
        u = torch.empty((c_in, c_in), dtype=torch.float32, device=h_full.device)
    ws = _gptq_ws(0, c_in, h_full.device, workspace)
    _check(lib.lh_gptq_prepare(_ptr(h2), c_in, h2.stride(0), float(damp), _ptr(u), u.stride(0), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(h_full)))
    return u


def lh_gptq_quantize(w: torch.Tensor, best_idx: torch.Tensor, amax: torch.Tensor, u: torch.Tensor,
                     w_q: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """GPTQ rounding of one layer's w [c_out, c_in] with fixed block scales
    (best_idx [c_out, c_in/16], global amax device scalar); returns the
    dequantised fp32 weights."""
    _require_device(w, best_idx, amax, u, w_q, workspace)
    w2 = w.reshape(w.shape[-2], w.shape[-1])
    if w2.stride(-1) != 1:
        raise ValueError("last dim of w must be contiguous")
    c_out, c_in = w2.shape
    if w_q is None:
        w_q = torch.empty((c_out, c_in), dtype=torch.float32, device=w.device)
    ws = _gptq_ws(c_out, c_in, w.device, workspace)
    ld_w = w2.stride(0) if c_out > 1 else c_in
    _check(lib.lh_gptq_quantize(_ptr(w2), _dtype(w2), c_out, c_in, ld_w, _ptr(best_idx), _ptr(amax), _ptr(u),
                                u.stride(0), _ptr(w_q), w_q.stride(0) if c_out > 1 else c_in, _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(w)))
    return w_q


def _row_stride(t: torch.Tensor) -> int:
    """Row stride of a 2-D or 3-D tensor (a single row, or a tensor without
    elements, has no meaningful one)."""
    return t.stride(-2) if t.shape[-2] > 1 and t.numel() > 0 else t.shape[-1]


def _whole_rows(t: torch.Tensor) -> bool:
    """Whether a row's elements follow one another (in a single column, or
    without elements, they do whatever the stride)."""
    return t.stride(-1) == 1 or t.shape[-1] == 1 or t.numel() == 0


def _dense(t: torch.Tensor | None, name: str, dtype, shape=None) -> None:
    """The library takes these as dense arrays of one type."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _scratch(first: torch.Tensor, t: torch.Tensor):
    """A caller's workspace and its bytes."""
    _on_device(first, t)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t, t.numel() * t.element_size()


def _on_device(first: torch.Tensor, *others) -> None:
    """All given tensors on one ROCm device."""
    d = first.get_device()
    if d < 0:
        raise ValueError("liblh works on device tensors only (got a %s tensor)" % first.device)
    for t in others:
        if t is not None and t.get_device() != d:
            if not t.is_cuda:
                raise ValueError("liblh works on device tensors only (got a %s tensor)" % t.device)
            raise ValueError("tensors on different devices (%s and %s)" % (first.device, t.device))


def lh_quantize_nvfp4(x: torch.Tensor, amax: torch.Tensor, values: bool | torch.Tensor = True,
                      packed: bool | torch.Tensor = False, scale_e4m3: bool | torch.Tensor = False,
                      global_scale: bool | torch.Tensor = False, values_dtype: torch.dtype | None = None) -> dict:
    """Activations to NVFP4 in one pass, block scales by the max rule.  x
    [rows, c_in] or [n_groups, rows, c_in]; amax fp32 [n_groups] (device),
    from the calibration or lh_absmax.  Returns a dict with the requested
    outputs: values [g, rows, c_in] = r * c in units of S_g (exact; x's dtype
    unless values_dtype says otherwise), packed, scale_e4m3, global_scale as
    lh_fake_quant_nvfp4.  The format has no infinity and no NaN: they leave as
    the block's largest value, and show in global_scale where amax is theirs."""
    _on_device(x, amax)
    x3 = _as3(x)
    if not _whole_rows(x3):
        raise ValueError("last dim of x must be contiguous")
    g, rows, c_in = x3.shape
    _dense(amax, "amax", torch.float32, (g,))
    dev = x.device

    def out(req, shape, dtype, name):
        if isinstance(req, torch.Tensor):
            _on_device(x, req)
            _dense(req, name, dtype, shape)
            return req
        return torch.empty(shape, dtype=dtype, device=dev) if req else None

    vdt = values.dtype if isinstance(values, torch.Tensor) else values_dtype or x.dtype
    res = dict(values=out(values, (g, rows, c_in), vdt, "values"),
               packed=out(packed, (g, rows, c_in // 2), torch.uint8, "packed"),
               scale_e4m3=out(scale_e4m3, (g, rows, c_in // BLOCK), torch.uint8, "scale_e4m3"),
               global_scale=out(global_scale, (g,), torch.float32, "global_scale"))
    v = res["values"]
    _check(lib.lh_quantize_nvfp4(_ptr(x3), _dtype(x3), rows, c_in, _row_stride(x3), g, _group_stride(x3), _ptr(amax),
                                 _ptr(v), LH_DTYPE_F32 if v is None else _dtype(v), _ptr(res["packed"]),
                                 _ptr(res["scale_e4m3"]), _ptr(res["global_scale"]), _stream(x)))
    return {k: t for k, t in res.items() if t is not None}


def lh_linear_nvfp4_workspace_bytes(n_rows: int, c_in: int, c_out: int, n_groups: int = 1,
                                    dtype: torch.dtype = torch.bfloat16, grad: bool = False, ragged: bool = False,
                                    max_group_rows: int = 0) -> int:
    code = LH_DTYPE_BF16 if dtype == torch.bfloat16 else LH_DTYPE_F32
    return int(lib.lh_linear_nvfp4_workspace_bytes(int(grad), int(ragged), code, n_rows, c_in, c_out, n_groups,
                                                   max_group_rows))


def _linear(x, offsets, packed, scale_e4m3, global_scale, x_scale, y, out_dtype, max_group_rows, workspace, grad):
    """The four product calls: x [rows, .] or [g, rows, .]; offsets None or int64 [g + 1]."""
    _on_device(x, offsets, packed, scale_e4m3, global_scale, x_scale, y)
    x3, p3, s3 = _as3(x), _as3(packed), _as3(scale_e4m3)
    g, c_out, half = p3.shape
    c_in = 2 * half
    _dense(p3, "packed", torch.uint8)
    _dense(s3, "scale_e4m3", torch.uint8, (g, c_out, c_in // BLOCK))
    _dense(global_scale, "global_scale", torch.float32)
    _dense(x_scale, "x_scale", torch.float32)
    if global_scale.numel() != g or x_scale is not None and x_scale.numel() != g:
        raise ValueError("global_scale and x_scale need one value for each of the %d groups" % g)
    k, m = (c_out, c_in) if grad else (c_in, c_out)
    rows = x3.shape[1]
    if x3.shape[2] != k:
        raise ValueError("the input has %d columns, the weights need %d" % (x3.shape[2], k))
    if not _whole_rows(x3):
        raise ValueError("last dim of the input must be contiguous")
    if offsets is None:
        if x3.shape[0] != g:
            raise ValueError("the input has %d groups, the weights %d" % (x3.shape[0], g))
    else:
        if x.dim() != 2:
            raise ValueError("ragged rows are a 2-D tensor")
        _dense(offsets, "offsets", torch.int64, (g + 1,))
    shape = tuple(x.shape[:-1]) + (m,)
    if y is None:
        y = torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    elif tuple(y.shape) != shape or not _whole_rows(y):
        raise ValueError("the output must have shape %s and a contiguous last dim" % (shape,))
    y3 = _as3(y)
    ws, ws_bytes = None, 0
    if workspace is True:
        ws_bytes = lh_linear_nvfp4_workspace_bytes(rows, c_in, c_out, g, x.dtype, grad, offsets is not None,
                                                   max_group_rows)
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    elif isinstance(workspace, torch.Tensor):
        ws, ws_bytes = _scratch(x, workspace)
    xa = (_ptr(x3), _dtype(x3), rows, k, _row_stride(x3))
    wa = (_ptr(p3), _ptr(s3), _ptr(global_scale), m)
    ya = (_ptr(y3), _dtype(y3), _row_stride(y3))
    end = (_ptr(ws), ws_bytes, _stream(x))
    xs = () if grad else (_ptr(x_scale),)
    if offsets is None:
        f = lib.lh_linear_nvfp4_grad if grad else lib.lh_linear_nvfp4
        _check(f(*xa, _group_stride(x3), *wa, g, *xs, *ya, _group_stride(y3), *end))
    else:
        f = lib.lh_linear_nvfp4_ragged_grad if grad else lib.lh_linear_nvfp4_ragged
        _check(f(*xa, _ptr(offsets), g, int(max_group_rows), *wa, *xs, *ya, *end))
    return y


def lh_linear_nvfp4(x: torch.Tensor, packed: torch.Tensor, scale_e4m3: torch.Tensor, global_scale: torch.Tensor,
                    x_scale: torch.Tensor | None = None, y: torch.Tensor | None = None,
                    out_dtype: torch.dtype | None = None,
                    workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """y = x W^T with NVFP4 weights as lh_fake_quant_nvfp4 / lh_calibrate_nvfp4
    return them (packed [g, c_out, c_in/2], scale_e4m3 [g, c_out, c_in/16],
    global_scale [g]).  x [n_tokens, c_in] (one group) or [g, n_tokens, c_in],
    bf16 or fp32; y in x's dtype unless out_dtype or y says otherwise.
    x_scale: S_g of activations given as lh_quantize_nvfp4 values."""
    return _linear(x, None, packed, scale_e4m3, global_scale, x_scale, y, out_dtype, 0, workspace, False)


def lh_linear_nvfp4_grad(dy: torch.Tensor, packed: torch.Tensor, scale_e4m3: torch.Tensor,
                         global_scale: torch.Tensor, dx: torch.Tensor | None = None,
                         out_dtype: torch.dtype | None = None,
                         workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """dx = dy W, the gradient of lh_linear_nvfp4 to its input (frozen weights)."""
    return _linear(dy, None, packed, scale_e4m3, global_scale, None, dx, out_dtype, 0, workspace, True)


def lh_linear_nvfp4_ragged(x: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor, scale_e4m3: torch.Tensor,
                           global_scale: torch.Tensor, x_scale: torch.Tensor | None = None,
                           y: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                           max_group_rows: int = 0, workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """lh_linear_nvfp4 for x [n_rows, c_in] whose rows offsets[g] ..
    offsets[g+1]-1 (device int64 [g + 1]) meet the weights of group g; rows of
    no group are not written."""
    return _linear(x, offsets, packed, scale_e4m3, global_scale, x_scale, y, out_dtype, max_group_rows, workspace,
                   False)


def lh_linear_nvfp4_ragged_grad(dy: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                                scale_e4m3: torch.Tensor, global_scale: torch.Tensor,
                                dx: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                                max_group_rows: int = 0,
                                workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """dx = dy W row by row, the gradient of lh_linear_nvfp4_ragged to its input."""
    return _linear(dy, offsets, packed, scale_e4m3, global_scale, None, dx, out_dtype, max_group_rows, workspace,
                   True)


def lh_moe_sort_workspace_bytes(n_tokens: int, top_k: int, n_groups: int) -> int:
    return int(lib.lh_moe_sort_workspace_bytes(n_tokens, top_k, n_groups))


def lh_moe_sort(expert_ids: torch.Tensor, n_groups: int, order: bool = True,
                workspace: torch.Tensor | None = None) -> dict:
    """Assignments [n_tokens, top_k] (int32 or int64 expert ids; outside
    [0, n_groups): dropped) sorted by expert, stable.  Returns offsets int64
    [n_groups + 1], position int32 [n_tokens, top_k] (the row, or -1 - row of
    a dropped one) and, with order=True, order int32 [n_tokens * top_k] (the
    assignment of each row, or -1 - it)."""
    _on_device(expert_ids)
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [n_tokens, top_k]")
    if expert_ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("expert_ids must be int32 or int64, got %s" % expert_ids.dtype)
    if not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be contiguous")
    t, k = expert_ids.shape
    i32 = dict(dtype=torch.int32, device=expert_ids.device)
    res = dict(offsets=torch.empty(n_groups + 1, dtype=torch.int64, device=expert_ids.device),
               position=torch.empty((t, k), **i32), order=torch.empty(t * k, **i32) if order else None)
    nbytes = 0
    if workspace is None:
        nbytes = lh_moe_sort_workspace_bytes(t, k, n_groups)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=expert_ids.device) if nbytes else None
    else:
        workspace, nbytes = _scratch(expert_ids, workspace)
    _check(lib.lh_moe_sort(_ptr(expert_ids), LH_INDEX_I64 if expert_ids.dtype == torch.int64 else LH_INDEX_I32, t, k,
                           n_groups, _ptr(res["offsets"]), _ptr(res["position"]), _ptr(res["order"]),
                           _ptr(workspace), nbytes, _stream(expert_ids)))
    return {key: v for key, v in res.items() if v is not None}


def _rows2(t: torch.Tensor, name: str, cols: int | None = None, like: torch.Tensor | None = None) -> torch.Tensor:
    if t.dim() != 2 or not _whole_rows(t):
        raise ValueError("%s must be 2-D with contiguous rows" % name)
    if cols is not None and t.shape[1] != cols:
        raise ValueError("%s has %d columns, expected %d" % (name, t.shape[1], cols))
    if like is not None and t.dtype != like.dtype:
        raise TypeError("%s must be %s, got %s" % (name, like.dtype, t.dtype))
    return t


def lh_moe_dispatch(x: torch.Tensor, position: torch.Tensor, xs: torch.Tensor | None = None) -> torch.Tensor:
    """Tokens' rows to their experts: xs[position[t, k]] = x[t], zero rows for
    dropped assignments; xs [n_tokens * top_k, cols] unless given.  Rows that
    position does not name are not written."""
    _on_device(x, position, xs)
    _rows2(x, "x")
    t, cols = x.shape
    _dense(position, "position", torch.int32)
    if position.dim() != 2 or position.shape[0] != t:
        raise ValueError("position must be [n_tokens, top_k]")
    k = position.shape[1]
    if xs is None:
        xs = torch.empty((t * k, cols), dtype=x.dtype, device=x.device)
    _rows2(xs, "xs", cols, x)
    _check(lib.lh_moe_dispatch(_ptr(x), _dtype(x), t, cols, _row_stride(x), _ptr(position), k, _ptr(xs), xs.shape[0],
                               _row_stride(xs), _stream(x)))
    return xs


def lh_moe_combine(ys: torch.Tensor, position: torch.Tensor, weights: torch.Tensor | None = None,
                   y: torch.Tensor | None = None) -> torch.Tensor:
    """Rows back to their tokens: y[t] = sum_k weights[t, k] ys[position[t, k]]
    over the assignments that have an expert (weights fp32, None: 1)."""
    _on_device(ys, position, weights, y)
    _rows2(ys, "ys")
    _dense(position, "position", torch.int32)
    if position.dim() != 2:
        raise ValueError("position must be [n_tokens, top_k]")
    t, k = position.shape
    _dense(weights, "weights", torch.float32, (t, k))
    cols = ys.shape[1]
    if y is None:
        y = torch.empty((t, cols), dtype=ys.dtype, device=ys.device)
    _rows2(y, "y", cols, ys)
    if y.shape[0] != t:
        raise ValueError("y must have one row per token")
    _check(lib.lh_moe_combine(_ptr(ys), _dtype(ys), ys.shape[0], cols, _row_stride(ys), _ptr(position),
                              _ptr(weights), t, k, _ptr(y), _row_stride(y), _stream(ys)))
    return y


def lh_moe_combine_grad(dy: torch.Tensor, ys: torch.Tensor, position: torch.Tensor,
                        weights: torch.Tensor | None = None, dys: torch.Tensor | bool = True,
                        dweights: torch.Tensor | bool = True):
    """Gradients of lh_moe_combine: (dys, dweights) with dys[position[t, k]] =
    weights[t, k] dy[t] (zero rows for dropped assignments) and dweights[t, k]
    = <dy[t], ys[position[t, k]]>; None where not requested (False).  Rows of
    ys beyond the assignments have no gradient: zero, or in a dys of the
    caller's left as they are.  (As many rows as assignments: position names
    each once, as lh_moe_sort leaves it.)"""
    _on_device(dy, ys, position, weights)
    _rows2(dy, "dy")
    t, cols = dy.shape
    _rows2(ys, "ys", cols, dy)
    _dense(position, "position", torch.int32)
    if position.dim() != 2 or position.shape[0] != t:
        raise ValueError("position must be [n_tokens, top_k]")
    k = position.shape[1]
    _dense(weights, "weights", torch.float32, (t, k))
    if dys is True:  # the kernel writes the rows that position names
        new = torch.empty if ys.shape[0] == t * k else torch.zeros
        dys = new(ys.shape, dtype=ys.dtype, device=ys.device)
    elif dys is False:
        dys = None
    if dys is not None:
        _on_device(dy, dys)
        _rows2(dys, "dys", cols, dy)
        if dys.shape[0] != ys.shape[0]:
            raise ValueError("dys must have ys's rows")
    if dweights is True:
        dweights = torch.empty((t, k), dtype=torch.float32, device=dy.device)
    elif dweights is False:
        dweights = None
    if dweights is not None:
        _on_device(dy, dweights)
        _dense(dweights, "dweights", torch.float32, (t, k))
    _check(lib.lh_moe_combine_grad(_ptr(dy), _dtype(dy), t, cols, _row_stride(dy), _ptr(ys), ys.shape[0],
                                   _row_stride(ys), _ptr(position), k, _ptr(weights), _ptr(dys),
                                   0 if dys is None else _row_stride(dys), _ptr(dweights), _stream(dy)))
    return dys, dweights


def _launch(first: torch.Tensor, f, *args) -> None:
    """The call with first's device as the current one, on that device's current stream."""
    d = first.get_device()
    if d == torch.cuda.current_device():
        _check(f(*args, _stream(first)))
    else:
        with torch.cuda.device(d):
            _check(f(*args, _stream(first)))


def _segments(first: torch.Tensor, n_rows: int, n_adapters: int, offsets, adapter_ids):
    """The arguments that say which rows take which adapter: (offsets, ids, type of the ids, segments)."""
    if offsets is not None:
        _dense(offsets, "offsets", torch.int64)
        if offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError("offsets must be [n_segments + 1]")
        n = offsets.shape[0] - 1
    else:
        n = n_rows if adapter_ids is not None and adapter_ids.shape != (1,) else 1
    kind = LH_INDEX_I32
    if adapter_ids is not None:
        if adapter_ids.dtype == torch.int64:
            kind = LH_INDEX_I64
        elif adapter_ids.dtype != torch.int32:
            raise TypeError("adapter_ids must be int32 or int64, got %s" % adapter_ids.dtype)
        _dense(adapter_ids, "adapter_ids", adapter_ids.dtype, (n,))
    elif n > n_adapters:
        raise ValueError("without adapter_ids the %d segments need an adapter each (there are %d)" % (n, n_adapters))
    _on_device(first, offsets, adapter_ids)
    return _ptr(offsets), _ptr(adapter_ids), kind, n


def lh_lora_workspace_bytes(n_rows: int, n_segments: int, c_in: int, c_out: int, rank: int, grad: bool = False) -> int:
    return int(lib.lh_lora_workspace_bytes(int(grad), n_rows, n_segments, c_in, c_out, rank))


def _lora(x, a, b, scale, offsets, adapter_ids, base, y, s, out_dtype, workspace, grad):
    """The product and its gradient: x [n_rows, .] into rows of the other factor's columns."""
    _on_device(x, a, b, scale, base, y)
    _rows2(x, "the input")
    a3, b3 = _as3(a), _as3(b)
    n, rank, c_in = a3.shape
    c_out = b3.shape[2]
    if b3.shape[:2] != a3.shape[:2]:
        raise ValueError("a and b must agree in adapters and rank, got %s and %s" % (tuple(a.shape), tuple(b.shape)))
    if b3.dtype != a3.dtype:
        raise TypeError("a and b must have one type, got %s and %s" % (a.dtype, b.dtype))
    _dense(a3, "a", a3.dtype)
    _dense(b3, "b", b3.dtype)
    _dense(scale, "scale", torch.float32, (n,))
    k, m = (c_out, c_in) if grad else (c_in, c_out)
    rows, cols = x.shape
    if cols != k:
        raise ValueError("the input has %d columns, the adapters need %d" % (cols, k))
    if y is None:
        y = torch.empty((rows, m), dtype=out_dtype or (x if base is None else base).dtype, device=x.device)
    _rows2(y, "the output", m)
    if base is not None:
        _rows2(base, "base", m, y)
    if y.shape[0] != rows or base is not None and base.shape[0] != rows:
        raise ValueError("the output and base must have the input's %d rows" % rows)
    off, ids, kind, segments = _segments(x, rows, n, offsets, adapter_ids)
    if s is True:
        s = torch.empty((rows, rank), dtype=torch.float32, device=x.device)
    elif s is False:
        s = None
    if s is not None:
        _on_device(x, s)
        _dense(s, "s", torch.float32, (rows, rank))
    if workspace is None:
        nbytes = int(lib.lh_lora_workspace_bytes(int(grad), rows, segments, c_in, c_out, rank))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    else:
        ws, nbytes = _scratch(x, workspace)
    _launch(x, lib.lh_lora_grad if grad else lib.lh_lora, _ptr(x), _dtype(x), rows, k, _row_stride(x), off, ids, kind,
            segments, _ptr(a3), _ptr(b3), _dtype(a3), n, rank, _ptr(scale), _ptr(base),
            m if base is None else _row_stride(base), m, _ptr(y), _dtype(y), _row_stride(y), _ptr(s), _ptr(ws), nbytes)
    return y if s is None else (y, s)


def lh_lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor | None = None,
            offsets: torch.Tensor | None = None, adapter_ids: torch.Tensor | None = None,
            base: torch.Tensor | None = None, y: torch.Tensor | None = None, s: torch.Tensor | bool = False,
            out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None):
    """y = base + scale[g] (x a[g]^T) b[g], row by row with the adapter g of the
    row's segment.  x [n_rows, c_in]; a [n_adapters, rank, c_in] and b
    [n_adapters, rank, c_out] (2-D: one adapter), rank-major both; scale fp32
    [n_adapters], times the global scale where x is in units of one (the values
    of lh_quantize_nvfp4).  offsets (device int64 [n_segments + 1]): segment i has the
    rows offsets[i] .. offsets[i+1]-1; without them every row is a segment (or
    all rows are one, with one adapter id or none).  adapter_ids (int32 or int64
    [n_segments], device): each segment's adapter, an id outside the adapters
    for none; without them segment i takes adapter i.  base [n_rows, c_out]:
    the projection's output (y=base adds to it in place); rows of no segment
    are not written.  y in base's dtype, else x's, unless out_dtype or y says
    otherwise.  With s=True (or a fp32 [n_rows, rank] tensor) returns (y, s), s
    = x a^T for lh_lora_weight_grad."""
    return _lora(x, a, b, scale, offsets, adapter_ids, base, y, s, out_dtype, workspace, False)


def lh_lora_grad(dy: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor | None = None,
                 offsets: torch.Tensor | None = None, adapter_ids: torch.Tensor | None = None,
                 base: torch.Tensor | None = None, dx: torch.Tensor | None = None, ds: torch.Tensor | bool = False,
                 out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None):
    """dx = base + scale[g] (dy b[g]^T) a[g], the gradient of lh_lora to its
    input; base is the projection's own (lh_linear_nvfp4_grad).  With ds=True
    (or a fp32 [n_rows, rank] tensor) returns (dx, ds), ds = dy b^T for
    lh_lora_weight_grad.  Other arguments as lh_lora."""
    return _lora(dy, a, b, scale, offsets, adapter_ids, base, dx, ds, out_dtype, workspace, True)


def lh_lora_weight_grad_workspace_bytes(n_rows: int, n_segments: int, n_adapters: int, rank: int, c_in: int,
                                        c_out: int) -> int:
    return int(lib.lh_lora_weight_grad_workspace_bytes(n_rows, n_segments, n_adapters, rank, c_in, c_out))


def lh_lora_weight_grad(x: torch.Tensor, dy: torch.Tensor, s: torch.Tensor | None, ds: torch.Tensor | None,
                        n_adapters: int, scale: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                        adapter_ids: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                        da: torch.Tensor | bool = True, db: torch.Tensor | bool = True, beta: float = 0.0,
                        out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None):
    """Gradients of lh_lora to its adapters: (da, db) with da[g] = scale[g]
    sum_t ds[t]^T x[t] [n_adapters, rank, c_in] and db[g] = scale[g] sum_t
    s[t]^T dy[t] [n_adapters, rank, c_out] over the rows of the segments with
    adapter g; None where not requested (False).  x as lh_lora had it, or the
    values of lh_checkpoint_pack (uint8) with x_scale its scales; s and ds from
    lh_lora and lh_lora_grad (None where only the other gradient is asked for).
    beta: what is added of da's and db's earlier contents, for which both must
    be given.  fp32 unless out_dtype, da or db says otherwise."""
    _on_device(x, dy, s, ds, scale, x_scale)
    p = ds if s is None else s
    if p is None:
        raise ValueError("s or ds is needed")
    rows, rank = p.shape
    _dense(s, "s", torch.float32, (rows, rank))
    _dense(ds, "ds", torch.float32, (rows, rank))
    _dense(scale, "scale", torch.float32, (n_adapters,))
    if x.dim() != 2 or dy.dim() != 2 or x.shape[0] != rows or dy.shape[0] != rows:
        raise ValueError("x and dy must be 2-D with the %d rows of s and ds" % rows)
    _rows2(dy, "dy")
    c_in, c_out = x.shape[1], dy.shape[1]
    if x_scale is None:
        _rows2(x, "x")
        x_code, ld_x = _dtype(x), _row_stride(x)
    else:
        _dense(x, "the checkpoint's values", torch.uint8)
        _dense(x_scale, "x_scale", torch.uint8, (rows, -(-c_in // CHECKPOINT_BLOCK)))
        x_code, ld_x = LH_DTYPE_E4M3, c_in
    if beta != 0.0 and not all(isinstance(t, torch.Tensor) or t is False for t in (da, db)):
        raise ValueError("beta needs the earlier da and db")
    given = [t.dtype for t in (da, db) if isinstance(t, torch.Tensor)]
    dtype = given[0] if given else out_dtype or torch.float32
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("the gradients must be float32 or bfloat16, got %s" % dtype)

    def out(t, cols, name):
        if t is True:
            return torch.empty((n_adapters, rank, cols), dtype=dtype, device=x.device)
        if t is False:
            return None
        _on_device(x, t)
        _dense(t, name, dtype, (n_adapters, rank, cols))
        return t

    da, db = out(da, c_in, "da"), out(db, c_out, "db")
    if da is not None and ds is None or db is not None and s is None:
        raise ValueError("da needs ds and db needs s")
    off, ids, kind, segments = _segments(x, rows, n_adapters, offsets, adapter_ids)
    if workspace is None:
        nbytes = int(lib.lh_lora_weight_grad_workspace_bytes(rows, segments, n_adapters, rank, c_in, c_out))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    else:
        ws, nbytes = _scratch(x, workspace)
    _launch(x, lib.lh_lora_weight_grad, _ptr(x), x_code, _ptr(x_scale), c_in, ld_x, _ptr(dy), _dtype(dy), c_out,
            _row_stride(dy), _ptr(s), _ptr(ds), rows, off, ids, kind, segments, n_adapters, rank, _ptr(scale),
            float(beta), _ptr(da), _ptr(db), LH_DTYPE_BF16 if dtype == torch.bfloat16 else LH_DTYPE_F32, _ptr(ws),
            nbytes)
    return da, db


def lh_checkpoint_pack(x: torch.Tensor, values: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """Activations [n_rows, cols] in 8 bits: (values, scales), uint8 [n_rows,
    cols] OCP E4M3FN codes and uint8 [n_rows, ceil(cols / 32)] E8M0 exponents of
    the power of two that 32 values of a row share (the smallest with which none
    exceeds 448).  Infinities and NaN become NaN."""
    _on_device(x, values, scales)
    _rows2(x, "x")
    rows, cols = x.shape
    blocks = -(-cols // CHECKPOINT_BLOCK)
    if values is None:
        values = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, blocks), dtype=torch.uint8, device=x.device)
    _dense(values, "values", torch.uint8, (rows, cols))
    _dense(scales, "scales", torch.uint8, (rows, blocks))
    _launch(x, lib.lh_checkpoint_pack, _ptr(x), _dtype(x), rows, cols, _row_stride(x), _ptr(values), _ptr(scales))
    return values, scales


def lh_checkpoint_unpack(values: torch.Tensor, scales: torch.Tensor, x: torch.Tensor | None = None,
                         out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The activations of lh_checkpoint_pack back: value * 2^(scale - 127), in x (bf16 or
    fp32 [n_rows, cols]) or a new tensor of out_dtype."""
    _on_device(values, scales, x)
    _dense(values, "values", torch.uint8)
    if values.dim() != 2:
        raise ValueError("values must be [n_rows, cols]")
    rows, cols = values.shape
    _dense(scales, "scales", torch.uint8, (rows, -(-cols // CHECKPOINT_BLOCK)))
    if x is None:
        x = torch.empty((rows, cols), dtype=out_dtype, device=values.device)
    _rows2(x, "x", cols)
    if x.shape[0] != rows:
        raise ValueError("x must have the values' rows")
    _launch(values, lib.lh_checkpoint_unpack, _ptr(values), _ptr(scales), rows, cols, _ptr(x), _dtype(x),
            _row_stride(x))
    return x
