"""ctypes binding of librib (the C-ABI declared in include/rib.h).

Argument marshalling only: tensors are passed as device pointers, the stream
is the caller's current torch stream, and every non-zero status raises
:class:`RibError` with the library's message. No step of the computation runs
here. There is no fallback: if librib.so is missing the import of the entry
points fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librib.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "rib.h")

RIB_BF16, RIB_F32, RIB_F16 = 0, 1, 2
STATUS = {0: "RIB_OK", 1: "RIB_ERR_INVALID_ARG", 2: "RIB_ERR_UNSUPPORTED", 3: "RIB_ERR_ALIGNMENT",
          4: "RIB_ERR_CUDA", 5: "RIB_ERR_TIMEOUT"}


# kernel launches of one training step through these entry points: forward
# (projection 1, gate 1, attention 1), rib_attention_bwd_prep 1,
# rib_window_attention_bwd 4, rib_pos_encode_bwd 3, rib_qkv_project_bwd 4
# (weight re-layout, token GEMM, token reduction, partial sums), cla_gate_bwd
# 7 (weight re-layout, token GEMM, token reduction, transposed depthwise,
# partial sums of dWpw, depthwise reductions and their sums)
LAUNCHES = {"train_step": 22}


def v_dtype():
    """torch dtype of V and dO in the padded head-major layout (the operand
    type of the P.V product)."""
    import torch
    return torch.bfloat16


class RibError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class MlpDesc(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("hidden", ctypes.c_int), ("heads", ctypes.c_int), ("R", ctypes.c_int),
                ("Wh", ctypes.c_void_p), ("bh", ctypes.c_void_p), ("Wpq", ctypes.c_void_p),
                ("Wpk", ctypes.c_void_p)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int), ("C", ctypes.c_int),
                ("heads", ctypes.c_int), ("R", ctypes.c_int), ("window", ctypes.c_int),
                ("softmax_scale", ctypes.c_float), ("mask_padding", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class ResidualNormDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_longlong), ("C", ctypes.c_int), ("rows_per_group", ctypes.c_longlong),
                ("x_dtype", ctypes.c_int), ("dtype", ctypes.c_int), ("pre", ctypes.c_int), ("post", ctypes.c_int),
                ("eps", ctypes.c_float), ("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class DiffAttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "q_len", "k_len", "q_heads", "kv_heads", "d", "dv", "dtype", "lam_dtype")] + \
        [("scale", ctypes.c_float)] + [(n, ctypes.c_int) for n in ("causal", "window", "width")] + \
        [(n, ctypes.c_longlong * 3) for n in ("q_stride", "k_stride", "v_stride", "o_stride")]


_lib: Optional[ctypes.CDLL] = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_SIGNATURES = {
    "rib_last_error": ([], ctypes.c_char_p),
    "rib_version": ([], _i),
    "rib_device_error": ([_vp], _i),
    "rib_head_pad": ([_i, _i], _i),
    "rib_pos_cache_bytes": ([ctypes.POINTER(MlpDesc), _i], _sz),
    "rib_pos_encode": ([ctypes.POINTER(MlpDesc), _i, _vp, _vp, _sz, _vp], _i),
    "rib_qkv_project": ([_vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _f, _vp, _vp, _vp, _vp], _i),
    "cla_gate_workspace_size": ([_i, _i, _i, _i], _sz),
    "cla_gate": ([_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "cla_gate_static_scratch": ([_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp], _i),
    "rib_window_attention": ([ctypes.POINTER(AttnDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i),
    "rib_layernorm": ([_vp, _i, _vp, _i, _i, _i, _vp, _vp, _f, _vp], _i),
    "rib_attention_bwd_prep": ([ctypes.POINTER(AttnDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i),
    "rib_window_attention_workspace_size": ([ctypes.POINTER(AttnDesc)], _sz),
    "rib_window_attention_bwd_workspace_size": ([ctypes.POINTER(AttnDesc)], _sz),
    "rib_window_attention_bwd": ([ctypes.POINTER(AttnDesc)] + [_vp] * 14 + [_sz, _vp], _i),
    "rib_pos_encode_bwd_workspace_size": ([ctypes.POINTER(MlpDesc), _i], _sz),
    "rib_pos_encode_bwd": ([ctypes.POINTER(MlpDesc), _i] + [_vp] * 7 + [_sz, _vp], _i),
    "rib_f32_to_bf16": ([_vp, _vp, _sz, _vp], _i),
    "rib_bf16_to_f32": ([_vp, _vp, _sz, _vp], _i),
    "rib_qkv_project_bwd_workspace_size": ([_i, _i, _i, _i, _i], _sz),
    "rib_qkv_project_bwd": ([_vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _f] + [_vp] * 7 + [_vp, _sz, _vp], _i),
    "cla_gate_bwd_workspace_size": ([_i, _i, _i, _i], _sz),
    "cla_gate_bwd": ([_vp, _i, _i, _i, _i, _i] + [_vp] * 9 + [_vp, _sz, _vp], _i),
    "rib_selftest_wait_timeout": ([_i, _vp], _i),
    "rib_selftest_mma_rate": ([_i, _i, _i, _i, _vp, _vp, _vp], _i),
    "rib_conv_ffn_workspace_size": ([_i, _i, _i, _i], _sz),
    "rib_conv_ffn": ([_vp, _i, _vp, _i, _i, _i, _i, _i] + [_vp] * 7 + [_sz, _vp], _i),
    "rib_dropout": ([_vp, _vp, _i, _sz, _f, ctypes.c_uint64, ctypes.c_uint64, _vp, _vp], _i),
    "rib_residual_norm": ([ctypes.POINTER(ResidualNormDesc)] + [_vp] * 12, _i),
    "rib_residual_norm_bwd_workspace_size": ([ctypes.POINTER(ResidualNormDesc)], _sz),
    "rib_residual_norm_bwd": ([ctypes.POINTER(ResidualNormDesc)] + [_vp] * 18 + [_sz, _vp, _vp], _i),
    "rib_diff_attention_workspace_size": ([ctypes.POINTER(DiffAttnDesc)], _sz),
    "rib_diff_attention": ([ctypes.POINTER(DiffAttnDesc)] + [_vp] * 11 + [_sz, _vp], _i),
    "rib_diff_attention_bwd_workspace_size": ([ctypes.POINTER(DiffAttnDesc)], _sz),
    "rib_diff_attention_bwd": ([ctypes.POINTER(DiffAttnDesc)] + [_vp] * 18 + [_sz, _vp], _i),
}


def header_symbols() -> list:
    """Names of the functions include/rib.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    text = "\n".join(line for line in text.splitlines() if not line.lstrip().startswith("#"))
    return sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) - {"if", "sizeof"})


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load librib.so (building it first if the sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if path is None:
        from . import build as _build
        if not _build.up_to_date():
            _build.build()
    if not os.path.exists(p):
        raise ImportError(f"librib.so not found at {p}; run python -m windowed_attention_b200.build")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        raise RibError(status, _lib.rib_last_error().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("librib entry points take device tensors")
    if not t.is_contiguous():
        raise ValueError("librib entry points take contiguous tensors")
    return t.data_ptr()


_raw_stream = None


def _stream(stream, device=None) -> Optional[int]:
    """Handle of `stream`, by default the current one of `device` (by default the current device)."""
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            # the stream's handle without a Stream object around it, where torch offers that
            get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            _raw_stream = (lambda d: get(dev() if d is None else d)) if get else (lambda d: torch.cuda.current_stream(d).cuda_stream)
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: RIB_F32, torch.float16: RIB_F16}.get(t.dtype, RIB_BF16)


# ----------------------------------------------------------------- entry points
def rib_version() -> int:
    return load().rib_version()


def rib_device_error(stream=None) -> None:
    load()
    _check(_lib.rib_device_error(_stream(stream)))


def rib_head_pad(C: int, heads: int) -> int:
    return load().rib_head_pad(C, heads)


def mlp_desc(L, hidden, heads, R, Wh, bh, Wpq, Wpk) -> MlpDesc:
    return MlpDesc(L, hidden, heads, R, _ptr(Wh), _ptr(bh), _ptr(Wpq), _ptr(Wpk))


def rib_pos_cache_bytes(desc: MlpDesc, window: int) -> int:
    return load().rib_pos_cache_bytes(ctypes.byref(desc), window)


def rib_pos_encode(desc: MlpDesc, window: int, qp_cache, kp_cache, stream=None) -> None:
    load()
    nbytes = min(qp_cache.numel() * qp_cache.element_size(), kp_cache.numel() * kp_cache.element_size())
    _check(_lib.rib_pos_encode(ctypes.byref(desc), window, _ptr(qp_cache), _ptr(kp_cache), nbytes,
                               _stream(stream)))


def rib_qkv_project(X, B, H, W, C, heads, window, Wq, Wk, Wv, q_scale, Qc, Kc, V, stream=None) -> None:
    load()
    _check(_lib.rib_qkv_project(_ptr(X), _dtype_code(X), B, H, W, C, heads, window, _ptr(Wq), _ptr(Wk), _ptr(Wv),
                                float(q_scale), _ptr(Qc), _ptr(Kc), _ptr(V), _stream(stream)))


def cla_gate_workspace_size(B, H, W, C) -> int:
    return load().cla_gate_workspace_size(B, H, W, C)


def cla_gate(X, B, H, W, C, Wdw, bdw, Wpw, bpw, sig_gate, workspace=None, stream=None) -> None:
    """sigmoid(PWConv(DWConv3x3(X))) into sig_gate; with a workspace, the
    depthwise output is left in it too (the backward's input)."""
    load()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.cla_gate(_ptr(X), _dtype_code(X), B, H, W, C, _ptr(Wdw), _ptr(bdw), _ptr(Wpw), _ptr(bpw),
                         _ptr(sig_gate), _ptr(workspace), nbytes, _stream(stream)))


def cla_gate_static_scratch(X, B, H, W, C, Wdw, bdw, Wpw, bpw, sig_gate, stream=None) -> None:
    """cla_gate for callers that cannot allocate device memory: the depthwise
    intermediate lives in the library's fixed 16 MiB per-device array (see
    include/rib.h for the size limit and the sharing rules)."""
    load()
    _check(_lib.cla_gate_static_scratch(_ptr(X), _dtype_code(X), B, H, W, C, _ptr(Wdw), _ptr(bdw), _ptr(Wpw),
                                        _ptr(bpw), _ptr(sig_gate), _stream(stream)))


def attn_desc(B, H, W, C, heads, R, window, softmax_scale=1.0, mask_padding=False, out_f32=False,
              out_f16=False) -> AttnDesc:
    """Descriptor of one attention call; Y (and the residual) are bf16, or
    fp32 with out_f32, or fp16 with out_f16."""
    out = RIB_F32 if out_f32 else (RIB_F16 if out_f16 else RIB_BF16)
    return AttnDesc(B, H, W, C, heads, R, window, float(softmax_scale), 1 if mask_padding else 0, out)


def rib_window_attention(desc: AttnDesc, Qc, Kc, V, qp_cache, kp_cache, sig_gate, residual, Y, lse=None,
                         O_out=None, stream=None) -> None:
    load()
    _check(_lib.rib_window_attention(ctypes.byref(desc), _ptr(Qc), _ptr(Kc), _ptr(V), _ptr(qp_cache),
                                     _ptr(kp_cache), _ptr(sig_gate), _ptr(residual), _ptr(Y), _ptr(lse),
                                     _ptr(O_out), _stream(stream)))


def rib_attention_bwd_prep(desc: AttnDesc, dY, sig_gate, O, dO, Dsum, dG=None, stream=None) -> None:
    load()
    _check(_lib.rib_attention_bwd_prep(ctypes.byref(desc), _ptr(dY), _ptr(sig_gate), _ptr(O), _ptr(dO), _ptr(Dsum),
                                       _ptr(dG), _stream(stream)))


def rib_window_attention_workspace_size(desc: AttnDesc) -> int:
    return load().rib_window_attention_workspace_size(ctypes.byref(desc))


def rib_window_attention_bwd_workspace_size(desc: AttnDesc) -> int:
    return load().rib_window_attention_bwd_workspace_size(ctypes.byref(desc))


def rib_window_attention_bwd(desc: AttnDesc, Qc, Kc, V, qp_cache, kp_cache, lse, dO, Dsum, dQc, dKc, dV, dQp, dKp,
                             workspace, stream=None) -> None:
    load()
    _check(_lib.rib_window_attention_bwd(ctypes.byref(desc), _ptr(Qc), _ptr(Kc), _ptr(V), _ptr(qp_cache),
                                         _ptr(kp_cache), _ptr(lse), _ptr(dO), _ptr(Dsum), _ptr(dQc), _ptr(dKc),
                                         _ptr(dV), _ptr(dQp), _ptr(dKp), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream)))


def rib_pos_encode_bwd_workspace_size(desc: MlpDesc, window: int) -> int:
    return load().rib_pos_encode_bwd_workspace_size(ctypes.byref(desc), window)


def rib_pos_encode_bwd(desc: MlpDesc, window, dqp_cache, dkp_cache, dWh, dbh, dWpq, dWpk, workspace,
                       stream=None) -> None:
    load()
    _check(_lib.rib_pos_encode_bwd(ctypes.byref(desc), window, _ptr(dqp_cache), _ptr(dkp_cache), _ptr(dWh),
                                   _ptr(dbh), _ptr(dWpq), _ptr(dWpk), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)))


def rib_qkv_project_bwd_workspace_size(B, H, W, C, heads) -> int:
    return load().rib_qkv_project_bwd_workspace_size(B, H, W, C, heads)


def rib_qkv_project_bwd(X, B, H, W, C, heads, window, Wq, Wk, Wv, q_scale, dQc, dKc, dV, dX, dWq, dWk, dWv,
                        workspace=None, stream=None) -> None:
    """workspace: a device tensor of at least rib_qkv_project_bwd_workspace_size
    bytes (allocated here when None)."""
    load()
    if workspace is None:
        import torch
        workspace = torch.empty(rib_qkv_project_bwd_workspace_size(B, H, W, C, heads), dtype=torch.uint8,
                                device=X.device)
    _check(_lib.rib_qkv_project_bwd(_ptr(X), _dtype_code(X), B, H, W, C, heads, window, _ptr(Wq), _ptr(Wk), _ptr(Wv),
                                    float(q_scale), _ptr(dQc), _ptr(dKc), _ptr(dV), _ptr(dX), _ptr(dWq), _ptr(dWk),
                                    _ptr(dWv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)))


def cla_gate_bwd_workspace_size(B, H, W, C) -> int:
    return load().cla_gate_bwd_workspace_size(B, H, W, C)


def cla_gate_bwd(X, B, H, W, C, Wdw, Wpw, D, dG, dX, dWdw, dbdw, dWpw, dbpw, workspace, stream=None) -> None:
    load()
    _check(_lib.cla_gate_bwd(_ptr(X), _dtype_code(X), B, H, W, C, _ptr(Wdw), _ptr(Wpw), _ptr(D), _ptr(dG), _ptr(dX),
                             _ptr(dWdw), _ptr(dbdw), _ptr(dWpw), _ptr(dbpw), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)))


def rib_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Make one bounded device wait run out (see include/rib.h); the next
    rib_device_error() raises RibError with the timeout status."""
    load()
    _check(_lib.rib_selftest_wait_timeout(int(limit_us), _stream(stream)))


def rib_selftest_mma_rate(ctas_per_sm: int, issuers_per_cta: int, n: int, mmas: int, stream=None):
    """Issue rate of tcgen05.mma (see include/rib.h): every SM runs
    ctas_per_sm CTAs, each with issuers_per_cta threads issuing a chain of
    `mmas` M=128, K=16, width-n products. Returns a dict with the median
    clock64 cycles per MMA of one issuing thread (to its last issue and to
    the chain's completion), the SM's aggregate cycles per MMA, and
    `overlap`: over the SMs, the smallest ratio of the time all of an SM's
    CTAs ran together to the mean CTA's run time (1 when they ran side by
    side; the aggregate figure assumes they did)."""
    import torch
    load()
    dev = torch.device("cuda", torch.cuda.current_device())
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    ctas = sms * ctas_per_sm
    cyc = torch.zeros(ctas * issuers_per_cta * 2, dtype=torch.int64, device=dev)
    spans = torch.zeros(ctas * 3, dtype=torch.int64, device=dev)
    _check(_lib.rib_selftest_mma_rate(int(ctas_per_sm), int(issuers_per_cta), int(n), int(mmas), _ptr(cyc),
                                      _ptr(spans), _stream(stream)))
    torch.cuda.synchronize(dev)
    rib_device_error()
    c = cyc.view(-1, 2).double().cpu()
    issue = float(c[:, 0].median()) / mmas
    done = float(c[:, 1].median()) / mmas
    sp = spans.view(-1, 3).cpu().tolist()
    by_sm = {}
    for smid, t0, t1 in sp:
        by_sm.setdefault(smid, []).append((t0, t1))
    overlap = 1.0
    for iv in by_sm.values():
        common = min(t1 for _, t1 in iv) - max(t0 for t0, _ in iv)
        mean = sum(t1 - t0 for t0, t1 in iv) / len(iv)
        overlap = min(overlap, max(0.0, common) / mean if mean > 0 else 0.0)
    return {"ctas_per_sm": ctas_per_sm, "issuers_per_cta": issuers_per_cta, "n": n, "mmas": mmas,
            "issue_cycles_per_mma": issue, "done_cycles_per_mma": done,
            "sm_cycles_per_mma": done / (ctas_per_sm * issuers_per_cta),
            "sms_used": len(by_sm), "max_ctas_on_an_sm": max(len(v) for v in by_sm.values()), "overlap": overlap}


def rib_layernorm(x, y, T, C, gamma=None, beta=None, eps=1e-5, stream=None) -> None:
    """y = LayerNorm(x) over C; x bf16, fp32 or fp16, y bf16 or fp16."""
    load()
    _check(_lib.rib_layernorm(_ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y), T, C, _ptr(gamma), _ptr(beta),
                              float(eps), _stream(stream)))


def rib_f32_to_bf16(x, y, stream=None) -> None:
    load()
    _check(_lib.rib_f32_to_bf16(_ptr(x), _ptr(y), x.numel(), _stream(stream)))


def rib_bf16_to_f32(x, y, stream=None) -> None:
    load()
    _check(_lib.rib_bf16_to_f32(_ptr(x), _ptr(y), x.numel(), _stream(stream)))


def rib_conv_ffn_workspace_size(B, H, W, hidden) -> int:
    return load().rib_conv_ffn_workspace_size(B, H, W, hidden)


def rib_conv_ffn(xn, x, B, H, W, C, hidden, W1, b1, Wf, bf, W2, b2, workspace, stream=None) -> None:
    """x += ConvFFN(xn) (see include/rib.h): xn bf16 or fp16, x fp32 in place."""
    load()
    _check(_lib.rib_conv_ffn(_ptr(xn), _dtype_code(xn), _ptr(x), B, H, W, C, hidden, _ptr(W1), _ptr(b1), _ptr(Wf),
                             _ptr(bf), _ptr(W2), _ptr(b2), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream)))


# ------------------------------------------------- training-block operators
# These calls check what the C interface cannot see: that every tensor is on
# the current device (the kernels run there), has its type and holds enough.
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_TORCH_CODE = {}   # filled when the first of these calls needs torch


def _codes() -> dict:
    if not _TORCH_CODE:
        import torch
        _TORCH_CODE.update({torch.bfloat16: RIB_BF16, torch.float32: RIB_F32, torch.float16: RIB_F16})
    return _TORCH_CODE


def _code(dtype) -> int:
    """RIB_* code of a torch dtype; anything but bf16, fp32 and fp16 is refused."""
    try:
        return (_TORCH_CODE or _codes())[dtype]
    except KeyError:
        raise ValueError(f"dtype {dtype}: librib takes bfloat16, float32 and float16") from None


_device_now = None


def _current_device(t) -> int:
    global _device_now
    if _device_now is None:
        import torch
        _device_now = torch.cuda.current_device
    at = t.get_device()
    if at < 0:
        raise ValueError("librib entry points take device tensors")
    if at != _device_now():
        raise ValueError(f"tensor on {t.device} while the current device is cuda:{_device_now()}: "
                         "make its device current for the call")
    return at


def _arg(name, t, numel, code, device) -> Optional[int]:
    """Pointer of a contiguous device tensor of at least `numel` values of type `code`; None stays None."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}: librib entry points take tensors of the current device, cuda:{device}")
    if _code(t.dtype) != code:
        raise ValueError(f"{name} is {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} values, {numel} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{name}: librib entry points take contiguous tensors")
    return t.data_ptr()


def _rows_of(t, want) -> bool:
    """True where `t` holds the values of a tensor of shape `want`, (rows, C) or (C,), by another shape: flat, or one that ends in C."""
    return t.numel() == want[0] * (want[1] if len(want) > 1 else 1) and (t.dim() == 1 or t.shape[-1:] == want[-1:])


def _row_arg(name, t, want, code, device) -> Optional[int]:
    """Pointer of a contiguous device tensor of type `code` that holds `want`, (rows, C) or (C,), values."""
    if t is None:
        return None
    if t.shape != want and not _rows_of(t, want):
        raise ValueError(f"{name} is {tuple(t.shape)}, the descriptor says {want}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}: librib entry points take tensors of the current device, cuda:{device}")
    if (_TORCH_CODE or _codes()).get(t.dtype) != code:
        raise ValueError(f"{name} is {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: librib entry points take contiguous tensors")
    return t.data_ptr()


def _step_arg(step, device) -> Optional[int]:
    """Pointer of the device word added to a dropout offset."""
    if step is None:
        return None
    import torch
    if step.dtype not in (torch.int64, torch.uint64) or step.numel() < 1 or step.get_device() != device:
        raise ValueError("step is one int64 or uint64 on the current device")
    return step.data_ptr()


def rib_dropout(x, y, p, seed, offset=0, step=None, stream=None) -> None:
    """y = x / keep where the element's random bits keep it, 0 elsewhere; the
    mask is a function of (element, seed, offset + step) and never stored, so
    the backward is the same call on the upstream gradient. y may be x."""
    load()
    dev, n = _current_device(x), x.numel()
    code = _code(x.dtype)
    if y.numel() != n:
        raise ValueError(f"y holds {y.numel()} values, x {n}")
    _check(_lib.rib_dropout(_arg("x", x, n, code, dev), _arg("y", y, n, code, dev), code, n, float(p), int(seed),
                            int(offset), _step_arg(step, dev), _stream(stream, dev)))


def residual_norm_desc(T, C, x_dtype, dtype, pre="layer", post="none", eps=1e-5, rows_per_group=None, p=0.0, seed=0,
                       offset=0) -> ResidualNormDesc:
    """Descriptor of one join of a block with its residual stream: T rows of C
    values, the stream in torch dtype x_dtype, the branch, gate and h in dtype;
    pre and post are "none", "layer" or "rms"; rows_per_group rows share a row
    of scale (all of them by default)."""
    for n in (pre, post):
        if n not in _NORMS:
            raise ValueError(f"norm {n!r}: one of {sorted(_NORMS)}")
    return ResidualNormDesc(T, C, max(1, T) if rows_per_group is None else rows_per_group, _code(x_dtype), _code(dtype),
                            _NORMS[pre], _NORMS[post], float(eps), float(p), int(seed), int(offset))


def _scale_shape(d: ResidualNormDesc, scale) -> tuple:
    """Rows and width of scale and its gradient; without rows of x any number of rows."""
    if d.T > 0 and d.rows_per_group > 0:
        return (-(-d.T // d.rows_per_group), d.C)
    return (0 if scale is None else scale.numel() // max(1, d.C), d.C)


def rib_residual_norm(desc: ResidualNormDesc, x, y=None, gate=None, scale=None, post_w=None, post_b=None, pre_w=None,
                      pre_b=None, x_out=None, h=None, step=None, stream=None) -> None:
    """x_out = x + dropout(scale * gate * (N_post(y) post_w + post_b)) and
    h = N_pre(x_out) pre_w + pre_b (see include/rib.h). Tensors hold the
    descriptor's rows of C values, in any shape that ends in C or flat."""
    load()
    dev, d, arg = _current_device(x), desc, _row_arg
    C, xc, c = d.C, d.x_dtype, d.dtype
    n, w = (d.T, C), (C,)
    _check(_lib.rib_residual_norm(
        ctypes.byref(d), arg("x", x, n, xc, dev), arg("y", y, n, c, dev), arg("gate", gate, n, c, dev),
        arg("scale", scale, _scale_shape(d, scale), RIB_F32, dev), arg("post_w", post_w, w, RIB_F32, dev), arg("post_b", post_b, w, RIB_F32, dev),
        arg("pre_w", pre_w, w, RIB_F32, dev), arg("pre_b", pre_b, w, RIB_F32, dev), arg("x_out", x_out, n, xc, dev), arg("h", h, n, c, dev),
        _step_arg(step, dev), _stream(stream, dev)))


def rib_residual_norm_bwd_workspace_size(desc: ResidualNormDesc) -> int:
    return load().rib_residual_norm_bwd_workspace_size(ctypes.byref(desc))


def rib_residual_norm_bwd(desc: ResidualNormDesc, x_out, y=None, gate=None, scale=None, post_w=None, post_b=None,
                          pre_w=None, dx_out=None, dh=None, dx=None, dy=None, dgate=None, dscale=None, dpost_w=None,
                          dpost_b=None, dpre_w=None, dpre_b=None, workspace=None, step=None, stream=None) -> None:
    """Gradients of rib_residual_norm from dx_out (the stream's, may be None)
    and dh; each output may be None (see include/rib.h)."""
    load()
    d, arg = desc, _row_arg
    dev = _current_device(x_out if x_out is not None else dx_out)
    C, xc, c = d.C, d.x_dtype, d.dtype
    n, w, g = (d.T, C), (C,), _scale_shape(d, dscale if scale is None else scale)
    _check(_lib.rib_residual_norm_bwd(
        ctypes.byref(d), arg("x_out", x_out, n, xc, dev), arg("y", y, n, c, dev), arg("gate", gate, n, c, dev),
        arg("scale", scale, g, RIB_F32, dev), arg("post_w", post_w, w, RIB_F32, dev), arg("post_b", post_b, w, RIB_F32, dev),
        arg("pre_w", pre_w, w, RIB_F32, dev), arg("dx_out", dx_out, n, xc, dev), arg("dh", dh, n, c, dev), arg("dx", dx, n, xc, dev),
        arg("dy", dy, n, c, dev), arg("dgate", dgate, n, c, dev), arg("dscale", dscale, g, RIB_F32, dev),
        arg("dpost_w", dpost_w, w, RIB_F32, dev), arg("dpost_b", dpost_b, w, RIB_F32, dev), arg("dpre_w", dpre_w, w, RIB_F32, dev),
        arg("dpre_b", dpre_b, w, RIB_F32, dev), *_workspace_arg(workspace, dev), _step_arg(step, dev), _stream(stream, dev)))


def diff_attn_desc(batch, q_len, k_len, q_heads, kv_heads, d, dv, scale, dtype, lam_dtype=None, causal=False, window=0, width=0,
                   q_stride=None, k_stride=None, v_stride=None, o_stride=None) -> DiffAttnDesc:
    """Descriptor of a differential attention: tensors [batch, tokens, heads,
    width] in torch dtype `dtype` (bfloat16 or float16), lam in lam_dtype
    (`dtype` by default, or float32). window and width: over the window x
    window cells of a map `width` wide instead of whole sequences. The strides
    are elements between batch items, tokens and heads (None: contiguous)."""
    s = [(ctypes.c_longlong * 3)(*(x or (0, 0, 0))) for x in (q_stride, k_stride, v_stride, o_stride)]
    return DiffAttnDesc(batch, q_len, k_len, q_heads, kv_heads, d, dv, _code(dtype), _code(dtype if lam_dtype is None else lam_dtype),
                        float(scale), int(bool(causal)), window, width, *s)


def _strided_arg(name, t, shape, strides, desc_code, device) -> Optional[int]:
    """Pointer of a device tensor [batch, tokens, heads, width] of that shape, laid out as the descriptor says."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}: librib entry points take tensors of the current device, cuda:{device}")
    if (_TORCH_CODE or _codes()).get(t.dtype) != desc_code:
        raise ValueError(f"{name} is {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, the descriptor says {shape}")
    if strides is not None:
        want = (*strides, 1)
        if t.stride() != want and any(n > 1 and a != b for n, a, b in zip(shape, t.stride(), want)):
            raise ValueError(f"{name} has strides {t.stride()}, the descriptor says {want}")
    elif not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous, and the descriptor names no strides")
    return t.data_ptr()


def _workspace_arg(ws, device):
    if ws is None:
        return None, 0
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError("workspace is a contiguous tensor of the current device")
    n = ws.numel() * ws.element_size()
    return (ws.data_ptr() if n else None), n


def _diff_layout(d):
    """Shapes and strides (None: contiguous) of the query, key, value and
    output tensors of a descriptor: kept on it for as long as its bytes stay."""
    key = bytes(d)
    kept = getattr(d, "_layout", None)
    if kept is None or kept[0] != key:
        b, nq, nk, hq, hk, e, ev = d.batch, d.q_len, d.k_len, d.q_heads, d.kv_heads, d.d, d.dv
        st = [tuple(f) if any(f) else None for f in (d.q_stride, d.k_stride, d.v_stride, d.o_stride)]
        kept = d._layout = (key, ((b, nq, hq, e), st[0]), ((b, nk, hk, e), st[1]), ((b, nk, hk, ev), st[2]), ((b, nq, hq, ev), st[3]),
                            d.dtype, d.lam_dtype, hq, b, 2 * b * hq * nq)
    return kept


def _lens_arg(k_lens, batch, device) -> Optional[int]:
    if k_lens is None:
        return None
    import torch
    if k_lens.dtype != torch.int32 or k_lens.numel() < batch or k_lens.get_device() != device or not k_lens.is_contiguous():
        raise ValueError("k_lens holds one int32 a batch item on the current device")
    return k_lens.data_ptr()


def rib_diff_attention_workspace_size(desc: DiffAttnDesc) -> int:
    return load().rib_diff_attention_workspace_size(ctypes.byref(desc))


def rib_diff_attention(desc: DiffAttnDesc, q1, q2, k1, k2, v, lam, k_lens=None, o=None, o2=None, lse=None, workspace=None,
                       stream=None) -> None:
    """o = (softmax(scale q1 k1^T) - lam softmax(scale q2 k2^T)) v; o2 and lse
    (None for inference) are what the backward needs (see include/rib.h)."""
    load()
    dev = _current_device(q1)
    _, (qs, qt), (ks, kt), (vs, vt), (os, ot), code, lam_code, heads, batch, rows = _diff_layout(desc)
    arg = _strided_arg
    _check(_lib.rib_diff_attention(
        ctypes.byref(desc), arg("q1", q1, qs, qt, code, dev), arg("q2", q2, qs, qt, code, dev), arg("k1", k1, ks, kt, code, dev),
        arg("k2", k2, ks, kt, code, dev), arg("v", v, vs, vt, code, dev), _arg("lam", lam, heads, lam_code, dev),
        _lens_arg(k_lens, batch, dev), arg("o", o, os, ot, code, dev), arg("o2", o2, os, ot, code, dev), _arg("lse", lse, rows, RIB_F32, dev),
        *_workspace_arg(workspace, dev), _stream(stream, dev)))


def rib_diff_attention_bwd_workspace_size(desc: DiffAttnDesc) -> int:
    return load().rib_diff_attention_bwd_workspace_size(ctypes.byref(desc))


def rib_diff_attention_bwd(desc: DiffAttnDesc, q1, q2, k1, k2, v, lam, k_lens, o, o2, lse, do, dq1, dq2, dk1, dk2, dv, dlam,
                           workspace, stream=None) -> None:
    """Every gradient of rib_diff_attention from do and the forward's o, o2 and
    lse (see include/rib.h)."""
    load()
    dev = _current_device(q1)
    _, (qs, qt), (ks, kt), (vs, vt), (os, ot), code, lam_code, heads, batch, rows = _diff_layout(desc)
    arg = _strided_arg
    _check(_lib.rib_diff_attention_bwd(
        ctypes.byref(desc), arg("q1", q1, qs, qt, code, dev), arg("q2", q2, qs, qt, code, dev), arg("k1", k1, ks, kt, code, dev),
        arg("k2", k2, ks, kt, code, dev), arg("v", v, vs, vt, code, dev), _arg("lam", lam, heads, lam_code, dev),
        _lens_arg(k_lens, batch, dev), arg("o", o, os, ot, code, dev), arg("o2", o2, os, ot, code, dev), _arg("lse", lse, rows, RIB_F32, dev),
        arg("do", do, os, ot, code, dev), arg("dq1", dq1, qs, qt, code, dev), arg("dq2", dq2, qs, qt, code, dev),
        arg("dk1", dk1, ks, kt, code, dev), arg("dk2", dk2, ks, kt, code, dev), arg("dv", dv, vs, vt, code, dev),
        _arg("dlam", dlam, heads, lam_code, dev), *_workspace_arg(workspace, dev), _stream(stream, dev)))
