"""KDA chunk-prefill forward for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI in ``include/kda_prefill.h``: argument
marshalling only.  Every step of the forward runs in the CUDA kernels of
``libkda_prefill.so``; there is no CPU path.  If the library is missing the
calls raise, they never fall back.

    o, final_state = forward(q, k, v, g, beta, initial_state=None, cu_seqlens=None)

Shapes ("KDA Chunk Prefill on Ascend A3", section "Function and tensor
contract"): q, k [B,T,H,128] bf16; v [B,T,HV,128] bf16; g [B,T,HV,128]
fp32; beta [B,T,HV] fp32; initial_state [N,HV,128,128] fp32 or None;
cu_seqlens [N+1] int32 or None (then B must be 1).  Returns o
[B,T,HV,128] bf16 and final_state [N,HV,128,128] fp32.

Softmax attention for the full-attention layers beside it: ``attention_forward`` and
``attention_backward`` over packed prompts, ``cache_plan``, ``cache_append`` and
``attention_decode`` over a paged 8-bit key/value cache.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libkda_prefill.so")

STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_MISALIGNED",
          4: "KDA_ERR_WORKSPACE", 5: "KDA_ERR_CUDA"}

EXPORTED = ("kda_status_string", "kda_prefill_workspace_size", "kda_prefill_forward",
            "kda_prefill_host_staging_size", "kda_prefill_forward_host", "kda_prefill_device_error",
            "kda_l2norm_bf16", "kda_prefill_kernel_launches", "kda_decode_step",
            "kda_prefill_backward_workspace_size", "kda_prefill_backward_kernel_launches", "kda_prefill_backward",
            "kda_prefill_state_bf16_workspace_size", "kda_prefill_forward_state_bf16",
            "kda_prefill_forward_save", "kda_prefill_backward_saved", "kda_prefill_forward_varlen",
            "kda_prefill_varlen_kernel_launches", "kda_attention_forward",
            "kda_attention_backward_workspace_size", "kda_attention_backward", "kda_cache_plan", "kda_cache_append",
            "kda_attention_decode_workspace_size", "kda_attention_decode")


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


_lock = threading.Lock()
_lib = None


def lib():
    """Load libkda_prefill.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run python -m kda_gated_delta_prefill_b200.build)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        L.kda_status_string.argtypes = [I]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_prefill_workspace_size.argtypes = [I] * 7
        L.kda_prefill_workspace_size.restype = Z
        L.kda_prefill_forward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, Z, P]
        L.kda_prefill_forward.restype = I
        L.kda_prefill_host_staging_size.argtypes = [I] * 9
        L.kda_prefill_host_staging_size.restype = Z
        L.kda_prefill_forward_host.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, Z, P]
        L.kda_prefill_forward_host.restype = I
        L.kda_prefill_device_error.argtypes = [P, I]
        L.kda_prefill_device_error.restype = I
        L.kda_l2norm_bf16.argtypes = [P, I64, I, P, P]
        L.kda_l2norm_bf16.restype = I
        L.kda_prefill_kernel_launches.argtypes = [I] * 7
        L.kda_prefill_kernel_launches.restype = I
        L.kda_decode_step.argtypes = [P, I64, P, I64, P, I64, P, P, P, I64, I, P, I, I, I, I, I, P, P]
        L.kda_decode_step.restype = I
        L.kda_prefill_backward_workspace_size.argtypes = [I] * 7
        L.kda_prefill_backward_workspace_size.restype = Z
        L.kda_prefill_backward_kernel_launches.argtypes = [I] * 7
        L.kda_prefill_backward_kernel_launches.restype = I
        L.kda_prefill_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, P, Z, P]
        L.kda_prefill_backward.restype = I
        L.kda_prefill_state_bf16_workspace_size.argtypes = [I] * 7
        L.kda_prefill_state_bf16_workspace_size.restype = Z
        L.kda_prefill_forward_state_bf16.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, Z, P]
        L.kda_prefill_forward_state_bf16.restype = I
        L.kda_prefill_forward_save.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, Z, P]
        L.kda_prefill_forward_save.restype = I
        L.kda_prefill_backward_saved.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, P, Z, P]
        L.kda_prefill_backward_saved.restype = I
        L.kda_prefill_forward_varlen.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, Z, P]
        L.kda_prefill_forward_varlen.restype = I
        L.kda_prefill_varlen_kernel_launches.argtypes = [I, I, I, I, I, I, P]
        L.kda_prefill_varlen_kernel_launches.restype = I
        S, F = ctypes.c_int64, ctypes.c_float
        L.kda_attention_forward.argtypes = [P, S, P, S, P, S, P, P] + [I] * 7 + [F, P, P, P]
        L.kda_attention_forward.restype = I
        L.kda_attention_backward_workspace_size.argtypes = [I] * 4
        L.kda_attention_backward_workspace_size.restype = Z
        L.kda_attention_backward.argtypes = [P, S, P, S, P, S, P, P, P, S, P, P] + [I] * 7 + [F, P, P, P, P, Z, P]
        L.kda_attention_backward.restype = I
        L.kda_cache_plan.argtypes = [P, P, I, P, S, I, P, I, I, P, P, P, I, P, P]
        L.kda_cache_plan.restype = I
        L.kda_cache_append.argtypes = [P, S, P, S, P, P, S, P, P, I, I, I, P, I, I, I, P]
        L.kda_cache_append.restype = I
        L.kda_attention_decode_workspace_size.argtypes = [I] * 6
        L.kda_attention_decode_workspace_size.restype = Z
        L.kda_attention_decode.argtypes = [P, S, P, P, S, P, P, I, I, I, P, S, I, P, I, I, I, I, F, P, P, P, Z, P]
        L.kda_attention_decode.restype = I
        _lib = L
        return L


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream, device=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _on(device):
    """The calls launch on the CUDA runtime's current device: make it the tensors' device for the call."""
    import torch
    return torch.cuda.device(device)


def _need_all(checks, device=None, *, host=False):
    """The library reads and writes raw pointers, so a tensor of another dtype or size would let its kernels run
    past the buffer.  ``checks``: (name, tensor or None, dtype, element count or None, contiguous); first every
    dtype and size, then placement (``device``, or host memory) and layout."""
    if device is not None and device.type == "cuda":  # one cheap pass when nothing is wrong
        index = device.index
        for _, t, dtype, numel, contiguous in checks:
            if t is not None and (t.dtype is not dtype or t.get_device() != index
                                  or (numel is not None and t.numel() != numel)
                                  or (contiguous and not t.is_contiguous())):
                break
        else:
            return
    checks = [c for c in checks if c[1] is not None]
    for name, t, dtype, numel, _ in checks:
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if numel is not None and t.numel() != numel:
            raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
    for name, t, _, _, contiguous in checks:
        if host:
            if t.is_cuda:
                raise ValueError(f"{name} must be a host tensor")
        else:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if device is not None and t.device != device:
                raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _need(name, t, dtype, numel, device=None, *, host=False, contiguous=True):
    _need_all([(name, t, dtype, numel, contiguous)], device, host=host)


def _need_inputs(q, k, v, g, beta, initial_state, cu_seqlens, state_dtype=None, host=False, more=None):
    """Checks of the forward's inputs, and of ``more(B, T, H, HV, K, V, N)``: further checks in ``_need_all``'s
    form.  Returns (B, T, H, HV, K, V, N, device)."""
    import torch
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B,T,H,K] and v [B,T,HV,V]")
    B, T, H, HV, K, V, N = _dims(q, v, cu_seqlens)
    dev = None if host else q.device
    bt = B * T
    checks = [("q", q, torch.bfloat16, bt * H * K, True), ("k", k, torch.bfloat16, bt * H * K, True),
              ("v", v, torch.bfloat16, bt * HV * V, True), ("g", g, torch.float32, bt * HV * K, True),
              ("beta", beta, torch.float32, bt * HV, True),
              ("initial_state", initial_state, state_dtype or torch.float32, N * HV * K * V, True),
              ("cu_seqlens", cu_seqlens, torch.int32, None, True)]
    if more is not None:
        checks += more(B, T, H, HV, K, V, N)
    _need_all(checks, dev, host=host)
    return B, T, H, HV, K, V, N, dev


def _check(rc: int, where: str):
    if rc != 0:
        raise KdaError(rc, where)


def _dims(q, v, cu_seqlens):
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    return B, T, H, HV, K, V, N


def workspace_size(B, T, H, HV, K=128, V=128, num_seqs=0) -> int:
    return int(lib().kda_prefill_workspace_size(B, T, H, HV, K, V, num_seqs))


def kernel_launches(B, T, H, HV, K=128, V=128, num_seqs=0) -> int:
    """Kernel launches one forward makes for these sizes on the current CUDA device (0 if rejected)."""
    return int(lib().kda_prefill_kernel_launches(B, T, H, HV, K, V, num_seqs))


def _host_cu(cu_seqlens_host):
    """A host copy of cu_seqlens (sequence, numpy array or CPU tensor) as contiguous int32 numpy."""
    import numpy as np
    if hasattr(cu_seqlens_host, "detach"):
        if cu_seqlens_host.device.type != "cpu":
            raise ValueError("cu_seqlens_host must be in host memory")
        cu_seqlens_host = cu_seqlens_host.detach().numpy()
    return np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))


def varlen_kernel_launches(T, H, HV, cu_seqlens_host, K=128, V=128) -> int:
    """Kernel launches forward(..., cu_seqlens_host=...) makes for these lengths (0 if rejected)."""
    cu = _host_cu(cu_seqlens_host)
    return int(lib().kda_prefill_varlen_kernel_launches(T, H, HV, K, V, cu.size - 1,
                                                        cu.ctypes.data_as(ctypes.c_void_p)))


def forward(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, o=None, final_state=None,
            workspace=None, stream=None, cu_seqlens_host=None):
    """Run the forward on CUDA tensors; returns (o, final_state).

    cu_seqlens_host: optional host copy of cu_seqlens (same values).  With it the library knows the sequence
    lengths and can overlap a packed batch's state carry with its intra-chunk work (kda_prefill_forward_varlen).
    """
    import torch
    B, T, H, HV, K, V, N, dev = _need_inputs(q, k, v, g, beta, initial_state, cu_seqlens)
    if cu_seqlens_host is not None and cu_seqlens is None:
        raise ValueError("cu_seqlens_host needs cu_seqlens")
    if o is None:
        o = torch.empty(B, T, HV, V, dtype=torch.bfloat16, device=dev)
    if final_state is None:
        final_state = torch.empty(N, HV, K, V, dtype=torch.float32, device=dev)
    _need("o", o, torch.bfloat16, B * T * HV * V, dev)
    _need("final_state", final_state, torch.float32, N * HV * K * V, dev)
    num_seqs = N if cu_seqlens is not None else 0
    ws_bytes = workspace_size(B, T, H, HV, K, V, num_seqs)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need("workspace", workspace, torch.uint8, None, dev)
    ws_n = workspace.numel() if workspace is not None else 0
    with _on(dev):
        if cu_seqlens_host is not None:
            cu_h = _host_cu(cu_seqlens_host)
            if cu_h.size != N + 1:
                raise ValueError(f"cu_seqlens_host has {cu_h.size} entries, expected {N + 1}")
            rc = lib().kda_prefill_forward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                                  _ptr(initial_state), _ptr(cu_seqlens),
                                                  cu_h.ctypes.data_as(ctypes.c_void_p), num_seqs, T, H, HV, K, V,
                                                  _ptr(o), _ptr(final_state), _ptr(workspace), ws_n,
                                                  _stream_ptr(stream, dev))
            _check(rc, "kda_prefill_forward_varlen")
            return o, final_state
        rc = lib().kda_prefill_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                       _ptr(cu_seqlens), num_seqs, B, T, H, HV, K, V, _ptr(o), _ptr(final_state),
                                       _ptr(workspace), ws_n, _stream_ptr(stream, dev))
    _check(rc, "kda_prefill_forward")
    return o, final_state


def forward_state_bf16(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, o=None, final_state=None,
                       workspace=None, stream=None):
    """The forward with a bf16 state: initial_state bf16 [N,HV,K,V] or None; returns (o, final_state bf16)."""
    import torch
    B, T, H, HV, K, V, N, dev = _need_inputs(q, k, v, g, beta, initial_state, cu_seqlens,
                                             state_dtype=torch.bfloat16)
    if o is None:
        o = torch.empty(B, T, HV, V, dtype=torch.bfloat16, device=dev)
    if final_state is None:
        final_state = torch.empty(N, HV, K, V, dtype=torch.bfloat16, device=dev)
    _need("o", o, torch.bfloat16, B * T * HV * V, dev)
    _need("final_state", final_state, torch.bfloat16, N * HV * K * V, dev)
    num_seqs = N if cu_seqlens is not None else 0
    ws_bytes = int(lib().kda_prefill_state_bf16_workspace_size(B, T, H, HV, K, V, num_seqs))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _need("workspace", workspace, torch.uint8, None, dev)
    with _on(dev):
        rc = lib().kda_prefill_forward_state_bf16(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                                  _ptr(initial_state), _ptr(cu_seqlens), num_seqs, B, T, H, HV, K,
                                                  V, _ptr(o), _ptr(final_state), _ptr(workspace), workspace.numel(),
                                                  _stream_ptr(stream, dev))
    _check(rc, "kda_prefill_forward_state_bf16")
    return o, final_state


def backward_workspace_size(B, T, H, HV, K=128, V=128, num_seqs=0) -> int:
    return int(lib().kda_prefill_backward_workspace_size(B, T, H, HV, K, V, num_seqs))


def backward_kernel_launches(B, T, H, HV, K=128, V=128, num_seqs=0) -> int:
    """Kernel launches one backward makes for these sizes (0 if rejected)."""
    return int(lib().kda_prefill_backward_kernel_launches(B, T, H, HV, K, V, num_seqs))


def forward_save(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, o=None, final_state=None, saved=None,
                 stream=None):
    """The forward that also keeps what the backward needs; returns (o, final_state, saved).  Pass ``saved`` to
    ``backward(..., saved=saved)`` with the same inputs."""
    import torch
    B, T, H, HV, K, V, N, dev = _need_inputs(q, k, v, g, beta, initial_state, cu_seqlens)
    if o is None:
        o = torch.empty(B, T, HV, V, dtype=torch.bfloat16, device=dev)
    if final_state is None:
        final_state = torch.empty(N, HV, K, V, dtype=torch.float32, device=dev)
    _need("o", o, torch.bfloat16, B * T * HV * V, dev)
    _need("final_state", final_state, torch.float32, N * HV * K * V, dev)
    num_seqs = N if cu_seqlens is not None else 0
    if saved is None:
        saved = torch.empty(max(backward_workspace_size(B, T, H, HV, K, V, num_seqs), 1), dtype=torch.uint8,
                            device=dev)
    _need("saved", saved, torch.uint8, None, dev)
    with _on(dev):
        rc = lib().kda_prefill_forward_save(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                            _ptr(cu_seqlens), num_seqs, B, T, H, HV, K, V, _ptr(o),
                                            _ptr(final_state), _ptr(saved), saved.numel(), _stream_ptr(stream, dev))
    _check(rc, "kda_prefill_forward_save")
    return o, final_state, saved


def backward(q, k, v, g, beta, dout, initial_state=None, dht=None, cu_seqlens=None, *, want_dh0=None,
             workspace=None, saved=None, stream=None):
    """Gradients of sum(o * dout) + sum(final_state * dht) for the forward on the same inputs (CUDA).

    Returns (dq, dk [B,T,H,K] bf16, dv [B,T,HV,V] bf16, dg [B,T,HV,K] fp32, dbeta [B,T,HV] fp32,
    dh0 [N,HV,K,V] fp32, or None when there is no initial state and want_dh0 is not set).  With ``saved`` (from
    ``forward_save`` on the same inputs) the forward is not recomputed.
    """
    import torch
    B, T, H, HV, K, V, N, dev = _need_inputs(
        q, k, v, g, beta, initial_state, cu_seqlens,
        more=lambda B, T, H, HV, K, V, N: [("dout", dout, torch.bfloat16, B * T * HV * V, True),
                                           ("dht", dht, torch.float32, N * HV * K * V, True)])
    dq = torch.empty(B, T, H, K, dtype=torch.bfloat16, device=dev)
    dk = torch.empty(B, T, H, K, dtype=torch.bfloat16, device=dev)
    dv = torch.empty(B, T, HV, V, dtype=torch.bfloat16, device=dev)
    dg = torch.empty(B, T, HV, K, dtype=torch.float32, device=dev)
    dbeta = torch.empty(B, T, HV, dtype=torch.float32, device=dev)
    if want_dh0 is None:
        want_dh0 = initial_state is not None
    dh0 = torch.empty(N, HV, K, V, dtype=torch.float32, device=dev) if want_dh0 else None
    num_seqs = N if cu_seqlens is not None else 0
    fn, name = lib().kda_prefill_backward, "kda_prefill_backward"
    if saved is not None:
        workspace, fn, name = saved, lib().kda_prefill_backward_saved, "kda_prefill_backward_saved"
    elif workspace is None:
        ws_bytes = backward_workspace_size(B, T, H, HV, K, V, num_seqs)
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _need("saved" if saved is not None else "workspace", workspace, torch.uint8, None, dev)
    with _on(dev):
        rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), num_seqs,
                B, T, H, HV, K, V, _ptr(dout), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta),
                _ptr(dh0), _ptr(workspace), workspace.numel(), _stream_ptr(stream, dev))
    _check(rc, name)
    return dq, dk, dv, dg, dbeta, dh0


def host_staging_size(B, T, H, HV, K=128, V=128, num_seqs=0, has_initial_state=False, has_cu_seqlens=False) -> int:
    return int(lib().kda_prefill_host_staging_size(B, T, H, HV, K, V, num_seqs, int(has_initial_state),
                                                    int(has_cu_seqlens)))


def forward_host(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, o, final_state, staging, stream=None):
    """Forward on HOST (ideally pinned) tensors through a device staging buffer.

    Enqueues the host->device copies, the forward and the device->host copies
    of o and final_state on ``stream``; the caller synchronises.
    """
    import torch
    B, T, H, HV, K, V, N, _ = _need_inputs(
        q, k, v, g, beta, initial_state, cu_seqlens, host=True,
        more=lambda B, T, H, HV, K, V, N: [("o", o, torch.bfloat16, B * T * HV * V, True),
                                           ("final_state", final_state, torch.float32, N * HV * K * V, True)])
    _need("staging", staging, torch.uint8, None)
    dev = staging.device
    num_seqs = N if cu_seqlens is not None else 0
    with _on(dev):
        rc = lib().kda_prefill_forward_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                            _ptr(cu_seqlens), num_seqs, B, T, H, HV, K, V, _ptr(o),
                                            _ptr(final_state), _ptr(staging), staging.numel(),
                                            _stream_ptr(stream, dev))
    _check(rc, "kda_prefill_forward_host")
    return o, final_state


def device_error(clear: bool = True) -> int:
    """Bits set on the current device (0 when none) by kernel waits that gave up (1, 2, 4, 8) and by the paged cache's
    calls: 16, a block, slot or length out of range; 32, blocks, table entries or slots that do not suffice.
    Synchronises."""
    w = ctypes.c_uint(0)
    _check(lib().kda_prefill_device_error(ctypes.byref(w), int(clear)), "kda_prefill_device_error")
    return int(w.value)


def decode_step(q, k, v, g, beta, state, state_indices, *, o=None, stream=None):
    """One recurrent decode step on a bf16 state pool (CUDA); returns o [B, HV, V].

    q, k: bf16 [B, H, K] and v: bf16 [B, HV, V], each row compact but rows may be strided (e.g. views of a
    packed [B, (2H + HV) * 128] QKV tensor); g: fp32 [B, HV, K]; beta: fp32 [B, HV]; state: bf16 pool
    [num_slots, HV, K, V] (compact inside a slot), updated in place; state_indices: int32 [B], -1 = padding row.
    """
    import torch
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[0] != q.shape[0]:
        raise ValueError("q and k must be [B,H,K] and v [B,HV,V]")
    if state.dim() != 4 or state.shape[1] != v.shape[1]:
        raise ValueError("state must be a pool [num_slots, HV, K, V]")
    B, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    dev = q.device
    _need_all([("q", q, torch.bfloat16, None, False), ("k", k, torch.bfloat16, None, False),
               ("v", v, torch.bfloat16, None, False), ("g", g, torch.float32, B * HV * K, True),
               ("beta", beta, torch.float32, B * HV, True), ("state", state, torch.bfloat16, None, False),
               ("state_indices", state_indices, torch.int32, B, True)], dev)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{name} must have compact rows")
    if tuple(state.shape[1:]) != (HV, K, V) or state[0].stride() != (K * V, V, 1):
        raise ValueError("state must be a pool [num_slots, HV, K, V] compact inside each slot")
    if o is None:
        o = torch.empty(B, HV, V, dtype=torch.bfloat16, device=dev)
    _need("o", o, torch.bfloat16, B * HV * V, dev)
    with _on(dev):
        rc = lib().kda_decode_step(_ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(v), v.stride(0), _ptr(g),
                                   _ptr(beta), _ptr(state), state.stride(0), state.shape[0], _ptr(state_indices),
                                   B, H, HV, K, V, _ptr(o), _stream_ptr(stream, dev))
    _check(rc, "kda_decode_step")
    return o


def l2norm_bf16(x, out=None, stream=None):
    """Exact-rounding L2 normalisation of rows of 128 bf16 values (CUDA)."""
    import torch
    _need("x", x, torch.bfloat16, None, x.device)
    if out is None:
        out = torch.empty_like(x)
    _need("out", out, torch.bfloat16, x.numel(), x.device)
    rows = x.numel() // x.shape[-1]
    with _on(x.device):
        rc = lib().kda_l2norm_bf16(_ptr(x), rows, x.shape[-1], _ptr(out), _stream_ptr(stream, x.device))
    _check(rc, "kda_l2norm_bf16")
    return out


def forward_noalloc(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, o=None, final_state=None,
                    stream=None):
    """The forward through kda_prefill_forward_noalloc: no workspace argument.

    For callers that may not allocate device memory during the call; the
    library's fixed 64 MiB scratch array limits the problem size (larger
    inputs raise KdaError with KDA_ERR_WORKSPACE).  Calls must not overlap.
    """
    import torch
    L = lib()
    f = L.kda_prefill_forward_noalloc
    P, I = ctypes.c_void_p, ctypes.c_int
    f.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P]
    f.restype = I
    B, T, H, HV, K, V, N, dev = _need_inputs(q, k, v, g, beta, initial_state, cu_seqlens)
    if o is None:
        o = torch.empty(B, T, HV, V, dtype=torch.bfloat16, device=dev)
    if final_state is None:
        final_state = torch.empty(N, HV, K, V, dtype=torch.float32, device=dev)
    _need("o", o, torch.bfloat16, B * T * HV * V, dev)
    _need("final_state", final_state, torch.float32, N * HV * K * V, dev)
    num_seqs = N if cu_seqlens is not None else 0
    with _on(dev):
        rc = f(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), num_seqs,
               B, T, H, HV, K, V, _ptr(o), _ptr(final_state), _stream_ptr(stream, dev))
    _check(rc, "kda_prefill_forward_noalloc")
    return o, final_state


# ---------------------------------------------------------------------------------------------- softmax attention
# These calls take a few microseconds on the GPU for short requests, so their host side is kept as short: pointers
# as plain integers, the device switched only where it is not the current one.
def _call(name, dev, *args):
    """Call a C entry whose last argument is the stream, on the tensors' device and its current stream."""
    import torch
    if torch.cuda.current_device() != dev.index:
        with _on(dev):
            return _call(name, dev, *args)
    rc = getattr(_lib or lib(), name)(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != 0:
        raise KdaError(rc, name)


def _under(stream, device):
    """Makes ``stream`` the current one for a call, so that the workspace and the results it allocates are that stream's:
    memory of another stream may still be in use there, or be given away again before this one is done with it."""
    import torch
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _scale(scale, D):
    return (max(D, 1) ** -0.5) if scale is None else scale


def _row_stride(name, shape, strides):
    """Elements between the rows of a [B,T,heads,D] (or [T,heads,D]) tensor, which are compact and evenly spaced."""
    D, heads = shape[-1], shape[-2]
    if (strides[-1] != 1 and D > 1) or (strides[-2] != D and heads > 1):
        raise ValueError(f"{name} must have compact rows")
    T = shape[-3]
    B = shape[0] if len(shape) == 4 else 1
    if T > 1:
        st = strides[-3]
        if B > 1 and strides[0] != T * st:
            raise ValueError(f"{name} must have evenly spaced rows")
        return st
    return strides[0] if B > 1 else heads * D


def _attention_inputs(q, k, v, cu_seqlens, cu_seqlens_k, more=()):
    """Checks of attention over whole prompts; returns the C calls' leading arguments (pointers and row strides of q, k
    and v), (cu_seqlens, cu_seqlens_k, num_seqs, B, T, Tk, H, HKV, D), and the device."""
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B,T,H,D], k and v [B,Tk,HKV,D]")
    qs, ks = q.shape, k.shape
    B, T, H, D = qs
    Bk, Tk, HKV, Dk = ks
    if Bk != B or Dk != D or v.shape != ks:
        raise ValueError("q must be [B,T,H,D], k and v [B,Tk,HKV,D]")
    num_seqs = 0
    if cu_seqlens is None:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
    else:
        num_seqs = cu_seqlens.numel() - 1
        if num_seqs < 1:
            raise ValueError("cu_seqlens must hold at least 2 elements")
        if cu_seqlens_k is None:
            if T != Tk:
                raise ValueError("keys of another length than the queries need cu_seqlens_k")
            cu_seqlens_k = cu_seqlens
    bf16 = torch.bfloat16
    dev = q.device
    _need_all([("q", q, bf16, None, False), ("k", k, bf16, None, False), ("v", v, bf16, None, False),
               ("cu_seqlens", cu_seqlens, torch.int32, None, True),
               ("cu_seqlens_k", cu_seqlens_k, torch.int32, num_seqs + 1, True), *more], dev)
    cu, cu_k = (None, None) if cu_seqlens is None else (cu_seqlens.data_ptr(), cu_seqlens_k.data_ptr())
    return ((q.data_ptr(), _row_stride("q", qs, q.stride()), k.data_ptr(), _row_stride("k", ks, k.stride()),
             v.data_ptr(), _row_stride("v", ks, v.stride())), (cu, cu_k, num_seqs, B, T, Tk, H, HKV, D), dev)


def attention_forward(q, k, v, cu_seqlens=None, cu_seqlens_k=None, *, scale=None, o=None, lse=None, stream=None):
    """Causal softmax attention over whole prompts (CUDA); returns (o [B,T,H,D] bf16, lse [B,H,T] fp32).

    q: bf16 [B,T,H,D]; k, v: bf16 [B,Tk,HKV,D], H a multiple of HKV, D 64 or 128.  Rows are compact but may be
    strided (views of a packed QKV tensor).  Query i of a sequence with Lq queries and Lk keys sees the keys
    j <= i + Lk - Lq; a row that sees none gets o = 0 and lse = -inf.  Packed sequences: B = 1 and cu_seqlens int32
    [N+1], with cu_seqlens_k where the keys' offsets differ; rows of no sequence are left as they were, and nothing of
    them reaches a result (infinities and NaN inside a sequence may reach all of its rows).
    scale: D^-0.5 when not given.  lse is the natural logarithm of the row's sum of exponentials.
    """
    import torch
    if stream is not None:
        with _under(stream, q.device):
            return attention_forward(q, k, v, cu_seqlens, cu_seqlens_k, scale=scale, o=o, lse=lse)
    rows, dims, dev = _attention_inputs(q, k, v, cu_seqlens, cu_seqlens_k)
    B, T, H, D = q.shape
    if o is None:
        o = torch.empty(B, T, H, D, dtype=torch.bfloat16, device=dev)
    else:
        _need("o", o, torch.bfloat16, B * T * H * D, dev)
    if lse is None:
        lse = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    else:
        _need("lse", lse, torch.float32, B * H * T, dev)
    _call("kda_attention_forward", dev, *rows, *dims, _scale(scale, D), o.data_ptr(),
          lse.data_ptr())
    return o, lse


def attention_backward_workspace_size(B, T, H, num_seqs=0) -> int:
    return int(lib().kda_attention_backward_workspace_size(B, T, H, num_seqs))


def attention_backward(q, k, v, o, lse, dout, cu_seqlens=None, cu_seqlens_k=None, *, scale=None, workspace=None,
                       stream=None):
    """Gradients of sum(o * dout) for ``attention_forward`` on the same inputs, from the o and lse it returned (CUDA).
    (Not from those of attention over further keys: a row's probabilities must sum to one over the keys given here.)

    Returns (dq [B,T,H,D], dk, dv [B,Tk,HKV,D]) in bf16; dk and dv are summed over the query heads that share a
    key/value head.  dout's rows may be strided like q's.  Rows of no sequence are not written.
    """
    import torch
    if stream is not None:
        with _under(stream, q.device):
            return attention_backward(q, k, v, o, lse, dout, cu_seqlens, cu_seqlens_k, scale=scale, workspace=workspace)
    if q.dim() != 4 or dout.shape != q.shape:
        raise ValueError("q must be [B,T,H,D], dout like it, k and v [B,Tk,HKV,D]")
    B, T, H, D = q.shape
    rows, dims, dev = _attention_inputs(
        q, k, v, cu_seqlens, cu_seqlens_k,
        (("o", o, torch.bfloat16, B * T * H * D, True), ("lse", lse, torch.float32, B * H * T, True),
         ("dout", dout, torch.bfloat16, None, False), ("workspace", workspace, torch.uint8, None, True)))
    dq = torch.empty(B, T, H, D, dtype=torch.bfloat16, device=dev)
    dk = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    dv = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(attention_backward_workspace_size(B, T, H, dims[2]), dtype=torch.uint8, device=dev)
    _call("kda_attention_backward", dev, *rows, o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
          _row_stride("dout", dout.shape, dout.stride()), *dims, _scale(scale, D), dq.data_ptr(),
          dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.numel())
    return dq, dk, dv


def _table_stride(block_table, B, width):
    sb, sw = block_table.stride()
    if sw != 1 and width > 1:
        raise ValueError("block_table must have compact rows")
    return sb if B > 1 else width


def cache_plan(context_lens, new_lens, block_table, free_blocks, block_size, num_tokens, *, stream=None):
    """Block tables and slot maps of a paged cache from request lengths, on the GPU (CUDA).

    context_lens, new_lens: int32 [B], tokens that each request holds and gets; block_table: int32 [B, width], updated
    in place; free_blocks: int32 [F], taken from the front; num_tokens: the slot map's length, at least the sum of
    new_lens.  Returns (cu_seqlens [B+1], seq_lens [B], slot_map [num_tokens], used [1]), all int32: the new tokens'
    offsets, the lengths with them, each new token's slot (-1 behind the last), the number of blocks taken.  What does
    not fit gets -1 and sets bit 5 of ``device_error``; such a row is planned anew from its length before.
    """
    import torch
    if stream is not None:
        with _under(stream, context_lens.device):
            return cache_plan(context_lens, new_lens, block_table, free_blocks, block_size, num_tokens)
    B = context_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, width]")
    if num_tokens < 0:
        raise ValueError("num_tokens must not be negative")
    if num_tokens >= 1 << 31:
        raise ValueError("num_tokens must be below 2^31")
    width = block_table.shape[1]
    dev = context_lens.device
    i32 = torch.int32
    _need_all((("context_lens", context_lens, i32, B, True), ("new_lens", new_lens, i32, B, True),
               ("block_table", block_table, i32, None, False), ("free_blocks", free_blocks, i32, None, True)), dev)
    table_stride = _table_stride(block_table, B, width)
    buf = torch.empty(2 * B + 2 + num_tokens, dtype=i32, device=dev)
    slots, cu, lens, used = torch.unsafe_split_with_sizes(buf, (num_tokens, B + 1, B, 1))
    at = buf.data_ptr()
    small = at + 4 * num_tokens
    _call("kda_cache_plan", dev, context_lens.data_ptr(), new_lens.data_ptr(), B, block_table.data_ptr(),
          table_stride, width, free_blocks.data_ptr(), free_blocks.numel(), block_size, small,
          small + 4 * (B + 1), at, num_tokens, small + 4 * (2 * B + 1))
    return cu, lens, slots, used


def _cache_inputs(k_cache, v_cache, k_scale, v_scale, device, more):
    """Checks of a cache's tensors; returns (code type, num_blocks, HKV, block_size, D, block stride)."""
    import torch
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [num_blocks, HKV, block_size, D]")
    dtype = k_cache.dtype
    if dtype is torch.float8_e4m3fn:
        code = 0
    elif dtype is torch.int8:
        code = 1
    else:
        raise ValueError(f"k_cache must be torch.float8_e4m3fn or torch.int8, got {dtype}")
    blocks, HKV, bs, D = shape
    _need_all((("k_cache", k_cache, dtype, None, False), ("v_cache", v_cache, dtype, None, False),
               ("k_scale", k_scale, torch.float32, blocks * HKV, True),
               ("v_scale", v_scale, torch.float32, blocks * HKV, True), *more), device)
    strides = k_cache.stride()
    inside = (bs * D, D, 1)
    if strides != v_cache.stride() or strides[1:] != inside:  # (the stride of an axis of length 1 says nothing)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if any(t.shape[i + 1] > 1 and t.stride(i + 1) != inside[i] for i in range(3)) or \
                    (blocks > 1 and t.stride(0) != strides[0]):
                raise ValueError(f"{name} must be compact inside each block, with k_cache's block stride")
    return code, blocks, HKV, bs, D, strides[0] if blocks > 1 else HKV * bs * D


def cache_append(k, v, k_cache, v_cache, k_scale, v_scale, slot_map, *, stream=None):
    """Store the rows of k and v (bf16 [T,HKV,D]) in a paged 8-bit cache, in place (CUDA).

    k_cache, v_cache: torch.float8_e4m3fn or torch.int8 [num_blocks,HKV,block_size,D], compact inside a block;
    k_scale, v_scale: fp32 [num_blocks,HKV]; slot_map: int32 [T], -1 = skipped (see ``cache_plan``); slots are unique,
    and the tokens of one block stand beside one another, in ascending order, none skipped between them.  The scale of a (block, head) is the
    smallest power of two that its tokens fit; it grows, and the block's earlier tokens are rounded again, when later ones
    need it.
    """
    import torch
    if stream is not None:
        with _under(stream, k.device):
            return cache_append(k, v, k_cache, v_cache, k_scale, v_scale, slot_map)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("k and v must be [T,HKV,D]")
    T, HKV, D = shape
    dev = k.device
    code, blocks, hkv, bs, d, stride = _cache_inputs(
        k_cache, v_cache, k_scale, v_scale, dev,
        (("k", k, torch.bfloat16, None, False), ("v", v, torch.bfloat16, None, False),
         ("slot_map", slot_map, torch.int32, T, True)))
    if hkv != HKV or d != D:
        raise ValueError("k and v must have the cache's heads")
    _call("kda_cache_append", dev, k.data_ptr(), _row_stride("k", shape, k.stride()), v.data_ptr(),
          _row_stride("v", shape, v.stride()), k_cache.data_ptr(), v_cache.data_ptr(), stride, k_scale.data_ptr(),
          v_scale.data_ptr(), code, blocks, bs, slot_map.data_ptr(), T, HKV, D)


@functools.lru_cache(maxsize=256)
def attention_decode_workspace_size(B, H, HKV, D, table_width, block_size) -> int:
    return int(lib().kda_attention_decode_workspace_size(B, H, HKV, D, table_width, block_size))


def attention_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, *, scale=None, o=None, lse=None,
                     workspace=None, stream=None):
    """One-token attention over a paged 8-bit cache (CUDA); returns (o [B,H,D] bf16, lse [B,H] fp32).

    q: bf16 [B,H,D], H a multiple of the cache's HKV, rows compact but they may be strided; the cache as in
    ``cache_append``; block_table: int32 [B,width]; seq_lens: int32 [B], the tokens that row b sees (0: o = 0 and
    lse = -inf).  scale: D^-0.5 when not given.  Blocks out of range do not count and set bit 4 of ``device_error``.
    """
    import torch
    if stream is not None:
        with _under(stream, q.device):
            return attention_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale=scale, o=o, lse=lse,
                                    workspace=workspace)
    qs, ts = q.shape, block_table.shape
    if len(qs) != 3 or len(ts) != 2 or ts[0] != qs[0]:
        raise ValueError("q must be [B,H,D] and block_table [B,width]")
    B, H, D = qs
    width = ts[1]
    dev = q.device
    code, blocks, HKV, bs, d, stride = _cache_inputs(
        k_cache, v_cache, k_scale, v_scale, dev,
        (("q", q, torch.bfloat16, None, False), ("block_table", block_table, torch.int32, None, False),
         ("seq_lens", seq_lens, torch.int32, B, True)))
    if d != D:
        raise ValueError("q must have the cache's head dimension")
    table_stride = _table_stride(block_table, B, width)
    if o is None:
        o = torch.empty(B, H, D, dtype=torch.bfloat16, device=dev)
    else:
        _need("o", o, torch.bfloat16, B * H * D, dev)
    if lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=dev)
    else:
        _need("lse", lse, torch.float32, B * H, dev)
    if workspace is None:
        workspace = torch.empty(attention_decode_workspace_size(B, H, HKV, D, width, bs), dtype=torch.uint8,
                                device=dev)
    else:
        _need("workspace", workspace, torch.uint8, None, dev)
    _call("kda_attention_decode", dev, q.data_ptr(), _row_stride("q", qs, q.stride()), k_cache.data_ptr(),
          v_cache.data_ptr(), stride, k_scale.data_ptr(), v_scale.data_ptr(), code, blocks, bs, block_table.data_ptr(),
          table_stride, width, seq_lens.data_ptr(), B, H, HKV, D, _scale(scale, D), o.data_ptr(),
          lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return o, lse
