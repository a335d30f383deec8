"""Python binding of libmoe.so, the GB300 gated Mixture-of-Experts FFN layer (forward).

Argument marshalling only: each function takes torch tensors (device memory owned by the
caller), passes their pointers and the current CUDA stream through the C ABI of
``include/moe.h`` and raises ``MoeError`` on a non-OK status.  Every step of the layer runs in
the library's CUDA kernels; there is no fallback.  The first call fails loudly when
the library has not been built (``python sparse_expert_ffn_layer_gb300/_build.py``).
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE_BOUNDS = 4, 5, 6
MOE_F32, MOE_F16 = 0, 1
MOE_MLP_STANDARD, MOE_MLP_RESIDUAL = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1

EXPORTED = ("moe_capacity", "moe_workspace_size", "moe_gate_topk", "moe_dispatch",
            "moe_expert_ffn", "moe_combine", "moe_layer_forward", "moe_status_read",
            "moe_status_string", "moe_selftest_wait", "moe_set_stage_events",
            "moe_expert_ffn_noalloc", "moe_dispatch_sharded", "moe_kernel_launches",
            "moe_balance_workspace_size", "moe_balance_loss", "moe_gate_backward_workspace_size",
            "moe_gate_topk_backward", "moe_combine_backward", "moe_adapter_workspace_size",
            "moe_adapter_forward", "moe_adapter_backward", "moe_route", "moe_route_backward",
            "moe_fp8_quantize", "moe_expert_fp8_workspace_size", "moe_expert_ffn_fp8", "moe_block_norm",
            "moe_block_norm_workspace_size", "moe_block_norm_backward")

_lib = None
MOE_STAGE_EVENTS = 7
STAGES = ("gate_logits", "softmax_topk", "dispatch", "expert_gemm1_gelu", "expert_gemm2_combine",
          "finalize")


def get_lib():
    """Load libmoe.so (once) and declare its signatures; raises if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python sparse_expert_ffn_layer_gb300/_build.py`"
                          " (or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sig = {
        "moe_capacity": ([I, I, F], I),
        "moe_workspace_size": ([I, I, I, I, I, F, I, I, I, ctypes.POINTER(S)], I),
        "moe_gate_topk": ([P, I, P, P, I, I, I, I, P, P, P, P, P], I),
        "moe_dispatch": ([P, I, I, I, F, P, P, P, P, P, P], I),
        "moe_expert_ffn": ([P, P, P, P, P, I, I, I, I, I, I, P, P, S, P], I),
        "moe_combine": ([P, P, P, P, I, I, I, I, P, P], I),
        "moe_layer_forward": ([P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, P, P, P, P, S, P], I),
        "moe_status_read": ([P, P], I),
        "moe_status_string": ([I], ctypes.c_char_p),
        "moe_selftest_wait": ([P, ctypes.c_uint64, P], I),
        "moe_set_stage_events": ([P, I], I),
        "moe_expert_ffn_noalloc": ([P, P, P, P, P, I, I, I, I, I, I, P, P], I),
        "moe_dispatch_sharded": ([P, I, I, I, F, I, P, I, I, P, P, P, P, P, P], I),
        "moe_kernel_launches": ([], ctypes.c_ulonglong),
        "moe_balance_workspace_size": ([I, I, ctypes.POINTER(S)], I),
        "moe_balance_loss": ([P, P, P, I, I, I, P, P, P, P, P, S, P], I),
        "moe_gate_backward_workspace_size": ([I, I, I, I, ctypes.POINTER(S)], I),
        "moe_gate_topk_backward": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, S, P], I),
        "moe_combine_backward": ([P, P, P, P, I, I, I, I, I, P, P, P], I),
        "moe_adapter_workspace_size": ([I, I, I, I, I, I, I, ctypes.POINTER(S)], I),
        "moe_adapter_forward": ([P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, S, P], I),
        "moe_adapter_backward": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, P, S, P], I),
        "moe_route": ([P, I, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, P, P, P, P], I),
        "moe_route_backward": ([P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P, P, S, P], I),
        "moe_fp8_quantize": ([P, I, I, I, I, P, P, P], I),
        "moe_expert_fp8_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(S)], I),
        "moe_expert_ffn_fp8": ([P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, S, P], I),
        "moe_block_norm": ([P, P, P, P, P, P, P, F, P, F, I, I, I, I, I, P, P, P, P, P], I),
        "moe_block_norm_workspace_size": ([I, I, I, I, ctypes.POINTER(S)], I),
        "moe_block_norm_backward": ([P] * 12 + [F] + [I] * 5 + [P] * 8 + [S, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def __getattr__(name):
    if name == "lib":
        return get_lib()
    raise AttributeError(name)


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {get_lib().moe_status_string(code).decode()}")


def _check(code: int, where: str) -> None:
    if code != MOE_OK:
        raise MoeError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return MOE_F16
    if t.dtype == torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def moe_kernel_launches() -> int:
    return get_lib().moe_kernel_launches()


def moe_capacity(T: int, E: int, capacity_factor: float) -> int:
    return get_lib().moe_capacity(T, E, capacity_factor)


def moe_workspace_size(T, d, f, E, k, capacity_factor, mlp_type, f_res, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(get_lib().moe_workspace_size(T, d, f, E, k, capacity_factor, mlp_type, f_res, dtype,
                                  ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_gate_topk(tokens, Wg, k, topk_idx, topk_w, logits_out=None, probs_out=None,
                  logits_in=None, stream=None):
    if logits_in is not None:
        T, E = logits_in.shape
        d = tokens.shape[1] if tokens is not None else 1
        dt = _dtype(tokens) if tokens is not None else MOE_F32
    else:
        T, d = tokens.shape
        E = Wg.shape[1]
        dt = _dtype(tokens)
    _check(get_lib().moe_gate_topk(_ptr(tokens), dt, _ptr(Wg), _ptr(logits_in), T, d, E, k,
                             _ptr(logits_out), _ptr(probs_out), _ptr(topk_idx), _ptr(topk_w),
                             _stream(stream)), "moe_gate_topk")


def moe_dispatch(topk_idx, E, capacity_factor, counts_raw, kept, offsets, perm, slot_of,
                 stream=None):
    T, k = topk_idx.shape
    _check(get_lib().moe_dispatch(_ptr(topk_idx), T, E, k, capacity_factor, _ptr(counts_raw), _ptr(kept),
                            _ptr(offsets), _ptr(perm), _ptr(slot_of), _stream(stream)),
           "moe_dispatch")


def moe_dispatch_sharded(topk_idx, E, capacity_factor, T_global, counts_all, rank, counts_raw, kept,
                         offsets, perm, slot_of, stream=None):
    T, k = topk_idx.shape
    n_ranks = counts_all.shape[0] if counts_all is not None else 1
    _check(get_lib().moe_dispatch_sharded(_ptr(topk_idx), T, E, k, capacity_factor, T_global,
                                          _ptr(counts_all), n_ranks, rank, _ptr(counts_raw),
                                          _ptr(kept), _ptr(offsets), _ptr(perm), _ptr(slot_of),
                                          _stream(stream)), "moe_dispatch_sharded")


def moe_expert_ffn(tokens, perm, offsets, W1, W2, S_max, expert_out, workspace, stream=None):
    T, d = tokens.shape
    E, _, f = W1.shape
    _check(get_lib().moe_expert_ffn(_ptr(tokens), _ptr(perm), _ptr(offsets), _ptr(W1), _ptr(W2),
                              _dtype(tokens), T, d, f, E, S_max, _ptr(expert_out), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_expert_ffn")


def moe_combine(expert_out, slot_of, topk_w, out, residual_in=None, stream=None):
    T, k = slot_of.shape
    d = out.shape[1]
    _check(get_lib().moe_combine(_ptr(expert_out), _ptr(slot_of), _ptr(topk_w), _ptr(residual_in),
                           _dtype(out), T, d, k, _ptr(out), _stream(stream)), "moe_combine")


def moe_layer_forward(tokens, Wg, W1, W2, k, capacity_factor, out, workspace, mlp_type=0,
                      Wr1=None, Wr2=None, topk_idx_out=None, slot_of_out=None, stream=None):
    T, d = tokens.shape
    E, _, f = W1.shape
    f_res = Wr1.shape[1] if Wr1 is not None else 0
    _check(get_lib().moe_layer_forward(_ptr(tokens), _ptr(Wg), _ptr(W1), _ptr(W2), _ptr(Wr1), _ptr(Wr2),
                                 _dtype(tokens), T, d, f, E, k, capacity_factor, mlp_type, f_res,
                                 _ptr(out), _ptr(topk_idx_out), _ptr(slot_of_out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_layer_forward")


def moe_status_read(workspace, stream=None) -> int:
    return get_lib().moe_status_read(_ptr(workspace), _stream(stream))


def moe_status_string(code: int) -> str:
    return get_lib().moe_status_string(code).decode()


def moe_selftest_wait(workspace, timeout_ns: int, stream=None):
    _check(get_lib().moe_selftest_wait(_ptr(workspace), timeout_ns, _stream(stream)), "moe_selftest_wait")


def moe_set_stage_events(events=None):
    """Record the given 7 torch.cuda.Event objects at the stage boundaries of this thread's next
    moe_layer_forward calls (None stops recording)."""
    if events is None:
        _check(get_lib().moe_set_stage_events(None, 0), "moe_set_stage_events")
        return
    handles = [e.cuda_event for e in events]
    if len(handles) != MOE_STAGE_EVENTS or not all(handles):
        raise ValueError("moe_set_stage_events needs 7 created events (record each once first)")
    arr = (ctypes.c_void_p * MOE_STAGE_EVENTS)(*[ctypes.c_void_p(h) for h in handles])
    _check(get_lib().moe_set_stage_events(arr, MOE_STAGE_EVENTS), "moe_set_stage_events")


def moe_expert_ffn_noalloc(tokens, perm, offsets, W1, W2, S_max, expert_out, stream=None):
    """moe_expert_ffn with the library's fixed scratch instead of a workspace (no allocation)."""
    T, d = tokens.shape
    E, _, f = W1.shape
    _check(get_lib().moe_expert_ffn_noalloc(_ptr(tokens), _ptr(perm), _ptr(offsets), _ptr(W1),
                                            _ptr(W2), _dtype(tokens), T, d, f, E, S_max,
                                            _ptr(expert_out), _stream(stream)),
           "moe_expert_ffn_noalloc")


# ---------------------------------------------------------------- training and adapters
# These calls take a few microseconds on the GPU at decode sizes, so their checks are kept to
# a few attribute reads per tensor: _device_of walks (tensor, dtype, shape) triples and only
# a call that fails builds a message.
def _device_of(where, names, given):
    """CUDA device index that every given tensor is on (None entries are skipped).

    The kernels read dense row-major memory of the stated type and shape; anything else is
    refused here rather than read wrongly."""
    dev = given[0][0].get_device()
    for t, dtype, shape in given:
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
                              or not t.is_contiguous()):
            _refuse(where, names, given, dev)
    if dev < 0:
        _refuse(where, names, given, dev)
    return dev


def _refuse(where, names, given, dev):
    for name, (t, dtype, shape) in zip(names.split(), given):
        if t is None:
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{where}: {name} is {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
        if t.get_device() != dev:
            raise ValueError(f"{where}: {name} is on {t.device}, expected the device of "
                             f"{names.split()[0]}, {given[0][0].device}")
    raise ValueError(f"{where}: tensors must be on a CUDA device")


def _mask_type(where, token_mask):
    """torch.bool or torch.uint8, whichever the mask is (a byte per token either way)."""
    import torch
    if token_mask is None:
        return None
    if token_mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"{where}: token_mask is {token_mask.dtype}, expected torch.bool or torch.uint8")
    return token_mask.dtype


def _required(where, **tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{where}: {name} is required")


def _adr(t):
    return None if t is None else t.data_ptr()


def _ws_bytes(workspace):
    return 0 if workspace is None else workspace.numel()


def _code(dtype) -> int:
    """MOE_F32 / MOE_F16 of a torch dtype (or of a code itself)."""
    if isinstance(dtype, int):
        return dtype
    import torch
    if dtype not in (torch.float16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}")
    return MOE_F16 if dtype == torch.float16 else MOE_F32


_fns = {}


def _call(where, dev, stream, *args):
    """The library call on device `dev`: its current stream unless one is given."""
    import torch
    fn = _fns.get(where)
    if fn is None:
        fn = _fns[where] = getattr(get_lib(), where)
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, handle)
    if code != MOE_OK:
        raise MoeError(code, where)


def _raw_stream(dev):
    """Handle of the device's current stream, without the stream object around it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev)


def moe_balance_workspace_size(T, E) -> int:
    n = ctypes.c_size_t(0)
    _check(get_lib().moe_balance_workspace_size(T, E, ctypes.byref(n)), "moe_balance_workspace_size")
    return n.value


def moe_balance_loss(logits, topk_idx, counts, prob_mean, losses, n_valid, workspace,
                     token_mask=None, stream=None):
    """Per-expert counts, mean probabilities and the balance and z losses of a routed batch."""
    import torch
    where = "moe_balance_loss"
    T, E = logits.shape
    k = topk_idx.shape[1]
    f32, i32 = torch.float32, torch.int32
    dev = _device_of(where, "logits topk_idx counts prob_mean losses n_valid workspace token_mask",
                     ((logits, f32, (T, E)), (topk_idx, i32, (T, k)), (counts, i32, (E,)),
                      (prob_mean, f32, (E,)), (losses, f32, (2,)), (n_valid, i32, (1,)),
                      (workspace, torch.uint8, workspace.shape),
                      (token_mask, _mask_type(where, token_mask), (T,))))
    _call(where, dev, stream, logits.data_ptr(), topk_idx.data_ptr(), _adr(token_mask), T, E, k,
          counts.data_ptr(), prob_mean.data_ptr(), losses.data_ptr(), n_valid.data_ptr(),
          workspace.data_ptr(), workspace.numel())


def moe_gate_backward_workspace_size(T, d, E, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(get_lib().moe_gate_backward_workspace_size(T, d, E, _code(dtype), ctypes.byref(n)),
           "moe_gate_backward_workspace_size")
    return n.value


def moe_gate_topk_backward(logits, topk_idx, dlogits, dtopk_w=None, dlosses=None, counts=None,
                           n_valid=None, token_mask=None, tokens=None, Wg=None, dWg=None,
                           dtokens=None, dtokens_in=None, workspace=None, stream=None):
    """Gradient of the gate weights and of the router losses: dlogits, and from it dWg and dtokens."""
    import torch
    where = "moe_gate_topk_backward"
    T, E = logits.shape
    k = topk_idx.shape[1]
    f32, i32 = torch.float32, torch.int32
    given = [(logits, f32, (T, E)), (topk_idx, i32, (T, k)), (dlogits, f32, (T, E)),
             (dtopk_w, f32, (T, k))]
    names = "logits topk_idx dlogits dtopk_w"
    if dlosses is not None:
        if counts is None or n_valid is None:
            _required(where, counts=counts, n_valid=n_valid)
        given += [(dlosses, f32, (2,)), (counts, i32, (E,)), (n_valid, i32, (1,))]
        names += " dlosses counts n_valid"
    if token_mask is not None:
        given.append((token_mask, _mask_type(where, token_mask), (T,)))
        names += " token_mask"
    code, d = MOE_F32, 4
    if dWg is not None or dtokens is not None:
        if dWg is not None:
            _required(where, tokens=tokens)
        if dtokens is not None:
            _required(where, Wg=Wg)
        like = tokens if dWg is not None else dtokens
        d, el, code = like.shape[1], like.dtype, _dtype(like)
        given += [(tokens if dWg is not None else None, el, (T, d)),
                  (Wg if dtokens is not None else None, f32, (d, E)), (dWg, f32, (d, E)),
                  (dtokens, el, (T, d)), (dtokens_in, el, (T, d)),
                  (workspace, torch.uint8, None if workspace is None else workspace.shape)]
        names += " tokens Wg dWg dtokens dtokens_in workspace"
    dev = _device_of(where, names, given)
    _call(where, dev, stream, logits.data_ptr(), topk_idx.data_ptr(), _adr(dtopk_w), _adr(dlosses),
          _adr(counts), _adr(n_valid), _adr(token_mask), _adr(tokens), _adr(Wg), code, T, d, E, k,
          dlogits.data_ptr(), _adr(dWg), _adr(dtokens_in), _adr(dtokens), _adr(workspace),
          _ws_bytes(workspace))


def moe_combine_backward(dout, expert_out, slot_of, topk_w, dexpert_out=None, dtopk_w=None,
                         stream=None):
    """Gradient of moe_combine: dexpert_out (topk_w is read) and dtopk_w (expert_out is read)."""
    import torch
    where = "moe_combine_backward"
    T, d = dout.shape
    k = slot_of.shape[1]
    code, el, f32 = _dtype(dout), dout.dtype, torch.float32
    if dtopk_w is not None:
        _required(where, expert_out=expert_out)
    rows = expert_out if expert_out is not None else dexpert_out
    S_max = rows.shape[0] if rows is not None else 0
    dev = _device_of(where, "dout slot_of expert_out topk_w dexpert_out dtopk_w",
                     ((dout, el, (T, d)), (slot_of, torch.int32, (T, k)), (expert_out, el, (S_max, d)),
                      (topk_w, f32, (T, k)), (dexpert_out, el, (S_max, d)), (dtopk_w, f32, (T, k))))
    _call(where, dev, stream, dout.data_ptr(), _adr(expert_out), slot_of.data_ptr(), _adr(topk_w), code,
          T, d, k, S_max, _adr(dexpert_out), _adr(dtopk_w))


def moe_adapter_workspace_size(T, d_in, d_out, r, N, S_max, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(get_lib().moe_adapter_workspace_size(T, d_in, d_out, r, N, S_max, _code(dtype),
                                                ctypes.byref(n)), "moe_adapter_workspace_size")
    return n.value


def moe_adapter_forward(tokens, perm, offsets, A, B, scale, out, workspace, base=None, hidden=None,
                        stream=None):
    """out[t] = base[t] + scale[n] (tokens[t] A[n]) B[n] for every slot of perm / offsets."""
    import torch
    where = "moe_adapter_forward"
    T, d_in = tokens.shape
    N, _, r = A.shape
    d_out, S_max = B.shape[2], perm.shape[0]
    code, el, f32, i32 = _dtype(tokens), tokens.dtype, torch.float32, torch.int32
    dev = _device_of(where, "tokens perm offsets A B scale out base hidden workspace",
                     ((tokens, el, (T, d_in)), (perm, i32, (S_max,)), (offsets, i32, (N + 1,)),
                      (A, el, (N, d_in, r)), (B, el, (N, r, d_out)), (scale, f32, (N,)),
                      (out, el, (T, d_out)), (base, el, (T, d_out)), (hidden, f32, (S_max, r)),
                      (workspace, torch.uint8, workspace.shape)))
    _call(where, dev, stream, tokens.data_ptr(), perm.data_ptr(), offsets.data_ptr(), A.data_ptr(),
          B.data_ptr(), scale.data_ptr(), _adr(base), code, T, d_in, d_out, r, N, S_max, out.data_ptr(),
          _adr(hidden), workspace.data_ptr(), workspace.numel())


def moe_adapter_backward(dout, tokens, hidden, perm, offsets, A, B, scale, workspace, dtokens=None,
                         dtokens_in=None, dA=None, dB=None, stream=None):
    """Gradients of moe_adapter_forward: dtokens (added to dtokens_in), dA and dB in float32."""
    import torch
    where = "moe_adapter_backward"
    T, d_out = dout.shape
    N, d_in, r = A.shape
    S_max = perm.shape[0]
    code, el, f32, i32 = _dtype(dout), dout.dtype, torch.float32, torch.int32
    dev = _device_of(where, "dout perm offsets A B scale tokens hidden dtokens dtokens_in dA dB workspace",
                     ((dout, el, (T, d_out)), (perm, i32, (S_max,)), (offsets, i32, (N + 1,)),
                      (A, el, (N, d_in, r)), (B, el, (N, r, d_out)), (scale, f32, (N,)),
                      (tokens, el, (T, d_in)), (hidden, f32, (S_max, r)), (dtokens, el, (T, d_in)),
                      (dtokens_in, el, (T, d_in)), (dA, f32, (N, d_in, r)), (dB, f32, (N, r, d_out)),
                      (workspace, torch.uint8, workspace.shape)))
    _call(where, dev, stream, dout.data_ptr(), _adr(tokens), _adr(hidden), perm.data_ptr(),
          offsets.data_ptr(), A.data_ptr(), B.data_ptr(), scale.data_ptr(), _adr(dtokens_in), code, T,
          d_in, d_out, r, N, S_max, _adr(dtokens), _adr(dA), _adr(dB), workspace.data_ptr(),
          workspace.numel())


# ---------------------------------------------------------------- a block of routed experts
def moe_route(tokens, Wg, k, topk_idx, topk_w, logits_out=None, logits_in=None, scores_out=None, bias=None,
              token_mask=None, score=MOE_SCORE_SOFTMAX, n_groups=1, top_groups=1, group_top=1,
              renormalize=True, scale=1.0, stream=None):
    """Routing by softmax or sigmoid scores: balance bias, groups of experts, top-k, weights."""
    import torch
    where = "moe_route"
    f32, i32 = torch.float32, torch.int32
    if logits_in is not None:
        T, E = logits_in.shape
        d, code = 1, MOE_F32
        given = [(logits_in, f32, (T, E))]
        names = "logits_in"
    else:
        _required(where, tokens=tokens, Wg=Wg, logits_out=logits_out)
        T, d = tokens.shape
        E, code = Wg.shape[1], _dtype(tokens)
        given = [(tokens, tokens.dtype, (T, d)), (Wg, f32, (d, E))]
        names = "tokens Wg"
    given += [(topk_idx, i32, (T, k)), (topk_w, f32, (T, k)), (logits_out, f32, (T, E)),
              (scores_out, f32, (T, E)), (bias, f32, (E,)), (token_mask, _mask_type(where, token_mask), (T,))]
    dev = _device_of(where, names + " topk_idx topk_w logits_out scores_out bias token_mask", given)
    x = None if logits_in is not None else tokens.data_ptr()
    _call(where, dev, stream, x, code, None if x is None else Wg.data_ptr(), _adr(logits_in), _adr(bias),
          _adr(token_mask), T, d, E, k, score, n_groups, top_groups, group_top, int(renormalize), scale,
          _adr(logits_out), _adr(scores_out), topk_idx.data_ptr(), topk_w.data_ptr())


def moe_route_backward(logits, topk_idx, dlogits, dtopk_w=None, dscores=None, token_mask=None,
                       score=MOE_SCORE_SOFTMAX, renormalize=True, scale=1.0, tokens=None, Wg=None, dWg=None,
                       dtokens=None, dtokens_in=None, workspace=None, stream=None):
    """Gradient of moe_route's weights and scores: dlogits, and from it dWg and dtokens.

    The workspace is moe_gate_backward_workspace_size's."""
    import torch
    where = "moe_route_backward"
    T, E = logits.shape
    k = topk_idx.shape[1]
    f32 = torch.float32
    given = [(logits, f32, (T, E)), (topk_idx, torch.int32, (T, k)), (dlogits, f32, (T, E)),
             (dtopk_w, f32, (T, k)), (dscores, f32, (T, E)), (token_mask, _mask_type(where, token_mask), (T,))]
    names = "logits topk_idx dlogits dtopk_w dscores token_mask"
    code, d = MOE_F32, 4
    if dWg is not None or dtokens is not None:
        if dWg is not None:
            _required(where, tokens=tokens)
        if dtokens is not None:
            _required(where, Wg=Wg)
        like = tokens if dWg is not None else dtokens
        d, el, code = like.shape[1], like.dtype, _dtype(like)
        given += [(tokens if dWg is not None else None, el, (T, d)),
                  (Wg if dtokens is not None else None, f32, (d, E)), (dWg, f32, (d, E)),
                  (dtokens, el, (T, d)), (dtokens_in, el, (T, d)),
                  (workspace, torch.uint8, None if workspace is None else workspace.shape)]
        names += " tokens Wg dWg dtokens dtokens_in workspace"
    dev = _device_of(where, names, given)
    _call(where, dev, stream, logits.data_ptr(), topk_idx.data_ptr(), _adr(dtopk_w), _adr(dscores),
          _adr(token_mask), _adr(tokens), _adr(Wg), code, T, d, E, k, score, int(renormalize), scale,
          dlogits.data_ptr(), _adr(dWg), _adr(dtokens_in), _adr(dtokens), _adr(workspace), _ws_bytes(workspace))


def _fp8_type(where, name, t):
    """torch.float8_e4m3fn, or torch.uint8 for the same bytes."""
    import torch
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"{where}: {name} is {t.dtype}, expected torch.float8_e4m3fn or torch.uint8")
    return t.dtype


def moe_fp8_quantize(W, Wq, scales, stream=None):
    """Expert weights W [E, K, N] to e4m3: Wq [E, N, K] and the scale of each 128 x 128 block."""
    import torch
    where = "moe_fp8_quantize"
    E, K, N = W.shape
    code = _dtype(W)
    dev = _device_of(where, "W Wq scales",
                     ((W, W.dtype, (E, K, N)), (Wq, _fp8_type(where, "Wq", Wq), (E, N, K)),
                      (scales, torch.float32, (E, N // 128, K // 128))))
    _call(where, dev, stream, W.data_ptr(), code, E, K, N, Wq.data_ptr(), scales.data_ptr())


def moe_expert_fp8_workspace_size(T, d, f, E, S_max, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(get_lib().moe_expert_fp8_workspace_size(T, d, f, E, S_max, _code(dtype), ctypes.byref(n)),
           "moe_expert_fp8_workspace_size")
    return n.value


def moe_expert_ffn_fp8(tokens, perm, offsets, W1q, W1s, W2q, W2s, S_max, expert_out, workspace, stream=None):
    """moe_expert_ffn with weights, tokens and hidden rows in e4m3, a scale for each 128."""
    import torch
    where = "moe_expert_ffn_fp8"
    T, d = tokens.shape
    E, f, _ = W1q.shape
    el, f32, i32 = tokens.dtype, torch.float32, torch.int32
    if perm.numel() < S_max or expert_out.shape[0] < S_max:
        raise ValueError(f"{where}: perm and expert_out need S_max = {S_max} rows")
    dev = _device_of(where, "tokens perm offsets W1q W1s W2q W2s expert_out workspace",
                     ((tokens, el, (T, d)), (perm, i32, (perm.numel(),)), (offsets, i32, (E + 1,)),
                      (W1q, _fp8_type(where, "W1q", W1q), (E, f, d)), (W1s, f32, (E, f // 128, d // 128)),
                      (W2q, _fp8_type(where, "W2q", W2q), (E, d, f)), (W2s, f32, (E, d // 128, f // 128)),
                      (expert_out, el, (expert_out.shape[0], d)), (workspace, torch.uint8, workspace.shape)))
    _call(where, dev, stream, tokens.data_ptr(), perm.data_ptr(), offsets.data_ptr(), W1q.data_ptr(),
          W1s.data_ptr(), W2q.data_ptr(), W2s.data_ptr(), _dtype(tokens), T, d, f, E, S_max,
          expert_out.data_ptr(), workspace.data_ptr(), workspace.numel())


def _experts_of(expert_out, slot_of, topk_w, el, T, d):
    """k, S_max and the checks of a block's expert rows (all None: a block without experts)."""
    import torch
    k = 0 if slot_of is None else slot_of.shape[1]
    S_max = 0 if expert_out is None else expert_out.shape[0]
    return k, S_max, [(expert_out, el, (S_max, d)), (slot_of, torch.int32, (T, k)),
                      (topk_w, torch.float32, (T, k))]


def moe_block_norm(residual, hidden_out=None, expert_out=None, slot_of=None, topk_w=None, shared=None, post_w=None,
                   gate=None, alpha=1.0, next_w=None, normed_out=None, eps=1e-6, rstd_post=None, rstd_next=None,
                   stream=None):
    """hidden = residual + alpha gate norm(sum of expert rows + shared) post_w;  normed = norm(hidden) next_w."""
    import torch
    where = "moe_block_norm"
    T, d = residual.shape
    code, el, f32 = _dtype(residual), residual.dtype, torch.float32
    k, S_max, experts = _experts_of(expert_out, slot_of, topk_w, el, T, d)
    dev = _device_of(where, "residual expert_out slot_of topk_w hidden_out shared post_w gate next_w normed_out "
                            "rstd_post rstd_next",
                     [(residual, el, (T, d))] + experts +
                     [(hidden_out, el, (T, d)), (shared, el, (T, d)), (post_w, f32, (d,)), (gate, f32, (d,)),
                      (next_w, f32, (d,)), (normed_out, el, (T, d)), (rstd_post, f32, (T,)), (rstd_next, f32, (T,))])
    _call(where, dev, stream, residual.data_ptr(), _adr(expert_out), _adr(slot_of), _adr(topk_w), _adr(shared),
          _adr(post_w), _adr(gate), alpha, _adr(next_w), eps, code, T, d, k, S_max, _adr(hidden_out),
          _adr(normed_out), _adr(rstd_post), _adr(rstd_next))


def moe_block_norm_workspace_size(T, d, k, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(get_lib().moe_block_norm_workspace_size(T, d, k, _code(dtype), ctypes.byref(n)),
           "moe_block_norm_workspace_size")
    return n.value


def moe_block_norm_backward(dhidden=None, dnormed=None, hidden=None, rstd_next=None, next_w=None, expert_out=None,
                            slot_of=None, topk_w=None, shared=None, post_w=None, rstd_post=None, gate=None,
                            alpha=1.0, dresidual=None, dexpert_out=None, dtopk_w=None, dshared=None, dpost_w=None,
                            dgate=None, dnext_w=None, workspace=None, stream=None):
    """Gradients of moe_block_norm from those of hidden_out and normed_out."""
    import torch
    where = "moe_block_norm_backward"
    like = dhidden if dhidden is not None else dnormed
    if like is None:
        raise ValueError(f"{where}: dhidden or dnormed is required")
    T, d = like.shape
    code, el, f32 = _dtype(like), like.dtype, torch.float32
    k, S_max, experts = _experts_of(expert_out, slot_of, topk_w, el, T, d)
    dev = _device_of(where, ("dhidden" if dhidden is not None else "dnormed") + " dnormed hidden rstd_next next_w "
                            "expert_out slot_of topk_w shared post_w rstd_post gate dresidual dexpert_out dtopk_w "
                            "dshared dpost_w dgate dnext_w workspace",
                     [(like, el, (T, d)), (dnormed, el, (T, d)), (hidden, el, (T, d)), (rstd_next, f32, (T,)),
                      (next_w, f32, (d,))] + experts +
                     [(shared, el, (T, d)), (post_w, f32, (d,)), (rstd_post, f32, (T,)), (gate, f32, (d,)),
                      (dresidual, el, (T, d)), (dexpert_out, el, (S_max, d)), (dtopk_w, f32, (T, k)),
                      (dshared, el, (T, d)), (dpost_w, f32, (d,)), (dgate, f32, (d,)), (dnext_w, f32, (d,)),
                      (workspace, torch.uint8, None if workspace is None else workspace.shape)])
    _call(where, dev, stream, _adr(dhidden), _adr(dnormed), _adr(hidden), _adr(rstd_next), _adr(next_w),
          _adr(expert_out), _adr(slot_of), _adr(topk_w), _adr(shared), _adr(post_w), _adr(rstd_post), _adr(gate),
          alpha, code, T, d, k, S_max, _adr(dresidual), _adr(dexpert_out), _adr(dtopk_w), _adr(dshared),
          _adr(dpost_w), _adr(dgate), _adr(dnext_w), _adr(workspace), _ws_bytes(workspace))
