"""ctypes binding of libkda_b200.so (see include/kda.h).

Argument marshalling only: PyTorch supplies device memory and the current
stream, every step of the layer runs in the library's CUDA kernels.  There is
no CPU fallback; if the library is missing or no CUDA device is present the
calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda_b200.so")
# the checked build (-DKDA_CHECK_G): the prefill also verifies the log-decay range
LIB_CHECKED_PATH = os.path.join(_HERE, "libkda_b200_checked.so")

KDA_DTYPE_F32 = 0
KDA_DTYPE_BF16 = 1

EXPORTS = ("kda_status_string", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd_plan",
           "kda_chunk_fwd", "kda_decode_step", "kda_chunk_fwd_ex", "kda_decode_step_ex",
           "kda_chunk_fwd_summary", "kda_state_compose", "kda_bwd_workspace_size", "kda_bwd",
           "kda_chunk_fwd_check", "kda_build_checks_g", "kda_chunk_fwd_noalloc",
           "kda_chunk_fwd_noalloc_check", "kda_chunk_fwd_sub_pieces",
           "kda_lin_chunk_fwd_workspace_size", "kda_lin_chunk_fwd", "kda_lin_decode_step",
           "kda_lin_bwd_workspace_size", "kda_lin_bwd", "kda_block_norm",
           "kda_block_norm_bwd_workspace_size", "kda_block_norm_bwd")

# flags of the extended entry points (include/kda.h)
FLAG_QK_L2NORM, FLAG_BETA_LOGITS, FLAG_GATE_LOGITS, FLAG_CLAMP_DECAY = 1, 2, 4, 8
# flags of the operators with one decay per head and of the block norms
LIN_DECAY_PER_HEAD = 1
NORM_POST, NORM_PRE, NORM_GATE_SIGMOID, NORM_GATE_SILU = 1, 2, 4, 8

_lib = None
_lib_checked = None


class KdaError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


def load(path: str = LIB_PATH):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if path == LIB_PATH and _lib is not None:
        return _lib
    lib = _open(path)
    if path == LIB_PATH:
        _lib = lib
    return lib


def load_checked():
    """The checked build of the library (a separate handle)."""
    global _lib_checked
    if _lib_checked is None:
        _lib_checked = _open(LIB_CHECKED_PATH)
    return _lib_checked


def _open(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} not found: build it first (python -m kda_linear_attention_fwd_b200.build)")
    lib = ctypes.CDLL(path)
    P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_chunk_fwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.c_int]
    lib.kda_chunk_fwd_workspace_size.restype = sz
    lib.kda_chunk_fwd_plan.argtypes = [i32, i32, i32, P, P, P]
    lib.kda_chunk_fwd_plan.restype = ctypes.c_int
    lib.kda_chunk_fwd_sub_pieces.argtypes = [i32, i32, i32]
    lib.kda_chunk_fwd_sub_pieces.restype = ctypes.c_int32
    lib.kda_chunk_fwd.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                  ctypes.c_int, f32, i32, P, P, P, sz, P]
    lib.kda_chunk_fwd.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, ctypes.c_int,
                                    f32, i32, P]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_chunk_fwd_ex.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                     ctypes.c_int, f32, i32, P, P, i32, P, P, P, sz, P]
    lib.kda_chunk_fwd_ex.restype = ctypes.c_int
    lib.kda_decode_step_ex.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, ctypes.c_int,
                                       f32, i32, P]
    lib.kda_decode_step_ex.restype = ctypes.c_int
    lib.kda_chunk_fwd_summary.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, ctypes.c_int,
                                          i32, P, P, P, sz, P]
    lib.kda_chunk_fwd_summary.restype = ctypes.c_int
    lib.kda_state_compose.argtypes = [P, P, i32, P, P, i32, i32, i32, i32, P]
    lib.kda_state_compose.restype = ctypes.c_int
    lib.kda_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.kda_bwd_workspace_size.restype = sz
    lib.kda_bwd.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, ctypes.c_int,
                            f32, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.kda_bwd.restype = ctypes.c_int
    lib.kda_chunk_fwd_check.argtypes = [P, sz, P]
    lib.kda_chunk_fwd_check.restype = ctypes.c_int
    lib.kda_build_checks_g.argtypes = []
    lib.kda_build_checks_g.restype = ctypes.c_int
    lib.kda_chunk_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                          ctypes.c_int, f32, i32, P, P, P]
    lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.kda_chunk_fwd_noalloc_check.argtypes = [P]
    lib.kda_chunk_fwd_noalloc_check.restype = ctypes.c_int
    i64 = ctypes.c_int64
    lib.kda_lin_chunk_fwd_workspace_size.argtypes = [i32] * 6 + [ctypes.c_int]
    lib.kda_lin_chunk_fwd_workspace_size.restype = sz
    lib.kda_lin_chunk_fwd.argtypes = [P] * 7 + [i32] * 6 + [ctypes.c_int, f32, i32, P, P, P, sz, P]
    lib.kda_lin_chunk_fwd.restype = ctypes.c_int
    lib.kda_lin_decode_step.argtypes = [P] * 6 + [i32] * 5 + [ctypes.c_int, f32, i32, P]
    lib.kda_lin_decode_step.restype = ctypes.c_int
    lib.kda_lin_bwd_workspace_size.argtypes = [i32] * 6
    lib.kda_lin_bwd_workspace_size.restype = sz
    lib.kda_lin_bwd.argtypes = [P] * 7 + [i32] * 6 + [ctypes.c_int, f32, i32] + [P] * 8 + [sz, P]
    lib.kda_lin_bwd.restype = ctypes.c_int
    lib.kda_block_norm.argtypes = [P, i64, P, P, i64, P, i64, P, P, P, i64, i32, ctypes.c_int, f32,
                                   f32, i32, P]
    lib.kda_block_norm.restype = ctypes.c_int
    lib.kda_block_norm_bwd_workspace_size.argtypes = [i64, i32, ctypes.c_int]
    lib.kda_block_norm_bwd_workspace_size.restype = sz
    lib.kda_block_norm_bwd.argtypes = [P, P, P, i64, P, P, i64, P, i64, P, P, P, P, P, P, i64, i32,
                                       ctypes.c_int, f32, f32, i32, P, sz, P]
    lib.kda_block_norm_bwd.restype = ctypes.c_int
    return lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def _check(fn, status):
    if status != 0:
        raise KdaError(fn, status, status_string(status))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")


def workspace_size(total_tokens, num_seqs, H, dk, dv, dtype=torch.bfloat16) -> int:
    code = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return int(load().kda_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, code))


def plan(total_tokens, num_seqs, H) -> dict:
    """Piece length, piece bound, launch count and sub-pieces of one
    kda_chunk_fwd call (bf16, dk = dv = 128)."""
    L, P, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    lib = load()
    _check("kda_chunk_fwd_plan", lib.kda_chunk_fwd_plan(
        total_tokens, num_seqs, H, ctypes.byref(L), ctypes.byref(P), ctypes.byref(n)))
    sub = int(lib.kda_chunk_fwd_sub_pieces(total_tokens, num_seqs, H))
    if sub < 1:
        _check("kda_chunk_fwd_sub_pieces", sub)
    return dict(piece_len=L.value, max_pieces=P.value, launches=n.value, sub_pieces=sub)


def _flags(qk_l2norm, beta_logits, gate_logits, clamp_decay):
    return ((FLAG_QK_L2NORM if qk_l2norm else 0) | (FLAG_BETA_LOGITS if beta_logits else 0) |
            (FLAG_GATE_LOGITS if gate_logits else 0) | (FLAG_CLAMP_DECAY if clamp_decay else 0))


def snapshot_offsets(lengths, snapshot_tokens):
    """Running sums of the per-sequence snapshot counts (L - 1) // B."""
    offs = [0]
    for L in lengths:
        offs.append(offs[-1] + (max(int(L), 1) - 1) // snapshot_tokens)
    return offs


def chunk_fwd(q, k, v, g, beta, gate, cu_seqlens, *, scale=1.0, qk_l2norm=False,
              initial_state=None, final_state=None, out=None, workspace=None,
              cu_seqlens_host=None, output_final_state=True, stream=None,
              beta_logits=False, gate_logits=False, clamp_decay=False, snapshot_tokens=0):
    """Prefill over packed sequences.  q, k, g [T, H, dk]; v, gate [T, H, dv];
    beta [T, H]; cu_seqlens int32 [N+1] (device).  Returns (out, final_state),
    plus the snapshots [count, H, dk, dv] fp32 when snapshot_tokens > 0 (the
    state after every snapshot_tokens tokens of each sequence, sequence-major;
    needs the offsets on the host: cu_seqlens_host, else one device read)."""
    lib = load()
    _require_cuda(q, k, v, g, beta, gate, cu_seqlens, initial_state, final_state, out, workspace)
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    code = _dtype_code(q)
    if out is None:
        out = torch.empty(T, H, dv, dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    need = int(lib.kda_chunk_fwd_workspace_size(T, N, H, dk, dv, code))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    host = None
    if cu_seqlens_host is not None:
        host_arr = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
        host = ctypes.cast(host_arr, ctypes.c_void_p)
    flags = _flags(qk_l2norm, beta_logits, gate_logits, clamp_decay)
    if flags & ~FLAG_QK_L2NORM == 0 and not snapshot_tokens:
        st = lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate),
                               _ptr(out), _ptr(cu_seqlens), host, N, T, H, dk, dv, code,
                               float(scale), flags, _ptr(initial_state), _ptr(final_state),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
        _check("kda_chunk_fwd", st)
        return out, final_state
    snaps = offs_dev = None
    if snapshot_tokens:
        cu = list(cu_seqlens_host) if cu_seqlens_host is not None else cu_seqlens.tolist()
        offs = snapshot_offsets([cu[i + 1] - cu[i] for i in range(N)], snapshot_tokens)
        offs_dev = torch.tensor(offs, dtype=torch.int32, device=q.device)
        snaps = torch.empty(max(offs[-1], 1), H, dk, dv, dtype=torch.float32, device=q.device)
    st = lib.kda_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate),
                              _ptr(out), _ptr(cu_seqlens), host, N, T, H, dk, dv, code,
                              float(scale), flags, _ptr(initial_state), _ptr(final_state),
                              int(snapshot_tokens), _ptr(snaps), _ptr(offs_dev), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check("kda_chunk_fwd_ex", st)
    if snapshot_tokens:
        return out, final_state, snaps[:offs[-1]]
    return out, final_state


def decode_step(q, k, v, g, beta, gate, state, *, scale=1.0, qk_l2norm=False, out=None,
                stream=None, beta_logits=False, gate_logits=False, clamp_decay=False):
    """One token per sequence.  q, k, g [N, H, dk]; v, gate [N, H, dv]; beta
    [N, H]; state [N, H, dk, dv] fp32, updated in place.  Returns out."""
    lib = load()
    _require_cuda(q, k, v, g, beta, gate, state, out)
    N, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(N, H, dv, dtype=q.dtype, device=q.device)
    st = lib.kda_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate),
                                _ptr(out), _ptr(state), N, H, dk, dv, _dtype_code(q),
                                float(scale), _flags(qk_l2norm, beta_logits, gate_logits,
                                                     clamp_decay), _stream(stream))
    _check("kda_decode_step_ex", st)
    return out


def chunk_summary(k, v, g, beta, cu_seqlens, *, qk_l2norm=False, beta_logits=False,
                  clamp_decay=False, cu_seqlens_host=None, workspace=None, stream=None):
    """The affine map S -> M S + Z of every sequence's tokens.  k, g [T, H, dk];
    v [T, H, dv]; beta [T, H].  Returns (M [N, H, dk, dk], Z [N, H, dk, dv]) fp32."""
    lib = load()
    _require_cuda(k, v, g, beta, cu_seqlens, workspace)
    T, H, dk = k.shape
    dv = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    code = _dtype_code(k)
    M = torch.empty(N, H, dk, dk, dtype=torch.float32, device=k.device)
    Z = torch.empty(N, H, dk, dv, dtype=torch.float32, device=k.device)
    need = int(lib.kda_chunk_fwd_workspace_size(T, N, H, dk, dv, code))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=k.device)
    host = None
    if cu_seqlens_host is not None:
        host_arr = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
        host = ctypes.cast(host_arr, ctypes.c_void_p)
    st = lib.kda_chunk_fwd_summary(_ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), host,
                                   N, T, H, dk, dv, code,
                                   _flags(qk_l2norm, beta_logits, False, clamp_decay),
                                   _ptr(M), _ptr(Z), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream))
    _check("kda_chunk_fwd_summary", st)
    return M, Z


def state_compose(M, Z, state_in=None, *, out=None, stream=None):
    """Apply the maps (M [R, N, H, dk, dk], Z [R, N, H, dk, dv]) in order to
    state_in [N, H, dk, dv] (None = zeros).  Returns the state."""
    lib = load()
    _require_cuda(M, Z, state_in, out)
    R, N, H, dk, _ = M.shape
    dv = Z.shape[-1]
    M, Z = M.contiguous(), Z.contiguous()
    if out is None:
        out = torch.empty(N, H, dk, dv, dtype=torch.float32, device=M.device)
    st = lib.kda_state_compose(_ptr(M), _ptr(Z), R, _ptr(state_in), _ptr(out), N, H, dk, dv,
                               _stream(stream))
    _check("kda_state_compose", st)
    return out


def bwd_workspace_size(total_tokens, num_seqs, H, dk, dv) -> int:
    return int(load().kda_bwd_workspace_size(total_tokens, num_seqs, H, dk, dv))


def bwd(q, k, v, g, beta, gate, dy, cu_seqlens, *, scale=1.0, initial_state=None,
        d_final_state=None, cu_seqlens_host=None, workspace=None, stream=None):
    """Gradients of the plain forward (kda_bwd): returns a dict of fp32
    tensors dq, dk, dg [T, H, dk]; dv, dgate [T, H, dv] (dgate None without a
    gate); dbeta [T, H]; ds0 [N, H, dk, dv]."""
    lib = load()
    _require_cuda(q, k, v, g, beta, gate, dy, cu_seqlens, initial_state, d_final_state)
    q, k, v, g, beta, dy = (t.contiguous() for t in (q, k, v, g, beta, dy))
    gate = None if gate is None else gate.contiguous()
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dq": torch.empty(T, H, dk, **f32), "dk": torch.empty(T, H, dk, **f32),
           "dg": torch.empty(T, H, dk, **f32), "dv": torch.empty(T, H, dv, **f32),
           "dbeta": torch.empty(T, H, **f32),
           "dgate": None if gate is None else torch.empty(T, H, dv, **f32),
           "ds0": torch.empty(N, H, dk, dv, **f32)}
    need = bwd_workspace_size(T, N, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    cu_arr = None
    if cu_seqlens_host is not None:
        cu_arr = (ctypes.c_int32 * len(cu_seqlens_host))(*cu_seqlens_host)
    s0 = None if initial_state is None else initial_state.float().contiguous()
    dsf = None if d_final_state is None else d_final_state.float().contiguous()
    st = lib.kda_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate), _ptr(dy),
                     _ptr(cu_seqlens), None if cu_arr is None else ctypes.cast(cu_arr, ctypes.c_void_p),
                     N, T, H, dk, dv, _dtype_code(q), float(scale), _ptr(s0), _ptr(dsf),
                     _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                     _ptr(out["dbeta"]), _ptr(out["dgate"]), _ptr(out["ds0"]), _ptr(workspace),
                     workspace.numel(), _stream(stream))
    _check("kda_bwd", st)
    return out


def chunk_fwd_check(workspace, stream=None, lib=None) -> int:
    """Status of the last prefill that used `workspace` (waits for the
    stream): 0 = KDA_OK, else a kda_status code (see include/kda.h)."""
    lib = lib or load()
    return int(lib.kda_chunk_fwd_check(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream(stream)))


# ---------------------------------------------- linear attention, one decay per head
# `stream`: another stream than the current one.  Results and workspaces made here
# belong to it; that the inputs are ready there is the caller's part.
_CODES = {torch.bfloat16: KDA_DTYPE_BF16, torch.float32: KDA_DTYPE_F32}


def _launch(fn, dev, stream, *args):
    """Calls a library function on the tensors' device (made current for the
    call) with the given stream or that device's current one; raises its error."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _launch(fn, dev, stream, *args)
    st = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(fn.__name__, st)


def _make(stream, make):
    """make()'s tensors, in the memory of the call's stream and filled on it: what
    the current stream has yet to do can neither use that memory nor come between."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _keep(stream, dev, *tensors):
    """The tensors of a call on a given stream: not to be given out again before
    that stream has passed the call and the current one has passed their use."""
    if stream is not None:
        here = torch.cuda.current_stream(dev)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
                t.record_stream(here)


def _tensor(name, t, shape, dtype, dev):
    """Address of a tensor, refused when the kernels could not read it as it is."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: want a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                     f"{'' if t.is_contiguous() else ', not contiguous'}")


def _opt(name, t, shape, dtype, dev):
    return None if t is None else _tensor(name, t, shape, dtype, dev)


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    return dev


def _code(t):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _space(workspace, dev, stream, need):
    """(tensor, address, bytes); need() sizes a new one."""
    if workspace is None:
        if torch._C._cuda_getDevice() != dev:  # the plan is the device's
            with torch.cuda.device(dev):
                return _space(None, dev, stream, need)
        workspace = _make(stream, lambda: torch.empty(max(need(), 16), dtype=torch.uint8, device="cuda"))
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: want a contiguous tensor on cuda:{dev}")
    # too small a one is refused by the library
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _lin_shapes(q, k, v, g):
    dev = _device(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k are [tokens, Hk, dk], v is [tokens, H, dv]")
    T, Hk, dk = shape = q.shape
    H, dv = v.shape[1], v.shape[2]
    per_head = g.dim() == 1
    dt = q.dtype
    code = _code(q)
    ptrs = (_tensor("q", q, shape, dt, dev), _tensor("k", k, shape, dt, dev), _tensor("v", v, (T, H, dv), dt, dev),
            _tensor("g", g, (H,) if per_head else (T, H), dt, dev))
    return dev, T, H, Hk, dk, dv, LIN_DECAY_PER_HEAD if per_head else 0, code, ptrs


def _host_offsets(cu_seqlens_host, N):
    if cu_seqlens_host is None:
        return None
    if len(cu_seqlens_host) != N + 1:
        raise ValueError("cu_seqlens_host and cu_seqlens differ in length")
    return (ctypes.c_int32 * (N + 1))(*cu_seqlens_host)


def lin_workspace_size(total_tokens, num_seqs, H, Hk, dk, dv, dtype=torch.bfloat16) -> int:
    return int(load().kda_lin_chunk_fwd_workspace_size(total_tokens, num_seqs, H, Hk, dk, dv,
                                                       _CODES[dtype]))


def lin_chunk_fwd(q, k, v, g, cu_seqlens, *, scale=1.0, initial_state=None, final_state=None,
                  out=None, workspace=None, cu_seqlens_host=None, output_final_state=True,
                  stream=None):
    """Linear attention with one decay per head over packed sequences:
    S <- exp(g) S + k v^T, o = S^T (scale q).  q, k [T, Hk, dk]; v [T, H, dv],
    H a multiple of Hk; g [T, H], or [H] for the same decay at every token;
    cu_seqlens int32 [N+1] (device).  Returns (out, final_state); final_state
    may be initial_state itself.  A device wait that gave up is recorded in the
    workspace: pass one to ask chunk_fwd_check for it."""
    lib = load()
    dev, T, H, Hk, dk, dv, flags, code, ptrs = _lin_shapes(q, k, v, g)
    N = cu_seqlens.shape[0] - 1
    p_cu = _tensor("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    states = (N, H, dk, dv)
    if out is None:
        out = _make(stream, lambda: torch.empty_like(v))
    if final_state is None and output_final_state:
        final_state = _make(stream, lambda: q.new_empty(states, dtype=torch.float32))
    p_out = _tensor("out", out, v.shape, q.dtype, dev)
    p_s0 = _opt("initial_state", initial_state, states, torch.float32, dev)
    p_s1 = _opt("final_state", final_state, states, torch.float32, dev)
    host = _host_offsets(cu_seqlens_host, N)
    ws, p_ws, n_ws = _space(workspace, dev, stream, lambda: lib.kda_lin_chunk_fwd_workspace_size(T, N, H, Hk, dk, dv, code))
    _launch(lib.kda_lin_chunk_fwd, dev, stream, *ptrs, p_out, p_cu, host, N, T, H, Hk, dk, dv, code, float(scale), flags,
            p_s0, p_s1, p_ws, n_ws)
    _keep(stream, dev, ws, out, final_state)
    return out, final_state


def lin_decode_step(q, k, v, g, state, *, scale=1.0, out=None, stream=None):
    """One token per sequence.  q, k [N, Hk, dk]; v [N, H, dv]; g [N, H] or
    [H]; state [N, H, dk, dv] fp32, updated in place.  Returns out."""
    lib = load()
    dev, N, H, Hk, dk, dv, flags, code, ptrs = _lin_shapes(q, k, v, g)
    if out is None:
        out = _make(stream, lambda: torch.empty_like(v))
    p_out = _tensor("out", out, v.shape, q.dtype, dev)
    p_s = _tensor("state", state, (N, H, dk, dv), torch.float32, dev)
    _launch(lib.kda_lin_decode_step, dev, stream, *ptrs, p_out, p_s, N, H, Hk, dk, dv, code, float(scale), flags)
    _keep(stream, dev, out)
    return out


def lin_bwd_workspace_size(total_tokens, num_seqs, H, Hk, dk, dv) -> int:
    return int(load().kda_lin_bwd_workspace_size(total_tokens, num_seqs, H, Hk, dk, dv))


def lin_bwd(q, k, v, g, dy, cu_seqlens, *, scale=1.0, initial_state=None, d_final_state=None,
            cu_seqlens_host=None, workspace=None, stream=None):
    """Gradients of lin_chunk_fwd: a dict of dq, dk [T, Hk, dk], dv [T, H, dv],
    dg (the shape of g), all in the inputs' dtype, and ds0 [N, H, dk, dv] fp32.
    Waits that gave up: as lin_chunk_fwd."""
    lib = load()
    dev, T, H, Hk, dk, dv, flags, code, ptrs = _lin_shapes(q, k, v, g)
    N = cu_seqlens.shape[0] - 1
    p_cu = _tensor("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    p_dy = _tensor("dy", dy, v.shape, q.dtype, dev)
    states = (N, H, dk, dv)
    p_s0 = _opt("initial_state", initial_state, states, torch.float32, dev)
    p_ds = _opt("d_final_state", d_final_state, states, torch.float32, dev)
    # tokens outside every sequence keep what is there: zeros only where the
    # offsets are not known to cover every token
    new = torch.empty_like if cu_seqlens_host is not None else torch.zeros_like
    out = _make(stream, lambda: {"dq": new(q), "dk": new(k), "dv": new(v), "dg": new(g),
                                 "ds0": q.new_empty(states, dtype=torch.float32)})
    host = _host_offsets(cu_seqlens_host, N)
    ws, p_ws, n_ws = _space(workspace, dev, stream, lambda: lib.kda_lin_bwd_workspace_size(T, N, H, Hk, dk, dv))
    _launch(lib.kda_lin_bwd, dev, stream, *ptrs, p_dy, p_cu, host, N, T, H, Hk, dk, dv, code, float(scale), flags, p_s0, p_ds,
            *(x.data_ptr() for x in out.values()), p_ws, n_ws)
    _keep(stream, dev, ws, *out.values())
    return out


# ------------------------------------------------------------ norms around a block
def _norm_rows(name, t, shape, dtype, dev):
    """(address, row stride) of a tensor whose rows (last dimension) are contiguous."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    D = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), D
    rows = t.unsqueeze(0) if t.dim() == 1 else t.flatten(0, -2) if t.dim() != 2 else t
    if rows.data_ptr() != t.data_ptr() or rows.stride(1) != 1 or (rows.shape[0] > 1 and rows.stride(0) < D):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced, got strides {t.stride()}")
    return t.data_ptr(), max(rows.stride(0), D)


def _row_length(shape):
    if not shape:
        raise ValueError("y has no rows: want [..., D]")
    return shape[-1]


def _norm_flags(post_norm, post_weight, pre_norm, pre_weight, gate, gate_logits, gate_silu):
    if gate_logits and gate_silu:
        raise ValueError("gate_logits and gate_silu exclude each other")
    if (post_weight is not None and not post_norm) or (pre_weight is not None and not pre_norm):
        raise ValueError("a weight without its norm")
    return ((NORM_POST if post_norm else 0) | (NORM_PRE if pre_norm else 0) |
            (NORM_GATE_SIGMOID if gate_logits and gate is not None else 0) |
            (NORM_GATE_SILU if gate_silu and gate is not None else 0))


def block_norm(y, *, post_norm=True, post_weight=None, gate=None, gate_logits=False, gate_silu=False,
               residual=None, res_scale=1.0, pre_norm=False, pre_weight=None, eps=1e-6, out=None,
               normed=None, stream=None):
    """The norm of a block's output with its gate and the scaled residual, and
    the next block's norm: u = act(gate) * rmsnorm(y) * post_weight, out =
    residual + res_scale * u, normed = rmsnorm(out) * pre_weight, over the last
    dimension of y [..., D].  Returns (out, normed); normed is None without
    pre_norm.  out and normed may be y, gate or residual themselves."""
    lib = load()
    dev = _device(y)
    shape = y.shape
    D = _row_length(shape)
    code, dt = _code(y), y.dtype
    flags = _norm_flags(post_norm, post_weight, pre_norm, pre_weight, gate, gate_logits, gate_silu)
    p_y, s_y = _norm_rows("y", y, shape, dt, dev)
    p_g, s_g = _norm_rows("gate", gate, shape, dt, dev)
    p_x, s_x = _norm_rows("residual", residual, shape, dt, dev)
    p_wp, p_wn = _opt("post_weight", post_weight, (D,), dt, dev), _opt("pre_weight", pre_weight, (D,), dt, dev)
    if out is None:
        out = _make(stream, lambda: y.new_empty(shape))
    if normed is None and pre_norm:
        normed = _make(stream, lambda: y.new_empty(shape))
    p_out, p_n = _tensor("out", out, shape, dt, dev), _opt("normed", normed, shape, dt, dev)
    _launch(lib.kda_block_norm, dev, stream, p_y, s_y, p_wp, p_g, s_g, p_x, s_x, p_wn, p_out, p_n,
            y.numel() // D if D else 0, D, code, float(res_scale), float(eps), flags)
    _keep(stream, dev, out, normed)
    return out, normed


def block_norm_bwd(dout, dnormed, y, *, post_norm=True, post_weight=None, gate=None, gate_logits=False,
                   gate_silu=False, residual=None, res_scale=1.0, pre_norm=False, pre_weight=None,
                   eps=1e-6, workspace=None, stream=None):
    """Gradients of block_norm for dout and dnormed (either None = zeros): a
    dict of dy, dgate, dresidual in y's dtype and dpost_weight, dpre_weight [D]
    fp32; None for what was not given."""
    lib = load()
    dev = _device(y)
    shape = y.shape
    D = _row_length(shape)
    code, dt = _code(y), y.dtype
    flags = _norm_flags(post_norm, post_weight, pre_norm, pre_weight, gate, gate_logits, gate_silu)
    if dout is None and dnormed is None:
        raise ValueError("dout and dnormed are both None")
    p_y, s_y = _norm_rows("y", y, shape, dt, dev)
    p_g, s_g = _norm_rows("gate", gate, shape, dt, dev)
    p_x, s_x = _norm_rows("residual", residual, shape, dt, dev)
    p_wp, p_wn = _opt("post_weight", post_weight, (D,), dt, dev), _opt("pre_weight", pre_weight, (D,), dt, dev)
    p_do, p_dn = _opt("dout", dout, shape, dt, dev), _opt("dnormed", dnormed, shape, dt, dev)
    rows = y.numel() // D if D else 0

    def like(t, shape=None, dtype=None):
        return None if t is None else y.new_empty(shape or t.shape, dtype=dtype or t.dtype)

    got = _make(stream, lambda: {"dy": like(y), "dgate": like(gate), "dresidual": like(residual),
                                 "dpost_weight": like(post_weight, (D,), torch.float32),
                                 "dpre_weight": like(pre_weight, (D,), torch.float32)})
    ws, p_ws, n_ws = _space(workspace, dev, stream, lambda: lib.kda_block_norm_bwd_workspace_size(rows, D, code))
    _launch(lib.kda_block_norm_bwd, dev, stream, p_do, p_dn, p_y, s_y, p_wp, p_g, s_g, p_x, s_x, p_wn,
            *(None if t is None else t.data_ptr() for t in got.values()), rows, D, code, float(res_scale), float(eps), flags, p_ws, n_ws)
    _keep(stream, dev, ws, *got.values())
    return got
