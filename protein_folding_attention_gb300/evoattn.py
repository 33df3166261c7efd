"""Python binding of the EvoAttention C ABI (``include/evoattn.h``).

Argument marshalling only: every step of the computation runs in the CUDA
library ``libevoattn.so`` built in-tree by ``build_lib.build()``.  PyTorch
provides device memory and the current stream; tensors are passed as raw
pointers plus element strides.  There is no fallback: if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import bisect
import contextlib
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libevoattn.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(7)
BF16, F32 = 0, 1
DBIAS_DETERMINISTIC, DBIAS_ATOMIC = 0, 1
DQ_DETERMINISTIC = 2  # OR-ed with either: dq bit-identical too
DBIAS_FUSED = 4  # dbias summed in the dK/dV pass (fp32 atomics)
NORM_LAYER, NORM_RMS = 0, 1
ADAMW_BLOCK = 256  # elements that share a scale in the 8-bit states
ADAMW_CLIP = 1

_lib = None
_I64_5 = ctypes.c_int64 * 5
_I64_4 = ctypes.c_int64 * 4
_I64_3 = ctypes.c_int64 * 3


class AdamwTensor(ctypes.Structure):
    """evoattn_adamw_tensor: one tensor of an AdamW step."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("weight_decay", ctypes.c_float), ("grad_dtype", ctypes.c_int32)]


class EvoAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def load(path: str = LIB_PATH):
    """Load the CUDA library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"EvoAttention CUDA library not built: {path} is missing "
                           "(run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i64p, u8p, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p, ctypes.c_void_p
    i, u, sz = ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
    lib.evoattn_fwd.argtypes = [vp, i64p, vp, i64p, vp, i64p, vp, i64p, u8p, i64p, vp, i64p,
                                vp, i64p, fp, i, i, i, i, i, i, vp]
    lib.evoattn_fwd.restype = i
    lib.evoattn_bwd_workspace_size.argtypes = [i, i, i, i, i, i, u]
    lib.evoattn_bwd_workspace_size.restype = sz
    lib.evoattn_bwd.argtypes = [vp, i64p, vp, i64p, vp, i64p, vp, i64p, u8p, i64p, vp, i64p,
                                vp, i64p, fp, vp, i64p, vp, i64p, vp, i64p, vp, i64p, fp,
                                vp, i64p, i, i, i, i, i, i, u, vp, sz, vp]
    lib.evoattn_bwd.restype = i
    lib.evoattn_bwd_profiled.argtypes = lib.evoattn_bwd.argtypes + [ctypes.POINTER(vp)]
    lib.evoattn_bwd_profiled.restype = i
    lib.evoattn_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.evoattn_get_device_status.restype = i
    lib.evoattn_status_string.argtypes = [i]
    lib.evoattn_status_string.restype = ctypes.c_char_p
    lib.evoattn_version.argtypes = []
    lib.evoattn_version.restype = i
    lib.evoattn_ln_proj.argtypes = [vp, fp, fp, vp, ctypes.c_float, vp, vp, vp, vp, vp,
                                    i, i, i, i, i, vp]
    lib.evoattn_ln_proj.restype = i
    lib.evoattn_transition.argtypes = [vp, vp, vp, fp, fp, vp, vp, ctypes.c_float, vp,
                                       i, i, i, i, i, vp]
    lib.evoattn_transition.restype = i
    f, d = ctypes.c_float, ctypes.c_double
    lib.evoattn_block_norm.argtypes = [vp, i64p] * 3 + [fp] * 5 + [vp, i64p] * 2 + [i] * 7 + [f, vp]
    lib.evoattn_block_norm.restype = i
    lib.evoattn_block_norm_bwd_workspace_size.argtypes = [i]
    lib.evoattn_block_norm_bwd_workspace_size.restype = sz
    lib.evoattn_block_norm_bwd.argtypes = ([vp, i64p] * 5 + [fp] * 4 + [vp, i64p] * 3 + [fp] * 5 +
                                           [i] * 7 + [f, vp, sz, vp])
    lib.evoattn_block_norm_bwd.restype = i
    lib.evoattn_block_norm_packed.argtypes = [ctypes.c_char_p, vp]
    lib.evoattn_block_norm_packed.restype = i
    lib.evoattn_block_norm_bwd_packed.argtypes = [ctypes.c_char_p, vp]
    lib.evoattn_block_norm_bwd_packed.restype = i
    lib.evoattn_grad_norm_workspace_size.argtypes = [i]
    lib.evoattn_grad_norm_workspace_size.restype = sz
    lib.evoattn_grad_norm.argtypes = [ctypes.POINTER(AdamwTensor), i, f, vp, vp, sz, vp]
    lib.evoattn_grad_norm.restype = i
    lib.evoattn_adamw.argtypes = [ctypes.POINTER(AdamwTensor), i, f, vp, d, d, f, i, u, vp, vp]
    lib.evoattn_adamw.restype = i
    lib.evoattn_debug_set_wait.argtypes = [ctypes.c_ulonglong, i]
    lib.evoattn_debug_set_wait.restype = i
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().evoattn_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s5(t):
    return None if t is None else _I64_5(*t.stride())


def _s4(t):
    return None if t is None else _I64_4(*t.stride())


def _s3(t):
    return None if t is None else _I64_3(*t.stride())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, what: str):
    if status != OK:
        raise EvoAttnError(status, what)


def fwd(q, k, v, pair_bias, mask=None, gate=None, out=None, lse=None, stream=None):
    """out = sigmoid(gate) * softmax(q k^T / sqrt(D) + pair_bias + mask_bias) v.

    q, k, v, gate: [B,S,H,N,D] (any strides; bf16 needs unit stride along D);
    pair_bias: [B,H,N,N]; mask: [B,S,N] uint8/bool (nonzero = keep) or None.
    Returns (out, lse); out defaults to a dense tensor like q, lse is fp32
    [B,S,H,N] contiguous.
    """
    lib = load()
    B, S, H, N, D = q.shape
    if out is None:
        out = torch.empty((B, S, H, N, D), device=q.device, dtype=q.dtype)
    if lse is None:
        lse = torch.empty((B, S, H, N), device=q.device, dtype=torch.float32)
    if mask is not None and mask.dtype != torch.uint8:
        mask = mask.to(torch.uint8)
    st = lib.evoattn_fwd(_ptr(q), _s5(q), _ptr(k), _s5(k), _ptr(v), _s5(v),
                         _ptr(pair_bias), _s4(pair_bias), _ptr(mask), _s3(mask),
                         _ptr(gate), _s5(gate), _ptr(out), _s5(out), _ptr(lse),
                         B, S, H, N, D, _dtype_code(q), _stream(stream))
    _check(st, "evoattn_fwd")
    return out, lse


def workspace_size(B, S, H, N, D, dtype=torch.bfloat16, flags=DBIAS_DETERMINISTIC) -> int:
    code = BF16 if dtype == torch.bfloat16 else F32
    return int(load().evoattn_bwd_workspace_size(B, S, H, N, D, code, flags))


def bwd(q, k, v, pair_bias, mask, gate, out, lse, dout, flags=DBIAS_DETERMINISTIC,
        dq=None, dk=None, dv=None, dbias=None, dgate=None, workspace=None, stream=None,
        stage_events=None):
    """Gradients of sum(out * dout).  Returns dict dq, dk, dv (like q), dbias
    (fp32 [B,H,N,N]) and dgate (None without a gate).  `stage_events`: five
    torch.cuda.Event recorded around the backward's kernels (see
    evoattn_bwd_profiled)."""
    lib = load()
    B, S, H, N, D = q.shape
    mk = lambda t: t if t is not None else torch.empty((B, S, H, N, D), device=q.device,
                                                       dtype=q.dtype)
    dq, dk, dv = mk(dq), mk(dk), mk(dv)
    if gate is not None:
        dgate = mk(dgate)
    else:
        dgate = None
    if dbias is None:
        dbias = torch.empty((B, H, N, N), device=q.device, dtype=torch.float32)
    if mask is not None and mask.dtype != torch.uint8:
        mask = mask.to(torch.uint8)
    need = workspace_size(B, S, H, N, D, q.dtype, flags)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    args = (_ptr(q), _s5(q), _ptr(k), _s5(k), _ptr(v), _s5(v),
            _ptr(pair_bias), _s4(pair_bias), _ptr(mask), _s3(mask),
            _ptr(gate), _s5(gate), _ptr(out), _s5(out), _ptr(lse),
            _ptr(dout), _s5(dout), _ptr(dq), _s5(dq), _ptr(dk), _s5(dk),
            _ptr(dv), _s5(dv), _ptr(dbias), _ptr(dgate), _s5(dgate),
            B, S, H, N, D, _dtype_code(q), flags, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if stage_events is None:
        st = lib.evoattn_bwd(*args)
    else:
        if len(stage_events) != 5:
            raise ValueError("stage_events needs 5 events")
        cur = stream if stream is not None else torch.cuda.current_stream()
        for e in stage_events:           # torch creates events lazily on first record
            if not getattr(e, "cuda_event", 0):
                e.record(cur)
        handles = (ctypes.c_void_p * 5)(*[ctypes.c_void_p(e.cuda_event) for e in stage_events])
        st = lib.evoattn_bwd_profiled(*args, handles)
    _check(st, "evoattn_bwd")
    return {"dq": dq, "dk": dk, "dv": dv, "dbias": dbias, "dgate": dgate}


def ln_proj(z, gamma, beta, w, H, D, eps=1e-5, out=None, stream=None):
    """EvoFusion upstream stack: LayerNorm of z [B, N, N, C] (bf16, dense) with
    gamma, beta [C] (fp32), then the bias-free projection w [4*H*D + H, C]
    (bf16).  Returns (q, k, v, g, pair_bias): q..g [B, N, N, H, D] bf16 and
    pair_bias [B, H, N, N] bf16 (see evoattn_ln_proj).  `out` may supply the
    five output tensors."""
    lib = load()
    B, N, N2, C = z.shape
    if N2 != N:
        raise ValueError("z must be [B, N, N, C]")
    if out is None:
        mk = lambda: torch.empty((B, N, N, H, D), device=z.device, dtype=torch.bfloat16)
        out = (mk(), mk(), mk(), mk(),
               torch.empty((B, H, N, N), device=z.device, dtype=torch.bfloat16))
    q, k, v, g, bias = out
    st = lib.evoattn_ln_proj(_ptr(z), _ptr(gamma), _ptr(beta), _ptr(w), float(eps),
                             _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(bias),
                             B, N, C, H, D, _stream(stream))
    _check(st, "evoattn_ln_proj")
    return q, k, v, g, bias


def transition(z, gamma, beta, w1, w2, eps=1e-5, o=None, w_o=None, out=None, stream=None):
    """EvoFusion downstream stack: z1 = z + o w_o^T (when o is given), then
    out = z1 + SwiGLU transition of LayerNorm(z1), for z [B, N, N, C] (bf16,
    dense), o [B, N, N, HD] and w_o [C, HD] (bf16), gamma, beta [C] (fp32),
    w1 [2F, C] and w2 [C, F] (bf16).  Returns out [B, N, N, C] bf16 (see
    evoattn_transition)."""
    lib = load()
    B, N, N2, C = z.shape
    if N2 != N:
        raise ValueError("z must be [B, N, N, C]")
    F = w2.shape[1]
    HD = o.shape[-1] if o is not None else 0
    if out is None:
        out = torch.empty_like(z)
    st = lib.evoattn_transition(_ptr(z), _ptr(o), _ptr(w_o), _ptr(gamma), _ptr(beta),
                                _ptr(w1), _ptr(w2), float(eps), _ptr(out), B, N, C, HD, F,
                                _stream(stream))
    _check(st, "evoattn_transition")
    return out


def _on_device(t):
    """Index of the tensor's device, which has to be the current one (the
    library enqueues on the current device's streams)."""
    index = t.get_device()
    if index < 0 or index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {t.device}: a CUDA tensor on the current device is needed")
    return index


_NO_ROWS = (0, 0, 0, 0, 0)
_PACK_FWD = struct.Struct("=37qd").pack
_PACK_BWD = struct.Struct("=56qd2q").pack


def _add_rows(words, operands, shape, index):
    """Checks [B, I, J, C] operands (tensor, dtype, name) on device `index`
    and appends the address and strides of each."""
    for t, dtype, name in operands:
        if t is None:
            words += _NO_ROWS
            continue
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
            raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on cuda:{index}, "
                             f"got {tuple(t.shape)} {t.dtype} on {t.device}")
        words.append(t.data_ptr())
        words += t.stride()


def _add_vectors(words, vectors, C, index):
    """Checks [C] fp32 parameters (tensor, name) and appends their addresses."""
    shape = (C,)
    for t, name in vectors:
        if t is None:
            words.append(0)
            continue
        if t.dtype is not torch.float32 or t.shape != shape or t.get_device() != index or \
                not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous fp32 [{C}] tensor on cuda:{index}")
        words.append(t.data_ptr())


def _raw_stream(stream, index):
    """The cudaStream_t of `stream` (None: the current one of device `index`)."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


_HERE_AND_NOW = contextlib.nullcontext()


def _allocate_on(stream):
    """Tensors made inside belong to `stream` (None: the current one), so that
    a workspace is not reused before the kernels on that stream are done."""
    return _HERE_AND_NOW if stream is None else torch.cuda.stream(stream)


def _used_on(stream, tensors):
    """The memory of `tensors` (None among them) goes to nobody else before the
    kernels enqueued on `stream` are done with it, whoever drops them."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _expanded(gate, shape):
    if gate is None or gate.shape == shape:
        return gate
    if gate.dim() != 4 or any(g != n and g != 1 for g, n in zip(gate.shape, shape)) or \
            gate.shape[3] != shape[3]:
        raise ValueError(f"gate {tuple(gate.shape)} does not broadcast to {tuple(shape)}")
    return gate.expand(shape)


def block_norm(x, u=None, gate=None, scale=None, gamma_post=None, beta_post=None, gamma_pre=None,
               beta_pre=None, kind=NORM_LAYER, eps=1e-5, pre=True, y_dtype=None, x1=None, y=None,
               stream=None):
    """The seam between two blocks (see evoattn_block_norm):

        x1 = x + scale * sigmoid(gate) * (n(u) * gamma_post + beta_post)
        y  = n(x1) * gamma_pre + beta_pre

    x [B, I, J, C]: the residual stream, bf16 or fp32; u (the block's output)
    and gate: bf16, or fp32 with an fp32 stream; gate may have extent 1 along
    any row axis and is then shared.  scale and the norms' parameters: [C]
    fp32.  `kind`: NORM_LAYER or NORM_RMS.  Any strides with unit stride along
    C (16-byte aligned rows run at full speed).  Without u the call is the
    norm before a block alone (x1 is x), with pre=False the norm after a block
    alone (y is None).  y has u's type; y_dtype names it where there is no u
    (default: x's).  Outputs take x's layout; x1=x updates the stream in place.
    No autograd node is made, whether inputs require gradients or not: the
    gradients are block_norm_bwd's.  Everything is enqueued on, and allocated
    for, `stream` (default: the current one); operands may be dropped after
    the call, but the caller orders `stream` behind the work that writes them.
    Returns (x1, y)."""
    shape = x.shape
    if len(shape) != 4:
        raise ValueError("x must be [B, I, J, C]")
    dev, sd = _on_device(x), x.dtype
    io = u.dtype if u is not None else (y_dtype or sd)
    if y_dtype is not None and y_dtype is not io:
        raise ValueError("y has the type of u")
    if (y is not None and not pre) or (x1 is not None and u is None):
        raise ValueError("y without pre, or x1 without u")
    if gate is not None:
        gate = _expanded(gate, shape)
    words = []
    _add_rows(words, ((x, sd, "x"), (u, io, "u"), (gate, io, "gate")), shape, dev)
    _add_vectors(words, ((scale, "scale"), (gamma_post, "gamma_post"), (beta_post, "beta_post"),
                         (gamma_pre, "gamma_pre"), (beta_pre, "beta_pre")), shape[3], dev)
    with _allocate_on(stream):
        if u is None:
            x1 = x
            words += _NO_ROWS
        elif x1 is None:
            x1 = torch.empty_like(x)
            words.append(x1.data_ptr())
            words += x1.stride()
        else:
            _add_rows(words, ((x1, sd, "x1"),), shape, dev)
        if not pre:
            words += _NO_ROWS
        elif y is None:
            y = torch.empty_like(x, dtype=io)
            words.append(y.data_ptr())
            words += y.stride()
        else:
            _add_rows(words, ((y, io, "y"),), shape, dev)
    if stream is not None:
        _used_on(stream, (x, u, gate, scale, gamma_post, beta_post, gamma_pre, beta_pre, x1, y))
    words += shape
    st = load().evoattn_block_norm_packed(
        _PACK_FWD(*words, _dtype_code(x), F32 if io is torch.float32 else BF16, kind, eps),
        _raw_stream(stream, dev))
    if st != OK:
        _check(st, "evoattn_block_norm")
    return x1, y


def block_norm_bwd(dx1, dy=None, x1=None, u=None, gate=None, scale=None, gamma_post=None,
                   beta_post=None, gamma_pre=None, beta_pre=None, kind=NORM_LAYER, eps=1e-5,
                   dx=None, workspace=None, stream=None):
    """Gradients of block_norm (see evoattn_block_norm_bwd).  dx1: the gradient
    of x1 from what else reads the stream (None for zero); dy: the gradient of
    y (None when the forward had pre=False); x1: the stream as the forward
    returned it (needed with dy); the rest as in the forward.  dx=dx1 works in
    place.  Returns a dict with dx (dx1 itself without dy), du, dgate (in the
    gate's own shape), and fp32 dscale, dgamma_post, dbeta_post, dgamma_pre,
    dbeta_pre of the parameters that were given.  `stream` as in block_norm."""
    lead = dx1 if dx1 is not None else x1
    if lead is None or (dy is None and (u is None or dx1 is None)):
        raise ValueError("dx1 with u, or dy with x1, is needed")
    shape = lead.shape
    if len(shape) != 4:
        raise ValueError("gradients must be [B, I, J, C]")
    if dy is None:
        x1 = None
        if dx is not None:
            raise ValueError("dx without dy: the gradient of x is dx1")
    elif x1 is None:
        raise ValueError("dy needs x1")
    dev, sd, C = _on_device(lead), lead.dtype, shape[3]
    io = u.dtype if u is not None else dy.dtype
    if gate is not None and 0 in gate.stride():
        if stream is not None:
            _used_on(stream, (gate,))
        with _allocate_on(stream):  # an expanded view: each of its rows has its own gradient
            gate = gate.contiguous()
    full = gate if gate is None else _expanded(gate, shape)
    words, out = [], {}
    _add_rows(words, ((dx1, sd, "dx1"), (dy, io, "dy"), (x1, sd, "x1"), (u, io, "u"),
                      (full, io, "gate")), shape, dev)
    _add_vectors(words, ((scale, "scale"), (gamma_post, "gamma_post"), (beta_post, "beta_post"),
                         (gamma_pre, "gamma_pre")), C, dev)
    lib = load()
    with _allocate_on(stream):
        if dy is None:
            words += _NO_ROWS
            out["dx"] = dx1
        else:
            if dx is None:
                dx = torch.empty_like(lead)
            _add_rows(words, ((dx, sd, "dx"),), shape, dev)
            out["dx"] = dx
        if u is None:
            words += _NO_ROWS
        else:
            out["du"] = du = torch.empty_like(u)
            words.append(du.data_ptr())
            words += du.stride()
        if gate is None:
            words += _NO_ROWS
        else:
            out["dgate"] = dgate = torch.empty_like(gate)
            words.append(dgate.data_ptr())
            words += (dgate if full is gate else dgate.expand(shape)).stride()
        for name, t in (("dscale", scale), ("dgamma_post", gamma_post), ("dbeta_post", beta_post),
                        ("dgamma_pre", gamma_pre), ("dbeta_pre", beta_pre)):
            if t is None:
                words.append(0)
            else:
                out[name] = t = torch.empty_like(t)
                words.append(t.data_ptr())
        if workspace is None:
            workspace = torch.empty(lib.evoattn_block_norm_bwd_workspace_size(C), device=lead.device,
                                    dtype=torch.uint8)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    if beta_pre is not None:
        _add_vectors([], ((beta_pre, "beta_pre"),), C, dev)
    if stream is not None:
        _used_on(stream, (dx1, dy, x1, u, gate, scale, gamma_post, beta_post, gamma_pre, dx, workspace))
    words += shape
    st = lib.evoattn_block_norm_bwd_packed(
        _PACK_BWD(*words, _dtype_code(lead), F32 if io is torch.float32 else BF16, kind, eps,
                  workspace.data_ptr(), workspace.numel() * workspace.element_size()),
        _raw_stream(stream, dev))
    if st != OK:
        _check(st, "evoattn_block_norm_bwd")
    return out


def _grad_table(grads):
    """An evoattn_adamw_tensor array with the gradients' fields filled in."""
    table = (AdamwTensor * len(grads))()
    for row, g in zip(table, grads):
        row.grad, row.n, row.grad_dtype = g.data_ptr(), g.numel(), _dtype_code(g)
    return table


def _check_flat(t, n, dtype, device, name):
    if t.dtype != dtype or t.numel() != n or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous {dtype} elements on {device}")


class AdamW:
    """AdamW over many tensors at once, states in 32 or 8 bits (see
    evoattn_adamw), optionally clipped by the norm of all gradients.

    params: fp32 tensors (contiguous); grads: the bf16 or fp32 gradient buffer
    of each, which the backward pass fills before every step (step(grads=...)
    takes others); copies: bf16 tensors that receive the rounded parameters,
    or None (for all or for some).  weight_decay: a number, or one per tensor.
    lr: a number (`opt.lr` may be changed), or a one-element fp32 CUDA tensor
    that the kernel reads (a captured step then follows it).

    The states are flat tensors in which each parameter starts at the next
    multiple of ADAMW_BLOCK elements (`opt.offsets`); exp_avg, exp_avg_sq and,
    for 8 bits, the scales of both (one fp32 per block) may be handed in to
    resume.  With state_bits=8 they are torch.float8_e4m3fn codes: the first
    moment is code * scale, the root of the second one code * scale.  Their
    padding is never written.  The step counter lives on the device.  One
    optimiser is used on one stream at a time.  The tensors' addresses are
    taken here (the gradients' by step(grads=...) too): none of them may be
    given other memory (`p.data = ...`) afterwards.

    One optimiser has one learning rate, and clips by the norm of its own
    gradients only.  The gradients' buffers exist when it is made.  A step
    changes the parameters without autograd's knowledge: a graph recorded
    before it must not be walked backwards after it.
    """

    def __init__(self, params, grads, *, copies=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01, state_bits=32, exp_avg=None, exp_avg_sq=None,
                 exp_avg_scale=None, exp_avg_sq_scale=None, step=0):
        self.params, self.grads = list(params), list(grads)
        n = len(self.params)
        self.copies = [None] * n if copies is None else list(copies)
        if n == 0 or len(self.grads) != n or len(self.copies) != n:
            raise ValueError("as many gradients and copies as parameters, at least one")
        if state_bits not in (32, 8):
            raise ValueError("state_bits is 32 or 8")
        if step < 0:
            raise ValueError("step: the number of steps already taken, not negative")
        decay = [weight_decay] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(decay) != n:
            raise ValueError("one weight_decay, or one per parameter")
        self._index = _on_device(self.params[0])
        self.device = dev = self.params[0].device
        self.lr, self.betas, self.eps, self.state_bits = lr, betas, eps, state_bits
        self.offsets, total = [], 0
        for p in self.params:
            self.offsets.append(total)
            total += -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
        wide = state_bits == 32
        dtype = torch.float32 if wide else torch.float8_e4m3fn

        def state(t, count, kind, name):
            if t is None:
                return torch.zeros(count, device=dev, dtype=kind)
            _check_flat(t, count, kind, dev, name)
            return t

        self.exp_avg = state(exp_avg, total, dtype, "exp_avg")
        self.exp_avg_sq = state(exp_avg_sq, total, dtype, "exp_avg_sq")
        if wide:
            if exp_avg_scale is not None or exp_avg_sq_scale is not None:
                raise ValueError("scales belong to 8-bit states")
            self.exp_avg_scale = self.exp_avg_sq_scale = None
        else:
            blocks = total // ADAMW_BLOCK
            self.exp_avg_scale = state(exp_avg_scale, blocks, torch.float32, "exp_avg_scale")
            self.exp_avg_sq_scale = state(exp_avg_sq_scale, blocks, torch.float32, "exp_avg_sq_scale")
        self._table = (AdamwTensor * n)()
        written = []
        size = self.exp_avg.element_size()
        for i, (row, p, c) in enumerate(zip(self._table, self.params, self.copies)):
            _check_flat(p, p.numel(), torch.float32, dev, f"parameter {i}")
            written.append((p.data_ptr(), 4 * p.numel()))
            if c is not None:
                _check_flat(c, p.numel(), torch.bfloat16, dev, f"copy {i}")
                written.append((c.data_ptr(), 2 * p.numel()))
                row.copy = c.data_ptr()
            at = self.offsets[i]
            row.param, row.n, row.weight_decay = p.data_ptr(), p.numel(), decay[i]
            row.exp_avg = self.exp_avg.data_ptr() + at * size
            row.exp_avg_sq = self.exp_avg_sq.data_ptr() + at * size
            if not wide:
                row.exp_avg_scale = self.exp_avg_scale.data_ptr() + at // ADAMW_BLOCK * 4
                row.exp_avg_sq_scale = self.exp_avg_sq_scale.data_ptr() + at // ADAMW_BLOCK * 4
        written += [(t.data_ptr(), t.numel() * t.element_size()) for t in
                    (self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)
                    if t is not None]
        written = sorted(w for w in written if w[1])
        if any(a + k > b for (a, k), (b, _) in zip(written, written[1:])):
            raise ValueError("parameters, copies and states overlap (is a tensor listed twice?)")
        self._used = set()  # streams whose kernels read and write the rest
        self._starts, self._ends = [a for a, _ in written], [a + k for a, k in written]
        self._bind(self.grads)
        # evoattn_optim_state: step, norm, clip, skip, tickets
        self._state = torch.zeros(8, device=dev, dtype=torch.int32)
        self._state[:2].view(torch.int64).fill_(step)
        #: norm of all gradients at the last clipped step (0-dim fp32, device)
        self.norm = self._state[2:3].view(torch.float32)[0]
        self._workspace = torch.empty(load().evoattn_grad_norm_workspace_size(n), device=dev,
                                      dtype=torch.uint8)

    def _bind(self, grads):
        if len(grads) != len(self.params):
            raise ValueError("as many gradients as parameters")
        for i, (row, g) in enumerate(zip(self._table, grads)):
            if g.dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"gradient {i}: bf16 or fp32, got {g.dtype}")
            _check_flat(g, row.n, g.dtype, self.device, f"gradient {i}")
            at = g.data_ptr()
            k = bisect.bisect_left(self._starts, at + g.numel() * g.element_size()) - 1
            if row.n and k >= 0 and self._ends[k] > at:
                raise ValueError(f"gradient {i} overlaps what a step writes")
        for row, g in zip(self._table, grads):  # all of them, or after an error none
            row.grad, row.grad_dtype = g.data_ptr(), _dtype_code(g)
        self.grads = grads
        self._grads_used = set()  # streams whose kernels read them

    def step(self, max_norm=None, grads=None, stream=None):
        """One step.  max_norm: clip by the norm of all gradients, which is
        returned (the tensor `norm`, overwritten by the next such step); a step
        whose norm is infinite or NaN then changes nothing.  grads: gradients
        to use from now on instead of those bound before.  Everything is
        enqueued on `stream` (default: the current one); gradients that a
        later step replaces may be dropped, but the caller orders `stream`
        behind the work that writes parameters, states and gradients."""
        _on_device(self._state)
        if grads is not None:
            self._bind(list(grads))
        lib, n = load(), len(self.params)
        st = _raw_stream(stream, self._index)
        if stream is not None:
            # (once for each stream: a tensor's memory remembers it until it is freed)
            if stream.cuda_stream not in self._used:
                self._used.add(stream.cuda_stream)
                _used_on(stream, (self._state, self._workspace, self.exp_avg, self.exp_avg_sq,
                                  self.exp_avg_scale, self.exp_avg_sq_scale, *self.params, *self.copies))
            if stream.cuda_stream not in self._grads_used:
                self._grads_used.add(stream.cuda_stream)
                _used_on(stream, self.grads)
        lr, lr_device = self.lr, None
        if isinstance(lr, torch.Tensor):
            _check_flat(lr, 1, torch.float32, self.device, "lr")
            if stream is not None:
                lr.record_stream(stream)
            lr, lr_device = 0.0, lr.data_ptr()
        state = self._state.data_ptr()
        if max_norm is not None:
            _check(lib.evoattn_grad_norm(self._table, n, max_norm, state,
                                         self._workspace.data_ptr(), self._workspace.numel(), st),
                   "evoattn_grad_norm")
        _check(lib.evoattn_adamw(self._table, n, lr, lr_device, self.betas[0], self.betas[1],
                                 self.eps, self.state_bits, 0 if max_norm is None else ADAMW_CLIP,
                                 state, st), "evoattn_adamw")
        return None if max_norm is None else self.norm

    def steps_taken(self) -> int:
        """Steps taken so far (waits for the device)."""
        return int(self._state[:2].view(torch.int64).item())


def grad_norm(grads, stream=None):
    """sqrt of the sum of squares of all elements of the bf16 or fp32 tensors
    `grads` (contiguous), as a 0-dim fp32 tensor (see evoattn_grad_norm).
    `stream` as in block_norm."""
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    index, dev = _on_device(grads[0]), grads[0].device
    for i, g in enumerate(grads):
        if g.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"gradient {i}: bf16 or fp32, got {g.dtype}")
        _check_flat(g, g.numel(), g.dtype, dev, f"gradient {i}")
    lib = load()
    with _allocate_on(stream):
        state = torch.zeros(8, device=dev, dtype=torch.int32)
        ws = torch.empty(lib.evoattn_grad_norm_workspace_size(len(grads)), device=dev, dtype=torch.uint8)
    if stream is not None:
        _used_on(stream, grads)
    _check(lib.evoattn_grad_norm(_grad_table(grads), len(grads), float("inf"), state.data_ptr(),
                                 ws.data_ptr(), ws.numel(), _raw_stream(stream, index)),
           "evoattn_grad_norm")
    return state[2:3].view(torch.float32)[0]


def debug_set_wait(limit_ns: int = 0, stall: bool = False) -> None:
    """Testing hook (evoattn_debug_set_wait): the wait limit of the kernels
    enqueued from now on (0 = the default 2 s) and whether their compute warps'
    first wait stalls until it gives up."""
    _check(load().evoattn_debug_set_wait(int(limit_ns), 1 if stall else 0),
           "evoattn_debug_set_wait")


def device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status word."""
    out = ctypes.c_int(-1)
    _check(load().evoattn_get_device_status(_stream(stream), ctypes.byref(out)),
           "evoattn_get_device_status")
    return out.value
