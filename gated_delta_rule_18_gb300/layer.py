"""The state-space layer's operators (include/gdn.h): residual RMS norm with
an optional 8-bit output, short causal convolution and selective scan, each
for prompts, single tokens and training.

Activations are (B, T, D), bf16 or fp32, with any strides over B and T and a
contiguous last dimension; norms take rows of any leading shape, single-token
calls (n, D). Parameters and scan states are contiguous fp32. Every call runs
on the current stream of its tensors' device, or on `stream`, which has to be
one of that device; what it allocates then belongs to that stream. Wrong
shapes raise ValueError, wrong types and layouts GDNError, both before anything
is launched.
"""
from __future__ import annotations

import ctypes

import torch

F32, BF16, E4M3 = 0, 1, 2
SILU = SOFTPLUS = 1
_F8 = torch.float8_e4m3fn
_CODE = {torch.float32: F32, torch.bfloat16: BF16}
_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_lib = None


def bind(L):
    """Argument types of the library's entry points."""
    act = [_P, _L, _L]
    L.gdn_rmsnorm_fwd.argtypes = [_P, _L, _I, _P, _L, _I, _P, _P, _L, _I, _P, _L, _P, _I, _I, _I, _F, _P]
    L.gdn_rmsnorm_bwd_workspace_size.argtypes = [_I, _I]
    L.gdn_rmsnorm_bwd.argtypes = [_P, _L, _I, _P, _L, _I, _P, _L, _P, _P, _L, _P, _I, _I, _F, _P, _Z, _P]
    L.gdn_conv_fwd.argtypes = act + [_P, _I, _P, _P, _P, _I] + act + [_P, _I, _I, _I, _I, _I, _P, _Z, _P]
    L.gdn_conv_bwd_workspace_size.argtypes = [_I] * 4
    L.gdn_conv_bwd.argtypes = act + [_P, _I, _P, _P, _P, _I] + act + [_P] * 5 + [_I] * 5 + [_P, _Z, _P]
    L.gdn_conv_step.argtypes = [_P, _L, _P, _I, _P, _P, _P, _I, _P, _L, _I, _I, _I, _I, _P]
    L.gdn_ssm_workspace_size.argtypes = [_I] * 6
    L.gdn_ssm_bwd_workspace_size.argtypes = [_I] * 6
    scan = act + act + [_P] + act + act + [_P] + act + [_P, _P, _P, _I] + act
    L.gdn_ssm_fwd.argtypes = scan + [_P] + [_I] * 6 + [_P, _Z, _P]
    L.gdn_ssm_bwd.argtypes = scan + [_P] * 10 + [_I] * 6 + [_P, _Z, _P]
    L.gdn_ssm_step.argtypes = [_P, _L, _P, _L, _P, _P, _L, _P, _L, _P, _P, _L, _P, _P, _P, _I, _P, _L] + [_I] * 5 + [_P]
    for name in ("gdn_rmsnorm_bwd_workspace_size", "gdn_conv_bwd_workspace_size", "gdn_ssm_workspace_size",
                 "gdn_ssm_bwd_workspace_size"):
        getattr(L, name).restype = _Z
    for name in ("gdn_rmsnorm_fwd", "gdn_rmsnorm_bwd", "gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_step",
                 "gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_ssm_step"):
        getattr(L, name).restype = _I


def _load():
    global _lib
    from . import lib
    _lib = lib()
    return _lib


def _fail(status, where):
    from . import GDNError
    raise GDNError(status, where)


def _code(t, name):
    c = _CODE.get(t.dtype)
    if c is None:
        _fail(3, f"{name}: unsupported dtype {t.dtype}")
    return c


def _wrong(t, name, shape, like):
    """Raises what is wrong with an activation."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != like.dtype:
        _fail(3, f"{name} must be {like.dtype} as x is, got {t.dtype}")
    _fail(4, f"{name} must be on {like.device} with a contiguous last dimension")


def _act(t, name, shape, like):
    """(pointer, stride over B, stride over T) of an activation; zeros for None."""
    if t is None:
        return 0, 0, 0
    if t.shape != shape or t.dtype is not like.dtype or t.get_device() != like.get_device():
        _wrong(t, name, shape, like)
    sb, st, sd = t.stride()
    if sd != 1 and shape[2] > 1:
        _wrong(t, name, shape, like)
    return t.data_ptr(), sb, st


def _rows(t, name, shape, like):
    """(pointer, row stride) of a (n, D) tensor; zeros for None."""
    if t is None:
        return 0, 0
    if t.shape != shape or t.dtype is not like.dtype or t.get_device() != like.get_device():
        _wrong(t, name, shape, like)
    st, sd = t.stride()
    if sd != 1 and shape[1] > 1:
        _wrong(t, name, shape, like)
    return t.data_ptr(), st


def _flat(t, name, shape, dtype, like):
    """Pointer of a contiguous tensor of this shape and type; 0 for None."""
    if t is None:
        return 0
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        _fail(3, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous() or t.get_device() != like.get_device():
        _fail(4, f"{name} must be contiguous on {like.device}")
    return t.data_ptr()


# (The library's sizes are 32-bit integers, and ctypes would pass the low half of
# a larger one. The checks stand inline: a call of its own is 0.2 us.)
def _too_large(*sizes):
    raise ValueError(f"a size must be at most 2147483647, got {max(sizes)}")


def _n_seq(cu_seqlens, B, like):
    """(pointer, sequences) of a batch."""
    if cu_seqlens is None:
        return 0, B
    if cu_seqlens.numel() >> 31:
        _too_large(cu_seqlens.numel())
    return _flat(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, like), cu_seqlens.numel() - 1


def _workspace(workspace, need, like):
    if workspace is not None and (workspace.get_device() != like.get_device() or not workspace.is_contiguous()):
        _fail(4, f"workspace must be contiguous on {like.device}")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(int(need), 256), dtype=torch.uint8, device=like.device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# The current stream's handle without building a Stream object (3 us of host
# time, more than a small call's kernel takes), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(like):
    if _raw_stream is not None:
        return _raw_stream(like.get_device())
    return torch.cuda.current_stream(like.device).cuda_stream


# of a tensor of the caller's that a call has written: autograd notices if it had saved one
_count_version = torch.autograd.graph.increment_version
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(x):
    """Whether x lies on another GPU than the current one."""
    if not x.is_cuda:
        _fail(4, "the tensors must be on a GPU")
    return x.get_device() != _current_device()


def _guard(x, stream):
    """The context of a call on x's device: its current stream, or `stream`."""
    if stream is None:
        return torch.cuda.device(x.get_device())
    if stream.device.index != x.get_device():
        _fail(4, f"stream must be on {x.device}, not on {stream.device}")
    return torch.cuda.stream(stream)


def _as_rows(t, name):
    if t is None or t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError:
        _fail(4, f"{name}'s rows must share one stride")


def gdn_rmsnorm_fwd(x, weight, residual=None, eps=1e-6, out_dtype=None, group=0, out=None, residual_out=None,
                    stream=None):
    """y = s / sqrt(mean(s^2) + eps) * weight over the last dimension, with
    s = x + residual (fp32). Returns a dict: "out"; with a residual,
    "residual": s in the residual's type (in residual_out, which may be the
    residual itself, or a new tensor); x's leading dimensions have to be rows
    of one stride; with out_dtype=torch.float8_e4m3fn,
    "scale": fp32, one for each `group` channels (32, 64, 128 or 256; 0: the
    row), out * scale being y."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_rmsnorm_fwd(x, weight, residual, eps, out_dtype, group, out, residual_out)
    L = _lib or _load()
    x2 = x if x.dim() == 2 else _as_rows(x, "x")
    R, D = x2.shape
    if (R | D | abs(group)) >> 31:
        _too_large(R, D, abs(group))
    q8 = out_dtype is _F8
    if out_dtype is not None and not q8 and out_dtype != x.dtype:
        _fail(3, f"out_dtype must be {x.dtype} or torch.float8_e4m3fn, got {out_dtype}")
    ty = out_dtype if q8 else x.dtype
    given = (out, residual_out)
    if out is None:
        out = torch.empty_like(x, dtype=ty, memory_format=torch.contiguous_format)
    elif out.shape != x.shape or out.dtype != ty:
        raise ValueError(f"out must be {tuple(x.shape)} {ty}, got {tuple(out.shape)} {out.dtype}")
    elif out.get_device() != x.get_device():
        _fail(4, f"out must be on {x.device}")
    o2 = _as_rows(out, "out")
    xp, xs = _rows(x2, "x", (R, D), x)
    op, os_ = _rows(o2, "out", (R, D), out)
    res = {"out": out}
    rp = rs = rop = ros = rc = sp = 0
    if residual is not None:
        rc = _code(residual, "residual")
        if residual_out is None:
            residual_out = torch.empty_like(residual, memory_format=torch.contiguous_format)
        elif residual_out.shape != x.shape or residual_out.dtype != residual.dtype:
            raise ValueError(f"residual_out must be {tuple(x.shape)} {residual.dtype}")
        if residual.shape != x.shape:
            raise ValueError(f"residual must have shape {tuple(x.shape)}, got {tuple(residual.shape)}")
        rp, rs = _rows(_as_rows(residual, "residual"), "residual", (R, D), residual)
        rop, ros = _rows(_as_rows(residual_out, "residual_out"), "residual_out", (R, D), residual)
        if residual.get_device() != x.get_device():
            _fail(4, f"residual must be on {x.device}")
        res["residual"] = residual_out
    if q8:
        scale = torch.empty(x.shape[:-1] + ((D + group - 1) // group if group > 0 else 1,), dtype=torch.float32,
                            device=x.device)
        res["scale"] = scale
        sp = scale.data_ptr()
    st = L.gdn_rmsnorm_fwd(xp, xs, _code(x, "x"), rp, rs, rc, _flat(weight, "weight", (D,), torch.float32, x), op, os_,
                           E4M3 if q8 else _CODE[ty], rop, ros, sp, R, D, group, eps, _stream(x))
    if st:
        _fail(st, "gdn_rmsnorm_fwd")
    for t in given:
        if t is not None:
            _count_version(t)
    return res


def gdn_rmsnorm_bwd(s, weight, dy, dres=None, eps=1e-6, workspace=None, stream=None):
    """Gradients of the norm for the sum s that gdn_rmsnorm_fwd returned (or
    x, without a residual), the output's gradient dy and the residual
    stream's own gradient dres (s's type): a dict of "dx" (s's type; the
    gradient of x and of the residual alike) and "dweight" (fp32)."""
    if stream is not None or _elsewhere(s):
        with _guard(s, stream):
            return gdn_rmsnorm_bwd(s, weight, dy, dres, eps, workspace)
    L = _lib or _load()
    s2 = _as_rows(s, "s")
    R, D = s2.shape
    if (R | D) >> 31:
        _too_large(R, D)
    if dy.shape != s.shape or dy.device != s.device:
        raise ValueError(f"dy must have shape {tuple(s.shape)} on {s.device}, got {tuple(dy.shape)}")
    dx = torch.empty(s.shape, dtype=s.dtype, device=s.device)
    dw = torch.empty(D, dtype=torch.float32, device=s.device)
    sp, ss = _rows(s2, "s", (R, D), s)
    yp, ys = _rows(_as_rows(dy, "dy"), "dy", (R, D), dy)
    rp, rs = _rows(_as_rows(dres, "dres"), "dres", (R, D), s)
    ws, wp, wn = _workspace(workspace, L.gdn_rmsnorm_bwd_workspace_size(R, D), s)
    st = L.gdn_rmsnorm_bwd(sp, ss, _code(s, "s"), yp, ys, _code(dy, "dy"), rp, rs,
                           _flat(weight, "weight", (D,), torch.float32, s), dx.data_ptr(), D, dw.data_ptr(), R, D,
                           eps, wp, wn, _stream(s))
    if st:
        _fail(st, "gdn_rmsnorm_bwd")
    return {"dx": dx, "dweight": dw}


def gdn_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, final_state=None, silu=True, out=None,
                 workspace=None, stream=None):
    """Causal depthwise convolution of W taps and SiLU. x (B, T, D); weight
    (D, W), bias (D) fp32; initial_state / final_state (n_seq, W - 1, D) in
    x's type, the inputs before and at the end of each sequence, oldest
    first; cu_seqlens int32 (n_seq + 1) with B == 1. Returns out."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_conv_fwd(x, weight, bias, initial_state, cu_seqlens, final_state, silu, out, workspace)
    L = _lib or _load()
    B, T, D = x.shape
    _, W = weight.shape
    if (B | T | D | W) >> 31:
        _too_large(B, T, D, W)
    cp, n = _n_seq(cu_seqlens, B, x)
    given = out
    if out is None:
        out = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    ws = wp = wn = 0
    if cp:
        ws, wp, wn = _workspace(workspace, 256, x)
    st = L.gdn_conv_fwd(*_act(x, "x", (B, T, D), x), _flat(weight, "weight", (D, W), torch.float32, x), W,
                        _flat(bias, "bias", (D,), torch.float32, x),
                        _flat(initial_state, "initial_state", (n, W - 1, D), x.dtype, x), cp, n,
                        *_act(out, "out", (B, T, D), x), _flat(final_state, "final_state", (n, W - 1, D), x.dtype, x),
                        B, T, D, _code(x, "x"), SILU if silu else 0, wp, wn, _stream(x))
    if st:
        _fail(st, "gdn_conv_fwd")
    for t in (given, final_state):
        if t is not None:
            _count_version(t)
    return out


def gdn_conv_bwd(x, weight, dout, bias=None, initial_state=None, cu_seqlens=None, dfinal_state=None, silu=True,
                 workspace=None, stream=None):
    """Gradients of gdn_conv_fwd for L = sum(dout * out) + sum(dfinal_state *
    final_state): a dict of "dx" (x's type), "dweight" (fp32), with a bias
    "dbias" (fp32) and with an initial state "dinitial_state" (x's type)."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_conv_bwd(x, weight, dout, bias, initial_state, cu_seqlens, dfinal_state, silu, workspace)
    L = _lib or _load()
    B, T, D = x.shape
    _, W = weight.shape
    if (B | T | D | W) >> 31:
        _too_large(B, T, D, W)
    cp, n = _n_seq(cu_seqlens, B, x)
    f32 = dict(dtype=torch.float32, device=x.device)
    r = {"dx": torch.empty((B, T, D), dtype=x.dtype, device=x.device), "dweight": torch.empty((D, W), **f32)}
    bp = ip = 0
    if bias is not None:
        r["dbias"] = torch.empty(D, **f32)
        bp = r["dbias"].data_ptr()
    if initial_state is not None:
        r["dinitial_state"] = torch.empty((n, W - 1, D), dtype=x.dtype, device=x.device)
        ip = r["dinitial_state"].data_ptr()
    ws, wp, wn = _workspace(workspace, L.gdn_conv_bwd_workspace_size(B, T, D, W), x)
    st = L.gdn_conv_bwd(*_act(x, "x", (B, T, D), x), _flat(weight, "weight", (D, W), torch.float32, x), W,
                        _flat(bias, "bias", (D,), torch.float32, x),
                        _flat(initial_state, "initial_state", (n, W - 1, D), x.dtype, x), cp, n,
                        *_act(dout, "dout", (B, T, D), x),
                        _flat(dfinal_state, "dfinal_state", (n, W - 1, D), x.dtype, x), r["dx"].data_ptr(),
                        r["dweight"].data_ptr(), bp, ip, B, T, D, _code(x, "x"), SILU if silu else 0, wp, wn, _stream(x))
    if st:
        _fail(st, "gdn_conv_bwd")
    return r


def gdn_conv_step(x, state, weight, bias=None, slots=None, silu=True, out=None, stream=None):
    """One token of n requests: x (n, D); state (n_slots, W - 1, D) in x's
    type, the requests' windows, shifted by x in place; slots int32 (n), each
    request's row of state (distinct; a value outside [0, n_slots) marks a
    padding row, whose output is 0), or None for rows 0 .. n - 1. Returns out."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_conv_step(x, state, weight, bias, slots, silu, out)
    L = _lib or _load()
    n, D = x.shape
    (_, W), (pool, _, _) = weight.shape, state.shape
    if (n | D | W | pool) >> 31:
        _too_large(n, D, W, pool)
    given = out
    if out is None:
        out = torch.empty((n, D), dtype=x.dtype, device=x.device)
        at = out.data_ptr(), D
    else:
        at = _rows(out, "out", (n, D), x)
    st = L.gdn_conv_step(*_rows(x, "x", (n, D), x), _flat(weight, "weight", (D, W), torch.float32, x), W,
                         _flat(bias, "bias", (D,), torch.float32, x),
                         _flat(state, "state", (pool, W - 1, D), x.dtype, x),
                         _flat(slots, "slots", (n,), torch.int32, x), pool, *at, n, D,
                         _code(x, "x"), SILU if silu else 0, _stream(x))
    if st:
        _fail(st, "gdn_conv_step")
    if given is not None:
        _count_version(given)
    _count_version(state)
    return out


def gdn_ssm_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None, cu_seqlens=None,
                h_final=None, out=None, workspace=None, stream=None):
    """The selective scan: with delta = softplus(dt + dt_bias), per channel d
    and state n, h <- exp(delta A) h + delta x Bm and out = (sum_n Cm h + D x)
    * silu(z). x, dt, z (B, T, C); Bm, Cm (B, T, N); A (C, N), D, dt_bias (C)
    fp32; h0 / h_final (n_seq, C, N) fp32; cu_seqlens int32 (n_seq + 1) with
    B == 1. Returns out."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_ssm_fwd(x, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus, h0, cu_seqlens, h_final, out, workspace)
    L = _lib or _load()
    B, T, C = x.shape
    _, N = A.shape
    if (B | T | C | N) >> 31:
        _too_large(B, T, C, N)
    cp, n = _n_seq(cu_seqlens, B, x)
    given = out
    if out is None:
        out = torch.empty((B, T, C), dtype=x.dtype, device=x.device)
    ws, wp, wn = _workspace(workspace, L.gdn_ssm_workspace_size(B, T, C, N, n, 1 if cp else 0), x)
    f = torch.float32
    st = L.gdn_ssm_fwd(*_act(x, "x", (B, T, C), x), *_act(dt, "dt", (B, T, C), x), _flat(A, "A", (C, N), f, x),
                       *_act(Bm, "Bm", (B, T, N), x), *_act(Cm, "Cm", (B, T, N), x), _flat(D, "D", (C,), f, x),
                       *_act(z, "z", (B, T, C), x), _flat(dt_bias, "dt_bias", (C,), f, x),
                       _flat(h0, "h0", (n, C, N), f, x), cp, n, *_act(out, "out", (B, T, C), x),
                       _flat(h_final, "h_final", (n, C, N), f, x), B, T, C, N, _code(x, "x"),
                       SOFTPLUS if dt_softplus else 0, wp, wn, _stream(x))
    if st:
        _fail(st, "gdn_ssm_fwd")
    for t in (given, h_final):
        if t is not None:
            _count_version(t)
    return out


def gdn_ssm_bwd(x, dt, A, Bm, Cm, dout, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None, cu_seqlens=None,
                dh_final=None, workspace=None, stream=None):
    """Gradients of gdn_ssm_fwd for L = sum(dout * out) + sum(dh_final *
    h_final), the forward recomputed: a dict of dx, ddt, dBm, dCm (x's type),
    dA (fp32) and, for what was given, dD, dz, ddt_bias, dh0."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_ssm_bwd(x, dt, A, Bm, Cm, dout, D, z, dt_bias, dt_softplus, h0, cu_seqlens, dh_final, workspace)
    L = _lib or _load()
    B, T, C = x.shape
    _, N = A.shape
    if (B | T | C | N) >> 31:
        _too_large(B, T, C, N)
    cp, n = _n_seq(cu_seqlens, B, x)
    like, f32 = dict(dtype=x.dtype, device=x.device), dict(dtype=torch.float32, device=x.device)
    r = {"dx": torch.empty((B, T, C), **like), "ddt": torch.empty((B, T, C), **like), "dA": torch.empty((C, N), **f32),
         "dBm": torch.empty((B, T, N), **like), "dCm": torch.empty((B, T, N), **like)}
    if D is not None:
        r["dD"] = torch.empty(C, **f32)
    if z is not None:
        r["dz"] = torch.empty((B, T, C), **like)
    if dt_bias is not None:
        r["ddt_bias"] = torch.empty(C, **f32)
    if h0 is not None:
        r["dh0"] = torch.empty((n, C, N), **f32)
    ws, wp, wn = _workspace(workspace, L.gdn_ssm_bwd_workspace_size(B, T, C, N, n, 1 if cp else 0), x)
    f = torch.float32

    def ptr(k):
        return r[k].data_ptr() if k in r else 0

    st = L.gdn_ssm_bwd(*_act(x, "x", (B, T, C), x), *_act(dt, "dt", (B, T, C), x), _flat(A, "A", (C, N), f, x),
                       *_act(Bm, "Bm", (B, T, N), x), *_act(Cm, "Cm", (B, T, N), x), _flat(D, "D", (C,), f, x),
                       *_act(z, "z", (B, T, C), x), _flat(dt_bias, "dt_bias", (C,), f, x),
                       _flat(h0, "h0", (n, C, N), f, x), cp, n, *_act(dout, "dout", (B, T, C), x),
                       _flat(dh_final, "dh_final", (n, C, N), f, x), ptr("dx"), ptr("ddt"), ptr("dA"), ptr("dBm"),
                       ptr("dCm"), ptr("dD"), ptr("dz"), ptr("ddt_bias"), ptr("dh0"), B, T, C, N, _code(x, "x"),
                       SOFTPLUS if dt_softplus else 0, wp, wn, _stream(x))
    if st:
        _fail(st, "gdn_ssm_bwd")
    return r


def gdn_ssm_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, dt_softplus=True, slots=None, out=None,
                 stream=None):
    """One token of n requests of the scan: x, dt, z (n, C); Bm, Cm (n, N);
    state (n_slots, C, N) fp32, updated in place; slots as for gdn_conv_step.
    Returns out."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_ssm_step(x, dt, A, Bm, Cm, state, D, z, dt_bias, dt_softplus, slots, out)
    L = _lib or _load()
    n, C = x.shape
    (_, N), (pool, _, _) = A.shape, state.shape
    if (n | C | N | pool) >> 31:
        _too_large(n, C, N, pool)
    given = out
    if out is None:
        out = torch.empty((n, C), dtype=x.dtype, device=x.device)
        at = out.data_ptr(), C
    else:
        at = _rows(out, "out", (n, C), x)
    f = torch.float32
    st = L.gdn_ssm_step(*_rows(x, "x", (n, C), x), *_rows(dt, "dt", (n, C), x), _flat(A, "A", (C, N), f, x),
                        *_rows(Bm, "Bm", (n, N), x), *_rows(Cm, "Cm", (n, N), x), _flat(D, "D", (C,), f, x),
                        *_rows(z, "z", (n, C), x), _flat(dt_bias, "dt_bias", (C,), f, x),
                        _flat(state, "state", (pool, C, N), f, x), _flat(slots, "slots", (n,), torch.int32, x), pool,
                        *at, n, C, N, _code(x, "x"), SOFTPLUS if dt_softplus else 0,
                        _stream(x))
    if st:
        _fail(st, "gdn_ssm_step")
    if given is not None:
        _count_version(given)
    _count_version(state)
    return out
