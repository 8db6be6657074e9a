"""The operators around a mixer and the recurrence that can stand in its place
(include/gdn.h): rotary positions of q and k, the norms behind and in front of a
block with its gate and residual scale, and the gated linear recurrence, each
for prompts, single tokens and training.

q and k are (B, T, H, D), as the gated delta rule takes them; activations
(B, T, D) or, in the block norm, rows of any leading shape; single-token calls
of the recurrence (n, C). bf16 or fp32, any strides and a contiguous last
dimension. Parameters and states of the recurrence are contiguous fp32. Streams,
devices and errors are those of the state-space layer's operators.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import layer
from .layer import (_act, _as_rows, _code, _count_version, _elsewhere, _fail, _flat, _guard, _n_seq, _rows,
                    _too_large, _workspace)

LRU_TILE = 64  # tokens a checkpoint of the recurrence stands for
INTERLEAVED, INVERSE = 1, 2
_ACT = {None: 1, "sigmoid": 2, "silu": 3}
_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_EMPTY = (0, 0, 0, 0)


def bind(L):
    """Argument types of the library's entry points."""
    act, heads = [_P, _L, _L], [_P, _L, _L, _L]
    L.gdn_rotary.argtypes = (heads + [_I] + heads) * 2 + [_P, _P, _I, _L, _L, _L] + [_I] * 4 + [_F, _I, _I, _P]
    row = [_P, _L]
    gate, norms = row + [_I, _I], [_P, _P, _P, _F]
    L.gdn_block_norm_fwd.argtypes = (row + [_I]) * 2 + gate + norms + row * 2 + [_I, _I, _F, _P]
    L.gdn_block_norm_bwd_workspace_size.argtypes = [_I] * 3
    L.gdn_block_norm_bwd.argtypes = ((row + [_I]) * 2 + gate + row * 2 + norms + row * 3 + [_P] * 3 +
                                     [_I, _I, _F, _P, _Z, _P])
    scan = act * 3 + [_P] + act + [_F, _P, _P, _I] + act
    L.gdn_lru_fwd.argtypes = scan + [_P, _P] + [_I] * 4 + [_P, _Z, _P]
    L.gdn_lru_bwd_workspace_size.argtypes = [_I] * 4
    L.gdn_lru_bwd.argtypes = scan + [_P] * 8 + [_I] * 4 + [_P, _Z, _P]
    L.gdn_lru_step.argtypes = row * 3 + [_P] + row + [_F, _P, _P, _I] + row + [_I] * 3 + [_P]
    for name in ("gdn_block_norm_bwd_workspace_size", "gdn_lru_bwd_workspace_size"):
        getattr(L, name).restype = _Z
    for name in ("gdn_rotary", "gdn_block_norm_fwd", "gdn_block_norm_bwd", "gdn_lru_fwd", "gdn_lru_bwd", "gdn_lru_step"):
        getattr(L, name).restype = _I


# ---------------------------------------------------------------- rotary ---


def rotary_frequencies(rot, base=10000.0, factor=1.0, original_length=None, beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(inv_freq, scale) of gdn_rotary for rot turning channels: inv_freq[j] =
    base^(-2 j / rot) radians a position, fp64. factor > 1 stretches the
    positions a model was trained on: every frequency is divided by it, or,
    with original_length (the trained positions), only those that make fewer
    than beta_slow turns in it; those of more than beta_fast turns stay, a linear
    ramp over the turns lies between, and scale is 0.1 log(factor) + 1. (Code
    released with checkpoints may ramp over the channel's index between rounded
    bounds instead, which gives other frequencies: such a model's own table is
    then inv_freq.)"""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if not base > 0 or not factor >= 1:
        raise ValueError(f"base must be positive and factor at least 1, got {base} and {factor}")
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if original_length is None:
        f = f / factor
    else:
        if not beta_fast > beta_slow:
            raise ValueError(f"beta_fast must be above beta_slow, got {beta_fast} and {beta_slow}")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
        scale = 0.1 * math.log(factor) + 1.0
    return f.to(device), scale


def _heads(t, name, shape, like):
    """(pointer, strides over B, T and H) of a (B, T, H, D) tensor."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not like.dtype:
        _fail(3, f"{name} must be {like.dtype} as q is, got {t.dtype}")
    sb, st, sh, sd = t.stride()
    if (sd != 1 and shape[3] > 1) or t.get_device() != like.get_device():
        _fail(4, f"{name} must be on {like.device} with a contiguous last dimension")
    return t.data_ptr(), sb, st, sh


def gdn_rotary(q, inv_freq, k=None, positions=None, offset=0, interleaved=False, scale=1.0, inverse=False, out=None,
               k_out=None, stream=None):
    """Turns the first rot = 2 len(inv_freq) channels of every head of q (B, T,
    Hq, D) and k (B, T, Hk, D) by their token's position p: pair j, channels
    (j, j + rot / 2) or with interleaved (2 j, 2 j + 1), by the angle p
    inv_freq[j] (fp64 radians), times scale. positions: int32 or int64, (T) or
    (B, T), or None for offset + 0 .. T - 1. inverse turns back: the gradient's
    map. out and k_out may be q and k. Positions of several axes (a video's frame,
    row and column) are a call each, in place on the axis' slice of the channels.
    Returns the turned q, or (q, k)."""
    if stream is not None or _elsewhere(q):
        with _guard(q, stream):
            return gdn_rotary(q, inv_freq, k, positions, offset, interleaved, scale, inverse, out, k_out)
    L = layer._lib or layer._load()
    B, T, H, D = q.shape
    pairs = inv_freq.numel()
    if (B | T | H | D | pairs) >> 30:
        _too_large(B, T, H, D, 2 * pairs)
    given = (out, k_out)
    shape = q.shape
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
        qo = out.data_ptr(), T * H * D, H * D, D
    else:
        qo = _heads(out, "out", shape, q)
    ka = ko = _EMPTY
    Hk = 0
    if k is not None:
        _, _, Hk, _ = k.shape
        if Hk >> 31:
            _too_large(Hk)
        k_shape = (B, T, Hk, D)
        ka = _heads(k, "k", k_shape, q)
        if k_out is None:
            k_out = torch.empty(k_shape, dtype=q.dtype, device=q.device)
            ko = k_out.data_ptr(), T * Hk * D, Hk * D, D
        else:
            ko = _heads(k_out, "k_out", k_shape, q)
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    pp = bits = pb = pt = 0
    if positions is not None:
        if positions.dtype is torch.int32:
            bits = 32
        elif positions.dtype is torch.int64:
            bits = 64
        else:
            _fail(3, f"positions must be int32 or int64, got {positions.dtype}")
        if positions.shape == (B, T):
            pb, pt = positions.stride()
        elif positions.shape == (T,):
            pt = positions.stride(0)
        else:
            raise ValueError(f"positions must have shape {(B, T)} or {(T,)}, got {tuple(positions.shape)}")
        if positions.get_device() != q.get_device():
            _fail(4, f"positions must be on {q.device}")
        pp = positions.data_ptr()
    elif not -2**63 <= offset < 2**63 - 2**31:
        raise ValueError(f"offset must fit 64 bits, got {offset}")
    st = L.gdn_rotary(*_heads(q, "q", shape, q), H, *qo, *ka, Hk, *ko,
                      _flat(inv_freq, "inv_freq", (pairs,), torch.float64, q), pp, bits, pb, pt, offset, B, T, D, 2 * pairs,
                      scale, _code(q, "q"), (INTERLEAVED if interleaved else 0) | (INVERSE if inverse else 0), layer._stream(q))
    if st:
        _fail(st, "gdn_rotary")
    for t in given:
        if t is not None:
            _count_version(t)
    return out if k is None else (out, k_out)


# ------------------------------------------------------------ block norm ---


def _lines(t, name, shape, like):
    """(pointer, row stride) of rows of any leading shape; zeros for None."""
    if t is None:
        return 0, 0
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is like.dtype and t.get_device() == like.get_device() and t.is_contiguous():
        return t.data_ptr(), shape[-1]
    rows = _as_rows(t, name)
    return _rows(rows, name, rows.shape, like)


def _sizes(y):
    """Rows and channels of y."""
    shape = y.shape
    if not shape:
        raise ValueError("y must have at least one dimension")
    D = shape[-1]
    R = y.numel() // D if D else 0
    if (R | D) >> 31:
        _too_large(R, D)
    return shape, R, D


def _gate(gate, gate_act, y):
    """(pointer, row stride, rows that share one, act) of the gate: y's shape,
    or (B, 1, D) for y (B, T, D)."""
    if gate is None:
        if gate_act is not None:
            raise ValueError("gate_act is given without a gate")
        return 0, 0, 1, 0
    if gate_act not in _ACT:
        raise ValueError(f"gate_act must be None, 'sigmoid' or 'silu', got {gate_act!r}")
    shape = y.shape
    if gate.shape == shape:
        return *_lines(gate, "gate", shape, y), 1, _ACT[gate_act]
    if len(shape) == 3 and gate.shape == (shape[0], 1, shape[2]):
        return *_lines(gate, "gate", gate.shape, y), max(shape[1], 1), _ACT[gate_act]
    raise ValueError(f"gate must have shape {tuple(shape)}, or one row a sequence of a (B, T, D) y, got {tuple(gate.shape)}")


def gdn_block_norm_fwd(y, residual, post_weight=None, pre_weight=None, gate=None, gate_act=None, scale=None, alpha=1.0,
                       eps=1e-6, residual_out=None, out=None, stream=None):
    """What stands between two blocks, over the last dimension (D): the norm of
    a block's output y, its gate and residual scale, the residual's addition
    and the norm in front of the next block,
      s = residual + alpha scale act(gate) (y post_weight / sqrt(mean(y^2) + eps)),
      out = s pre_weight / sqrt(mean(s^2) + eps),
    where a weight of None leaves its norm out (post: y as it is; pre: no out).
    gate: y's shape, or (B, 1, D) for a y of (B, T, D), in y's type; gate_act
    None (the gate itself), "sigmoid" or "silu". scale (D) fp32. Returns a dict
    of "residual": s in the residual's type (in residual_out, which may be the
    residual), and with pre_weight "out" in y's type."""
    if stream is not None or _elsewhere(y):
        with _guard(y, stream):
            return gdn_block_norm_fwd(y, residual, post_weight, pre_weight, gate, gate_act, scale, alpha, eps, residual_out,
                                      out)
    L = layer._lib or layer._load()
    shape, R, D = _sizes(y)
    if post_weight is None and pre_weight is None:
        raise ValueError("at least one of post_weight and pre_weight must be given")
    at = _lines(residual, "residual", shape, residual)
    if residual.get_device() != y.get_device():
        _fail(4, f"residual must be on {y.device}")
    given = (residual_out, out)
    if residual_out is None:
        residual_out = torch.empty(shape, dtype=residual.dtype, device=y.device)
        ro = residual_out.data_ptr(), D
    else:
        ro = _lines(residual_out, "residual_out", shape, residual)
    res = {"residual": residual_out}
    o = 0, 0
    if pre_weight is not None:
        if out is None:
            out = torch.empty(shape, dtype=y.dtype, device=y.device)
            o = out.data_ptr(), D
        else:
            o = _lines(out, "out", shape, y)
        res["out"] = out
    elif out is not None:
        raise ValueError("out is given without pre_weight")
    f = torch.float32
    st = L.gdn_block_norm_fwd(*_lines(y, "y", shape, y), _code(y, "y"), *at, _code(residual, "residual"), *_gate(gate, gate_act, y),
                              _flat(post_weight, "post_weight", (D,), f, y), _flat(pre_weight, "pre_weight", (D,), f, y),
                              _flat(scale, "scale", (D,), f, y), alpha, *ro, *o, R, D, eps, layer._stream(y))
    if st:
        _fail(st, "gdn_block_norm_fwd")
    for t in given:
        if t is not None:
            _count_version(t)
    return res


def gdn_block_norm_bwd(y, s, dout=None, dres=None, post_weight=None, pre_weight=None, gate=None, gate_act=None, scale=None,
                       alpha=1.0, eps=1e-6, workspace=None, stream=None):
    """Gradients of gdn_block_norm_fwd at the sum s that it returned
    ("residual"), for dout (y's type, with pre_weight) and the stream's own
    gradient dres (s's type; with pre_weight it may be None): a dict of "dy",
    "dresidual" and, for what was given, "dgate" (the gate's shape and type),
    "dpost_weight", "dpre_weight" and "dscale" (fp32)."""
    if stream is not None or _elsewhere(y):
        with _guard(y, stream):
            return gdn_block_norm_bwd(y, s, dout, dres, post_weight, pre_weight, gate, gate_act, scale, alpha, eps, workspace)
    L = layer._lib or layer._load()
    shape, R, D = _sizes(y)
    if post_weight is None and pre_weight is None:
        raise ValueError("at least one of post_weight and pre_weight must be given")
    if (dout is None) != (pre_weight is None):
        raise ValueError("dout goes with pre_weight")
    if dout is None and dres is None:
        raise ValueError("without pre_weight dres must be given")
    s_at = _lines(s, "s", shape, s)
    if s.get_device() != y.get_device():
        _fail(4, f"s must be on {y.device}")
    f32 = dict(dtype=torch.float32, device=y.device)
    gp, gs, each, act = _gate(gate, gate_act, y)
    r = {"dy": torch.empty(y.shape, dtype=y.dtype, device=y.device),
         "dresidual": torch.empty(s.shape, dtype=s.dtype, device=s.device)}
    dg = 0
    if gate is not None:
        r["dgate"] = (torch.empty if R else torch.zeros)(gate.shape, dtype=y.dtype, device=y.device)
        dg = r["dgate"].data_ptr()
    for name, w in (("dpost_weight", post_weight), ("dpre_weight", pre_weight), ("dscale", scale)):
        if w is not None:
            r[name] = torch.empty(D, **f32)

    def ptr(k):
        return r[k].data_ptr() if k in r else 0

    f = torch.float32
    ws, wp, wn = _workspace(workspace, L.gdn_block_norm_bwd_workspace_size(R, D, each), y)
    st = L.gdn_block_norm_bwd(*_lines(y, "y", shape, y), _code(y, "y"), *s_at, _code(s, "s"), gp, gs, each, act,
                              *_lines(dout, "dout", shape, y), *_lines(dres, "dres", shape, s),
                              _flat(post_weight, "post_weight", (D,), f, y), _flat(pre_weight, "pre_weight", (D,), f, y),
                              _flat(scale, "scale", (D,), f, y), alpha, r["dy"].data_ptr(), D, r["dresidual"].data_ptr(), D,
                              dg, D, ptr("dpost_weight"), ptr("dpre_weight"), ptr("dscale"), R, D, eps, wp, wn, layer._stream(y))
    if st:
        _fail(st, "gdn_block_norm_bwd")
    return r


# ------------------------------------------------------ gated recurrence ---


def gdn_lru_fwd(x, r, i, lam, z=None, c=8.0, h0=None, cu_seqlens=None, h_final=None, checkpoints=None, out=None,
                workspace=None, stream=None):
    """The gated linear recurrence: with u = c softplus(lam) sigmoid(r) and a =
    exp(-u), per channel h <- a h + sqrt(1 - a^2) sigmoid(i) x and out = h
    silu(z) (h without z). Every token's input takes the root, a sequence's first
    too: for a model that leaves it out there, that token's x is given divided by
    it; for another gate than SiLU, z is left out. x, r, i, z (B, T, C); lam (C) fp32; h0 / h_final
    (n_seq, C) fp32; cu_seqlens int32 (n_seq + 1) with B == 1; checkpoints (B,
    ceil(T / LRU_TILE), C) fp32, written: the states gdn_lru_bwd starts its
    tiles from. out may be x, r, i or z. workspace: 256 bytes, whose error word
    (gdn_last_device_error) tells of malformed cu_seqlens and of a wait that ran
    out, which leaves NaN. Returns out."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_lru_fwd(x, r, i, lam, z, c, h0, cu_seqlens, h_final, checkpoints, out, workspace)
    L = layer._lib or layer._load()
    B, T, C = shape = x.shape
    if (B | T | C) >> 31:
        _too_large(B, T, C)
    cp, n = _n_seq(cu_seqlens, B, x)
    given = out
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        at = out.data_ptr(), T * C, C
    else:
        at = _act(out, "out", shape, x)
    ws = wp = wn = 0
    if cp or workspace is not None:
        ws, wp, wn = _workspace(workspace, 256, x)
    f = torch.float32
    st = L.gdn_lru_fwd(*_act(x, "x", shape, x), *_act(r, "r", shape, x), *_act(i, "i", shape, x), _flat(lam, "lam", (C,), f, x),
                       *_act(z, "z", shape, x), c, _flat(h0, "h0", (n, C), f, x), cp, n, *at,
                       _flat(h_final, "h_final", (n, C), f, x),
                       _flat(checkpoints, "checkpoints", (B, (T + LRU_TILE - 1) // LRU_TILE, C), f, x), B, T, C,
                       _code(x, "x"), wp, wn, layer._stream(x))
    if st:
        _fail(st, "gdn_lru_fwd")
    for t in (given, h_final, checkpoints):
        if t is not None:
            _count_version(t)
    return out


def gdn_lru_bwd(x, r, i, lam, dout, z=None, c=8.0, h0=None, cu_seqlens=None, dh_final=None, checkpoints=None,
                workspace=None, stream=None):
    """Gradients of gdn_lru_fwd for L = sum(dout * out) + sum(dh_final *
    h_final): a dict of dx, dr, di (x's type), dlam (fp32) and, for what was
    given, dz and dh0. checkpoints: what the forward wrote for the same
    inputs; without them the states are formed again."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_lru_bwd(x, r, i, lam, dout, z, c, h0, cu_seqlens, dh_final, checkpoints, workspace)
    L = layer._lib or layer._load()
    B, T, C = shape = x.shape
    if (B | T | C) >> 31:
        _too_large(B, T, C)
    cp, n = _n_seq(cu_seqlens, B, x)
    like, f32 = dict(dtype=x.dtype, device=x.device), dict(dtype=torch.float32, device=x.device)
    g = {k: torch.empty(shape, **like) for k in (("dx", "dr", "di") if z is None else ("dx", "dr", "di", "dz"))}
    g["dlam"] = torch.empty(C, **f32)
    if h0 is not None:
        g["dh0"] = torch.empty((n, C), **f32)

    def ptr(k):
        return g[k].data_ptr() if k in g else 0

    f = torch.float32
    ws, wp, wn = _workspace(workspace, L.gdn_lru_bwd_workspace_size(B, T, C, checkpoints is not None), x)
    st = L.gdn_lru_bwd(*_act(x, "x", shape, x), *_act(r, "r", shape, x), *_act(i, "i", shape, x), _flat(lam, "lam", (C,), f, x),
                       *_act(z, "z", shape, x), c, _flat(h0, "h0", (n, C), f, x), cp, n, *_act(dout, "dout", shape, x),
                       _flat(dh_final, "dh_final", (n, C), f, x),
                       _flat(checkpoints, "checkpoints", (B, (T + LRU_TILE - 1) // LRU_TILE, C), f, x),
                       ptr("dx"), ptr("dr"), ptr("di"), ptr("dlam"), ptr("dz"), ptr("dh0"), B, T, C, _code(x, "x"), wp, wn,
                       layer._stream(x))
    if st:
        _fail(st, "gdn_lru_bwd")
    return g


def gdn_lru_step(x, r, i, lam, state, z=None, c=8.0, slots=None, out=None, stream=None):
    """One token of n requests of the recurrence: x, r, i, z (n, C); state
    (n_slots, C) fp32, updated in place; slots as for gdn_conv_step. Returns
    out."""
    if stream is not None or _elsewhere(x):
        with _guard(x, stream):
            return gdn_lru_step(x, r, i, lam, state, z, c, slots, out)
    L = layer._lib or layer._load()
    n, C = shape = x.shape
    pool, _ = state.shape
    if (n | C | pool) >> 31:
        _too_large(n, C, pool)
    given = out
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        at = out.data_ptr(), C
    else:
        at = _rows(out, "out", shape, x)
    f = torch.float32
    st = L.gdn_lru_step(*_rows(x, "x", shape, x), *_rows(r, "r", shape, x), *_rows(i, "i", shape, x),
                        _flat(lam, "lam", (C,), f, x), *_rows(z, "z", shape, x), c, _flat(state, "state", (pool, C), f, x),
                        _flat(slots, "slots", (n,), torch.int32, x), pool, *at, n, C, _code(x, "x"), layer._stream(x))
    if st:
        _fail(st, "gdn_lru_step")
    if given is not None:
        _count_version(given)
    _count_version(state)
    return out
