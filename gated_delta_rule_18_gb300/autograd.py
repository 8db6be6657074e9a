"""torch.autograd functions over the library's forward and backward calls.

Each function's forward runs the CUDA forward through the C ABI; its
backward runs the matching gradient kernels (gdn_chunk_bwd, gdn_frame_bwd,
gdn_merge_bwd, gdn_prep_bwd; of the state-space layer gdn_rmsnorm_bwd,
gdn_conv_bwd, gdn_ssm_bwd; around a mixer gdn_rotary, gdn_block_norm_bwd,
gdn_lru_bwd).
Nothing here computes on its own: the wrappers marshal tensors and sum the
two directions' gradients.

The gradient kernels take the upstream gradient of the output in the
inputs' precision: for bf16 inputs an fp32 upstream gradient is rounded to
bf16 first; fp32 inputs (the fp32 path) keep it in fp32.

A backward pass is captured into a CUDA graph only while no eager graph of the
same leaves is alive: torch's nodes that accumulate their gradients would wait
on the eager graph's stream amid the capture, which ends the process.
"""
from __future__ import annotations

import functools

import torch

from . import (PREP_RELU, PREP_RMS, gdn_chunk_bwd, gdn_chunk_fwd, gdn_chunk_fwd_bidir, gdn_frame_bwd,
               gdn_frame_fwd, gdn_merge, gdn_merge_bwd, gdn_prep, gdn_prep_bwd)
from .block import (LRU_TILE, gdn_block_norm_bwd, gdn_block_norm_fwd, gdn_lru_bwd, gdn_lru_fwd, gdn_rotary)
from .layer import (gdn_conv_bwd, gdn_conv_fwd, gdn_rmsnorm_bwd, gdn_rmsnorm_fwd, gdn_ssm_bwd, gdn_ssm_fwd)


def _bf16(t):
    return None if t is None else t.to(torch.bfloat16).contiguous()


class _ChunkGDR(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, g, gk, h0, cu_seqlens, reverse, qk_l2norm, final_state):
        n_seq = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        H, K, V = q.shape[2], q.shape[3], v.shape[3]
        hf = (torch.empty((n_seq, H, K, V), dtype=torch.float32, device=q.device)
              if final_state else None)
        o = gdn_chunk_fwd(q, k, v, beta, g=g, gk=gk, h0=h0, cu_seqlens=cu_seqlens, h_final=hf,
                          reverse=reverse, qk_l2norm=qk_l2norm)
        ctx.save_for_backward(q, k, v, beta, g, gk, h0, cu_seqlens)
        ctx.reverse, ctx.qk_l2norm = reverse, qk_l2norm
        return o, hf

    @staticmethod
    def backward(ctx, do, dhf):
        q, k, v, beta, g, gk, h0, cu_seqlens = ctx.saved_tensors
        want_h0 = h0 is not None and ctx.needs_input_grad[6]
        do = do.float().contiguous() if q.dtype == torch.float32 else _bf16(do)
        res = gdn_chunk_bwd(q, k, v, beta, g, do, h0=h0,
                            dh_final=None if dhf is None else dhf.float().contiguous(),
                            reverse=ctx.reverse, qk_l2norm=ctx.qk_l2norm, with_dh0=want_h0,
                            gk=gk, cu_seqlens=cu_seqlens)
        dg = res["dg"]
        return (res["dq"].to(q.dtype), res["dk"].to(k.dtype), res["dv"].to(v.dtype), res["dbeta"],
                None if gk is not None else dg, dg if gk is not None else None, res.get("dh0"),
                None, None, None, None)


def chunk_gated_delta_rule(q, k, v, beta, g=None, gk=None, initial_state=None,
                           output_final_state=False, cu_seqlens=None, reverse=False,
                           use_qk_l2norm=True):
    """One direction of the chunked gated delta rule, differentiable in q, k,
    v, beta, g (or the per-key gk) and initial_state. Shapes and meanings as
    gdn_chunk_fwd: q, k (B, T, H, K), v (B, T, H, V) bf16 (or all fp32: the
    fp32 path and its backward); beta, g (B, T, H)
    fp32; gk (B, T, H, K) fp32; initial_state (n_seq, H, K, V) fp32;
    cu_seqlens int32 (n_seq + 1) with B == 1. use_qk_l2norm normalises q and
    k per (token, head) inside the kernels. Returns (o, final_state or None)."""
    return _ChunkGDR.apply(q, k, v, beta, g, gk, initial_state, cu_seqlens, bool(reverse),
                           bool(use_qk_l2norm), bool(output_final_state))


class _BidirMerge(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, g, gk, g_bwd, beta_bwd, gate, cu_seqlens, eps, qk_l2norm):
        B, T, H = q.shape[0], q.shape[1], q.shape[2]
        den = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
        num = gdn_chunk_fwd_bidir(q, k, v, beta, g=g, gk=gk, g_bwd=g_bwd, beta_bwd=beta_bwd,
                                  cu_seqlens=cu_seqlens, den=den, qk_l2norm=qk_l2norm)
        out = gdn_merge(num, den, gate=gate, eps=eps)
        ctx.save_for_backward(q, k, v, beta, g, gk, g_bwd, beta_bwd, gate, cu_seqlens, num, den)
        ctx.eps, ctx.qk_l2norm = eps, qk_l2norm
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, beta, g, gk, g_bwd, beta_bwd, gate, cu_seqlens, num, den = ctx.saved_tensors
        m = gdn_merge_bwd(num, den, dout.float().contiguous(), gate=gate, eps=ctx.eps)
        dnum, dden = _bf16(m["dnum"]), m["dden"]
        fwd = gdn_chunk_bwd(q, k, v, beta, g, dnum, qk_l2norm=ctx.qk_l2norm, with_dh0=False,
                            cu_seqlens=cu_seqlens, dden=dden, gk=gk)
        rev = gdn_chunk_bwd(q, k, v, beta if beta_bwd is None else beta_bwd,
                            g if g_bwd is None else g_bwd, dnum, reverse=True,
                            qk_l2norm=ctx.qk_l2norm, with_dh0=False, cu_seqlens=cu_seqlens,
                            dden=dden, gk=gk)
        dq = (fwd["dq"] + rev["dq"]).to(q.dtype)
        dk = (fwd["dk"] + rev["dk"]).to(k.dtype)
        dv = (fwd["dv"] + rev["dv"]).to(v.dtype)
        dbeta = fwd["dbeta"] if beta_bwd is not None else fwd["dbeta"] + rev["dbeta"]
        dbeta_bwd = rev["dbeta"] if beta_bwd is not None else None
        dg = fwd["dg"] if g_bwd is not None else fwd["dg"] + rev["dg"]
        dg_bwd = rev["dg"] if g_bwd is not None else None
        dgate = m.get("dgate")
        return (dq, dk, dv, dbeta, None if gk is not None else dg, dg if gk is not None else None,
                dg_bwd, dbeta_bwd, None if dgate is None else dgate.to(gate.dtype), None, None, None)


def bidirectional_gated_delta_rule(q, k, v, beta, g=None, g_bwd=None, beta_bwd=None, gate=None,
                                   cu_seqlens=None, eps=1e-6, use_qk_l2norm=True, gk=None):
    """The bidirectional form with its denominator and merge (SANA
    `fused_gdn.py` page, `fused_bigdn_func`): out = (num_fwd + num_bwd) /
    (den_fwd + den_bwd + eps) * silu(gate), differentiable in q, k, v, beta,
    g (or the per-key gk), g_bwd, beta_bwd and gate. g_bwd / beta_bwd: the
    reverse direction's own log gates / betas (the chunk-causal form; g_bwd
    with a scalar gate only), or None for g / beta."""
    return _BidirMerge.apply(q, k, v, beta, g, gk, g_bwd, beta_bwd, gate, cu_seqlens, float(eps),
                             bool(use_qk_l2norm))


class _FrameVideo(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, g_frame, gate, frame, eps, prep_eps):
        K = q.shape[3]
        B, T, H = q.shape[0], q.shape[1], q.shape[2]
        mode = PREP_RMS | PREP_RELU
        qn = gdn_prep(q, mode=mode, scale=1.0, eps=prep_eps)
        kn = gdn_prep(k, mode=mode, scale=K ** -0.5, eps=prep_eps)
        den = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
        num = gdn_frame_fwd(qn, kn, v, beta, g_frame, frame, den=den, direction=2)
        out = gdn_merge(num, den, gate=gate, eps=eps)
        ctx.save_for_backward(q, k, qn, kn, v, beta, g_frame, gate, num, den)
        ctx.frame, ctx.eps, ctx.prep_eps = frame, eps, prep_eps
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, qn, kn, v, beta, g_frame, gate, num, den = ctx.saved_tensors
        K = q.shape[3]
        m = gdn_merge_bwd(num, den, dout.float().contiguous(), gate=gate, eps=ctx.eps)
        r = gdn_frame_bwd(qn, kn, v, beta, g_frame, ctx.frame, _bf16(m["dnum"]), dden=m["dden"],
                          direction=2)
        mode = PREP_RMS | PREP_RELU
        dq = gdn_prep_bwd(q, r["dq"], mode=mode, scale=1.0, eps=ctx.prep_eps)
        dk = gdn_prep_bwd(k, r["dk"], mode=mode, scale=K ** -0.5, eps=ctx.prep_eps)
        dgate = m.get("dgate")
        return (dq.to(q.dtype), dk.to(k.dtype), r["dv"].to(v.dtype), r["dbeta"], r["dg_frame"],
                None if dgate is None else dgate.to(gate.dtype), None, None, None)


def frame_video_gated_delta_rule(q, k, v, beta, g_frame, frame, gate=None, eps=1e-6, prep_eps=1e-5):
    """The video form of the SANA pages, differentiable end to end: q and k
    through the full-channel RMSNorm and ReLU (k scaled by K^-1/2), the
    frame-causal rule in both directions with its denominator (frames of
    `frame` tokens, one log decay per frame and head, g_frame (B, T / frame,
    H)), and the merge num / (den + eps) * silu(gate). q, k, v (B, T, H, D)
    bf16 (views of an interleaved qkv tensor work); beta (B, T, H) fp32."""
    return _FrameVideo.apply(q, k, v, beta, g_frame, gate, int(frame), float(eps), float(prep_eps))


class _Once(torch.autograd.Function):
    """Passes a backward's results on; to differentiate them again raises."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of the layer's and the block's operators are not differentiable")


def _once(backward):
    # (torch's once_differentiable guards the path over the upstream gradients
    # only: a second derivative of y.sum() would go by it)
    @functools.wraps(backward)
    def call(ctx, *grads):
        with torch.no_grad():
            r = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return r
        return _Once.apply(torch.ones((), requires_grad=True), *r)
    return call


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        r = gdn_rmsnorm_fwd(x, weight, residual=residual, eps=eps)
        s = r.get("residual", x)
        ctx.save_for_backward(s, weight)
        ctx.eps, ctx.with_residual = eps, residual is not None
        return r["out"], s if residual is not None else None

    @staticmethod
    @_once
    def backward(ctx, dy, ds):
        s, weight = ctx.saved_tensors
        r = gdn_rmsnorm_bwd(s, weight, dy.contiguous(), dres=None if ds is None else ds.to(s.dtype).contiguous(),
                            eps=ctx.eps)
        return r["dx"].to(dy.dtype), r["dweight"], r["dx"] if ctx.with_residual else None, None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """The norm in front of a mixer, differentiable in x, weight (fp32) and
    residual: (y, s) with s = x + residual in the residual's type, the
    residual stream that goes on (None without a residual). The gradient takes
    s as stored."""
    return _RMSNorm.apply(x, weight, residual, float(eps))


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, silu, output_final_state):
        n_seq = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        final = (torch.empty((n_seq, weight.shape[1] - 1, x.shape[2]), dtype=x.dtype, device=x.device)
                 if output_final_state else None)
        y = gdn_conv_fwd(x, weight, bias=bias, initial_state=initial_state, cu_seqlens=cu_seqlens, final_state=final,
                         silu=silu)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu = silu
        return y, final

    @staticmethod
    @_once
    def backward(ctx, dy, dfinal):
        x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
        r = gdn_conv_bwd(x, weight, dy.contiguous(), bias=bias, initial_state=initial_state, cu_seqlens=cu_seqlens,
                         dfinal_state=None if dfinal is None else dfinal.contiguous(), silu=ctx.silu)
        return r["dx"], r["dweight"], r.get("dbias"), r.get("dinitial_state"), None, None, None


def causal_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, silu=True, output_final_state=False):
    """The short causal convolution (gdn_conv_fwd), differentiable in x,
    weight, bias and initial_state. Returns (y, final_state or None)."""
    return _CausalConv.apply(x, weight, bias, initial_state, cu_seqlens, bool(silu), bool(output_final_state))


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, Bm, Cm, D, z, dt_bias, h0, cu_seqlens, dt_softplus, output_final_state):
        n_seq = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        final = (torch.empty((n_seq,) + tuple(A.shape), dtype=torch.float32, device=x.device)
                 if output_final_state else None)
        y = gdn_ssm_fwd(x, dt, A, Bm, Cm, D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus, h0=h0,
                        cu_seqlens=cu_seqlens, h_final=final)
        ctx.save_for_backward(x, dt, A, Bm, Cm, D, z, dt_bias, h0, cu_seqlens)
        ctx.dt_softplus = dt_softplus
        return y, final

    @staticmethod
    @_once
    def backward(ctx, dy, dfinal):
        x, dt, A, Bm, Cm, D, z, dt_bias, h0, cu_seqlens = ctx.saved_tensors
        r = gdn_ssm_bwd(x, dt, A, Bm, Cm, dy.contiguous(), D=D, z=z, dt_bias=dt_bias, dt_softplus=ctx.dt_softplus,
                        h0=h0, cu_seqlens=cu_seqlens, dh_final=None if dfinal is None else dfinal.contiguous())
        return (r["dx"], r["ddt"], r["dA"], r["dBm"], r["dCm"], r.get("dD"), r.get("dz"), r.get("ddt_bias"),
                r.get("dh0"), None, None, None)


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                   dt_softplus=True, output_final_state=False):
    """The selective state-space scan (gdn_ssm_fwd), differentiable in every
    tensor but cu_seqlens. Returns (y, final_state or None)."""
    return _SelectiveScan.apply(x, dt, A, Bm, Cm, D, z, dt_bias, initial_state, cu_seqlens, bool(dt_softplus),
                                bool(output_final_state))


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, inv_freq, positions, offset, interleaved, scale):
        ctx.save_for_backward(inv_freq, positions)
        ctx.how = offset, interleaved, scale
        r = gdn_rotary(q, inv_freq, k=k, positions=positions, offset=offset, interleaved=interleaved, scale=scale)
        return (r, None) if k is None else r

    @staticmethod
    @_once
    def backward(ctx, dq, dk):
        inv_freq, positions = ctx.saved_tensors
        offset, interleaved, scale = ctx.how
        r = gdn_rotary(dq.contiguous(), inv_freq, k=None if dk is None else dk.contiguous(), positions=positions,
                       offset=offset, interleaved=interleaved, scale=scale, inverse=True)
        dq, dk = (r, None) if dk is None else r
        return dq, dk, None, None, None, None, None


def rotary(q, inv_freq, k=None, positions=None, offset=0, interleaved=False, scale=1.0):
    """Rotary positions (gdn_rotary), differentiable in q and k. Returns the
    turned q, or (q, k)."""
    q, k = _Rotary.apply(q, k, inv_freq, positions, int(offset), bool(interleaved), float(scale))
    return q if k is None else (q, k)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, post, pre, gate, scale, gate_act, alpha, eps):
        r = gdn_block_norm_fwd(y, residual, post_weight=post, pre_weight=pre, gate=gate, gate_act=gate_act, scale=scale,
                               alpha=alpha, eps=eps)
        ctx.save_for_backward(y, r["residual"], post, pre, gate, scale)
        ctx.how = gate_act, alpha, eps
        return r.get("out"), r["residual"]

    @staticmethod
    @_once
    def backward(ctx, dout, dres):
        y, s, post, pre, gate, scale = ctx.saved_tensors
        gate_act, alpha, eps = ctx.how
        r = gdn_block_norm_bwd(y, s, dout=None if pre is None else dout.contiguous(), dres=dres.to(s.dtype).contiguous(),
                               post_weight=post, pre_weight=pre, gate=gate, gate_act=gate_act, scale=scale, alpha=alpha,
                               eps=eps)
        return (r["dy"], r["dresidual"], r.get("dpost_weight"), r.get("dpre_weight"), r.get("dgate"), r.get("dscale"), None,
                None, None)


def block_norm(y, residual, post_weight=None, pre_weight=None, gate=None, gate_act=None, scale=None, alpha=1.0, eps=1e-6):
    """What stands between two blocks (gdn_block_norm_fwd), differentiable in
    every tensor: (out, s), the normed input of the next block (None without
    pre_weight) and the residual stream that goes on. The gradient takes s as
    stored."""
    return _BlockNorm.apply(y, residual, post_weight, pre_weight, gate, scale, gate_act, float(alpha), float(eps))


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, lam, z, h0, cu_seqlens, c, output_final_state):
        B, T, C = x.shape
        f32 = dict(dtype=torch.float32, device=x.device)
        n_seq = B if cu_seqlens is None else cu_seqlens.numel() - 1
        final = torch.empty((n_seq, C), **f32) if output_final_state else None
        saved = torch.empty((B, (T + LRU_TILE - 1) // LRU_TILE, C), **f32)
        y = gdn_lru_fwd(x, r, i, lam, z=z, c=c, h0=h0, cu_seqlens=cu_seqlens, h_final=final, checkpoints=saved)
        ctx.save_for_backward(x, r, i, lam, z, h0, cu_seqlens, saved)
        ctx.c = c
        return y, final

    @staticmethod
    @_once
    def backward(ctx, dy, dfinal):
        x, r, i, lam, z, h0, cu_seqlens, saved = ctx.saved_tensors
        g = gdn_lru_bwd(x, r, i, lam, dy.contiguous(), z=z, c=ctx.c, h0=h0, cu_seqlens=cu_seqlens,
                        dh_final=None if dfinal is None else dfinal.contiguous(), checkpoints=saved)
        return g["dx"], g["dr"], g["di"], g["dlam"], g.get("dz"), g.get("dh0"), None, None, None


def gated_recurrence(x, r, i, lam, z=None, initial_state=None, cu_seqlens=None, c=8.0, output_final_state=False):
    """The gated linear recurrence (gdn_lru_fwd), differentiable in every tensor
    but cu_seqlens. Returns (y, final_state or None)."""
    return _GatedRecurrence.apply(x, r, i, lam, z, initial_state, cu_seqlens, float(c), bool(output_final_state))
