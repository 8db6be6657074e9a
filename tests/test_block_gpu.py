"""The block's operators on the GPU against plain fp64 forms.

Tolerances, as max|got - ref| / max|ref|, fixed from the arithmetic:
  * bf16 results: one rounding, at most half a step, eps / 2 = 2^-8 of the
    value, beside an fp32 error far below it: 2^-8 (1 + 2^-6).
  * rotary, fp32: the angle is right to 2^-25 of half a turn (pi 2^-25 = 1e-7),
    its cosine and sine to 2 units in the last place (2^-23), and each result
    is two products and a sum (3 half steps of 2^-24): 4e-7, of the largest
    value of a pair, which max|ref| bounds up to sqrt(2): 6e-7.
  * block norm, fp32: sums of at most D terms with errors of a few 2^-24, in
    chains of at most a few thousand: 2e-5.
  * recurrence, fp32: a step multiplies the state by a with a relative error of
    2^-22 (the exponential) and a few 2^-24, and errors of one sign add up over
    min(T, 1 / (1 - a)) steps; T <= 600 where fp32 is compared: 600 2^-22 =
    1.4e-4. Its gradients multiply two such walks: 2.8e-4.
  * central differences of a loss of fp32 outputs with step h along a random
    direction: the third derivative gives h^2 / 6 of the loss's scale and the
    outputs' rounding 2^-22 / h of it; h = 2^-7: 1e-5 + 3e-5, and the loss is
    at most some tens of times the derivative's size: 2e-3.
"""
import math

import pytest
import torch

import gated_delta_rule_18_gb300 as gdn
from gated_delta_rule_18_gb300 import autograd as gdr, layer
from test_layer_gpu import BF, DEV, F32, F64, built, cu_of, dev, f64, randn, rel, spans, strided  # noqa: F401

pytestmark = pytest.mark.gpu

TOL_BF = 2.0**-8 * (1 + 2.0**-6)
TOL_ROT, TOL_NORM, TOL_LRU, TOL_LRU_BWD, TOL_DIFF = 6e-7, 2e-5, 1.4e-4, 2.8e-4, 2e-3


def tol(dtype, f32):
    return TOL_BF if dtype == BF else f32


# ---------------------------------------------------------------- rotary ---


def freqs(rot, base=10000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=F64) / rot)


def ref_rotary(x, pos, f, interleaved, scale, inverse=False):
    """pos (B, T) integers, exactly reduced: whole turns go first."""
    x, rot = f64(x).clone(), 2 * f.numel()
    turn = torch.tensor([[[math.fmod(int(p) * float(w) / (2 * math.pi), 1.0) for w in f] for p in row] for row in pos.tolist()],
                        dtype=F64).reshape(*pos.shape, 1, f.numel())
    ang = 2 * math.pi * turn * (-1 if inverse else 1)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = scale * (u * ang.cos() - v * ang.sin()), scale * (v * ang.cos() + u * ang.sin())
    return x


@pytest.mark.parametrize("B,T,Hq,Hk,D,rot", [
    (1, 1, 1, 1, 2, 2), (1, 1, 4, 2, 64, 64), (3, 5, 2, 1, 128, 128), (2, 7, 3, 3, 112, 64), (2, 300, 4, 1, 96, 32), (5, 1, 32, 8, 128, 64),
    (1, 33, 2, 2, 7, 4), (2, 3, 2, 1, 80, 20), (1, 9, 1, 1, 512, 512), (2, 65, 5, 1, 33, 33 - 1), (1, 2000, 2, 1, 16, 16), (700, 1, 3, 1, 64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary(B, T, Hq, Hk, D, rot, interleaved, dtype):
    q, k, f = randn((B, T, Hq, D), dtype, 1), randn((B, T, Hk, D), dtype, 2), freqs(rot)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 100000, (B, T), generator=g, dtype=torch.int32)
    for inverse in (False, True):
        kw = dict(interleaved=interleaved, scale=1.25, inverse=inverse)
        gq, gk = gdn.gdn_rotary(dev(q), dev(f), k=dev(k), positions=dev(pos), **kw)
        for got, x in ((gq, q), (gk, k)):
            ref = ref_rotary(x, pos, f, interleaved, 1.25, inverse)
            assert got.dtype == dtype and rel(got, ref) <= tol(dtype, TOL_ROT)
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])  # what does not turn is copied


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_layouts_and_in_place(dtype):
    B, T, H, D, f = 2, 37, 3, 64, freqs(32)
    x, pos = randn((B, T, H, D), dtype, 4), torch.arange(T, dtype=torch.int64).expand(B, T) + 11
    for interleaved in (False, True):
        ref = ref_rotary(x, pos, f, interleaved, 1.0)
        layouts = [dev(x), strided(dev(x)), dev(x.transpose(1, 2).contiguous()).transpose(1, 2), dev(x.transpose(0, 1).contiguous()).transpose(0, 1),
                   strided(dev(x), 8, 8), strided(dev(x.transpose(1, 2).contiguous()), 1, 2).transpose(1, 2)]
        for t in layouts:
            got = gdn.gdn_rotary(t, dev(f), offset=11, interleaved=interleaved)
            assert got.is_contiguous() and rel(got, ref) <= tol(dtype, TOL_ROT)
            before = t.clone()
            back = gdn.gdn_rotary(t, dev(f), offset=11, interleaved=interleaved, out=t)
            assert back is t and torch.equal(t, got)
            t.copy_(before)
        # q and k as slices of one projection; positions of one row for all; the gaps stay
        qkv = torch.cat([x, x + 1, x - 1], 2).to(DEV)
        kept = qkv.clone()
        q, k = qkv[:, :, :H], qkv[:, :, H:2 * H]
        gq, gk = gdn.gdn_rotary(q, dev(f), k=k, positions=dev(pos[0].contiguous()), interleaved=interleaved, out=q, k_out=k)
        assert rel(gq, ref) <= tol(dtype, TOL_ROT) and gk.data_ptr() == k.data_ptr()
        assert rel(gk, ref_rotary((x + 1), pos, f, interleaved, 1.0)) <= tol(dtype, TOL_ROT)
        assert torch.equal(qkv[:, :, 2 * H:], kept[:, :, 2 * H:]) and torch.equal(qkv[..., 32:], kept[..., 32:])


@pytest.mark.parametrize("p", [0, 1, -1, 2**20 + 1, 2**31 - 1, -2**31, 2**40 + 12345, -2**62])
def test_rotary_far_positions(p):
    """The angle of a far position to a small part of a turn: frequencies that are whole parts of one have known angles."""
    n = torch.tensor([1, 2, 3, 5, 64, 1000, 2**20, 2**30])
    f = 2 * math.pi / n.to(F64)
    x = torch.zeros(1, 1, 1, 16)
    x[..., :8] = 1.0
    got = gdn.gdn_rotary(dev(x), dev(f), positions=torch.tensor([[p]], dtype=torch.int64, device=DEV)).cpu().to(F64)[0, 0, 0]
    turn = torch.tensor([(p % int(k)) / int(k) for k in n], dtype=F64)
    # f is a double near 2 pi / n: off by 2^-53 of it, times p, beside the fp32 result's 4e-7
    bound = 4e-7 + abs(p) * (2 * math.pi / n.to(F64)) * 2.0**-52
    for k in range(8):
        assert abs(got[k] - math.cos(2 * math.pi * turn[k])) <= bound[k] and abs(got[8 + k] - math.sin(2 * math.pi * turn[k])) <= bound[k], k


def test_rotary_without_tokens_and_fast_frequencies():
    f = dev(torch.tensor([math.pi, 5.0, 100.0, 0.0], dtype=F64))
    assert gdn.gdn_rotary(torch.empty(2, 0, 3, 16, device=DEV), f).shape == (2, 0, 3, 16)
    assert gdn.gdn_rotary(torch.empty(0, 4, 3, 16, device=DEV), f, positions=torch.empty(0, 4, dtype=torch.int32, device=DEV)).shape == (0, 4, 3, 16)
    x, pos = randn((1, 9, 2, 16), F32, 5), torch.arange(9)[None]
    assert rel(gdn.gdn_rotary(dev(x), f), ref_rotary(x, pos, f.cpu(), False, 1.0)) <= TOL_ROT
    # another element than the pair's stays out of a NaN
    x[0, 3, 1, 2] = float("nan")
    got = gdn.gdn_rotary(dev(x), f)
    assert torch.nonzero(got.isnan()).cpu().tolist() == [[0, 3, 1, 2], [0, 3, 1, 6]]


def test_rotary_gradient():
    q, k, f = (randn((2, 19, 4, 48), F32, 6).to(DEV).requires_grad_(), randn((2, 19, 2, 48), F32, 7).to(DEV).requires_grad_(), dev(freqs(32)))
    gq, gk = randn((2, 19, 4, 48), F32, 8).to(DEV), randn((2, 19, 2, 48), F32, 9).to(DEV)
    a, b = gdr.rotary(q, f, k=k, offset=5, interleaved=True, scale=0.5)
    dq, dk = torch.autograd.grad((a * gq).sum() + (b * gk).sum(), (q, k))
    # the map is linear: <g, R v> = <R' g, v>
    v = randn(q.shape, F32, 10).to(DEV)
    lhs = (gq.double() * gdn.gdn_rotary(v, f, offset=5, interleaved=True, scale=0.5).double()).sum()
    assert abs(lhs - (dq.double() * v.double()).sum()) <= 1e-6 * gq.double().norm() * v.double().norm()
    pos = (torch.arange(19) + 5).expand(2, 19)
    for got, g in ((dq, gq), (dk, gk)):
        assert rel(got, ref_rotary(g.cpu(), pos, f.cpu(), True, 0.5, True)) <= TOL_ROT
    (only,) = torch.autograd.grad(gdr.rotary(q, f).sum(), q)  # (an expanded gradient)
    assert rel(only, ref_rotary(torch.ones(q.shape), torch.arange(19).expand(2, 19), f.cpu(), False, 1.0, True)) <= TOL_ROT


# ------------------------------------------------------------ block norm ---


def act_of(g, act):
    return g if act is None else torch.sigmoid(g) if act == "sigmoid" else g * torch.sigmoid(g)


def norm(x, w, eps):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w


def ref_block(y, res, post, pre, gate, act, scale, alpha, eps):
    u = norm(y, post, eps) if post is not None else y
    if gate is not None:
        u = act_of(gate, act) * u
    s = res + alpha * (scale * u if scale is not None else u)
    return s, norm(s, pre, eps) if pre is not None else None


def block_inputs(B, T, D, dtype, res, post, pre, gate, scale, seed=20):
    y, r = randn((B, T, D), dtype, seed), randn((B, T, D), res, seed + 1, 2.0)
    w = [randn((D,), F32, seed + 2 + i, 0.1, m) if on else None for i, (on, m) in enumerate(((post, 1.0), (pre, 1.0), (scale, 0.5)))]
    g = {None: None, "token": (B, T, D), "sequence": (B, 1, D)}[gate]
    return y, r, w[0], w[1], None if g is None else randn(g, dtype, seed + 5), w[2]


SIZES = [(1, 1, 1), (1, 3, 7), (2, 5, 64), (1, 1, 2048), (3, 70, 100), (2, 9, 1000), (2, 33, 4096), (1, 2, 5000), (1, 3, 16384), (3, 43, 72),
         (1, 5, 8192), (2, 700, 40), (12, 5, 48), (9, 33, 1792)]
FORMS = [  # dtype, residual, post, pre, gate, act, scale
    (BF, BF, True, True, None, None, False), (BF, F32, True, True, "token", "sigmoid", True), (F32, F32, True, True, "sequence", "silu", True),
    (F32, BF, True, False, "token", None, False), (BF, BF, False, True, "sequence", None, False), (F32, F32, False, True, "token", "silu", True),
    (BF, F32, True, False, "sequence", "sigmoid", True)]


@pytest.mark.parametrize("B,T,D", SIZES)
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_block_norm(B, T, D, form):
    dtype, res, post, pre, gate, act, scale = FORMS[form]
    y, r, wp, wn, g, sc = block_inputs(B, T, D, dtype, res, post, pre, gate, scale)
    s, out = ref_block(*(f64(t) for t in (y, r)), f64(wp), f64(wn), f64(g), act, f64(sc), 0.75, 1e-6)
    kw = dict(post_weight=dev(wp), pre_weight=dev(wn), gate=dev(g), gate_act=act, scale=dev(sc), alpha=0.75)
    got = gdn.gdn_block_norm_fwd(dev(y), dev(r), **kw)
    assert ("out" in got) == pre and got["residual"].dtype == res
    assert rel(got["residual"], s) <= tol(res, TOL_NORM)
    if pre:
        assert got["out"].dtype == dtype and rel(got["out"], out) <= tol(dtype, TOL_NORM)


@pytest.mark.parametrize("B,T,D", SIZES)
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_block_norm_bwd(B, T, D, form):
    dtype, res, post, pre, gate, act, scale = FORMS[form]
    y, r, wp, wn, g, sc = block_inputs(B, T, D, dtype, res, post, pre, gate, scale)
    do, dr = randn((B, T, D), dtype, 30) if pre else None, randn((B, T, D), res, 31)
    if pre and form == 2:
        dr = None
    kw = dict(gate_act=act, alpha=0.75)
    fwd = dict(post_weight=dev(wp), pre_weight=dev(wn), gate=dev(g), scale=dev(sc), **kw)
    s = gdn.gdn_block_norm_fwd(dev(y), dev(r), **fwd)["residual"]
    names = dict(y="dy", r="dresidual", wp="dpost_weight", wn="dpre_weight", g="dgate", sc="dscale")
    leaf = {k: f64(t).requires_grad_() for k, t in dict(y=y, r=r, wp=wp, wn=wn, g=g, sc=sc).items() if t is not None}
    t, _ = ref_block(leaf["y"], leaf["r"], leaf.get("wp"), None, leaf.get("g"), act, leaf.get("sc"), 0.75, 1e-6)
    t = t + (f64(s) - t.detach())  # at the sum as stored
    loss = (t * f64(dr)).sum() if dr is not None else 0.0
    if pre:
        loss = loss + (norm(t, leaf["wn"], 1e-6) * f64(do)).sum()
    want = dict(zip((names[k] for k in leaf), torch.autograd.grad(loss, tuple(leaf.values()))))
    got = gdn.gdn_block_norm_bwd(dev(y), s, dout=dev(do), dres=dev(dr), **fwd)
    assert set(got) == set(want)
    for k, v in got.items():
        assert rel(v, want[k]) <= tol(v.dtype, TOL_NORM), k
        assert v.dtype == {"dy": dtype, "dresidual": res, "dgate": dtype}.get(k, F32)
    again = gdn.gdn_block_norm_bwd(dev(y), s, dout=dev(do), dres=dev(dr), **fwd)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_block_norm_strides_rows_and_in_place():
    y, r, wp, wn, g, sc = block_inputs(2, 7, 100, BF, BF, True, True, "sequence", True)
    s, out = ref_block(*(f64(t) for t in (y, r, wp, wn, g)), "silu", f64(sc), 1.0, 1e-5)
    rr, yy = dev(r), dev(y)
    kw = dict(post_weight=dev(wp), pre_weight=dev(wn), gate_act="silu", scale=dev(sc), eps=1e-5)
    got = gdn.gdn_block_norm_fwd(strided(dev(y)), strided(dev(r)), gate=strided(dev(g)), **kw)
    assert rel(got["out"], out) <= TOL_BF and rel(got["residual"], s) <= TOL_BF
    got = gdn.gdn_block_norm_fwd(yy, rr, gate=dev(g), residual_out=rr, out=yy, **kw)
    assert got["out"] is yy and got["residual"] is rr and rel(yy, out) <= TOL_BF and rel(rr, s) <= TOL_BF
    # rows of any leading shape: the token's gate at T = 1, four dimensions, two
    flat = gdn.gdn_block_norm_fwd(dev(y).view(14, 1, 100), dev(r).view(14, 1, 100), gate=dev(g.expand(2, 7, 100).reshape(14, 1, 100)), **kw)
    four = gdn.gdn_block_norm_fwd(dev(y).view(2, 1, 7, 100), dev(r).view(2, 1, 7, 100), gate=dev(g.expand(2, 7, 100).reshape(2, 1, 7, 100)), **kw)
    two = gdn.gdn_block_norm_fwd(dev(y).view(14, 100), dev(r).view(14, 100), gate=dev(g.expand(2, 7, 100).reshape(14, 100)), **kw)
    for x in (flat, four, two):
        assert torch.equal(x["out"].flatten(), yy.flatten()) and torch.equal(x["residual"].flatten(), rr.flatten())
    # no rows
    empty = gdn.gdn_block_norm_fwd(dev(y)[:0], dev(r)[:0], gate=dev(g)[:0], **kw)
    assert empty["out"].shape == (0, 7, 100)
    z = gdn.gdn_block_norm_bwd(dev(y)[:0], dev(r)[:0], dout=dev(y)[:0], gate=dev(g)[:0], **kw)
    assert (z["dpost_weight"] == 0).all() and (z["dscale"] == 0).all() and (z["dpre_weight"] == 0).all() and z["dgate"].shape == (0, 1, 100)


def test_block_norm_of_sequences_without_tokens():
    """A shared gate row nobody takes: its gradient is zeros, and so are the weights'; below Python nothing of it is touched."""
    y, g, w = torch.empty(2, 0, 64, device=DEV), dev(randn((2, 1, 64), F32, 43)), dev(randn((64,), F32, 44))
    kw = dict(post_weight=w, pre_weight=w, gate=g, gate_act="silu")
    got = gdn.gdn_block_norm_fwd(y, y.clone(), **kw)
    assert got["out"].shape == got["residual"].shape == (2, 0, 64)
    b = gdn.gdn_block_norm_bwd(y, got["residual"], dout=y.clone(), **kw)
    assert b["dgate"].shape == (2, 1, 64) and all((b[k] == 0).all() for k in ("dgate", "dpost_weight", "dpre_weight"))
    L = layer._load()
    dg, dw, ws = torch.full((2, 64), 7.0, device=DEV), torch.ones(64, device=DEV), torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    st = L.gdn_block_norm_bwd(0, 64, 0, 0, 64, 0, g.data_ptr(), 64, 5, 3, 0, 64, 0, 64, w.data_ptr(), w.data_ptr(), 0, 1.0, 0, 64, 0, 64,
                              dg.data_ptr(), 64, dw.data_ptr(), 0, 0, 0, 64, 1e-6, ws.data_ptr(), ws.numel(),
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and (dg == 7).all() and (dw == 0).all()


def test_block_norm_closed_and_non_finite_rows_stay_apart():
    """A gate of the lowest value lets nothing through; a row's NaN or infinity reaches no other row."""
    y, r, wp, wn, g, sc = block_inputs(1, 6, 256, F32, F32, True, True, "token", True)
    low = torch.finfo(F32).min
    g[0, 0] = low
    y[0, 1, 3], g[0, 2, 7], r[0, 3, 9] = float("nan"), float("nan"), float("inf")
    y[0, 4] = 0
    for act in ("sigmoid", "silu"):
        kw = dict(post_weight=dev(wp), pre_weight=dev(wn), gate=dev(g), gate_act=act, scale=dev(sc))
        got = gdn.gdn_block_norm_fwd(dev(y), dev(r), **kw)
        assert torch.equal(got["residual"][0, 0].cpu(), r[0, 0]) and torch.equal(got["residual"][0, 4].cpu(), r[0, 4])
        s, out = ref_block(*(f64(t)[0, [0, 4, 5]] for t in (y, r)), f64(wp), f64(wn), f64(g)[0, [0, 4, 5]], act, f64(sc), 1.0, 1e-6)
        assert rel(got["out"][0, [0, 4, 5]], out) <= TOL_NORM
        assert got["residual"][0, 1].isnan().all() and got["residual"][0, 2].isnan().sum() == 1 and got["out"][0, 2].isnan().all()
        assert got["out"][0, 3, 9].isnan() and (got["out"][0, 3, :9] == 0).all()
        bwd = gdn.gdn_block_norm_bwd(dev(y), got["residual"], dout=dev(randn((1, 6, 256), F32, 40)), **kw)
        for k in ("dy", "dresidual", "dgate"):
            assert bwd[k][0, [0, 4, 5]].isfinite().all(), k
        assert (bwd["dy"][0, 0] == 0).all() and (bwd["dgate"][0, 0] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [256, 100, 1792])
@pytest.mark.parametrize("gate", ["token", "sequence"])
def test_block_norm_padding_of_extreme_values(dtype, D, gate):
    """Padded rows of the type's lowest value, whose squares pass fp32's range: they are normed to zeros and add none to the
    weights' gradients, and a stream row of them passes its own gradient on."""
    y, r, wp, wn, g, sc = block_inputs(1, 9, D, dtype, dtype, True, True, gate, True)
    do, dr = randn((1, 9, D), dtype, 45), randn((1, 9, D), dtype, 46)
    low = torch.finfo(dtype).min
    pad, keep = [2, 6], [0, 1, 3, 4, 5, 7, 8]
    kw = dict(post_weight=dev(wp), pre_weight=dev(wn), gate=dev(g), gate_act="sigmoid", scale=dev(sc))
    y[0, pad] = low
    f = gdn.gdn_block_norm_fwd(dev(y), dev(r), **kw)
    assert torch.equal(f["residual"][0, pad].cpu(), r[0, pad])
    b = gdn.gdn_block_norm_bwd(dev(y), f["residual"], dout=dev(do), dres=dev(dr), **kw)
    assert all(b[k].isfinite().all() for k in b) and (b["dy"][0, pad] == 0).all()
    s = f["residual"].clone()
    s[0, pad] = low
    b = gdn.gdn_block_norm_bwd(dev(y), s, dout=dev(do), dres=dev(dr), **kw)
    assert all(b[k].isfinite().all() for k in b) and torch.equal(b["dresidual"][0, pad].cpu(), dr[0, pad])
    few = dict(kw, gate=dev(g)[:, keep].contiguous() if gate == "token" else dev(g))
    alone = gdn.gdn_block_norm_bwd(dev(y)[:, keep].contiguous(), s[:, keep].contiguous(), dout=dev(do)[:, keep].contiguous(),
                                   dres=dev(dr)[:, keep].contiguous(), **few)
    for k in ("dpost_weight", "dpre_weight", "dscale"):
        assert rel(b[k], f64(alone[k])) <= TOL_NORM, k


def test_block_norm_gradient_by_differences():
    y, r, wp, wn, g, sc = block_inputs(2, 6, 72, F32, F32, True, True, "sequence", True)
    do, dr = dev(randn((2, 6, 72), F32, 41)), dev(randn((2, 6, 72), F32, 42))
    leaves = [dev(t).requires_grad_() for t in (y, r, wp, wn, g, sc)]

    def loss(y, r, wp, wn, g, sc):
        out, s = gdr.block_norm(y, r, post_weight=wp, pre_weight=wn, gate=g, gate_act="silu", scale=sc, alpha=0.5)
        return (out.double() * do).sum() + (s.double() * dr).sum()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    for i in range(6):
        v = dev(randn(leaves[i].shape, F32, 50 + i))
        h = 2.0**-7
        with torch.no_grad():
            at = [loss(*[t + (sign * h * v if j == i else 0) for j, t in enumerate(leaves)]) for sign in (1, -1)]
        d, e = ((at[0] - at[1]) / (2 * h)).item(), (grads[i].double() * v).sum().item()
        assert abs(d - e) <= TOL_DIFF * (grads[i].double().norm() * v.double().norm()).item(), i


# ------------------------------------------------------ gated recurrence ---


def decays(C, lo=0.9, hi=0.999, c=8.0, seed=60):
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(C, generator=g, dtype=F64) * (hi - lo) + lo
    return torch.log(torch.expm1(-torch.log(a) / c)).float()


def ref_lru(x, r, i, lam, z, h0, lens, c=8.0):
    B, T, C = x.shape
    u = c * torch.nn.functional.softplus(lam, threshold=200) * torch.sigmoid(r)
    a, b = torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u)) * torch.sigmoid(i) * x
    rows, final = [[] for _ in range(B)], []
    for k, (row, p, q) in enumerate(spans(B, T, lens)):
        h = h0[k] if h0 is not None else torch.zeros(C, dtype=F64)
        for t in range(p, q):
            h = a[row, t] * h + b[row, t]
            rows[row].append(h)
        final.append(h)
    h = torch.stack([torch.stack(v) if v else torch.zeros(0, C, dtype=F64) for v in rows])
    return h if z is None else h * z * torch.sigmoid(z), torch.stack(final)


def lru_inputs(B, T, C, lens, dtype, full, seed=61):
    n = B if lens is None else len(lens)
    x, r, i = (randn((B, T, C), dtype, seed + k) for k in range(3))
    z = randn((B, T, C), dtype, seed + 3) if full else None
    return x, r, i, decays(C), z, randn((n, C), F32, seed + 4) if full else None, n


LRU = [  # B, T, C, lens
    (1, 1, 8, None), (2, 5, 3, None), (1, 7, 1, None), (2, 8, 64, None), (1, 9, 66, None), (3, 64, 40, None), (1, 65, 129, None),
    (1, 600, 257, None), (2, 513, 200, None), (1, 128, 1024, None), (1, 64, 24, [64]), (1, 50, 33, [1, 0, 2, 3, 0, 0, 40, 4]),
    (1, 333, 136, [5, 0, 200, 1, 1, 126, 0]), (1, 6, 16, [0, 6, 0]), (1, 600, 72, [8, 56, 64, 100, 28, 256, 88]), (2, 0, 16, None),
    (1, 0, 16, [0, 0, 0]), (1, 40, 64, [1] * 40)]


@pytest.mark.parametrize("B,T,C,lens", LRU)
@pytest.mark.parametrize("dtype,full", [(BF, True), (BF, False), (F32, True), (F32, False)])
def test_lru(B, T, C, lens, dtype, full):
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, lens, dtype, full)
    ref, fin = ref_lru(*(f64(t) for t in (x, r, i, lam, z, h0)), lens)
    final = torch.full((n, C), float("nan"), device=DEV)
    ck = torch.full((B, (T + 63) // 64, C), float("nan"), device=DEV)
    args = [strided(dev(t)) if full else dev(t) for t in (x, r, i)] + [dev(lam)]
    kw = dict(z=dev(z), h0=dev(h0), cu_seqlens=dev(cu_of(lens)))
    got = gdn.gdn_lru_fwd(*args, h_final=final, checkpoints=ck, **kw)
    assert rel(got, ref) <= tol(dtype, TOL_LRU) and rel(final, fin) <= TOL_LRU
    assert ck.isfinite().all()
    if full:  # wide rows walk the same tiles
        again = gdn.gdn_lru_fwd(*(dev(t) for t in (x, r, i)), dev(lam), **kw)
        assert rel(again, ref) <= tol(dtype, TOL_LRU)


@pytest.mark.parametrize("B,T,C,lens", LRU)
@pytest.mark.parametrize("dtype,full", [(BF, True), (BF, False), (F32, True), (F32, False)])
def test_lru_bwd(B, T, C, lens, dtype, full):
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, lens, dtype, full)
    do, dh = randn((B, T, C), dtype, 70), randn((n, C), F32, 71) if full else None
    leaf = {k: f64(t).requires_grad_() for k, t in dict(x=x, r=r, i=i, lam=lam, z=z, h0=h0).items() if t is not None}
    out, fin = ref_lru(leaf["x"], leaf["r"], leaf["i"], leaf["lam"], leaf.get("z"), leaf.get("h0"), lens)
    loss = (out * f64(do)).sum() + ((fin * f64(dh)).sum() if full else 0)
    want = dict(zip(("d" + k for k in leaf), torch.autograd.grad(loss, tuple(leaf.values()), allow_unused=True))) if T or full else {}
    args = [strided(dev(t)) if full else dev(t) for t in (x, r, i)] + [dev(lam), strided(dev(do)) if full else dev(do)]
    kw = dict(z=dev(z), h0=dev(h0), cu_seqlens=dev(cu_of(lens)), dh_final=dev(dh))
    ck = torch.empty((B, (T + 63) // 64, C), device=DEV)
    gdn.gdn_lru_fwd(*args[:4], h0=dev(h0), cu_seqlens=dev(cu_of(lens)), checkpoints=ck)
    got = gdn.gdn_lru_bwd(*args, checkpoints=ck, **kw)
    assert set(got) == {"dx", "dr", "di", "dlam"} | ({"dz", "dh0"} if full else set())
    for k, v in got.items():
        w = want.get(k)
        assert rel(v, w if w is not None else torch.zeros(v.shape, dtype=F64)) <= tol(v.dtype, TOL_LRU_BWD), k
    # the states formed again: the same, and the same bits each time
    for other in (gdn.gdn_lru_bwd(*args, **kw), gdn.gdn_lru_bwd(*args, checkpoints=ck, **kw)):
        assert all(torch.equal(got[k], other[k]) for k in got)


@pytest.mark.parametrize("B,T,C,dtype", [(24, 300, 640, BF), (24, 300, 636, BF), (24, 300, 640, F32), (8, 300, 2560, BF), (8, 300, 2560, F32)])
def test_lru_many_lines(B, T, C, dtype):
    """As many lines and channels as fill the GPU alone (whole lines, eight warps), or leave a part of it (clusters)."""
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, None, dtype, True, seed=140)
    do, dh = randn((B, T, C), dtype, 150), randn((n, C), F32, 151)
    leaf = [f64(t).requires_grad_() for t in (x, r, i, lam, z, h0)]
    u = 8 * torch.nn.functional.softplus(leaf[3], threshold=200) * torch.sigmoid(leaf[1])
    a, b = torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u)) * torch.sigmoid(leaf[2]) * leaf[0]
    h, rows = leaf[5], []
    for t in range(T):
        h = a[:, t] * h + b[:, t]
        rows.append(h)
    ref = torch.stack(rows, 1) * leaf[4] * torch.sigmoid(leaf[4])
    want = torch.autograd.grad((ref * f64(do)).sum() + (h * f64(dh)).sum(), leaf)
    args, kw = [dev(t) for t in (x, r, i, lam)], dict(z=dev(z), h0=dev(h0))
    final, ck = torch.empty(n, C, device=DEV), torch.empty(B, (T + 63) // 64, C, device=DEV)
    got = gdn.gdn_lru_fwd(*args, h_final=final, checkpoints=ck, **kw)
    assert rel(got, ref.detach()) <= tol(dtype, TOL_LRU) and rel(final, h.detach()) <= TOL_LRU
    g = gdn.gdn_lru_bwd(*args, dev(do), dh_final=dev(dh), checkpoints=ck, **kw)
    for k, w in zip(("dx", "dr", "di", "dlam", "dz", "dh0"), want):
        assert rel(g[k], w) <= tol(g[k].dtype, TOL_LRU_BWD), k


def test_lru_long_lines_cross_tiles_and_clusters():
    """Every place of a sequence's end in a warp, a tile, a cluster's step; more tokens than one step of a cluster takes."""
    lens = [1500, 63, 1, 64, 65, 7, 8, 9, 511, 512, 513, 30]
    T, C = sum(lens), 128
    x, r, i, lam, z, h0, n = lru_inputs(1, T, C, lens, F32, True)
    lam = decays(C, 0.5, 0.9)  # (short memory: the tolerance's steps stay below 600)
    ref, fin = ref_lru(*(f64(t) for t in (x, r, i, lam, z, h0)), lens)
    final = torch.empty(n, C, device=DEV)
    cu = dev(cu_of(lens))
    got = gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), z=dev(z), h0=dev(h0), cu_seqlens=cu, h_final=final)
    assert rel(got, ref) <= TOL_LRU and rel(final, fin) <= TOL_LRU
    # each sequence alone
    at = 0
    for k, n_tok in enumerate(lens):
        part = [dev(t[:, at:at + n_tok].contiguous()) for t in (x, r, i, z)]
        alone = gdn.gdn_lru_fwd(*part[:3], dev(lam), z=part[3], h0=dev(h0[k:k + 1]))
        assert rel(alone, got[:, at:at + n_tok]) <= TOL_LRU
        at += n_tok
    # a line in two calls, the state carried, is the line
    state = torch.empty(1, C, device=DEV)
    a, b = slice(0, 1001), slice(1001, 1500)
    first = gdn.gdn_lru_fwd(*(dev(t[:, a]) for t in (x, r, i)), dev(lam), h0=dev(h0[:1]), h_final=state)
    second = gdn.gdn_lru_fwd(*(dev(t[:, b]) for t in (x, r, i)), dev(lam), h0=state)
    whole = gdn.gdn_lru_fwd(*(dev(t[:, :1500]) for t in (x, r, i)), dev(lam), h0=dev(h0[:1]))
    assert rel(torch.cat([first, second], 1), whole) <= TOL_LRU


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lru_masked_tokens_and_extremes(dtype):
    """Gates of the lowest and of the greatest value: r closed keeps the state, i closed adds nothing; the gradients
    there are finite."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    B, T, C = 1, 200, 72
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, None, dtype, True)
    for closed in (low, float("-inf"), -1000.0):
        rr, ii = r.clone(), i.clone()
        rr[:, 20:150] = closed  # a = 1 and no input
        ii[:, 150:] = closed    # decay alone
        h = torch.empty(n, C, device=DEV)
        out = gdn.gdn_lru_fwd(dev(x), dev(rr), dev(ii), dev(lam), h0=dev(h0), h_final=h)
        # To the bit inside each run of eight tokens. From run to run the state is walked, joined over runs or joined
        # over tiles: each of these is off by at most 64 multiply-adds, 8 + 8 joins and one more rounding of 2^-24, of
        # |A v| + |H| <= 2 max|h|; two of them differ by at most 2 * 81 * 2 * 2^-24 max|h|.
        for s in (20, *range(24, 150, 8)):
            e = min(s // 8 * 8 + 8, 150)
            assert (out[:, s:e] == out[:, s:s + 1]).all(), s
        if dtype == F32:
            assert (out[:, 20:150] - out[:, 19:20]).abs().max() <= 324 * 2.0**-24 * out.abs().max()
        ref, fin = ref_lru(*(f64(t) for t in (x, rr, ii, lam)), None, f64(h0), None)
        assert rel(out, ref) <= tol(dtype, TOL_LRU) and rel(h, fin) <= TOL_LRU
        g = gdn.gdn_lru_bwd(dev(x), dev(rr), dev(ii), dev(lam), dev(z), h0=dev(h0))
        assert all(v.isfinite().all() for v in g.values())
        assert (g["dr"][:, 20:150] == 0).all() and (g["dx"][:, 20:150] == 0).all() and (g["di"][:, 20:] == 0).all()
        assert (g["dx"][:, 150:] == 0).all()
    rr, zz = r.clone(), z.clone()
    rr[:, 50], zz[:, 60], zz[:, 61] = high, low, high
    lam[0], lam[1], lam[2] = -200.0, -30.0, 80.0
    x[..., 0] = 0.0
    zz = zz.clamp(max=1e30)
    out = gdn.gdn_lru_fwd(dev(x), dev(rr), dev(i), dev(lam), z=dev(zz), h0=dev(h0))
    assert out.isfinite().all() and (out[:, 60] == 0).all()
    g = gdn.gdn_lru_bwd(dev(x), dev(rr), dev(i), dev(lam), dev(z), z=dev(zz), h0=dev(h0))
    assert all(v.isfinite().all() for v in g.values())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lru_largest_inputs_behind_a_closed_gate(dtype):
    """Padding of the type's lowest or largest value under a closed r adds nothing, forward or back."""
    B, T, C = 2, 70, 40
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, None, dtype, True, seed=160)
    do, pad = randn((B, T, C), dtype, 170), slice(20, 45)
    r[:, pad] = torch.finfo(dtype).min
    x[:, pad] = 0.0
    args = lambda: ([dev(t) for t in (x, r, i, lam)], dict(z=dev(z), h0=dev(h0)))  # noqa: E731
    a, kw = args()
    want, grads = gdn.gdn_lru_fwd(*a, **kw), gdn.gdn_lru_bwd(*a, dev(do), **kw)
    for value in (torch.finfo(dtype).min, torch.finfo(dtype).max):
        x[:, pad] = value
        a, kw = args()
        assert torch.equal(gdn.gdn_lru_fwd(*a, **kw), want)
        got = gdn.gdn_lru_bwd(*a, dev(do), **kw)
        assert all(torch.equal(got[k], grads[k]) for k in got)
        assert all((got[k][:, pad] == 0).all() for k in ("dx", "dr", "di"))


def test_lru_non_finite_values_stay_in_their_channel_and_sequence():
    lens = [70, 3, 500, 27]
    T, C = sum(lens), 64
    for where, value in (("x", float("nan")), ("r", float("nan")), ("i", float("nan")), ("x", float("inf"))):
        x, r, i, lam, z, h0, n = lru_inputs(1, T, C, lens, F32, True)
        clean = gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), z=dev(z), h0=dev(h0), cu_seqlens=dev(cu_of(lens)))
        dict(x=x, r=r, i=i)[where][0, 100, 5] = value
        final = torch.empty(n, C, device=DEV)
        args = (dev(x), dev(r), dev(i), dev(lam))
        kw = dict(z=dev(z), h0=dev(h0), cu_seqlens=dev(cu_of(lens)))
        got = gdn.gdn_lru_fwd(*args, h_final=final, **kw)
        bad = ~got.isfinite()
        assert bad[0, 100:573, 5].all() and bad.sum() == 473
        assert torch.equal(got[~bad], clean[~bad]) and (~final.isfinite()).nonzero().tolist() == [[2, 5]]
        g = gdn.gdn_lru_bwd(*args, dev(z), dh_final=torch.ones(n, C, device=DEV), **kw)
        for k in ("dx", "dr", "di", "dz"):
            b = (~g[k].isfinite()).nonzero().cpu()
            assert (b[:, 2] == 5).all() and (b[:, 1] >= 73).all() and (b[:, 1] < 573).all(), k
        assert (~g["dlam"].isfinite()).nonzero().flatten().tolist() in ([], [5])
        assert set((~g["dh0"].isfinite()).nonzero()[:, 0].tolist()) <= {2}
    # and in a state
    h0[1, 7] = float("nan")
    x, r, i, lam, z, _, n = lru_inputs(1, T, C, lens, F32, True)
    got = gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), h0=dev(h0), cu_seqlens=dev(cu_of(lens)))
    assert (~got.isfinite()).nonzero().tolist() == [[0, t, 7] for t in (70, 71, 72)]


def test_lru_out_in_place():
    x, r, i, lam, z, h0, n = lru_inputs(2, 700, 96, None, BF, True)
    want = gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), z=dev(z), h0=dev(h0))
    for k in range(4):
        t = [dev(v) for v in (x, r, i, z)]
        got = gdn.gdn_lru_fwd(*t[:3], dev(lam), z=t[3], h0=dev(h0), out=t[k])
        assert got is t[k] and torch.equal(got, want)


def test_lru_malformed_cu_seqlens_is_reported():
    import ctypes
    x, r, i, lam, z, h0, _ = lru_inputs(1, 100, 64, [50, 50], F32, True)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    for cu in ([0, 70, 60], [5, 50, 100], [0, 50, 1 << 30], [0, -7, 100]):
        t = torch.tensor(cu, dtype=torch.int32, device=DEV)
        gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), z=dev(z), h0=dev(h0), cu_seqlens=t, workspace=ws, h_final=torch.empty(2, 64, device=DEV))
        word = ctypes.c_int(0)
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert gdn.lib().gdn_last_device_error(ctypes.c_void_p(ws.data_ptr()), stream, ctypes.byref(word)) == 9 and word.value == 1
        gdn.gdn_lru_bwd(dev(x), dev(r), dev(i), dev(lam), dev(x), z=dev(z), h0=dev(h0), cu_seqlens=t, workspace=ws)
        assert gdn.lib().gdn_last_device_error(ctypes.c_void_p(ws.data_ptr()), stream, ctypes.byref(word)) == 9


def test_lru_decays_near_one():
    """A state of one and no input leave a itself. For u = c softplus(lam) sigmoid(r) below 1/8 it is 1 - t, rounded to half a
    step of the values below one (2^-25), with t = 1 - exp(-u) right to 2^-20: the sigmoid's exponential, sum and reciprocal
    2^-21.4, softplus and its product 2^-22, the series 2^-22.5. (An exponential good to 2^-22 would not pass where t < 2^-5.)"""
    C = 4096
    lam = decays(C, 0.985, 0.9999, seed=97)
    r = torch.linspace(-9, 9, C, dtype=F64)[torch.randperm(C, generator=torch.Generator().manual_seed(98))].float()[None]
    u = 8 * torch.nn.functional.softplus(f64(lam), threshold=200) * torch.sigmoid(f64(r))
    assert u.max() < 0.125
    state, zero = torch.ones(1, C, device=DEV), torch.zeros(1, C, device=DEV)
    gdn.gdn_lru_step(zero, dev(r), zero, dev(lam), state)
    t = -torch.expm1(-u)
    off = (state.cpu().double() - (1 - t)).abs()
    assert (off <= 2.0**-25 + t * 2.0**-20).all(), (off / (2.0**-25 + t * 2.0**-20)).max()
    # the same a in whole sequences: the final state of one token
    final = torch.empty(1, C, device=DEV)
    gdn.gdn_lru_fwd(zero[None], dev(r)[None], zero[None], dev(lam), h0=torch.ones(1, C, device=DEV), h_final=final)
    assert torch.equal(final, state)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lru_channels_do_not_see_their_neighbours_decay(dtype):
    """Warps whose channels all decay slowly take a shorter way to a; one fast channel sends them the other one, to the same bits."""
    B, T, C = 2, 150, 128
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, None, dtype, True, seed=180)
    do, fast = dev(randn((B, T, C), dtype, 190)), lam.clone()
    fast[[5, 127]] = 4.0
    rest = [c for c in range(C) if c not in (5, 127)]
    out = []
    for v in (lam, fast):
        args, kw = [dev(t) for t in (x, r, i, v)], dict(z=dev(z), h0=dev(h0))
        final = torch.empty(n, C, device=DEV)
        g = gdn.gdn_lru_bwd(*args, do, **kw)
        out.append([gdn.gdn_lru_fwd(*args, h_final=final, **kw), final, *(g[k] for k in sorted(g))])
    for a, b in zip(*out):
        assert torch.equal(a[..., rest], b[..., rest])


@pytest.mark.parametrize("n,C,pool", [(1, 4096, 1), (1, 1, 1), (5, 64, 9), (3, 7, 3), (64, 130, 80), (256, 512, 300)])
@pytest.mark.parametrize("dtype,full", [(BF, True), (F32, False)])
def test_lru_step(n, C, pool, dtype, full):
    x, r, i, z = (randn((n, C), dtype, 80 + k) for k in range(4))
    lam, state = decays(C), randn((pool, C), F32, 85)
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(86))[:n].to(torch.int32) if full else None
    z = z if full else None
    pad = full and n > 2
    if pad:
        slots[1], slots[2] = -1, pool
    at = slots.long() if full else torch.arange(n)
    live = (at >= 0) & (at < pool)
    st = dev(state)
    args = [strided(dev(t)) if full else dev(t) for t in (x, r, i)]
    got = gdn.gdn_lru_step(*args, dev(lam), st, z=dev(z), slots=dev(slots))
    ref, fin = ref_lru(*(f64(t)[live, None] for t in (x, r, i)), f64(lam), f64(z)[live, None] if full else None, f64(state)[at[live]], None)
    want = f64(state).clone()
    want[at[live]] = fin
    assert rel(got[dev(live)], ref[:, 0]) <= tol(dtype, 1e-6) and rel(st, want) <= 1e-6
    assert (got[~dev(live)] == 0).all()
    rest = torch.ones(pool, dtype=torch.bool)
    rest[at[live]] = False
    assert torch.equal(st.cpu()[rest], state[rest])  # other rows to the bit


def test_lru_steps_continue_a_prompt():
    x, r, i, lam, z, h0, n = lru_inputs(3, 80, 96, None, F32, True)
    whole = gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), z=dev(z), h0=dev(h0))
    state = torch.empty(3, 96, device=DEV)
    gdn.gdn_lru_fwd(*(dev(t[:, :70]) for t in (x, r, i)), dev(lam), h0=dev(h0), h_final=state)
    for t in range(70, 80):
        out = gdn.gdn_lru_step(*(dev(v[:, t]) for v in (x, r, i)), dev(lam), state, z=dev(z[:, t]))
        assert rel(out, whole[:, t]) <= TOL_LRU


def test_lru_gradient_by_differences():
    lens = [30, 0, 70, 20]
    x, r, i, lam, z, h0, n = lru_inputs(1, 120, 40, lens, F32, True)
    do, dh, cu = dev(randn((1, 120, 40), F32, 90)), dev(randn((n, 40), F32, 91)), dev(cu_of(lens))
    leaves = [dev(t).requires_grad_() for t in (x, r, i, lam, z, h0)]

    def loss(x, r, i, lam, z, h0):
        y, fin = gdr.gated_recurrence(x, r, i, lam, z=z, initial_state=h0, cu_seqlens=cu, output_final_state=True)
        return (y.double() * do).sum() + (fin.double() * dh).sum()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    for k in range(6):
        v = dev(randn(leaves[k].shape, F32, 92 + k))
        h = 2.0**-7
        with torch.no_grad():
            at = [loss(*[t + (sign * h * v if j == k else 0) for j, t in enumerate(leaves)]) for sign in (1, -1)]
        d, e = ((at[0] - at[1]) / (2 * h)).item(), (grads[k].double() * v).sum().item()
        assert abs(d - e) <= TOL_DIFF * (grads[k].double().norm() * v.double().norm()).item(), k


# ---------------------------------------------------------- as used together ---


def _cell(p, h, s, cu, h0):
    """A recurrent block between two norms, then the gated delta rule with rotary positions, on fp32 parameters."""
    B, T, D = h.shape
    x, r, i, z = (h.flatten(0, 1) @ p["proj"]).view(B, T, 4 * D).split(D, -1)
    x, _ = gdr.causal_conv(x, p["taps"], cu_seqlens=cu, silu=False)
    y, fin = gdr.gated_recurrence(x, r, i, p["lam"], z=z, initial_state=h0, cu_seqlens=cu, output_final_state=True)
    h, s = gdr.block_norm(y, s, post_weight=p["post"], pre_weight=p["pre"], gate=h, gate_act="sigmoid", scale=p["scale"])
    q, k, v = (t.reshape(B, T, 2, D // 2) for t in (h.flatten(0, 1) @ p["qkv"]).view(B, T, 3 * D).split(D, -1))
    q, k = gdr.rotary(q, p["freq"], k=k)
    beta, g = torch.sigmoid(h[..., :2]), -torch.sigmoid(h[..., 2:4])
    o, _ = gdr.chunk_gated_delta_rule(q, k, v, beta.contiguous(), g=g.contiguous(), cu_seqlens=cu)
    out, s = gdr.block_norm(o.reshape(B, T, D), s, post_weight=p["post"], pre_weight=p["pre"], alpha=0.5)
    return out, s, fin


def _cell_ref(p, h, s, lens, h0):
    B, T, D = h.shape
    x, r, i, z = (h @ p["proj"]).split(D, -1)
    W, rows = p["taps"].shape[1], []
    for row, a, b in spans(B, T, lens):
        line = torch.cat([torch.zeros(W - 1, D, dtype=F64), x[row, a:b]])
        rows.append(sum(p["taps"][:, j] * line[j:j + b - a] for j in range(W)))
    x = torch.cat(rows).view(B, T, D)
    y, fin = ref_lru(x, r, i, p["lam"], z, h0, lens)
    s, h = ref_block(y, s, p["post"], p["pre"], h, "sigmoid", p["scale"], 1.0, 1e-6)
    q, k, v = (t.reshape(B, T, 2, D // 2) for t in (h @ p["qkv"]).split(D, -1))

    def turned(t):
        ang = torch.arange(T, dtype=F64)[:, None, None] * p["freq"]
        u, w = t[..., :p["freq"].numel()], t[..., p["freq"].numel():2 * p["freq"].numel()]
        return torch.cat([u * ang.cos() - w * ang.sin(), w * ang.cos() + u * ang.sin(), t[..., 2 * p["freq"].numel():]], -1)

    q, k = turned(q), turned(k)
    q, k = (t / torch.sqrt(t.square().sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    beta, g = torch.sigmoid(h[..., :2]), -torch.sigmoid(h[..., 2:4])
    outs = []
    for row, a, b in spans(B, T, lens):
        S = torch.zeros(2, D // 2, D // 2, dtype=F64)
        for t in range(a, b):
            S = S * torch.exp(g[row, t])[:, None, None]
            d = beta[row, t][:, None] * (v[row, t] - torch.einsum("hkv,hk->hv", S, k[row, t]))
            S = S + torch.einsum("hk,hv->hkv", k[row, t], d)
            outs.append(torch.einsum("hkv,hk->hv", S, q[row, t]))
    o = torch.stack(outs).view(B, T, D)
    s, out = ref_block(o, s, p["post"], p["pre"], None, None, None, 0.5, 1e-6)
    return out, s, fin


def _cell_inputs(D=32, T=90, seed=110):
    p = dict(proj=randn((D, 4 * D), F32, seed, D**-0.5), qkv=randn((D, 3 * D), F32, seed + 1, D**-0.5), taps=randn((D, 4), F32, seed + 2, 0.5),
             lam=decays(D), post=randn((D,), F32, seed + 3, 0.1, 1.0), pre=randn((D,), F32, seed + 4, 0.1, 1.0),
             scale=randn((D,), F32, seed + 5, 0.1, 0.5), freq=freqs(8))
    return p, randn((1, T, D), F32, seed + 6), randn((1, T, D), F32, seed + 7), [40, 1, 49], randn((3, D), F32, seed + 8)


def test_blocks_of_both_mixers():
    """Norms, convolution, recurrence, rotary positions and the gated delta rule in a row, outputs and every gradient. The
    errors of each pass on to the next and are not amplified beyond the norms' gains: ten times the recurrence's."""
    p, h, s, lens, h0 = _cell_inputs()
    grad = [k for k in p if k != "freq"]
    P = {k: dev(v).requires_grad_(k != "freq") for k, v in p.items()}
    Q = {k: f64(v).requires_grad_(k != "freq") for k, v in p.items()}
    hg, hr = dev(h).requires_grad_(), f64(h).requires_grad_()
    got = _cell(P, hg, dev(s), dev(cu_of(lens)), dev(h0))
    ref = _cell_ref(Q, hr, f64(s), lens, f64(h0))
    w = [randn(t.shape, F32, 130 + k) for k, t in enumerate(ref)]
    for a, b in zip(got, ref):
        assert rel(a, b) <= 10 * TOL_LRU
    G = torch.autograd.grad(sum((a * dev(b)).sum() for a, b in zip(got, w)), [P[k] for k in grad] + [hg])
    R = torch.autograd.grad(sum((a * f64(b)).sum() for a, b in zip(ref, w)), [Q[k] for k in grad] + [hr])
    for name, a, b in zip(grad + ["h"], G, R):
        assert rel(a, b) <= 10 * TOL_LRU_BWD, name


def test_calls_on_another_stream_and_in_graphs():
    """A captured run of the operators, replayed on new inputs, beside a second graph; and calls on a side stream."""
    B, T, D = 2, 130, 64
    x, r, i, lam, z, h0, n = lru_inputs(B, T, D, None, BF, True)
    w, f = dev(randn((D,), F32, 120, 0.1, 1.0)), dev(freqs(16))
    bufs = [dev(t) for t in (x, r, i, z)]
    res, state, lam = dev(randn((B, T, D), BF, 121)), dev(randn((B, D), F32, 122)), dev(lam)

    def run(x, r, i, z, st):
        y = gdn.gdn_lru_fwd(x, r, i, lam, z=z, h0=st)
        b = gdn.gdn_block_norm_fwd(y, res, post_weight=w, pre_weight=w, gate=z, gate_act="silu")
        q = gdn.gdn_rotary(b["out"].view(B, T, 4, 16), f)
        g = gdn.gdn_lru_bwd(x, r, i, lam, b["out"], z=z, h0=st)
        g.update(gdn.gdn_block_norm_bwd(y, b["residual"], dout=b["out"], post_weight=w, pre_weight=w, gate=z, gate_act="silu"))
        st2 = st.clone()
        o = gdn.gdn_lru_step(x[:, 0], r[:, 0], i[:, 0], lam, st2, z=z[:, 0])
        return [y, b["out"], b["residual"], q, o, st2] + [g[k] for k in sorted(g)]

    want = run(*bufs, state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*bufs, state)
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(run(*bufs, state))
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for k in range(2):
        graphs[k].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    for t in bufs:
        t.copy_(t.flip(1).clone())
    want = run(*bufs, state)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    got = gdn.gdn_lru_fwd(*bufs[:3], lam, z=bufs[3], h0=state, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])


def test_rows_behind_the_outputs_stay():
    """Outputs in the middle of larger buffers: what lies around them is left as it was."""
    for C in (64, 71):
        x, r, i, lam, z, h0, n = lru_inputs(2, 77, C, None, BF, True)
        big = torch.full((2, 90, C + 40), 7.0, dtype=BF, device=DEV)
        out = big[:, 5:82, 8:8 + C]
        gdn.gdn_lru_fwd(dev(x), dev(r), dev(i), dev(lam), z=dev(z), out=out)
        big2 = torch.full((2, 90, C + 40), 7.0, dtype=BF, device=DEV)
        rows = big2.view(180, C + 40)[:154, 8:8 + C]
        gdn.gdn_block_norm_fwd(dev(x).view(154, C), dev(r).view(154, C), post_weight=torch.ones(C, device=DEV), residual_out=rows)
        big3 = torch.full((2, 90, 4, C + 40), 7.0, dtype=BF, device=DEV)
        turned = big3[:, 5:82, 1:3, 8:8 + C]
        gdn.gdn_rotary(dev(randn((2, 77, 2, C), BF, 99)), dev(freqs(32)), out=turned)
        for b, o in ((big, out), (big2, rows), (big3, turned)):
            assert not (o == 7.0).all()
            o.fill_(7.0)
            assert (b == 7.0).all()
