"""The state-space layer's entry points refuse bad arguments on the host,
before any launch (no GPU needed): the C entry points with fake device
addresses that nothing dereferences, the Python ones with CPU tensors."""
import ctypes

import pytest
import torch

import gated_delta_rule_18_gb300 as gdn
from gated_delta_rule_18_gb300 import GDNError
from gated_delta_rule_18_gb300.build import build

OK, NULL, SHAPE, DTYPE, LAYOUT, UNSUP, CUDA, TIMEOUT, WS, DEVICE = range(10)
A = 1 << 20
BIG = 1 << 40  # workspace bytes


@pytest.fixture(scope="module")
def L():
    build()
    return gdn.lib()


def call(fn, spec, **kw):
    """fn(*spec's values), with those named in kw replaced."""
    unknown = set(kw) - {k for k, _ in spec}
    assert not unknown, unknown
    return fn(*[kw.get(k, v) for k, v in spec])


def p(i):
    return A * (i + 1)


NORM = [("x", p(0)), ("x_st", 64), ("x_dtype", 1), ("res", p(1)), ("res_st", 64), ("res_dtype", 0), ("w", p(2)),
        ("out", p(3)), ("out_st", 64), ("out_dtype", 1), ("ro", p(4)), ("ro_st", 64), ("scale", 0), ("R", 4), ("D", 64),
        ("group", 0), ("eps", 1e-6), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(out=0), NULL), (dict(ro=0), NULL), (dict(res=0), NULL),
    (dict(out_dtype=2), NULL), (dict(scale=p(5)), NULL), (dict(R=-1), SHAPE), (dict(D=0), SHAPE), (dict(D=16385), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(out_dtype=2, scale=p(5), group=48), SHAPE),
    (dict(x_dtype=2), DTYPE), (dict(res_dtype=7), DTYPE), (dict(out_dtype=0), DTYPE), (dict(x=p(0) + 1), LAYOUT),
    (dict(res=p(1) + 2), LAYOUT), (dict(x_st=-64), LAYOUT), (dict(out_dtype=2, scale=p(5) + 1), LAYOUT), (dict(R=0), OK),
])
def test_rmsnorm_fwd_refuses(L, kw, code):
    assert call(L.gdn_rmsnorm_fwd, NORM, **kw) == code


NORM_BWD = [("s", p(0)), ("s_st", 64), ("s_dtype", 1), ("dy", p(1)), ("dy_st", 64), ("dy_dtype", 1), ("dres", 0),
            ("dres_st", 0), ("w", p(2)), ("dx", p(3)), ("dx_st", 64), ("dw", p(4)), ("R", 4), ("D", 64), ("eps", 1e-6),
            ("ws", p(5)), ("ws_bytes", BIG), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(s=0), NULL), (dict(dy=0), NULL), (dict(dw=0), NULL), (dict(D=20000), SHAPE), (dict(dy_dtype=2), DTYPE),
    (dict(dx=p(3) + 1), LAYOUT), (dict(dw=p(4) + 2), LAYOUT), (dict(ws=0), WS), (dict(ws_bytes=100), WS),
    (dict(ws=p(5) + 16), WS),
])
def test_rmsnorm_bwd_refuses(L, kw, code):
    assert call(L.gdn_rmsnorm_bwd, NORM_BWD, **kw) == code
    assert L.gdn_rmsnorm_bwd_workspace_size(4, 0) == 0 and L.gdn_rmsnorm_bwd_workspace_size(-1, 64) == 0


CONV = [("x", p(0)), ("x_sb", 6400), ("x_st", 64), ("w", p(1)), ("W", 4), ("b", p(2)), ("init", p(3)), ("cu", 0), ("n_seq", 2),
        ("out", p(4)), ("o_sb", 6400), ("o_st", 64), ("final", p(5)), ("B", 2), ("T", 100), ("D", 64), ("dtype", 1), ("flags", 1),
        ("ws", 0), ("ws_bytes", 0), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(out=0), NULL), (dict(W=1), SHAPE), (dict(W=9), SHAPE), (dict(B=0), SHAPE),
    (dict(n_seq=3), SHAPE), (dict(T=-1), SHAPE), (dict(D=0), SHAPE), (dict(cu=p(6)), SHAPE),
    (dict(cu=p(6), B=1, n_seq=0), SHAPE), (dict(dtype=2), DTYPE), (dict(flags=2), UNSUP), (dict(out=p(0)), UNSUP),
    (dict(final=p(3)), UNSUP), (dict(x=p(0) + 1), LAYOUT), (dict(x_st=-1), LAYOUT), (dict(b=p(2) + 2), LAYOUT),
    (dict(cu=p(6), B=1, n_seq=3), WS), (dict(cu=p(6), B=1, n_seq=3, ws=p(7), ws_bytes=8), WS),
    (dict(cu=p(6) + 2, B=1, n_seq=3, ws=p(7), ws_bytes=256), LAYOUT),
])
def test_conv_fwd_refuses(L, kw, code):
    assert call(L.gdn_conv_fwd, CONV, **kw) == code


CONV_BWD = [("x", p(0)), ("x_sb", 6400), ("x_st", 64), ("w", p(1)), ("W", 4), ("b", p(2)), ("init", p(3)), ("cu", 0),
            ("n_seq", 2), ("dout", p(4)), ("do_sb", 6400), ("do_st", 64), ("dfinal", p(5)), ("dx", p(6)), ("dw", p(7)),
            ("db", p(8)), ("dinit", p(9)), ("B", 2), ("T", 100), ("D", 64), ("dtype", 1), ("flags", 1), ("ws", p(10)),
            ("ws_bytes", BIG), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(dout=0), NULL), (dict(dx=0), NULL), (dict(dw=0), NULL), (dict(W=10), SHAPE), (dict(n_seq=1), SHAPE),
    (dict(dtype=5), DTYPE), (dict(flags=4), UNSUP), (dict(dw=p(7) + 1), LAYOUT), (dict(dout=p(4) + 1), LAYOUT),
    (dict(ws=0), WS), (dict(ws_bytes=256), WS),
])
def test_conv_bwd_refuses(L, kw, code):
    assert call(L.gdn_conv_bwd, CONV_BWD, **kw) == code
    assert L.gdn_conv_bwd_workspace_size(1, 1, 1, 1) == 0 and L.gdn_conv_bwd_workspace_size(0, 1, 1, 4) == 0


CONV_STEP = [("x", p(0)), ("x_st", 64), ("w", p(1)), ("W", 4), ("b", 0), ("state", p(2)), ("slots", p(3)), ("n_slots", 8),
             ("out", p(4)), ("out_st", 64), ("n", 3), ("D", 64), ("dtype", 1), ("flags", 1), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(state=0), NULL), (dict(out=0), NULL), (dict(n=-1), SHAPE), (dict(n=70000), SHAPE),
    (dict(slots=0, n=9), SHAPE), (dict(n_slots=-1), SHAPE), (dict(W=0), SHAPE), (dict(dtype=3), DTYPE), (dict(flags=8), UNSUP),
    (dict(state=p(2) + 1), LAYOUT), (dict(slots=p(3) + 1), LAYOUT), (dict(n=0), OK),
])
def test_conv_step_refuses(L, kw, code):
    assert call(L.gdn_conv_step, CONV_STEP, **kw) == code


def act(name, i):
    return [(name, p(i)), (name + "_sb", 6400), (name + "_st", 64)]


SCAN = (act("x", 0) + act("dt", 1) + [("A", p(2))] + act("bm", 3) + act("cm", 4) + [("Dv", p(5))] + act("z", 6) +
        [("bias", p(7)), ("h0", p(8)), ("cu", 0), ("n_seq", 2)])
SSM = SCAN + act("out", 9) + [("h_final", p(10)), ("B", 2), ("T", 100), ("D", 64), ("N", 16), ("dtype", 1), ("flags", 1),
                              ("ws", p(11)), ("ws_bytes", BIG), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(dt=0), NULL), (dict(A=0), NULL), (dict(bm=0), NULL), (dict(cm=0), NULL), (dict(out=0), NULL),
    (dict(N=0), SHAPE), (dict(N=129), SHAPE), (dict(D=0), SHAPE), (dict(B=0), SHAPE), (dict(n_seq=1), SHAPE),
    (dict(cu=p(12)), SHAPE), (dict(T=-1), SHAPE), (dict(dtype=2), DTYPE), (dict(flags=2), UNSUP), (dict(h_final=p(8)), UNSUP),
    (dict(x=p(0) + 1), LAYOUT), (dict(bm=p(3) + 1), LAYOUT), (dict(z_st=-8), LAYOUT), (dict(A=p(2) + 2), LAYOUT),
    (dict(h_final=p(10) + 1), LAYOUT), (dict(ws=0), WS), (dict(ws_bytes=16), WS), (dict(ws=p(11) + 8), WS),
])
def test_ssm_fwd_refuses(L, kw, code):
    assert call(L.gdn_ssm_fwd, SSM, **kw) == code


SSM_BWD = SCAN + act("dout", 9) + [("dh_final", p(10)), ("dx", p(11)), ("ddt", p(12)), ("dA", p(13)), ("dbm", p(14)),
                                   ("dcm", p(15)), ("dD", p(16)), ("dz", p(17)), ("dbias", p(18)), ("dh0", p(19)), ("B", 2),
                                   ("T", 100), ("D", 64), ("N", 16), ("dtype", 1), ("flags", 1), ("ws", p(20)),
                                   ("ws_bytes", BIG), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(dout=0), NULL), (dict(dx=0), NULL), (dict(ddt=0), NULL), (dict(dA=0), NULL), (dict(dbm=0), NULL),
    (dict(z=0), NULL), (dict(N=200), SHAPE), (dict(n_seq=3), SHAPE), (dict(dtype=9), DTYPE), (dict(flags=16), UNSUP),
    (dict(dx=p(11) + 1), LAYOUT), (dict(dcm=p(15) + 1), LAYOUT), (dict(dh0=p(19) + 2), LAYOUT), (dict(ws=0), WS),
    (dict(ws_bytes=4096), WS),
])
def test_ssm_bwd_refuses(L, kw, code):
    assert call(L.gdn_ssm_bwd, SSM_BWD, **kw) == code


STEP = [("x", p(0)), ("x_st", 64), ("dt", p(1)), ("dt_st", 64), ("A", p(2)), ("bm", p(3)), ("bm_st", 16), ("cm", p(4)),
        ("cm_st", 16), ("Dv", 0), ("z", 0), ("z_st", 0), ("bias", 0), ("state", p(5)), ("slots", p(6)), ("n_slots", 8),
        ("out", p(7)), ("out_st", 64), ("n", 3), ("D", 64), ("N", 16), ("dtype", 1), ("flags", 1), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(A=0), NULL), (dict(state=0), NULL), (dict(N=0), SHAPE), (dict(N=130), SHAPE),
    (dict(slots=0, n=9), SHAPE), (dict(n=65536), SHAPE), (dict(dtype=2), DTYPE), (dict(flags=2), UNSUP),
    (dict(state=p(5) + 2), LAYOUT), (dict(bm=p(3) + 1), LAYOUT), (dict(n=0), OK),
])
def test_ssm_step_refuses(L, kw, code):
    assert call(L.gdn_ssm_step, STEP, **kw) == code


def test_workspace_sizes(L):
    assert L.gdn_ssm_workspace_size(1, 10, 64, 129, 1, 0) == 0 and L.gdn_ssm_workspace_size(2, 10, 64, 16, 1, 0) == 0
    assert L.gdn_ssm_workspace_size(2, 10, 64, 16, 2, 1) == 0
    small, large = L.gdn_ssm_bwd_workspace_size(1, 64, 64, 16, 1, 0), L.gdn_ssm_bwd_workspace_size(4, 4096, 64, 16, 4, 0)
    assert 0 < small < large
    # one line of few channels is cut into chunks whose states lie in the workspace; many channels need none
    assert L.gdn_ssm_workspace_size(1, 32768, 2048, 16, 1, 0) > 1 << 20
    assert L.gdn_ssm_workspace_size(64, 4096, 4096, 16, 64, 0) <= 4096


def test_python_refuses_cpu_tensors_before_anything_else():
    x = torch.zeros(2, 8)
    w = torch.ones(8)
    for f in (lambda: gdn.gdn_rmsnorm_fwd(x, w), lambda: gdn.gdn_rmsnorm_bwd(x, w, x),
              lambda: gdn.gdn_conv_fwd(x[None], torch.ones(8, 4)),
              lambda: gdn.gdn_conv_bwd(x[None], torch.ones(8, 4), x[None]),
              lambda: gdn.gdn_conv_step(x, torch.zeros(2, 3, 8), torch.ones(8, 4)),
              lambda: gdn.gdn_ssm_fwd(x[None], x[None], torch.ones(8, 4), x[None, :, :4], x[None, :, :4]),
              lambda: gdn.gdn_ssm_bwd(x[None], x[None], torch.ones(8, 4), x[None, :, :4], x[None, :, :4], x[None]),
              lambda: gdn.gdn_ssm_step(x, x, torch.ones(8, 4), x[:, :4], x[:, :4], torch.zeros(2, 8, 4))):
        with pytest.raises(GDNError) as e:
            f()
        assert e.value.name == "GDN_ERR_LAYOUT"


@pytest.mark.gpu
def test_python_checks_shapes_types_and_layouts():
    dev = "cuda:0"
    x, w = torch.zeros(2, 6, 16, device=dev), torch.ones(16, device=dev)
    taps, a = torch.ones(16, 4, device=dev), -torch.ones(16, 8, device=dev)
    bc = torch.zeros(2, 6, 8, device=dev)
    bad_shape = [
        lambda: gdn.gdn_rmsnorm_fwd(x, w[:8]), lambda: gdn.gdn_rmsnorm_fwd(x, w, residual=x[:1]),
        lambda: gdn.gdn_rmsnorm_bwd(x, w, x[:1]), lambda: gdn.gdn_conv_fwd(x, taps[:8]),
        lambda: gdn.gdn_conv_fwd(x, taps, bias=w[:3]), lambda: gdn.gdn_conv_fwd(x, taps, initial_state=x[:, :2]),
        lambda: gdn.gdn_conv_step(x[:, 0], x[:, :2], taps), lambda: gdn.gdn_ssm_fwd(x, x[:1], a, bc, bc),
        lambda: gdn.gdn_ssm_fwd(x, x, a, bc[..., :4], bc), lambda: gdn.gdn_ssm_fwd(x, x, a, bc, bc, h0=a[None]),
        lambda: gdn.gdn_ssm_bwd(x, x, a, bc, bc, x[:, :3]), lambda: gdn.gdn_ssm_step(x[:, 0], x[:, 0], a, bc[:, 0], bc[:, 0], a[None, :4]),
    ]
    for f in bad_shape:
        with pytest.raises(ValueError):
            f()
    bad = [
        (DTYPE, lambda: gdn.gdn_rmsnorm_fwd(x.half(), w)), (DTYPE, lambda: gdn.gdn_rmsnorm_fwd(x, w.bfloat16())),
        (DTYPE, lambda: gdn.gdn_rmsnorm_fwd(x, w, out_dtype=torch.bfloat16)), (DTYPE, lambda: gdn.gdn_conv_fwd(x.double(), taps)),
        (DTYPE, lambda: gdn.gdn_ssm_fwd(x, x.bfloat16(), a, bc, bc)), (DTYPE, lambda: gdn.gdn_ssm_fwd(x, x, a.double(), bc, bc)),
        (LAYOUT, lambda: gdn.gdn_conv_fwd(x.transpose(1, 2), torch.ones(6, 4, device=dev))),
        (LAYOUT, lambda: gdn.gdn_ssm_fwd(x, x, torch.ones(8, 16, device=dev).t(), bc, bc)),
        (LAYOUT, lambda: gdn.gdn_conv_fwd(x, taps.cpu())), (SHAPE, lambda: gdn.gdn_rmsnorm_fwd(x, w, out_dtype=torch.float8_e4m3fn, group=7)),
        (SHAPE, lambda: gdn.gdn_conv_fwd(x, torch.ones(16, 1, device=dev))),
        (DTYPE, lambda: gdn.gdn_conv_fwd(x, taps, cu_seqlens=torch.tensor([0, 6], device=dev))),
        (UNSUP, lambda: gdn.gdn_conv_fwd(x, taps, out=x)),
    ]
    for code, f in bad:
        with pytest.raises(GDNError) as e:
            f()
        assert e.value.status == code
