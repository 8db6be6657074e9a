"""The Python checks of the state-space layer's operators, on the CPU: tensors
that claim a GPU, and a library that records its calls instead of launching."""
import contextlib

import pytest
import torch

import gated_delta_rule_18_gb300 as gdn
from gated_delta_rule_18_gb300 import GDNError, layer

LAYOUT = "GDN_ERR_LAYOUT"
F8 = torch.float8_e4m3fn


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    index = 0
    is_cuda = True

    def get_device(self):
        return self.index

    def view(self, *shape):
        return claim(super().view(*shape), self.index)

    __torch_function__ = torch._C._disabled_torch_function_impl


def claim(t, index=0):
    t = t.as_subclass(OnGpu)
    t.index = index
    return t


def on(index, *shape, dtype=torch.float32):
    return claim(torch.zeros(shape, dtype=dtype), index)


class Library:
    """Every entry point: returns 0 (for sizes, 1024) and notes its name and the current device."""

    def __init__(self):
        self.current, self.calls = 0, []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, self.current))
            return 1024 if name.endswith("_size") else 0
        return entry

    @property
    def launched(self):
        return [(n, d) for n, d in self.calls if not n.endswith("_size")]


@pytest.fixture
def L(monkeypatch):
    lib = Library()
    monkeypatch.setattr(layer, "_lib", lib)
    monkeypatch.setattr(layer, "_stream", lambda like: 0)
    monkeypatch.setattr(layer, "_current_device", lambda: lib.current)
    return lib


def refused(L, name, f):
    with pytest.raises(GDNError) as e:
        f()
    assert e.value.name == name
    assert L.launched == []


@pytest.mark.parametrize("q8", [False, True])
def test_norm_output_on_another_device_is_refused(L, q8):
    x, w = on(0, 4, 64), on(0, 64)
    kw = dict(out_dtype=F8) if q8 else {}
    ty = F8 if q8 else x.dtype
    refused(L, LAYOUT, lambda: gdn.gdn_rmsnorm_fwd(x, w, out=torch.zeros(4, 64).to(ty), **kw))
    refused(L, LAYOUT, lambda: gdn.gdn_rmsnorm_fwd(x, w, out=on(1, 4, 64, dtype=ty), **kw))
    gdn.gdn_rmsnorm_fwd(x, w, out=on(0, 4, 64, dtype=ty), **kw)
    assert len(L.launched) == 1


def packed(index):
    """The calls that take a workspace, on a packed batch."""
    x, cu = on(index, 1, 6, 16), on(index, 3, dtype=torch.int32)
    taps, a, bc = on(index, 16, 4), on(index, 16, 8), on(index, 1, 6, 8)
    out = on(index, 1, 6, 16)
    return [
        lambda **k: gdn.gdn_rmsnorm_bwd(x, on(index, 16), x, **k),
        lambda **k: gdn.gdn_conv_fwd(x, taps, cu_seqlens=cu, out=out, **k),
        lambda **k: gdn.gdn_conv_bwd(x, taps, out, cu_seqlens=cu, **k),
        lambda **k: gdn.gdn_ssm_fwd(x, x, a, bc, bc, cu_seqlens=cu, out=out, **k),
        lambda **k: gdn.gdn_ssm_bwd(x, x, a, bc, bc, out, cu_seqlens=cu, **k),
    ]


@pytest.mark.parametrize("call", range(5))
def test_workspace_on_another_device_or_with_gaps_is_refused(L, call):
    f = packed(0)[call]
    plain = torch.zeros(1 << 16, dtype=torch.uint8)
    for ws in (plain, claim(plain, 1), claim(plain[::2])):
        refused(L, LAYOUT, lambda: f(workspace=ws))
    f(workspace=on(0, 1 << 16, dtype=torch.uint8))
    f()
    assert len(L.launched) == 2


def calls(index):
    """Every call of the layer on tensors of a device, outputs given where the call takes them."""
    x, w, taps, a, bc = on(index, 4, 16), on(index, 16), on(index, 16, 4), on(index, 16, 8), on(index, 4, 8)
    out = on(index, 4, 16)
    step = [
        lambda **k: gdn.gdn_rmsnorm_fwd(x, w, out=out, **k),
        lambda **k: gdn.gdn_conv_step(x, on(index, 4, 3, 16), taps, out=out, **k),
        lambda **k: gdn.gdn_ssm_step(x, x, a, bc, bc, on(index, 4, 16, 8), out=out, **k),
    ]
    return step + packed(index)


class FakeStream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.mark.parametrize("call", range(8))
def test_calls_run_on_the_device_of_their_tensors(L, monkeypatch, call):
    @contextlib.contextmanager
    def device(d):
        before, L.current = L.current, d.index if isinstance(d, torch.device) else d
        yield
        L.current = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: device(s.device))
    calls(1)[call]()
    calls(0)[call]()
    calls(1)[call](stream=FakeStream(1))
    assert [d for _, d in L.launched] == [1, 0, 1] and L.current == 0
    L.calls.clear()
    refused(L, LAYOUT, lambda: calls(1)[call](stream=FakeStream(0)))
    refused(L, LAYOUT, lambda: calls(0)[call](stream=FakeStream(1)))


def test_tensors_written_in_place_count_a_version(L):
    """A tensor saved for a gradient and then overwritten by a call is noticed."""
    x, w, taps, a, bc = on(0, 4, 16), on(0, 16), on(0, 16, 4), on(0, 16, 8), on(0, 4, 8)
    line, rows = on(0, 4, 1, 16), on(0, 4, 1, 8)
    res, window, h = on(0, 4, 16), on(0, 4, 3, 16), on(0, 4, 16, 8)
    out, out3 = on(0, 4, 16), on(0, 4, 1, 16)
    for written, f in (
            ([out, res], lambda: gdn.gdn_rmsnorm_fwd(x, w, residual=res, residual_out=res, out=out)),
            ([out3, window], lambda: gdn.gdn_conv_fwd(line, taps, final_state=window, out=out3)),
            ([out, window], lambda: gdn.gdn_conv_step(x, window, taps, out=out)),
            ([out3, h], lambda: gdn.gdn_ssm_fwd(line, line, a, rows, rows, h_final=h, out=out3)),
            ([out, h], lambda: gdn.gdn_ssm_step(x, x, a, bc, bc, h, out=out))):
        before = [t._version for t in written]
        f()
        assert all(t._version > b for t, b in zip(written, before))
    assert [t._version for t in (x, w, taps, a, bc, line, rows)] == [0] * 7
    leaf = torch.ones(4, 16, requires_grad=True)
    h = on(0, 4, 16, 8)
    loss = (leaf[..., None] * h).sum()
    gdn.gdn_ssm_step(x, x, a, bc, bc, h, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", ["rms_norm", "causal_conv", "selective_scan"])
def test_second_derivatives_are_refused(monkeypatch, name):
    """The gradient calls are not differentiable: a loss of a gradient raises instead of missing its part."""
    from gated_delta_rule_18_gb300 import autograd as gdr

    def gradients(x, *args, **kw):
        return {k: torch.ones_like(x) for k in ("dx", "ddt", "dBm", "dCm")} | {"dweight": torch.ones(16), "dA": torch.ones(16, 8)}
    for k in ("gdn_rmsnorm", "gdn_conv", "gdn_ssm"):
        monkeypatch.setattr(gdr, k + "_fwd", lambda x, *a, **kw: {"out": x * 2} if kw.get("eps") else x * 2)
        monkeypatch.setattr(gdr, k + "_bwd", gradients)
    x, w, a = torch.randn(1, 4, 16, requires_grad=True), torch.ones(16), torch.ones(16, 8)
    y = {"rms_norm": lambda: gdr.rms_norm(x, w)[0], "causal_conv": lambda: gdr.causal_conv(x, torch.ones(16, 4))[0],
         "selective_scan": lambda: gdr.selective_scan(x, x, a, x.detach()[..., :8], x.detach()[..., :8])[0]}[name]()
    for loss in (y.sum(), y.square().sum()):
        (g,) = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError, match="not differentiable"):
            (g.square().sum() + loss).backward(retain_graph=True)
    y.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0 if name == "selective_scan" else 1.0))


def tall(*shape, dtype=torch.float32):
    """A tensor of any size in a few bytes (stride 0)."""
    return claim(torch.zeros((1,) * len(shape), dtype=dtype).expand(*shape))


@pytest.mark.parametrize("n", [2**31, 2**32 + 4])
def test_sizes_past_32_bits_are_refused_and_not_cut(L, n):
    """The library's sizes are 32-bit: a larger one must not arrive as its low half."""
    x, out = tall(n, 1), tall(n, 1)
    line, w, taps, a = tall(1, n, 1), on(0, 1), on(0, 1, 4), on(0, 1, 8)
    rows = tall(1, n, 8)
    for f in (lambda: gdn.gdn_rmsnorm_fwd(x, w, out=out),
              lambda: gdn.gdn_rmsnorm_fwd(on(0, 4, 64), on(0, 64), out_dtype=F8, group=2**32 + 32,
                                          out=on(0, 4, 64, dtype=F8)),
              lambda: gdn.gdn_rmsnorm_bwd(x, w, out),
              lambda: gdn.gdn_conv_fwd(line, taps, out=line),
              lambda: gdn.gdn_conv_bwd(line, taps, line),
              lambda: gdn.gdn_conv_step(x, on(0, 1, 3, 1), taps, out=out),
              lambda: gdn.gdn_conv_step(on(0, 4, 1), tall(n, 3, 1), taps, out=on(0, 4, 1)),
              lambda: gdn.gdn_conv_fwd(on(0, 1, 4, 1), tall(1, n), out=on(0, 1, 4, 1)),
              lambda: gdn.gdn_ssm_fwd(line, line, a, rows, rows, out=line),
              lambda: gdn.gdn_ssm_bwd(line, line, a, rows, rows, line),
              lambda: gdn.gdn_ssm_step(x, x, a, tall(n, 8), tall(n, 8), on(0, 4, 1, 8), out=out)):
        with pytest.raises(ValueError, match="2147483647"):
            f()
    assert L.launched == []


def test_lengths_whose_sums_would_pass_32_bits_are_refused():
    """Kernels and workspace sizes add a tile's or a group's tokens to T and R: room for that is kept."""
    from gated_delta_rule_18_gb300.build import build
    from test_layer_abi import CONV, CONV_BWD, NORM, NORM_BWD, SHAPE, SSM, SSM_BWD, call
    build()
    lib, most = gdn.lib(), 2**31 - 1
    for fn, spec, kw in ((lib.gdn_rmsnorm_fwd, NORM, dict(R=most)), (lib.gdn_rmsnorm_bwd, NORM_BWD, dict(R=most)),
                         (lib.gdn_conv_fwd, CONV, dict(T=most)), (lib.gdn_conv_bwd, CONV_BWD, dict(T=most)),
                         (lib.gdn_ssm_fwd, SSM, dict(T=most)), (lib.gdn_ssm_bwd, SSM_BWD, dict(T=most))):
        assert call(fn, spec, **kw) == SHAPE, fn
    assert lib.gdn_rmsnorm_bwd_workspace_size(most, 64) == 0 and lib.gdn_conv_bwd_workspace_size(1, most, 64, 4) == 0
    assert lib.gdn_ssm_workspace_size(1, most, 64, 16, 1, 0) == 0
    assert lib.gdn_ssm_bwd_workspace_size(1, most, 64, 16, 1, 0) == 0
    long = 2**31 - 2**16
    assert lib.gdn_conv_bwd_workspace_size(1, long, 64, 4) > 0 and lib.gdn_rmsnorm_bwd_workspace_size(long, 64) > 0
    assert lib.gdn_ssm_bwd_workspace_size(1, long, 64, 16, 1, 0) > 2**31


def test_tensors_of_too_few_dimensions_raise_value_errors(L):
    line, x, w, one = on(0, 1, 4, 16), on(0, 4, 16), on(0, 16), on(0)
    taps, a, bc, rows = on(0, 16, 4), on(0, 16, 8), on(0, 4, 8), on(0, 1, 4, 8)
    for f in (lambda: gdn.gdn_rmsnorm_fwd(one, w), lambda: gdn.gdn_rmsnorm_bwd(one, w, one),
              lambda: gdn.gdn_conv_fwd(line, w), lambda: gdn.gdn_conv_bwd(line, w, line),
              lambda: gdn.gdn_conv_step(x, on(0, 4, 3, 16), w), lambda: gdn.gdn_conv_step(x, one, taps),
              lambda: gdn.gdn_ssm_fwd(line, line, w, rows, rows), lambda: gdn.gdn_ssm_bwd(line, line, w, rows, rows, line),
              lambda: gdn.gdn_ssm_step(x, x, w, bc, bc, on(0, 4, 16, 8)), lambda: gdn.gdn_ssm_step(x, x, a, bc, bc, one),
              lambda: gdn.gdn_conv_fwd(x, taps), lambda: gdn.gdn_ssm_step(line, x, a, bc, bc, on(0, 4, 16, 8))):
        with pytest.raises(ValueError):
            f()
    assert L.launched == []


@pytest.mark.parametrize("outside", [False, True])
def test_calls_run_in_inference_mode(L, outside):
    """Inference tensors have no version to count; others written there count theirs."""
    h, x, bc, out = (on(0, *s) for s in ((4, 16, 8), (4, 16), (4, 8), (4, 16)))
    with torch.inference_mode():
        if not outside:
            h, x, bc, out = (on(0, *s) for s in ((4, 16, 8), (4, 16), (4, 8), (4, 16)))
        assert gdn.gdn_ssm_step(x, x, on(0, 16, 8), bc, bc, h, out=out) is out
    assert len(L.launched) == 1 and (not outside or h._version == 1)
