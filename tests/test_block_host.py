"""The Python checks of the block's operators, on the CPU: tensors that claim a
GPU, and a library that records its calls instead of launching; and the
frequencies of rotary positions."""
import contextlib
import math

import pytest
import torch

import gated_delta_rule_18_gb300 as gdn
from gated_delta_rule_18_gb300 import GDNError
from test_layer_host import LAYOUT, FakeStream, L, claim, on, refused, tall  # noqa: F401

BF = torch.bfloat16


def tensors(index):
    """One valid call of each operator on tensors of a device, outputs given where the call takes them."""
    q, k, f = on(index, 2, 6, 4, 16), on(index, 2, 6, 2, 16), on(index, 4, dtype=torch.float64)
    y, w = on(index, 2, 6, 16), on(index, 16)
    rows, state = on(index, 4, 16), on(index, 5, 16)
    return {
        "rotary": (gdn.gdn_rotary, (q, f), dict(k=k, positions=on(index, 2, 6, dtype=torch.int32), out=q, k_out=k)),
        "block_fwd": (gdn.gdn_block_norm_fwd, (y, on(index, 2, 6, 16)),
                      dict(post_weight=w, pre_weight=w, gate=on(index, 2, 1, 16), gate_act="silu", scale=w,
                           residual_out=on(index, 2, 6, 16), out=on(index, 2, 6, 16))),
        "block_bwd": (gdn.gdn_block_norm_bwd, (y, y), dict(dout=y, dres=y, post_weight=w, pre_weight=w, gate=y, scale=w)),
        "lru_fwd": (gdn.gdn_lru_fwd, (y, y, y, w), dict(z=y, h0=on(index, 2, 16), h_final=on(index, 2, 16),
                                                        checkpoints=on(index, 2, 1, 16), out=on(index, 2, 6, 16))),
        "lru_bwd": (gdn.gdn_lru_bwd, (y, y, y, w, y), dict(z=y, h0=on(index, 2, 16), dh_final=on(index, 2, 16),
                                                           checkpoints=on(index, 2, 1, 16))),
        "lru_step": (gdn.gdn_lru_step, (rows, rows, rows, w, state), dict(z=rows, slots=on(index, 4, dtype=torch.int32),
                                                                          out=on(index, 4, 16))),
    }


NAMES = list(tensors(0))


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_checked(L, monkeypatch, name):  # noqa: F811
    """Each tensor in turn on another device, of another type, of another shape, with a strided last dimension."""
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext(setattr(L, "current", d)))
    f, args, kw = tensors(0)[name]
    f(*args, **kw)
    assert len(L.launched) == 1
    L.calls.clear()
    places = [("arg", i) for i in range(len(args))] + [("kw", k) for k, v in kw.items() if isinstance(v, torch.Tensor)]

    def with_one(place, t):
        a, k = list(args), dict(kw)
        if place[0] == "arg":
            a[place[1]] = t
        else:
            k[place[1]] = t
        return lambda: f(*a, **k)

    for place in places:
        t = args[place[1]] if place[0] == "arg" else kw[place[1]]
        plain = t.as_subclass(torch.Tensor)
        wrong = [claim(plain.clone(), 1), plain.clone(), claim(plain.to(torch.float16 if t.dtype != torch.int32 else torch.int16)),
                 claim(torch.zeros(tuple(plain.shape) + (2,), dtype=t.dtype)),
                 claim(torch.zeros(tuple(n + 1 for n in plain.shape), dtype=t.dtype)),
                 claim(torch.zeros(tuple(plain.shape[:-1]) + (2 * plain.shape[-1],), dtype=t.dtype)[..., ::2])]
        if place == ("kw", "positions"):
            wrong.pop()  # positions may have any strides
        if name == "rotary" and place == ("arg", 1):
            wrong.pop(4)  # more frequencies turn more channels
        if place == ("arg", 0) or (name == "lru_step" and place == ("arg", 4)):
            wrong.pop(4)  # a larger pool or batch is what the other tensors are held against
            if name == "lru_step" and place == ("arg", 4):
                wrong.append(claim(torch.zeros(5, 17)))
        for t in wrong:
            L.current = 0
            with pytest.raises((GDNError, ValueError)):
                with_one(place, t)()
            assert L.launched == [], (place, t.shape, t.dtype)


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_the_device_of_their_tensors(L, monkeypatch, name):  # noqa: F811
    @contextlib.contextmanager
    def device(d):
        before, L.current = L.current, d.index if isinstance(d, torch.device) else d
        yield
        L.current = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: device(s.device))
    for index, stream in ((1, None), (0, None), (1, FakeStream(1))):
        f, args, kw = tensors(index)[name]
        f(*args, **kw, **({} if stream is None else {"stream": stream}))
    assert [d for _, d in L.launched] == [1, 0, 1] and L.current == 0
    L.calls.clear()
    f, args, kw = tensors(1)[name]
    refused(L, LAYOUT, lambda: f(*args, **kw, stream=FakeStream(0)))


def test_tensors_written_in_place_count_a_version(L):  # noqa: F811
    for name, written in (("rotary", ("out", "k_out")), ("block_fwd", ("residual_out", "out")),
                          ("lru_fwd", ("h_final", "checkpoints", "out")), ("lru_step", ("out",))):
        f, args, kw = tensors(0)[name]
        tracked = [kw[k] for k in written] + ([args[4]] if name == "lru_step" else [])
        before = [t._version for t in tracked]
        f(*args, **kw)
        assert all(t._version > b for t, b in zip(tracked, before)), name


@pytest.mark.parametrize("name", ["block_bwd", "lru_bwd", "lru_fwd"])
def test_workspace_on_another_device_or_with_gaps_is_refused(L, name):  # noqa: F811
    f, args, kw = tensors(0)[name]
    if name == "lru_fwd":  # only a packed batch takes one
        y, w = on(0, 1, 6, 16), on(0, 16)
        args, kw = (y, y, y, w), dict(cu_seqlens=on(0, 3, dtype=torch.int32))
    plain = torch.zeros(1 << 16, dtype=torch.uint8)
    for ws in (plain, claim(plain, 1), claim(plain[::2])):
        refused(L, LAYOUT, lambda: f(*args, **kw, workspace=ws))
    f(*args, **kw, workspace=on(0, 1 << 16, dtype=torch.uint8))
    assert len(L.launched) == 1


def test_calls_that_do_not_go_together_are_refused(L):  # noqa: F811
    q, k, f = on(0, 2, 6, 4, 16), on(0, 2, 6, 2, 16), on(0, 4, dtype=torch.float64)
    y, w = on(0, 2, 6, 16), on(0, 16)
    for call in (
            lambda: gdn.gdn_rotary(q, f, k_out=k), lambda: gdn.gdn_rotary(q, f, positions=on(0, 5, dtype=torch.int32)),
            lambda: gdn.gdn_rotary(q, f, positions=on(0, 2, 1, dtype=torch.int64)), lambda: gdn.gdn_rotary(q, f, offset=2**63),
            lambda: gdn.gdn_rotary(on(0, 6, 4, 16), f), lambda: gdn.gdn_rotary(q, f, k=on(0, 6, 2, 16)),
            lambda: gdn.gdn_block_norm_fwd(y, y), lambda: gdn.gdn_block_norm_fwd(y, y, post_weight=w, out=on(0, 2, 6, 16)),
            lambda: gdn.gdn_block_norm_fwd(y, y, post_weight=w, gate_act="silu"),
            lambda: gdn.gdn_block_norm_fwd(y, y, post_weight=w, gate=y, gate_act="relu"),
            lambda: gdn.gdn_block_norm_fwd(y, y, post_weight=w, gate=on(0, 1, 1, 16)),
            lambda: gdn.gdn_block_norm_fwd(on(0, 12, 16), on(0, 12, 16), post_weight=w, gate=on(0, 1, 16)),
            lambda: gdn.gdn_block_norm_fwd(on(0), on(0), post_weight=w),
            lambda: gdn.gdn_block_norm_bwd(y, y, dres=y, pre_weight=w), lambda: gdn.gdn_block_norm_bwd(y, y, dout=y, post_weight=w),
            lambda: gdn.gdn_block_norm_bwd(y, y, post_weight=w), lambda: gdn.gdn_block_norm_bwd(y, y, dres=y),
            lambda: gdn.gdn_lru_fwd(on(0, 12, 16), y, y, w), lambda: gdn.gdn_lru_step(y, y, y, w, on(0, 4, 16)),
            lambda: gdn.gdn_lru_step(on(0, 4, 16), on(0, 4, 16), on(0, 4, 16), w, w),
            lambda: gdn.gdn_lru_fwd(y, y, y, w, checkpoints=on(0, 2, 2, 16))):
        with pytest.raises(ValueError):
            call()
    assert L.launched == []


@pytest.mark.parametrize("n", [2**31, 2**32 + 4])
def test_sizes_past_32_bits_are_refused_and_not_cut(L, n):  # noqa: F811
    f, w = on(0, 1, dtype=torch.float64), on(0, 1)
    line, rows, heads = tall(1, n, 1), tall(n, 1), tall(1, n, 1, 2)
    for call in (lambda: gdn.gdn_rotary(heads, f, out=heads), lambda: gdn.gdn_rotary(tall(1, 1, n, 2), f, out=tall(1, 1, n, 2)),
                 lambda: gdn.gdn_rotary(on(0, 1, 1, 1, 2), f, k=tall(1, 1, n, 2)),
                 lambda: gdn.gdn_rotary(on(0, 1, 1, 1, 2), tall(n, dtype=torch.float64)),
                 lambda: gdn.gdn_block_norm_fwd(rows, rows, post_weight=w, residual_out=rows),
                 lambda: gdn.gdn_block_norm_bwd(rows, rows, dres=rows, post_weight=w),
                 lambda: gdn.gdn_lru_fwd(line, line, line, w, out=line), lambda: gdn.gdn_lru_bwd(line, line, line, w, line),
                 lambda: gdn.gdn_lru_step(rows, rows, rows, w, rows, out=rows),
                 lambda: gdn.gdn_lru_step(on(0, 4, 1), on(0, 4, 1), on(0, 4, 1), w, rows)):
        with pytest.raises(ValueError, match="at most"):
            call()
    assert L.launched == []


@pytest.mark.parametrize("name", ["rotary", "block_norm", "gated_recurrence"])
def test_second_derivatives_are_refused(monkeypatch, name):
    from gated_delta_rule_18_gb300 import autograd as gdr

    def gradients(x, *args, **kw):
        return {k: torch.ones_like(x) for k in ("dx", "dr", "di", "dy", "dresidual")} | {k: torch.ones(16) for k in ("dlam", "dpost_weight")}
    monkeypatch.setattr(gdr, "gdn_rotary", lambda q, f, k=None, **kw: q * 2 if k is None else (q * 2, k * 2))
    monkeypatch.setattr(gdr, "gdn_block_norm_fwd", lambda y, r, **kw: {"residual": y * 2 + r})
    monkeypatch.setattr(gdr, "gdn_lru_fwd", lambda x, *a, **kw: x * 2)
    for k in ("gdn_block_norm_bwd", "gdn_lru_bwd"):
        monkeypatch.setattr(gdr, k, gradients)
    x, w = torch.randn(1, 4, 16, requires_grad=True), torch.ones(16)
    y = {"rotary": lambda: gdr.rotary(x[None], torch.ones(4, dtype=torch.float64)),
         "block_norm": lambda: gdr.block_norm(x, x.detach(), post_weight=w)[1],
         "gated_recurrence": lambda: gdr.gated_recurrence(x, x.detach(), x.detach(), w)[0]}[name]()
    for loss in (y.sum(), y.square().sum()):
        (g,) = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError, match="not differentiable"):
            (g.square().sum() + loss).backward(retain_graph=True)
    y.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0 if name == "rotary" else 1.0))


@pytest.mark.parametrize("outside", [False, True])
def test_calls_run_in_inference_mode(L, outside):  # noqa: F811
    h, x, out = (on(0, *s) for s in ((4, 16), (4, 16), (4, 16)))
    with torch.inference_mode():
        if not outside:
            h, x, out = (on(0, *s) for s in ((4, 16), (4, 16), (4, 16)))
        assert gdn.gdn_lru_step(x, x, x, on(0, 16), h, out=out) is out
    assert len(L.launched) == 1 and (not outside or h._version == 1)


def test_rotary_frequencies():
    f, s = gdn.rotary_frequencies(8, base=10000.0, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    g, s = gdn.rotary_frequencies(8, factor=4.0, device="cpu")
    assert torch.equal(g, f / 4) and s == 1.0
    # 4096 trained positions: 652, 65, 6.5 and 0.65 turns; the ramp runs from 32 turns down to one
    g, s = gdn.rotary_frequencies(8, factor=4.0, original_length=4096, device="cpu")
    keep = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    want = torch.tensor([1.0, 0.1, 0.01 * (keep + (1 - keep) / 4), 0.001 / 4], dtype=torch.float64)
    assert torch.allclose(g, want, rtol=1e-14) and s == 0.1 * math.log(4.0) + 1.0
    for kw in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=0.5),
               dict(rot=8, factor=2.0, original_length=100, beta_fast=1.0, beta_slow=1.0), dict(rot=8, base=float("nan"))):
        with pytest.raises(ValueError):
            gdn.rotary_frequencies(kw.pop("rot"), device="cpu", **kw)
