"""The state-space layer's operators where rounding, non-finite values, extreme
gates and layouts matter, against plain fp64 forms. Tolerances are those of
test_layer_gpu.py unless a test derives its own."""
import pytest
import torch

import gated_delta_rule_18_gb300 as gdn
from test_layer_gpu import (BF, DEV, F32, TOL_BF, TOL_F32, TOL_SCAN, built, cu_of, dev, f64, randn, ref_conv,  # noqa: F401
                            ref_norm, ref_scan, rel, scan_case, strided)

pytestmark = pytest.mark.gpu


def scan_gradients(v, do, lens=None, df=None, softplus=True, place=lambda k, t: t):
    """gdn_ssm_bwd of scan_case's tensors; place(name, tensor on the GPU) may lay them out anew."""
    a = {k: place(k, dev(t)) for k, t in v.items()}
    return gdn.gdn_ssm_bwd(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], place("dout", dev(do)), D=a.get("D"),
                           z=a.get("z"), dt_bias=a.get("dt_bias"), dt_softplus=softplus, h0=a.get("h0"),
                           cu_seqlens=dev(cu_of(lens)), dh_final=dev(df))


def ref_gradients(v, do, lens=None, df=None, softplus=True):
    leaf = {k: f64(t).requires_grad_() for k, t in v.items()}
    out, fin = ref_scan(leaf, lens, softplus)
    loss = (out * f64(do)).sum() + (0.0 if df is None else (fin * f64(df)).sum())
    return {"d" + k: g for k, g in zip(leaf, torch.autograd.grad(loss, tuple(leaf.values())))}


@pytest.mark.parametrize("N", [5, 16, 40, 100])
def test_channel_sums_of_the_scan_gradient_are_rounded_once(N):
    """dB and dC are sums over the channels in fp32, rounded once to bf16.
    All terms are positive here, so a sum's relative error is at most that of
    fp32 sums (2e-5), and the chance that it takes a value to the other side
    of a rounding boundary 2 * 2e-5 / 2^-8 = 1 %. Products cut to ten bits
    shrink every sum by some 3.4e-4 and move four to nine in a hundred."""
    v = {k: t if k == "A" else t.abs() for k, t in scan_case(1, 64, 512, N, None, BF, True, 200).items()}
    v["dt_bias"] = -v["dt_bias"] - 4
    do = randn((1, 64, 512), BF, 210).abs()
    got, ref = scan_gradients(v, do), ref_gradients(v, do)
    for k in ("dBm", "dCm"):
        assert (got[k].cpu() != ref[k].to(BF)).float().mean().item() <= 0.01, k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [5, 16, 40, 100])
def test_non_finite_values_stay_in_their_state_of_the_channel_sums(dtype, N):
    T, C, at, n = 150, 48, 70, 3
    v, do = scan_case(1, T, C, N, None, dtype, True, 220), randn((1, T, C), dtype, 230)
    clean, tol = scan_gradients(v, do), TOL_BF if dtype == BF else TOL_SCAN
    others = [i for i in range(N) if i != n]

    def same(got, key, rows, states):
        return rel(got[key][0, rows][:, states], clean[key][0, rows][:, states]) <= tol
    # B of one state: dB does not depend on it, dC of that state alone does
    bad = dict(v, Bm=v["Bm"].clone())
    bad["Bm"][0, at, n] = float("nan")
    got = scan_gradients(bad, do)
    assert same(got, "dBm", slice(0, T), slice(0, N)) and same(got, "dCm", slice(0, T), others)
    assert same(got, "dCm", slice(0, at), [n]) and got["dCm"][0, at:, n].isnan().all()
    # an output's gradient: dC of its token, dB of that token and those before
    bad_do = do.clone()
    bad_do[0, at, 10] = float("nan")
    got = scan_gradients(v, bad_do)
    rest = [t for t in range(T) if t != at]
    assert same(got, "dCm", rest, slice(0, N)) and got["dCm"][0, at].isnan().all()
    assert same(got, "dBm", slice(at + 1, T), slice(0, N)) and got["dBm"][0, :at + 1].isnan().all()
    # an infinite input: dB of its token, dC from there on
    bad = dict(v, x=v["x"].clone())
    bad["x"][0, at, 10] = float("inf")
    got = scan_gradients(bad, do)
    assert same(got, "dBm", rest, slice(0, N)) and not got["dBm"][0, at].isfinite().any()
    assert same(got, "dCm", slice(0, at), slice(0, N)) and not got["dCm"][0, at:].isfinite().any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [64, 37])  # wide rows, and rows of any alignment
def test_very_low_and_high_gates(dtype, C):
    """silu(z) -> -0 for z down to the type's lowest value, as a mask has it;
    a prompt, its continuation and the gradients agree with the definition."""
    T, N = 300, 16
    v, do = scan_case(1, T, C, N, None, dtype, True, 240), randn((1, T, C), dtype, 250)
    gates = torch.tensor([torch.finfo(dtype).min, -1e30, -1e20, -1e4, -100.0, -60.0, -45.0, -41.0, -20.0, 60.0, 1e4])
    v["z"][0, 10:10 + 11 * 20] = gates.to(dtype).repeat(20)[:, None]
    silu = f64(v["z"]) * torch.sigmoid(f64(v["z"]))
    ref, fin = ref_scan({k: f64(t) for k, t in v.items()}, None, True)
    y, _ = ref_scan({k: f64(t) for k, t in v.items() if k != "z"}, None, True)
    a = {k: dev(t) for k, t in v.items()}
    got = gdn.gdn_ssm_fwd(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], D=a["D"], z=a["z"], dt_bias=a["dt_bias"], h0=a["h0"])
    # y's error is relative to the largest y, and its gate scales it (the smallest normal number: what may be flushed)
    tol = (TOL_BF if dtype == BF else TOL_SCAN) * silu.abs() * y.abs().max() + torch.finfo(F32).tiny * y.abs().max()
    assert ((f64(got) - ref).abs() <= tol).all()
    state, steps = a["h0"].clone(), []
    for t in range(T):
        steps.append(gdn.gdn_ssm_step(a["x"][:, t], a["dt"][:, t], a["A"], a["Bm"][:, t], a["Cm"][:, t], state, D=a["D"],
                                      z=a["z"][:, t], dt_bias=a["dt_bias"]))
    assert ((f64(torch.stack(steps, 1)) - ref).abs() <= tol).all() and rel(state, fin) <= TOL_SCAN
    got, ref = scan_gradients(v, do), ref_gradients(v, do)
    for k, r in ref.items():
        act = k in ("dx", "ddt", "dBm", "dCm", "dz")
        assert rel(got[k], r) <= (TOL_BF if dtype == BF and act else TOL_SCAN), k


@pytest.mark.parametrize("C", [64, 37])
def test_outputs_in_place_of_an_input(C):
    T, N = 400, 16
    v = {k: dev(t) for k, t in scan_case(2, T, C, N, None, BF, True, 260).items()}

    def scan(out):
        return gdn.gdn_ssm_fwd(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                               h0=v["h0"], out=out)
    want = scan(None)
    for k in ("x", "dt", "z"):
        keep = v[k].clone()
        assert torch.equal(scan(v[k]), want) and torch.equal(v[k], want)
        v[k].copy_(keep)
    x, r, w = randn((700, C), BF, 270).to(DEV), randn((700, C), BF, 271).to(DEV), randn((C,), F32, 272, 0.1, 1.0).to(DEV)
    want = gdn.gdn_rmsnorm_fwd(x, w, residual=r)
    got = gdn.gdn_rmsnorm_fwd(x, w, residual=r, out=x, residual_out=r)
    assert torch.equal(got["out"], want["out"]) and torch.equal(r, want["residual"]) and got["out"] is x


# How the rows of a call's activations lie: whole tensors; slices of wider rows that keep 16-byte
# boundaries, as halves and parts of projections do; slices at odd offsets.
PLACES = {"whole": lambda t: t, "wide": lambda t: strided(t, 8, 24), "odd": strided}
places = pytest.mark.parametrize("place", PLACES)


@places
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C,N,lens", [(2, 300, 64, 16, None), (1, 700, 136, 16, [3, 0, 500, 190, 7]),
                                          (3, 260, 40, 32, None), (1, 300, 24, 64, [100, 200]), (2, 200, 16, 128, None)])
def test_scan_and_gradient_over_rows_of_any_layout(place, dtype, B, T, C, N, lens):
    """Gated, with softplus, skip, bias and states, over lines cut into chunks and runs."""
    n = B if lens is None else len(lens)
    v, do, df = scan_case(B, T, C, N, lens, dtype, True, 300), randn((B, T, C), dtype, 310), randn((n, C, N), F32, 311)
    lay = lambda k, t: PLACES[place](t) if k in ("x", "dt", "z", "Bm", "Cm", "dout") else t  # noqa: E731
    a = {k: lay(k, dev(t)) for k, t in v.items()}
    final, out = torch.full((n, C, N), float("nan"), device=DEV), lay("x", torch.zeros(B, T, C, dtype=dtype, device=DEV))
    got = gdn.gdn_ssm_fwd(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], D=a["D"], z=a["z"], dt_bias=a["dt_bias"], h0=a["h0"],
                          cu_seqlens=dev(cu_of(lens)), h_final=final, out=out)
    ref, fin = ref_scan({k: f64(t) for k, t in v.items()}, lens, True)
    assert rel(got, ref) <= (TOL_BF if dtype == BF else TOL_SCAN) and rel(final, fin) <= TOL_SCAN
    got, ref = scan_gradients(v, do, lens, df, place=lay), ref_gradients(v, do, lens, df)
    assert set(got) == set(ref)
    for k, r in ref.items():
        act = k in ("dx", "ddt", "dBm", "dCm", "dz")
        assert rel(got[k], r) <= (TOL_BF if dtype == BF and act else TOL_SCAN), k


@places
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("B,T,D,lens", [(2, 129, 264, None), (1, 333, 136, [5, 0, 200, 1, 1, 126, 0])])
def test_convolution_and_gradient_over_rows_of_any_layout(place, dtype, W, B, T, D, lens):
    n, lay = B if lens is None else len(lens), PLACES[place]
    leaf = dict(x=randn((B, T, D), dtype, 320), weight=randn((D, W), F32, 321, 0.5), bias=randn((D,), F32, 322),
                initial_state=randn((n, W - 1, D), dtype, 323))
    do, df = randn((B, T, D), dtype, 324), randn((n, W - 1, D), dtype, 325)
    v = {k: f64(t).requires_grad_() for k, t in leaf.items()}
    ref, fin = ref_conv(v["x"], v["weight"], v["bias"], v["initial_state"], lens, True)
    grad = torch.autograd.grad((ref * f64(do)).sum() + (fin * f64(df)).sum(), tuple(v.values()))
    a = {k: dev(t) for k, t in leaf.items()}
    final, out = torch.full((n, W - 1, D), float("nan"), dtype=dtype, device=DEV), lay(torch.zeros(B, T, D, dtype=dtype, device=DEV))
    kw = dict(bias=a["bias"], initial_state=a["initial_state"], cu_seqlens=dev(cu_of(lens)))
    got = gdn.gdn_conv_fwd(lay(a["x"]), a["weight"], final_state=final, out=out, **kw)
    assert rel(got, ref) <= (TOL_BF if dtype == BF else TOL_F32) and torch.equal(f64(final), fin)
    got = gdn.gdn_conv_bwd(lay(a["x"]), a["weight"], lay(dev(do)), dfinal_state=dev(df), **kw)
    for k, r in zip(v, grad):
        assert rel(got["d" + k], r) <= (TOL_BF if dtype == BF and k in ("x", "initial_state") else TOL_F32), k


@places
@pytest.mark.parametrize("ds,dy", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,D", [(700, 72), (40, 1000), (9, 4096), (5, 9000), (3, 16384)])
def test_norm_and_gradient_over_rows_of_any_layout(place, ds, dy, rows, D):
    """The norm of an input of one type with a residual stream of the other, and its gradient."""
    lay = PLACES[place]
    x, r, w = randn((rows, D), dy, 330), randn((rows, D), ds, 331, 2.0), randn((D,), F32, 332, 0.1, 1.0)
    ref_s, ref = ref_norm(x, w, r, 1e-6)
    got = gdn.gdn_rmsnorm_fwd(lay(dev(x)), dev(w), residual=lay(dev(r)), out=lay(torch.zeros(rows, D, dtype=dy, device=DEV)),
                              residual_out=lay(torch.zeros(rows, D, dtype=ds, device=DEV)))
    assert rel(got["out"], ref) <= (TOL_BF if dy == BF else TOL_F32)
    assert rel(got["residual"], ref_s) <= (TOL_BF if ds == BF else TOL_F32)
    g, q = randn((rows, D), dy, 333), randn((rows, D), ds, 334)
    u, wr = f64(r).requires_grad_(), f64(w).requires_grad_()
    loss = (ref_norm(u, wr, None, 1e-6)[1] * f64(g)).sum() + (u * f64(q)).sum()
    dx, dw = torch.autograd.grad(loss, (u, wr))
    got = gdn.gdn_rmsnorm_bwd(lay(dev(r)), dev(w), lay(dev(g)), dres=lay(dev(q)))
    assert rel(got["dx"], dx) <= (TOL_BF if ds == BF else TOL_F32) and rel(got["dweight"], dw) <= TOL_F32


@pytest.mark.parametrize("C", [64, 37])
def test_growing_states_that_no_input_has_reached_stay_zero(C):
    """A > 0 and a line that begins with zeros: a chunk's growth passes fp32's range, the zero state does not."""
    T, N = 1024, 16
    v = scan_case(1, T, C, N, None, F32, False, 340)
    v["A"], v["dt"] = v["A"].abs() * 0 + 2, torch.ones(1, T, C)
    v["x"][:, :T - 8] = 0
    ref, fin = ref_scan({k: f64(t) for k, t in v.items()}, None, False)
    final = torch.empty(1, C, N, device=DEV)
    a = {k: dev(t) for k, t in v.items()}
    got = gdn.gdn_ssm_fwd(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], dt_softplus=False, h_final=final)
    assert rel(got, ref) <= TOL_SCAN and rel(final, fin) <= TOL_SCAN
    do = randn((1, T, C), F32, 350)
    do[:, :T - 8] = 0
    got, ref = scan_gradients(v, do, softplus=False), ref_gradients(v, do, softplus=False)
    assert rel(got["dCm"], ref["dCm"]) <= TOL_SCAN


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("size", [1e-36, 1e-28, 3e-26, 1e-20, 1.0, 1e20, 1e29, 1e34])
def test_eight_bit_values_are_the_nearest_to_the_quotient(group, size):
    """out = e4m3(y / scale) with the quotient rounded to nearest, for scales of any size."""
    rows, D = 40, 4096
    x, w = randn((rows, D), F32, 360).to(DEV), (randn((D,), F32, 361, 0.1, 1.0) * size).to(DEV)
    y = gdn.gdn_rmsnorm_fwd(x, w)["out"].cpu()
    got = gdn.gdn_rmsnorm_fwd(x, w, out_dtype=torch.float8_e4m3fn, group=group)
    g = group or D
    scale = got["scale"].cpu()
    assert torch.equal(scale, y.view(rows, -1, g).abs().amax(-1) / 448)
    want = (y.view(rows, -1, g) / scale[..., None]).view(rows, D).to(torch.float8_e4m3fn)
    assert torch.equal(got["out"].cpu().float(), want.float())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("low", ["lowest", "-inf"])
@pytest.mark.parametrize("C", [64, 37])
def test_steps_masked_by_the_lowest_dt_leave_the_state(dtype, low, C):
    """softplus(dt) = 0 there: the state passes, the token's x and B have no part, and no gradient is lost."""
    T, N = 300, 16
    v, do = scan_case(1, T, C, N, None, dtype, True, 370), randn((1, T, C), dtype, 380)
    masked = torch.zeros(T, dtype=torch.bool)
    masked[20:60] = masked[128:200] = masked[299] = True
    v["dt"][0, masked] = torch.finfo(dtype).min if low == "lowest" else float("-inf")
    a = {k: dev(t) for k, t in v.items()}
    final = torch.empty(1, C, N, device=DEV)
    got = gdn.gdn_ssm_fwd(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], D=a["D"], z=a["z"], dt_bias=a["dt_bias"], h0=a["h0"],
                          h_final=final)
    v["dt"][0, masked] = -1e30  # (the reference's softplus of -inf has no gradient of its own)
    ref, fin = ref_scan({k: f64(t) for k, t in v.items()}, None, True)
    assert rel(got, ref) <= (TOL_BF if dtype == BF else TOL_SCAN) and rel(final, fin) <= TOL_SCAN
    ref = ref_gradients(v, do)
    v["dt"][0, masked] = torch.finfo(dtype).min if low == "lowest" else float("-inf")
    got = scan_gradients(v, do)
    for k, r in ref.items():
        act = k in ("dx", "ddt", "dBm", "dCm", "dz")
        assert rel(got[k], r) <= (TOL_BF if dtype == BF and act else TOL_SCAN), k
    assert (got["ddt"][0, dev(masked)] == 0).all() and (got["dBm"][0, dev(masked)] == 0).all()
