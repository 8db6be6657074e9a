"""The block's operators on the GPU at the ends of their ranges, against plain
fp64 forms: rows of very large values, non-finite values beside a sequence's
end, waits that run out, callers on two threads, far positions, lines of several
steps of a cluster, forms of rows that few calls have.

Tolerances as derived in test_block_gpu.py; others beside their tests.
"""
import math
import threading
from fractions import Fraction

import pytest
import torch

import gated_delta_rule_18_gb300 as gdn
import test_block_gpu as base
from test_block_gpu import TOL_LRU, TOL_LRU_BWD, TOL_NORM, TOL_ROT, block_inputs, decays, freqs, lru_inputs, norm, ref_block, ref_lru, ref_rotary, tol
from test_layer_gpu import BF, DEV, F32, F64, built, cu_of, dev, f64, randn, rel, spans, strided  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rotary ---


def _two_pi(bits=320):
    """2 pi by Machin's formula, to about `bits` bits."""
    def arctan(x):
        s = t = (1 << bits) // x
        n, sign = 3, -1
        while t:
            t //= x * x
            s += sign * (t // n)
            n, sign = n + 2, -sign
        return s
    return Fraction(8 * (4 * arctan(5) - arctan(239)), 1 << bits)


@pytest.mark.parametrize("p", [1, 2**30 + 1, 2**40 + 12345, 2**53 + 1, -2**53 - 1, 2**60 + 3, 2**62, -2**62, 2**63 - 1, -2**63])
def test_rotary_far_positions_of_exact_frequencies(p):
    """Frequencies as the doubles they are, reduced exactly. The kernel's 2 / pi is rounded to 64 bits: 0.0151 of its last
    place, which is 1.28e-21 of it, so the angle is 1.3e-21 |p| f radians off, beside the fp32 result's 4e-7."""
    f = torch.tensor([1.0, 0.5, 3.0, math.pi, 10000.0**-0.125, 1e-4, 1.5e-7, 2.0**-40], dtype=F64)
    x = torch.zeros(1, 1, 1, 16)
    x[..., :8] = 1.0
    got = gdn.gdn_rotary(dev(x), dev(f), positions=torch.tensor([[p]], dtype=torch.int64, device=DEV)).cpu().to(F64)[0, 0, 0]
    turn = _two_pi()
    for k in range(8):
        angle = float(p * Fraction(f[k].item()) % turn)
        bound = 4e-7 + abs(p) * f[k].item() * 1.3e-21
        assert abs(got[k] - math.cos(angle)) <= bound and abs(got[8 + k] - math.sin(angle)) <= bound, (k, bound)


@pytest.mark.parametrize("D,axes,interleaved", [(112, (32, 40, 40), True), (112, (32, 40, 40), False), (128, (64, 32, 32), True), (96, (24, 36, 36), False)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_of_several_axes(D, axes, interleaved, dtype):
    """A video's tokens by frame, row and column: each axis turns channels of its own, a call on a slice of the head, in place."""
    B, F, H, W, n = 2, 3, 5, 4, 6
    q, k = randn((B, F * H * W, n, D), dtype, 300), randn((B, F * H * W, 2, D), dtype, 301)
    at = torch.stack(torch.meshgrid(torch.arange(F), torch.arange(H), torch.arange(W), indexing="ij")).reshape(3, -1)
    gq, gk, want, c = dev(q), dev(k), [f64(q), f64(k)], 0
    for pos, rot in zip(at, axes):
        f = freqs(rot)
        a, b = (t[..., c:c + rot] for t in (gq, gk))
        gdn.gdn_rotary(a, dev(f), k=b, positions=dev(pos.to(torch.int32)), interleaved=interleaved, out=a, k_out=b)
        for t, x in zip(want, (q, k)):
            t[..., c:c + rot] = ref_rotary(x[..., c:c + rot], pos.expand(B, -1), f, interleaved, 1.0)
        c += rot
    assert rel(gq, want[0]) <= tol(dtype, TOL_ROT) and rel(gk, want[1]) <= tol(dtype, TOL_ROT)


@pytest.mark.parametrize("D,rot", [(96, 24), (80, 20), (80, 40), (112, 28), (112, 56), (64, 12), (72, 72)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_parts_off_whole_vectors(D, rot, interleaved, dtype):
    """Parts of a head whose half is not whole 16-byte vectors, of more heads and tokens than a CTA has under way."""
    B, T, Hq, Hk = 2, 150, 20, 3
    q, k, f = randn((B, T, Hq, D), dtype, 310), randn((B, T, Hk, D), dtype, 311), freqs(rot)
    pos = torch.randint(0, 1 << 20, (B, T), generator=torch.Generator().manual_seed(312))
    for t in ((dev(q), dev(k)), (strided(dev(q), 8, 8), strided(dev(k), 8, 8))):
        gq, gk = gdn.gdn_rotary(t[0], dev(f), k=t[1], positions=dev(pos), interleaved=interleaved)
        for got, x in ((gq, q), (gk, k)):
            assert rel(got, ref_rotary(x, pos, f, interleaved, 1.0)) <= tol(dtype, TOL_ROT)
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


# ------------------------------------------------------------ block norm ---


@pytest.mark.parametrize("B,T,D", [(1, 3, 5001), (2, 2, 9001), (1, 3, 4097), (1, 2, 16383)])
@pytest.mark.parametrize("form", range(len(base.FORMS)))
def test_block_norm_of_wide_rows_off_vectors(B, T, D, form):
    """Rows of two and of four vectors a thread that are taken by elements."""
    base.test_block_norm(B, T, D, form)
    base.test_block_norm_bwd(B, T, D, form)


def rows_rel(got, ref):
    """Largest error of any row, of the row's largest value."""
    got, ref = f64(got).flatten(0, -2), f64(ref).flatten(0, -2)
    assert got.isfinite().all()
    return ((got - ref).abs().amax(-1) / ref.abs().amax(-1).clamp(min=1e-300)).max().item()


@pytest.mark.parametrize("D", [8, 100, 256, 1792, 4096, 9000])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", [None, "token", "sequence"])
def test_block_norm_gradient_of_large_rows(D, dtype, gate):
    """Rows of up to the largest values whose squares' sum fp32 holds, of one value and of random ones, beside usual rows and
    rows near zero: the norms' gradients are inv gw and its projections, however small inv is. Row by row, as their sizes
    differ by 1e30; errors are those of a usual row (the scaling by a power of two adds none). Where a row's sum does pass
    fp32's range (of 9000 channels 2.5e17), it is normed to zeros and has zeros for that norm's gradients."""
    top = math.sqrt(0.9 * torch.finfo(F32).max / D)
    sizes = [1.0, 1e-12, 1e8, 1e12, 1e13, 1e14, 1e15, 1e16, 1e17, 1e18 if D <= 256 else 2.5e17, top]
    T = 2 * len(sizes)
    y, r, wp, wn, g, _ = block_inputs(1, T, D, dtype, dtype, True, True, gate, False, seed=200)
    do, dr = randn((1, T, D), dtype, 210, 1.5), randn((1, T, D), dtype, 211)
    for t in (y, r):
        for k, v in enumerate(sizes):
            t[0, 2 * k] = -v * 0.99                                                       # padding of one value
            t[0, 2 * k + 1] = (t[0, 2 * k + 1].float().clamp(-4, 4) * (v / 4)).to(dtype)  # (sum of squares below the constant row's)
    kw = dict(post_weight=dev(wp), pre_weight=dev(wn), gate=dev(g), gate_act=None if gate is None else "sigmoid")
    # the stream's norm alone, at large s and usual y; then y's norm alone, at large y and usual s
    usual, small = block_inputs(1, T, D, dtype, dtype, True, True, gate, False, seed=220)[:2]
    for yy, s, dres in ((usual, r, None), (y, small, dr)):
        none = {k: f64(t).square().sum(-1, keepdim=True) > torch.finfo(F32).max for k, t in dict(y=yy, s=s).items()}
        leaf = {k: f64(t).requires_grad_() for k, t in dict(y=yy, s=s, wp=wp, wn=wn, g=g).items() if t is not None}
        t, _ = ref_block(leaf["y"].masked_fill(none["y"], 0), torch.zeros(1, T, D, dtype=F64), leaf["wp"], None, leaf.get("g"), kw["gate_act"], None, 1.0, 1e-6)
        t = t - t.detach() + leaf["s"]
        loss = (norm(t.masked_fill(none["s"], 0), leaf["wn"], 1e-6) * f64(do)).sum()
        if dres is not None:
            loss = loss + (t * f64(dres)).sum()
        want = dict(zip(leaf, torch.autograd.grad(loss, tuple(leaf.values()))))
        b = gdn.gdn_block_norm_bwd(dev(yy), dev(s), dout=dev(do), dres=dev(dres), **kw)
        assert rows_rel(b["dresidual"], want["s"]) <= tol(dtype, TOL_NORM)
        assert rows_rel(b["dy"], want["y"]) <= tol(dtype, TOL_NORM)
        assert rows_rel(b["dpost_weight"][None], want["wp"][None]) <= TOL_NORM
        assert rows_rel(b["dpre_weight"][None], want["wn"][None]) <= TOL_NORM
        if gate is not None:
            assert rows_rel(b["dgate"], want["g"]) <= tol(dtype, TOL_NORM)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rms_norm_weights_gradient_beside_large_rows(dtype):
    """The layer's norm has no finite dx for rows whose sum of squares comes near the end of fp32's range; the weights' gradient
    and the other rows' stay right."""
    s, w, dy = randn((12, 256), dtype, 320), randn((256,), F32, 321, 0.1, 1.0), randn((12, 256), dtype, 322, 1.5)
    s[3], s[7], s[8], s[11] = -1e18, torch.finfo(dtype).min, 1e12, 1e16
    leaf = f64(s).requires_grad_(), f64(w).requires_grad_()
    ds, dw = torch.autograd.grad((norm(leaf[0].masked_fill(f64(s) == f64(s[7]).min(), 0), leaf[1], 1e-6) * f64(dy)).sum(), leaf)
    got = gdn.gdn_rmsnorm_bwd(dev(s), dev(w), dev(dy))
    rest = [k for k in range(12) if k not in (3, 7)]
    assert rows_rel(got["dx"][rest], ds[rest]) <= tol(dtype, TOL_NORM) and rows_rel(got["dweight"][None], dw[None]) <= TOL_NORM


def test_block_norm_gradient_with_a_small_eps():
    """Rows of zeros under a small eps, whose inverse root's third power fp32 does not hold: the gradient is gw / sqrt(eps)."""
    y, do, w = torch.zeros(1, 2, 64, device=DEV), dev(randn((1, 2, 64), F32, 230)), torch.ones(64, device=DEV)
    b = gdn.gdn_block_norm_bwd(y, y, dres=do, post_weight=w, eps=1e-30)
    assert rows_rel(b["dy"], f64(do) * 1e15) <= TOL_NORM


# ------------------------------------------------------ gated recurrence ---


@pytest.mark.parametrize("lens,at", [
    ([70, 3, 500, 27], 75),       # a sequence starts at 73, in a run of eight from 72: 12 tiles, a cluster
    ([20, 40], 22),               # one tile
    ([3, 2, 2, 90, 5], 6),        # several in a run; the second to last of those before it
    ([64, 64, 64], 65), ([1] * 40, 17), ([13, 650, 20], 664), ([700, 9, 3000, 1], 703), ([2500, 64, 1], 2502)])
@pytest.mark.parametrize("where", ["x", "r", "i", "z", "dout"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lru_non_finite_values_beside_a_cut(lens, at, where, dtype):
    """A NaN among the first tokens of a packed sequence, in the run of tokens in which it begins: the sequences before and
    behind keep their outputs and gradients to the bit."""
    T, C = sum(lens), 70
    x, r, i, lam, z, h0, n = lru_inputs(1, T, C, lens, dtype, True, seed=240)
    do, dh = randn((1, T, C), dtype, 250), randn((n, C), F32, 251)
    (seq, (_, p, q)), = [(k, s) for k, s in enumerate(spans(1, T, lens)) if s[1] <= at < s[2]]
    cu, out = dev(cu_of(lens)), []
    for value in (0.5, float("nan")):
        dict(x=x, r=r, i=i, z=z, dout=do)[where][0, at] = value
        args, kw = [dev(t) for t in (x, r, i, lam)], dict(z=dev(z), h0=dev(h0), cu_seqlens=cu)
        final, ck = torch.empty(n, C, device=DEV), torch.empty(1, (T + 63) // 64, C, device=DEV)
        y = gdn.gdn_lru_fwd(*args, h_final=final, checkpoints=ck, **kw)
        b = gdn.gdn_lru_bwd(*args, dev(do), dh_final=dev(dh), checkpoints=ck, **kw)
        out.append(([y] + [b[k] for k in ("dx", "dr", "di", "dz")], [final, b["dh0"]]))
    rest = torch.ones(T, dtype=torch.bool)
    rest[p:q] = False
    for a, b in zip(out[0][0], out[1][0]):
        assert torch.equal(a[0, dev(rest)], b[0, dev(rest)])
    rest = [k for k in range(n) if k != seq]
    for a, b in zip(out[0][1], out[1][1]):
        assert torch.equal(a[rest], b[rest])
    assert not all(a.isfinite().all() for a in out[1][0])


@pytest.mark.parametrize("B,T,C,lens", [
    (1, 50, 192, None), (3, 700, 192, None), (1, 2500, 128, None), (1, 2500, 128, [3, 0, 1900, 597]), (2, 2500, 126, None),
    (1, 1500, 130, [700, 800]), (4, 300, 130, None)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cta", [0, 1, 7])
def test_lru_waits_that_run_out(B, T, C, lens, dtype, cta):
    """A CTA that asks for no rows (the library's testing aid) gives up after 20 ms: the error word says so, all that it or the
    CTAs of its cluster would have written (one line of 64 channels) is NaN, the rest is right to the bit, and so is the
    next call. Where rows go by words or elements there is no wait for them, and the CTA gives up without one."""
    x, r, i, lam, z, h0, n = lru_inputs(B, T, C, lens, dtype, True, seed=260)
    args, cu = [dev(t) for t in (x, r, i, lam)], dev(cu_of(lens))
    kw = dict(z=dev(z), h0=dev(h0), cu_seqlens=cu)
    do, dh = dev(randn((B, T, C), dtype, 270)), dev(randn((n, C), F32, 271))
    ws = torch.zeros(gdn.lib().gdn_lru_bwd_workspace_size(B, T, C, 0), dtype=torch.uint8, device=DEV)

    def forward():
        final, ck = torch.zeros(n, C, device=DEV), torch.zeros(B, (T + 63) // 64, C, device=DEV)
        y = gdn.gdn_lru_fwd(*args, h_final=final, checkpoints=ck, workspace=ws, **kw)
        return dict(y=y, final=final, ck=ck)

    saved = forward()["ck"]

    def backward(**how):
        return gdn.gdn_lru_bwd(*args, do, dh_final=dh, workspace=ws, **how, **kw)

    for run, how in ((forward, {}), (backward, dict(checkpoints=saved)), (backward, {})):
        want = run(**how)
        assert gdn.gdn_last_device_error(ws) == 0
        gdn.gdn_set_stall_test(cta, 20000)
        try:
            got = run(**how)
            word = gdn.gdn_last_device_error(ws)
        finally:
            gdn.gdn_set_stall_test(-1, 0)
        again = run(**how)
        assert gdn.gdn_last_device_error(ws) == 0 and all(torch.equal(want[k], again[k]) for k in want)
        lost = got["y" if run is forward else "dr"].isnan()
        if not lost.any():  # (fewer CTAs than that)
            assert word == 0
            continue
        assert word == 2
        tiles = sorted({(line, c // 64) for line, c in lost.any(1).nonzero().tolist()})
        here = torch.zeros(B, 1, C, dtype=torch.bool, device=DEV)
        for line, c in tiles:
            here[line, 0, 64 * c:64 * c + 64] = True
        # without checkpoints the states are formed by a launch of its own, one of whose CTAs gives up, too: what follows
        # from them (dr, dz, dlam) is NaN there as far as its states go
        alone = run is forward or how
        assert len(tiles) == 1 or (not alone and len(tiles) == 2)
        for k in got:
            if k == "dlam":
                mine = here.any(0)[0]
            elif k in ("final", "dh0"):
                some = torch.ones(n, 1, dtype=torch.bool, device=DEV) if lens is None else dev(torch.tensor(lens) > 0)[:, None]
                mine = (here[:, 0] if lens is None else here[0]).expand(n, C) & some
            else:
                mine = here.expand(got[k].shape)
            assert not alone or got[k][mine].isnan().all(), k
            assert torch.equal(got[k][~mine], want[k][~mine]), k


@pytest.mark.parametrize("B,T,C,lens,off", [
    (2, 2501, 72, None, False),                                 # tensor copies
    (1, 2501, 128, [1500, 63, 1, 0, 64, 65, 200, 608], False),  # sequences that end inside, at and across steps
    (1, 2501, 66, [768, 768, 768, 197], True), (2, 1300, 34, None, True),    # words (in bf16 of pairs)
    (1, 2501, 65, [1024, 1024, 453], True), (2, 1300, 33, None, True)])      # bf16: elements
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lru_lines_of_several_cluster_steps(B, T, C, lens, off, dtype):
    """Lines that a cluster walks in three steps and more, so that its barriers and the runs' places are used again, forward
    and back, by clusters of the default size (12, or 16 where rows are not wide), of the size taken where those do not fit,
    and of few CTAs, whose lines have up to 40 steps. Short memories: the tolerances' steps stay below 600."""
    x, r, i, _, z, h0, n = lru_inputs(B, T, C, lens, dtype, True, seed=280)
    lam, do, dh = decays(C, 0.5, 0.9), randn((B, T, C), dtype, 290), randn((n, C), F32, 291)
    leaf = [f64(t).requires_grad_() for t in (x, r, i, lam, z, h0)]
    ref, fin = ref_lru(*leaf, lens)
    want = torch.autograd.grad((ref * f64(do)).sum() + (fin * f64(dh)).sum(), leaf)
    at = (lambda t: strided(dev(t))) if off else dev
    args, kw = [at(t) for t in (x, r, i)] + [dev(lam)], dict(z=at(z), h0=dev(h0), cu_seqlens=dev(cu_of(lens)))
    for most in (0, 8, 1, 2, 3):
        gdn.gdn_set_lru_cluster(most)
        try:
            final, ck = torch.empty(n, C, device=DEV), torch.empty(B, (T + 63) // 64, C, device=DEV)
            got = gdn.gdn_lru_fwd(*args, h_final=final, checkpoints=ck, **kw)
            grads = [gdn.gdn_lru_bwd(*args, at(do), dh_final=dev(dh), **saved, **kw) for saved in (dict(checkpoints=ck), {})]
        finally:
            gdn.gdn_set_lru_cluster(0)
        assert rel(got, ref.detach()) <= tol(dtype, TOL_LRU) and rel(final, fin.detach()) <= TOL_LRU, most
        for g in grads:
            for k, w in zip(("dx", "dr", "di", "dlam", "dz", "dh0"), want):
                assert rel(g[k], w) <= tol(g[k].dtype, TOL_LRU_BWD), (most, k)


def test_lru_without_tokens_clears_the_error_word():
    t, lam, ws = torch.empty(1, 0, 64, dtype=BF, device=DEV), torch.zeros(64, device=DEV), torch.full((512,), 255, dtype=torch.uint8, device=DEV)
    final = torch.empty(1, 64, device=DEV)
    for call in (lambda: gdn.gdn_lru_fwd(t, t, t, lam, h_final=final, workspace=ws), lambda: gdn.gdn_lru_bwd(t, t, t, lam, t, workspace=ws),
                 lambda: gdn.gdn_lru_fwd(t, t, t, lam, cu_seqlens=torch.zeros(3, dtype=torch.int32, device=DEV), workspace=ws)):
        ws.fill_(255)
        call()
        assert gdn.gdn_last_device_error(ws) == 0


def test_lru_large_clusters_in_a_graph():
    """Whether a cluster of twelve fits is asked on the host, in a captured call as well."""
    x, r, i, lam, z, h0, n = lru_inputs(1, 1500, 72, None, BF, True, seed=300)
    args, kw = [dev(t) for t in (x, r, i, lam)], dict(z=dev(z), h0=dev(h0))

    def run():
        g = gdn.gdn_lru_bwd(*args, args[0], **kw)
        return [gdn.gdn_lru_fwd(*args, **kw)] + [g[k] for k in sorted(g)]

    want, graph, side = run(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# --------------------------------------------------------- as used together ---


def _sizes_of(name):
    """Two calls that one kernel takes with different amounts of shared memory."""
    bf = dict(dtype=BF, device=DEV)
    if name.startswith("lru"):
        def call(T):
            t, lam = torch.zeros(1, T, 64, **bf), torch.zeros(64, device=DEV)
            ws = torch.zeros(gdn.lib().gdn_lru_bwd_workspace_size(1, T, 64, 0), dtype=torch.uint8, device=DEV)
            if name == "lru_bwd":
                return lambda: gdn.gdn_lru_bwd(t, t, t, lam, t, z=t, workspace=ws)
            return lambda: gdn.gdn_lru_fwd(t, t, t, lam, z=t, out=torch.empty_like(t))
        return call(1500), call(100)
    if name.startswith("chunk"):
        def call(V):
            q, v, b = torch.zeros(1, 64, 1, 64, **bf), torch.zeros(1, 64, 1, V, **bf), torch.zeros(1, 64, 1, device=DEV)
            gk = torch.zeros(1, 64, 1, 64, device=DEV) if name == "chunk_gk" else None
            return lambda: gdn.gdn_chunk_fwd(q, q, v, b, g=None if gk is not None else b, gk=gk)
        return call(256), call(64)

    def call(D):
        t, w = torch.zeros(2, D, **bf), torch.zeros(D, device=DEV)
        if name == "rms_bwd":
            return lambda: gdn.gdn_rmsnorm_bwd(t, w, t)
        kw = dict(post_weight=w, pre_weight=w, gate=t, gate_act="silu")
        if name == "block_bwd":
            return lambda: gdn.gdn_block_norm_bwd(t, t, dout=t, dres=t, **kw)
        return lambda: gdn.gdn_block_norm_fwd(t, t, **kw)
    return call(8192), call(5120)


@pytest.mark.parametrize("name", ["lru", "lru_bwd", "block", "block_bwd", "rms_bwd", "chunk", "chunk_gk"])
def test_calls_of_different_sizes_on_two_threads(name):
    """Each call sets what shared memory its kernel may take; a smaller call between another's setting and launch must not
    lower it."""
    calls, failed = _sizes_of(name), []
    for call in calls:
        call()
    start = threading.Barrier(len(calls))

    def work(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for k in range(4000):
                    call()
                    if k % 500 == 0:
                        torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
