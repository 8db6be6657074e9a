"""Cases of the state-space layer's operators: the residual root-mean-square
norm (with an 8-bit output), the short causal convolution and the selective
scan, each for prompts, for single tokens and (norm, convolution, scan) for
training.

`run` makes one pass through one operator. With `own` false it computes the
operator from elementary torch operations in fp32; with `own` true it makes
the framework's calls. `exact` computes the same outputs in fp64.

Layouts: x, dt, z, out (B, T, D); Bm, Cm (B, T, N); A (D, N) fp32; states of
the scan (n, D, N) fp32; taps of the convolution (D, W) fp32, its states
(n, W - 1, D), oldest input first; norms over rows (R, D). Packed batches have
B = 1 and cu_seqlens.
"""
import math
import random

import torch

own = False

EPS = 1e-6
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# the largest scan: B T D N of the prompt and training cases
MOST_SCAN = 4 * 4096 * 4096 * 16
# the largest norm or convolution, in elements of x
MOST_ROWS = 4 * 4096 * 4096


def listed():
    return [
        # decoding: 8 requests through the norm before the 8-bit input projection
        dict(name="norm_token_q8", op="norm", rows=8, d=2048, dtype="bf16", res="bf16", group=128),
        # a prompt's norm with an fp32 residual stream, one scale per 128 channels
        dict(name="norm_prompt_q8", op="norm", rows=16384, d=4096, dtype="bf16", res="f32", group=128),
        # training: gradient of the norm, with the residual stream's own gradient
        dict(name="norm_train_bwd", op="norm_bwd", rows=16384, d=2048, dtype="bf16", res="bf16"),
        # decoding: 64 requests, their windows in a pool of 96 slots
        dict(name="conv_token", op="conv_step", reqs=64, pool=96, d=4096, w=4, dtype="bf16"),
        # packed prompts of very different lengths, windows carried in and out
        dict(name="conv_prompt", op="conv", batch=1, t=16384, seqs=24, d=4096, w=4, dtype="bf16", states=True),
        # training: input, tap and bias gradients
        dict(name="conv_train_bwd", op="conv_bwd", batch=4, t=4096, seqs=0, d=4096, w=4, dtype="bf16", states=False),
        # decoding one request: latency
        dict(name="ssm_token_1", op="ssm_step", reqs=1, pool=1, d=4096, n=16, dtype="bf16"),
        # decoding 256 requests out of a pool of 384 states
        dict(name="ssm_token_256", op="ssm_step", reqs=256, pool=384, d=4096, n=16, dtype="bf16"),
        # a batch of prompts, states kept for decoding
        dict(name="ssm_prompt", op="ssm", batch=4, t=4096, seqs=0, d=4096, n=16, dtype="bf16", states=True),
        # one long prompt over few channels: too few rows to fill the GPU
        dict(name="ssm_long", op="ssm", batch=1, t=32768, seqs=0, d=2048, n=16, dtype="bf16", states=True),
        # packed ragged prompts in fp32, a channel count that is no power of two
        dict(name="ssm_packed_f32", op="ssm", batch=1, t=5003, seqs=9, d=1792, n=16, dtype="f32", states=True),
        # training: every gradient of the scan
        dict(name="ssm_train_bwd", op="ssm_bwd", batch=4, t=4096, seqs=0, d=4096, n=16, dtype="bf16", states=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _channels(rng):
    d = _log(rng, 64, 8192)
    return d if rng.random() < 0.3 else max(8, d // 8 * 8)  # some odd, most of whole 16-byte rows


def _tokens(rng, most):
    """(batch, t, seqs): dense batches, or one packed line of `seqs` sequences."""
    t = _log(rng, 1, max(1, min(32768, most)))
    if rng.random() < 0.5:
        return 1, t, rng.randint(1, 40)
    b = max(1, min(rng.randint(1, 8), most // t))
    return b, t, 0


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "conv_step", "conv", "conv_bwd", "ssm_step", "ssm", "ssm", "ssm_bwd", "ssm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = _channels(rng)
    if op in ("norm", "norm_bwd"):
        c = dict(op=op, rows=_log(rng, 1, MOST_ROWS // 2 // d), d=d, dtype=dtype, res=rng.choice(["bf16", "f32", "none"]))
        if op == "norm":
            c["group"] = rng.choice([-1, 0, 32, 64, 128, 256])  # -1: no 8-bit output, 0: one scale a row
        elif c["res"] == "none":
            c["res"] = dtype
        return c
    if op in ("conv_step", "ssm_step"):
        c = dict(op=op, reqs=_log(rng, 1, 256), d=min(d, 4096), dtype=dtype)
        c["pool"] = c["reqs"] + rng.randint(0, 64)
    else:
        most = (MOST_ROWS if op.startswith("conv") else MOST_SCAN // 16) // 2 // d
    if op.startswith("conv"):
        w = rng.choice([2, 3, 4, 4, 4, 5, 8])
        if op == "conv_step":
            return dict(c, w=w)
        b, t, seqs = _tokens(rng, most)
        return dict(op=op, batch=b, t=t, seqs=seqs, d=d, w=w, dtype=dtype, states=rng.random() < 0.5)
    n = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 40)])
    if op == "ssm_step":
        return dict(c, n=n)
    b, t, seqs = _tokens(rng, max(1, most * 16 // max(16, n)))
    return dict(op=op, batch=b, t=t, seqs=seqs, d=d, n=n, dtype=dtype, states=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs ---


def _lengths(case):
    """Token counts of a packed batch: uniform cuts, so some are short and a few may be empty."""
    r = random.Random(case["t"] * 1009 + case["seqs"])
    cuts = sorted(r.randint(0, case["t"]) for _ in range(case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["t"]])]


class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, std=1.0, mean=0.0):
        x = torch.empty(shape, device="cuda", dtype=dtype)
        return x.normal_(mean, std, generator=self.g)

    def uniform(self, lo, hi, *shape):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=self.g)

    def slots(self, pool, reqs):
        return torch.randperm(pool, generator=self.g, device="cuda")[:reqs].to(torch.int32)


def _cu(case):
    if not case["seqs"]:
        return None
    at = [0]
    for n in _lengths(case):
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _scan_inputs(m, case, s, lead):
    """x, dt, z, Bm, Cm as a layer has them: z is half of the input
    projection, Bm and Cm are slices of one projection's rows."""
    d, n, ty = case["d"], case["n"], TYPES[case["dtype"]]
    rank = max(8, d // 16 // 8 * 8)
    s["x"] = m.normal(*lead, d, dtype=ty)
    s["z"] = m.normal(*lead, 2 * d, dtype=ty)[..., d:]
    s["dt"] = m.normal(*lead, d, dtype=ty, std=0.5)
    p = m.normal(*lead, rank + 2 * n, dtype=ty)
    s["Bm"], s["Cm"] = p[..., rank : rank + n], p[..., rank + n :]
    s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * m.uniform(0.8, 1.25, d, n)
    s["D"] = m.normal(d, std=0.1, mean=1.0)
    # time steps between 1e-3 and 1e-1: the inverse of softplus gives the bias
    step = torch.exp(m.uniform(math.log(1e-3), math.log(1e-1), d))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))


def prepare(case, seed):
    m, op, ty = _Maker(seed), case["op"], TYPES[case["dtype"]]
    d = case["d"]
    s = dict(op=op, ty=ty)
    if op in ("norm", "norm_bwd"):
        rows, res = case["rows"], TYPES.get(case["res"])
        s["weight"] = m.normal(d, std=0.1, mean=1.0)
        if op == "norm":
            s["x"] = m.normal(rows, d, dtype=ty)
            s["res"] = None if res is None else m.normal(rows, d, dtype=res, std=2.0)
            s["group"] = case["group"]
        else:
            s["s"] = m.normal(rows, d, dtype=res, std=2.0)
            s["dy"] = m.normal(rows, d, dtype=ty)
            s["dres"] = m.normal(rows, d, dtype=res)
        return s
    n_seq = case.get("seqs") or case.get("batch")
    if op.startswith("conv"):
        w = case["w"]
        s["weight"], s["bias"] = m.normal(d, w, std=0.3), m.normal(d, std=0.1)
        if op == "conv_step":
            s["x"] = m.normal(case["reqs"], 2 * d, dtype=ty)[:, :d]
            s["state"] = m.normal(case["pool"], w - 1, d, dtype=ty)
            s["slots"] = m.slots(case["pool"], case["reqs"])
            return s
        b, t = case["batch"], case["t"]
        s["cu"] = _cu(case)
        s["x"] = m.normal(b, t, 2 * d, dtype=ty)[..., :d]
        s["init"] = m.normal(n_seq, w - 1, d, dtype=ty) if case["states"] else None
        if op == "conv":
            s["final"] = torch.empty(n_seq, w - 1, d, device="cuda", dtype=ty) if case["states"] else None
        else:
            s["dout"] = m.normal(b, t, d, dtype=ty)
            s["dfinal"] = m.normal(n_seq, w - 1, d, dtype=ty) if case["states"] else None
        return s
    n = case["n"]
    if op == "ssm_step":
        _scan_inputs(m, case, s, (case["reqs"],))
        s["state"] = m.normal(case["pool"], d, n, std=0.1)
        s["slots"] = m.slots(case["pool"], case["reqs"])
        return s
    b, t = case["batch"], case["t"]
    _scan_inputs(m, case, s, (b, t))
    s["cu"] = _cu(case)
    s["h0"] = m.normal(n_seq, d, n, std=0.1) if case["states"] else None
    if op == "ssm":
        s["final"] = torch.empty(n_seq, d, n, device="cuda") if case["states"] else None
    else:
        s["dout"] = m.normal(b, t, d, dtype=ty)
        s["dfinal"] = m.normal(n_seq, d, n, std=0.1) if case["states"] else None
    return s


# ------------------------------------------------------------------- plain ---


def _plain_norm(s):
    x, res, group = s["x"].float(), s["res"], s["group"]
    r = {}
    if res is not None:
        x = x + res.float()
        r["residual"] = x.to(res.dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"]
    if group < 0:
        return dict(r, out=y.to(s["ty"]))
    rows, d = y.shape
    group = group or d
    pad = -d % group
    v = torch.nn.functional.pad(y, (0, pad)).view(rows, -1, group)
    scale = v.abs().amax(-1) / F8_MAX
    q = v / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    return dict(r, out=q.reshape(rows, -1)[:, :d].to(F8), scale=scale)


def _plain_norm_bwd(s):
    x, w, dy = s["s"].float(), s["weight"], s["dy"].float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = dy * w
    dx = inv * g - x * inv**3 * (g * x).mean(-1, keepdim=True) + s["dres"].float()
    return dict(dx=dx.to(s["s"].dtype), dweight=(dy * x * inv).sum(0))


def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def _lines(s, w):
    """The packed line with each sequence's W - 1 earlier inputs before its
    tokens: (fp32 rows, the tokens' places in it, the places of the first
    earlier input of each sequence and of each sequence's end)."""
    b, t, d = s["x"].shape
    n = s["cu"].numel() - 1 if s["cu"] is not None else b
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device="cuda") * t
    tok = torch.arange(b * t, device="cuda")
    seg = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    at = tok + (seg + 1) * (w - 1)
    first, end = cu[:-1] + torch.arange(n, device="cuda") * (w - 1), cu[1:] + torch.arange(1, n + 1, device="cuda") * (w - 1)
    line = torch.zeros(b * t + n * (w - 1), d, device="cuda")
    line[at] = s["x"].reshape(b * t, d).float()
    k = torch.arange(w - 1, device="cuda")
    if s["init"] is not None:
        line[first[:, None] + k] = s["init"].float()
    return line, at, first[:, None] + k, end[:, None] - (w - 1) + k


def _plain_conv(s):
    w = s["weight"].shape[1]
    line, at, _, last = _lines(s, w)
    pre = (line.unfold(0, w, 1) * s["weight"]).sum(-1)[at - (w - 1)] + s["bias"]
    r = dict(out=_silu(pre).to(s["ty"]).view(s["x"].shape))
    if s["final"] is not None:
        s["final"].copy_(line[last])
        r["final"] = s["final"]
    return r


def _plain_conv_bwd(s):
    w, wt = s["weight"].shape[1], s["weight"]
    line, at, first, last = _lines(s, w)
    win = line.unfold(0, w, 1)[at - (w - 1)]
    dpre = s["dout"].reshape(at.numel(), -1).float() * _dsilu((win * wt).sum(-1) + s["bias"])
    g = torch.zeros(line.shape[0] + w - 1, line.shape[1], device="cuda")
    g[at] = dpre
    dline = (g.unfold(0, w, 1) * wt.flip(1)).sum(-1)
    if s["dfinal"] is not None:
        dline.index_put_((last,), s["dfinal"].float(), accumulate=True)
    r = dict(dx=dline[at].to(s["ty"]).view(s["x"].shape), dweight=(win * dpre[..., None]).sum(0), dbias=dpre.sum(0))
    if s["init"] is not None:
        r["dinitial"] = dline[first].to(s["ty"])
    return r


def _plain_conv_step(s):
    at = s["slots"].long()
    win = torch.cat([s["state"][at].float(), s["x"].float()[:, None]], 1)
    s["state"][at] = win[:, 1:].to(s["ty"])
    out = _silu((win * s["weight"].t()).sum(1) + s["bias"])
    return dict(out=out.to(s["ty"]), state=s["state"])


def _steps(s):
    """softplus(dt + bias), its argument, and the gated-scan inputs in fp32."""
    v = s["dt"].float() + s["dt_bias"]
    soft = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    return soft, v


def _plain_ssm_step(s):
    at = s["slots"].long()
    delta, _ = _steps(s)
    x = s["x"].float()
    h = s["state"][at] * torch.exp(delta[..., None] * s["A"]) + (delta * x)[..., None] * s["Bm"].float()[:, None]
    s["state"][at] = h
    y = (h * s["Cm"].float()[:, None]).sum(-1) + s["D"] * x
    return dict(out=(y * _silu(s["z"].float())).to(s["ty"]), state=s["state"])


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling: both are overwritten."""
    k = 1
    while k < a.shape[1]:
        b[:, k:] += a[:, k:] * b[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return b


def _bounds(s):
    """(row, first token), (row, last token) and nonempty of each sequence."""
    b, t, _ = s["x"].shape
    if s["cu"] is None:
        row, zero = torch.arange(b, device="cuda"), torch.zeros(b, dtype=torch.long, device="cuda")
        return (row, zero), (row, zero + t - 1), zero == 0
    cu = s["cu"].long()
    zero = torch.zeros_like(cu[1:])
    return (zero, cu[:-1].clamp(max=t - 1)), (zero, (cu[1:] - 1).clamp(min=0)), cu[1:] > cu[:-1]


def _scan_terms(s):
    """The decays with zeros where a sequence begins, the states, and what made them."""
    delta, v = _steps(s)
    x = s["x"].float()
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * s["Bm"].float()[:, :, None]
    first, last, some = _bounds(s)
    if s["h0"] is not None:
        b.index_put_(first, a[first] * s["h0"] * some[:, None, None], accumulate=True)
    begins = torch.zeros(s["x"].shape[:2], device="cuda").index_put_(first, some.float(), accumulate=True) > 0
    cut = a.masked_fill(begins[..., None, None], 0.0)
    return delta, v, x, a, cut, b, first, last, some, begins


def _plain_ssm(s):
    _, _, x, _, cut, b, _, last, some, _ = _scan_terms(s)
    h = _recur(cut, b)
    y = (h * s["Cm"].float()[:, :, None]).sum(-1) + s["D"] * x
    r = dict(out=(y * _silu(s["z"].float())).to(s["ty"]))
    if s["final"] is not None:
        s["final"].copy_(torch.where(some[:, None, None], h[last], s["h0"]))
        r["final"] = s["final"]
    return r


def _plain_ssm_bwd(s):
    delta, v, x, a, cut, b, first, last, some, begins = _scan_terms(s)
    bm, cm, z, do = (s[k].float() for k in ("Bm", "Cm", "z", "dout"))
    h = _recur(cut.clone(), b)
    y = (h * cm[:, :, None]).sum(-1) + s["D"] * x
    dz, dy = do * y * _dsilu(z), do * _silu(z)
    g = dy[..., None] * cm[:, :, None]
    if s["dfinal"] is not None:
        g.index_put_(last, s["dfinal"] * some[:, None, None], accumulate=True)
    # g_t += a_{t+1} g_{t+1}, with no step over a sequence's end
    nxt = torch.cat([torch.zeros_like(cut[:, :1]), cut[:, 1:].flip(1)], 1)
    g = _recur(nxt, g.flip(1)).flip(1)
    back = a * g
    r = dict(dz=dz.to(s["ty"]), dD=(dy * x).sum((0, 1)))
    r["dCm"] = (dy[..., None] * h).sum(2).to(s["ty"])
    r["dBm"] = ((delta * x)[..., None] * g).sum(2).to(s["ty"])
    gb = (g * bm[:, :, None]).sum(-1)
    r["dx"] = (s["D"] * dy + delta * gb).to(s["ty"])
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1).masked_fill_(begins[..., None, None], 0.0)
    if s["h0"] is not None:
        prev.index_put_(first, s["h0"] * some[:, None, None], accumulate=True)
        r["dh0"] = torch.where(some[:, None, None], back[first], s["dfinal"])
    prev *= back
    ddelta = (prev * s["A"]).sum(-1) + x * gb
    r["dA"] = (prev * delta[..., None]).sum((0, 1))
    dv = ddelta * torch.sigmoid(v)
    r["ddt"], r["ddt_bias"] = dv.to(s["ty"]), dv.sum((0, 1))
    return r


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "conv": _plain_conv, "conv_bwd": _plain_conv_bwd,
         "conv_step": _plain_conv_step, "ssm": _plain_ssm, "ssm_bwd": _plain_ssm_bwd, "ssm_step": _plain_ssm_step}


# --------------------------------------------------------------- framework ---


def _own(s):
    import gated_delta_rule_18_gb300 as gdn

    op = s["op"]
    if op == "norm":
        if s["group"] < 0:
            return gdn.gdn_rmsnorm_fwd(s["x"], s["weight"], residual=s["res"], eps=EPS)
        return gdn.gdn_rmsnorm_fwd(s["x"], s["weight"], residual=s["res"], eps=EPS, out_dtype=F8, group=s["group"])
    if op == "norm_bwd":
        return gdn.gdn_rmsnorm_bwd(s["s"], s["weight"], s["dy"], dres=s["dres"], eps=EPS)
    if op == "conv":
        r = dict(out=gdn.gdn_conv_fwd(s["x"], s["weight"], bias=s["bias"], initial_state=s["init"], cu_seqlens=s["cu"], final_state=s["final"]))
        if s["final"] is not None:
            r["final"] = s["final"]
        return r
    if op == "conv_bwd":
        r = gdn.gdn_conv_bwd(s["x"], s["weight"], s["dout"], bias=s["bias"], initial_state=s["init"], cu_seqlens=s["cu"], dfinal_state=s["dfinal"])
        if "dinitial_state" in r:
            r["dinitial"] = r.pop("dinitial_state")
        return r
    if op == "conv_step":
        return dict(out=gdn.gdn_conv_step(s["x"], s["state"], s["weight"], bias=s["bias"], slots=s["slots"]), state=s["state"])
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    if op == "ssm_step":
        out = gdn.gdn_ssm_step(*args, s["state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], slots=s["slots"])
        return dict(out=out, state=s["state"])
    if op == "ssm":
        r = dict(out=gdn.gdn_ssm_fwd(*args, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], h0=s["h0"], cu_seqlens=s["cu"], h_final=s["final"]))
        if s["final"] is not None:
            r["final"] = s["final"]
        return r
    return gdn.gdn_ssm_bwd(*args, s["dout"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], h0=s["h0"], cu_seqlens=s["cu"], dh_final=s["dfinal"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work ---


def work(case):
    op, d, e = case["op"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        rows, r = case["rows"], {"bf16": 2, "f32": 4, "none": 0}[case["res"]]
        if op == "norm_bwd":
            return dict(bytes=rows * d * (e + 3 * r) + 8 * d, flops=12 * rows * d)
        out = e if case["group"] < 0 else 1
        scales = 0 if case["group"] < 0 else 4 * rows * (-(-d // case["group"]) if case["group"] else 1)
        return dict(bytes=rows * d * (e + 2 * r + out) + scales + 4 * d, flops=6 * rows * d)
    if op == "conv_step":
        return dict(bytes=case["reqs"] * (d * e * (2 + 2 * (case["w"] - 1)) + 4) + 4 * d * (case["w"] + 1), flops=case["reqs"] * d * (2 * case["w"] + 5))
    if op == "ssm_step":
        n = case["n"]
        return dict(bytes=case["reqs"] * (8 * d * n + e * (4 * d + 2 * n) + 4) + 4 * d * (n + 2), flops=case["reqs"] * d * (7 * n + 15))
    tok = case["batch"] * case["t"]
    n_seq = case["seqs"] or case["batch"]
    if op.startswith("conv"):
        w = case["w"]
        state = 2 * n_seq * (w - 1) * d * e if case["states"] else 0
        if op == "conv":
            return dict(bytes=2 * tok * d * e + state + 4 * d * (w + 1), flops=tok * d * (2 * w + 5))
        return dict(bytes=3 * tok * d * e + (1.5 * state) + 8 * d * (w + 1), flops=tok * d * (6 * w + 9))
    n = case["n"]
    state = 4 * n_seq * d * n * (2 if op == "ssm" else 3) if case["states"] else 0
    if op == "ssm":
        return dict(bytes=tok * e * (4 * d + 2 * n) + state + 4 * d * (n + 2), flops=tok * d * (7 * n + 15))
    return dict(bytes=tok * e * (7 * d + 4 * n) + state + 8 * d * (n + 2), flops=tok * d * (24 * n + 40))


# ------------------------------------------------------------------- exact ---


def _exact_e4m3(v):
    """fp64 to the nearest e4m3 value (ties to even), in fp64."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0**-20))).clamp(min=-6, max=8)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-F8_MAX, F8_MAX)


def _exact_norm(s):
    r = {}
    u = s["x"].double()
    if s["res"] is not None:
        u = u + s["res"].double()
        r["residual"] = u
    y = s["weight"].double() * (u / torch.sqrt(u.square().sum(1, keepdim=True) / u.shape[1] + EPS))
    if s["group"] < 0:
        return dict(r, out=y)
    parts = torch.split(y, s["group"] or y.shape[1], dim=1)
    scales = [p.abs().max(1, keepdim=True).values / F8_MAX for p in parts]
    return dict(r, out=torch.cat([_exact_e4m3(p / c) for p, c in zip(parts, scales)], 1), scale=torch.cat(scales, 1))


def _exact_norm_bwd(s):
    u = s["s"].double().requires_grad_()
    w = s["weight"].double().requires_grad_()
    y = w * (u / torch.sqrt(u.square().sum(1, keepdim=True) / u.shape[1] + EPS))
    loss = (y * s["dy"].double()).sum() + (u * s["dres"].double()).sum()
    dx, dw = torch.autograd.grad(loss, (u, w))
    return dict(dx=dx, dweight=dw)


def _spans(s):
    b, t, _ = s["x"].shape
    if s["cu"] is None:
        return [(i, 0, t) for i in range(b)]
    at = s["cu"].tolist()
    return [(0, p, q) for p, q in zip(at[:-1], at[1:])]


def _exact_conv_all(s, x, wt, bias, init):
    """(out, final) by sequence and tap, in fp64."""
    w = wt.shape[1]
    out, final = [], []
    for k, (row, p, q) in enumerate(_spans(s)):
        head = init[k] if init is not None else torch.zeros(w - 1, x.shape[2], device="cuda", dtype=torch.float64)
        line = torch.cat([head, x[row, p:q]], 0)
        pre = bias.expand(q - p, -1)
        for j in range(w):
            pre = pre + wt[:, j] * line[j : j + q - p]
        out.append(pre / (1 + torch.exp(-pre)))
        final.append(line[q - p :])
    return torch.cat(out, 0).view(x.shape), torch.stack(final)


def _exact_conv(s):
    init = None if s["init"] is None else s["init"].double()
    out, final = _exact_conv_all(s, s["x"].double(), s["weight"].double(), s["bias"].double(), init)
    return dict(out=out, **({} if s["final"] is None else dict(final=final)))


def _exact_conv_bwd(s):
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "weight", "bias", "init") if s[k] is not None}
    out, final = _exact_conv_all(s, leaf["x"], leaf["weight"], leaf["bias"], leaf.get("init"))
    loss = (out * s["dout"].double()).sum()
    if s["dfinal"] is not None:
        loss = loss + (final * s["dfinal"].double()).sum()
    names = dict(x="dx", weight="dweight", bias="dbias", init="dinitial")
    return dict(zip((names[k] for k in leaf), torch.autograd.grad(loss, tuple(leaf.values()))))


def _exact_conv_step(s):
    state = s["state"].double()
    at = s["slots"].long()
    pre = s["bias"].double() + s["weight"].double()[:, -1] * s["x"].double()
    for j in range(state.shape[1]):
        pre = pre + s["weight"].double()[:, j] * state[at, j]
    new = torch.cat([state[at, 1:], s["x"].double()[:, None]], 1)
    state[at] = new
    return dict(out=pre / (1 + torch.exp(-pre)), state=state)


def _exact_cell(h, x, dt, a, bm, cm, dd, z, bias):
    """One token: the new state and the gated output."""
    delta = torch.nn.functional.softplus(dt + bias, threshold=700)
    h = torch.exp(delta.unsqueeze(-1) * a) * h + delta.unsqueeze(-1) * x.unsqueeze(-1) * bm.unsqueeze(-2)
    y = torch.matmul(h, cm.unsqueeze(-1)).squeeze(-1) + dd * x
    return h, y * z / (1 + torch.exp(-z))


def _exact_ssm_step(s):
    state, at = s["state"].double(), s["slots"].long()
    h, out = _exact_cell(state[at], *(s[k].double() for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")))
    state[at] = h
    return dict(out=out, state=state)


def _exact_ssm_all(s, v):
    """(out, final), token by token."""
    x, b = v["x"], s["x"].shape[0]
    if s["cu"] is None:
        h = v["h0"] if "h0" in v else torch.zeros(b, *v["A"].shape, device="cuda", dtype=torch.float64)
        spans, whole = [(0, s["x"].shape[1])], True
    else:
        spans, whole = [(p, q) for _, p, q in _spans(s)], False
    out, final = [], []
    for k, (p, q) in enumerate(spans):
        if not whole:
            h = v["h0"][k : k + 1] if "h0" in v else torch.zeros(1, *v["A"].shape, device="cuda", dtype=torch.float64)
        for t in range(p, q):
            h, o = _exact_cell(h, x[:, t], v["dt"][:, t], v["A"], v["Bm"][:, t], v["Cm"][:, t], v["D"], v["z"][:, t], v["dt_bias"])
            out.append(o)
        final.append(h)
    return torch.stack(out, 1), torch.cat(final, 0)


LEAVES = dict(x="dx", dt="ddt", A="dA", Bm="dBm", Cm="dCm", D="dD", z="dz", dt_bias="ddt_bias", h0="dh0")


def _exact_ssm(s):
    with torch.no_grad():
        out, final = _exact_ssm_all(s, {k: s[k].double() for k in LEAVES if s[k] is not None})
    return dict(out=out, **({} if s["final"] is None else dict(final=final)))


def _exact_ssm_bwd(s):
    v = {k: s[k].double().requires_grad_() for k in LEAVES if s[k] is not None}
    out, final = _exact_ssm_all(s, v)
    loss = (out * s["dout"].double()).sum()
    if s["dfinal"] is not None:
        loss = loss + (final * s["dfinal"].double()).sum()
    return dict(zip((LEAVES[k] for k in v), torch.autograd.grad(loss, tuple(v.values()))))


EXACT = {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "conv": _exact_conv, "conv_bwd": _exact_conv_bwd,
         "conv_step": _exact_conv_step, "ssm": _exact_ssm, "ssm_bwd": _exact_ssm_bwd, "ssm_step": _exact_ssm_step}


def exact(case, seed):
    if case["op"] == "ssm_bwd":
        # the recorded token loop: about 10 fp64 copies of every token's state and 60 launches a token
        if case["batch"] * case["t"] * case["d"] * case["n"] * 80 > 150e9 or case["t"] > 6000:
            return None
    return EXACT[case["op"]](prepare(case, seed))
