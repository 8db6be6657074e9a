"""Cases of the operators around a mixer and of the gated linear recurrence that
can stand in its place: rotary positions of q and k, the norms behind and in
front of a block with its gate and residual scale, and the recurrence itself,
for prompts, for single tokens and for training.

`run` makes one pass through one operator. With `own` false it computes the
operator from elementary torch operations in fp32; with `own` true it makes
the framework's calls. `exact` computes the same outputs in fp64.

Layouts: q, k (B, T, H, D), slices of one projection's rows; positions (B, T)
int32; the recurrence's x, r, i, z (B, T, C), lam (C) fp32, its states (n, C)
fp32; y, residual, gate (B, T, D), a gate of one row a sequence (B, 1, D).
Packed batches have B = 1 and cu_seqlens.

  rotary       (a, b) -> s (a cos p f - b sin p f, a sin p f + b cos p f) for the
               pairs of the first `rot` channels of a head, f one frequency a pair
  recurrence   u = c softplus(lam) sigmoid(r), h <- exp(-u) h + sqrt(1 - exp(-2 u))
               sigmoid(i) x, out = h silu(z)
  block norm   s = residual + alpha scale act(gate) N(y; post), out = N(s; pre)
"""
import math
import random

import torch

own = False

EPS = 1e-6
C_DECAY = 8.0
TILE = 64  # tokens a saved state of the recurrence stands for
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# the largest case in elements of one activation
MOST = 4 * 4096 * 4096


def listed():
    return [
        # decoding: 32 requests at far positions, 32 query and 8 key heads
        dict(name="rotary_token", op="rotary", batch=32, t=1, hq=32, hk=8, d=128, rot=128, half=True, dtype="bf16", start=90000),
        # a batch of prompts, grouped heads, positions past the trained length by scaled frequencies
        dict(name="rotary_prompt", op="rotary", batch=4, t=4096, hq=32, hk=8, d=128, rot=128, half=True, dtype="bf16", start=0),
        # training heads of 112 channels of which 64 turn, interleaved: the rotation and its gradient
        dict(name="rotary_train", op="rotary_train", batch=2, t=8192, hq=16, hk=16, d=112, rot=64, half=False, dtype="bf16", start=0),
        # decoding one request: latency
        dict(name="lru_token_1", op="lru_step", reqs=1, pool=1, c=4096, dtype="bf16"),
        # decoding 256 requests out of a pool of 384 states
        dict(name="lru_token_256", op="lru_step", reqs=256, pool=384, c=4096, dtype="bf16"),
        # a batch of prompts, states kept for decoding
        dict(name="lru_prompt", op="lru", batch=4, t=4096, seqs=0, c=4096, dtype="bf16", gate=True, states=True),
        # one long prompt over few channels: too few rows to fill the GPU
        dict(name="lru_long", op="lru", batch=1, t=32768, seqs=0, c=1024, dtype="bf16", gate=True, states=True),
        # packed ragged prompts in fp32, a channel count that is no power of two
        dict(name="lru_packed_f32", op="lru", batch=1, t=5003, seqs=9, c=1792, dtype="f32", gate=False, states=True),
        # training: the outputs and every gradient
        dict(name="lru_train", op="lru_train", batch=4, t=4096, seqs=0, c=4096, dtype="bf16", gate=True, states=False),
        # decoding: 8 requests between two blocks
        dict(name="block_token", op="block", batch=8, t=1, d=2048, dtype="bf16", res="bf16", post=True, pre=True, gate="none", act="none", scale=False),
        # a prompt with an fp32 residual stream, a gate row a token
        dict(name="block_prompt", op="block", batch=4, t=4096, d=4096, dtype="bf16", res="f32", post=True, pre=True, gate="token", act="sigmoid", scale=True),
        # training a video block: one gate row a sequence, every gradient
        dict(name="block_train", op="block_train", batch=2, t=8192, d=1792, dtype="bf16", res="bf16", post=True, pre=True, gate="sequence", act="none", scale=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _channels(rng):
    d = _log(rng, 64, 8192)
    return d if rng.random() < 0.3 else max(8, d // 8 * 8)  # some odd, most of whole 16-byte rows


def draw(rng):
    op = rng.choice(["rotary", "rotary", "rotary_train", "lru_step", "lru", "lru", "lru_train", "lru_train", "block", "block", "block_train", "block_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("rotary"):
        d = rng.choice([64, 80, 96, 112, 128, 128, 192, 256])
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 1, 4, 8])
        rot = rng.choice([d, d, d // 2, d // 4])
        tokens = _log(rng, 1, max(1, MOST // 4 // (hq * d)))
        batch = rng.randint(1, min(8, tokens))
        if rng.random() < 0.3:
            batch, tokens = min(tokens, 256), min(tokens, 256)
        return dict(op=op, batch=batch, t=max(1, tokens // batch), hq=hq, hk=hk, d=d, rot=rot - rot % 2, half=rng.random() < 0.6, dtype=dtype, start=_log(rng, 1, 1000000))
    if op == "lru_step":
        reqs = _log(rng, 1, 256)
        return dict(op=op, reqs=reqs, pool=reqs + rng.randint(0, 64), c=min(4096, _channels(rng)), dtype=dtype)
    d = _channels(rng)
    t = _log(rng, 1, min(32768, MOST // 2 // d))
    if op.startswith("lru"):
        batch, seqs = 1, rng.randint(1, 40)
        if rng.random() < 0.5:
            batch, seqs = max(1, min(rng.randint(1, 8), MOST // 2 // d // t)), 0
        return dict(op=op, batch=batch, t=t, seqs=seqs, c=d, dtype=dtype, gate=rng.random() < 0.6, states=rng.random() < 0.5)
    batch = max(1, min(rng.randint(1, 8), MOST // 2 // d // t))
    post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
    return dict(op=op, batch=batch, t=t, d=d, dtype=dtype, res=rng.choice([dtype, "f32"]), post=post, pre=pre, gate=rng.choice(["none", "token", "sequence"]),
                act=rng.choice(["none", "sigmoid", "silu"]), scale=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs ---


def _lengths(case):
    """Token counts of a packed batch: uniform cuts, so some are short and a few may be empty."""
    r = random.Random(case["t"] * 1013 + case["seqs"])
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


def _prepare_rotary(m, case, s, ty):
    b, t, hq, hk, d, rot = (case[k] for k in ("batch", "t", "hq", "hk", "d", "rot"))
    qkv = m.normal(b, t, hq + 2 * hk, d, dtype=ty)
    s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq : hq + hk]
    s["half"], s["rot"] = case["half"], rot
    if t == 1:
        s["positions"] = torch.randint(0, case["start"] + 1, (b, 1), generator=m.g, device="cuda", dtype=torch.int32)
    else:
        s["positions"] = (case["start"] + torch.arange(t, device="cuda", dtype=torch.int32)).expand(b, t).contiguous()
    # frequencies of base 10000 for a context four times the trained one: the fast pairs
    # as they are, the slow ones four times slower, a ramp between them
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ramp = ((f * 8192 / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
    s["inv_freq"] = f * (ramp + (1 - ramp) / 4.0)
    s["scale"] = 0.1 * math.log(4.0) + 1.0
    if case["op"] == "rotary_train":
        s["dq"], s["dk"] = m.normal(b, t, hq, d, dtype=ty), m.normal(b, t, hk, d, dtype=ty)


def _prepare_lru(m, case, s, ty):
    c = case["c"]
    lead = (case["reqs"],) if case["op"] == "lru_step" else (case["batch"], case["t"])
    # x and z are the halves of one projection, the gates those of another
    xz, ri = m.normal(*lead, 2 * c, dtype=ty), m.normal(*lead, 2 * c, dtype=ty)
    s["x"], s["z"], s["r"], s["i"] = xz[..., :c], xz[..., c:], ri[..., :c], ri[..., c:]
    # exp(-c softplus(lam)) between 0.9 and 0.999: decays at an open gate
    s["lam"] = torch.log(torch.expm1(-torch.log(m.uniform(0.9, 0.999, c)) / C_DECAY))
    if case["op"] == "lru_step":
        s["state"] = m.normal(case["pool"], c)
        s["slots"] = torch.randperm(case["pool"], generator=m.g, device="cuda")[: case["reqs"]].to(torch.int32)
        return
    if not case["gate"]:
        s["z"] = None
    n = case["seqs"] or case["batch"]
    s["cu"] = None
    if case["seqs"]:
        at = [0]
        for k in _lengths(case):
            at.append(at[-1] + k)
        s["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    s["h0"] = m.normal(n, c) if case["states"] else None
    s["final"] = torch.empty(n, c, device="cuda") if case["states"] else None
    if case["op"] == "lru_train":
        s["dout"] = m.normal(*lead, c, dtype=ty)
        s["dfinal"] = m.normal(n, c) if case["states"] else None


def _prepare_block(m, case, s, ty):
    b, t, d = case["batch"], case["t"], case["d"]
    s["y"] = m.normal(b, t, d, dtype=ty)
    s["residual"] = m.normal(b, t, d, dtype=TYPES[case["res"]], std=2.0)
    s["post"] = m.normal(d, std=0.1, mean=1.0) if case["post"] else None
    s["pre"] = m.normal(d, std=0.1, mean=1.0) if case["pre"] else None
    s["gate"] = {"none": lambda: None, "token": lambda: m.normal(b, t, d, dtype=ty), "sequence": lambda: m.normal(b, 1, d, dtype=ty)}[case["gate"]]()
    s["act"] = None if case["act"] == "none" or s["gate"] is None else case["act"]
    s["scale"] = m.normal(d, std=0.1, mean=0.5) if case["scale"] else None
    s["alpha"] = 0.5
    if case["op"] == "block_train":
        s["dout"] = m.normal(b, t, d, dtype=ty) if case["pre"] else None
        s["dres"] = m.normal(b, t, d, dtype=TYPES[case["res"]])


def prepare(case, seed):
    m, ty = _Maker(seed), TYPES[case["dtype"]]
    s = dict(op=case["op"], ty=ty)
    {"rotary": _prepare_rotary, "lru": _prepare_lru, "block": _prepare_block}[case["op"].split("_")[0]](m, case, s, ty)
    return s


# ------------------------------------------------------------------- plain ---


def _turn(x, cos, sin, half, rot):
    """The first rot channels of x (fp32) turned, the others as they are."""
    y = x.float().clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * cos - v * sin, v * cos + u * sin
    return y.to(x.dtype)


def _plain_rotary(s):
    angle = s["positions"].double()[..., None, None] * s["inv_freq"]  # (fp64: far positions)
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    r = {n: _turn(s[n], cos, sin, s["half"], s["rot"]) for n in ("q", "k")}
    if "dq" in s:
        r.update({n: _turn(s[n], cos, -sin, s["half"], s["rot"]) for n in ("dq", "dk")})
    return r


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


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


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_lru(s):
    x, gr, gi = s["x"].float(), _sigmoid(s["r"].float()), _sigmoid(s["i"].float())
    u = C_DECAY * _softplus(s["lam"]) * gr
    a, beta = torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))
    b = beta * gi * x
    first, last, some = _bounds(s)
    if s["h0"] is not None:
        b.index_put_(first, a[first] * s["h0"] * some[:, None], accumulate=True)
    begins = torch.zeros(x.shape[:2], device="cuda").index_put_(first, some.float(), accumulate=True) > 0
    cut = a.masked_fill(begins[..., None], 0.0)
    h = _recur(cut.clone(), b)
    z = None if s["z"] is None else s["z"].float()
    r = dict(out=(h if z is None else h * z * _sigmoid(z)).to(s["ty"]))
    if s["final"] is not None:
        s["final"].copy_(torch.where(some[:, None], h[last], s["h0"]))
        r["final"] = s["final"]
    if s["op"] == "lru":
        return r
    do = g = s["dout"].float()
    if z is not None:
        gz = _sigmoid(z)
        r["dz"] = (do * h * gz * (1 + z * (1 - gz))).to(s["ty"])
        g = do * z * gz
    if s["dfinal"] is not None:
        g = g.clone().index_put_(last, s["dfinal"] * some[:, None], accumulate=True)
    # g_t += a_{t+1} g_{t+1}, with no step over a sequence's end
    nxt = torch.cat([torch.zeros_like(cut[:, :1]), cut[:, 1:].flip(1)], 1)
    g = _recur(nxt, g.flip(1)).flip(1)
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1).masked_fill_(begins[..., None], 0.0)
    if s["h0"] is not None:
        prev.index_put_(first, s["h0"] * some[:, None], accumulate=True)
        r["dh0"] = torch.where(some[:, None], (a * g)[first], s["dfinal"])
    r["dx"], r["di"] = (g * beta * gi).to(s["ty"]), (g * beta * x * gi * (1 - gi)).to(s["ty"])
    du = g * (u * a * a / beta * gi * x - u * a * prev)  # u times the gradient of u
    r["dr"] = (du * (1 - gr)).to(s["ty"])
    r["dlam"] = du.sum((0, 1)) * _sigmoid(s["lam"]) / _softplus(s["lam"])
    return r


def _plain_lru_step(s):
    at = s["slots"].long()
    x, z = s["x"].float(), s["z"].float()
    u = C_DECAY * _softplus(s["lam"]) * _sigmoid(s["r"].float())
    h = torch.exp(-u) * s["state"][at] + torch.sqrt(-torch.expm1(-2 * u)) * _sigmoid(s["i"].float()) * x
    s["state"][at] = h
    return dict(out=(h * z * _sigmoid(z)).to(s["ty"]), state=s["state"])


def _act(x, act):
    """The gate's factor and its derivative."""
    if act is None:
        return x, torch.ones_like(x)
    g = _sigmoid(x)
    return (g, g * (1 - g)) if act == "sigmoid" else (x * g, g * (1 + x * (1 - g)))


def _norm(x, w):
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * inv * w, inv


def _dnorm(x, inv, w, g):
    gw = g * w
    return inv * gw - x * inv**3 * (gw * x).mean(-1, keepdim=True)


def _plain_block(s):
    y = s["y"].float()
    u, inv = (y, None) if s["post"] is None else _norm(y, s["post"])
    f, df = (1.0, None) if s["gate"] is None else _act(s["gate"].float(), s["act"])
    k = s["alpha"] if s["scale"] is None else s["alpha"] * s["scale"]
    t = s["residual"].float() + k * f * u
    r = dict(residual=t.to(s["residual"].dtype))
    if s["pre"] is not None:
        r["out"] = _norm(t, s["pre"])[0].to(s["ty"])
    if s["op"] == "block":
        return r
    t, ds = r["residual"].float(), s["dres"].float()  # the gradient takes the sum as stored
    if s["pre"] is not None:
        do = s["dout"].float()
        _, inv_s = _norm(t, s["pre"])
        ds = ds + _dnorm(t, inv_s, s["pre"], do)
        r["dpre_weight"] = (do * t * inv_s).sum((0, 1))
    r["dresidual"] = ds.to(s["residual"].dtype)
    if s["scale"] is not None:
        r["dscale"] = (ds * s["alpha"] * f * u).sum((0, 1))
    if s["gate"] is not None:
        dg = ds * k * u * df
        r["dgate"] = (dg if dg.shape == s["gate"].shape else dg.sum(1, keepdim=True)).to(s["ty"])
    du = ds * k * f
    if s["post"] is not None:
        r["dpost_weight"] = (du * y * inv).sum((0, 1))
        du = _dnorm(y, inv, s["post"], du)
    r["dy"] = du.to(s["ty"])
    return r


PLAIN = {"rotary": _plain_rotary, "rotary_train": _plain_rotary, "lru": _plain_lru, "lru_train": _plain_lru, "lru_step": _plain_lru_step, "block": _plain_block, "block_train": _plain_block}


# --------------------------------------------------------------- framework ---


def _own_rotary(gdn, s):
    kw = dict(positions=s["positions"], interleaved=not s["half"], scale=s["scale"])
    q, k = gdn.gdn_rotary(s["q"], s["inv_freq"], k=s["k"], **kw)
    r = dict(q=q, k=k)
    if "dq" in s:
        r["dq"], r["dk"] = gdn.gdn_rotary(s["dq"], s["inv_freq"], k=s["dk"], inverse=True, **kw)
    return r


def _own_lru(gdn, s):
    b, t, c = s["x"].shape
    args, kw = (s["x"], s["r"], s["i"], s["lam"]), dict(z=s["z"], c=C_DECAY, h0=s["h0"], cu_seqlens=s["cu"])
    saved = None
    if s["op"] == "lru_train":
        saved = torch.empty(b, -(-t // TILE), c, device=s["x"].device)
    r = dict(out=gdn.gdn_lru_fwd(*args, h_final=s["final"], checkpoints=saved, **kw))
    if s["final"] is not None:
        r["final"] = s["final"]
    if s["op"] == "lru_train":
        r.update(gdn.gdn_lru_bwd(*args, s["dout"], dh_final=s["dfinal"], checkpoints=saved, **kw))
    return r


def _own_lru_step(gdn, s):
    out = gdn.gdn_lru_step(s["x"], s["r"], s["i"], s["lam"], s["state"], z=s["z"], c=C_DECAY, slots=s["slots"])
    return dict(out=out, state=s["state"])


def _own_block(gdn, s):
    kw = dict(post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"], gate_act=s["act"], scale=s["scale"], alpha=s["alpha"], eps=EPS)
    r = gdn.gdn_block_norm_fwd(s["y"], s["residual"], **kw)
    if s["op"] == "block_train":
        r.update(gdn.gdn_block_norm_bwd(s["y"], r["residual"], dout=s["dout"], dres=s["dres"], **kw))
    return r


OWN = {"rotary": _own_rotary, "rotary_train": _own_rotary, "lru": _own_lru, "lru_train": _own_lru, "lru_step": _own_lru_step, "block": _own_block, "block_train": _own_block}


def run(state):
    if own:
        import gated_delta_rule_18_gb300 as gdn

        return OWN[state["op"]](gdn, state)
    return PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work ---


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("rotary"):
        tok, heads = case["batch"] * case["t"], case["hq"] + case["hk"]
        passes = 2 if op == "rotary_train" else 1
        return dict(bytes=passes * 2 * e * tok * heads * case["d"] + 4 * tok + 4 * case["rot"], flops=passes * 3 * tok * heads * case["rot"])
    if op == "lru_step":
        n, c = case["reqs"], case["c"]
        return dict(bytes=n * c * (8 + 5 * e) + 4 * n + 4 * c, flops=20 * n * c)
    if op.startswith("lru"):
        c, el = case["c"], case["batch"] * case["t"] * case["c"]
        n, z = case["seqs"] or case["batch"], 1 if case["gate"] else 0
        states = 4 * n * c * (2 if op == "lru" else 4) if case["states"] else 0
        moved = el * e * (4 + z)
        if op == "lru_train":  # x, r, i, z and dout again, dx, dr, di and dz
            moved += el * e * (7 + 2 * z) + 4 * c
        return dict(bytes=moved + states + 4 * c, flops=el * (20 if op == "lru" else 70))
    d, el, r = case["d"], case["batch"] * case["t"] * case["d"], 2 if case["res"] == "bf16" else 4
    pre = 1 if case["pre"] else 0
    gate = e * {"none": 0, "token": el, "sequence": case["batch"] * d}[case["gate"]]
    vectors = 4 * d * (pre + (1 if case["post"] else 0) + (1 if case["scale"] else 0))
    moved = el * (e * (1 + pre) + 2 * r) + gate + vectors
    if op == "block_train":  # y, s, the gate, dout and the stream's gradient; dy, its gradient, the gate's
        moved += el * (e * (2 + pre) + 3 * r) + 2 * gate + 2 * vectors
    return dict(bytes=moved, flops=el * (14 if op == "block" else 50))


# ------------------------------------------------------------------- exact ---


def _exact_rotary(s):
    def turned(x, back):
        f = torch.arange(s["rot"] // 2, device="cuda")
        i = f if s["half"] else 2 * f
        j = f + s["rot"] // 2 if s["half"] else 2 * f + 1
        angle = s["positions"].double().unsqueeze(-1) * s["inv_freq"] * (-1 if back else 1)
        w = torch.polar(torch.full_like(angle, s["scale"]), angle)
        v = torch.complex(x[..., i].double(), x[..., j].double()) * w.unsqueeze(2)
        out = x.double()
        out[..., i], out[..., j] = v.real, v.imag
        return out

    r = dict(q=turned(s["q"], False), k=turned(s["k"], False))
    if "dq" in s:
        r.update(dq=turned(s["dq"], True), dk=turned(s["dk"], True))
    return r


def _exact_spans(s):
    """(rows, first token, end, rows of the states) of the parts that are walked on their own."""
    if s["cu"] is None:
        return [(slice(None), 0, s["x"].shape[1], slice(None))]
    at = s["cu"].tolist()
    return [(slice(0, 1), p, q, slice(k, k + 1)) for k, (p, q) in enumerate(zip(at[:-1], at[1:]))]


def _exact_lru(s):
    """Token by token in fp64; the gradients of a_t and b_t by the walk back, of what they are made of by autograd."""
    train = s["op"] == "lru_train"
    leaf = {k: s[k].double().requires_grad_(train) for k in ("x", "r", "i", "lam", "z") if s[k] is not None}
    u = C_DECAY * torch.nn.functional.softplus(leaf["lam"], threshold=100) * torch.sigmoid(leaf["r"])
    a, b = torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u)) * torch.sigmoid(leaf["i"]) * leaf["x"]
    av, bv = a.detach(), b.detach()
    rows, _, c = av.shape
    h = torch.empty_like(av)
    n = rows if s["cu"] is None else s["cu"].numel() - 1
    h0 = torch.zeros(n, c, device="cuda", dtype=torch.float64) if s["h0"] is None else s["h0"].double()
    final = h0.clone()
    for row, p, q, k in _exact_spans(s):
        st = h0[k]
        for t in range(p, q):
            st = torch.addcmul(bv[row, t], av[row, t], st)
            h[row, t] = st
        final[k] = st
    out = h if s["z"] is None else h * torch.nn.functional.silu(leaf["z"])
    r = dict(out=out.detach())
    if s["final"] is not None:
        r["final"] = final
    if not train:
        return r
    do = s["dout"].double()
    g = do if s["z"] is None else do * torch.nn.functional.silu(leaf["z"].detach())
    da, db, dh0 = torch.empty_like(av), torch.empty_like(av), torch.zeros_like(h0)
    for row, p, q, k in _exact_spans(s):
        back = s["dfinal"][k].double() if s["dfinal"] is not None else torch.zeros_like(h0[k])
        for t in reversed(range(p, q)):
            back = back + g[row, t]
            db[row, t] = back
            da[row, t] = back * (h[row, t - 1] if t > p else h0[k])
            back = back * av[row, t]
        dh0[k] = back
    loss = (a * da).sum() + (b * db).sum()
    if s["z"] is not None:
        loss = loss + (out * do).sum()
    r.update(zip(("d" + k for k in leaf), torch.autograd.grad(loss, tuple(leaf.values()))))
    if s["h0"] is not None:
        r["dh0"] = dh0
    return r


def _exact_lru_step(s):
    state, at = s["state"].double(), s["slots"].long()
    x, r, i, z, lam = (s[k].double() for k in ("x", "r", "i", "z", "lam"))
    a = torch.sigmoid(-lam) ** (C_DECAY * torch.sigmoid(r))  # exp(-softplus(v)) = sigmoid(-v)
    state[at] = a * state[at] + torch.sqrt((1 - a) * (1 + a)) * torch.sigmoid(i) * x
    return dict(out=state[at] * torch.nn.functional.silu(z), state=state)


def _exact_block(s):
    train = s["op"] == "block_train"
    names = dict(y="dy", residual="dresidual", post="dpost_weight", pre="dpre_weight", gate="dgate", scale="dscale")
    leaf = {k: s[k].double().requires_grad_(train) for k in names if s[k] is not None}

    def norm(x, w):
        return leaf[w] * (x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS))

    v = norm(leaf["y"], "post") if "post" in leaf else leaf["y"]
    if "gate" in leaf:
        v = v * {None: lambda x: x, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[s["act"]](leaf["gate"])
    t = leaf["residual"] + s["alpha"] * v * leaf.get("scale", 1.0)
    r = dict(residual=t.detach())
    if not train:
        return dict(r, out=norm(t, "pre")) if "pre" in leaf else r
    loss = (t * s["dres"].double()).sum()
    if "pre" in leaf:
        r["out"] = norm(t.detach(), "pre").detach()
        # the second norm's gradient is taken at the sum as stored
        rounded = t + (t.detach().to(s["residual"].dtype).double() - t.detach())
        loss = loss + (norm(rounded, "pre") * s["dout"].double()).sum()
    return dict(r, **dict(zip((names[k] for k in leaf), torch.autograd.grad(loss, tuple(leaf.values())))))


EXACT = {"rotary": _exact_rotary, "rotary_train": _exact_rotary, "lru": _exact_lru, "lru_train": _exact_lru, "lru_step": _exact_lru_step, "block": _exact_block, "block_train": _exact_block}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
