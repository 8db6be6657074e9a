"""The entry points of the block's operators refuse bad arguments on the host,
before any launch (no GPU needed), with fake device addresses that nothing
dereferences; calls that pass every check stop at a missing workspace or do
nothing."""
import pytest

import gated_delta_rule_18_gb300 as gdn
from gated_delta_rule_18_gb300.build import build
from test_layer_abi import BIG, DTYPE, LAYOUT, NULL, OK, SHAPE, UNSUP, WS, call, p


@pytest.fixture(scope="module")
def L():
    build()
    return gdn.lib()


INF, NAN = float("inf"), float("nan")


def heads(name, i, h=4):
    return [(name, p(i)), (name + "_sb", 100 * h * 64), (name + "_st", h * 64), (name + "_sh", 64)]


ROTARY = (heads("q", 0) + [("Hq", 4)] + heads("qo", 1) + heads("k", 2, 2) + [("Hk", 2)] + heads("ko", 3, 2) +
          [("freq", p(4)), ("pos", p(5)), ("bits", 32), ("pos_sb", 100), ("pos_st", 1), ("offset", 0), ("B", 2), ("T", 100),
           ("D", 64), ("rot", 32), ("scale", 1.0), ("dtype", 1), ("flags", 0), ("stream", 0)])
NOTHING = dict(B=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), NULL), (dict(qo=0), NULL), (dict(k=0), NULL), (dict(ko=0), NULL), (dict(freq=0), NULL),
    (dict(Hq=0), SHAPE), (dict(Hk=0), SHAPE), (dict(k=0, ko=0), SHAPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(B=65536, T=65536), SHAPE), (dict(D=0), SHAPE), (dict(D=513), SHAPE), (dict(rot=0), SHAPE), (dict(rot=31), SHAPE),
    (dict(rot=66), SHAPE), (dict(Hq=65536), SHAPE), (dict(dtype=2), DTYPE), (dict(bits=16), DTYPE), (dict(flags=4), UNSUP),
    (dict(q=p(0) + 1), LAYOUT), (dict(q_st=-256), LAYOUT), (dict(freq=p(4) + 4), LAYOUT), (dict(pos=p(5) + 2), LAYOUT),
    (dict(pos=p(5) + 4, bits=64), LAYOUT), (dict(pos_st=-1), LAYOUT),
    # outputs whose rows share bytes, overlap an input, one another
    (dict(qo_sh=32), LAYOUT), (dict(qo_st=0), LAYOUT), (dict(qo_sb=0), LAYOUT),
    (dict(qo=p(0) + 128), UNSUP), (dict(qo=p(2)), UNSUP), (dict(ko=p(0)), UNSUP), (dict(ko=p(1)), UNSUP),
    (dict(qo=p(0), qo_st=512, qo_sb=51200), UNSUP),
    (NOTHING, OK), (dict(T=0), OK), (dict(NOTHING, k=0, ko=0, Hk=0), OK), (dict(NOTHING, pos=0, bits=0), OK),
])
def test_rotary_refuses(L, kw, code):
    assert call(L.gdn_rotary, ROTARY, **kw) == code


def test_rotary_overlap_agrees_with_the_bytes(L):
    """Random small layouts of q and its output against the sets of their elements: every overlap is refused, by the
    status of its kind where two strides describe the rows (three separate ones are judged by ranges)."""
    import random
    rng, seen = random.Random(1), set()
    for _ in range(6000):
        n = [rng.randint(1, 3) for _ in range(3)]
        qs, os_ = ([rng.randint(0, 30) for _ in range(3)] for _ in range(2))
        if rng.random() < 0.5:
            os_ = list(qs)
        shift = rng.choice([0, rng.randint(-150, 150)])
        at = lambda base, s: [base + b * s[0] + t * s[1] + h * s[2] + d  # noqa: E731
                              for b in range(n[0]) for t in range(n[1]) for h in range(n[2]) for d in range(2)]
        q, out = at(0, qs), at(shift, os_)
        same = shift == 0 and all(k == 1 or a == b for k, a, b in zip(n, qs, os_))
        want = LAYOUT if len(set(out)) < len(out) else UNSUP if set(q) & set(out) and not same else OK
        if want == OK:
            continue  # it would launch
        got = call(L.gdn_rotary, ROTARY, k=0, ko=0, Hk=0, B=n[0], T=n[1], Hq=n[2], D=2, rot=2, qo=p(0) + 2 * shift,
                   q_sb=qs[0], q_st=qs[1], q_sh=qs[2], qo_sb=os_[0], qo_st=os_[1], qo_sh=os_[2])
        assert got == want or (min(n) > 1 and got in (LAYOUT, UNSUP)), (n, qs, os_, shift)
        seen.add(got)
    assert seen == {LAYOUT, UNSUP}


BLOCK = [("y", p(0)), ("y_st", 64), ("y_dtype", 1), ("res", p(1)), ("res_st", 64), ("res_dtype", 0), ("gate", p(2)),
         ("gate_st", 64), ("gate_rows", 1), ("act", 2), ("post", p(3)), ("pre", p(4)), ("scale", p(5)), ("alpha", 1.0),
         ("ro", p(6)), ("ro_st", 64), ("out", p(7)), ("out_st", 64), ("R", 6), ("D", 64), ("eps", 1e-6), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(y=0), NULL), (dict(res=0), NULL), (dict(ro=0), NULL), (dict(out=0), NULL), (dict(pre=0), NULL),
    (dict(post=0, pre=0, out=0), NULL), (dict(gate=0), SHAPE), (dict(act=0), SHAPE), (dict(act=4), SHAPE), (dict(act=-1), SHAPE),
    (dict(gate_rows=4), SHAPE), (dict(gate_rows=0), SHAPE), (dict(gate=0, act=0, gate_rows=2), SHAPE),
    (dict(R=2 * 65536, gate_rows=2), SHAPE), (dict(R=-1), SHAPE), (dict(R=2**31 - 1), SHAPE), (dict(D=0), SHAPE),
    (dict(D=16385), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(y_dtype=2), DTYPE), (dict(res_dtype=2), DTYPE),
    (dict(y=p(0) + 1), LAYOUT), (dict(gate_st=-1), LAYOUT), (dict(scale=p(5) + 2), LAYOUT), (dict(ro_st=32), LAYOUT),
    (dict(out_st=0), LAYOUT), (dict(ro=p(1) + 256), UNSUP), (dict(out=p(0) + 128), UNSUP), (dict(out=p(1)), UNSUP),
    (dict(ro=p(7)), UNSUP), (dict(gate_rows=2, out=p(2)), UNSUP), (dict(R=0), OK),
])
def test_block_norm_fwd_refuses(L, kw, code):
    assert call(L.gdn_block_norm_fwd, BLOCK, **kw) == code


BLOCK_BWD = [("y", p(0)), ("y_st", 64), ("y_dtype", 1), ("s", p(1)), ("s_st", 64), ("s_dtype", 0), ("gate", p(2)),
             ("gate_st", 64), ("gate_rows", 1), ("act", 2), ("dout", p(3)), ("dout_st", 64), ("dres", p(4)), ("dres_st", 64),
             ("post", p(5)), ("pre", p(6)), ("scale", p(7)), ("alpha", 1.0), ("dy", p(8)), ("dy_st", 64), ("ds", p(9)),
             ("ds_st", 64), ("dgate", p(10)), ("dgate_st", 64), ("dpost", p(11)), ("dpre", p(12)), ("dscale", p(13)), ("R", 6),
             ("D", 64), ("eps", 1e-6), ("ws", p(14)), ("ws_bytes", BIG), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(y=0), NULL), (dict(s=0), NULL), (dict(dout=0), NULL), (dict(dy=0), NULL), (dict(ds=0), NULL), (dict(dgate=0), NULL),
    (dict(post=0), NULL), (dict(pre=0), NULL), (dict(scale=0), NULL), (dict(post=0, pre=0, dpost=0, dpre=0), NULL),
    (dict(pre=0, dpre=0, dres=0), NULL), (dict(gate=0), NULL), (dict(gate=0, dgate=0), SHAPE), (dict(gate_rows=4), SHAPE),
    (dict(D=20000), SHAPE), (dict(eps=NAN), SHAPE), (dict(s_dtype=2), DTYPE), (dict(dy=p(8) + 1), LAYOUT),
    (dict(dscale=p(13) + 2), LAYOUT), (dict(dy=p(0)), UNSUP), (dict(ds=p(4)), UNSUP), (dict(dgate=p(2)), UNSUP),
    (dict(dpost=p(5)), UNSUP), (dict(dy=p(9)), UNSUP), (dict(ds_st=32), LAYOUT), (dict(ws=0), WS), (dict(ws_bytes=256), WS),
    (dict(ws=p(14) + 16), WS), (dict(dres=0, ws=0), WS), (dict(pre=0, dpre=0, s=0, dout=0, ws=0), WS),
    (dict(gate_rows=3, ws=0), WS),
])
def test_block_norm_bwd_refuses(L, kw, code):
    assert call(L.gdn_block_norm_bwd, BLOCK_BWD, **kw) == code


def test_block_norm_workspace_sizes(L):
    size = L.gdn_block_norm_bwd_workspace_size
    assert size(-1, 64, 1) == size(6, 0, 1) == size(6, 64, 0) == size(6, 64, 4) == size(2 * 65536, 64, 2) == 0
    assert size(6, 64, 3) > size(6, 64, 1) > 0 and size(0, 64, 1) > 0
    # the parts are never more than the rows they stand for, nor more than four a SM and sequence
    assert size(10**6, 4096, 1) <= 608 * 2 * 4096 * 4 + 4096


def test_block_norm_workspace_of_an_empty_batch(L):
    """A shared gate without rows: a size, and no division by the number of its rows."""
    assert L.gdn_block_norm_bwd_workspace_size(0, 64, 5) > 0


def act(name, i):
    return [(name, p(i)), (name + "_sb", 6400), (name + "_st", 64)]


SCAN = act("x", 0) + act("r", 1) + act("i", 2) + [("lam", p(3))] + act("z", 4) + [("c", 8.0), ("h0", p(5)), ("cu", 0), ("n_seq", 2)]
TAIL = [("B", 2), ("T", 100), ("C", 64), ("dtype", 1), ("ws", p(20)), ("ws_bytes", BIG), ("stream", 0)]
LRU = SCAN + act("out", 6) + [("h_final", p(7)), ("ck", p(8))] + TAIL


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(r=0), NULL), (dict(i=0), NULL), (dict(lam=0), NULL), (dict(out=0), NULL), (dict(B=0), SHAPE),
    (dict(B=65536), SHAPE), (dict(T=-1), SHAPE), (dict(T=2**31 - 1), SHAPE), (dict(C=0), SHAPE), (dict(C=(1 << 20) + 1), SHAPE),
    (dict(n_seq=3), SHAPE), (dict(cu=p(9)), SHAPE), (dict(cu=p(9), B=1, n_seq=0), SHAPE), (dict(c=-1.0), SHAPE),
    (dict(c=NAN), SHAPE), (dict(c=INF), SHAPE), (dict(dtype=2), DTYPE), (dict(x=p(0) + 1), LAYOUT), (dict(z_st=-64), LAYOUT),
    (dict(lam=p(3) + 2), LAYOUT), (dict(h0=p(5) + 2), LAYOUT), (dict(ck=p(8) + 1), LAYOUT), (dict(h_final=p(7) + 1), LAYOUT),
    (dict(out_st=32), LAYOUT), (dict(out=p(0) + 128), UNSUP), (dict(out=p(4), out_st=128, out_sb=12800), UNSUP),
    (dict(h_final=p(5)), UNSUP), (dict(ck=p(7)), UNSUP), (dict(ck=p(0)), UNSUP), (dict(h_final=p(3)), UNSUP),
    (dict(cu=p(9), B=1, n_seq=3, ws=0), WS), (dict(cu=p(9), B=1, n_seq=3, ws_bytes=8), WS),
    (dict(cu=p(9) + 2, B=1, n_seq=3), LAYOUT), (dict(T=0, h_final=0), OK),
    # in place, element by element, is what passes: the call then stops at the workspace
    (dict(out=p(0), cu=p(9), B=1, n_seq=3, ws=0), WS), (dict(out=p(4), cu=p(9), B=1, n_seq=3, ws=0), WS),
])
def test_lru_fwd_refuses(L, kw, code):
    assert call(L.gdn_lru_fwd, LRU, **kw) == code


LRU_BWD = SCAN + act("dout", 6) + [("dh_final", p(7)), ("ck", p(8)), ("dx", p(10)), ("dr", p(11)), ("di", p(12)), ("dlam", p(13)),
                                   ("dz", p(14)), ("dh0", p(15))] + TAIL


@pytest.mark.parametrize("kw,code", [
    (dict(dout=0), NULL), (dict(dx=0), NULL), (dict(dr=0), NULL), (dict(di=0), NULL), (dict(dlam=0), NULL), (dict(dz=0), NULL),
    (dict(z=0), NULL), (dict(h0=0), NULL), (dict(n_seq=1), SHAPE), (dict(c=NAN), SHAPE), (dict(dtype=5), DTYPE),
    (dict(dlam=p(13) + 2), LAYOUT), (dict(dx=p(10) + 1), LAYOUT), (dict(dx=p(0)), UNSUP), (dict(dx=p(6)), UNSUP),
    (dict(dr=p(10)), UNSUP), (dict(dh0=p(5)), UNSUP), (dict(dh0=p(8)), UNSUP), (dict(ws=0), WS), (dict(ws_bytes=256), WS),
    (dict(ws=p(20) + 16), WS), (dict(dh0=0, ws=0), WS), (dict(z=0, dz=0, ws=0), WS),
])
def test_lru_bwd_refuses(L, kw, code):
    assert call(L.gdn_lru_bwd, LRU_BWD, **kw) == code


def test_lru_workspace_sizes(L):
    size = L.gdn_lru_bwd_workspace_size
    assert size(0, 5, 64, 0) == size(1, -1, 64, 0) == size(1, 2**31 - 1, 64, 0) == size(1, 5, 0, 1) == 0
    assert size(2, 1000, 64, 0) - size(2, 1000, 64, 1) == 2 * 16 * 64 * 4
    assert size(1, 2**31 - 2**16, 64, 0) > 2**32  # 64-bit sums


STEP = [("x", p(0)), ("x_st", 64), ("r", p(1)), ("r_st", 64), ("i", p(2)), ("i_st", 64), ("lam", p(3)), ("z", p(4)), ("z_st", 64),
        ("c", 8.0), ("state", p(5)), ("slots", p(6)), ("n_slots", 8), ("out", p(7)), ("out_st", 64), ("n", 3), ("C", 64),
        ("dtype", 1), ("stream", 0)]


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), NULL), (dict(lam=0), NULL), (dict(state=0), NULL), (dict(out=0), NULL), (dict(n=-1), SHAPE), (dict(n=70000), SHAPE),
    (dict(slots=0, n=9), SHAPE), (dict(n_slots=-1), SHAPE), (dict(C=0), SHAPE), (dict(c=-2.0), SHAPE), (dict(dtype=3), DTYPE),
    (dict(state=p(5) + 2), LAYOUT), (dict(slots=p(6) + 1), LAYOUT), (dict(i_st=-1), LAYOUT), (dict(out_st=8), LAYOUT),
    (dict(out=p(0) + 16), UNSUP), (dict(out=p(5) + 16), UNSUP), (dict(x=p(5) + 16), UNSUP), (dict(state=p(3)), UNSUP), (dict(n=0), OK),
])
def test_lru_step_refuses(L, kw, code):
    assert call(L.gdn_lru_step, STEP, **kw) == code
