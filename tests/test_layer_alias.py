"""Outputs that overlap inputs, or their own rows, are refused on the host: the
C entry points with fake device addresses that nothing dereferences. Calls
that pass the checks stop at a missing workspace."""
import pytest

import gated_delta_rule_18_gb300 as gdn
from gated_delta_rule_18_gb300.build import build
from test_layer_abi import (CONV, CONV_BWD, CONV_STEP, LAYOUT, NORM, NORM_BWD, SSM, SSM_BWD, STEP, UNSUP, WS, call, p)


@pytest.fixture(scope="module")
def L():
    build()
    return gdn.lib()


# tensors of the specs: 2 x 100 tokens (4 rows in NORM, 3 in the steps) of 64 bf16 channels, rows of 128 bytes,
# lines of 12800, states fp32
LINE, ROW = 12800, 128


@pytest.mark.parametrize("fn,spec,kw", [
    ("gdn_rmsnorm_fwd", NORM, dict(out=p(0) + 16)), ("gdn_rmsnorm_fwd", NORM, dict(out=p(0) + ROW)),
    ("gdn_rmsnorm_fwd", NORM, dict(ro=p(1) + 256)), ("gdn_rmsnorm_fwd", NORM, dict(ro=p(0))),  # fp32 over bf16
    ("gdn_rmsnorm_fwd", NORM, dict(out=p(4))), ("gdn_rmsnorm_fwd", NORM, dict(out=p(1))),
    ("gdn_rmsnorm_fwd", NORM, dict(out=p(0), out_st=128)),
    ("gdn_rmsnorm_fwd", NORM, dict(out_dtype=2, out=p(0), scale=p(5))),
    ("gdn_rmsnorm_fwd", NORM, dict(out_dtype=2, scale=p(3))),
    ("gdn_rmsnorm_bwd", NORM_BWD, dict(dx=p(0) + ROW)), ("gdn_rmsnorm_bwd", NORM_BWD, dict(dx=p(1) - ROW)),
    ("gdn_conv_fwd", CONV, dict(out=p(0))), ("gdn_conv_fwd", CONV, dict(out=p(0) + ROW)),
    ("gdn_conv_fwd", CONV, dict(out=p(0) + LINE)), ("gdn_conv_fwd", CONV, dict(out=p(0) - LINE - 99 * ROW)),
    ("gdn_conv_fwd", CONV, dict(x_st=128, x_sb=12800, out=p(0) + ROW - 16, o_st=128, o_sb=12800)),
    ("gdn_conv_fwd", CONV, dict(final=p(3))), ("gdn_conv_fwd", CONV, dict(final=p(3) + 16)),
    ("gdn_conv_fwd", CONV, dict(final=p(0) + 64)), ("gdn_conv_fwd", CONV, dict(final=p(4) + 64)),
    ("gdn_conv_fwd", CONV, dict(out=p(3) + 16)),
    ("gdn_conv_bwd", CONV_BWD, dict(dx=p(0))), ("gdn_conv_bwd", CONV_BWD, dict(dx=p(4) + ROW)),
    ("gdn_conv_bwd", CONV_BWD, dict(dinit=p(3))), ("gdn_conv_bwd", CONV_BWD, dict(dinit=p(5) + 16)),
    ("gdn_conv_step", CONV_STEP, dict(out=p(0) + 16)), ("gdn_conv_step", CONV_STEP, dict(out=p(2) + 16)),
    ("gdn_conv_step", CONV_STEP, dict(x=p(2) + 16)),
    ("gdn_ssm_fwd", SSM, dict(out=p(0) + ROW)), ("gdn_ssm_fwd", SSM, dict(out=p(6) + 16)),
    ("gdn_ssm_fwd", SSM, dict(out=p(3))), ("gdn_ssm_fwd", SSM, dict(out=p(4) + ROW)),
    ("gdn_ssm_fwd", SSM, dict(h_final=p(8))), ("gdn_ssm_fwd", SSM, dict(h_final=p(8) + 16)),
    ("gdn_ssm_fwd", SSM, dict(h_final=p(9) + 16)), ("gdn_ssm_fwd", SSM, dict(h_final=p(0) + 16)),
    ("gdn_ssm_bwd", SSM_BWD, dict(dx=p(9) + ROW)), ("gdn_ssm_bwd", SSM_BWD, dict(dbm=p(3))),
    ("gdn_ssm_bwd", SSM_BWD, dict(dx=p(12))), ("gdn_ssm_bwd", SSM_BWD, dict(dh0=p(8))),
    ("gdn_ssm_bwd", SSM_BWD, dict(dh0=p(10) + 16)),
    ("gdn_ssm_step", STEP, dict(out=p(0) + 16)), ("gdn_ssm_step", STEP, dict(out=p(3))),
    ("gdn_ssm_step", STEP, dict(out=p(5) + 16)), ("gdn_ssm_step", STEP, dict(x=p(5) + 16)),
])
def test_overlapping_outputs_are_refused(L, fn, spec, kw):
    assert call(getattr(L, fn), spec, **kw) == UNSUP


@pytest.mark.parametrize("fn,spec,kw", [
    ("gdn_rmsnorm_fwd", NORM, dict(out_st=0)), ("gdn_rmsnorm_fwd", NORM, dict(ro_st=63)),
    ("gdn_rmsnorm_bwd", NORM_BWD, dict(dx_st=32)), ("gdn_conv_fwd", CONV, dict(o_st=0)),
    ("gdn_conv_fwd", CONV, dict(o_sb=0)), ("gdn_conv_fwd", CONV, dict(o_sb=64 * 99)),
    ("gdn_conv_fwd", CONV, dict(o_sb=32, o_st=128)), ("gdn_ssm_fwd", SSM, dict(out_sb=64)),
    ("gdn_ssm_fwd", SSM, dict(out_st=8)), ("gdn_conv_step", CONV_STEP, dict(out_st=8)),
    ("gdn_ssm_step", STEP, dict(out_st=0)),
])
def test_outputs_whose_rows_overlap_are_refused(L, fn, spec, kw):
    assert call(getattr(L, fn), spec, **kw) == LAYOUT


@pytest.mark.parametrize("fn,spec,kw", [
    # halves of rows of one tensor, lines between lines, tokens between tokens
    ("gdn_ssm_fwd", SSM, dict(x_st=128, x_sb=12800, out=p(0) + ROW, out_st=128, out_sb=12800)),
    ("gdn_ssm_fwd", SSM, dict(x_sb=2 * 6400, out=p(0) + LINE, out_sb=2 * 6400)),
    ("gdn_ssm_fwd", SSM, dict(out=p(0) + 2 * LINE)), ("gdn_ssm_fwd", SSM, dict(out=p(0) - 2 * LINE)),
    ("gdn_ssm_fwd", SSM, dict(x_st=192, x_sb=19200, out=p(0) + ROW, out_st=384, out_sb=38400)),
    ("gdn_ssm_fwd", SSM, dict(out_sb=64, out_st=128)),                       # lines interleaved by token
    ("gdn_ssm_fwd", SSM, dict(out=p(0))), ("gdn_ssm_fwd", SSM, dict(out=p(6))),  # in place, element by element
    ("gdn_ssm_fwd", SSM, dict(bm=p(0), cm=p(0) + 32, z=p(0))),               # inputs may share
    ("gdn_ssm_fwd", SSM, dict(x_sb=0, x_st=0)),                              # and repeat
    ("gdn_ssm_bwd", SSM_BWD, dict(dx=p(9))), ("gdn_rmsnorm_bwd", NORM_BWD, dict(dx=p(0))),
    ("gdn_conv_fwd", CONV, dict(cu=p(30), B=1, n_seq=2, x_st=128, out=p(0) + ROW, o_st=128)),
])
def test_outputs_apart_from_inputs_pass(L, fn, spec, kw):
    assert call(getattr(L, fn), spec, ws=0, **kw) == WS


def test_overlap_agrees_with_the_bytes(L):
    """Random small layouts of x and out against the sets of their elements."""
    import random
    rng, seen = random.Random(0), set()
    for _ in range(6000):
        B, T, D = rng.randint(1, 3), rng.randint(1, 5), rng.randint(1, 4)
        x_sb, x_st, o_sb, o_st = (rng.randint(0, 24) for _ in range(4))
        if rng.random() < 0.5:
            o_sb, o_st = x_sb, x_st
        shift = rng.randint(-40, 40)
        at = lambda base, sb, st: [base + b * sb + t * st + d for b in range(B) for t in range(T) for d in range(D)]  # noqa: E731
        x, out = at(0, x_sb, x_st), at(shift, o_sb, o_st)
        same = shift == 0 and (B == 1 or x_sb == o_sb) and (T == 1 or x_st == o_st)
        want = LAYOUT if len(set(out)) < len(out) else UNSUP if set(x) & set(out) and not same else WS
        got = call(L.gdn_ssm_fwd, SSM, B=B, T=T, D=D, n_seq=B, x_sb=x_sb, x_st=x_st, out=p(0) + 2 * shift, out_sb=o_sb,
                   out_st=o_st, ws=0)
        assert got == want, (B, T, D, x_sb, x_st, o_sb, o_st, shift)
        seen.add(got)
    assert seen == {LAYOUT, UNSUP, WS}
