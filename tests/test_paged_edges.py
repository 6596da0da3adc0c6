"""Edges of the paged operators (GPU): ill-formed boundaries, waits that run
out, extreme sinks and scales, full sequences, and the sizes at which a
kernel's rule takes another form.  Tolerances are test_paged.py's unless a test
derives its own."""
import numpy as np
import pytest
import torch

from oracle import paged as OP
from tests.paged_cases import Case, values
from tests.test_paged import append, attend, check_append, check_attend, fa  # noqa: F401

pytestmark = pytest.mark.gpu
INVALID = 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mn", [2, 64])
def test_falling_boundaries_leave_the_others_right(fa, mn, fp8):  # noqa: F811
    """cu_new falls after runs of empty sequences, in a call with more tiles
    than CTAs: reported, and the well-formed sequences' rows are those of the
    call without the fall."""
    c = Case([30000, 0, 0, 20000, 0, 0], [2, 0, 0, 2, 0, 0], ps=64, fp8=fp8, seed=41)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, want, wl = attend(fa, c, t, max_new=mn)
    assert st == 0
    check_attend(c, t, want, wl, chunk=mn > 8)
    t["cu"] = torch.tensor([0, 2, 2, 2, 4, 2, 2], dtype=torch.int32, device="cuda")
    st, out, lse = attend(fa, c, t, max_new=mn)
    assert st == INVALID and torch.equal(out, want) and torch.equal(lse, wl)
    t["ctx"][5] = 5000000                                 # no new token: its length is not looked up
    st, out, lse = attend(fa, c, t, max_new=mn)
    assert st == INVALID and torch.equal(out, want) and torch.equal(lse, wl)
    assert append(fa, c, t) == INVALID


_TIMEOUT_CHILD = """
import sys
sys.path.insert(0, %r)
import numpy as np
import torch
import full_gqa_learned_b200 as fa
from tests.paged_cases import Case
from tests.test_paged import append, attend, check_attend
c = Case([20000], [1], ps=64, seed=42)
t = c.to("cuda")
assert append(fa, c, t) == 0
ws = torch.zeros(fa.paged_workspace_bytes(1, 1, 1, c.table.shape[1], 64, window=0), dtype=torch.uint8, device="cuda")
# an earlier call's notes: fold the parts of CTAs 0 and 1 into row 0, head 0
# (status, fold, first and last CTA, second, row, head, rows, pad)
note = torch.tensor([0, 1, 0, 1, 0, 0, 0, 8, 0], dtype=torch.int32, device="cuda")
ws[256:256 + 296 * 36].view(torch.int32).view(296, 9).copy_(note.expand(296, 9))
out = torch.full((1, 4096), 7.0, dtype=torch.bfloat16, device="cuda")
lse = torch.full((32, 1), 7.0, device="cuda")
st, _, _ = attend(fa, c, t, out=out, lse=lse, workspace=ws)
assert st == 4, st                                   # FLINT_ERR_TIMEOUT
assert (out == 7).all() and (lse == 7).all(), "a stale note was folded"
st, out, lse = attend(fa, c, t, workspace=ws)        # the hook is one-shot
assert st == 0
check_attend(c, t, out, lse)
print("TIMEOUT_CHILD_OK")
"""


def test_step_wait_that_runs_out_folds_nothing():
    """A test hook makes the first launch's consumer warps wait 20 ms on a
    barrier nothing arrives on, so no CTA reaches a pair.  The workspace holds
    an earlier call's notes (within the call's bounds): the status reads
    FLINT_ERR_TIMEOUT, nothing is folded, and the next call is right.  In a
    fresh process, where the hook is read."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _TIMEOUT_CHILD % root], env=dict(os.environ, FLINT_TEST_WAIT_TIMEOUT_MS="20"),
                       cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "TIMEOUT_CHILD_OK" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 2], [1, 20]])
def test_largest_finite_sinks(fa, new, fp8):  # noqa: F811
    """Sinks whose multiple by log2(e) leaves FP32's range: they take all the
    weight (output 0, LSE the sink), as the lowest take none."""
    top = float(np.finfo(np.float32).max)
    c = Case([300, 70], new, ps=32, fp8=fp8, seed=43, sinks=[top, -top, 2.4e38, -2.4e38, 2.3e38, 0, 1, 2] * 4)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse, chunk=max(new) > 8)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_full_sequence_may_idle(fa, fp8):  # noqa: F811
    """A sequence at the most positions there can be, without new tokens, is
    no error: no position of it is past the limit."""
    c = Case([40, 7, 3], [2, 0, 1], ps=16, fp8=fp8, seed=44)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    want = {mn: attend(fa, c, t, max_new=mn)[1:] for mn in (2, 64)}
    at, cu = torch.tensor([3, 0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, 20, 20, 22], dtype=torch.int32, device="cuda")
    sc = dict(k_scales=t["k_scales"], v_scales=t["v_scales"])
    kv = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], at, cu, 22, **sc)
    t["ctx"][1] = at[1] = 1 << 24
    assert append(fa, c, t) == 0
    for mn, (o, l) in want.items():
        st, out, lse = attend(fa, c, t, max_new=mn)
        assert st == 0 and torch.equal(out, o) and torch.equal(lse, l)
    k2, v2 = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], at, cu, 22, **sc)
    assert fa.device_status(fa.paged_read.last_workspace) == 0 and torch.equal(kv[0], k2) and torch.equal(kv[1], v2)
    t["ctx"][1] = (1 << 24) + 1                           # past the limit it is one
    assert append(fa, c, t) == INVALID
    for mn in want:
        assert attend(fa, c, t, max_new=mn)[0] == INVALID


@pytest.mark.parametrize("new", [1, 2])
def test_value_scales_far_apart_on_8_bit_pages(fa, new):  # noqa: F811
    """One cached token with a weight and a value scale far above the others',
    and values in one channel only: what the others leave in the remaining
    channels is small beside it but not lost.

    The kernel multiplies P' = p 2^e in FP16, in units 2^(m - 7) with m at most
    the largest log2(p 2^e) of the row: a term is rounded to 2^-11 of itself, or
    by at most 2^-25 x 2^(m - 7), which a code of at most 448 < 2^9 multiplies.
    So the N positions add at most N 2^-23 max_j p_j 2^(e_j) to the usual
    tolerance."""
    B, ctx, g = 24, 300, 2
    c = Case([ctx] * B, [new] * B, ps=16, fp8=True, g=g, seed=45, sinks=[-np.inf] * 16)
    r = np.random.default_rng(46)
    one = r.standard_normal(128)
    c.q = torch.from_numpy(np.broadcast_to(one.astype(np.float32), (c.T, 8 * g, 128)).copy()).bfloat16()
    qt = OP.norm_rope(c.q[0, 0].double().numpy(), c.wq, 0, False)
    kv = [x.float() for x in (c.k_pages, c.v_pages)]
    ks, vs = (x.view(torch.uint8).clone() for x in (c.k_scales, c.v_scales))
    for b in range(B):
        for p in range(ctx):
            page, slot = c.table[b, p // 16], p % 16
            k, v = np.zeros((g, 128)), 1.0 + 0.5 * np.abs(r.standard_normal((g, 128)))
            if p == 37:
                k[:] = qt * (0.2 + 0.05 * b)              # logits of 2.3 to 16
                v[:], v[:, 5] = 0, 2.0 ** 7
            for x, s, y, most in ((kv[0], ks, k, 7), (kv[1], vs, v, 40)):
                code, e = OP.quantise(y, most)
                x[page, :, slot], s[page, :, slot] = torch.from_numpy(code).float(), torch.from_numpy(e + 127).to(torch.uint8)
    c.k_pages, c.v_pages = (x.to(torch.float8_e4m3fn) for x in kv)
    c.k_scales, c.v_scales = (x.view(torch.float8_e8m0fnu) for x in (ks, vs))
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    K, V = values(t["k_pages"], t["k_scales"]), values(t["v_pages"], t["v_scales"])
    E = np.exp2(t["v_scales"].cpu().view(torch.uint8).double().numpy() - 127)
    args = (c.q.double().numpy(), c.wq, c.sinks, K, V, c.table, c.ctx, c.cu)
    ref, rl, ab, spread = OP.attn(*args, window=0, use_rope=False)
    dz = (2.0 ** -11 * spread + 2e-5)[..., None]
    # max_j p_j 2^(e_j) / Z of a row
    top = np.zeros((c.T, 8 * g, 1))
    for i in range(c.T):
        b, p = i // new, ctx + i % new
        j = np.arange(p + 1)
        page = c.table[b][j // 16]
        for h in range(8 * g):
            z = K[page, h // 8, j % 16] @ OP.norm_rope(c.q[i, h].double().numpy(), c.wq, p, False) / np.sqrt(128.0)
            top[i, h] = (np.exp(z - rl[h, i]) * E[page, h // 8, j % 16]).max()
    tol = 2.0 ** -8 * np.abs(ref) + (2 * dz + 2.0 ** -15 + 2.0 ** -11) * ab + (ctx + new) * 2.0 ** -23 * top
    err = np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref)
    rel = np.delete(err / np.abs(ref), 5, -1)
    print("largest error relative to the output, other channels: %.3e" % rel.max())
    assert (err <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx,new", [(40, [1, 1]), (40, [20, 3]), (9000, [1, 2])])
def test_nan_reaches_the_lse(fa, ctx, new, fp8):  # noqa: F811
    """A NaN sink makes its head's outputs and LSE NaN, a NaN key its
    sequence's and KV head's; no other row's."""
    c = Case([ctx, 18], new, fp8=fp8, ps=16, seed=47)
    c.sinks[3] = np.nan
    t = c.to("cuda")
    t["k"][0, 1, 5] = float("nan")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    want = np.zeros((32, c.T), bool)
    want[3] = want[8:16, :new[0]] = True
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), want)
    nan = torch.isnan(out.reshape(c.T, 32, 128)).cpu().numpy()
    assert np.array_equal(nan.all(-1).T, want) and np.array_equal(nan.any(-1).T, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 2], [33, 100]])
def test_a_window_larger_than_any_position(fa, new, fp8):  # noqa: F811
    """The largest window there is sees what no window does."""
    c = Case([300, 90], new, ps=16, fp8=fp8, seed=48)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, want, wl = attend(fa, c, t)
    assert st == 0
    c.window = 2 ** 31 - 1
    st, out, lse = attend(fa, c, t)
    assert st == 0 and torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx,new", [([40, 18, 300], [1, 1, 1]), ([40, 18, 300], [2, 1, 3]), ([700, 18, 0], [40, 5, 20]), ([9000, 18], [2, 1])])
def test_nan_queries_stay_in_their_rows(fa, ctx, new, fp8):  # noqa: F811
    """NaN in a token's query, and in the rows behind the last sequence,
    reaches no other row, of the same tile or group either."""
    c = Case(ctx, new, fp8=fp8, ps=16, seed=49, extra=9)
    t = c.to("cuda")
    row = new[0] - 1
    t["q"][row, 9] = t["q"][c.rows:] = t["k"][c.rows:] = t["v"][c.rows:] = float("nan")
    assert append(fa, c, t) == 0
    check_append(c, t)
    out, lse = torch.full((c.T, 4096), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((32, c.T), 7.0, device="cuda")
    st, out, lse = attend(fa, c, t, out=out, lse=lse)
    assert st == 0 and (out[c.rows:] == 7).all() and (lse[:, c.rows:] == 7).all()
    o = out.reshape(c.T, 32, 128)
    assert torch.isnan(o[row, 9]).all() and torch.isnan(lse[9, row])
    # in the place of the NaN head: the oracle's own, so that the rest is compared
    t["q"] = torch.where(torch.isnan(t["q"]), 0, t["q"])
    st, ref, rl = attend(fa, c, t)
    assert st == 0
    c.q[row, 9], c.q[c.rows:] = 0, 0
    o[row, 9], lse[9, row] = ref.reshape(c.T, 32, 128)[row, 9], rl[9, row]
    check_attend(c, t, out, lse, chunk=max(new) > 8)


@pytest.mark.parametrize("where", ["length", "fall"])
def test_one_ill_formed_sequence_among_the_most(fa, where):  # noqa: F811
    """As many sequences as a call may have, most of them idle: the call with
    an ill-formed one walks all of them and still ends with the others' rows
    as they are without it."""
    B = 65535
    r = np.random.default_rng(50)
    ctx, new = np.zeros(B, int), np.zeros(B, int)
    live = np.sort(r.choice(B - 2, 60, replace=False))
    ctx[live], new[live] = r.integers(0, 3000, 60), r.integers(1, 3, 60)
    c = Case(ctx.tolist(), new.tolist(), g=1, ps=128, seed=51)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, want, wl = attend(fa, c, t, max_new=2)
    assert st == 0
    check_attend(c, t, want, wl)
    if where == "length":
        t["ctx"][B - 2] = -1
    else:
        t["cu"][B - 1] = 0                                # falls at an idle sequence, and rises for the next one
    st, out, lse = attend(fa, c, t, max_new=2)
    assert st == INVALID and torch.equal(out, want) and torch.equal(lse, wl)
