"""GPU parity of the paged cache (flint_paged_append, flint_paged_read,
flint_attn_paged through the package's entry points) with the FP64 oracle.

Tolerances, from the roundings that the kernels make:
* 16-bit keys: one rounding to FP16 (2^-11 relative, 2^-25 near zero) of an
  FP32 result whose error is a few FP32 last places of the row's largest
  entry (|k~| <= sqrt(128) max|w|): 2e-6 of it.  8-bit keys: one rounding to
  E4M3 (2^-4 relative, 2^-10 x scale near zero) of the same.  Values and what
  is read back: exact bits.
* Attention: the output's BF16 rounding (2^-8 relative), and relative to
  A = sum p |V| / Z: the rounding of P and twice the error of the logits.
  q~ is rounded to FP16 (2^-11 relative): a logit is off by at most dz =
  2^-11 spread + 2e-5, with spread = max_j sum_c |q~_c K_jc| / sqrt(128) (the
  constant: FP32 sums, the rotation's and the exponential's approximations).
  The step kernel keeps P to 2^-16 (two BF16 parts; 8-bit values: 2^-11 once,
  in FP16) and its sums to 2^-16: 2 dz + 2^-15 of A (8-bit values: + 2^-11).
  The chunk kernel (a sequence of the call has over 8 new tokens) rounds P to
  BF16: 2 dz + 2^-8 of A.  LSE: dz and an FP32 last place or two of itself.
"""
import numpy as np
import pytest
import torch

from oracle import paged as OP
from tests.paged_cases import Case, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import full_gqa_learned_b200 as m
    return m


def scales(t):
    return dict(k_scales=t["k_scales"], v_scales=t["v_scales"])


def append(fa, c, t, **kw):
    fa.paged_append(t["k"], t["v"], t["wk"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"],
                    use_rope=c.rope, rope_theta=c.theta, **scales(t), **kw)
    return fa.device_status(kw.get("workspace", fa.paged_append.last_workspace))


def attend(fa, c, t, **kw):
    kw.setdefault("max_new", int(c.new.max()))
    out, lse = fa.attn_paged(t["q"], t["wq"], t["sinks"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"],
                             window=c.window, use_rope=c.rope, rope_theta=c.theta, **scales(t), **kw)
    return fa.device_status(kw.get("workspace", fa.attn_paged.last_workspace)), out, lse


def bits(x):
    return x.cpu().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]).numpy()


def check_append(c, t):
    page, slot = c.slots()
    _, pos = OP.rows_of(c.ctx, c.cu)
    kept = page >= 0
    want = OP.norm_rope(c.k[:c.rows].double().numpy(), c.wk, pos[:, None].repeat(c.g, 1), c.rope, c.theta)
    got = values(t["k_pages"], t["k_scales"])[page[kept], :, slot[kept]]
    want, v = want[kept], c.v[:c.rows].double().numpy()[kept]
    fp32 = 2e-6 * np.sqrt(128) * np.abs(c.wk).max()
    if c.fp8:
        # the scale is that of the exact row, or of one that FP32 puts across its border
        e = t["k_scales"].cpu().view(torch.uint8).numpy()[page[kept], :, slot[kept]].astype(np.int64) - 127
        lo, hi = OP.scale_exponent(want * (1 - 1e-6)), OP.scale_exponent(want * (1 + 1e-6))
        assert ((e >= lo) & (e <= hi)).all()
        tol = np.abs(want) * 2.0 ** -4 + 2.0 ** -10 * np.exp2(e)[..., None] + fp32
        vc, ve = OP.quantise(v)
        assert np.array_equal(t["v_pages"].cpu().double().numpy()[page[kept], :, slot[kept]], vc)
        assert np.array_equal(t["v_scales"].cpu().view(torch.uint8).numpy()[page[kept], :, slot[kept]], ve + 127)
    else:
        tol = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + fp32
        assert np.array_equal(values(t["v_pages"], None)[page[kept], :, slot[kept]], v)
    assert (np.abs(got - want) <= tol).all()
    # every other slot keeps its bits
    touched = np.zeros((c.P, c.ps), bool)
    touched[page[kept], slot[kept]] = True
    for n in ("k_pages", "v_pages", "k_scales", "v_scales"):
        if t[n] is not None:
            a, b = bits(t[n]), bits(getattr(c, n).contiguous())
            same = (a == b).reshape(c.P, c.g, c.ps, -1).all(-1)
            assert same[~np.broadcast_to(touched[:, None], same.shape)].all(), n


def check_attend(c, t, out, lse, chunk=False):
    K, V = values(t["k_pages"], t["k_scales"]), values(t["v_pages"], t["v_scales"])
    ref, rl, ab, spread = OP.attn(c.q.double().numpy(), c.wq, c.sinks, K, V, c.table, c.ctx, c.cu, window=c.window,
                                  use_rope=c.rope, theta=c.theta)
    n = c.rows
    got = out.float().cpu().numpy().reshape(c.T, 8 * c.g, 128)[:n].astype(np.float64)
    ref, ab, spread, rl = ref[:n], ab[:n], spread[:n], rl[:, :n]
    dz = 2.0 ** -11 * spread + 2e-5
    p_off = 2.0 ** -8 if chunk else 2.0 ** -15 + (2.0 ** -11 if c.fp8 else 0.0)
    tol = 2.0 ** -8 * np.abs(ref) + (2 * dz[..., None] + p_off) * ab
    err = np.abs(got - ref)
    print("rel %.2e" % (np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300)))
    assert (err <= tol).all()
    if lse is not None:
        gl = lse.cpu().numpy()[:, :n].astype(np.float64)
        fin = np.isfinite(rl)
        assert np.array_equal(gl[~fin], rl[~fin])
        lt = dz.T + 2.0 ** -22 * np.abs(np.where(fin, rl, 0))
        assert (np.abs(gl[fin] - rl[fin]) <= lt[fin]).all()


# ragged lengths: no context, one position, ends on and off page and tile
# borders, sequences without new rows
LENS = {
    "one": ([300], [1]),
    "first": ([0, 0, 0], [1, 1, 1]),
    "ones": ([0, 1, 15, 16, 17, 63, 64, 127, 128, 255, 513, 700], [1] * 12),
    "some_none": ([5, 40, 0, 129, 64], [1, 0, 0, 1, 0]),
    "pairs": ([0, 14, 31, 100, 250, 511], [2, 2, 2, 1, 2, 2]),
    "few": ([0, 3, 60, 127, 300], [3, 5, 1, 8, 7]),
    "rows": ([0, 100, 37, 5, 511], [40, 17, 1, 33, 9]),
}
FORMS = [(16, False, 4), (32, True, 4), (64, False, 2), (128, True, 1), (64, True, 2), (128, False, 1)]


@pytest.mark.parametrize("ps,fp8,g", FORMS)
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("window,rope", [(0, False), (513, True), (33, True), (1, False)])
def test_append_and_attend(fa, lens, ps, fp8, g, window, rope):
    ctx, new = LENS[lens]
    c = Case(ctx, new, g=g, ps=ps, fp8=fp8, window=window, rope=rope, seed=len(lens) + ps + window, extra=3)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    check_append(c, t)
    out = torch.full((c.T, 8 * g * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8 * g, c.T), 7.0, device="cuda")
    st, out, lse = attend(fa, c, t, out=out, lse=lse)
    assert st == 0
    check_attend(c, t, out, lse, chunk=c.new.max() > 8)
    assert (out[c.rows:] == 7).all() and (lse[:, c.rows:] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ps,g", [(16, 4), (128, 2), (32, 1)])
def test_read_gives_back_the_bits(fa, ps, g, fp8):
    c = Case([300, 17, 0, 128], [0, 0, 0, 0], g=g, ps=ps, fp8=fp8, seed=3)
    t = c.to("cuda")
    start, count = np.array([13, 0, 0, 16], np.int32), np.array([287, 17, 0, 100], np.int32)
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    T = int(cu[-1]) + 5
    k = torch.full((T, g, 128), 9.0, dtype=torch.float16, device="cuda")
    v = torch.full((T, g, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    fa.paged_read(t["k_pages"], t["v_pages"], t["table"], torch.from_numpy(start).cuda(), torch.from_numpy(cu).cuda(), T,
                  k=k, v=v, **scales(t))
    assert fa.device_status(fa.paged_read.last_workspace) == 0
    b, pos = OP.rows_of(start, cu)
    page, slot = c.table[b, pos // ps], pos % ps
    K, V = values(t["k_pages"], t["k_scales"]), values(t["v_pages"], t["v_scales"])
    assert np.array_equal(k[:cu[-1]].cpu().double().numpy(), K[page, :, slot])
    assert np.array_equal(v[:cu[-1]].cpu().double().numpy(), V[page, :, slot])
    assert (k[cu[-1]:] == 9).all() and (v[cu[-1]:] == 9).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_axis_is_split_and_repeatable(fa, fp8):
    c = Case([20000, 3, 9001], [1, 1, 1], ps=64, fp8=fp8, seed=5)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse)
    for _ in range(3):
        _, o2, l2 = attend(fa, c, t)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("ps,fp8", [(16, False), (128, False), (64, True)])
@pytest.mark.parametrize("ctx,new,window", [([2500], [70], 0), ([900, 0, 130, 4000, 64], [33, 129, 16, 1, 100], 0),
                                            ([700, 5000, 0], [300, 40, 17], 257)])
def test_chunks(fa, ps, fp8, ctx, new, window):
    c = Case(ctx, new, ps=ps, fp8=fp8, window=window, rope=window > 0, seed=8, extra=2)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse, chunk=True)
    # again, and in the least workspace (8-bit pages: converted on chip): the same bits
    least = fa.paged_workspace_bytes(c.B, c.T, int(c.new.max()), c.table.shape[1], ps, window=window)
    for kw in ({}, {"workspace": torch.empty(least, dtype=torch.uint8, device="cuda")}):
        st, o2, l2 = attend(fa, c, t, **kw)
        assert st == 0
        assert torch.equal(out[:c.rows], o2[:c.rows]) and torch.equal(lse[:, :c.rows], l2[:, :c.rows])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", [0, 60, 200])
def test_chunks_of_unlike_pairs(fa, fp8, where):
    """One long sequence among 200 whose pairs have a chunk or two: where a
    CTA's share begins goes by a pair's cost, not by its chunks alone."""
    r = np.random.default_rng(31)
    ctx, new = r.integers(0, 140, 200).tolist(), r.integers(0, 4, 200).tolist()
    ctx.insert(where, 9001)
    new.insert(where, 40)
    c = Case(ctx, new, ps=32, fp8=fp8, seed=32)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse, chunk=True)
    if fp8:                                               # converted on chip
        least = fa.paged_workspace_bytes(c.B, c.T, 40, c.table.shape[1], 32, window=0)
        st, out, lse = attend(fa, c, t, workspace=torch.empty(least, dtype=torch.uint8, device="cuda"))
        assert st == 0
        check_attend(c, t, out, lse, chunk=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_positions_and_extreme_sinks(fa, fp8):
    sinks = np.array([np.inf, -np.inf, 80.0, -80.0] * 8, np.float32)
    c = Case([262100, 1 << 20, 12], [1, 2, 1], ps=32, fp8=fp8, window=129, rope=True, seed=6, sinks=sinks)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w_scale,v_scale", [(4.0, 1.0), (1e-3, 1.0), (1.0, 1e4), (1.0, 1e-4)])
def test_large_and_small_rows(fa, fp8, w_scale, v_scale):
    c = Case([200, 70, 513], [1, 2, 2], ps=16, fp8=fp8, seed=7, w_scale=w_scale, v_scale=v_scale)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    check_append(c, t)
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse)
