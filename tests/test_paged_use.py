"""The paged operators as a serving loop uses them (GPU): prompts in chunks,
then single and drafted tokens, against the full-sequence oracle; captured
graphs, streams, shared and missing pages, and what the calls refuse on the
device.

Tolerances of the loop are the forward's (output max abs 2e-2, relative L2
5e-3, LSE 2e-3: short rows carry the raw error of single FP16 products).  On
8-bit pages the oracle attends to what the pages hold, so the loop is checked
against OP.attn there, with the kernels' own tolerances (test_paged.py)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from oracle import decode as OD
from tests.paged_cases import Case, values
from tests.test_paged import append, attend, check_append, check_attend, fa, scales  # noqa: F401

pytestmark = pytest.mark.gpu
INVALID = 1


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x)).view(torch.bfloat16).cuda()


@pytest.mark.parametrize("window,rope,ps", [(0, False, 32), (65, True, 16), (513, True, 128)])
def test_serving_loop_equals_the_forward(fa, window, rope, ps):  # noqa: F811
    """Three documents fed in steps (chunks, single tokens, drafts, pauses):
    every row equals the row of the packed forward."""
    lens = [150, 61, 333]
    cu_docs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu_docs[-1])
    w = W.make_small(T, seed=31, window=window, use_rope=rope, cu_seqlens=cu_docs)
    ref, ref_l = oracle.attn_fwd_workload(w, rows=None)
    q, k, v = bf(w.q).view(T, 32, 128), bf(w.k).view(T, 4, 128), bf(w.v).view(T, 4, 128)
    wq, wk = torch.from_numpy(w.q_norm_w).cuda(), torch.from_numpy(w.k_norm_w).cuda()
    sinks = torch.from_numpy(np.asarray(w.sinks, np.float32)).cuda()
    width = (max(lens) + ps - 1) // ps + 1
    r = np.random.default_rng(5)
    table = torch.from_numpy(r.permutation(3 * width).reshape(3, width).astype(np.int32)).cuda()
    kp = torch.full((3 * width, 4, ps, 128), float("nan"), dtype=torch.float16, device="cuda")
    vp = torch.full((3 * width, 4, ps, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    got, got_l = np.zeros((T, 32, 128)), np.zeros((T, 32))
    at = [0, 0, 0]
    steps = [(100, 1, 0), (1, 33, 200), (1, 1, 1), (4, 2, 3), (1, 0, 1), (40, 20, 120)]
    while any(a < n for a, n in zip(at, lens)):
        new = [min(s, n - a) for s, a, n in zip(steps.pop(0) if steps else (8, 8, 8), at, lens)]
        rows = np.concatenate([np.arange(cu_docs[b] + at[b], cu_docs[b] + at[b] + new[b]) for b in range(3)])
        sel = torch.from_numpy(rows).cuda()
        cl = torch.tensor(at, dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        fa.paged_append(k[sel], v[sel], wk, kp, vp, table, cl, cu, use_rope=rope)
        out, lse = fa.attn_paged(q[sel], wq, sinks, kp, vp, table, cl, cu, max_new=max(new), window=window, use_rope=rope)
        assert fa.device_status(fa.attn_paged.last_workspace) == 0
        got[rows] = out.float().cpu().numpy().reshape(-1, 32, 128)
        got_l[rows] = lse.cpu().numpy().T
        at = [a + n for a, n in zip(at, new)]
    err = np.abs(got - ref)
    rel = np.linalg.norm(err) / np.linalg.norm(ref)
    print("max %.2e rel %.2e lse %.2e" % (err.max(), rel, np.abs(got_l - ref_l).max()))
    assert err.max() <= 2e-2 and rel <= 5e-3 and np.abs(got_l - ref_l).max() <= 2e-3


@pytest.mark.parametrize("fp8", [False, True])
def test_read_back_feeds_the_contiguous_decode(fa, fp8):  # noqa: F811
    """A sequence moved out of its pages into attn_decode's cache decodes to
    what the paged step gives (keys rounded to BF16 on the way: 2^-9 of each
    logit's products)."""
    c = Case([200, 90], [1, 1], fp8=fp8, ps=32, seed=12)
    t = c.to("cuda")
    cap = 208
    cu = torch.tensor([0, 200, 290], dtype=torch.int32, device="cuda")
    k, v = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], torch.zeros(2, dtype=torch.int32, device="cuda"), cu, 290, **scales(t))
    kc = torch.zeros(2, 4, cap, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    for b, (x, y) in enumerate([(0, 200), (200, 290)]):
        kc[b, :, :y - x] = k[x:y].transpose(0, 1).bfloat16()
        vc[b, :, :y - x] = v[x:y].transpose(0, 1)
    kc0, vc0 = kc.cpu().double().numpy(), vc.cpu().double().numpy()
    od, ld = fa.attn_decode(t["q"], t["k"], t["v"], t["wq"], t["wk"], t["sinks"], kc, vc, t["ctx"], window=0, use_rope=False)
    ref, rl, _ = OD.decode_step(c.q.double().numpy(), c.k.double().numpy(), c.v.double().numpy(), kc0, vc0, c.ctx, c.wq, c.wk,
                                c.sinks, window=0, use_rope=False)
    assert np.abs(od.float().cpu().numpy().reshape(2, 32, 128) - ref).max() <= 2e-2
    assert append(fa, c, t) == 0
    st, op, lp = attend(fa, c, t)
    assert st == 0
    # the new token's own row is exact in one cache and rounded (8-bit pages: to E4M3) in the other
    assert (op.float() - od.float()).abs().max() <= (0.15 if fp8 else 3e-2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 40, 1]])
def test_captured_step_replays_on_new_contents(fa, fp8, new):  # noqa: F811
    c = Case([100, 300, 17], new, fp8=fp8, ps=32, window=65, rope=True, seed=13)
    t = c.to("cuda")
    need = fa.paged_workspace_bytes(c.B, c.T, max(new), c.table.shape[1], 32, window=65, eight_bit=fp8)
    ws, ws2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, 256))
    out = torch.empty(c.T, 4096, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(32, c.T, device="cuda")

    def step():
        append(fa, c, t, workspace=ws2) if not torch.cuda.is_current_stream_capturing() else fa.paged_append(
            t["k"], t["v"], t["wk"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"], use_rope=True, workspace=ws2, **scales(t))
        fa.attn_paged(t["q"], t["wq"], t["sinks"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"], max_new=max(new),
                      window=65, use_rope=True, out=out, lse=lse, workspace=ws, **scales(t))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (g1, g2):                                    # two graphs, one workspace, one after the other
        with torch.cuda.graph(g):
            step()
    for seed, g in ((1, g1), (2, g2), (3, g1)):
        d = Case([100, 300, 17], new, fp8=fp8, ps=32, window=65, rope=True, seed=20 + seed)
        for n, x in d.to("cuda").items():
            if x is not None:
                if x.dtype is torch.float8_e8m0fnu:
                    t[n].view(torch.uint8).copy_(x.view(torch.uint8))
                elif t[n].shape == x.shape:
                    t[n].copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert fa.device_status(ws) == 0 and fa.device_status(ws2) == 0
        # table contents of d are t's now
        check_append(d, t)
        check_attend(d, t, out, lse, chunk=max(new) > 8)


def test_calls_on_two_streams(fa):  # noqa: F811
    cases = [Case([500, 20], [1, 2], seed=14), Case([300, 64], [40, 9], fp8=True, ps=64, seed=15)]
    ts = [c.to("cuda") for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for c, t, s in zip(cases, ts, streams):
            fa.paged_append(t["k"], t["v"], t["wk"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"], use_rope=False,
                            stream=s, **scales(t))
            # the stream as an object, and as a number
            outs.append(fa.attn_paged(t["q"], t["wq"], t["sinks"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"],
                                      max_new=int(c.new.max()), window=0, use_rope=False,
                                      stream=s if c is cases[0] else s.cuda_stream, **scales(t)))
    torch.cuda.synchronize()
    for c, t, (o, l) in zip(cases, ts, outs):
        check_append(c, t)
        check_attend(c, t, o, l, chunk=c.new.max() > 8)


def test_another_stream_gets_its_own_memory(fa):  # noqa: F811
    """What the call allocates must not be memory that the current stream has
    freed on the host and still writes on the device."""
    c = Case([300, 20], [1, 2], seed=28)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    _, want, wl = attend(fa, c, t)
    cu = torch.tensor([0, 300, 320], dtype=torch.int32, device="cuda")
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    wk, wv = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], at, cu, 320)
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):
        busy.fill_(1)                                     # about 6 ms of the current stream
    for like in (want, wl, wk, wv):
        for _ in range(3):
            torch.empty_like(like).fill_(7)
    got = fa.attn_paged(t["q"], t["wq"], t["sinks"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"], max_new=2,
                        window=0, use_rope=False, stream=side)
    read = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], at, cu, 320, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], wl)
    assert torch.equal(read[0], wk) and torch.equal(read[1], wv)


def test_default_stream_from_a_side_stream(fa):  # noqa: F811
    """The default stream by object and by number, while another is current."""
    c = Case([70, 9], [2, 1], seed=34)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    _, want, wl = attend(fa, c, t)
    args = [t[n] for n in ("q", "wq", "sinks", "k_pages", "v_pages", "table", "ctx", "cu")]
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream()):
        with torch.cuda.stream(torch.cuda.Stream()):
            out, lse = fa.attn_paged(*args, max_new=2, window=0, use_rope=False, stream=stream)
        assert fa.device_status(fa.attn_paged.last_workspace, stream) == 0
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("given", [False, True])
def test_empty_calls_have_a_status(fa, given):  # noqa: F811
    """No sequences, or no tokens: nothing is launched, and the status is not
    an earlier call's."""
    c = Case([20, 5], [1, 2], seed=29)
    t = c.to("cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for B, T in ((0, 0), (0, 3), (2, 0)):
        table, at, cu = t["table"][:B], torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
        kw = {}
        if given:
            kw["workspace"] = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        else:
            torch.full((256,), 255, dtype=torch.uint8, device="cuda")       # what the allocator hands out next
        fa.paged_append(t["k"][:T], t["v"][:T], t["wk"], t["k_pages"], t["v_pages"], table, at, cu, **kw)
        assert fa.device_status(fa.paged_append.last_workspace) == 0
        k, v = fa.paged_read(t["k_pages"], t["v_pages"], table, at, cu, T, **kw)
        assert fa.device_status(fa.paged_read.last_workspace) == 0 and k.shape == v.shape == (T, 4, 128)
        out, lse = fa.attn_paged(t["q"][:T], t["wq"], t["sinks"], t["k_pages"], t["v_pages"], table, at, cu, max_new=1, **kw)
        assert fa.device_status(fa.attn_paged.last_workspace) == 0 and out.shape == (T, 4096) and lse.shape == (32, T)


def test_sequences_share_prefix_pages(fa):  # noqa: F811
    """Two sequences whose first pages are the same page."""
    c = Case([64, 64], [1, 1], ps=16, seed=16)
    c.table[1, :4] = c.table[0, :4]
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse)


def test_dropped_tokens_and_freed_pages(fa):  # noqa: F811
    """A sliding layer's long prompt: pages that nothing sees later are -1.
    Append drops their tokens; attention of the last rows never reads them."""
    c = Case([0], [200], ps=16, window=33, rope=True, seed=17)
    c.table[0, :8] = -1                                   # positions 0 .. 127
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    check_append(c, t)
    # the next token's step sees positions 168 .. 200
    d = Case([200], [1], ps=16, window=33, rope=True, seed=18)
    t["cu"], t["ctx"] = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([200], dtype=torch.int32, device="cuda")
    for n in ("q", "k", "v"):
        t[n] = getattr(d, n).cuda()
    c.ctx, c.new, c.cu, c.rows, c.T = np.array([200], np.int32), np.array([1], np.int32), np.array([0, 1], np.int32), 1, 1
    c.q, c.k, c.v = d.q, d.k, d.v
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t)
    assert st == 0
    check_attend(c, t, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [2, 40]])
@pytest.mark.parametrize("page", [-1, -2, 10 ** 6, 2 ** 31 - 1])
def test_bad_pages_are_reported_and_not_read(fa, page, new, fp8):  # noqa: F811
    c = Case([100, 50], new, fp8=fp8, ps=16, seed=19)
    good = c.to("cuda")
    assert append(fa, c, good) == 0
    _, want, wl = attend(fa, c, good)
    t = dict(good, table=good["table"].clone())
    t["table"][0, 2] = page                               # a page that sequence 0's rows need
    least = fa.paged_workspace_bytes(c.B, c.T, max(new), c.table.shape[1], 16, window=0)
    for kw in ({}, {"workspace": torch.empty(least, dtype=torch.uint8, device="cuda")}):
        st, out, lse = attend(fa, c, t, **kw)
        assert st == INVALID
        n = new[0]
        assert torch.equal(out[n:], want[n:]) and torch.equal(lse[:, n:], wl[:, n:])     # sequence 1 is untouched by it
    # append: a bad page (-1 drops) is reported; read: its rows are zeros
    t["table"][0, 2], t["table"][0, 6] = good["table"][0, 2], page
    before = [t[n].clone().view(torch.uint8) for n in ("k_pages", "v_pages")]
    c2 = dict(t)
    st = append(fa, c, c2)
    assert st == (0 if page == -1 else INVALID)
    assert all(torch.equal(x, t[n].view(torch.uint8)) for x, n in zip(before, ("k_pages", "v_pages")))   # the same rows again
    cu = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    t["table"][0, 2] = page
    k, v = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], torch.zeros(2, dtype=torch.int32, device="cuda"), cu, 150, **scales(t))
    assert fa.device_status(fa.paged_read.last_workspace) == INVALID
    assert (k[32:48] == 0).all() and (v[32:48] == 0).all() and (k[48:100] != 0).any()


@pytest.mark.parametrize("what", ["cu_start", "cu_down", "cu_repeats", "cu_past", "len_neg", "len_past", "table_past", "max_new"])
@pytest.mark.parametrize("new", [[1, 1, 1], [2, 40, 1]])
def test_ill_formed_calls_are_reported(fa, what, new):  # noqa: F811
    c = Case([100, 50, 20], new, ps=16, seed=21)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    _, want, _ = attend(fa, c, t)
    mn = max(new)
    if what == "cu_start":
        t["cu"][0] = 1
    elif what == "cu_down":
        t["cu"][1] = -3
    elif what == "cu_repeats":                            # the same rows named over and over
        B = 300
        t["cu"] = torch.tensor([0, c.T] * (B // 2) + [0], dtype=torch.int32, device="cuda")
        t["ctx"] = torch.full((B,), 5, dtype=torch.int32, device="cuda")
        t["table"] = t["table"][:1].repeat(B, 1).clamp(min=0)
        mn = c.T
        st, _, _ = attend(fa, c, t, max_new=mn)
        assert st == INVALID and append(fa, c, t) == INVALID
        return
    elif what == "cu_past":
        t["cu"][3] = c.T + 1000
    elif what == "len_neg":
        t["ctx"][1] = -1
    elif what == "len_past":
        t["ctx"][1] = 1 << 24
    elif what == "table_past":
        t["ctx"][1] = c.table.shape[1] * 16
    else:
        mn = max(new) - 1
    st, out, _ = attend(fa, c, t, max_new=mn)
    assert st == INVALID
    if what in ("len_neg", "len_past", "table_past"):     # the others' rows are as they were
        keep = np.r_[0:c.cu[1], c.cu[2]:c.cu[3]]
        assert torch.equal(out[keep], want[keep])
    if what != "max_new":
        assert append(fa, c, t) == INVALID


def test_nobody_has_new_tokens(fa):  # noqa: F811
    c = Case([40, 0], [0, 0], ps=16, seed=22, extra=4)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    check_append(c, t)
    for mn in (0, 1, 2, 64):
        out = torch.full((4, 4096), 3.0, dtype=torch.bfloat16, device="cuda")
        st, _, _ = attend(fa, c, t, max_new=mn, out=out)
        assert st == 0 and (out == 3).all()


@pytest.mark.parametrize("mn", [2, 64])
@pytest.mark.parametrize("B,share", [(5000, 0.05), (40000, 0.002)])
def test_many_sequences(fa, mn, B, share):  # noqa: F811
    """More sequences than a plan's threads, most without new tokens."""
    r = np.random.default_rng(23)
    ctx = np.where(r.random(B) < 0.1, r.integers(0, 20, B), 0)
    new = np.where(r.random(B) < share, r.integers(1, 3, B), 0)
    new[17], new[B - 1] = 2, 1
    c = Case([int(x) for x in ctx], [int(x) for x in new], g=1, ps=16, seed=24)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, out, lse = attend(fa, c, t, max_new=mn)
    assert st == 0
    check_attend(c, t, out, lse, chunk=mn > 8)


def test_keys_saturate_within_fp16(fa):  # noqa: F811
    """Norm weights far beyond any model's: keys stay finite in both formats."""
    for fp8, top in ((False, 65504.0), (True, 57344.0)):
        c = Case([3], [2], fp8=fp8, seed=27, w_scale=4e4)
        t = c.to("cuda")
        assert append(fa, c, t) == 0
        cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
        k, _ = fa.paged_read(t["k_pages"], t["v_pages"], t["table"], t["ctx"], cu, 2, **scales(t))
        assert torch.isfinite(k).all() and k.abs().max().item() == top


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [20, 3]])
def test_nan_of_a_token_is_not_hidden(fa, fp8, new):  # noqa: F811
    """A NaN in a key or value stays one in the pages and in the outputs that
    see it; other sequences and heads do not."""
    c = Case([40, 18], new, fp8=fp8, ps=16, seed=33)
    t = c.to("cuda")
    t["k"][0, 1, 5] = float("nan")
    t["v"][0, 2, 7] = float("nan")
    assert append(fa, c, t) == 0
    page, slot = c.slots()
    K, V = values(t["k_pages"], t["k_scales"]), values(t["v_pages"], t["v_scales"])
    assert np.isnan(K[page[0], 1, slot[0]]).all()          # the whole row: its norm is NaN
    assert np.isnan(V[page[0], 2, slot[0], 7]) and np.isnan(V[page[0], 2, slot[0]]).sum() == 1
    assert not np.isnan(K[page[0], [0, 2, 3], slot[0]]).any()
    st, out, _ = attend(fa, c, t)
    assert st == 0
    out = out.float().reshape(c.T, 32, 128).cpu()
    n = new[0]
    assert torch.isnan(out[:n, 8:16]).all() and torch.isnan(out[:n, 16:24, 7]).all()
    assert not torch.isnan(out[:n, 16:24, :7]).any() and not torch.isnan(out[:n, :8]).any() and not torch.isnan(out[:n, 24:]).any()
    assert not torch.isnan(out[n:]).any()


def test_offsets_past_32_bits(fa):  # noqa: F811
    """A pool of over 2^31 elements: the pages in use are its last ones."""
    c = Case([300, 65], [2, 1], ps=128, seed=25)
    t = c.to("cuda")
    P = (1 << 31) // (4 * 128 * 128) + 40
    shift = P - c.P
    big = {}
    for n, dt in (("k_pages", torch.float16), ("v_pages", torch.bfloat16)):
        big[n] = torch.empty(P, 4, 128, 128, dtype=dt, device="cuda")
        big[n][shift:] = t[n]
    t2 = dict(t, k_pages=big["k_pages"], v_pages=big["v_pages"], table=torch.where(t["table"] >= 0, t["table"] + shift, t["table"]))
    assert append(fa, c, t) == 0 and append(fa, c, t2) == 0
    assert torch.equal(t2["k_pages"][shift:].view(torch.int16), t["k_pages"].view(torch.int16))
    _, o1, l1 = attend(fa, c, t)
    st, o2, l2 = attend(fa, c, t2)
    assert st == 0 and torch.equal(o1, o2) and torch.equal(l1, l2)
    st, o3, l3 = attend(fa, c, t2, max_new=9)             # the chunk kernel
    assert st == 0
    check_attend(c, t, o3, l3, chunk=True)
    del big, t2
    torch.cuda.empty_cache()


def test_argument_checks_on_cuda_tensors(fa):  # noqa: F811
    c = Case([20, 5], [1, 2], seed=26)
    t = c.to("cuda")
    kw = dict(max_new=2, window=0, use_rope=False)
    args = [t["q"], t["wq"], t["sinks"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"]]

    def bad(i, x, err, **more):
        a = list(args)
        a[i] = x
        with pytest.raises(err):
            fa.attn_paged(*a, **dict(kw, **more))
    bad(0, t["q"].float(), TypeError)
    bad(0, t["q"][:, :16], ValueError)
    bad(0, t["q"].transpose(0, 1).contiguous().transpose(0, 1), ValueError)
    bad(2, t["sinks"][:16], ValueError)
    bad(3, t["k_pages"].bfloat16(), TypeError)
    bad(4, t["v_pages"][:2], ValueError)
    bad(5, t["table"].long(), TypeError)
    bad(5, t["table"][:, ::2], ValueError)
    bad(6, t["ctx"].cpu(), ValueError)
    bad(7, t["cu"][:2], ValueError)
    with pytest.raises(TypeError):
        fa.attn_paged(*args, out=torch.empty(3, 4096, device="cuda"), **kw)
    with pytest.raises(fa.FlintError):
        fa.attn_paged(*args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **kw)
    with pytest.raises(fa.FlintError):
        fa.attn_paged(*args, **dict(kw, window=-1))
    with pytest.raises(TypeError):
        fa.paged_append(t["k"].half(), t["v"], t["wk"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"])
    with pytest.raises(ValueError):
        fa.paged_read(t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"], 3, k=torch.empty(2, 4, 128, dtype=torch.float16, device="cuda"))
    odd = torch.zeros(5, 4, 24, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(fa.FlintError):
        fa.paged_read(odd, odd.bfloat16(), t["table"], t["ctx"], t["cu"], 3)
    # a view that starts off a 16-byte boundary
    raw = torch.zeros(4 * 128 * 3 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa.FlintError):
        fa.paged_append(raw[1:1 + 4 * 128 * 3].view(3, 4, 128), t["v"], t["wk"], t["k_pages"], t["v_pages"], t["table"], t["ctx"], t["cu"])
